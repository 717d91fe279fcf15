// paged_decode.cu -- relpos_paged_decode: argument checks, the choice of the
// kernel variant, scratch and launches (the kernels are in paged_decode.cuh).

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include "../../include/relpos_attn.h"
#include "paged_decode.cuh"
#include "relpos_internal.h"
#include "serving_internal.h"

namespace relpos {
namespace {

PagedDecodeVariant variant_of(int d, int dtype, int rows8) {
  if (dtype == RELPOS_E4M3) return d == 64 ? paged_decode_e4m3_64(rows8) : paged_decode_e4m3_128(rows8);
  return d == 64 ? paged_decode_bf16_64(rows8) : paged_decode_bf16_128(rows8);
}

constexpr int kDevices = 64;
std::mutex g_mu;  // guards what is kept between calls below

// What is set up once may come up first in a call under stream capture, where
// calls that touch no stream are refused too unless the thread says that they are
// meant.
struct OutsideCapture {
  cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
  OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
  ~OutsideCapture() { cudaThreadExchangeStreamCaptureMode(&mode); }
};

// Blocks of a variant's decode kernel that an SM of the current device holds,
// asked once for each device (with the shared memory allowed for the kernel's
// launches); 0 on failure.
int resident_blocks(int d, int dtype, int rows8, const PagedDecodeVariant& v) {
  static int known[kDevices][8];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
  int& n = known[dev][(d == 128) * 4 + (dtype == RELPOS_E4M3) * 2 + rows8 - 1];
  std::lock_guard<std::mutex> lk(g_mu);
  if (n == 0) {
    OutsideCapture mode;
    if (cudaFuncSetAttribute(v.decode, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess ||
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, v.decode, kPdThreads, v.smem) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
  }
  return n;
}

// The pool that scratch comes from, one of the library's own for each device:
// the default pool gives its memory back whenever the host waits for the GPU,
// and a call after that took 200 us for its scratch (every step of a decode loop
// that looks at its token). This one keeps up to 64 MB.
cudaMemPool_t scratch_pool() {
  static cudaMemPool_t pools[kDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return nullptr;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!pools[dev]) {
    OutsideCapture mode;
    cudaMemPoolProps props = {};
    props.allocType = cudaMemAllocationTypePinned;
    props.location.type = cudaMemLocationTypeDevice;
    props.location.id = dev;
    cudaMemPool_t pool = nullptr;
    cuuint64_t keep = 64ull << 20;
    if (cudaMemPoolCreate(&pool, &props) != cudaSuccess ||
        cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &keep) != cudaSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    pools[dev] = pool;
  }
  return pools[dev];
}

// The T5 thresholds (t5_setup, which walks the distances up to max_distance in
// logarithms) and the buckets of the first distances, for parameters that the
// last calls did not have; they depend on nothing else.
int set_t5(int num_buckets, int max_distance, int longest, PagedDecodeParams* p) {
  struct Known {
    int num_buckets, max_distance, longest, R;
    T5Index ix;
    uint8_t bucket[kPdBuckets];
  };
  static Known known[8];
  static int next = 0;
  std::lock_guard<std::mutex> lk(g_mu);
  const Known* k = nullptr;
  for (const Known& e : known)
    if (e.num_buckets == num_buckets && e.max_distance == max_distance && e.longest == longest) k = &e;
  if (!k) {
    Known e = {num_buckets, max_distance, longest};
    const int rc = t5_setup(num_buckets, max_distance, 1, longest, &e.ix, &e.R);
    if (rc != RELPOS_OK) return rc;
    for (int i = 0; i < kPdBuckets; ++i) e.bucket[i] = static_cast<uint8_t>(t5_bucket_dev(-i, e.ix));
    known[next] = e;
    k = &known[next];
    next = (next + 1) % 8;
  }
  p->t5 = k->ix;
  p->t5_R = k->R;
  std::memcpy(p->bucket, k->bucket, sizeof(k->bucket));
  return RELPOS_OK;
}

// How a call is cut up: the variant, rows of a unit and units that a key/value
// head takes, blocks, and whether each unit has its block and there is no second
// launch.
struct Split {
  PagedDecodeVariant v;
  int rows, rt, blocks, direct;
};

int split_of(const RelposPagedCache* cache, int B, int Hq, int Lq, int max_pages, Split* out) {
  const int G = Hq / cache->H;
  if (G > 65535) return RELPOS_ERR_UNSUPPORTED;
  const long long capacity = static_cast<long long>(max_pages) * cache->page;
  if (capacity > (1 << 28)) return RELPOS_ERR_UNSUPPORTED;
  out->v = variant_of(cache->d, cache->dtype, 1);
  out->rt = (G * Lq + 7) / 8;
  long long units = static_cast<long long>(B) * cache->H * out->rt;
  const long long tiles = (capacity + out->v.tile - 1) / out->v.tile;  // of a unit, with every page in use
  if (units > (1 << 30) || units * (tiles + kPdUnitCost) > (1 << 30)) return RELPOS_ERR_UNSUPPORTED;
  if (static_cast<long long>(cache->num_pages) * cache->H > 0x7fffffffll) return RELPOS_ERR_UNSUPPORTED;
  const int sms = device_sms();
  if (sms <= 0) return RELPOS_ERR_CUDA;
  // Rows of a unit: 8, or 16 where a key/value head has more than 8 and a warp
  // more than 16 tiles. 16 rows read each tile once instead of twice but keep a
  // third fewer warps on an SM and take longer a tile. us with 8 / 16 rows for 16
  // sequences x 4 heads x 16 rows at 2048, 4096, 8192 and 16384 tokens:
  //   bf16  d =  64   16 / 20   25 / 30   51 / 47   94 / 75   16 rows from 9728 on
  //   bf16  d = 128   27 / 25   54 / 36   97 / 58  181 / 97   from 3648
  //   e4m3  d =  64   15 / 17   19 / 21   29 / 30   48 / 43   from 9728
  //   e4m3  d = 128   20 / 21   28 / 28   53 / 40   97 / 62   from 7296
  // 24 and 32 rows lose to both.
  int occ = resident_blocks(cache->d, cache->dtype, 1, out->v);
  if (occ < 1) return RELPOS_ERR_CUDA;
  const bool wide = out->rt > 1 && units * tiles > 16ll * kPdWarps * occ * sms;
  if (wide) {
    out->v = variant_of(cache->d, cache->dtype, 2);
    out->rt = (out->rt + 1) / 2;
    units = static_cast<long long>(B) * cache->H * out->rt;
    occ = resident_blocks(cache->d, cache->dtype, 2, out->v);
    if (occ < 1) return RELPOS_ERR_CUDA;
  }
  out->rows = wide ? 16 : 8;
  // Sequences of up to 16 tiles at most (four of a warp) have a block for each
  // unit and no second launch: 5.0 against 7.3 us for 113 tokens of 16 heads.
  out->direct = tiles <= 4 * kPdMinTiles;
  out->blocks = static_cast<int>(out->direct ? units
                                             : std::min<long long>(static_cast<long long>(occ) * sms,
                                                                   (units * tiles + kPdMinTiles - 1) / kPdMinTiles));
  return RELPOS_OK;
}

}  // namespace
}  // namespace relpos

using namespace relpos;

extern "C" int relpos_selftest_paged_decode_split(const RelposPagedCache* cache, int B, int Hq, int Lq, int max_pages,
                                                  int* rows, int* launches) {
  const int rc = check_paged_cache(cache);
  if (rc != RELPOS_OK) return rc;
  if (!rows || !launches || cache->H < 1 || cache->num_pages < 1 || B < 1 || Hq < 1 || Hq % cache->H || Lq < 1 ||
      max_pages < 1)
    return RELPOS_ERR_INVALID_ARG;
  if (Lq > 8) return RELPOS_ERR_UNSUPPORTED;
  Split split;
  const int err = split_of(cache, B, Hq, Lq, max_pages, &split);
  if (err != RELPOS_OK) return err;
  *rows = split.rows;
  *launches = split.direct ? 1 : 2;
  return RELPOS_OK;
}

extern "C" int relpos_paged_decode(const RelposPagedCache* cache, const void* Q, const RelposRowStrides* qs, int B,
                                   int Hq, int Lq, const int* block_table, long long table_stride, int max_pages,
                                   const int* lens, int bias_mode, const void* bias, int num_buckets,
                                   int max_distance, float scale, void* out, const RelposRowStrides* os,
                                   void* stream) {
  int rc = check_paged_cache(cache);
  if (rc != RELPOS_OK) return rc;
  if (bias_mode != RELPOS_NO_BIAS && bias_mode != RELPOS_T5 && bias_mode != RELPOS_ALIBI)
    return RELPOS_ERR_INVALID_ARG;
  if (bias_mode == RELPOS_T5) {
    rc = check_rel_params(RELPOS_T5, num_buckets, max_distance, 1);
    if (rc != RELPOS_OK) return rc;
  }
  if (!qs || !os || B < 0 || Hq < 0 || Lq < 0 || max_pages < 0 || !std::isfinite(scale)) return RELPOS_ERR_INVALID_ARG;
  if (Lq > 8) return RELPOS_ERR_UNSUPPORTED;
  if (B == 0 || Hq == 0 || Lq == 0) return RELPOS_OK;
  if (cache->H == 0 || Hq % cache->H) return RELPOS_ERR_INVALID_ARG;
  const uintptr_t ints = reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(lens) |
                         reinterpret_cast<uintptr_t>(bias);
  if (!Q || !out || !lens || !block_table || (ints & 3u)) return RELPOS_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(Q) | reinterpret_cast<uintptr_t>(out)) & 1u) return RELPOS_ERR_INVALID_ARG;
  if (rows_overlap(B, os->batch, cache->d) || rows_overlap(Hq, os->head, cache->d) || rows_overlap(Lq, os->row, cache->d))
    return RELPOS_ERR_INVALID_ARG;
  if (bias_mode != RELPOS_NO_BIAS && !bias) return RELPOS_ERR_INVALID_ARG;
  if (max_pages == 0 || cache->num_pages == 0) return RELPOS_ERR_INVALID_ARG;
  if (B > 1 && table_stride < max_pages) return RELPOS_ERR_INVALID_ARG;
  Split split;
  rc = split_of(cache, B, Hq, Lq, max_pages, &split);
  if (rc != RELPOS_OK) return rc;
  const PagedDecodeVariant& v = split.v;
  const long long capacity = static_cast<long long>(max_pages) * cache->page;

  PagedDecodeParams p;
  std::memset(&p, 0, sizeof(p));
  p.k = static_cast<const uint8_t*>(cache->k);
  p.v = static_cast<const uint8_t*>(cache->v);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.num_pages = cache->num_pages;
  p.Hkv = cache->H;
  p.log_page = cache->page == 32 ? 5 : cache->page == 64 ? 6 : 7;
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.q_batch = qs->batch, p.q_head = qs->head, p.q_row = qs->row;
  p.q_vec = aligned16(Q) && (qs->batch | qs->head | qs->row) % 8 == 0;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.o_vec = aligned16(out) && (os->batch | os->head | os->row) % 8 == 0;
  p.o_batch = os->batch, p.o_head = os->head, p.o_row = os->row;
  p.table = block_table;
  p.table_stride = table_stride;
  p.max_len = static_cast<int>(capacity);
  p.lens = lens;
  p.B = B, p.Hq = Hq, p.Lq = Lq, p.G = Hq / cache->H, p.rows = split.rows, p.rt = split.rt;
  p.bias = static_cast<const float*>(bias);
  p.mode = bias_mode;
  if (bias_mode == RELPOS_T5) {
    rc = set_t5(num_buckets, max_distance, static_cast<int>(capacity), &p);
    if (rc != RELPOS_OK) return rc;
  }
  p.scale_log2 = (scale != 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(cache->d))) * kLog2e;
  p.status = device_status();
  if (!p.status) return RELPOS_ERR_CUDA;
  p.direct = split.direct;
  p.blocks = split.blocks;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  float* scratch = nullptr;
  if (!p.direct) {
    const size_t slots = static_cast<size_t>(p.blocks) * 2 * p.rows;  // a multiple of 16
    const size_t bytes = slots * (cache->d + 2) * sizeof(float) + p.blocks * 2 * sizeof(int4);
    cudaMemPool_t pool = scratch_pool();
    if (!pool || cudaMallocFromPoolAsync(reinterpret_cast<void**>(&scratch), bytes, pool, s) != cudaSuccess) {
      cudaGetLastError();
      return RELPOS_ERR_CUDA;
    }
    p.part_o = scratch;
    p.part_ml = scratch + slots * cache->d;
    p.ends = reinterpret_cast<int4*>(p.part_ml + slots * 2);
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.blocks);
  cfg.blockDim = dim3(kPdThreads);
  cfg.dynamicSmemBytes = v.smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  bool ok = cudaLaunchKernelEx(&cfg, v.decode, p) == cudaSuccess;
  if (!p.direct) {
    cfg.dynamicSmemBytes = 0;
    ok = ok && cudaLaunchKernelEx(&cfg, v.combine, p) == cudaSuccess;
    ok = cudaFreeAsync(scratch, s) == cudaSuccess && ok;
  }
  if (!ok) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  return RELPOS_OK;
}
