// paged_append.cu -- new tokens' keys and values into the pages of a paged
// cache, keys turned by their rotary positions on the way ("Relative Position
// Embeddings, in depth", sections "ALiBi and RoPE: the two endpoints" and
// "Kernels and the KV cache"). 16-bit caches hold bf16; 8-bit caches hold
// e4m3 codes with one power-of-two scale for each page and head.
//
// Why powers of two: e4m3 carries its own exponent, so a scale only has to
// place the page's largest value below 448; a power of two costs no mantissa
// bit and makes dividing by the scale, moving codes to a larger scale and the
// value (code * scale) exact, up to the codes that fall below e4m3's smallest
// normal. A page's scale only grows while tokens are appended to it. Keys take
// sqrt(2) * amplitude times their largest magnitude: no angle turns a pair
// beyond that, so the scale is known before the rotation and does not depend
// on the position.

#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/relpos_attn.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "relpos_internal.h"
#include "rotary.cuh"

namespace relpos {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppSlots = 4;  // 16-element units of a key and a value that a thread holds

struct AppendParams {
  RelposRotaryPlan plan;  // rot_dim 0: no rotation
  RelposPagedCache cache;
  const __nv_bfloat16* K;
  const __nv_bfloat16* V;
  long long k_batch, k_head, k_row, v_batch, v_head, v_row;
  int vec;                // every row of K and V is 16-byte aligned
  const int* cu;          // [B + 1] first new row of each sequence, or null: n rows each
  int n, rows, B;
  const int* table;
  long long table_stride;
  int max_pages;
  const int* lens;
  int log_page, log_units;  // page and d / 16, powers of two
  int group;              // heads of a block
  double reach;           // largest rotated magnitude over the largest one
  int* status;
};

// The smallest power of two s with amax * reach <= 448 s, clamped to
// 2^-120 .. 2^120: the exponent comes from the bits of the quotient.
RP_DEVI float scale_for(float amax, double reach) {
  if (!(amax > 0.f)) return __int_as_float((127 - 120) << 23);
  const unsigned long long r = __double_as_longlong(static_cast<double>(amax) * reach / 448.0);
  int e = static_cast<int>((r >> 52) & 0x7ff) - 1023;  // floor(log2)
  if (r & 0xfffffffffffffull) ++e;
  e = min(120, max(-120, e));
  return __int_as_float((e + 127) << 23);
}

RP_DEVI uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// A value in 64 bits to its e4m3 code: rounded to fp32 with the last bit made
// odd where that dropped anything, so that the second rounding sees on which
// side of a border the value lies.
RP_DEVI uint32_t e4m3_of(double v) {
  float f = __double2float_rz(v);
  if (static_cast<double>(f) != v) f = __int_as_float(__float_as_int(f) | 1);
  return e4m3x2(f, 0.f) & 0xffu;
}

// The pair's codes from the rotation in 64 bits (y1's in the low byte). Taken
// where the fp32 rotation cannot tell on which side of a border of the e4m3
// grid its result lies, about once in 10^5 values.
__device__ __noinline__ uint32_t rotated_codes_exact(float x1, float x2, unsigned long long turns, int pos,
                                                     double amplitude, float inv) {
  const long long t =
      static_cast<long long>(turns * static_cast<unsigned long long>(static_cast<long long>(pos)));
  double s, c;
  sincospi(static_cast<double>(t) * 1.0842021724855044e-19, &s, &c);  // t / 2^63 half turns
  const double a = amplitude * inv;
  const double u = x1, v = x2;
  return e4m3_of((u * c - v * s) * a) | (e4m3_of((u * s + v * c) * a) << 8);
}

// Blocks of 256 threads take one page that gets new tokens and `group` heads;
// a thread holds up to four 16-element units of the keys and of the values in
// registers, all loads in flight at once, so both the page's largest value
// and its codes come from one read.
template <bool FP8>
__global__ void __launch_bounds__(kAppThreads) relpos_paged_append_kernel(const __grid_constant__ AppendParams p) {
  __shared__ int amax_s[8][2];
  __shared__ float inv_s[8][2];
  __shared__ float move_s[8][2];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31;

  // The sequence of this block: sequence b has the blocks from
  // floor(first row / page) + 2 b on, at least as many as the pages its rows
  // can touch (n rows touch at most floor(n / page) + 2).
  auto first_row = [&](int b) { return p.cu ? __ldg(p.cu + b) : b * p.n; };
  const int blk = blockIdx.x;
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {  // 32 probes at a time
    const int step = (hi - lo + 31) >> 5;
    const int i = lo + lane * step;
    const bool at_or_before = i < hi && (first_row(i) >> p.log_page) + 2 * i <= blk;
    const int k = __popc(__ballot_sync(0xffffffffu, at_or_before));
    if (k == 0) return;  // first rows that do not ascend: checked below for the others
    lo += (k - 1) * step;
    hi = min(hi, lo + step);
  }
  const int b = lo;
  const int row0 = first_row(b), row1 = first_row(b + 1);
  const int len = __ldg(p.lens + b);
  if (len <= 0 || row1 == row0) return;  // an unused entry of the batch
  const int n = row1 - row0;
  if (row0 < 0 || n < 0 || row1 > p.rows || len < n || len > (p.max_pages << p.log_page)) {
    if (tid == 0) atomicCAS(p.status, 0, RELPOS_ERR_PAGE);
    return;
  }
  const int start = len - n;  // position of the first new token
  const int k = blk - ((row0 >> p.log_page) + 2 * b);
  const int pg = (start >> p.log_page) + k;
  if (k < 0 || pg > (len - 1) >> p.log_page) return;
  const int page_id = __ldg(p.table + b * p.table_stride + pg);
  if (page_id < 0 || page_id >= p.cache.num_pages) {
    if (tid == 0) atomicCAS(p.status, 0, RELPOS_ERR_PAGE);
    return;
  }
  const int page = 1 << p.log_page;
  const int t_lo = max(start - pg * page, 0), t_hi = min(len - pg * page, page);  // new slots of the page
  const int h0 = blockIdx.y * p.group;
  const int nheads = min(p.group, p.cache.H - h0);
  const int d = p.cache.d;
  const int log_items = p.log_page + p.log_units;  // units of one head's page
  const int rot_units = p.plan.rot_dim >> 4;
  const bool interleaved = p.plan.layout == RELPOS_ROTARY_INTERLEAVED;

  // dims of a unit: 8 pairs of the rotation, or 16 neighbouring values
  auto dims = [&](int unit, int& d1, int& d2) {
    if (unit < rot_units && !interleaved) {
      d1 = unit * 8;
      d2 = (p.plan.rot_dim >> 1) + d1;
    } else {
      d1 = unit * 16;
      d2 = d1 + 8;
    }
  };

  uint4 kr[kAppSlots][2], vr[kAppSlots][2];
  bool live[kAppSlots];
#pragma unroll
  for (int i = 0; i < kAppSlots; ++i) {
    const int item = i * kAppThreads + tid;
    const int hs = item >> log_items;
    const int slot = (item >> p.log_units) & (page - 1);
    const int unit = item & ((1 << p.log_units) - 1);
    live[i] = hs < nheads && slot >= t_lo && slot < t_hi;
    kr[i][0] = kr[i][1] = vr[i][0] = vr[i][1] = make_uint4(0, 0, 0, 0);
    if (live[i]) {
      const long long r = pg * page + slot - start;  // new row of the sequence
      const long long kb = p.cu ? (row0 + r) * p.k_row : b * p.k_batch + r * p.k_row;
      const long long vb = p.cu ? (row0 + r) * p.v_row : b * p.v_batch + r * p.v_row;
      const __nv_bfloat16* kp = p.K + kb + (h0 + hs) * p.k_head;
      const __nv_bfloat16* vp = p.V + vb + (h0 + hs) * p.v_head;
      int d1, d2;
      dims(unit, d1, d2);
      if (p.vec) {
        kr[i][0] = *reinterpret_cast<const uint4*>(kp + d1);
        kr[i][1] = *reinterpret_cast<const uint4*>(kp + d2);
        vr[i][0] = *reinterpret_cast<const uint4*>(vp + d1);
        vr[i][1] = *reinterpret_cast<const uint4*>(vp + d2);
      } else {
        kr[i][0] = load8_unaligned(kp + d1);
        kr[i][1] = load8_unaligned(kp + d2);
        vr[i][0] = load8_unaligned(vp + d1);
        vr[i][1] = load8_unaligned(vp + d2);
      }
    }
  }

  const size_t page_rows = static_cast<size_t>(page_id) * p.cache.H;
  if constexpr (FP8) {
    float* const scales[2] = {p.cache.k_scale, p.cache.v_scale};
    // thread 2 h + w looks after head h's scale of the keys (w = 0) or values
    const bool keeper = tid < 2 * nheads;
    float had = 0.f;
    if (keeper) {
      amax_s[tid >> 1][tid & 1] = 0;
      if (t_lo > 0) had = scales[tid & 1][page_rows + h0 + (tid >> 1)];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kAppSlots; ++i) {
      const int hs = (i * kAppThreads + tid) >> log_items;  // the same for the whole warp
      if (hs >= nheads) break;
      // magnitudes of bf16 order like their bits; infinities and NaN: an
      // infinity takes the largest scale, NaN has no magnitude
      uint32_t mk = max(absmax_bf16(kr[i][0]), absmax_bf16(kr[i][1]));
      uint32_t mv = max(absmax_bf16(vr[i][0]), absmax_bf16(vr[i][1]));
      mk = __reduce_max_sync(0xffffffffu, mk);
      mv = __reduce_max_sync(0xffffffffu, mv);
      if (lane == 0) {
        if (mk) atomicMax(&amax_s[hs][0], static_cast<int>(mk << 16));
        if (mv) atomicMax(&amax_s[hs][1], static_cast<int>(mv << 16));
      }
    }
    __syncthreads();
    if (keeper) {
      const float want =
          scale_for(__int_as_float(amax_s[tid >> 1][tid & 1]), (tid & 1) ? 1.0 : p.reach);
      const float now = t_lo > 0 ? fmaxf(want, had) : want;
      move_s[tid >> 1][tid & 1] = t_lo > 0 ? had / now : 1.f;
      inv_s[tid >> 1][tid & 1] = 1.f / now;
      if (t_lo == 0 || now != had) scales[tid & 1][page_rows + h0 + (tid >> 1)] = now;
    }
    __syncthreads();
  }

  const float amplitude = static_cast<float>(p.plan.amplitude);
  float s[8], c[8];
#pragma unroll
  for (int i = 0; i < kAppSlots; ++i) {
    const int item = i * kAppThreads + tid;
    const int hs = item >> log_items;
    if (hs >= nheads) break;
    const int slot = (item >> p.log_units) & (page - 1);
    const int unit = item & ((1 << p.log_units) - 1);
    int d1, d2;
    dims(unit, d1, d2);
    const size_t at = ((page_rows + h0 + hs) * page + slot) * d;
    if constexpr (FP8) {
      if (slot < t_lo) {  // codes that were there, to the page's new scale
        move_codes(static_cast<uint8_t*>(p.cache.k) + at, d1, d2, move_s[hs][0]);
        move_codes(static_cast<uint8_t*>(p.cache.v) + at, d1, d2, move_s[hs][1]);
      }
    }
    if (!live[i]) continue;
    const bool turns = unit < rot_units;
    const int pos = pg * page + slot;
    // threads keep their unit and slot from head to head when a head's page
    // has at most 256 units
    if (turns && (i == 0 || log_items > 8)) {
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        rotary_sincos(p.plan.turns[8 * unit + m], pos, s[m], c[m]);
        s[m] *= amplitude;
        c[m] *= amplitude;
      }
    }
    float x1[8], x2[8];
    unpack8(kr[i][0], x1);
    unpack8(kr[i][1], x2);
    if constexpr (!FP8) {
      __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(p.cache.k) + at;
      __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(p.cache.v) + at;
      if (turns) {
        rotate_unit<8>(x1, x2, s, c, interleaved);
        store_vec<8>(ko + d1, x1);
        store_vec<8>(ko + d2, x2);
      } else {
        *reinterpret_cast<uint4*>(ko + d1) = kr[i][0];
        *reinterpret_cast<uint4*>(ko + d2) = kr[i][1];
      }
      *reinterpret_cast<uint4*>(vo + d1) = vr[i][0];
      *reinterpret_cast<uint4*>(vo + d2) = vr[i][1];
    } else {
      uint8_t* ko = static_cast<uint8_t*>(p.cache.k) + at;
      uint8_t* vo = static_cast<uint8_t*>(p.cache.v) + at;
      const float ik = inv_s[hs][0], iv = inv_s[hs][1];
      uint2 o1, o2;
      if (turns) {
        uint32_t code[8];  // of pair m: first member's code, second's in the next byte
#pragma unroll
        for (int m = 0; m < 8; ++m) {
          const float a = interleaved ? (m < 4 ? x1[2 * (m & 3)] : x2[2 * (m & 3)]) : x1[m];
          const float q = interleaved ? (m < 4 ? x1[2 * (m & 3) + 1] : x2[2 * (m & 3) + 1]) : x2[m];
          float y1, y2;
          rotate_pair(a, q, s[m], c[m], y1, y2);
          // the fp32 rotation is off by less than 2^-21 (|a| + |q|) amplitude:
          // where both ends of that round to one code it is the right one
          const float off = (fabsf(a) + fabsf(q)) * (4.76837158e-07f * amplitude);
          code[m] = e4m3x2((y1 - off) * ik, (y2 - off) * ik);
          if (code[m] != e4m3x2((y1 + off) * ik, (y2 + off) * ik))
            code[m] = rotated_codes_exact(a, q, p.plan.turns[8 * unit + m], pos, p.plan.amplitude, ik);
        }
        if (interleaved) {
          o1 = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
          o2 = make_uint2(code[4] | code[5] << 16, code[6] | code[7] << 16);
        } else {
          const uint32_t a0 = __byte_perm(code[0], code[1], 0x5140), a1 = __byte_perm(code[2], code[3], 0x5140);
          const uint32_t a2 = __byte_perm(code[4], code[5], 0x5140), a3 = __byte_perm(code[6], code[7], 0x5140);
          o1 = make_uint2(__byte_perm(a0, a1, 0x5410), __byte_perm(a2, a3, 0x5410));
          o2 = make_uint2(__byte_perm(a0, a1, 0x7632), __byte_perm(a2, a3, 0x7632));
        }
      } else {
        o1 = codes8(x1, ik);
        o2 = codes8(x2, ik);
      }
      *reinterpret_cast<uint2*>(ko + d1) = o1;
      *reinterpret_cast<uint2*>(ko + d2) = o2;
      unpack8(vr[i][0], x1);
      unpack8(vr[i][1], x2);
      *reinterpret_cast<uint2*>(vo + d1) = codes8(x1, iv);
      *reinterpret_cast<uint2*>(vo + d2) = codes8(x2, iv);
    }
  }
}

}  // namespace

int check_paged_cache(const RelposPagedCache* c) {
  if (!c) return RELPOS_ERR_INVALID_ARG;
  if (c->dtype != RELPOS_BF16 && c->dtype != RELPOS_E4M3) return RELPOS_ERR_INVALID_ARG;
  if (c->num_pages < 0 || c->H < 0 || c->d <= 0 || c->page <= 0) return RELPOS_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return RELPOS_ERR_UNSUPPORTED;
  if (c->page != 32 && c->page != 64 && c->page != 128) return RELPOS_ERR_UNSUPPORTED;
  if (c->H > 65535) return RELPOS_ERR_UNSUPPORTED;
  if (c->num_pages > 0 && c->H > 0) {
    if (!c->k || !c->v || !aligned16(c->k) || !aligned16(c->v)) return RELPOS_ERR_INVALID_ARG;
    if (c->dtype == RELPOS_E4M3 &&
        (!c->k_scale || !c->v_scale || (reinterpret_cast<uintptr_t>(c->k_scale) & 3u) ||
         (reinterpret_cast<uintptr_t>(c->v_scale) & 3u)))
      return RELPOS_ERR_INVALID_ARG;
  }
  return RELPOS_OK;
}

}  // namespace relpos

using namespace relpos;

extern "C" int relpos_paged_append(const RelposPagedCache* cache, const RelposRotaryPlan* plan, const void* K,
                                   const void* V, const RelposRowStrides* ks, const RelposRowStrides* vs,
                                   const int* cu_new, int rows, int n, int B, const int* block_table,
                                   long long table_stride, int max_pages, const int* lens, void* stream) {
  int rc = check_paged_cache(cache);
  if (rc != RELPOS_OK) return rc;
  if (plan && !rotary_plan_ok(plan)) return RELPOS_ERR_INVALID_ARG;
  if (!ks || !vs || B < 0 || rows < 0 || n < 0 || max_pages < 0) return RELPOS_ERR_INVALID_ARG;
  if (plan && plan->rot_dim > cache->d) return RELPOS_ERR_INVALID_ARG;
  if (plan && plan->rot_dim % 16) return RELPOS_ERR_UNSUPPORTED;
  const long long total = cu_new ? rows : static_cast<long long>(B) * n;
  if (B == 0 || cache->H == 0 || total == 0) return RELPOS_OK;
  if (!K || !V || !block_table || !lens || max_pages == 0 || cache->num_pages == 0) return RELPOS_ERR_INVALID_ARG;
  const uintptr_t ints = reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(lens) |
                         reinterpret_cast<uintptr_t>(cu_new);
  const uintptr_t rowp = reinterpret_cast<uintptr_t>(K) | reinterpret_cast<uintptr_t>(V);
  if ((ints & 3u) || (rowp & 1u)) return RELPOS_ERR_INVALID_ARG;
  if (B > 1 && table_stride < max_pages) return RELPOS_ERR_INVALID_ARG;
  const long long capacity = static_cast<long long>(max_pages) * cache->page;
  if (total > (1 << 28) || B > (1 << 24) || capacity > (1 << 28)) return RELPOS_ERR_UNSUPPORTED;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  if (plan) p.plan = *plan;
  p.cache = *cache;
  p.K = static_cast<const __nv_bfloat16*>(K);
  p.V = static_cast<const __nv_bfloat16*>(V);
  p.k_batch = ks->batch, p.k_head = ks->head, p.k_row = ks->row;
  p.v_batch = vs->batch, p.v_head = vs->head, p.v_row = vs->row;
  const long long odd = p.k_head | p.k_row | p.v_head | p.v_row | (cu_new ? 0 : p.k_batch | p.v_batch);
  p.vec = (rowp & 15u) == 0 && odd % 8 == 0;
  p.cu = cu_new;
  p.n = n;
  p.rows = static_cast<int>(total);
  p.B = B;
  p.table = block_table;
  p.table_stride = table_stride;
  p.max_pages = max_pages;
  p.lens = lens;
  p.log_page = cache->page == 32 ? 5 : cache->page == 64 ? 6 : 7;
  p.log_units = cache->d == 64 ? 2 : 3;
  p.group = (kAppThreads * kAppSlots) >> (p.log_page + p.log_units);  // 8 .. 1 heads
  p.reach = plan ? 1.4142135623730951 * plan->amplitude : 1.0;
  p.status = device_status();
  if (!p.status) return RELPOS_ERR_CUDA;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((total >> p.log_page) + 2 * static_cast<long long>(B)),
                     (cache->H + p.group - 1) / p.group);
  cfg.blockDim = dim3(kAppThreads);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cache->dtype == RELPOS_E4M3 ? cudaLaunchKernelEx(&cfg, relpos_paged_append_kernel<true>, p)
                                                    : cudaLaunchKernelEx(&cfg, relpos_paged_append_kernel<false>, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  return RELPOS_OK;
}
