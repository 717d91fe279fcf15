// paged_decode.cu -- attention of a few new rows over a paged key/value cache,
// bf16 or e4m3 with a scale for each page and head ("Relative Position
// Embeddings, in depth", section "Kernels and the KV cache"), with no bias, the
// T5 bucket bias or ALiBi, and grouped heads.
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale q_r . k_j + bias_rj - m_r)
//
// The cache is streamed once, about one product per byte and row, so the kernel
// is built around keeping loads in flight; the products of the up to 16 rows
// that share a key/value head (query heads of the group times new rows) run on
// the tensor cores' m16n8k16 form, whose operands come straight out of the
// streamed tile's registers.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <type_traits>

#include "../../include/relpos_attn.h"
#include "ptx.cuh"
#include "relpos_common.cuh"
#include "relpos_internal.h"

namespace relpos {
namespace {

constexpr int kPdWarps = 4;
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdRows = 16;     // rows of a unit: the m of the matrix instruction
constexpr int kPdMinTiles = 4;  // fewest tiles of a block's share: one for each warp
// exponent offset of the weights p: they reach 2^12, so that fp16 weights (8-bit
// caches) keep 11 bits down to 2^-26 of the largest and vanish below 2^-36
constexpr float kPdShift = 12.f;

struct PagedDecodeParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int num_pages, Hkv, log_page;
  const __nv_bfloat16* Q;
  long long q_batch, q_head, q_row;
  __nv_bfloat16* out;
  long long o_batch, o_head, o_row;
  const int* table;
  long long table_stride;
  int max_len;  // tokens that the block table's row can name
  const int* lens;
  int B, Hq, Lq, G;  // G: query heads of a key/value head
  int rt;            // 16-row tiles of the G * Lq rows of a key/value head
  const float* bias;
  int t5_R;
  T5Index t5;
  float scale_log2;
  float* part_o;   // [blocks][2][16][d] partial outputs
  float* part_ml;  // [blocks][2][16][2] their maxima and sums
  int blocks;
  int* status;
};

// A unit is one sequence, key/value head and 16-row tile; units follow one
// another in that order, each with the sequence's key tiles. A block takes an
// equal share of the tiles of all units, whatever the lengths, and its warps
// every fourth tile of it.

RP_DEVI int seq_tiles(const PagedDecodeParams& p, int b, int KT) {
  const int len = __ldg(p.lens + b);
  return (min(max(len, 0), p.max_len) + KT - 1) / KT;
}

// Key tiles of the units before sequence b (b = B: of all), summed by a warp.
RP_DEVI int tiles_before(const PagedDecodeParams& p, int b, int KT, int lane) {
  int sum = 0;
  for (int i = lane; i < b; i += 32) sum += seq_tiles(p, i, KT);
  return __reduce_add_sync(0xffffffffu, sum) * p.Hkv * p.rt;
}

RP_DEVI int share_of(int total, int blocks) { return max((total + blocks - 1) / blocks, kPdMinTiles); }

// Place in the sequence of tiles: sequence, unit of it, tile of the unit.
struct Cursor {
  int b, u, t, nt;
  RP_DEVI void skip_empty(const PagedDecodeParams& p, int KT) {
    while (nt == 0 && b < p.B) {
      ++b;
      nt = b < p.B ? seq_tiles(p, b, KT) : 0;
    }
  }
  RP_DEVI void forward(const PagedDecodeParams& p, int KT, int by) {
    t += by;
    while (b < p.B && t >= nt) {
      t -= nt;
      if (++u == p.Hkv * p.rt) {
        u = 0;
        ++b;
        nt = b < p.B ? seq_tiles(p, b, KT) : 0;
        skip_empty(p, KT);
      }
    }
  }
};

// The cursor at tile x of all; warp-uniform.
RP_DEVI Cursor seek(const PagedDecodeParams& p, int KT, int x, int lane) {
  const int per = p.Hkv * p.rt;
  int before = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int nt = b0 + lane < p.B ? seq_tiles(p, b0 + lane, KT) : 0;
    int upto = nt;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    // the first sequence whose tiles end behind x
    const unsigned past = __ballot_sync(0xffffffffu, (before + upto) * per > x);
    if (past) {
      const int l = __ffs(past) - 1;
      Cursor c;
      c.b = b0 + l;
      c.nt = __shfl_sync(0xffffffffu, nt, l);
      const int rest = x - (before + __shfl_sync(0xffffffffu, upto - nt, l)) * per;
      c.u = rest / c.nt;
      c.t = rest - c.u * c.nt;
      return c;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  return Cursor{p.B, 0, 0, 0};
}

RP_DEVI void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
RP_DEVI void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
RP_DEVI void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
RP_DEVI void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
RP_DEVI uint4 lds128(uint32_t a) {
  uint4 u;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(a) : "memory");
  return u;
}
RP_DEVI uint2 lds64(uint32_t a) {
  uint2 u;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u.x), "=r"(u.y) : "r"(a) : "memory");
  return u;
}
RP_DEVI float lds32f(uint32_t a) {
  float f;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(a) : "memory");
  return f;
}

// two e4m3 codes to two fp16 values (exact), from the low or high half of w
RP_DEVI uint32_t half2_lo(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(w));
  return h;
}
RP_DEVI uint32_t half2_hi(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, b;\n\t}" : "=r"(h) : "r"(w));
  return h;
}

template <bool F16>
RP_DEVI void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

RP_DEVI uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
RP_DEVI uint32_t pack_bf2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Shapes of a variant: head dimension, cache type, keys of a tile, ring stages.
// A tile divides a page, so it has one page number and one pair of scales.
template <int D, bool FP8, int KT, int STAGES>
struct Shape {
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;       // 16-byte chunks of a key's row
  static constexpr int kTileBytes = KT * kRowBytes;    // of the keys, and of the values
  static constexpr int kStageBytes = 2 * kTileBytes + 16;  // and the two scales
  static constexpr int kRingBytes = STAGES * kStageBytes;  // of a warp
  static constexpr int kOutPitch = D + 4;
  static constexpr int kSmem = kPdWarps * kRingBytes + kPdRows * kOutPitch * 4 + kPdWarps * kPdRows * 2 * 4;
  static constexpr int kIters = KT * kChunks / 32;     // 16-byte copies of a lane, of each of K and V
};

// Chunk c of row r lies at chunk c ^ f(r) of its row in shared memory. A
// quarter-warp reads the keys by 4 chunks of rows 2i, 2i + 1, the values by 2
// chunks of rows 2t + o for t = 0..3; with this f both meet 8 different banks
// groups (rows of 64 bytes, two to a bank line, need only the row pair's index).
template <int CHUNKS>
RP_DEVI constexpr int swizzle(int r) {
  return CHUNKS == 4 ? (r >> 1) & 3 : (((r >> 1) & 3) << 1) ^ ((r & 1) << 2);
}

// MODE: RELPOS_NO_BIAS, RELPOS_T5 or RELPOS_ALIBI
template <int D, bool FP8, int KT, int STAGES, int MODE>
__global__ void __launch_bounds__(kPdThreads) relpos_paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  using S = Shape<D, FP8, KT, STAGES>;
  constexpr int NT = KT / 8;    // 8-key tiles of the scores
  constexpr int KS = D / 16;    // 16-dim steps of q . k
  constexpr int ND = D / 8;     // 8-dim tiles of the output
  constexpr int KK = KT / 16;   // 16-key steps of p v
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * S::kRingBytes;
  float* const out_s = reinterpret_cast<float*>(smem + kPdWarps * S::kRingBytes);
  float* const ml_s = out_s + kPdRows * S::kOutPitch;

  griddep_wait();
  const int total = tiles_before(p, p.B, KT, lane);
  const int share = share_of(total, p.blocks);
  const int x0 = min(static_cast<int>(blockIdx.x) * share, total), x1 = min(x0 + share, total);
  if (x0 >= x1) {
    griddep_launch_dependents();
    return;
  }

  // ---- producer: this warp's tiles x0 + warp, x0 + warp + 4, ... into its ring
  Cursor pc = seek(p, KT, x0, lane);
  const Cursor first = pc;
  pc.forward(p, KT, warp);
  int px = x0 + warp;
  auto page_of = [&](const Cursor& c) {
    return __ldg(p.table + c.b * p.table_stride + ((c.t * KT) >> p.log_page));
  };
  int next_page = px < x1 ? page_of(pc) : 0;  // a step ahead: its load does not delay the copies
  const int r0 = lane / S::kChunks, ch = lane % S::kChunks;
  const uint32_t dst0 = r0 * S::kRowBytes + ((ch ^ swizzle<S::kChunks>(r0)) << 4);
  auto produce = [&](int stage) {
    if (px < x1) {
      const int key0 = pc.t * KT;
      int valid = min(__ldg(p.lens + pc.b), p.max_len) - key0;
      int page = next_page;
      if (page < 0 || page >= p.num_pages) {  // zeros in its place, and the error on record
        if (lane == 0) atomicCAS(p.status, 0, RELPOS_ERR_PAGE);
        page = 0;
        valid = 0;
      }
      const int h = pc.u / p.rt;
      const size_t ph = static_cast<size_t>(page) * p.Hkv + h;
      const size_t at = ((ph << p.log_page) + (key0 & ((1 << p.log_page) - 1))) * S::kRowBytes + lane * 16;
      const uint32_t base = ring + stage * S::kStageBytes;
#pragma unroll
      for (int i = 0; i < S::kIters; ++i) {
        const int row = r0 + i * (32 / S::kChunks);
        const uint32_t dst = (dst0 ^ (swizzle<S::kChunks>(i * (32 / S::kChunks)) << 4)) + i * 512;
        const int bytes = row < valid ? 16 : 0;  // zeros behind the sequence's end
        cp_async16(base + dst, p.k + at + i * 512, bytes);
        cp_async16(base + S::kTileBytes + dst, p.v + at + i * 512, bytes);
      }
      if constexpr (FP8) {
        if (lane < 2) cp_async4(base + 2 * S::kTileBytes + lane * 4, (lane ? p.v_scale : p.k_scale) + ph);
      }
      px += kPdWarps;
      if (px < x1) {
        pc.forward(p, KT, kPdWarps);
        next_page = page_of(pc);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < STAGES - 1; ++i) produce(i);

  // ---- consumer: the block's units one after another
  uint32_t k_off[FP8 ? D / 64 : D / 32], v_off[2];
#pragma unroll
  for (int j = 0; j < (FP8 ? D / 64 : D / 32); ++j)
    k_off[j] = g * S::kRowBytes + (((t + 4 * j) ^ swizzle<S::kChunks>(g)) << 4);
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int row = 2 * t + o;
    if constexpr (FP8 && D == 64)
      v_off[o] = row * S::kRowBytes + (((g >> 1) ^ swizzle<S::kChunks>(row)) << 4) + (g & 1) * 8;
    else
      v_off[o] = row * S::kRowBytes + ((g ^ swizzle<S::kChunks>(row)) << 4);
  }

  int stage = 0;
  int x = x0;
  Cursor cc = first;
  while (x < x1) {
    const int xe = min(x1, x + cc.nt - cc.t);  // the unit's tiles in this block
    const int len_raw = __ldg(p.lens + cc.b);
    const int len = min(len_raw, p.max_len);
    if (len_raw > p.max_len && threadIdx.x == 0) atomicCAS(p.status, 0, RELPOS_ERR_PAGE);
    const int h = cc.u / p.rt, row0 = (cc.u - h * p.rt) * kPdRows;
    const int rows = min(p.G * p.Lq - row0, kPdRows);
    // this lane's rows g and g + 8: query row, head, last key that it sees
    int vis[2];
    float slope[2], bias_far[2];
    uint32_t q[KS][4];
    float qs[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = g + 8 * e;
      const int i = (row0 + r) / p.G;
      const int hq = h * p.G + (row0 + r) - i * p.G;
      const bool real = r < rows;
      vis[e] = real ? len - p.Lq + i : -1;
      slope[e] = bias_far[e] = 0.f;
      if (MODE == RELPOS_ALIBI && real) slope[e] = __ldg(p.bias + hq) * kLog2e;
      if (MODE == RELPOS_T5 && real) {
        // a finite bias stays finite in log2 units
        const float far = __ldg(p.bias + (p.t5.slots - 1) * p.Hq + hq);
        bias_far[e] = fabsf(far) <= FLT_MAX ? fminf(fmaxf(far * kLog2e, -FLT_MAX), FLT_MAX) : far;
      }
      const __nv_bfloat16* qp = p.Q + cc.b * p.q_batch + hq * p.q_head + i * p.q_row;
      float f[KS][4];
      float big = 0.f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int dim = FP8 ? 16 * (t + 4 * (s / 4)) + 4 * (s % 4) : 8 * (t + 4 * (s / 2)) + 4 * (s % 2);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          f[s][m] = real ? __bfloat162float(qp[dim + m]) : 0.f;
          big = fmaxf(big, fabsf(f[s][m]));
        }
      }
      qs[e] = p.scale_log2;
      if constexpr (FP8) {
        // to fp16 by way of a power of two that brings the row's largest
        // value into [1, 2): exact but for values below 2^-14 of it
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int ex = min(126, max(-126, static_cast<int>(__float_as_uint(big) >> 23) - 127));
        const float down = __int_as_float((127 - ex) << 23);
        qs[e] *= __int_as_float((127 + ex) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          q[s][e] = pack_half2(f[s][0] * down, f[s][1] * down);
          q[s][2 + e] = pack_half2(f[s][2] * down, f[s][3] * down);
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          q[s][e] = pack_bf2(f[s][0], f[s][1]);
          q[s][2 + e] = pack_bf2(f[s][2], f[s][3]);
        }
      }
    }
    const int vis_first = len - p.Lq + row0 / p.G;  // last key that every row sees
    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    float o[ND][4];
#pragma unroll
    for (int j = 0; j < ND; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;

    // this warp's tiles of the unit: x + k with (x - x0 + k) mod 4 = warp
    for (int y = x + ((warp - (x - x0)) & (kPdWarps - 1)); y < xe; y += kPdWarps) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      produce(stage == 0 ? STAGES - 1 : stage - 1);
      const uint32_t ks = ring + stage * S::kStageBytes, vs = ks + S::kTileBytes;
      if (++stage == STAGES) stage = 0;
      const int key0 = (cc.t + y - x) * KT;

      // scores of KT keys: lane (g, t) holds rows g, g + 8 and keys 8 n + 2 t, + 1
      float sc[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.f;
        if constexpr (FP8) {
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            const uint4 u = lds128(ks + k_off[j] + n * 8 * S::kRowBytes);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) mma16816<true>(sc[n], q[4 * j + i], half2_lo(w[i]), half2_hi(w[i]));
          }
        } else {
#pragma unroll
          for (int j = 0; j < D / 32; ++j) {
            const uint4 u = lds128(ks + k_off[j] + n * 8 * S::kRowBytes);
            mma16816<false>(sc[n], q[2 * j], u.x, u.y);
            mma16816<false>(sc[n], q[2 * j + 1], u.z, u.w);
          }
        }
      }
      float v_scale = 1.f, cs[2] = {qs[0], qs[1]};
      if constexpr (FP8) {
        const float k_scale = lds32f(vs + S::kTileBytes);
        v_scale = lds32f(vs + S::kTileBytes + 4);
        cs[0] *= k_scale;
        cs[1] *= k_scale;
      }
      const bool edge = key0 + KT - 1 > vis_first;  // some row does not see every key
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const bool far = MODE == RELPOS_T5 && vis[e] - (key0 + KT - 1) >= p.t5_R;
        const int hq = MODE == RELPOS_T5 ? h * p.G + (row0 + g + 8 * e) % p.G : 0;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float& z = sc[n][2 * e + m];
            const int back = vis[e] - (key0 + 8 * n + 2 * t + m);
            if (MODE == RELPOS_ALIBI) {
              z = fmaf(z, cs[e], -slope[e] * fabsf(static_cast<float>(back)));
            } else if (MODE == RELPOS_T5) {
              float bias = bias_far[e];
              if (!far && back >= 0) {
                const float w = __ldg(p.bias + t5_bucket_dev(-back, p.t5) * p.Hq + hq);
                bias = fabsf(w) <= FLT_MAX ? fminf(fmaxf(w * kLog2e, -FLT_MAX), FLT_MAX) : w;
              }
              z = fmaf(z, cs[e], bias);
            } else {
              z *= cs[e];
            }
            if (edge && back < 0) z = -INFINITY;
            mx[e] = fmaxf(mx[e], z);
          }
        }
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 1));
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], 2));
      }
      float keep[2] = {1.f, 1.f}, off[2];
      const bool grew = mx[0] > m_run[0] || mx[1] > m_run[1];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float m_new = fmaxf(m_run[e], mx[e]);
        // a row that has seen no key yet keeps zero weights
        off[e] = m_new == -INFINITY ? 0.f : m_new - kPdShift;
        if (grew) keep[e] = m_run[e] == -INFINITY ? 0.f : ex2_approx(m_run[e] - m_new);
        m_run[e] = m_new;
        l_run[e] *= keep[e];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float& z = sc[n][2 * e + m];
            z = ex2_approx(z - off[e]);
            l_run[e] += z;
          }
        }
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int j = 0; j < ND; ++j) {
          o[j][0] *= keep[0];
          o[j][1] *= keep[0];
          o[j][2] *= keep[1];
          o[j][3] *= keep[1];
        }
      }

      // o += p v, for the rows and the keys of one query position (ONE) or all
      auto add_values = [&](auto one, int last) {
        constexpr bool ONE = decltype(one)::value;
        const bool mine[2] = {!ONE || vis[0] == last, !ONE || vis[1] == last};
        uint32_t ph[KK][4];
        [[maybe_unused]] uint32_t pl[FP8 ? 1 : KK][4];
#pragma unroll
        for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
          for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = mine[e] ? sc[2 * kk + n][2 * e] : 0.f, c = mine[e] ? sc[2 * kk + n][2 * e + 1] : 0.f;
              if constexpr (FP8) {
                // 11 bits of a weight: its rounding (2^-12) is far below the
                // output's (2^-9)
                ph[kk][2 * n + e] = pack_half2(a, c);
              } else {
                // bf16 alone would round the weights as coarsely as the
                // output: a second part carries the next 8 bits
                const uint32_t hi = pack_bf2(a, c);
                ph[kk][2 * n + e] = hi;
                pl[kk][2 * n + e] = pack_bf2(a - __uint_as_float(hi << 16), c - __uint_as_float(hi & 0xffff0000u));
              }
            }
          }
        }
        // value rows of the lane: 16 kk + 8 n + 2 t + o
        auto row_words = [&](int kk, int n, int oo, int half, uint32_t (&w)[4]) {
          const uint32_t a = vs + v_off[oo] + (16 * kk + 8 * n) * S::kRowBytes + half * 128;
          if constexpr (FP8 && D == 64) {
            const uint2 u = lds64(a);
            w[0] = u.x, w[1] = u.y, w[2] = w[3] = 0;
          } else {
            const uint4 u = lds128(a);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
          }
          if (ONE && key0 + 16 * kk + 8 * n + 2 * t + oo > last) w[0] = w[1] = w[2] = w[3] = 0;
        };
        if constexpr (FP8) {
          constexpr int W = D / 32;  // words of 4 dims that a lane holds of a row
          uint32_t r[KK][2][2][4];
#pragma unroll
          for (int kk = 0; kk < KK; ++kk)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int oo = 0; oo < 2; ++oo) row_words(kk, n, oo, 0, r[kk][n][oo]);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            float acc[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
            for (int kk = 0; kk < KK; ++kk) {
              const uint32_t a0 = __byte_perm(r[kk][0][0][w], r[kk][0][1][w], 0x5140);
              const uint32_t a1 = __byte_perm(r[kk][0][0][w], r[kk][0][1][w], 0x7362);
              const uint32_t b0 = __byte_perm(r[kk][1][0][w], r[kk][1][1][w], 0x5140);
              const uint32_t b1 = __byte_perm(r[kk][1][0][w], r[kk][1][1][w], 0x7362);
              mma16816<true>(acc[0], ph[kk], half2_lo(a0), half2_lo(b0));
              mma16816<true>(acc[1], ph[kk], half2_hi(a0), half2_hi(b0));
              mma16816<true>(acc[2], ph[kk], half2_lo(a1), half2_lo(b1));
              mma16816<true>(acc[3], ph[kk], half2_hi(a1), half2_hi(b1));
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (mine[e >> 1]) o[4 * w + j][e] = fmaf(acc[j][e], v_scale, o[4 * w + j][e]);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < KK; ++kk) {
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
              uint32_t r[2][2][4];
#pragma unroll
              for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int oo = 0; oo < 2; ++oo) row_words(kk, n, oo, half, r[n][oo]);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  float(&d)[4] = o[8 * half + 2 * w + j];
                  const float was[4] = {d[0], d[1], d[2], d[3]};
                  const uint32_t b0 = __byte_perm(r[0][0][w], r[0][1][w], j ? 0x7632 : 0x5410);
                  const uint32_t b1 = __byte_perm(r[1][0][w], r[1][1][w], j ? 0x7632 : 0x5410);
                  mma16816<false>(d, ph[kk], b0, b1);
                  mma16816<false>(d, pl[kk], b0, b1);
                  if (ONE) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = mine[e >> 1] ? d[e] : was[e];
                  }
                }
              }
            }
          }
        }
      };
      // Where rows of one tile see different keys, the rows of each query
      // position go alone, with the values that they do not see as zeros, so
      // that what lies there (it may be NaN) cannot reach them.
      if (edge && p.Lq > 1) {
        for (int i = 0; i < p.Lq; ++i) add_values(std::true_type{}, len - p.Lq + i);
      } else {
        add_values(std::false_type{}, 0);
      }
    }

    // ---- the four warps' parts of the unit, joined in a fixed order
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 1);
      l_run[e] += __shfl_xor_sync(0xffffffffu, l_run[e], 2);
      if (t == 0) {
        ml_s[(warp * kPdRows + g + 8 * e) * 2] = m_run[e];
        ml_s[(warp * kPdRows + g + 8 * e) * 2 + 1] = l_run[e];
      }
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m = -INFINITY;
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w) m = fmaxf(m, ml_s[(w * kPdRows + g + 8 * e) * 2]);
      f[e] = m_run[e] == -INFINITY ? 0.f : ex2_approx(m_run[e] - m);
    }
    for (int w = 0; w < kPdWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float* row = out_s + (g + 8 * e) * S::kOutPitch;
#pragma unroll
          for (int j = 0; j < ND; ++j) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              // dim of column 2 t + c of output tile j, as the values were read
              const int n = 2 * t + c;
              const int dim = FP8 ? (D / 8) * n + j : (j / 8) * 64 + 8 * n + j % 8;
              const float val = o[j][2 * e + c] * f[e];
              row[dim] = w ? row[dim] + val : val;
            }
          }
        }
      }
      __syncthreads();
    }
    const bool whole = cc.t == 0 && xe - x == cc.nt;
    const int slot = 2 * blockIdx.x + (cc.t == 0 ? 1 : 0);
    for (int i = threadIdx.x; i < rows * (D / 4); i += kPdThreads) {
      const int r = i / (D / 4), d4 = i % (D / 4);
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w) m = fmaxf(m, ml_s[(w * kPdRows + r) * 2]);
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w) {
        const float mw = ml_s[(w * kPdRows + r) * 2];
        if (mw != -INFINITY) l = fmaf(ex2_approx(mw - m), ml_s[(w * kPdRows + r) * 2 + 1], l);
        else l += ml_s[(w * kPdRows + r) * 2 + 1];
      }
      const float4 v = *reinterpret_cast<const float4*>(out_s + r * S::kOutPitch + 4 * d4);
      if (whole) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int qi = (row0 + r) / p.G;
        const int hq = h * p.G + (row0 + r) - qi * p.G;
        __nv_bfloat16* op = p.out + cc.b * p.o_batch + hq * p.o_head + qi * p.o_row + 4 * d4;
        op[0] = __float2bfloat16_rn(v.x * inv);
        op[1] = __float2bfloat16_rn(v.y * inv);
        op[2] = __float2bfloat16_rn(v.z * inv);
        op[3] = __float2bfloat16_rn(v.w * inv);
      } else {
        *reinterpret_cast<float4*>(p.part_o + (static_cast<size_t>(slot) * kPdRows + r) * D + 4 * d4) = v;
        if (d4 == 0) {
          p.part_ml[(slot * kPdRows + r) * 2] = m;
          p.part_ml[(slot * kPdRows + r) * 2 + 1] = l;
        }
      }
    }
    __syncthreads();  // out_s and ml_s are free again
    cc.forward(p, KT, xe - x);
    x = xe;
  }
  cp_async_wait<0>();
  griddep_launch_dependents();
}

// One block for each unit and row: units that several blocks shared, joined in
// block order; units without keys, zero.
template <int D, int KT>
__global__ void __launch_bounds__(kPdThreads) relpos_paged_combine_kernel(const __grid_constant__ PagedDecodeParams p) {
  constexpr int LANES = D / 4, PARTS = kPdThreads / LANES;
  __shared__ float red[PARTS][D + 4];
  __shared__ float lsum[PARTS];
  griddep_launch_dependents();
  griddep_wait();
  const int per = p.Hkv * p.rt;
  const int b = blockIdx.x / per, u = blockIdx.x - b * per;
  const int h = u / p.rt, row = (u - h * p.rt) * kPdRows + blockIdx.y;
  if (row >= p.G * p.Lq) return;
  const int lane = threadIdx.x & 31;
  const int nt = seq_tiles(p, b, KT);
  const int total = tiles_before(p, p.B, KT, lane);
  const int share = share_of(total, p.blocks);
  const int xs = tiles_before(p, b, KT, lane) + u * nt, xe = xs + nt;
  const int c0 = xs / share, c1 = nt ? (xe - 1) / share : c0 - 1;
  if (c1 == c0) return;  // one block had the whole unit
  const int d4 = threadIdx.x % LANES, part = threadIdx.x / LANES;
  float m = -INFINITY;
  for (int c = c0; c <= c1; ++c) {
    const size_t slot = (2 * static_cast<size_t>(c) + (c * share <= xs ? 1 : 0)) * kPdRows + blockIdx.y;
    m = fmaxf(m, p.part_ml[2 * slot]);
  }
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int c = c0 + part; c <= c1; c += PARTS) {
    const size_t slot = (2 * static_cast<size_t>(c) + (c * share <= xs ? 1 : 0)) * kPdRows + blockIdx.y;
    const float mc = p.part_ml[2 * slot];
    const float w = mc == -INFINITY ? 0.f : ex2_approx(mc - m);
    const float lc = p.part_ml[2 * slot + 1];
    l += mc == -INFINITY ? lc : w * lc;
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + slot * D + 4 * d4);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
    acc.z = fmaf(w, v.z, acc.z);
    acc.w = fmaf(w, v.w, acc.w);
  }
  *reinterpret_cast<float4*>(&red[part][4 * d4]) = acc;
  if (d4 == 0) lsum[part] = l;
  __syncthreads();
  if (threadIdx.x < D) {
    float a = 0.f, s = 0.f;
#pragma unroll
    for (int i = 0; i < PARTS; ++i) {
      a += red[i][threadIdx.x];
      s += lsum[i];
    }
    const int qi = row / p.G, hq = h * p.G + row - qi * p.G;
    p.out[b * p.o_batch + hq * p.o_head + qi * p.o_row + threadIdx.x] =
        __float2bfloat16_rn(s == 0.f ? 0.f : a / s);
  }
}

// What a variant needs to be launched: its kernels, tile size and shared memory.
struct Variant {
  void (*decode)(PagedDecodeParams);
  void (*combine)(PagedDecodeParams);
  int tile, smem;
};

template <int D, bool FP8, int KT, int STAGES>
Variant variant_of(int mode) {
  Variant v;
  v.decode = mode == RELPOS_T5 ? relpos_paged_decode_kernel<D, FP8, KT, STAGES, RELPOS_T5>
             : mode == RELPOS_ALIBI ? relpos_paged_decode_kernel<D, FP8, KT, STAGES, RELPOS_ALIBI>
                                    : relpos_paged_decode_kernel<D, FP8, KT, STAGES, RELPOS_NO_BIAS>;
  v.combine = relpos_paged_combine_kernel<D, KT>;
  v.tile = KT;
  v.smem = Shape<D, FP8, KT, STAGES>::kSmem;
  return v;
}

// Tiles and stages by head dimension and type, so that a warp has 8 to 16 KB
// in flight.
Variant pick(int d, int dtype, int mode) {
  if (dtype == RELPOS_E4M3) return d == 64 ? variant_of<64, true, 32, 3>(mode) : variant_of<128, true, 32, 3>(mode);
  return d == 64 ? variant_of<64, false, 32, 3>(mode) : variant_of<128, false, 16, 3>(mode);
}

}  // namespace
}  // namespace relpos

using namespace relpos;

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
  if (bias_mode != RELPOS_NO_BIAS && !bias) return RELPOS_ERR_INVALID_ARG;
  if (max_pages == 0 || cache->num_pages == 0) return RELPOS_ERR_INVALID_ARG;
  if (B > 1 && table_stride < max_pages) return RELPOS_ERR_INVALID_ARG;
  const int G = Hq / cache->H;
  if (G > 65535) return RELPOS_ERR_UNSUPPORTED;
  const int rt = (G * Lq + kPdRows - 1) / kPdRows;
  const long long capacity = static_cast<long long>(max_pages) * cache->page;
  if (capacity > (1 << 28)) return RELPOS_ERR_UNSUPPORTED;
  const Variant v = pick(cache->d, cache->dtype, bias_mode);
  const long long units = static_cast<long long>(B) * cache->H * rt;
  const long long most = units * ((capacity + v.tile - 1) / v.tile);  // tiles, with every page in use
  if (units > 0x7fffffffll || most > 0x7fffffffll) return RELPOS_ERR_UNSUPPORTED;

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
  p.out = static_cast<__nv_bfloat16*>(out);
  p.o_batch = os->batch, p.o_head = os->head, p.o_row = os->row;
  p.table = block_table;
  p.table_stride = table_stride;
  p.max_len = static_cast<int>(capacity);
  p.lens = lens;
  p.B = B, p.Hq = Hq, p.Lq = Lq, p.G = G, p.rt = rt;
  p.bias = static_cast<const float*>(bias);
  if (bias_mode == RELPOS_T5) {
    rc = t5_setup(num_buckets, max_distance, 1, capacity, &p.t5, &p.t5_R);
    if (rc != RELPOS_OK) return rc;
  }
  p.scale_log2 = (scale != 0.f ? scale : 1.0f / std::sqrt(static_cast<float>(cache->d))) * kLog2e;
  p.status = device_status();
  const int sms = device_sms();
  if (!p.status || sms <= 0) return RELPOS_ERR_CUDA;
  if (cudaFuncSetAttribute(v.decode, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  int occ = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, v.decode, kPdThreads, v.smem) != cudaSuccess || occ < 1) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  p.blocks = static_cast<int>(std::min<long long>(static_cast<long long>(occ) * sms, (most + kPdMinTiles - 1) / kPdMinTiles));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const size_t slots = static_cast<size_t>(p.blocks) * 2 * kPdRows;
  float* scratch = nullptr;
  if (cudaMallocAsync(&scratch, slots * (cache->d + 2) * sizeof(float), s) != cudaSuccess) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  p.part_o = scratch;
  p.part_ml = scratch + slots * cache->d;
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
  cfg.gridDim = dim3(static_cast<unsigned>(units), std::min(G * Lq, kPdRows));
  cfg.dynamicSmemBytes = 0;
  ok = ok && cudaLaunchKernelEx(&cfg, v.combine, p) == cudaSuccess;
  ok = cudaFreeAsync(scratch, s) == cudaSuccess && ok;
  if (!ok) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  return RELPOS_OK;
}
