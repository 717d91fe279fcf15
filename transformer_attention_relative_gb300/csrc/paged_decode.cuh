// paged_decode.cuh -- the kernels of attention of a few new rows over a paged
// key/value cache, bf16 or e4m3 with a scale for each page and head ("Relative
// Position Embeddings, in depth", section "Kernels and the KV cache"), with no
// bias, the T5 bucket bias or ALiBi, and grouped heads.
//
//   out_r = sum_j p_rj v_j / sum_j p_rj,  p_rj = exp(scale q_r . k_j + bias_rj - m_r)
//
// The cache is streamed once, about one product per byte and row, so the kernel
// is built around keeping loads in flight: each warp has its own ring of tiles
// in shared memory, filled by asynchronous copies. The products of the up to 16
// rows that share a key/value head (query heads of the group times new rows)
// run on the tensor cores' m16n8k16 form, whose operands come straight out of
// the streamed tile.
//
// Bounded by HBM for large batches: 32 x 4096 tokens of 16 heads in 8 bits (269
// MB) 51 us, 5.3 TB/s, 93 % of a copy's rate while it streams (slope over the
// length) and 9 us for its start, the spread of the blocks' ends and the joining
// kernel; 2 x 131075 tokens, d = 128, 16 query and 4 key heads 56 us. Small
// batches are bounded by the chain lengths, table, tile, products, joining: 113
// tokens 5 us.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "../../include/relpos_attn.h"
#include "ptx.cuh"
#include "relpos_common.cuh"

namespace relpos {

constexpr int kPdWarps = 4;
constexpr int kPdThreads = 32 * kPdWarps;
constexpr int kPdMinTiles = 4;  // fewest tiles of a block's share: one for each warp
constexpr int kPdUnitCost = 12;  // what a unit costs a block beside its tiles, in tiles
constexpr int kPdBuckets = 256;

// The weights p are kept as 2^(logit - off) for a row offset `off` that starts
// below every logit and moves up only when a logit comes more than kPdMost above
// it, to kPdShift below the largest: most tiles then need no maximum across the
// warp and no rescaling. Weights stay below 2^13, and fp16 ones (8-bit caches)
// take a factor between 1/2 and 4 with their page's scale: they keep 11 bits
// down to 2^-18 of a row's largest weight, 2^5 or more, and below that are off by
// 2^-29 of it at most: n keys together by n 2^-29 (2^-12 of it for 131072).
constexpr float kPdShift = 5.f, kPdMost = 13.f;

// 8-bit values: the output is kept in units of v_unit, a power of two near the
// scales of the pages, and the weights of a page take its scale's ratio to it.
// Where a page's ratio is outside [kPdRatioLow, kPdRatioHigh] the unit moves to
// its scale, but only between these bounds: a page may have any scale (zero
// values 2^-120, an infinite one 2^120), and sums of weights (2^13), codes (448)
// and ratios over 2^28 keys, 2^53, stay finite when they move from the upper
// bound's unit to the lower one's. Pages of smaller scale add their products
// with the ratio in fp32, and so do all tiles from a page of larger scale on, in
// units of twice the upper bound.
constexpr float kPdRatioLow = 0.5f, kPdRatioHigh = 4.f;
constexpr float kPdUnitLow = 0x1p-32f, kPdUnitHigh = 0x1p32f;

struct PagedDecodeParams {
  const uint8_t* k;
  const uint8_t* v;
  const float* k_scale;
  const float* v_scale;
  int num_pages, Hkv, log_page;
  const __nv_bfloat16* Q;
  long long q_batch, q_head, q_row;
  int q_vec, o_vec;  // rows of Q and of out are 16-byte aligned
  __nv_bfloat16* out;
  long long o_batch, o_head, o_row;
  const int* table;
  long long table_stride;
  int max_len;  // tokens that the block table's row can name
  const int* lens;
  int B, Hq, Lq, G;  // G: query heads of a key/value head
  int rows;          // rows of a unit (a multiple of 8)
  int rt;            // units that the G * Lq rows of a key/value head take
  const float* bias;
  int mode;          // RELPOS_NO_BIAS, RELPOS_T5 or RELPOS_ALIBI
  int t5_R;
  T5Index t5;
  uint8_t bucket[kPdBuckets];  // T5 buckets of the first distances
  float scale_log2;
  float* part_o;   // [blocks][2][rows][d] partial outputs
  float* part_ml;  // [blocks][2][rows][2] their offsets and sums
  // [blocks][2] what a slot holds: first block and number of blocks of its unit
  // (0: nothing), sequence, unit
  int4* ends;
  int blocks;
  int direct;      // a block for each unit: nothing to combine
  int* status;
};

// A variant's kernels, tile size and shared memory; one translation unit each
// for the head dimensions and types. `rows8`: 8-row groups of a unit.
struct PagedDecodeVariant {
  void (*decode)(PagedDecodeParams);
  void (*combine)(PagedDecodeParams);
  int tile, smem;
};
PagedDecodeVariant paged_decode_e4m3_64(int rows8);
PagedDecodeVariant paged_decode_e4m3_128(int rows8);
PagedDecodeVariant paged_decode_bf16_64(int rows8);
PagedDecodeVariant paged_decode_bf16_128(int rows8);

namespace {

// A unit is one sequence, key/value head and up to 16 rows; units follow one
// another in that order, each with the sequence's key tiles. A block takes an
// equal share of all units' work, whatever the lengths, and its warps every
// fourth tile of it.

// Tokens of a sequence; none where the block table cannot hold them (which the
// kernel that writes the sequence's zero rows reports).
RP_DEVI int seq_len(const PagedDecodeParams& p, int b) {
  const int len = b < p.B ? __ldg(p.lens + b) : 0;
  return len <= p.max_len ? max(len, 0) : 0;
}
RP_DEVI void report_length(const PagedDecodeParams& p, int b) {
  if (__ldg(p.lens + b) > p.max_len) atomicCAS(p.status, 0, RELPOS_ERR_PAGE);
}

// Place in the sequence of tiles: sequence and its length, unit of it, tile of
// the unit.
struct Cursor {
  int b, u, t, nt, len;
  int h;             // key/value head of the unit
  const int* pages;  // the sequence's row of the block table
  template <int KT>
  RP_DEVI void enter(const PagedDecodeParams& p) {  // the first sequence from b on that has tiles
    nt = len = 0;
    for (; b < p.B; ++b) {
      len = seq_len(p, b);
      nt = (len + KT - 1) / KT;
      pages = p.table + b * p.table_stride;
      if (nt) return;
    }
  }
  template <int KT>
  RP_DEVI void forward(const PagedDecodeParams& p, int by) {
    t += by;
    while (t >= nt && b < p.B) {
      t -= nt;
      if (++u == p.Hkv * p.rt) {
        u = 0;
        ++b;
        enter<KT>(p);
      }
      h = u / p.rt;
    }
  }
};

// A block's share of the work. A unit counts its tiles and kPdUnitCost more, for
// what a block spends on each unit that it touches (its query rows, its first
// logits, the joining of its warps); equal shares of that sum end closer together
// than equal shares of the tiles. len0 are the lengths of the first 32
// sequences, a lane each; all of this is warp-uniform.

// Cost of a sequence's unit
template <int KT>
RP_DEVI int unit_cost(int len) {
  return len > 0 ? (len + KT - 1) / KT + kPdUnitCost : 0;
}

template <int KT>
RP_DEVI int total_cost(const PagedDecodeParams& p, int lane, int len0) {
  int sum = unit_cost<KT>(len0);
  for (int b = lane + 32; b < p.B; b += 32) sum += unit_cost<KT>(seq_len(p, b));
  return __reduce_add_sync(0xffffffffu, sum) * p.Hkv * p.rt;
}

// The cursor at the first tile at or behind cost x of all units (behind the last
// one: sequence p.B), the cost at which its unit starts and the number of tiles
// before it.
template <int KT>
RP_DEVI Cursor locate(const PagedDecodeParams& p, int lane, int len0, int x, int& unit_at, int& before) {
  const int per = p.Hkv * p.rt;
  Cursor c{p.B, 0, 0, 0, 0, 0, p.table};
  int cost = 0, seqs = 0;  // of the sequences looked at, a unit each
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    const int len = b0 ? seq_len(p, b0 + lane) : len0;
    const int mine = unit_cost<KT>(len);
    const unsigned some = __ballot_sync(0xffffffffu, mine > 0);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    // the first sequence whose units end behind x
    const unsigned past = __ballot_sync(0xffffffffu, (cost + upto) * per > x);
    if (past) {
      const int l = __ffs(past) - 1;
      const int unit = __shfl_sync(0xffffffffu, mine, l);
      cost += __shfl_sync(0xffffffffu, upto, l) - unit;
      seqs += __popc(some & ((1u << l) - 1));
      c.b = b0 + l;
      c.len = __shfl_sync(0xffffffffu, len, l);
      c.nt = unit - kPdUnitCost;
      c.pages = p.table + c.b * p.table_stride;
      c.u = (x - cost * per) / unit;
      unit_at = cost * per + c.u * unit;
      c.t = max(x - unit_at - kPdUnitCost, 0);
      c.h = c.u / p.rt;
      before = (cost - seqs * kPdUnitCost) * per + c.u * c.nt + c.t;
      return c;
    }
    cost += __shfl_sync(0xffffffffu, upto, 31);
    seqs += __popc(some);
  }
  unit_at = cost * per;
  before = (cost - seqs * kPdUnitCost) * per;
  return c;
}

template <int DST, int SRC>
RP_DEVI void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(DST), "n"(SRC)
               : "memory");
}
// `bytes` (16 or 0) are copied, the rest is zero
template <int DST, int SRC>
RP_DEVI void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16, %4;" ::"r"(dst), "l"(src), "n"(DST), "n"(SRC),
               "r"(bytes)
               : "memory");
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
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(a)
               : "memory");
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

// an 8 x 8 matrix of 16-bit values, transposed across the warp
RP_DEVI uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

RP_DEVI uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
RP_DEVI uint32_t pack_bf2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Shapes of a variant: head dimension, cache type, 8-row groups of a unit, keys
// of a tile, ring stages. A tile divides a page, so it has one page number and
// one pair of scales.
template <int D, bool FP8, int NQ, int KT, int STAGES>
struct Shape {
  static constexpr int kRows = 8 * NQ;
  static constexpr int kRowBytes = D * (FP8 ? 1 : 2);
  static constexpr int kChunks = kRowBytes / 16;       // 16-byte chunks of a key's row
  static constexpr int kTileBytes = KT * kRowBytes;    // of the keys, and of the values
  static constexpr int kStageBytes = 2 * kTileBytes + 16;  // and the two scales
  static constexpr int kRingBytes = STAGES * kStageBytes;  // of a warp
  static constexpr int kSmem = kPdWarps * kRingBytes + 2 * kRows * D * 4 + kPdWarps * kRows * 2 * 4;
  static constexpr int kIters = KT * kChunks / 32;     // 16-byte copies of a lane, of each of K and V
};

// Chunk c of row r lies at chunk c ^ f(r) of its row in shared memory. A
// quarter-warp reads the keys by 4 chunks of rows 2i, 2i + 1, the values by 2
// chunks of rows 2t + o for t = 0..3; with this f both meet 8 different groups
// of banks (rows of 64 bytes, two to a bank line, need only the row pair's
// index).
template <int CHUNKS>
RP_DEVI constexpr int swizzle(int r) {
  return CHUNKS == 4 ? (r >> 1) & 3 : (((r >> 1) & 3) << 1) ^ ((r & 1) << 2);
}

template <int... I, typename F>
RP_DEVI void for_each(std::integer_sequence<int, I...>, F&& f) {
  (f(std::integral_constant<int, I>{}), ...);
}

// 1 / x for a normal power of two
RP_DEVI float inverse_pow2(float x) { return __uint_as_float(0x7f000000u - __float_as_uint(x)); }

// log2 units, a finite value staying finite (a table may hold the type's lowest)
RP_DEVI float to_log2(float x) {
  return fabsf(x) <= FLT_MAX ? fminf(fmaxf(x * kLog2e, -FLT_MAX), FLT_MAX) : x;
}

// The products are formed the other way round, keys and output dimensions as
// the rows of the matrix instruction (16) and query rows as its columns (8):
// one query row of one head, the common case, then wastes 7 of 8 columns
// instead of 15 of 16 rows, and everything that is done per score or per output
// value halves. K's rows are the A operand as they lie in memory; V^T's A
// operand is V's words of two keys interleaved; p^T, the B operand, is the
// scores' tile transposed across the warp (movmatrix). 8-bit keys and values
// become fp16, exactly (the e4m3 form of the instruction takes more
// instructions here: 510 a tile against 453).
template <int D, bool FP8, int NQ, int KT, int STAGES>
__global__ void __launch_bounds__(kPdThreads, NQ * D <= 64 ? 4 : NQ * D <= 128 ? 3 : 2)
    relpos_paged_decode_kernel(const __grid_constant__ PagedDecodeParams p) {
  using S = Shape<D, FP8, NQ, KT, STAGES>;
  constexpr int MT = KT / 16;   // 16-key tiles of the scores, 16-key steps of v^T p^T
  constexpr int KS = D / 16;    // 16-dim steps of k . q, 16-dim tiles of the output
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_u32(smem) + warp * S::kRingBytes;
  float* const out_s = reinterpret_cast<float*>(smem + kPdWarps * S::kRingBytes);
  float* const ml_s = out_s + 2 * S::kRows * D;

  griddep_wait();
  int tiles;             // of this block
  int size = 0, at = 0;  // cost of a block's share, and that at which the present unit starts
  Cursor pc;
  if (p.direct) {
    const int per = p.Hkv * p.rt;
    pc.b = blockIdx.x / per;
    pc.u = blockIdx.x - pc.b * per;
    pc.t = 0;
    pc.len = seq_len(p, pc.b);
    pc.nt = tiles = (pc.len + KT - 1) / KT;
    pc.h = pc.u / p.rt;
    pc.pages = p.table + pc.b * p.table_stride;
    if (tiles == 0) {  // no key is seen: zero rows
      if (threadIdx.x == 0) report_length(p, pc.b);
      const int row0 = (pc.u - pc.h * p.rt) * S::kRows;
      for (int i = threadIdx.x; i < min(p.G * p.Lq - row0, S::kRows) * D; i += kPdThreads) {
        const int r = row0 + i / D, qi = r / p.G;
        p.out[pc.b * p.o_batch + (pc.h * p.G + r - qi * p.G) * p.o_head + qi * p.o_row + i % D] =
            __float2bfloat16_rn(0.f);
      }
      return;
    }
  } else {
    const int len0 = seq_len(p, lane);
    const int total = total_cost<KT>(p, lane, len0);
    size = max((total + p.blocks - 1) / p.blocks, kPdMinTiles + kPdUnitCost);
    if (threadIdx.x == 0) p.ends[2 * blockIdx.x] = p.ends[2 * blockIdx.x + 1] = make_int4(0, 0, 0, 0);
    const int begin = min(static_cast<int>(blockIdx.x) * size, total);
    if (begin == total) return;
    int first, last, unused;
    locate<KT>(p, lane, len0, min(begin + size, total), unused, last);
    pc = locate<KT>(p, lane, len0, begin, at, first);
    tiles = last - first;
  }

  // ---- producer: this warp's tiles, warp, warp + 4, ... of the block's, into its ring
  Cursor cc = pc;
  pc.forward<KT>(p, warp);
  int px = warp;
  auto page_of = [&](const Cursor& c) { return __ldg(c.pages + ((c.t * KT) >> p.log_page)); };
  int next_page = px < tiles ? page_of(pc) : 0;  // a step ahead: its load does not delay the copies
  unsigned missing = 0;  // bit s: stage s is of a page that does not exist
  const int r0 = lane / S::kChunks, ch = lane % S::kChunks;
  const uint32_t dst0 = r0 * S::kRowBytes + ((ch ^ swizzle<S::kChunks>(r0)) << 4);
  constexpr int kStep = 32 / S::kChunks;  // rows between a lane's copies
  const uint32_t page_bytes = S::kRowBytes << p.log_page;
  const uint8_t *k_lane = p.k + lane * 16, *v_lane = p.v + lane * 16;
  auto produce = [&](int stage) {
    if (px < tiles) {
      const int key0 = pc.t * KT;
      int valid = pc.len - key0;
      uint32_t page = next_page;
      missing &= ~(1u << stage);
      if (page >= static_cast<uint32_t>(p.num_pages)) {  // zeros in its place, and the error on record
        if (lane == 0) atomicCAS(p.status, 0, RELPOS_ERR_PAGE);
        page = 0;
        valid = 0;
        missing |= 1u << stage;
      }
      const uint32_t ph = page * p.Hkv + pc.h;  // (page, head) pairs of a pool are fewer than 2^31
      const size_t at = static_cast<size_t>(ph) * page_bytes + (key0 & ((1 << p.log_page) - 1)) * S::kRowBytes;
      const uint32_t base = ring + stage * S::kStageBytes;
      const uint8_t *kp = k_lane + at, *vp = v_lane + at;
      // row r0 + i kStep goes to dst0 ^ (f(i kStep) << 4) + 512 i: two bases
      const uint32_t even = base + dst0, odd = base + (dst0 ^ (swizzle<S::kChunks>(kStep) << 4));
      auto copy = [&](auto index, auto full) {
        constexpr int i = decltype(index)::value;
        constexpr uint32_t x = swizzle<S::kChunks>(i * kStep) << 4;
        const uint32_t dst = x == 0 ? even : x == (swizzle<S::kChunks>(kStep) << 4) ? odd : base + (dst0 ^ x);
        if constexpr (decltype(full)::value) {
          cp_async16<i * 512, i * 512>(dst, kp);
          cp_async16<S::kTileBytes + i * 512, i * 512>(dst, vp);
        } else {  // zeros behind the sequence's end
          const int bytes = r0 + i * kStep < valid ? 16 : 0;
          cp_async16<i * 512, i * 512>(dst, kp, bytes);
          cp_async16<S::kTileBytes + i * 512, i * 512>(dst, vp, bytes);
        }
      };
      if (valid >= KT)
        for_each(std::make_integer_sequence<int, S::kIters>{}, [&](auto i) { copy(i, std::true_type{}); });
      else
        for_each(std::make_integer_sequence<int, S::kIters>{}, [&](auto i) { copy(i, std::false_type{}); });
      if constexpr (FP8) {
        if (lane < 2) cp_async4(base + 2 * S::kTileBytes + lane * 4, (lane ? p.v_scale : p.k_scale) + ph);
      }
      px += kPdWarps;
      if (px < tiles) {
        pc.forward<KT>(p, kPdWarps);
        next_page = page_of(pc);
      }
    }
    cp_async_commit();
  };
#pragma unroll 1
  for (int i = 0; i < STAGES - 1; ++i) produce(i);

  // ---- consumer: the block's units one after another
  constexpr int KC = FP8 ? D / 64 : D / 32;  // chunks that a lane reads of a key's row
  uint32_t k_off[KC], v_off[2];
#pragma unroll
  for (int j = 0; j < KC; ++j) k_off[j] = g * S::kRowBytes + (((t + 4 * j) ^ swizzle<S::kChunks>(g)) << 4);
#pragma unroll
  for (int o = 0; o < 2; ++o) {
    const int row = 2 * t + o;
    if constexpr (FP8 && D == 64)
      v_off[o] = row * S::kRowBytes + (((g >> 1) ^ swizzle<S::kChunks>(row)) << 4) + (g & 1) * 8;
    else
      v_off[o] = row * S::kRowBytes + ((g ^ swizzle<S::kChunks>(row)) << 4);
  }

  // the first of the 4 dims that a lane holds of q and of a key for step s
  auto dim_of = [&](int s) { return FP8 ? 16 * (t + 4 * (s / 4)) + 4 * (s % 4) : 8 * (t + 4 * (s / 2)) + 4 * (s % 2); };

  int stage = 0;
  int x = 0;
  while (x < tiles) {
    const int xe = min(tiles, x + cc.nt - cc.t);  // the unit's tiles in this block
    const int len = cc.len;
    const int h = cc.h, row0 = (cc.u - h * p.rt) * S::kRows;
    const int rows = min(p.G * p.Lq - row0, S::kRows);

    // T5: the biases of the distances below the last bucket's, for each head
    // of the group, in the joining buffers (free while tiles are read)
    const int lut_len = p.t5_R + 1;
    const bool lut = p.mode == RELPOS_T5 && p.G * static_cast<long long>(lut_len) <= 2 * S::kRows * D &&
                     len - p.Lq - (cc.t + xe - x) * KT + 1 < p.t5_R;
    if (lut) {
      for (int i = threadIdx.x; i < p.G * lut_len; i += kPdThreads) {
        const int hl = i / lut_len, back = i - hl * lut_len;
        const int bucket = back < kPdBuckets ? p.bucket[back] : t5_bucket_dev(-back, p.t5);
        out_s[i] = to_log2(__ldg(p.bias + bucket * p.Hq + h * p.G + hl));
      }
      __syncthreads();
    }

    // row 8 n + g of the unit as the B operand of k . q
    uint32_t q[NQ][KS][2];
    // this lane's score columns, rows 8 n + 2 t and + 1: scale of the products,
    // last key seen, constant and slope of the bias
    float qs[NQ][2], add[NQ][2], slope[NQ][2];
    int vis[NQ][2];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int r = row0 + 8 * n + g;
      const int i = r / p.G, hq = h * p.G + r - i * p.G;
      const bool real = 8 * n + g < rows;
      const __nv_bfloat16* qp = p.Q + cc.b * p.q_batch + hq * p.q_head + i * p.q_row;
      float f[KS][4];
#pragma unroll
      for (int s = 0; s < KS; ++s) f[s][0] = f[s][1] = f[s][2] = f[s][3] = 0.f;
      if (real && p.q_vec) {
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(qp + dim_of(s)));
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            f[s + m / 2][2 * (m & 1)] = __uint_as_float(w[m] << 16);
            f[s + m / 2][2 * (m & 1) + 1] = __uint_as_float(w[m] & 0xffff0000u);
          }
        }
      } else if (real) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int m = 0; m < 4; ++m) f[s][m] = __bfloat162float(qp[dim_of(s) + m]);
      }
      float up = p.scale_log2;
      if constexpr (FP8) {
        // to fp16 by way of a power of two that brings the row's largest
        // value into [1, 2): exact but for values below 2^-14 of it
        float big = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int m = 0; m < 4; ++m) big = fmaxf(big, fabsf(f[s][m]));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
        const int ex = min(126, max(-126, static_cast<int>(__float_as_uint(big) >> 23) - 127));
        const float down = __int_as_float((127 - ex) << 23);
        up *= __int_as_float((127 + ex) << 23);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          q[n][s][0] = pack_half2(f[s][0] * down, f[s][1] * down);
          q[n][s][1] = pack_half2(f[s][2] * down, f[s][3] * down);
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          q[n][s][0] = pack_bf2(f[s][0], f[s][1]);
          q[n][s][1] = pack_bf2(f[s][2], f[s][3]);
        }
      }
      int last = -1;
      float far = 0.f, sl = 0.f;
      if (real) {
        last = len - p.Lq + i;
        if (p.mode == RELPOS_ALIBI) {
          // from 2^90 on a row has its own key alone; times a distance it
          // stays finite
          sl = __ldg(p.bias + hq) * kLog2e;
          if (fabsf(sl) > 0x1p90f) sl = copysignf(0x1p90f, sl);
        }
        if (p.mode == RELPOS_T5) far = to_log2(__ldg(p.bias + (p.t5.slots - 1) * p.Hq + hq));
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {  // from the lanes of row 8 n + 2 t + c
        const int from = 4 * (2 * t + c);
        qs[n][c] = __shfl_sync(0xffffffffu, up, from);
        vis[n][c] = __shfl_sync(0xffffffffu, last, from);
        add[n][c] = __shfl_sync(0xffffffffu, far, from);
        slope[n][c] = __shfl_sync(0xffffffffu, sl, from);
      }
    }
    const int vis_first = len - p.Lq + row0 / p.G;  // last key that every row sees
    // a constant bias beside which products lose bits (a mask of -1e9, the
    // type's lowest value): every tile then has to lose them alike
    bool odd = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) odd |= !(fabsf(add[n][0]) <= 4096.f && fabsf(add[n][1]) <= 4096.f);
    odd = __any_sync(0xffffffffu, odd);
    [[maybe_unused]] float v_inv = 0.f;  // 1 / v_unit, 0 before the first tile
    float off[NQ][2], l_run[NQ][2], o[NQ][KS][4];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      off[n][0] = off[n][1] = 0.f;
      l_run[n][0] = l_run[n][1] = 0.f;
#pragma unroll
      for (int j = 0; j < KS; ++j) o[n][j][0] = o[n][j][1] = o[n][j][2] = o[n][j][3] = 0.f;
    }

    bool first = true;  // no tile of the unit yet
    // this warp's tiles of the unit: those with y mod 4 = warp
    for (int y = x + ((warp - x) & (kPdWarps - 1)); y < xe; y += kPdWarps) {
      cp_async_wait<STAGES - 2>();
      __syncwarp();
      produce(stage == 0 ? STAGES - 1 : stage - 1);
      const uint32_t ks = ring + stage * S::kStageBytes, vs = ks + S::kTileBytes;
      const bool skip = missing >> stage & 1;
      if (++stage == STAGES) stage = 0;
      if (skip) continue;
      const int key0 = (cc.t + y - x) * KT;

      // scores: lane (g, t) holds keys 16 i + g (+ 8) and rows 8 n + 2 t, + 1
      float sc[NQ][MT][4];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) sc[n][i][0] = sc[n][i][1] = sc[n][i][2] = sc[n][i][3] = 0.f;
#pragma unroll
        for (int j = 0; j < KC; ++j) {
          const uint4 u = lds128(ks + k_off[j] + 16 * i * S::kRowBytes);
          const uint4 w = lds128(ks + k_off[j] + (16 * i + 8) * S::kRowBytes);
          const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {w.x, w.y, w.z, w.w};
          if constexpr (FP8) {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              const uint32_t f[4] = {half2_lo(a[s]), half2_lo(b[s]), half2_hi(a[s]), half2_hi(b[s])};
#pragma unroll
              for (int n = 0; n < NQ; ++n) mma16816<true>(sc[n][i], f, q[n][4 * j + s][0], q[n][4 * j + s][1]);
            }
          } else {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const uint32_t f[4] = {a[2 * s], b[2 * s], a[2 * s + 1], b[2 * s + 1]};
#pragma unroll
              for (int n = 0; n < NQ; ++n) mma16816<false>(sc[n][i], f, q[n][2 * j + s][0], q[n][2 * j + s][1]);
            }
          }
        }
      }
      float k_scale = 1.f;
      [[maybe_unused]] float ratio = 1.f;
      [[maybe_unused]] auto outside = [&] { return !(fabsf(ratio) >= kPdRatioLow && fabsf(ratio) <= kPdRatioHigh); };
      if constexpr (FP8) {
        k_scale = lds32f(vs + S::kTileBytes);
        const float v_scale = lds32f(vs + S::kTileBytes + 4);
        ratio = v_scale * v_inv;
        if (outside()) {  // NaN too
          const float size = fabsf(v_scale), v_unit = v_inv == 0.f ? 0.f : inverse_pow2(v_inv);
          const float unit = size > kPdUnitHigh   ? 2.f * kPdUnitHigh
                             : size >= kPdUnitLow ? __uint_as_float(__float_as_uint(size) & 0x7f800000u)
                                                  : fmaxf(v_unit, kPdUnitLow);
          if (v_unit <= kPdUnitHigh && unit != v_unit) {
            v_inv = inverse_pow2(unit);
            const float down = v_unit * v_inv;
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int j = 0; j < KS; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[n][j][e] *= down;
            ratio = v_scale * v_inv;
          }
        }
      }
      const bool edge = key0 + KT - 1 > vis_first;  // some row does not see every key
      const bool near = p.mode == RELPOS_T5 && vis_first - (key0 + KT - 1) < p.t5_R;
      // The common tile: every row sees it, its biases are linear in the key's
      // position, and no logit passes its row's offset by too much.
      float z[NQ][MT][4];
      bool above = edge || near || odd || first;
      if (!above) {
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float cs = qs[n][c] * k_scale;
            const float base =
                fmaf(-slope[n][c], static_cast<float>(vis[n][c] - key0 - g), add[n][c] - off[n][c]);
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                z[n][i][2 * e + c] = fmaf(sc[n][i][2 * e + c], cs, fmaf(slope[n][c], 16 * i + 8 * e, base));
          }
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) above |= z[n][i][e] > kPdMost;
        }
        above = __any_sync(0xffffffffu, above);
      }
      if (above) {
        float slow[NQ * MT * 4];  // biases, where a table of them does not fit
        if (near && !lut) {
#pragma unroll 1
          for (int i = 0; i < NQ * MT * 4; ++i) {
            const int r = row0 + 8 * (i / (4 * MT)) + 2 * t + i / (2 * MT) % 2, qi = r / p.G;
            const int back = len - p.Lq + qi - (key0 + 16 * (i / 2 % MT) + 8 * (i % 2) + g);
            const int bucket = t5_bucket_dev(-min(max(back, 0), p.t5_R), p.t5);
            slow[i] = to_log2(__ldg(p.bias + bucket * p.Hq + h * p.G + r - qi * p.G));
          }
        }
        // logit of row 8 n + 2 t + c and key 16 i + 8 e + g, less its row's offset
        auto logits = [&](float (&z)[NQ][MT][4]) {
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float cs = qs[n][c] * k_scale;
              const int back0 = vis[n][c] - key0 - g;  // to key 16 i + 8 e: less 16 i + 8 e
              if (near && lut) {
                const float* biases = out_s + (row0 + 8 * n + 2 * t + c) % p.G * lut_len;
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    z[n][i][2 * e + c] = fmaf(sc[n][i][2 * e + c], cs,
                                              biases[min(max(back0 - 16 * i - 8 * e, 0), p.t5_R)]) - off[n][c];
              } else if (near) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    z[n][i][2 * e + c] = fmaf(sc[n][i][2 * e + c], cs, slow[((n * 2 + c) * MT + i) * 2 + e]) - off[n][c];
              } else if (p.mode != RELPOS_ALIBI) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    z[n][i][2 * e + c] = fmaf(sc[n][i][2 * e + c], cs, add[n][c]) - off[n][c];
              } else {
                const float back_f = static_cast<float>(back0);
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    z[n][i][2 * e + c] =
                        fmaf(sc[n][i][2 * e + c], cs, fmaf(-slope[n][c], back_f - (16 * i + 8 * e), -off[n][c]));
              }
              if (edge) {
#pragma unroll
                for (int i = 0; i < MT; ++i)
#pragma unroll
                  for (int e = 0; e < 2; ++e)
                    if (back0 < 16 * i + 8 * e) z[n][i][2 * e + c] = -INFINITY;
              }
            }
          }
        };
        // Offsets move by the logits themselves (less an offset far below them
        // these have no bits left): the rows concerned take offset 0 and the
        // logits are formed anew. At the warp's first tile of the unit that is
        // where they stand.
        float was[NQ][2];
        bool moves[NQ][2], settle = first;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            was[n][c] = -FLT_MAX;
            moves[n][c] = true;
          }
        }
        auto largest = [&](int n, int c) {
          float top = -INFINITY;
#pragma unroll
          for (int i = 0; i < MT; ++i) top = fmaxf(top, fmaxf(z[n][i][c], z[n][i][2 + c]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
          return fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
        };
        while (true) {
          logits(z);
          if (settle) break;
          above = false;
#pragma unroll
          for (int n = 0; n < NQ; ++n)
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) above |= z[n][i][e] > kPdMost;
          if (!__any_sync(0xffffffffu, above)) break;
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              was[n][c] = off[n][c];
              moves[n][c] = largest(n, c) > kPdMost;
              if (moves[n][c]) off[n][c] = 0.f;
            }
          }
          settle = true;
        }
        if (settle) {
#pragma unroll
          for (int n = 0; n < NQ; ++n) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float top = fmaxf(largest(n, c) - kPdShift, -FLT_MAX);  // a row may see no key
              if (moves[n][c]) {
                off[n][c] = top;
                const float down = ex2_approx(was[n][c] - top);
                l_run[n][c] *= down;
#pragma unroll
                for (int i = 0; i < MT; ++i) z[n][i][c] -= top, z[n][i][2 + c] -= top;
#pragma unroll
                for (int j = 0; j < KS; ++j) o[n][j][c] *= down, o[n][j][2 + c] *= down;
              }
            }
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sc[n][i][e] = ex2_approx(z[n][i][e]);
            l_run[n][e & 1] += sc[n][i][e];
          }
        }
      }

      first = false;

      // o^T += v^T p^T. SLOW: each product by itself, times the page's ratio,
      // for the rows and the keys of one query position or (`all`) of every one.
      auto add_values = [&](auto slow_path, int last, bool all) {
        constexpr bool SLOW = decltype(slow_path)::value;
        [[maybe_unused]] const float factor = SLOW ? 1.f : ratio;
        uint32_t ph[NQ][MT][2];
        [[maybe_unused]] uint32_t pl[FP8 ? 1 : NQ][MT][2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          const bool mine[2] = {!SLOW || all || vis[n][0] == last, !SLOW || all || vis[n][1] == last};
#pragma unroll
          for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float a = mine[0] ? sc[n][i][2 * e] : 0.f, c = mine[1] ? sc[n][i][2 * e + 1] : 0.f;
              if constexpr (FP8) {
                // 11 bits of a weight: its rounding (2^-12) is far below the
                // output's (2^-9)
                ph[n][i][e] = transpose8(pack_half2(a * factor, c * factor));
              } else {
                // bf16 alone would round the weights as coarsely as the
                // output: a second part carries the next 8 bits
                const uint32_t hi = pack_bf2(a, c);
                ph[n][i][e] = transpose8(hi);
                pl[n][i][e] =
                    transpose8(pack_bf2(a - __uint_as_float(hi << 16), c - __uint_as_float(hi & 0xffff0000u)));
              }
            }
          }
        }
        // value rows of the lane: 16 i + 8 e + 2 t + o
        auto row_words = [&](int i, int e, int oo, int half, uint32_t (&w)[4]) {
          const uint32_t a = vs + v_off[oo] + (16 * i + 8 * e) * S::kRowBytes + half * 128;
          if constexpr (FP8 && D == 64) {
            const uint2 u = lds64(a);
            w[0] = u.x, w[1] = u.y, w[2] = w[3] = 0;
          } else {
            const uint4 u = lds128(a);
            w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
          }
          if (SLOW && !all && key0 + 16 * i + 8 * e + 2 * t + oo > last) w[0] = w[1] = w[2] = w[3] = 0;
        };
        if constexpr (FP8) {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
            uint32_t r[2][2][4];
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
              for (int oo = 0; oo < 2; ++oo) row_words(i, e, oo, 0, r[e][oo]);
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {  // words of 4 dims that a lane holds of a row
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t a = __byte_perm(r[0][0][w], r[0][1][w], j ? 0x7362 : 0x5140);
                const uint32_t b = __byte_perm(r[1][0][w], r[1][1][w], j ? 0x7362 : 0x5140);
                const uint32_t f[4] = {half2_lo(a), half2_hi(a), half2_lo(b), half2_hi(b)};
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                  float(&d)[4] = o[n][2 * w + j];
                  if constexpr (SLOW) {
                    float y[4] = {0.f, 0.f, 0.f, 0.f};
                    mma16816<true>(y, f, ph[n][i][0], ph[n][i][1]);
                    // d = 128: the ratio anew, since held through the loop it
                    // makes 8 rows' variant spill (3 % longer)
                    auto times = [&] { return D == 128 && NQ == 1 ? lds32f(vs + S::kTileBytes + 4) * v_inv : ratio; };
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                      if (all || vis[n][e & 1] == last) d[e] = fmaf(y[e], times(), d[e]);
                  } else {
                    mma16816<true>(d, f, ph[n][i][0], ph[n][i][1]);
                  }
                }
              }
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
              uint32_t r[2][2][4];
#pragma unroll
              for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int oo = 0; oo < 2; ++oo) row_words(i, e, oo, half, r[e][oo]);
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t f[4] = {
                    __byte_perm(r[0][0][w], r[0][1][w], 0x5410), __byte_perm(r[0][0][w], r[0][1][w], 0x7632),
                    __byte_perm(r[1][0][w], r[1][1][w], 0x5410), __byte_perm(r[1][0][w], r[1][1][w], 0x7632)};
#pragma unroll
                for (int n = 0; n < NQ; ++n) {
                  float(&d)[4] = o[n][4 * half + w];
                  const float was[4] = {d[0], d[1], d[2], d[3]};
                  mma16816<false>(d, f, ph[n][i][0], ph[n][i][1]);
                  mma16816<false>(d, f, pl[n][i][0], pl[n][i][1]);
                  if (SLOW) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) d[e] = vis[n][e & 1] == last ? d[e] : was[e];
                  }
                }
              }
            }
          }
        }
      };
      // Where rows of one tile see different keys and a value that some of
      // them do not see, or the page's scale, is not finite (0 times it is
      // NaN), the rows of each query position that see a key go alone, with
      // the values that they do not see as zeros.
      bool foul = false;
      if (edge && p.Lq > 1) {
        if constexpr (FP8) foul = !(fabsf(ratio) <= FLT_MAX);
#pragma unroll
        for (int i = lane; i < KT * S::kChunks; i += 32) {
          const uint4 u = lds128(vs + 16 * i);
          if (key0 + i / S::kChunks > vis_first) {
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int m = 0; m < 4; ++m)
              foul |= FP8 ? __vcmpeq4(w[m] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0
                          : __vcmpeq2(w[m] & 0x7f807f80u, 0x7f807f80u) != 0;
          }
        }
        foul = __any_sync(0xffffffffu, foul);
      }
      if (foul || (FP8 && outside())) {
#pragma unroll 1
        for (int i = foul ? 0 : p.Lq - 1; i < p.Lq; ++i)
          if (len - p.Lq + i >= key0) add_values(std::true_type{}, len - p.Lq + i, !foul);
      } else {
        add_values(std::false_type{}, 0, true);
      }
    }

    // ---- the four warps' parts of the unit, joined in a fixed order: 2 into 0
    // and 3 into 1, then 1 into 0
    const int had = xe - x;  // tiles of the unit in this block
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (first) off[n][c] = -FLT_MAX;  // a warp without tiles
        l_run[n][c] += __shfl_xor_sync(0xffffffffu, l_run[n][c], 4);
        l_run[n][c] += __shfl_xor_sync(0xffffffffu, l_run[n][c], 8);
        l_run[n][c] += __shfl_xor_sync(0xffffffffu, l_run[n][c], 16);
        if (g == 0) {
          float* ml = ml_s + (warp * S::kRows + 8 * n + 2 * t + c) * 2;
          ml[0] = off[n][c];
          ml[1] = l_run[n][c];
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float2* ml = reinterpret_cast<const float2*>(ml_s) + 8 * n + 2 * t + c;
        float top = -FLT_MAX;
#pragma unroll
        for (int w = 0; w < kPdWarps; ++w) top = fmaxf(top, ml[w * S::kRows].x);
        const float down = ex2_approx(off[n][c] - top) * (FP8 && v_inv != 0.f ? inverse_pow2(v_inv) : 1.f);
#pragma unroll
        for (int j = 0; j < KS; ++j) o[n][j][c] *= down, o[n][j][2 + c] *= down;
      }
    }
    // a lane's values of a row: 16 bytes at a time, lane after lane
    auto give = [&](float* to) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (8 * n + 2 * t + c < rows)
#pragma unroll
            for (int j = 0; j < KS; j += 2)
              reinterpret_cast<float4*>(to)[((n * 2 + c) * (KS / 2) + j / 2) * 32 + lane] =
                  make_float4(o[n][j][c], o[n][j][2 + c], o[n][j + 1][c], o[n][j + 1][2 + c]);
    };
    auto take = [&](const float* from) {
#pragma unroll
      for (int n = 0; n < NQ; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c)
          if (8 * n + 2 * t + c < rows)
#pragma unroll
            for (int j = 0; j < KS; j += 2) {
              const float4 v = reinterpret_cast<const float4*>(from)[((n * 2 + c) * (KS / 2) + j / 2) * 32 + lane];
              o[n][j][c] += v.x, o[n][j][2 + c] += v.y, o[n][j + 1][c] += v.z, o[n][j + 1][2 + c] += v.w;
            }
    };
    if (warp >= 2) give(out_s + (warp - 2) * S::kRows * D);
    __syncthreads();
    if (warp < 2) take(out_s + warp * S::kRows * D);
    if (warp == 1) give(out_s + S::kRows * D);
    __syncthreads();
    if (warp == 0) {  // and the rows in order
      take(out_s + S::kRows * D);
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (8 * n + 2 * t + c >= rows) continue;
          float4* row = reinterpret_cast<float4*>(out_s + (8 * n + 2 * t + c) * D);
#pragma unroll
          for (int j = 0; j < KS; j += 2) {  // the lane's dims as the values were read
            const int dim = FP8 ? 2 * KS * g + 2 * j : (j / 4) * 64 + 8 * g + 2 * (j % 4);
            row[dim / 4] = make_float4(o[n][j][c], o[n][j][2 + c], o[n][j + 1][c], o[n][j + 1][2 + c]);
          }
        }
      }
    }
    __syncthreads();
    const bool whole = cc.t == 0 && had == cc.nt;
    const int slot = 2 * blockIdx.x + (cc.t == 0 ? 1 : 0);
    if (!whole && threadIdx.x == 0) {  // the same thread wrote the zeros before
      const int c0 = (at + kPdUnitCost) / size;
      p.ends[slot] = make_int4(c0, (at + kPdUnitCost + cc.nt - 1) / size - c0 + 1, cc.b, cc.u);
    }
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (D / 8); i += kPdThreads) {
      const int r = i / (D / 8), dim = 8 * (i % (D / 8));
      const float2* ml = reinterpret_cast<const float2*>(ml_s) + r;
      float top = -FLT_MAX, sum = 0.f;
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w) top = fmaxf(top, ml[w * S::kRows].x);
#pragma unroll
      for (int w = 0; w < kPdWarps; ++w) sum = fmaf(ex2_approx(ml[w * S::kRows].x - top), ml[w * S::kRows].y, sum);
      const float4* v = reinterpret_cast<const float4*>(out_s + r * D + dim);
      float4 a = v[0], b = v[1];
      if (whole) {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        const uint32_t w[4] = {pack_bf2(a.x * inv, a.y * inv), pack_bf2(a.z * inv, a.w * inv),
                               pack_bf2(b.x * inv, b.y * inv), pack_bf2(b.z * inv, b.w * inv)};
        const int qi = (row0 + r) / p.G;
        const int hq = h * p.G + (row0 + r) - qi * p.G;
        __nv_bfloat16* op = p.out + cc.b * p.o_batch + hq * p.o_head + qi * p.o_row + dim;
        if (p.o_vec) {
          *reinterpret_cast<uint4*>(op) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            op[2 * e] = __ushort_as_bfloat16(static_cast<unsigned short>(w[e]));
            op[2 * e + 1] = __ushort_as_bfloat16(static_cast<unsigned short>(w[e] >> 16));
          }
        }
      } else {
        const size_t at = static_cast<size_t>(slot) * S::kRows + r;
        float4* to = reinterpret_cast<float4*>(p.part_o + at * D + dim);
        to[0] = a;
        to[1] = b;
        if (dim == 0) *reinterpret_cast<float2*>(p.part_ml + 2 * at) = make_float2(top, sum);
      }
    }
    __syncthreads();  // ml_s and the buffers are free again
    at += kPdUnitCost + cc.nt;
    cc.forward<KT>(p, had);
    x = xe;
  }
  cp_async_wait<0>();
}

// Joins the parts of the units that several blocks shared, in block order, and
// writes the zeros of empty sequences. Each of the k blocks of such a unit takes
// a k-th of its output, so that every block reads about one unit's worth of
// parts for either end of its share, however many blocks a unit has; half of
// its threads for each end. What a slot holds the decode kernel has noted, so
// that nothing is searched for here: these blocks mostly start when that
// kernel's leave their SM.
template <int D>
__global__ void __launch_bounds__(kPdThreads) relpos_paged_combine_kernel(const __grid_constant__ PagedDecodeParams p) {
  griddep_launch_dependents();
  griddep_wait();
  constexpr int kHalf = kPdThreads / 2;
  const int end = threadIdx.x / kHalf, tid = threadIdx.x % kHalf;
  const int4 what = __ldcg(p.ends + 2 * blockIdx.x + end);
  const int c0 = what.x, k = what.y, b = what.z, u = what.w;
  for (int i = blockIdx.x; i < p.B; i += gridDim.x) {
    if (seq_len(p, i) > 0) continue;
    if (threadIdx.x == 0) report_length(p, i);
    for (int r = threadIdx.x / 32; r < p.Hq * p.Lq; r += kPdWarps)
      for (int j = threadIdx.x % 32; j < D; j += 32)
        p.out[i * p.o_batch + r / p.Lq * p.o_head + r % p.Lq * p.o_row + j] = __float2bfloat16_rn(0.f);
  }
  if (k == 0) return;
  const int h = u / p.rt, row0 = (u - h * p.rt) * p.rows, rows = min(p.G * p.Lq - row0, p.rows);
  // this block's columns (4 dims of a row) of the unit's rows * D / 4
  const int me = blockIdx.x - c0, cols = rows * (D / 4);
  const int first = cols * me / k, count = cols * (me + 1) / k - first;
  int lanes = 1;  // that share a column, a power of two
  while (lanes < 32 && lanes < k && 2 * lanes * count <= kHalf) lanes *= 2;
  const int part = tid & (lanes - 1);
  for (int i0 = 0; i0 < count; i0 += kHalf / lanes) {  // whole warps take part
    const int i = i0 + tid / lanes;
    const int col = first + min(i, count - 1), r = col / (D / 4), d4 = col % (D / 4);
    float m = -FLT_MAX, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    auto join = [&](float m2, float l2, const float4& v) {
      const float top = fmaxf(m, m2), w = ex2_approx(m2 - top), down = ex2_approx(m - top);
      m = top;
      l = fmaf(w, l2, l * down);
      acc.x = fmaf(w, v.x, acc.x * down);
      acc.y = fmaf(w, v.y, acc.y * down);
      acc.z = fmaf(w, v.z, acc.z * down);
      acc.w = fmaf(w, v.w, acc.w * down);
    };
#pragma unroll 4
    for (int j = part; j < k; j += lanes) {
      // the unit begins in its first block's second slot
      const size_t at = (2 * static_cast<size_t>(c0 + j) + (j == 0 ? 1 : 0)) * p.rows + r;
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(p.part_ml + 2 * at));
      join(ml.x, ml.y, __ldcg(reinterpret_cast<const float4*>(p.part_o + at * D + 4 * d4)));
    }
    for (int o = 1; o < lanes; o *= 2) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
      const float4 v = make_float4(__shfl_xor_sync(0xffffffffu, acc.x, o), __shfl_xor_sync(0xffffffffu, acc.y, o),
                                   __shfl_xor_sync(0xffffffffu, acc.z, o), __shfl_xor_sync(0xffffffffu, acc.w, o));
      join(m2, l2, v);
    }
    if (i < count && part == 0) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int qi = (row0 + r) / p.G, hq = h * p.G + (row0 + r) - qi * p.G;
      __nv_bfloat16* op = p.out + b * p.o_batch + hq * p.o_head + qi * p.o_row + 4 * d4;
      const uint32_t w[2] = {pack_bf2(acc.x * inv, acc.y * inv), pack_bf2(acc.z * inv, acc.w * inv)};
      if (p.o_vec) {
        *reinterpret_cast<uint2*>(op) = make_uint2(w[0], w[1]);
      } else {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          op[2 * e] = __ushort_as_bfloat16(static_cast<unsigned short>(w[e]));
          op[2 * e + 1] = __ushort_as_bfloat16(static_cast<unsigned short>(w[e] >> 16));
        }
      }
    }
  }
}

template <int D, bool FP8, int NQ, int KT, int STAGES>
PagedDecodeVariant paged_decode_variant() {
  return {relpos_paged_decode_kernel<D, FP8, NQ, KT, STAGES>, relpos_paged_combine_kernel<D>, KT,
          Shape<D, FP8, NQ, KT, STAGES>::kSmem};
}

}  // namespace
}  // namespace relpos
