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
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/relpos_attn.h"
#include "paged.cuh"
#include "ptx.cuh"
#include "relpos_internal.h"
#include "serving_internal.h"
#include "rotary.cuh"

namespace relpos {
namespace {

constexpr int kAppMaxGroup = 64;  // heads of a block at most

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
  int exp_k[2], exp_v[2]; // scale_exponents of keys and values
  int* status;
};

// The scale of a largest magnitude (bf16 bits without the sign): the smallest
// power of two s with magnitude * reach <= 448 s. For a magnitude m 2^k with
// 7 bits after the point its exponent is k + ex[0], one more from the
// mantissa ex[1] on; clamped to -120 .. 120.
RP_DEVI float scale_for(uint32_t bits, const int (&ex)[2]) {
  int e = static_cast<int>(bits >> 7) - 127 + ex[0] + (static_cast<int>(bits & 127u) >= ex[1]);
  e = min(120, max(-120, e));
  return __int_as_float((e + 127) << 23);
}

RP_DEVI uint32_t e4m3x2(float lo, float hi) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

// Sine and cosine of `turn` 2^-64ths of a turn in units of 2^-62, off by at most 4
// of them: the Taylor series of the distance to the nearest quarter turn (at most
// pi / 4; the first terms left out are below 2^-63), in units of 2^-64.
RP_DEVI void sincos_fixed(unsigned long long turn, long long& s, long long& c) {
  const unsigned quarter = static_cast<unsigned>((turn + (1ull << 61)) >> 62);
  const long long rest = static_cast<long long>(turn - (static_cast<unsigned long long>(quarter) << 62));
  const unsigned long long far = rest < 0 ? -static_cast<unsigned long long>(rest) : rest;
  const unsigned long long x = __umul64hi(far << 2, 0xc90fdaa22168c234ull) << 1;  // times pi / 4 in 2^-64
  const unsigned long long z = __umul64hi(x, x);
  // 1 / 3! - z / 5! + ... - z^7 / 17! and 1 / 4! - z / 6! + ... - z^7 / 18!
  constexpr unsigned long long kSin[8] = {0x2aaaaaaaaaaaaaabull, 0x222222222222222ull, 0xd00d00d00d00dull, 0x2e3bc74aad8eull,
                                          0x6b99159fd5ull, 0xb092309dull, 0xd73f9full, 0xca96ull};
  constexpr unsigned long long kCos[8] = {0xaaaaaaaaaaaaaabull, 0x5b05b05b05b05bull, 0x1a01a01a01a02ull, 0x49f93edde28ull,
                                          0x8f76c77fcull, 0xc9cba54ull, 0xd73faull, 0xb41ull};
  unsigned long long p = kSin[7], q = kCos[7];
#pragma unroll
  for (int i = 6; i >= 0; --i) {
    p = kSin[i] - __umul64hi(z, p);
    q = kCos[i] - __umul64hi(z, q);
  }
  s = static_cast<long long>((x - __umul64hi(__umul64hi(z, x), p)) >> 2);
  c = static_cast<long long>((1ull << 62) - (z >> 3) + (__umul64hi(__umul64hi(z, z), q) >> 2));
  if (rest < 0) s = -s;
  if (quarter & 1) {
    const long long was = s;
    s = c;
    c = -was;
  }
  if (quarter & 2) s = -s, c = -c;
}

// m 2^e, as u with the top bit set times 2^e
struct Scaled {
  unsigned long long u;
  int e;
  RP_DEVI void normalize() {
    const int n = __clzll(u) & 63;
    u <<= n, e -= n;
  }
  RP_DEVI void times(unsigned long long by, int by_e) {  // `by` with its top bit set too
    u = __umul64hi(u, by), e += by_e + 64;
    normalize();
  }
};

// The pair's codes from the rotation in 64-bit integers (y1's in the low byte).
// Taken where the fp32 rotation cannot tell on which side of a border of the e4m3
// grid its result lies, about once in 3 x 10^4 values. Each product of an 8-bit
// mantissa and a sine or cosine of 2^-54 is exact; their sum is multiplied by inv,
// a power of two, (DIVIDED) divided by a 24-bit mantissa, divisor / 2^23, and cut to
// 24 bits, the last made odd where that dropped anything, so that the rounding to
// a code sees on which side of a border the value lies. Fixed point since 64-bit
// floating point is slow here: a token's step took 6.2 us with it against 5.5,
// prompts 21.6 against 20.3.
template <bool DIVIDED>
__device__ __noinline__ uint32_t rotated_codes_exact(float x1, float x2, unsigned long long turns, int pos,
                                                     double amplitude, float inv, uint32_t divisor = 0) {
  long long s, c;
  sincos_fixed(turns * static_cast<unsigned long long>(static_cast<long long>(pos)), s, c);
  const uint32_t b1 = __float_as_uint(x1), b2 = __float_as_uint(x2);
  const int f1 = b1 >> 23 & 255, f2 = b2 >> 23 & 255;
  const int e1 = max(f1, 1), e2 = max(f2, 1), top = max(e1, e2);
  long long m1 = (b1 >> 16 & 127) | (f1 ? 128 : 0), m2 = (b2 >> 16 & 127) | (f2 ? 128 : 0);
  if (b1 >> 31) m1 = -m1;
  if (b2 >> 31) m2 = -m2;
  const int d1 = min(top - e1, 63), d2 = min(top - e2, 63);
  s >>= 8, c >>= 8;
  const long long y[2] = {(m1 * c >> d1) - (m2 * s >> d2), (m1 * s >> d1) + (m2 * c >> d2)};
  const unsigned long long amp = __double_as_longlong(amplitude);
  const uint32_t inv_bits = __float_as_uint(inv);
  Scaled by = {inv_bits & 0x7fffffu, max(static_cast<int>(inv_bits >> 23), 1) - 150};
  if (inv_bits >> 23) by.u |= 1u << 23;
  const bool plain = f1 < 255 && f2 < 255 && by.u != 0;
  by.normalize();
  const float sf = static_cast<float>(s) * 0x1p-54f, cf = static_cast<float>(c) * 0x1p-54f;
  uint32_t code = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float f;
    if (plain && y[i] != 0) {
      Scaled v = {static_cast<unsigned long long>(y[i] < 0 ? -y[i] : y[i]), top - 134 - 54};
      v.normalize();
      v.times(amp << 11 | 1ull << 63, static_cast<int>(amp >> 52) - 1023 - 63);
      v.times(by.u, by.e);
      if constexpr (DIVIDED) {
        const unsigned long long whole = v.u / divisor;  // 40 bits or more
        v.u = whole | (whole * divisor != v.u), v.e += 23;
        v.normalize();
      }
      const uint32_t cut = static_cast<uint32_t>(v.u >> 40) | ((v.u & ((1ull << 40) - 1)) != 0);
      // what is below half of the smallest code may be so by more or less
      f = static_cast<float>(cut) * __int_as_float((min(max(v.e + 40, -120), 100) + 127) << 23);
      if (y[i] < 0) f = -f;
    } else {  // zeros, infinities and NaN
      f = (i ? fmaf(x1, sf, x2 * cf) : fmaf(x1, cf, x2 * -sf)) * inv;
    }
    code |= (e4m3x2(f, 0.f) & 0xffu) << 8 * i;
  }
  return code;
}

// The codes of a page that was quantised elsewhere, with a scale that is no power
// of two, and keeps it: the block's tokens t_lo .. t_hi - 1 of the heads that are
// so, divided by it, over the codes by its rounded inverse. After a block's other
// work, and out of line, so that it costs the others no registers.
template <bool INTERLEAVED>
__device__ __noinline__ void divided_codes(const AppendParams& p, const float (&had)[2][kAppMaxGroup],
                                           const int (&amax)[2][kAppMaxGroup], int nheads, size_t page_rows, int page0,
                                           int t_lo, int t_hi, const __nv_bfloat16* K, const __nv_bfloat16* V) {
  const int d = p.cache.d, pairs = p.plan.rot_dim >> 1;
  for (int i = 0; i < 2 * nheads; ++i) {
    const int w = i >= nheads, h = i - w * nheads;
    const float scale = had[w][h];
    if (is_pow2(scale) || !(scale_for(amax[w][h], w ? p.exp_v : p.exp_k) <= scale)) continue;
    const uint32_t bits = __float_as_uint(scale);
    const float inv = 1.f / __uint_as_float(bits & 0x7f800000u);  // a power of two
    const __nv_bfloat16* x = w ? V + h * p.v_head : K + h * p.k_head;
    const long long step = w ? p.v_row : p.k_row;
    uint8_t* codes = static_cast<uint8_t*>(w ? p.cache.v : p.cache.k) + ((page_rows + h) << p.log_page) * d;
    const int turned = w ? 0 : pairs, units = d - turned;  // of a token: pairs, then single values
    for (int j = threadIdx.x; j < (t_hi - t_lo) * units; j += blockDim.x) {
      const int slot = t_lo + j / units, m = j % units;
      const __nv_bfloat16* row = x + slot * step;
      uint8_t* to = codes + slot * d;
      if (m < turned) {
        const int e1 = INTERLEAVED ? 2 * m : m, e2 = INTERLEAVED ? e1 + 1 : e1 + pairs;
        const uint32_t both =
            rotated_codes_exact<true>(__bfloat162float(row[e1]), __bfloat162float(row[e2]), p.plan.turns[m],
                                      page0 + slot, p.plan.amplitude, inv, (bits & 0x7fffffu) | 0x800000u);
        to[e1] = static_cast<uint8_t>(both);
        to[e2] = static_cast<uint8_t>(both >> 8);
      } else {
        to[m + turned] = code_over(__bfloat162float(row[m + turned]), scale);
      }
    }
  }
}

// A block takes one page that gets new tokens and `group` heads of it. Its
// items are the heads' new tokens in units of 16 elements, a thread holding
// UNITS of them (keys and values, all loads in flight at once) in registers,
// so that a page's largest value and its codes come from one read; heads
// follow one another, as many at a time as the block has threads for, the next
// ones' loads ahead of the present ones' arithmetic. Sines and cosines are
// formed once for the block, in shared memory: [4][slots * units] float4, the
// two sines, then the two cosines, of pairs 2 j and 2 j + 1 of a unit in plane j.
//
// 8531 tokens of 16 heads, d = 64, e4m3: 20.8 us for 52 MB. The launch is one wave
// of 408 blocks with work, of 6, 6 and 4 heads, three to an SM at most, whose
// loads are uneven; in it issue is 59 % busy (640 instructions for a warp's 32 x 16
// keys and values) with a third of the warps resident. The test for borders is 1 us
// of it, the decisions next to one, long chains in single lanes, 2.4. A token a
// sequence: 5.4 us, its chain of loads (lengths, table, rows, scales). Decisions noted down and taken together at the block's end: 0.2 us
// less for the prompts, 0.4 more for a token. Three blocks of 256 threads share an
// SM for e4m3 (80 registers); with the decisions still in floating point the
// prompts took 22.2 us so, 22.6 with two (128) and 32 with four (64, which spills
// 152 bytes). 16-bit caches, with no codes to decide, go with two: 4.7 us for
// 4 x 1001 tokens of 8 heads, d = 128, against 5.8 with three and 6.1 with four.
template <bool FP8, bool INTERLEAVED, int THREADS, int UNITS>
__global__ void __launch_bounds__(THREADS, UNITS == 1 ? (FP8 ? 768 : 512) / THREADS : 1)
    relpos_paged_append_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float4 turn_s[];
  __shared__ int amax_s[2][kAppMaxGroup];
  __shared__ float had_s[2][kAppMaxGroup];      // scales so far (0 for a page taken anew)
  __shared__ float had_inv_s[2][kAppMaxGroup];  // and 1 over them
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
  const int page = 1 << p.log_page, page0 = pg << p.log_page;
  const int t_lo = max(start - page0, 0), t_hi = min(len - page0, page);  // new slots of the page
  const int h0 = blockIdx.y * p.group;
  const int nheads = min(p.group, p.cache.H - h0);
  const int d = p.cache.d;
  const int rot_units = p.plan.rot_dim >> 4;
  const size_t page_rows = static_cast<size_t>(page_id) * p.cache.H + h0;

  // items of a head: its new tokens, rounded up to a power of two, by units
  const int log_tok = 32 - __clz(t_hi - t_lo - 1);
  const int log_items = log_tok + p.log_units;
  constexpr int kSpan = THREADS * UNITS;
  const int step_heads = max(1, kSpan >> log_items);
  // unit i of the thread: item tid + i * THREADS of the block's span
  auto place = [&](int i, int& hs, int& slot, int& unit, int& d1, int& d2) {
    const int item = i * THREADS + tid;
    hs = item >> log_items;
    slot = t_lo + ((item >> p.log_units) & ((1 << log_tok) - 1));
    unit = item & ((1 << p.log_units) - 1);
    if (unit < rot_units && !INTERLEAVED) {  // 8 pairs of the rotation's halves
      d1 = unit * 8;
      d2 = (p.plan.rot_dim >> 1) + d1;
    } else {  // 16 neighbours
      d1 = unit * 16;
      d2 = d1 + 8;
    }
  };
  const long long k_base = (p.cu ? (row0 - static_cast<long long>(start - page0)) * p.k_row
                                 : b * p.k_batch - (start - page0) * p.k_row) + h0 * p.k_head;
  const long long v_base = (p.cu ? (row0 - static_cast<long long>(start - page0)) * p.v_row
                                 : b * p.v_batch - (start - page0) * p.v_row) + h0 * p.v_head;
  uint4 kr[UNITS][2], vr[UNITS][2];
  const __nv_bfloat16 *kp[UNITS], *vp[UNITS];  // the next head's row of each unit
#pragma unroll
  for (int i = 0; i < UNITS; ++i) {
    int hs, slot, unit, d1, d2;
    place(i, hs, slot, unit, d1, d2);
    kp[i] = p.K + k_base + slot * p.k_row + hs * p.k_head + d1;
    vp[i] = p.V + v_base + slot * p.v_row + hs * p.v_head + d1;
  }
  auto load = [&](int head) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      int hs, slot, unit, d1, d2;
      place(i, hs, slot, unit, d1, d2);
      kr[i][0] = kr[i][1] = vr[i][0] = vr[i][1] = make_uint4(0, 0, 0, 0);
      if (hs < step_heads && head + hs < nheads && slot < t_hi) {
        if (p.vec) {
          kr[i][0] = *reinterpret_cast<const uint4*>(kp[i]);
          kr[i][1] = *reinterpret_cast<const uint4*>(kp[i] + d2 - d1);
          vr[i][0] = *reinterpret_cast<const uint4*>(vp[i]);
          vr[i][1] = *reinterpret_cast<const uint4*>(vp[i] + d2 - d1);
        } else {
          kr[i][0] = load8_unaligned(kp[i]);
          kr[i][1] = load8_unaligned(kp[i] + d2 - d1);
          vr[i][0] = load8_unaligned(vp[i]);
          vr[i][1] = load8_unaligned(vp[i] + d2 - d1);
        }
      }
      kp[i] += step_heads * p.k_head;
      vp[i] += step_heads * p.v_head;
    }
  };
  load(0);

  bool odd = false;  // a scale so far that is no power of two
  if constexpr (FP8) {
    for (int i = tid; i < 2 * nheads; i += THREADS) {
      const int w = i >= nheads, h = i - w * nheads;
      amax_s[w][h] = 0;
      const float had = t_lo > 0 ? (w ? p.cache.v_scale : p.cache.k_scale)[page_rows + h] : 0.f;
      had_s[w][h] = had;
      had_inv_s[w][h] = 1.f / had;
      odd |= !is_pow2(had);
    }
  }
  const float amplitude = static_cast<float>(p.plan.amplitude);
  const int planes = (t_hi - t_lo) << p.log_units;  // float4 of a plane
  {
    // a warp at one pair of frequencies (their loads are uniform), its lanes
    // at the tokens
    for (int m = 2 * (tid >> 5); m < p.plan.rot_dim >> 1; m += THREADS / 16) {
      const unsigned long long w0 = p.plan.turns[m], w1 = p.plan.turns[m + 1];
      for (int tok = lane; tok < t_hi - t_lo; tok += 32) {
        float4 f;
        rotary_sincos(w0, page0 + t_lo + tok, f.x, f.y);
        rotary_sincos(w1, page0 + t_lo + tok, f.z, f.w);
        f.x *= amplitude, f.y *= amplitude, f.z *= amplitude, f.w *= amplitude;
        f = make_float4(f.x, f.z, f.y, f.w);
        turn_s[((m >> 1) & 3) * planes + (tok << p.log_units) + (m >> 3)] = f;
      }
    }
  }
  if constexpr (FP8)
    odd = __syncthreads_or(odd);
  else
    __syncthreads();

  for (int head = 0; head < nheads; head += step_heads) {
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < UNITS; ++i) {
        int hs, slot, unit, d1, d2;
        place(i, hs, slot, unit, d1, d2);
        uint32_t both = absmax_bf16(kr[i][0], kr[i][1]) << 16 | absmax_bf16(vr[i][0], vr[i][1]);
        if (log_items >= 5) {  // the warp has one head
          both = __reduce_max_sync(0xffffffffu, both >> 16) << 16 | __reduce_max_sync(0xffffffffu, both & 0xffffu);
        } else {
#pragma unroll
          for (int o = 8; o > 0; o >>= 1) {  // lanes of one head
            const uint32_t other = __shfl_xor_sync(0xffffffffu, both, o);
            if (o < (1 << log_items)) both = __vmaxu2(both, other);
          }
        }
        if ((lane & ((1 << log_items) - 1)) == 0 && head + hs < nheads && hs < step_heads) {
          if (both >> 16) atomicMax(&amax_s[0][head + hs], static_cast<int>(both >> 16));
          if (both & 0xffffu) atomicMax(&amax_s[1][head + hs], static_cast<int>(both & 0xffffu));
        }
      }
      __syncthreads();
      // each head's scales, and the codes that are in the page to a larger one
      const int heads_now = min(step_heads, nheads - head);
      for (int i = tid; i < 2 * heads_now; i += THREADS) {
        const int w = i >= heads_now, h = head + i - w * heads_now;
        const float want = w ? scale_for(amax_s[1][h], p.exp_v) : scale_for(amax_s[0][h], p.exp_k);
        const float now = t_lo > 0 ? fmaxf(want, had_s[w][h]) : want;
        if (t_lo == 0 || now != had_s[w][h]) (w ? p.cache.v_scale : p.cache.k_scale)[page_rows + h] = now;
      }
      if (t_lo > 0) {
        for (int w = 0; w < 2; ++w) {
          uint8_t* base = static_cast<uint8_t*>(w ? p.cache.v : p.cache.k);
          for (int h = head; h < head + heads_now; ++h) {
            const float want = w ? scale_for(amax_s[1][h], p.exp_v) : scale_for(amax_s[0][h], p.exp_k);
            const float had = had_s[w][h], now = fmaxf(want, had);
            if (now == had) continue;
            uint2* row = reinterpret_cast<uint2*>(base + ((page_rows + h) << p.log_page) * d);
            for (int i = tid; i < t_lo * d / 8; i += THREADS) row[i] = moved8(row[i], had / now);
          }
        }
      }
    }

    uint4 kc[UNITS][2], vc[UNITS][2];
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) kc[i][j] = kr[i][j], vc[i][j] = vr[i][j];
    if (head + step_heads < nheads) load(head + step_heads);

#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      int hs, slot, unit, d1, d2;
      place(i, hs, slot, unit, d1, d2);
      if (hs >= step_heads || head + hs >= nheads || slot >= t_hi) continue;
      const int h = head + hs;
      const size_t at = (((page_rows + h) << p.log_page) + slot) * d;
      const bool turns = unit < rot_units;
      float s[8], c[8];
      if (turns) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float4 f = turn_s[j * planes + ((slot - t_lo) << p.log_units) + unit];
          s[2 * j] = f.x, s[2 * j + 1] = f.y, c[2 * j] = f.z, c[2 * j + 1] = f.w;
        }
      }
      float x1[8], x2[8];
      unpack8(kc[i][0], x1);
      unpack8(kc[i][1], x2);
      if constexpr (!FP8) {
        __nv_bfloat16* ko = static_cast<__nv_bfloat16*>(p.cache.k) + at;
        __nv_bfloat16* vo = static_cast<__nv_bfloat16*>(p.cache.v) + at;
        if (turns) {
          rotate_unit<8>(x1, x2, s, c, INTERLEAVED);
          store_vec<8>(ko + d1, x1);
          store_vec<8>(ko + d2, x2);
        } else {
          *reinterpret_cast<uint4*>(ko + d1) = kc[i][0];
          *reinterpret_cast<uint4*>(ko + d2) = kc[i][1];
        }
        *reinterpret_cast<uint4*>(vo + d1) = vc[i][0];
        *reinterpret_cast<uint4*>(vo + d2) = vc[i][1];
      } else {
        uint8_t* ko = static_cast<uint8_t*>(p.cache.k) + at;
        uint8_t* vo = static_cast<uint8_t*>(p.cache.v) + at;
        const float want_k = scale_for(amax_s[0][h], p.exp_k), want_v = scale_for(amax_s[1][h], p.exp_v);
        // 1 over the scale: exact from a power of two's bits, but the page's
        // scale so far may be any number (whose codes are divided below)
        const bool same_k = want_k <= had_s[0][h], same_v = want_v <= had_s[1][h];
        const float ik = same_k ? had_inv_s[0][h] : __int_as_float((254 << 23) - __float_as_int(want_k));
        const float iv = same_v ? had_inv_s[1][h] : __int_as_float((254 << 23) - __float_as_int(want_v));
        uint2 o1, o2;
        // The fp32 rotation is off by less than 2^-22 (|a| + |q|): sine and
        // cosine by 2^-23, two products and a sum by 2^-24 each; by twice that
        // times the amplitude where there is one; by nothing at position 0,
        // where many values do lie on a border. A head with magnitudes of the
        // largest scale leaves all but its zeros open: an amplitude may take
        // them past fp32, and 0 times an infinity would be NaN.
        const float slack = want_k == 0x1p120f ? FLT_MAX
                            : amplitude != 1.f ? ik * 4.76837158e-07f * amplitude
                            : page0 + slot     ? ik * 2.38418579e-07f
                                               : 0.f;
        uint32_t doubt = 0;  // pairs whose codes the fp32 rotation leaves open
        if (turns) {
          uint32_t code[8];  // of pair m: first member's code, second's in the next byte
          const float2 scale2 = make_float2(ik, ik);
#pragma unroll
          for (int m = 0; m < 8; m += 2) {  // two pairs at a time in packed fp32
            float2 a, q;
            if (INTERLEAVED) {
              const float(&x)[8] = m < 4 ? x1 : x2;
              const int e = 2 * (m & 3);
              a = make_float2(x[e], x[e + 2]);
              q = make_float2(x[e + 1], x[e + 3]);
            } else {
              a = make_float2(x1[m], x1[m + 1]);
              q = make_float2(x2[m], x2[m + 1]);
            }
            const float2 sm = make_float2(s[m], s[m + 1]), cm = make_float2(c[m], c[m + 1]);
            const float2 y1 = fma2(a, cm, mul2(q, make_float2(-sm.x, -sm.y))), y2 = fma2(a, sm, mul2(q, cm));
            // where both ends of the rotation's error bound round to one
            // code it is the right one
            const float2 off = make_float2((fabsf(a.x) + fabsf(q.x)) * slack, (fabsf(a.y) + fabsf(q.y)) * slack);
            const float2 neg = make_float2(-off.x, -off.y);
            const float2 l1 = fma2(y1, scale2, neg), l2 = fma2(y2, scale2, neg);
            const float2 u1 = fma2(y1, scale2, off), u2 = fma2(y2, scale2, off);
            code[m] = e4m3x2(l1.x, l2.x);
            code[m + 1] = e4m3x2(l1.y, l2.y);
            if (code[m] != e4m3x2(u1.x, u2.x)) doubt |= 1u << m;
            if (code[m + 1] != e4m3x2(u1.y, u2.y)) doubt |= 2u << m;
          }
          if (INTERLEAVED) {
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
        unpack8(vc[i][0], x1);
        unpack8(vc[i][1], x2);
        *reinterpret_cast<uint2*>(vo + d1) = codes8(x1, iv);
        *reinterpret_cast<uint2*>(vo + d2) = codes8(x2, iv);
        const __nv_bfloat16* row = p.K + k_base + slot * p.k_row + h * p.k_head;
        while (doubt) {
          const int m = __ffs(doubt) - 1;
          doubt &= doubt - 1;
          const int e1 = INTERLEAVED ? d1 + 2 * m : d1 + m, e2 = INTERLEAVED ? e1 + 1 : d2 + m;
          const uint32_t both = rotated_codes_exact<false>(__bfloat162float(row[e1]), __bfloat162float(row[e2]),
                                                           p.plan.turns[8 * unit + m], page0 + slot,
                                                           p.plan.amplitude, ik);
          ko[e1] = static_cast<uint8_t>(both);
          ko[e2] = static_cast<uint8_t>(both >> 8);
        }
      }
    }
  }
  if (FP8 && odd) {
    __syncthreads();
    divided_codes<INTERLEAVED>(p, had_s, amax_s, nheads, page_rows, page0, t_lo, t_hi, p.K + k_base, p.V + v_base);
  }
}

// {e0, threshold}: see scale_for. The quotient is formed as its definition
// says, magnitude times reach over 448 in 64 bits, for every 7-bit mantissa.
void scale_exponents(double reach, int (&ex)[2]) {
  auto exponent = [&](int m) {  // smallest e with (1 + m / 128) reach / 448 <= 2^e
    int e;
    return std::frexp((1.0 + m / 128.0) * reach / 448.0, &e) == 0.5 ? e - 1 : e;
  };
  ex[0] = exponent(0);
  ex[1] = 0;
  while (ex[1] < 128 && exponent(ex[1]) == ex[0]) ++ex[1];
}

template <bool FP8, bool INTERLEAVED>
void (*append_kernel(int threads, int units))(AppendParams) {
  if (units == 2) return relpos_paged_append_kernel<FP8, INTERLEAVED, 512, 2>;
  if (threads == 512) return relpos_paged_append_kernel<FP8, INTERLEAVED, 512, 1>;
  if (threads == 256) return relpos_paged_append_kernel<FP8, INTERLEAVED, 256, 1>;
  return relpos_paged_append_kernel<FP8, INTERLEAVED, 128, 1>;
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
  scale_exponents(plan ? 1.4142135623730951 * plan->amplitude : 1.0, p.exp_k);
  scale_exponents(1.0, p.exp_v);
  p.status = device_status();
  const int sms = device_sms();
  if (!p.status || sms <= 0) return RELPOS_ERR_CUDA;
  // a thread for each 16-element unit of a head's page, two units from 1024 on
  const int items = 1 << (p.log_page + p.log_units);
  const int threads = std::min(items, 512), units = items / threads;
  const long long pages = (total >> p.log_page) + 2 * static_cast<long long>(B);
  // heads of a block: as few as fill the GPU's SMs, since a block walks them
  const long long groups = std::min<long long>(
      cache->H, std::max<long long>((cache->H + kAppMaxGroup - 1) / kAppMaxGroup, (2 * sms + pages - 1) / pages));
  p.group = static_cast<int>((cache->H + groups - 1) / groups);
  const bool inter = p.plan.layout == RELPOS_ROTARY_INTERLEAVED;
  const auto kernel = cache->dtype == RELPOS_E4M3
                          ? (inter ? append_kernel<true, true>(threads, units)
                                   : append_kernel<true, false>(threads, units))
                          : (inter ? append_kernel<false, true>(threads, units)
                                   : append_kernel<false, false>(threads, units));
  const int smem = p.plan.rot_dim ? 64 * items : 0;
  if (smem > 48 * 1024 &&
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pages), (cache->H + p.group - 1) / p.group);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  return RELPOS_OK;
}
