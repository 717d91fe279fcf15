// paged.cuh -- device helpers of the paged key/value cache: bf16 and e4m3
// vectors as the append kernel reads, scales and writes them.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "ptx.cuh"

namespace relpos {

// two fp32 operations in one instruction
RP_DEVI float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
RP_DEVI float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }

// 8 bf16 values from a pointer that is only 2-byte aligned
RP_DEVI uint4 load8_unaligned(const __nv_bfloat16* p) {
  const unsigned short* u = reinterpret_cast<const unsigned short*>(p);
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = u[2 * e] | static_cast<uint32_t>(u[2 * e + 1]) << 16;
  return make_uint4(w[0], w[1], w[2], w[3]);
}

RP_DEVI void unpack8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
  }
}

// The largest magnitude among 16 bf16 values, as the bits of a bf16: they
// order like the magnitudes, infinity last. NaN counts as nothing.
RP_DEVI uint32_t absmax_bf16(const uint4& u, const uint4& v) {
  const uint32_t w[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
  uint32_t m = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = __vmaxu2(m, w[e] & 0x7fff7fffu);
  m = max(m & 0xffffu, m >> 16);
  if (m > 0x7f80u) {  // a NaN among them
    m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
      m = max(m, lo > 0x7f80u ? 0u : lo);
      m = max(m, hi > 0x7f80u ? 0u : hi);
    }
  }
  return m;
}

// 8 values times inv (a power of two) as e4m3 codes, rounded to nearest even,
// saturating at 448
RP_DEVI uint2 codes8(const float (&f)[8], float inv) {
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e)
    c[e] = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * e] * inv, f[2 * e + 1] * inv), __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

RP_DEVI bool is_pow2(float x) { return (__float_as_uint(x) & 0x7fffffu) == 0; }

// A result y of an operation that rounded towards zero, its last bit made odd
// where the operation dropped something: rounded to a code it then falls on the
// side of a border that the exact result lies on.
RP_DEVI float sticky(float y, bool dropped) { return __uint_as_float(__float_as_uint(y) | (dropped ? 1u : 0u)); }

// The code of x / scale for a scale (2^-120 or more) that is no power of two
RP_DEVI uint8_t code_over(float x, float scale) {
  const float up = scale < 0x1p-60f ? 0x1p60f : 1.f;  // the division's remainder has to be representable
  x *= up;
  scale *= up;
  const float q = __fdiv_rz(x, scale);
  // beyond 1024 it saturates (infinity and NaN stay as they are)
  return __nv_cvt_float_to_fp8(sticky(q, fabsf(q) < 1024.f && fmaf(-q, scale, x) != 0.f), __NV_SATFINITE, __NV_E4M3);
}

// 8 codes times ratio = old scale / new scale, the new one a power of two
RP_DEVI uint2 moved8(const uint2& u, float ratio) {
  uint32_t w[2] = {u.x, u.y};
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    uint32_t out = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2_raw r =
          __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>((w[e] >> (16 * h)) & 0xffffu), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      // towards zero and sticky: the product may have more than fp32's 24 bits
      float2 y = make_float2(__fmul_rz(f.x, ratio), __fmul_rz(f.y, ratio));
      y.x = sticky(y.x, fmaf(f.x, ratio, -y.x) != 0.f);
      y.y = sticky(y.y, fmaf(f.y, ratio, -y.y) != 0.f);
      const uint32_t c = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
      out |= c << (16 * h);
    }
    w[e] = out;
  }
  return make_uint2(w[0], w[1]);
}

}  // namespace relpos
