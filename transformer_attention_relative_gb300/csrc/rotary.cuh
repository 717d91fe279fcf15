// rotary.cuh -- the rotation of rotary positions, shared by the kernel that
// rotates queries and keys and the one that appends keys to a paged cache.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "../../include/relpos_attn.h"
#include "ptx.cuh"

namespace relpos {

// sin and cos of the angle position * w. The plan holds w / 2 pi as a 64-bit
// fraction of a turn, so the product modulo 2^64 is the angle modulo a full
// turn, exact for every 32-bit position (an fp32 product would lose a far
// position's angle: at position 10^6 its rounding alone is 0.03 radians). What
// is left of it after the nearest quarter turn lies in [-pi/4, pi/4], where the
// Taylor series to y^9 (sine) and y^10 (cosine) are below half an fp32 ulp off.
RP_DEVI void rotary_sincos(unsigned long long turns, int pos, float& s, float& c) {
  const uint32_t u = static_cast<uint32_t>((turns * static_cast<unsigned long long>(static_cast<long long>(pos))) >> 32);
  const uint32_t q = (u + 0x20000000u) >> 30;  // nearest quarter turn
  const int r = static_cast<int>(u - (q << 30));
  const float y = static_cast<float>(r) * 1.46291807926715968e-09f;  // 2 pi / 2^32
  const float z = y * y;
  float ps = fmaf(z, 2.75573192e-06f, -1.98412698e-04f);
  ps = fmaf(z, ps, 8.33333333e-03f);
  ps = fmaf(z, ps, -1.66666667e-01f);
  ps = fmaf(y * z, ps, y);
  float pc = fmaf(z, -2.75573192e-07f, 2.48015873e-05f);
  pc = fmaf(z, pc, -1.38888889e-03f);
  pc = fmaf(z, pc, 4.16666667e-02f);
  pc = fmaf(z, pc, -0.5f);
  pc = fmaf(z, pc, 1.0f);
  const float a = (q & 1u) ? pc : ps, b = (q & 1u) ? ps : pc;
  s = (q & 2u) ? -a : a;
  c = ((q + 1u) & 2u) ? -b : b;
}

// (x1, x2) turned by the angle; the amplitude is in s and c.
RP_DEVI void rotate_pair(float x1, float x2, float s, float c, float& y1, float& y2) {
  y1 = fmaf(x1, c, -(x2 * s));
  y2 = fmaf(x1, s, x2 * c);
}

// P consecutive values to and from fp32 registers; the pointer is aligned to
// P * sizeof(T) bytes (16 for the widest).
template <int P>
RP_DEVI void load_vec(const __nv_bfloat16* p, float (&f)[P]) {
  if constexpr (P == 1) {
    f[0] = __bfloat162float(*p);
  } else {
    uint32_t w[P / 2];
    if constexpr (P == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      w[0] = u.x, w[1] = u.y, w[2] = u.z, w[3] = u.w;
    } else {
      static_assert(P == 4, "vector width");
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      w[0] = u.x, w[1] = u.y;
    }
#pragma unroll
    for (int e = 0; e < P / 2; ++e) {
      f[2 * e] = __uint_as_float(w[e] << 16);
      f[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
  }
}
template <int P>
RP_DEVI void load_vec(const float* p, float (&f)[P]) {
  if constexpr (P == 1) {
    f[0] = *p;
  } else {
#pragma unroll
    for (int e = 0; e < P / 4; ++e) {
      const float4 u = reinterpret_cast<const float4*>(p)[e];
      f[4 * e] = u.x, f[4 * e + 1] = u.y, f[4 * e + 2] = u.z, f[4 * e + 3] = u.w;
    }
  }
}
template <int P>
RP_DEVI void store_vec(__nv_bfloat16* p, const float (&f)[P]) {
  if constexpr (P == 1) {
    *p = __float2bfloat16_rn(f[0]);
  } else {
    uint32_t w[P / 2];
#pragma unroll
    for (int e = 0; e < P / 2; ++e) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    if constexpr (P == 8) {
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
  }
}
template <int P>
RP_DEVI void store_vec(float* p, const float (&f)[P]) {
  if constexpr (P == 1) {
    *p = f[0];
  } else {
#pragma unroll
    for (int e = 0; e < P / 4; ++e)
      reinterpret_cast<float4*>(p)[e] = make_float4(f[4 * e], f[4 * e + 1], f[4 * e + 2], f[4 * e + 3]);
  }
}

// The 2P values a thread turns as P pairs: v1 and v2 are the first and second
// members of the pairs ("half"), or 2P neighbouring values ("interleaved").
template <int P>
RP_DEVI void rotate_unit(float (&v1)[P], float (&v2)[P], const float (&s)[P], const float (&c)[P], bool interleaved) {
  if (interleaved) {
    if constexpr (P == 1) {
      rotate_pair(v1[0], v2[0], s[0], c[0], v1[0], v2[0]);
    } else {
#pragma unroll
      for (int m = 0; m < P / 2; ++m) {
        rotate_pair(v1[2 * m], v1[2 * m + 1], s[m], c[m], v1[2 * m], v1[2 * m + 1]);
        rotate_pair(v2[2 * m], v2[2 * m + 1], s[P / 2 + m], c[P / 2 + m], v2[2 * m], v2[2 * m + 1]);
      }
    }
  } else {
#pragma unroll
    for (int m = 0; m < P; ++m) rotate_pair(v1[m], v2[m], s[m], c[m], v1[m], v2[m]);
  }
}

// true when the plan can have come from relpos_rotary_plan_init
inline bool rotary_plan_ok(const RelposRotaryPlan* p) {
  return p && p->rot_dim >= 2 && p->rot_dim <= RELPOS_ROTARY_MAX_DIM && p->rot_dim % 2 == 0 &&
         (p->layout == RELPOS_ROTARY_HALF || p->layout == RELPOS_ROTARY_INTERLEAVED) && p->amplitude > 0.0;
}

}  // namespace relpos
