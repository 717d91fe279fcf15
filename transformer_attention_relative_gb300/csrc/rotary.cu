// rotary.cu -- rotary positions: queries and keys turned by their position
// before attention ("Relative Position Embeddings, in depth", section "ALiBi
// and RoPE: the two endpoints"), and the gradient, the turn by the opposite
// angle. The work is a stream: every element read once and written once, with
// a sine and a cosine for each (token, frequency) that all heads share. Measured:
// 4 x 2048 tokens of 32 heads, d = 64, bf16, 12.2 us (5.5 TB/s, 81 % of a copy's
// rate); 16411 tokens of 20 heads, d = 128, fp32, 55 us (6.1 TB/s, 90 %).

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/relpos_attn.h"
#include "ptx.cuh"
#include "rotary.cuh"
#include "serving_internal.h"

namespace relpos {
namespace {

constexpr int kRotThreads = 256;

struct RotaryParams {
  RelposRotaryPlan plan;
  RelposRotaryTensor t[2];
  const int* positions;   // or null: position offset + l
  long long pos_stride;   // between batch elements, 0 when they share the positions
  int offset;
  int heads, heads0;      // of both tensors, of the first
  int group;              // heads a thread turns with its sines and cosines
  int units, rot_units;   // 2P-element units of a head, and those that turn
  int L;
  unsigned n;             // tokens * units
  float sign;             // -1: the gradient
};

// A thread owns one unit (2P elements) of one token and walks `group` heads
// with the unit's P sines and cosines in registers: 28 instructions for each
// angle, against 12 for each pair and head. Consecutive threads have consecutive
// units and tokens, so a warp's 16-byte accesses cover whole rows.
template <typename T, int P>
__global__ void __launch_bounds__(kRotThreads) relpos_rotary_kernel(const __grid_constant__ RotaryParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const unsigned idx = blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= p.n) return;
  const unsigned tok = idx / p.units;
  const int unit = static_cast<int>(idx - tok * p.units);
  const int b = static_cast<int>(tok / p.L), l = static_cast<int>(tok - static_cast<unsigned>(b) * p.L);
  const bool interleaved = p.plan.layout == RELPOS_ROTARY_INTERLEAVED;
  const bool turns = unit < p.rot_units;
  int d1, d2;
  if (!turns) {
    d1 = 2 * P * unit;
    d2 = d1 + P;
  } else if (interleaved) {
    d1 = 2 * P * unit;
    d2 = d1 + P;
  } else {
    d1 = P * unit;
    d2 = p.plan.rot_dim / 2 + d1;
  }
  float s[P], c[P];
  if (turns) {
    const float amplitude = static_cast<float>(p.plan.amplitude);
    const int pos = p.positions ? p.positions[b * p.pos_stride + l] : p.offset + l;
#pragma unroll
    for (int m = 0; m < P; ++m) {
      rotary_sincos(p.plan.turns[P * unit + m], pos, s[m], c[m]);
      s[m] *= p.sign * amplitude;
      c[m] *= amplitude;
    }
  }
  const int h_end = min(p.heads, static_cast<int>(blockIdx.y + 1) * p.group);
#pragma unroll 2
  for (int h = blockIdx.y * p.group; h < h_end; ++h) {
    const RelposRotaryTensor& t = p.t[h >= p.heads0];
    const int ht = h >= p.heads0 ? h - p.heads0 : h;
    const T* x = static_cast<const T*>(t.x) + b * t.x_batch + ht * t.x_head + l * t.x_row;
    T* y = static_cast<T*>(t.out) + b * t.out_batch + ht * t.out_head + l * t.out_row;
    float v1[P], v2[P];
    load_vec<P>(x + d1, v1);
    load_vec<P>(x + d2, v2);
    if (turns) rotate_unit<P>(v1, v2, s, c, interleaved);
    store_vec<P>(y + d1, v1);
    store_vec<P>(y + d2, v2);
  }
}

template <typename T>
cudaError_t launch_rotary(const RotaryParams& p, int P, dim3 grid, int threads, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (P == 8) return cudaLaunchKernelEx(&cfg, relpos_rotary_kernel<T, 8>, p);
  if (P == 4) return cudaLaunchKernelEx(&cfg, relpos_rotary_kernel<T, 4>, p);
  return cudaLaunchKernelEx(&cfg, relpos_rotary_kernel<T, 1>, p);
}

// whether every row of the tensor starts on a multiple of `bytes`
bool rows_aligned(const RelposRotaryTensor& t, size_t esize, size_t bytes) {
  const uintptr_t p = reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.out);
  const unsigned long long st = static_cast<unsigned long long>(t.x_batch) | static_cast<unsigned long long>(t.x_head) |
                                static_cast<unsigned long long>(t.x_row) | static_cast<unsigned long long>(t.out_batch) |
                                static_cast<unsigned long long>(t.out_head) | static_cast<unsigned long long>(t.out_row);
  return p % bytes == 0 && st * esize % bytes == 0;
}

}  // namespace
}  // namespace relpos

using namespace relpos;

extern "C" int relpos_rotary_plan_init(RelposRotaryPlan* plan, int rot_dim, int layout, double base, int scaling,
                                       double factor, double original_len, double fast_turns, double slow_turns) {
  if (!plan) return RELPOS_ERR_INVALID_ARG;
  if (rot_dim < 2 || rot_dim > RELPOS_ROTARY_MAX_DIM || rot_dim % 2) return RELPOS_ERR_INVALID_ARG;
  if (layout != RELPOS_ROTARY_HALF && layout != RELPOS_ROTARY_INTERLEAVED) return RELPOS_ERR_INVALID_ARG;
  if (!(base > 1.0) || !std::isfinite(base)) return RELPOS_ERR_INVALID_ARG;
  if (scaling < RELPOS_ROTARY_PLAIN || scaling > RELPOS_ROTARY_YARN) return RELPOS_ERR_INVALID_ARG;
  if (scaling != RELPOS_ROTARY_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor))) return RELPOS_ERR_INVALID_ARG;
  if (scaling == RELPOS_ROTARY_NTK && rot_dim < 4) return RELPOS_ERR_INVALID_ARG;
  if (scaling == RELPOS_ROTARY_YARN &&
      (!(original_len > 0.0) || !(slow_turns >= 0.0) || !(fast_turns > slow_turns) || !std::isfinite(original_len) ||
       !std::isfinite(fast_turns)))
    return RELPOS_ERR_INVALID_ARG;
  std::memset(plan, 0, sizeof(*plan));
  plan->rot_dim = rot_dim;
  plan->layout = layout;
  plan->amplitude = scaling == RELPOS_ROTARY_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  const double two_pi = 6.283185307179586476925;
  const double b = scaling == RELPOS_ROTARY_NTK ? base * std::pow(factor, rot_dim / (rot_dim - 2.0)) : base;
  for (int m = 0; m < rot_dim / 2; ++m) {
    double w = std::pow(b, -2.0 * m / rot_dim);
    if (scaling == RELPOS_ROTARY_LINEAR) w /= factor;
    if (scaling == RELPOS_ROTARY_YARN) {
      double keep = (original_len * w / two_pi - slow_turns) / (fast_turns - slow_turns);
      keep = std::min(1.0, std::max(0.0, keep));
      w = w / factor * (1.0 - keep) + w * keep;
    }
    // w <= 1, so the fraction of a turn is below 1 / 2 pi
    plan->turns[m] = static_cast<unsigned long long>(w / two_pi * 18446744073709551616.0 + 0.5);
  }
  return RELPOS_OK;
}

extern "C" int relpos_rotary(const RelposRotaryPlan* plan, int dtype, int inverse, const RelposRotaryTensor* tensors,
                             int ntensors, int B, int L, int d, const int* positions, long long pos_stride, int offset,
                             void* stream) {
  if (!rotary_plan_ok(plan)) return RELPOS_ERR_INVALID_ARG;
  if (dtype != RELPOS_BF16 && dtype != RELPOS_FP32) return RELPOS_ERR_INVALID_ARG;
  if (inverse != 0 && inverse != 1) return RELPOS_ERR_INVALID_ARG;
  if (!tensors || ntensors < 1 || ntensors > 2) return RELPOS_ERR_INVALID_ARG;
  if (B < 0 || L < 0 || d < plan->rot_dim || d % 2) return RELPOS_ERR_INVALID_ARG;
  int heads = 0;
  for (int i = 0; i < ntensors; ++i) {
    if (tensors[i].H < 0) return RELPOS_ERR_INVALID_ARG;
    if (tensors[i].H > 65535) return RELPOS_ERR_UNSUPPORTED;
    heads += tensors[i].H;
  }
  if (B == 0 || L == 0 || heads == 0) return RELPOS_OK;
  if (reinterpret_cast<uintptr_t>(positions) & 3u) return RELPOS_ERR_INVALID_ARG;
  if (!positions && static_cast<long long>(offset) + L - 1 > 0x7fffffffll) return RELPOS_ERR_INVALID_ARG;
  const size_t esize = dtype == RELPOS_FP32 ? 4 : 2;
  for (int i = 0; i < ntensors; ++i)
    if (tensors[i].H > 0 && (!tensors[i].x || !tensors[i].out || !rows_aligned(tensors[i], esize, esize)))
      return RELPOS_ERR_INVALID_ARG;
  // the widest unit that the sizes, pointers and strides allow: 16-byte loads
  // (8 bf16; 4 fp32, two of them for 8 pairs), 8-byte loads, single values
  int P = 1;
  for (int w : {8, 4}) {
    bool ok = plan->rot_dim % (2 * w) == 0 && d % (2 * w) == 0;
    for (int i = 0; i < ntensors; ++i)
      ok = ok && (tensors[i].H == 0 || rows_aligned(tensors[i], esize, std::min<size_t>(16, w * esize)));
    if (ok) {
      P = w;
      break;
    }
  }
  RotaryParams p;
  std::memset(&p, 0, sizeof(p));
  p.plan = *plan;
  for (int i = 0; i < ntensors; ++i) p.t[i] = tensors[i];
  p.positions = positions;
  p.pos_stride = pos_stride;
  p.offset = offset;
  p.heads = heads;
  p.heads0 = tensors[0].H;
  p.units = d / (2 * P);
  p.rot_units = plan->rot_dim / (2 * P);
  p.L = L;
  p.sign = inverse ? -1.f : 1.f;
  const long long n = static_cast<long long>(B) * L * p.units;
  if (n > 0x7fffffffll) return RELPOS_ERR_UNSUPPORTED;
  for (int i = 0; i < ntensors; ++i)
    if (tensors[i].H > 0 && (rows_overlap(B, tensors[i].out_batch, d) || rows_overlap(L, tensors[i].out_row, d) ||
                             rows_overlap(tensors[i].H, tensors[i].out_head, d)))
      return RELPOS_ERR_INVALID_ARG;
  p.n = static_cast<unsigned>(n);
  const int sms = device_sms();
  if (sms <= 0) return RELPOS_ERR_CUDA;
  // heads a thread walks: as many as leave every SM its fill of threads, since
  // the sines and cosines (about 25 instructions each) are shared among them
  // (1024 threads an SM, 52 registers each; 4 x 2048 tokens of 32 heads: 11.8 us
  // against 12.7 with twice and 14.6 with four times as many)
  const long long want = (static_cast<long long>(sms) * 1024 + n - 1) / n;
  const int groups = static_cast<int>(std::min<long long>({want, heads, 65535}));
  p.group = (heads + groups - 1) / groups;
  const int threads = static_cast<int>(std::min<long long>(kRotThreads, (n + 31) / 32 * 32));
  const dim3 grid(static_cast<unsigned>((n + threads - 1) / threads), (heads + p.group - 1) / p.group);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == RELPOS_FP32 ? launch_rotary<float>(p, P, grid, threads, s)
                                             : launch_rotary<__nv_bfloat16>(p, P, grid, threads, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return RELPOS_ERR_CUDA;
  }
  return RELPOS_OK;
}
