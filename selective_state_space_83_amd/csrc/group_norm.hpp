// group_norm.hpp -- gfx950 device code of the group norm with an activation or
// a gate over the channels of each row (token):
//
//   u = x or x silu(z);  n = (u - mean) r, r = 1 / sqrt(var + eps)  (rms: mean = 0)
//   a = n w + b;         y = a, silu(a) or a silu(z)
//
// and its gradients.  With s(z) = 1 / (1 + exp(-z)), silu'(z) = s (1 + z (1 - s)):
//   da = dy, dy silu'(a) or dy silu(z);   dw = sum_rows da n;   db = sum_rows da
//   dn = da w;   du = r (dn - mean(dn) - n mean(dn n))          (rms: no mean(dn))
//   dx = du or du silu(z);   dz = dy a silu'(z) or du x silu'(z)
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssmn {

using bf16_t = uint16_t;

constexpr int kWave = 64;
constexpr float kLog2e = 1.4426950408889634f;

enum Mode : int { kPlain = 0, kSilu = 1, kGate = 2, kGateFirst = 3 };

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const bf16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(bf16_t* p, float v) {
  *p = __builtin_bit_cast(bf16_t, static_cast<__bf16>(v));   // to nearest even
}

// 1 / (1 + exp(-z)): the exp overflows to inf for z -> -inf and rcp gives 0
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * kLog2e));
}

struct NormParams {
  const void* x;
  const void* z;
  const void* dy;
  const float* w;
  const float* b;
  void* y;               // forward: y; backward: dx
  void* dz;
  float* stats;          // (rows, groups, 2): mean, r, for the column sums; or null
  float* dw;
  float* db;
  int64_t rows, C, G, gs;
  int64_t xs, zs, ds;    // row strides of x, z, dy
  int32_t mode, rms;
  float eps;
};

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int w = 32; w; w >>= 1) v += __shfl_xor(v, w);
  return v;
}

// One wave per (row, group), three reads of the row from the caches.
template <typename T>
__device__ __forceinline__ float norm_input(const NormParams& p, int64_t row, int64_t c) {
  const float x = ld(static_cast<const T*>(p.x) + row * p.xs + c);
  if (p.mode != kGateFirst) return x;
  const float z = ld(static_cast<const T*>(p.z) + row * p.zs + c);
  return x * (z * sigmoid(z));
}

template <typename T>
__device__ __forceinline__ void norm_stats(const NormParams& p, int64_t row, int64_t c0, float* mean,
                                           float* r) {
  const int lane = threadIdx.x;
  float m = 0.0f;
  if (!p.rms) {
    for (int64_t i = lane; i < p.gs; i += kWave) m += norm_input<T>(p, row, c0 + i);
    m = wave_sum(m) / float(p.gs);
  }
  float v = 0.0f;
  for (int64_t i = lane; i < p.gs; i += kWave) {
    const float d = norm_input<T>(p, row, c0 + i) - m;
    v += d * d;
  }
  v = wave_sum(v) / float(p.gs);
  *mean = m;
  *r = 1.0f / sqrtf(v + p.eps);
}

template <typename T>
__global__ __launch_bounds__(kWave) void k_norm_simple(NormParams p) {
  const int64_t row = blockIdx.x / p.G, c0 = blockIdx.x % p.G * p.gs;
  float mean, r;
  norm_stats<T>(p, row, c0, &mean, &r);
  for (int64_t i = threadIdx.x; i < p.gs; i += kWave) {
    const int64_t c = c0 + i;
    float a = (norm_input<T>(p, row, c) - mean) * r;
    a = a * (p.w ? p.w[c] : 1.0f) + (p.b ? p.b[c] : 0.0f);
    if (p.mode == kSilu) a *= sigmoid(a);
    if (p.mode == kGate) {
      const float z = ld(static_cast<const T*>(p.z) + row * p.zs + c);
      a *= z * sigmoid(z);
    }
    st(static_cast<T*>(p.y) + row * p.C + c, a);
  }
}

// da and n of one channel; *dz the gate's gradient in the gate mode.
template <typename T>
__device__ __forceinline__ float norm_da(const NormParams& p, int64_t row, int64_t c, float mean, float r,
                                         float* n, float* dz) {
  *n = (norm_input<T>(p, row, c) - mean) * r;
  const float dy = ld(static_cast<const T*>(p.dy) + row * p.ds + c);
  const float a = *n * (p.w ? p.w[c] : 1.0f) + (p.b ? p.b[c] : 0.0f);
  if (p.mode == kSilu) {
    const float s = sigmoid(a);
    return dy * (s * (1.0f + a * (1.0f - s)));
  }
  if (p.mode == kGate) {
    const float z = ld(static_cast<const T*>(p.z) + row * p.zs + c), s = sigmoid(z);
    *dz = dy * a * (s * (1.0f + z * (1.0f - s)));
    return dy * (z * s);
  }
  return dy;
}

template <typename T>
__global__ __launch_bounds__(kWave) void k_norm_bwd_simple(NormParams p) {
  const int64_t row = blockIdx.x / p.G, c0 = blockIdx.x % p.G * p.gs;
  float mean, r;
  norm_stats<T>(p, row, c0, &mean, &r);
  if (p.stats && threadIdx.x == 0) {
    p.stats[blockIdx.x * int64_t(2)] = mean;
    p.stats[blockIdx.x * int64_t(2) + 1] = r;
  }
  float sd = 0.0f, sdn = 0.0f, n, dz = 0.0f;
  for (int64_t i = threadIdx.x; i < p.gs; i += kWave) {
    const float dn = norm_da<T>(p, row, c0 + i, mean, r, &n, &dz) * (p.w ? p.w[c0 + i] : 1.0f);
    sd += dn;
    sdn += dn * n;
  }
  sd = p.rms ? 0.0f : wave_sum(sd) / float(p.gs);
  sdn = wave_sum(sdn) / float(p.gs);
  for (int64_t i = threadIdx.x; i < p.gs; i += kWave) {
    const int64_t c = c0 + i;
    const float dn = norm_da<T>(p, row, c, mean, r, &n, &dz) * (p.w ? p.w[c] : 1.0f);
    float du = r * (dn - sd - n * sdn);
    if (p.mode == kGateFirst) {
      const float x = ld(static_cast<const T*>(p.x) + row * p.xs + c);
      const float z = ld(static_cast<const T*>(p.z) + row * p.zs + c), s = sigmoid(z);
      dz = du * x * (s * (1.0f + z * (1.0f - s)));
      du *= z * s;
    }
    st(static_cast<T*>(p.y) + row * p.C + c, du);
    if (p.mode >= kGate) st(static_cast<T*>(p.dz) + row * p.C + c, dz);
  }
}

// A lane per channel, the rows one after another.
template <typename T>
__global__ __launch_bounds__(kWave) void k_norm_cols_simple(NormParams p) {
  const int64_t c = blockIdx.x * int64_t(kWave) + threadIdx.x;
  if (c >= p.C) return;
  float dw = 0.0f, db = 0.0f, n, dz;
  for (int64_t row = 0; row < p.rows; ++row) {
    const float* s = p.stats + (row * p.G + c / p.gs) * 2;
    const float da = norm_da<T>(p, row, c, s[0], s[1], &n, &dz);
    dw += da * n;
    db += da;
  }
  if (p.dw) p.dw[c] = dw;
  if (p.db) p.db[c] = db;
}

}  // namespace ssmn
