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
  float* dw;             // backward: (blocks of rows, C), each block's sums over its rows; or null
  float* db;
  int64_t rows, C, G, gs;
  int64_t xs, zs, ds;    // row strides of x, z, dy
  int64_t per;           // rows of a block: a lane walks them with its channels' weights in registers
  int32_t mode, rms;
  float eps;
};

template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// Sum over the TG neighbouring lanes that share a group, for all of them.
template <int TG>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (TG >= 2) v = dpp_add<0xB1>(v);    // lane ^ 1
  if constexpr (TG >= 4) v = dpp_add<0x4E>(v);    // lane ^ 2
  if constexpr (TG >= 8) v = dpp_add<0x141>(v);   // mirrored within 8
  if constexpr (TG >= 16) v = dpp_add<0x140>(v);  // mirrored within 16
  if constexpr (TG >= 32) v += __shfl_xor(v, 16);
  if constexpr (TG >= 64) v += __shfl_xor(v, 32);
  return v;
}

// The same for two sums; with TG = 256 the workgroup's four waves join in LDS.
template <int TG>
__device__ __forceinline__ void group_sum(float& a, float& b, float* part) {
  a = lanes_sum<TG>(a);
  b = lanes_sum<TG>(b);
  if constexpr (TG == 256) {
    const int w = threadIdx.x >> 6;
    __syncthreads();   // the last use of part
    if ((threadIdx.x & 63) == 0) {
      part[w] = a;
      part[4 + w] = b;
    }
    __syncthreads();
    a = part[0] + part[1] + part[2] + part[3];
    b = part[4] + part[5] + part[6] + part[7];
  }
}

// A lane's channels of one row: R times V of them, V side by side (V = 1, or 16
// bytes' worth), the lanes of a group taking turns.
template <typename T, int V, int R>
struct Slice {
  float v[R * V];
  template <int TG>
  __device__ __forceinline__ void load(const T* p, int lane, int gs) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (k * TG + lane) * V;
      if constexpr (V == 1) {
        v[k] = c < gs ? ld(p + c) : 0.0f;
      } else if constexpr (sizeof(T) == 4) {
        float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (c < gs) u = *reinterpret_cast<const float4*>(p + c);
        v[4 * k] = u.x;
        v[4 * k + 1] = u.y;
        v[4 * k + 2] = u.z;
        v[4 * k + 3] = u.w;
      } else {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (c < gs) u = *reinterpret_cast<const uint4*>(p + c);
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[8 * k + 2 * i] = __uint_as_float(a[i] << 16);
          v[8 * k + 2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
        }
      }
    }
  }
  template <int TG>
  __device__ __forceinline__ void store(T* p, int lane, int gs) const {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (k * TG + lane) * V;
      if (c >= gs) continue;
      if constexpr (V == 1) {
        st(p + c, v[k]);
      } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p + c) = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
      } else {
        typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
        bf16x8 u;
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = static_cast<__bf16>(v[8 * k + i]);
        *reinterpret_cast<bf16x8*>(p + c) = u;
      }
    }
  }
};

// Weight and bias of a lane's channels (1 and 0 without).
template <int V, int R, int TG>
__device__ __forceinline__ void load_affine(const NormParams& p, int64_t c0, int lane, float (&w)[R * V],
                                            float (&b)[R * V]) {
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int c = (k * TG + lane) * V;
    if constexpr (V == 1) {
      w[k] = p.w && c < p.gs ? p.w[c0 + c] : 1.0f;
      b[k] = p.b && c < p.gs ? p.b[c0 + c] : 0.0f;
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        float4 x = make_float4(1.0f, 1.0f, 1.0f, 1.0f), y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (p.w && c < p.gs) x = *reinterpret_cast<const float4*>(p.w + c0 + c + i);
        if (p.b && c < p.gs) y = *reinterpret_cast<const float4*>(p.b + c0 + c + i);
        w[k * V + i] = x.x;
        w[k * V + i + 1] = x.y;
        w[k * V + i + 2] = x.z;
        w[k * V + i + 3] = x.w;
        b[k * V + i] = y.x;
        b[k * V + i + 1] = y.y;
        b[k * V + i + 2] = y.z;
        b[k * V + i + 3] = y.w;
      }
    }
  }
}

// The normalized values of a row's slice in place of u (0 past the group's
// end); returns r.  The variance is the mean square of the differences: the
// values are in registers, so a second sum costs no second read.
template <int V, int R, int TG>
__device__ __forceinline__ float normalize(float (&u)[R * V], int lane, const NormParams& p, float inv, float* part) {
  const int gs = int(p.gs);
  float mean = 0.0f, zero = 0.0f;
  if (!p.rms) {
#pragma unroll
    for (int i = 0; i < R * V; ++i) mean += u[i];
    group_sum<TG>(mean, zero, part);
    mean *= inv;
  }
  float var = 0.0f;
#pragma unroll
  for (int k = 0; k < R; ++k)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float& d = u[k * V + i];
      d = (k * TG + lane) * V + i < gs ? d - mean : 0.0f;
      var += d * d;
    }
  group_sum<TG>(var, zero, part);
  const float r = 1.0f / sqrtf(var * inv + p.eps);
#pragma unroll
  for (int i = 0; i < R * V; ++i) u[i] *= r;
  return r;
}

// Forward: TG lanes share a group of a row and walk p.per rows of it; a
// workgroup of 256 holds 256 / TG of them, numbered (block of rows, group).
// Bound by memory: 32768 x 2560 gated bf16 in 98 us, 5.1 TB/s (122 us with the
// weights read a channel at a time).
template <typename T, int V, int TG, int R, bool Z>
__global__ __launch_bounds__(256) void k_norm(NormParams p) {
  __shared__ float part[8];
  const int lane = threadIdx.x & (TG - 1);
  const uint32_t item = blockIdx.x * uint32_t(256 / TG) + threadIdx.x / TG;   // the host keeps them below 2^31
  const uint32_t block = item / uint32_t(p.G), group = item % uint32_t(p.G);
  const int64_t row0 = block * p.per, c0 = group * p.gs;
  const int64_t end = row0 + p.per < p.rows ? row0 + p.per : p.rows;
  if (row0 >= end) return;
  const int gs = int(p.gs);
  const float inv = 1.0f / float(gs);
  float w[R * V], b[R * V];
  load_affine<V, R, TG>(p, c0, lane, w, b);
  Slice<T, V, R> x, z;
  const T* px = static_cast<const T*>(p.x) + row0 * p.xs + c0;
  const T* pz = Z ? static_cast<const T*>(p.z) + row0 * p.zs + c0 : nullptr;
  T* py = static_cast<T*>(p.y) + row0 * p.C + c0;
  x.template load<TG>(px, lane, gs);
  if constexpr (Z) z.template load<TG>(pz, lane, gs);
  for (int64_t row = row0; row < end; ++row) {
    Slice<T, V, R> nx, nz;
    const bool more = row + 1 < end;   // the next row is on its way while this one is worked on
    if (more) {
      nx.template load<TG>(px += p.xs, lane, gs);
      if constexpr (Z) nz.template load<TG>(pz += p.zs, lane, gs);
    }
    if (Z && p.mode == kGateFirst) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) x.v[i] *= z.v[i] * sigmoid(z.v[i]);
    }
    normalize<V, R, TG>(x.v, lane, p, inv, part);
#pragma unroll
    for (int i = 0; i < R * V; ++i) x.v[i] = x.v[i] * w[i] + b[i];
    if (Z && p.mode == kGate) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) x.v[i] *= z.v[i] * sigmoid(z.v[i]);
    }
    if (!Z && p.mode == kSilu) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) x.v[i] *= sigmoid(x.v[i]);
    }
    x.template store<TG>(py, lane, gs);
    py += p.C;
    if (more) {
      x = nx;
      if constexpr (Z) z = nz;
    }
  }
}

// Backward, the same walk: dx (and dz) of every row, and the sums over the
// block's rows for the gradients of weight and bias.  Bound by memory: 16384 x
// 1536 gated fp32 in 93 us, 5.4 TB/s.
template <typename T, int V, int TG, int R, bool Z>
__global__ __launch_bounds__(256) void k_norm_bwd(NormParams p) {
  __shared__ float part[8];
  const int lane = threadIdx.x & (TG - 1);
  const uint32_t item = blockIdx.x * uint32_t(256 / TG) + threadIdx.x / TG;
  const uint32_t block = item / uint32_t(p.G), group = item % uint32_t(p.G);
  const int64_t row0 = block * p.per, c0 = group * p.gs;
  const int64_t end = row0 + p.per < p.rows ? row0 + p.per : p.rows;
  if (row0 >= end) return;
  const int gs = int(p.gs);
  const float inv = 1.0f / float(gs);
  float w[R * V], b[R * V], dw[R * V], db[R * V];
  load_affine<V, R, TG>(p, c0, lane, w, b);
#pragma unroll
  for (int i = 0; i < R * V; ++i) dw[i] = db[i] = 0.0f;
  const T* px = static_cast<const T*>(p.x) + row0 * p.xs + c0;
  const T* pd = static_cast<const T*>(p.dy) + row0 * p.ds + c0;
  const T* pz = Z ? static_cast<const T*>(p.z) + row0 * p.zs + c0 : nullptr;
  T* py = static_cast<T*>(p.y) + row0 * p.C + c0;
  T* pdz = Z ? static_cast<T*>(p.dz) + row0 * p.C + c0 : nullptr;
  Slice<T, V, R> x, d, z;
  x.template load<TG>(px, lane, gs);
  d.template load<TG>(pd, lane, gs);
  if constexpr (Z) z.template load<TG>(pz, lane, gs);
  for (int64_t row = row0; row < end; ++row) {
    Slice<T, V, R> nx, nd, nz;
    const bool more = row + 1 < end;
    if (more) {
      nx.template load<TG>(px += p.xs, lane, gs);
      nd.template load<TG>(pd += p.ds, lane, gs);
      if constexpr (Z) nz.template load<TG>(pz += p.zs, lane, gs);
    }
    float n[R * V];
#pragma unroll
    for (int i = 0; i < R * V; ++i) n[i] = x.v[i];
    if (Z && p.mode == kGateFirst) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) n[i] *= z.v[i] * sigmoid(z.v[i]);
    }
    const float r = normalize<V, R, TG>(n, lane, p, inv, part);
    // d becomes da; in the gate mode z becomes dz
    if (Z && p.mode == kGate) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) {
        const float s = sigmoid(z.v[i]), a = n[i] * w[i] + b[i], dy = d.v[i];
        d.v[i] = dy * (z.v[i] * s);
        z.v[i] = dy * a * (s * (1.0f + z.v[i] * (1.0f - s)));
      }
    }
    if (!Z && p.mode == kSilu) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) {
        const float a = n[i] * w[i] + b[i], s = sigmoid(a);
        d.v[i] *= s * (1.0f + a * (1.0f - s));
      }
    }
    float sd = 0.0f, sdn = 0.0f;
#pragma unroll
    for (int i = 0; i < R * V; ++i) {
      dw[i] += d.v[i] * n[i];
      db[i] += d.v[i];
      d.v[i] *= w[i];   // dn
      sd += d.v[i];
      sdn += d.v[i] * n[i];
    }
    group_sum<TG>(sd, sdn, part);
    sd = p.rms ? 0.0f : sd * inv;
    sdn *= inv;
#pragma unroll
    for (int i = 0; i < R * V; ++i) d.v[i] = r * (d.v[i] - sd - n[i] * sdn);   // du
    if (Z && p.mode == kGateFirst) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) {
        const float s = sigmoid(z.v[i]), du = d.v[i];
        d.v[i] = du * (z.v[i] * s);
        z.v[i] = du * x.v[i] * (s * (1.0f + z.v[i] * (1.0f - s)));
      }
    }
    d.template store<TG>(py, lane, gs);
    py += p.C;
    if constexpr (Z) {
      z.template store<TG>(pdz, lane, gs);
      pdz += p.C;
    }
    if (more) {
      x = nx;
      d = nd;
      if constexpr (Z) z = nz;
    }
  }
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int c = (k * TG + lane) * V;
    if (c >= gs) continue;
    const int64_t at = int64_t(block) * p.C + c0 + c;
    if constexpr (V == 1) {
      if (p.dw) p.dw[at] = dw[k];
      if (p.db) p.db[at] = db[k];
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 4) {
        const int j = k * V + i;
        if (p.dw) *reinterpret_cast<float4*>(p.dw + at + i) = make_float4(dw[j], dw[j + 1], dw[j + 2], dw[j + 3]);
        if (p.db) *reinterpret_cast<float4*>(p.db + at + i) = make_float4(db[j], db[j + 1], db[j + 2], db[j + 3]);
      }
    }
  }
}

// Groups too long for registers: a workgroup to each, its rows read again for
// every pass over them (from the caches), a lane per channel in turn.
template <typename T>
__device__ __forceinline__ float long_input(const NormParams& p, int64_t row, int64_t c) {
  const float x = ld(static_cast<const T*>(p.x) + row * p.xs + c);
  if (p.mode != kGateFirst) return x;
  const float z = ld(static_cast<const T*>(p.z) + row * p.zs + c);
  return x * (z * sigmoid(z));
}

template <typename T>
__device__ __forceinline__ void long_stats(const NormParams& p, int64_t row, int64_t c0, float inv, float* mean,
                                           float* r, float* part) {
  float m = 0.0f, v = 0.0f, zero = 0.0f;
  if (!p.rms) {
    for (int64_t i = threadIdx.x; i < p.gs; i += 256) m += long_input<T>(p, row, c0 + i);
    group_sum<256>(m, zero, part);
    m *= inv;
  }
  for (int64_t i = threadIdx.x; i < p.gs; i += 256) {
    const float d = long_input<T>(p, row, c0 + i) - m;
    v += d * d;
  }
  group_sum<256>(v, zero, part);
  *mean = m;
  *r = 1.0f / sqrtf(v * inv + p.eps);
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_long(NormParams p) {
  __shared__ float part[8];
  const int64_t row = blockIdx.x / uint32_t(p.G), c0 = blockIdx.x % uint32_t(p.G) * p.gs;
  float mean, r;
  long_stats<T>(p, row, c0, 1.0f / float(p.gs), &mean, &r, part);
  for (int64_t i = threadIdx.x; i < p.gs; i += 256) {
    const int64_t c = c0 + i;
    float a = (long_input<T>(p, row, c) - mean) * r;
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
__device__ __forceinline__ float long_da(const NormParams& p, int64_t row, int64_t c, float mean, float r, float* n,
                                         float* dz) {
  *n = (long_input<T>(p, row, c) - mean) * r;
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
__global__ __launch_bounds__(256) void k_norm_bwd_long(NormParams p) {
  __shared__ float part[8];
  const int64_t block = blockIdx.x / uint32_t(p.G), c0 = blockIdx.x % uint32_t(p.G) * p.gs;
  const int64_t row0 = block * p.per, end = row0 + p.per < p.rows ? row0 + p.per : p.rows;
  const float inv = 1.0f / float(p.gs);
  for (int64_t row = row0; row < end; ++row) {
    float mean, r;
    long_stats<T>(p, row, c0, inv, &mean, &r, part);
    float sd = 0.0f, sdn = 0.0f, n, dz = 0.0f;
    for (int64_t i = threadIdx.x; i < p.gs; i += 256) {
      const int64_t c = c0 + i, at = block * p.C + c;
      const float da = long_da<T>(p, row, c, mean, r, &n, &dz), dn = da * (p.w ? p.w[c] : 1.0f);
      sd += dn;
      sdn += dn * n;
      // the block's sums, this lane's channels from row to row
      if (p.dw) p.dw[at] = (row == row0 ? 0.0f : p.dw[at]) + da * n;
      if (p.db) p.db[at] = (row == row0 ? 0.0f : p.db[at]) + da;
    }
    group_sum<256>(sd, sdn, part);
    sd = p.rms ? 0.0f : sd * inv;
    sdn *= inv;
    for (int64_t i = threadIdx.x; i < p.gs; i += 256) {
      const int64_t c = c0 + i;
      const float dn = long_da<T>(p, row, c, mean, r, &n, &dz) * (p.w ? p.w[c] : 1.0f);
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
}

// The blocks' sums of dweight and dbias (blocks, C) into one, in order: 16 lanes
// of a workgroup share a column, each with every 16th block, and join in LDS.
// blockIdx.y: which of the two.
struct ColsParams {
  const float* in[2];
  float* out[2];
  int64_t blocks, C;
};

static __global__ __launch_bounds__(256) void k_norm_cols(ColsParams p) {
  __shared__ float part[16][17];
  const float* in = p.in[blockIdx.y];
  float* out = p.out[blockIdx.y];
  if (!out) return;
  const int col = threadIdx.x & 15, lane = threadIdx.x >> 4;
  const int64_t c = int64_t(blockIdx.x) * 16 + col, C = p.C, blocks = p.blocks;
  float s = 0.0f;
  if (c < C) {
    int64_t k = lane;
    for (; k + 112 < blocks; k += 128) {
      float a[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) a[u] = in[(k + 16 * u) * C + c];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += a[u];
    }
    for (; k < blocks; k += 16) s += in[k * C + c];
  }
  part[lane][col] = s;
  __syncthreads();
  if (lane == 0 && c < C) {
    float t = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) t += part[k][col];
    out[c] = t;
  }
}

}  // namespace ssmn
