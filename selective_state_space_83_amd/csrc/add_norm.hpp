// add_norm.hpp -- gfx950 device code of the residual's addition with the
// root-mean-square norm, row by row:
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//
// in x's type, or as e4m3 values q = round(y / scale) with scale = max|y| / 448
// of each block of channels; and its gradients, with n = s r:
//   dn = dy w,  ds = dsum + r (dn - n mean(dn n)),  dw = sum_rows dy n.
#pragma once

#include "group_norm.hpp"

namespace ssma {

using ssmn::bf16_t;
using ssmn::group_sum;
using ssmn::ld;
using ssmn::st;

struct fp8_t {   // a byte that holds an e4m3 value
  uint8_t v;
};

constexpr float kE4m3Max = 448.0f;

struct AddNormParams {
  const void* x;
  const void* res;       // or null
  const float* w;        // or null
  void* sum;             // or null
  void* y;
  float* scale;          // e4m3: (rows, nblk)
  int64_t rows, C;
  int64_t xs, rs;        // row strides of x and the residual
  int64_t per;           // rows of a block: a lane walks them with its channels' weights in registers
  int32_t block, nblk;   // channels per scale (C: one scale per row) and scales per row
  float eps;
};

struct AddNormBwdParams {
  const void* sum;
  const void* dy;
  const void* dsum;      // or null
  const float* w;        // or null
  void* dx;
  void* dres;            // or null
  float* dw;             // (blocks of rows, C), each block's sums over its rows; or null
  int64_t rows, C;
  int64_t ss, ds, gs;    // row strides of sum, dy and dsum
  int64_t per;
  float eps;
};

// V neighbouring channels at p: V = 1, or 16 bytes' worth of the narrowest type
// of the row (a wider one takes two loads).
template <int V>
__device__ __forceinline__ void load_v(float* v, const float* p) {
  if constexpr (V == 1) {
    v[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 u = *reinterpret_cast<const float4*>(p + i);
      v[i] = u.x;
      v[i + 1] = u.y;
      v[i + 2] = u.z;
      v[i + 3] = u.w;
    }
  }
}
template <int V>
__device__ __forceinline__ void load_v(float* v, const bf16_t* p) {
  if constexpr (V == 1) {
    v[0] = ld(p);
  } else {
    static_assert(V == 8 || V == 4, "16 or 8 bytes of bf16");
    uint32_t a[V / 2];
    if constexpr (V == 8) {
      const uint4 u = *reinterpret_cast<const uint4*>(p);
      a[0] = u.x;
      a[1] = u.y;
      a[2] = u.z;
      a[3] = u.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(p);
      a[0] = u.x;
      a[1] = u.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
    }
  }
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float* v) {
  if constexpr (V == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store_v(bf16_t* p, const float* v) {
  if constexpr (V == 1) {
    st(p, v[0]);
  } else {
    typedef __bf16 bf16s __attribute__((ext_vector_type(V)));
    bf16s u;
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = static_cast<__bf16>(v[i]);
    *reinterpret_cast<bf16s*>(p) = u;
  }
}

// Within +-448 (a product with the scale's reciprocal may round past it); NaN stays.
__device__ __forceinline__ float to_range(float v) {
  return v != v ? v : __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max);
}
// To e4m3, to nearest even.
template <int V>
__device__ __forceinline__ void store_v(fp8_t* p, const float* v) {
  if constexpr (V == 1) {
    p->v = uint8_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[0], 0.0f, 0, false));
  } else {
    uint32_t u[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i], v[4 * i + 1], 0, false);
      u[i] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2], v[4 * i + 3], lo, true));
    }
    if constexpr (V == 8)
      *reinterpret_cast<uint2*>(p) = make_uint2(u[0], u[1]);
    else
      *reinterpret_cast<uint32_t*>(p) = u[0];
  }
}

// The scale of a block whose largest magnitude is top, and its reciprocal.
__device__ __forceinline__ float scale_of(float top, float* inverse) {
  const float s = top > 0.0f ? fmaxf(top / kE4m3Max, 0x1p-126f) : 1.0f;
  *inverse = 1.0f / s;
  return s;
}

template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
  return fmaxf(v, __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true)));
}
// Largest value (of values not below 0) over `n` neighbouring lanes, 1 to 64, for all of them.
__device__ __forceinline__ float lanes_max(float v, int n) {
  if (n >= 2) v = dpp_max<0xB1>(v);
  if (n >= 4) v = dpp_max<0x4E>(v);
  if (n >= 8) v = dpp_max<0x141>(v);
  if (n >= 16) v = dpp_max<0x140>(v);
  if (n >= 32) v = fmaxf(v, __shfl_xor(v, 16));
  if (n >= 64) v = fmaxf(v, __shfl_xor(v, 32));
  return v;
}
// Over the TG lanes that share a row; with 256 the workgroup's waves join in LDS.
template <int TG>
__device__ __forceinline__ float row_max(float v, float* part) {
  v = lanes_max(v, TG < 64 ? TG : 64);
  if constexpr (TG == 256) {
    __syncthreads();   // the last use of part
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  }
  return v;
}

// A lane's channels of a row, R times V of them, the TG lanes of a row taking turns;
// 0 past the end.
template <int V, int R, int TG, typename T>
__device__ __forceinline__ void load_row(float (&v)[R * V], const T* p, int lane, int C) {
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int c = (k * TG + lane) * V;
    if (c < C) {
      load_v<V>(v + k * V, p + c);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) v[k * V + i] = 0.0f;
    }
  }
}
template <int V, int R, int TG, typename T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[R * V], int lane, int C) {
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int c = (k * TG + lane) * V;
    if (c < C) store_v<V>(p + c, v + k * V);
  }
}

// Forward: TG lanes share a row and walk p.per rows; a workgroup of 256 holds
// 256 / TG of them.
template <typename InT, typename ResT, typename OutT, int V, int TG, int R>
__global__ __launch_bounds__(256) void k_add_norm(AddNormParams p) {
  constexpr bool kQuant = sizeof(OutT) == 1;
  __shared__ float part[8];
  const int lane = threadIdx.x & (TG - 1);
  const int64_t row0 = (int64_t(blockIdx.x) * (256 / TG) + threadIdx.x / TG) * p.per;
  const int64_t end = row0 + p.per < p.rows ? row0 + p.per : p.rows;
  if (row0 >= end) return;
  const int C = int(p.C);
  const float inv = 1.0f / float(C);
  float w[R * V];
#pragma unroll
  for (int i = 0; i < R * V; ++i) w[i] = 1.0f;
  if (p.w) load_row<V, R, TG>(w, p.w, lane, C);
  const InT* px = static_cast<const InT*>(p.x) + row0 * p.xs;
  const ResT* pr = static_cast<const ResT*>(p.res) + row0 * p.rs;
  float x[R * V], q[R * V];
  load_row<V, R, TG>(x, px, lane, C);
  if (p.res) load_row<V, R, TG>(q, pr, lane, C);
  for (int64_t row = row0; row < end; ++row) {
    if (p.res) {
#pragma unroll
      for (int i = 0; i < R * V; ++i) x[i] += q[i];
    }
    float nx[R * V];
    const bool more = row + 1 < end;   // the next row is on its way while this one is worked on
    if (more) {
      load_row<V, R, TG>(nx, px += p.xs, lane, C);
      if (p.res) load_row<V, R, TG>(q, pr += p.rs, lane, C);
    }
    if (p.sum) store_row<V, R, TG>(static_cast<ResT*>(p.sum) + row * p.C, x, lane, C);
    float ss = 0.0f, zero = 0.0f;
#pragma unroll
    for (int i = 0; i < R * V; ++i) ss += x[i] * x[i];
    group_sum<TG>(ss, zero, part);
    const float r = 1.0f / sqrtf(ss * inv + p.eps);
#pragma unroll
    for (int i = 0; i < R * V; ++i) x[i] = x[i] * r * w[i];
    if constexpr (kQuant) {
      float top[R];
#pragma unroll
      for (int k = 0; k < R; ++k) {
        top[k] = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) top[k] = fmaxf(top[k], fabsf(x[k * V + i]));
      }
      float* ps = p.scale + row * p.nblk;
      if (p.nblk == 1) {
#pragma unroll
        for (int k = 1; k < R; ++k) top[0] = fmaxf(top[0], top[k]);
        float inverse;
        const float s = scale_of(row_max<TG>(top[0], part), &inverse);
        if (lane == 0) *ps = s;
#pragma unroll
        for (int i = 0; i < R * V; ++i) x[i] = to_range(x[i] * inverse);
      } else {
        // a block is the same turn of block / V neighbouring lanes (the host sees to it)
        const int lanes = p.block / V;
#pragma unroll
        for (int k = 0; k < R; ++k) {
          float inverse;
          const float s = scale_of(lanes_max(top[k], lanes), &inverse);
          const int c = (k * TG + lane) * V;
          if ((lane & (lanes - 1)) == 0 && c < C) ps[c / p.block] = s;
#pragma unroll
          for (int i = 0; i < V; ++i) x[k * V + i] = to_range(x[k * V + i] * inverse);
        }
      }
    }
    store_row<V, R, TG>(static_cast<OutT*>(p.y) + row * p.C, x, lane, C);
#pragma unroll
    for (int i = 0; i < R * V; ++i) x[i] = nx[i];
  }
}

// Rows too long for registers, and blocks of channels that no lane group of one turn
// covers: a workgroup to a row, read again for every pass over it (from the caches).
// Nothing is written before the last pass, which reads an element before it writes
// it: the sum may take the residual's place.
template <typename InT, typename ResT>
__device__ __forceinline__ float long_sum(const AddNormParams& p, int64_t row, int64_t c) {
  const float x = ld(static_cast<const InT*>(p.x) + row * p.xs + c);
  return p.res ? x + ld(static_cast<const ResT*>(p.res) + row * p.rs + c) : x;
}

template <typename InT, typename ResT, typename OutT>
__global__ __launch_bounds__(256) void k_add_norm_long(AddNormParams p) {
  constexpr bool kQuant = sizeof(OutT) == 1;
  __shared__ float part[8];
  const int64_t row = blockIdx.x;
  float ss = 0.0f, zero = 0.0f;
  for (int64_t c = threadIdx.x; c < p.C; c += 256) {
    const float s = long_sum<InT, ResT>(p, row, c);
    ss += s * s;
  }
  group_sum<256>(ss, zero, part);
  const float r = 1.0f / sqrtf(ss * (1.0f / float(p.C)) + p.eps);
  ResT* sum = static_cast<ResT*>(p.sum) + row * p.C;
  OutT* y = static_cast<OutT*>(p.y) + row * p.C;
  auto value = [&](float s, int64_t c) { return s * r * (p.w ? p.w[c] : 1.0f); };
  auto finish = [&](int64_t c, float inverse) {
    const float s = long_sum<InT, ResT>(p, row, c);
    float v = value(s, c);
    if constexpr (kQuant) v = to_range(v * inverse);
    if (p.sum) st(sum + c, s);
    store_v<1>(y + c, &v);
  };
  if constexpr (!kQuant) {
    for (int64_t c = threadIdx.x; c < p.C; c += 256) finish(c, 1.0f);
  } else if (p.nblk == 1) {
    float top = 0.0f, inverse;
    for (int64_t c = threadIdx.x; c < p.C; c += 256) top = fmaxf(top, fabsf(value(long_sum<InT, ResT>(p, row, c), c)));
    const float s = scale_of(row_max<256>(top, part), &inverse);
    if (threadIdx.x == 0) p.scale[row] = s;
    for (int64_t c = threadIdx.x; c < p.C; c += 256) finish(c, inverse);
  } else {
    // a wave to a block of channels
    const int lane = threadIdx.x & 63;
    for (int64_t k = threadIdx.x >> 6; k < p.nblk; k += 4) {
      const int64_t c0 = k * p.block, c1 = c0 + p.block < p.C ? c0 + p.block : p.C;
      float top = 0.0f, inverse;
      for (int64_t c = c0 + lane; c < c1; c += 64) top = fmaxf(top, fabsf(value(long_sum<InT, ResT>(p, row, c), c)));
      const float s = scale_of(lanes_max(top, 64), &inverse);
      if (lane == 0) p.scale[row * p.nblk + k] = s;
      for (int64_t c = c0 + lane; c < c1; c += 64) finish(c, inverse);
    }
  }
}

// Backward, the same walk: ds of every row, and the sums over the block's rows
// for the weight's gradient.
template <typename InT, typename SumT, int V, int TG, int R>
__global__ __launch_bounds__(256) void k_add_norm_bwd(AddNormBwdParams p) {
  __shared__ float part[8];
  const int lane = threadIdx.x & (TG - 1);
  const int64_t block = int64_t(blockIdx.x) * (256 / TG) + threadIdx.x / TG;
  const int64_t row0 = block * p.per;
  const int64_t end = row0 + p.per < p.rows ? row0 + p.per : p.rows;
  if (row0 >= end) return;
  const int C = int(p.C);
  const float inv = 1.0f / float(C);
  float w[R * V], dw[R * V];
#pragma unroll
  for (int i = 0; i < R * V; ++i) {
    w[i] = 1.0f;
    dw[i] = 0.0f;
  }
  if (p.w) load_row<V, R, TG>(w, p.w, lane, C);
  const SumT* ps = static_cast<const SumT*>(p.sum) + row0 * p.ss;
  const InT* pd = static_cast<const InT*>(p.dy) + row0 * p.ds;
  const SumT* pg = static_cast<const SumT*>(p.dsum) + row0 * p.gs;
  float s[R * V], d[R * V], g[R * V];
  load_row<V, R, TG>(s, ps, lane, C);
  load_row<V, R, TG>(d, pd, lane, C);
#pragma unroll
  for (int i = 0; i < R * V; ++i) g[i] = 0.0f;
  if (p.dsum) load_row<V, R, TG>(g, pg, lane, C);
  for (int64_t row = row0; row < end; ++row) {
    float ns[R * V], nd[R * V], ng[R * V];
    const bool more = row + 1 < end;
    if (more) {
      load_row<V, R, TG>(ns, ps += p.ss, lane, C);
      load_row<V, R, TG>(nd, pd += p.ds, lane, C);
      if (p.dsum) load_row<V, R, TG>(ng, pg += p.gs, lane, C);
    }
    float ss = 0.0f, sdn = 0.0f;
#pragma unroll
    for (int i = 0; i < R * V; ++i) {
      ss += s[i] * s[i];
      sdn += d[i] * w[i] * s[i];
    }
    group_sum<TG>(ss, sdn, part);
    const float r = 1.0f / sqrtf(ss * inv + p.eps);
    const float m = sdn * inv * r;   // mean(dn n)
#pragma unroll
    for (int i = 0; i < R * V; ++i) {
      const float n = s[i] * r;
      dw[i] += d[i] * n;
      g[i] += r * (d[i] * w[i] - n * m);
    }
    store_row<V, R, TG>(static_cast<InT*>(p.dx) + row * p.C, g, lane, C);
    if constexpr (sizeof(SumT) != sizeof(InT))
      if (p.dres) store_row<V, R, TG>(static_cast<SumT*>(p.dres) + row * p.C, g, lane, C);
#pragma unroll
    for (int i = 0; i < R * V; ++i) {
      s[i] = ns[i];
      d[i] = nd[i];
      g[i] = p.dsum ? ng[i] : 0.0f;
    }
  }
  if (p.dw) store_row<V, R, TG>(p.dw + block * p.C, dw, lane, C);
}

template <typename InT, typename SumT>
__global__ __launch_bounds__(256) void k_add_norm_bwd_long(AddNormBwdParams p) {
  __shared__ float part[8];
  const int64_t row0 = blockIdx.x * p.per, end = row0 + p.per < p.rows ? row0 + p.per : p.rows;
  float* dw = p.dw ? p.dw + blockIdx.x * p.C : nullptr;
  for (int64_t row = row0; row < end; ++row) {
    const SumT* ps = static_cast<const SumT*>(p.sum) + row * p.ss;
    const InT* pd = static_cast<const InT*>(p.dy) + row * p.ds;
    const SumT* pg = static_cast<const SumT*>(p.dsum) + row * p.gs;
    float ss = 0.0f, sdn = 0.0f;
    for (int64_t c = threadIdx.x; c < p.C; c += 256) {
      const float s = ld(ps + c);
      ss += s * s;
      sdn += ld(pd + c) * (p.w ? p.w[c] : 1.0f) * s;
    }
    group_sum<256>(ss, sdn, part);
    const float inv = 1.0f / float(p.C), r = 1.0f / sqrtf(ss * inv + p.eps), m = sdn * inv * r;
    for (int64_t c = threadIdx.x; c < p.C; c += 256) {
      const float n = ld(ps + c) * r, dy = ld(pd + c);
      // the block's sums, this lane's channels from row to row
      if (dw) dw[c] = (row == row0 ? 0.0f : dw[c]) + dy * n;
      const float g = (p.dsum ? ld(pg + c) : 0.0f) + r * (dy * (p.w ? p.w[c] : 1.0f) - n * m);
      st(static_cast<InT*>(p.dx) + row * p.C + c, g);
      if constexpr (sizeof(SumT) != sizeof(InT))
        if (p.dres) st(static_cast<SumT*>(p.dres) + row * p.C + c, g);
    }
  }
}

}  // namespace ssma
