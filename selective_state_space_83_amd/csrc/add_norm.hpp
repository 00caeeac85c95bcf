// add_norm.hpp -- gfx950 device code of the residual's addition with the
// root-mean-square norm, row by row:
//
//   s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r w
//
// in x's type, or as e4m3 values q = round(y / scale) with scale = max|y| / 448
// of each block of channels; and its gradients, with n = s r:
//   dn = dy w,  ds = dsum + r (dn - n mean(dn n)),  dw = sum_rows dy n,
// from the sum as it was kept, or from x and the residual, whose sum is formed again as
// the forward pass forms it, before any rounding to the sum's type.
#pragma once

#include <type_traits>

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
  int32_t block, nblk;   // channels per scale (C: one scale per row) and scales per row
  int32_t stream;        // outputs larger than the L2 caches
  float eps;
};

struct AddNormBwdParams {
  const void* sum;       // the kept sum, or x where res is given
  const void* res;       // or null
  const void* dy;
  const void* dsum;      // or null
  const float* w;        // or null
  void* dx;
  void* dres;            // or null
  float* dw;             // (blocks of rows, C), each block's sums over its rows; or null
  int64_t rows, C;
  int64_t ss, rs, ds, gs;   // row strides of sum, the residual, dy and dsum
  int64_t per;           // rows of a block: a lane walks them with its channels' weights in registers
  int32_t stream;        // as AddNormParams'
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
// The same as they lie in memory: what is requested ahead takes half the registers
// with bf16.
template <typename T, int V>
struct Raw {
  static constexpr int W = V * int(sizeof(T)) / 4 > 0 ? V * int(sizeof(T)) / 4 : 1;
  uint32_t w[W];
  // KEEP: in the caches, for rows that another tile reads too; else past them
  template <bool KEEP = false>
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      w[0] = __builtin_bit_cast(uint32_t, ld(p));
    } else {
      constexpr int L = W < 4 ? W : 4;
      typedef uint32_t words __attribute__((ext_vector_type(L)));
#pragma unroll
      for (int i = 0; i < W; i += L) {
        const words* q = reinterpret_cast<const words*>(p) + i / L;
        const words u = KEEP ? *q : __builtin_nontemporal_load(q);
#pragma unroll
        for (int k = 0; k < L; ++k) w[i + k] = u[k];
      }
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0;
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (V == 1 || sizeof(T) == 4)
      return __uint_as_float(w[i]);
    else
      return __uint_as_float(i % 2 == 0 ? w[i / 2] << 16 : w[i / 2] & 0xffff0000u);
  }
};

// STREAM: past the caches, for outputs that they cannot hold until they are read.
template <int V, bool STREAM = false>
__device__ __forceinline__ void store_v(float* p, const float* v) {
  if constexpr (V == 1) {
    *p = v[0];
  } else {
    typedef float f32x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const f32x4 u = {v[i], v[i + 1], v[i + 2], v[i + 3]};
      if constexpr (STREAM)
        __builtin_nontemporal_store(u, reinterpret_cast<f32x4*>(p + i));
      else
        *reinterpret_cast<f32x4*>(p + i) = u;
    }
  }
}
template <int V, bool STREAM = false>
__device__ __forceinline__ void store_v(bf16_t* p, const float* v) {
  if constexpr (V == 1) {
    st(p, v[0]);
  } else {
    typedef __bf16 bf16s __attribute__((ext_vector_type(V)));
    bf16s u;
#pragma unroll
    for (int i = 0; i < V; ++i) u[i] = static_cast<__bf16>(v[i]);
    if constexpr (STREAM)
      __builtin_nontemporal_store(u, reinterpret_cast<bf16s*>(p));
    else
      *reinterpret_cast<bf16s*>(p) = u;
  }
}

// Within +-448 (a product with the scale's reciprocal may round past it); NaN stays.
__device__ __forceinline__ float to_range(float v) {
  return v != v ? v : __builtin_amdgcn_fmed3f(v, -kE4m3Max, kE4m3Max);
}
// To e4m3, to nearest even.
template <int V, bool STREAM = false>
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
    typedef uint32_t words __attribute__((ext_vector_type(V / 4)));
    words q;
#pragma unroll
    for (int i = 0; i < V / 4; ++i) q[i] = u[i];
    if constexpr (STREAM)
      __builtin_nontemporal_store(q, reinterpret_cast<words*>(p));
    else
      *reinterpret_cast<words*>(p) = q;
  }
}

// To 8 bits: y is p m with p = (s 2^e) w and r = 2^e m, so that a value in units of its
// block's scale, p (448 / max|p|), does not depend on the rounding of r.  The product's
// rest and the quotient's go along, and q is rounded but once before its 8 bits: of
// 7.9 million values 3 lay a step off those of 64 bits, and 7 with every operation
// rounded.  32768 x 2560 to 8 bits takes as long either way.
struct Unit {
  float up, m;   // 2^e, and r without it
  __device__ __forceinline__ explicit Unit(float r) {
    const uint32_t b = __float_as_uint(r);
    up = r != r ? r : __uint_as_float(b & 0x7f800000u);   // (a row of NaN has no largest value)
    m = __uint_as_float((b & 0x007fffffu) | 0x3f800000u);
  }
};
// The scale of a block whose largest |p| is top (of its numbers; 0 if it has none), and
// what takes p to q.
struct Step {
  float scale, c, rest;
  __device__ __forceinline__ Step(float top, const Unit& u) {
    const float y = top * u.m;
    scale = y > 0.0f ? fmaxf(y / kE4m3Max, 0x1p-126f) : 1.0f;
    rest = 0.0f;
    if (scale == 0x1p-126f || !(y > 0.0f)) {   // at its least, or a block of zeros
      c = u.m / scale;
    } else {
      c = kE4m3Max / top;
      if (c > 0.0f) rest = fmaf(-c, top, kE4m3Max) * (c * (1.0f / kE4m3Max));
    }
  }
  __device__ __forceinline__ float operator()(float s, float w) const {
    const float p = s * w, low = fmaf(s, w, -p);
    return to_range(fmaf(p, c, fmaf(p, rest, low * c)));
  }
};

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
template <int V, int R, int TG, bool STREAM = false, typename T>
__device__ __forceinline__ void store_row(T* p, const float (&v)[R * V], int lane, int C) {
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int c = (k * TG + lane) * V;
    if (c < C) store_v<V, STREAM>(p + c, v + k * V);
  }
}

// A row as it lies in memory.
template <typename T, int V, int R>
struct RawRow {
  Raw<T, V> v[R];
  template <int TG>
  __device__ __forceinline__ void load(const T* p, int lane, int C) {
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int c = (k * TG + lane) * V;
      v[k].clear();
      if (c < C) v[k].load(p + c);
    }
  }
  __device__ __forceinline__ float at(int i) const { return v[i / V].at(i % V); }
};

// Forward: TG lanes to a row, 256 / TG rows to a workgroup.  Bound by memory; rows
// enough are on their way in the waves a SIMD holds.  (A lane that walks 8 rows, the
// weights in registers and the next row requested ahead: 32768 x 2560 bf16 131 us
// for 120, to 8 bits with an fp32 residual 190 for 175.  Loads past the caches 116 ->
// 109 and 159 -> 147, outputs 118 -> 111 and 161 -> 147; those that the L2 caches hold
// are left there.)
template <typename InT, typename ResT, typename OutT, int V, int TG, int R>
__global__ __launch_bounds__(256) void k_add_norm(AddNormParams p) {
  constexpr bool kQuant = sizeof(OutT) == 1;
  __shared__ float part[8];
  const int lane = threadIdx.x & (TG - 1);
  const int64_t row = int64_t(blockIdx.x) * (256 / TG) + threadIdx.x / TG;
  if (row >= p.rows) return;
  const int C = int(p.C);
  float x[R * V];
  {
    RawRow<InT, V, R> a;
    RawRow<ResT, V, R> b;
    a.template load<TG>(static_cast<const InT*>(p.x) + row * p.xs, lane, C);
    if (p.res) b.template load<TG>(static_cast<const ResT*>(p.res) + row * p.rs, lane, C);
#pragma unroll
    for (int i = 0; i < R * V; ++i) x[i] = p.res ? a.at(i) + b.at(i) : a.at(i);
  }
  if (p.sum) {
    ResT* sum = static_cast<ResT*>(p.sum) + row * p.C;
    if (p.stream)
      store_row<V, R, TG, true>(sum, x, lane, C);
    else
      store_row<V, R, TG>(sum, x, lane, C);
  }
  float w[R * V];
#pragma unroll
  for (int i = 0; i < R * V; ++i) w[i] = 1.0f;
  if (p.w) load_row<V, R, TG>(w, p.w, lane, C);
  float ss = 0.0f, zero = 0.0f;
#pragma unroll
  for (int i = 0; i < R * V; ++i) ss += x[i] * x[i];
  group_sum<TG>(ss, zero, part);
  const float r = 1.0f / sqrtf(ss * (1.0f / float(C)) + p.eps);
  if constexpr (!kQuant) {
#pragma unroll
    for (int i = 0; i < R * V; ++i) x[i] = x[i] * r * w[i];
  } else {
    const Unit unit(r);
    float top[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      top[k] = 0.0f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        x[k * V + i] *= unit.up;
        top[k] = fmaxf(top[k], fabsf(x[k * V + i] * w[k * V + i]));
      }
    }
    float* ps = p.scale + row * p.nblk;
    if (p.nblk == 1) {
#pragma unroll
      for (int k = 1; k < R; ++k) top[0] = fmaxf(top[0], top[k]);
      const Step q(row_max<TG>(top[0], part), unit);
      if (lane == 0) *ps = q.scale;
#pragma unroll
      for (int i = 0; i < R * V; ++i) x[i] = q(x[i], w[i]);
    } else {
      // a block is the same turn of block / V neighbouring lanes (the host sees to it)
      const int lanes = p.block / V;
#pragma unroll
      for (int k = 0; k < R; ++k) {
        const Step q(lanes_max(top[k], lanes), unit);
        const int c = (k * TG + lane) * V;
        if ((lane & (lanes - 1)) == 0 && c < C) ps[c / p.block] = q.scale;
#pragma unroll
        for (int i = 0; i < V; ++i) x[k * V + i] = q(x[k * V + i], w[k * V + i]);
      }
    }
  }
  OutT* y = static_cast<OutT*>(p.y) + row * p.C;
  if (p.stream)
    store_row<V, R, TG, true>(y, x, lane, C);
  else
    store_row<V, R, TG>(y, x, lane, C);
}

// Rows too long for registers, and blocks of channels that no lane group of one turn
// covers: a workgroup to a row, read again for every pass over it (from the caches), V
// channels to a lane in turn.  Nothing is written before the last pass, which reads an
// element before it writes it: the sum may take the residual's place.
template <typename InT, typename ResT, typename OutT, int V>
__global__ __launch_bounds__(256) void k_add_norm_long(AddNormParams p) {
  constexpr bool kQuant = sizeof(OutT) == 1;
  __shared__ float part[8];
  const int64_t row = blockIdx.x;
  const InT* x = static_cast<const InT*>(p.x) + row * p.xs;
  const ResT* res = static_cast<const ResT*>(p.res) + row * p.rs;
  auto load = [&](float (&s)[V], int64_t c) {
    load_v<V>(s, x + c);
    if (p.res) {
      float q[V];
      load_v<V>(q, res + c);
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] += q[i];
    }
  };
  float ss = 0.0f, zero = 0.0f;
  for (int64_t c = threadIdx.x * V; c < p.C; c += 256 * V) {
    float s[V];
    load(s, c);
#pragma unroll
    for (int i = 0; i < V; ++i) ss += s[i] * s[i];
  }
  group_sum<256>(ss, zero, part);
  const float r = 1.0f / sqrtf(ss * (1.0f / float(p.C)) + p.eps);
  ResT* sum = static_cast<ResT*>(p.sum) + row * p.C;
  OutT* y = static_cast<OutT*>(p.y) + row * p.C;
  // s of V channels, and their weights
  auto values = [&](float (&s)[V], float (&w)[V], int64_t c) {
    load(s, c);
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = 1.0f;
    if (p.w) load_v<V>(w, p.w + c);
  };
  if constexpr (!kQuant) {
    for (int64_t c = threadIdx.x * V; c < p.C; c += 256 * V) {
      float s[V], w[V], v[V];
      values(s, w, c);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = s[i] * r * w[i];
      if (p.sum) store_v<V>(sum + c, s);
      store_v<V>(y + c, v);
    }
  } else {
    const Unit unit(r);
    auto largest = [&](float top, int64_t c) {
      float s[V], w[V];
      values(s, w, c);
#pragma unroll
      for (int i = 0; i < V; ++i) top = fmaxf(top, fabsf(s[i] * unit.up * w[i]));
      return top;
    };
    auto finish = [&](int64_t c, const Step& q) {
      float s[V], w[V], v[V];
      values(s, w, c);
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = q(s[i] * unit.up, w[i]);
      if (p.sum) store_v<V>(sum + c, s);
      store_v<V>(y + c, v);
    };
    if (p.nblk == 1) {
      float top = 0.0f;
      for (int64_t c = threadIdx.x * V; c < p.C; c += 256 * V) top = largest(top, c);
      const Step q(row_max<256>(top, part), unit);
      if (threadIdx.x == 0) p.scale[row] = q.scale;
      for (int64_t c = threadIdx.x * V; c < p.C; c += 256 * V) finish(c, q);
    } else {
      // a wave to a block of channels
      const int lane = threadIdx.x & 63;
      for (int64_t k = threadIdx.x >> 6; k < p.nblk; k += 4) {
        const int64_t c0 = k * p.block, c1 = c0 + p.block < p.C ? c0 + p.block : p.C;
        float top = 0.0f;
        for (int64_t c = c0 + lane * V; c < c1; c += 64 * V) top = largest(top, c);
        const Step q(lanes_max(top, 64), unit);
        if (lane == 0) p.scale[row * p.nblk + k] = q.scale;
        for (int64_t c = c0 + lane * V; c < c1; c += 64 * V) finish(c, q);
      }
    }
  }
}

// Backward: TG lanes walk the p.per rows of a block: ds of every row, and the sums
// over the block's rows for the weight's gradient.  (16384 x 1536 bf16 beside an fp32 sum,
// with the forward pass: loads past the caches 134 -> 125 us, stores of large outputs
// 131 -> 125.)  RES: s is x + residual (16384 x 1536 bf16: 55 us, from the kept sum 46).
template <typename InT, typename SumT, bool RES, int V, int TG, int R>
__global__ __launch_bounds__(256) void k_add_norm_bwd(AddNormBwdParams p) {
  using FirstT = std::conditional_t<RES, InT, SumT>;
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
  const FirstT* ps = static_cast<const FirstT*>(p.sum) + row0 * p.ss;
  const SumT* pr = static_cast<const SumT*>(p.res) + row0 * p.rs;
  const InT* pd = static_cast<const InT*>(p.dy) + row0 * p.ds;
  const SumT* pg = static_cast<const SumT*>(p.dsum) + row0 * p.gs;
  RawRow<FirstT, V, R> ns;
  RawRow<SumT, V, R> nr, ng;
  RawRow<InT, V, R> nd;
  auto request = [&] {
    ns.template load<TG>(ps, lane, C);
    if constexpr (RES) nr.template load<TG>(pr, lane, C);
    nd.template load<TG>(pd, lane, C);
    if (p.dsum) ng.template load<TG>(pg, lane, C);
  };
  request();
  for (int64_t row = row0; row < end; ++row) {
    float s[R * V], d[R * V], g[R * V];
#pragma unroll
    for (int i = 0; i < R * V; ++i) {
      s[i] = ns.at(i);
      if constexpr (RES) s[i] += nr.at(i);
      d[i] = nd.at(i);
      g[i] = p.dsum ? ng.at(i) : 0.0f;
    }
    if (row + 1 < end) {
      ps += p.ss;
      if constexpr (RES) pr += p.rs;
      pd += p.ds;
      pg += p.gs;
      request();
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
    InT* dx = static_cast<InT*>(p.dx) + row * p.C;
    SumT* dres = static_cast<SumT*>(p.dres) + row * p.C;
    if (p.stream) {
      store_row<V, R, TG, true>(dx, g, lane, C);
      if constexpr (sizeof(SumT) != sizeof(InT))
        if (p.dres) store_row<V, R, TG, true>(dres, g, lane, C);
    } else {
      store_row<V, R, TG>(dx, g, lane, C);
      if constexpr (sizeof(SumT) != sizeof(InT))
        if (p.dres) store_row<V, R, TG>(dres, g, lane, C);
    }
  }
  if (p.dw) store_row<V, R, TG>(p.dw + block * p.C, dw, lane, C);
}

// Rows too long for registers, read twice.
template <typename InT, typename SumT, bool RES, int V>
__global__ __launch_bounds__(256) void k_add_norm_bwd_long(AddNormBwdParams p) {
  using FirstT = std::conditional_t<RES, InT, SumT>;
  __shared__ float part[8];
  const int64_t row0 = blockIdx.x * p.per, end = row0 + p.per < p.rows ? row0 + p.per : p.rows;
  float* dw = p.dw ? p.dw + blockIdx.x * p.C : nullptr;
  for (int64_t row = row0; row < end; ++row) {
    const FirstT* ps = static_cast<const FirstT*>(p.sum) + row * p.ss;
    const SumT* pr = static_cast<const SumT*>(p.res) + row * p.rs;
    const InT* pd = static_cast<const InT*>(p.dy) + row * p.ds;
    const SumT* pg = static_cast<const SumT*>(p.dsum) + row * p.gs;
    auto values = [&](float (&s)[V], int64_t c) {
      load_v<V>(s, ps + c);
      if constexpr (RES) {
        float q[V];
        load_v<V>(q, pr + c);
#pragma unroll
        for (int i = 0; i < V; ++i) s[i] += q[i];
      }
    };
    auto weight = [&](float (&w)[V], int64_t c) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = 1.0f;
      if (p.w) load_v<V>(w, p.w + c);
    };
    float ss = 0.0f, sdn = 0.0f;
    for (int64_t c = threadIdx.x * V; c < p.C; c += 256 * V) {
      float s[V], d[V], w[V];
      values(s, c);
      load_v<V>(d, pd + c);
      weight(w, c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss += s[i] * s[i];
        sdn += d[i] * w[i] * s[i];
      }
    }
    group_sum<256>(ss, sdn, part);
    const float inv = 1.0f / float(p.C), r = 1.0f / sqrtf(ss * inv + p.eps), m = sdn * inv * r;
    for (int64_t c = threadIdx.x * V; c < p.C; c += 256 * V) {
      float s[V], d[V], w[V], g[V], sum[V];
      values(s, c);
      load_v<V>(d, pd + c);
      weight(w, c);
#pragma unroll
      for (int i = 0; i < V; ++i) g[i] = sum[i] = 0.0f;
      if (p.dsum) load_v<V>(g, pg + c);
      // the block's sums, this lane's channels from row to row
      if (dw && row > row0) load_v<V>(sum, dw + c);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float n = s[i] * r;
        sum[i] += d[i] * n;
        g[i] += r * (d[i] * w[i] - n * m);
      }
      if (dw) store_v<V>(dw + c, sum);
      store_v<V>(static_cast<InT*>(p.dx) + row * p.C + c, g);
      if constexpr (sizeof(SumT) != sizeof(InT))
        if (p.dres) store_v<V>(static_cast<SumT*>(p.dres) + row * p.C + c, g);
    }
  }
}

}  // namespace ssma
