// decay_attn.hpp -- gfx950 device code of decay attention, linear attention
// with a decay for each head:
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t       per (batch row, head)
//
// One kernel covers the forward and the gradients, which are the same sum with
// the roles changed.  With "rows" a, b (contracted, M wide) and c (N wide),
//
//   S_t = exp(g_t) S_{t-1} + b_t c_t^T,   out_t = S_t^T a_t      S (M, N)
//
//   forward   a, b, c = q, k, v          S = the state
//   dq        a, b, c = dout, v, k       S = the state, transposed
//   dv        a, b, c = k, q, dout       backward in time, S = G
//   dk        a, b, c = v, dout, q       backward in time, S = G transposed
//
// where G_t = q_t dout_t^T + exp(g_{t+1}) G_{t+1} is the state's gradient: going
// backward, token t's decay is that of its successor in time.
//
// The decay's gradient needs no state: dq_i.q_i and dk_i.k_i sum the same pairs
// (i, j <= i) by reader and by writer, so with u_i = dq_i.q_i, w_i = dk_i.k_i
// (per value head) and P the gradient's flow through the end of the sequence,
// P = <S_last, dh_last>,
//   dg_t = sum_{i >= t} (u_i - w_i) + P.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssma {

using bf16_t = uint16_t;

constexpr int kWave = 64;
constexpr float kLog2e = 1.4426950408889634f;
// exp of a decay below this is 0 in fp32; clamped there, sums of log decays
// stay finite and differences of them are defined (a reset is log decay -inf)
constexpr float kMinLogDecay = -128.0f;

__device__ __forceinline__ float ld(const float* p) { return *p; }
__device__ __forceinline__ float ld(const bf16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(*p) << 16);
}
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(bf16_t* p, float v) {
  *p = __builtin_bit_cast(bf16_t, static_cast<__bf16>(v));   // to nearest even
}

struct Rows {
  const void* p;
  int64_t sb, st, sh;   // elements between batch rows, tokens, heads
  int32_t per;          // value heads that read one of its heads
};

template <typename T>
__device__ __forceinline__ const T* row_base(const Rows& r, int64_t b, int64_t h) {
  return static_cast<const T*>(r.p) + b * r.sb + (h / r.per) * r.sh;
}

struct Decay {
  const void* p;
  int64_t sb, st, sh;
  int32_t bf16;
};

__device__ __forceinline__ float log_decay(const Decay& d, int64_t b, int64_t t, int64_t h) {
  const int64_t i = b * d.sb + t * d.st + h * d.sh;
  const float g = d.bf16 ? ld(static_cast<const bf16_t*>(d.p) + i) : static_cast<const float*>(d.p)[i];
  return g < kMinLogDecay ? kMinLogDecay : g;   // a NaN stays one
}

__device__ __forceinline__ int64_t live_tokens(const int32_t* lengths, int64_t b, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > L ? L : n;
}

struct MixParams {
  Rows a, b, c, x;       // x: rows like out, for the dots (dots null: unused)
  Decay g;
  const int32_t* lengths;
  const float* s0;       // state before the first token, or null
  float* s_last;         // state after the last, or null
  int64_t sm, sn;        // strides of S(m, n) within a head's state
  void* out;             // (B, L, H, N)
  float* dots;           // (tiles of N, B, L, H): out_t . x_t over the tile
  int64_t B, L, H;
  int32_t M, N;
  int32_t reverse;
};

// The recurrence as written: a lane holds a column of S.
template <typename T, typename OutT, int MP>
__global__ __launch_bounds__(kWave) void k_mix_simple(MixParams p) {
  const int lane = threadIdx.x;
  const int64_t bh = blockIdx.x, b = bh / p.H, h = bh % p.H;
  const int n = blockIdx.y * kWave + lane;
  const bool on = n < p.N;
  const T* pa = row_base<T>(p.a, b, h);
  const T* pb = row_base<T>(p.b, b, h);
  const T* pc = row_base<T>(p.c, b, h);
  const T* px = p.dots ? row_base<T>(p.x, b, h) : nullptr;
  OutT* out = static_cast<OutT*>(p.out) + (b * p.L * p.H + h) * p.N;
  float* dots = p.dots ? p.dots + (int64_t(blockIdx.y) * p.B + b) * p.L * p.H + h : nullptr;
  const int64_t len = live_tokens(p.lengths, b, p.L);
  const int64_t sbase = bh * p.M * p.N;
  float S[MP];
#pragma unroll
  for (int m = 0; m < MP; ++m)
    S[m] = (p.s0 && on && m < p.M) ? p.s0[sbase + m * p.sm + n * p.sn] : 0.0f;
  for (int64_t i = 0; i < len; ++i) {
    const int64_t t = p.reverse ? len - 1 - i : i;
    const float g = !p.reverse ? log_decay(p.g, b, t, h)
                               : t + 1 < len ? log_decay(p.g, b, t + 1, h) : 0.0f;
    const float e = expf(g);
    const float c = on ? ld(pc + t * p.c.st + n) : 0.0f;
    float acc = 0.0f;
#pragma unroll
    for (int m = 0; m < MP; ++m) {
      if (m < p.M) {
        S[m] = S[m] * e + ld(pb + t * p.b.st + m) * c;
        acc += S[m] * ld(pa + t * p.a.st + m);
      }
    }
    if (on) st(out + t * p.H * p.N + n, acc);
    if (dots) {
      float d = on ? acc * ld(px + t * p.x.st + n) : 0.0f;
#pragma unroll
      for (int w = 32; w; w >>= 1) d += __shfl_xor(d, w);
      if (lane == 0) dots[t * p.H] = d;
    }
  }
  if (on)
    for (int64_t t = len; t < p.L; ++t) st(out + t * p.H * p.N + n, 0.0f);
  if (p.s_last) {
    // going backward, the first token's own decay stands between G_0 and h0
    const float e = p.reverse && len > 0 ? expf(log_decay(p.g, b, 0, h)) : 1.0f;
#pragma unroll
    for (int m = 0; m < MP; ++m)
      if (on && m < p.M) p.s_last[sbase + m * p.sm + n * p.sn] = S[m] * e;
  }
}

struct DecayGradParams {
  const float* u;        // (utiles, B, L, H)
  const float* w;        // (wtiles, B, L, H)
  const float* s_last;   // (B, H, dk, dv), with dh_last; null: no flow through the end
  const float* dh_last;
  const int32_t* lengths;
  void* dg;              // (B, L, H)
  int64_t B, L, H, inner;
  int32_t utiles, wtiles, bf16;
};

// One wave per (batch row, head): the flow through the end, then the suffix sums.
static __global__ __launch_bounds__(kWave) void k_decay_grad_simple(DecayGradParams p) {
  const int lane = threadIdx.x;
  const int64_t bh = blockIdx.x, b = bh / p.H, h = bh % p.H;
  const int64_t len = live_tokens(p.lengths, b, p.L), n = p.B * p.L * p.H;
  double acc = 0.0;
  if (p.s_last)
    for (int64_t i = lane; i < p.inner; i += kWave)
      acc += double(p.s_last[bh * p.inner + i]) * p.dh_last[bh * p.inner + i];
#pragma unroll
  for (int w = 32; w; w >>= 1) acc += __shfl_xor(acc, w);
  if (lane) return;
  for (int64_t t = p.L - 1; t >= 0; --t) {
    const int64_t i = (b * p.L + t) * p.H + h;
    if (t < len) {
      for (int k = 0; k < p.utiles; ++k) acc += p.u[k * n + i];
      for (int k = 0; k < p.wtiles; ++k) acc -= p.w[k * n + i];
    }
    const float v = t < len ? float(acc) : 0.0f;
    if (p.bf16)
      st(static_cast<bf16_t*>(p.dg) + i, v);
    else
      static_cast<float*>(p.dg)[i] = v;
  }
}

// Sum over the value heads of a key head: (rows, heads, n) fp32 to (rows, key heads, n).
template <typename T>
__global__ void k_sum_heads(T* out, const float* in, int64_t total, int32_t n, int32_t per) {
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= total) return;
  const int64_t row = i / n, c = i % n;   // row: (batch, token, key head)
  float acc = 0.0f;
  for (int k = 0; k < per; ++k) acc += in[(row * per + k) * n + c];
  st(out + i, acc);
}

struct AttnStepParams {
  const void* q;
  const void* k;
  const void* v;
  const void* g;
  int64_t qs[2], ks[2], vs[2], gs[2];
  float* h;
  void* o;
  int64_t B, H;
  int32_t per, dk, dv, g_bf16;
};

template <typename T>
__global__ __launch_bounds__(kWave) void k_attn_step_simple(AttnStepParams p) {
  const int64_t bh = blockIdx.x, b = bh / p.H, h = bh % p.H;
  const int n = blockIdx.y * kWave + threadIdx.x;
  if (n >= p.dv) return;
  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + h / p.per * p.qs[1];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + h / p.per * p.ks[1];
  const float v = ld(static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[1] + n);
  const Decay d{p.g, p.gs[0], 0, p.gs[1], p.g_bf16};
  const float e = expf(log_decay(d, b, 0, h));
  float* S = p.h + bh * p.dk * p.dv + n;
  float acc = 0.0f;
  for (int m = 0; m < p.dk; ++m) {
    const float s = S[int64_t(m) * p.dv] * e + ld(k + m) * v;
    S[int64_t(m) * p.dv] = s;
    acc += s * ld(q + m);
  }
  st(static_cast<T*>(p.o) + bh * p.dv + n, acc);
}

static __global__ void k_attn_state_copy(float* dst, const float* src, int64_t n) {
  const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i < n) dst[i] = src ? src[i] : 0.0f;
}

}  // namespace ssma
