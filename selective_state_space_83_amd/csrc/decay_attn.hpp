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
// Long sequences of few heads are cut into spans walked side by side: a first
// pass forms each span's end state from zero, k_join_spans the states entering
// the spans.
//
// The decay's gradient needs no state per token: dq_i.q_i and dk_i.k_i sum the
// same pairs (i, j <= i) by reader and by writer, so with u_i = dq_i.q_i,
// w_i = dk_i.k_i (per value head), any e > t, and P_e the gradient's flow
// through the boundary before e, P_e = <S_{e-1}, exp(g_e) G_e> (at the
// sequence's end <S_last, dh_last>),
//   dg_t = sum_{t <= i < e} (u_i - w_i) + P_e.
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
  int64_t sm, sn;        // strides of S(m, n) within a head's state (s0, s_last)
  const float* carry;    // (B, H, spans, M x N): state entering each span; null with one span
  int64_t cm, cn;        // strides of S(m, n) within a carry
  float* sum;            // (B, H, spans, M, N): a span's end state from zero (the state pass)
  float* total;          // (B, H, spans): a span's decay (the state pass)
  void* out;             // (B, L, H, N)
  float* dots;           // (slices of N, B, H, L): out_t . x_t over a wave's slice
  int64_t B, L, H, span; // span: tokens per span, a multiple of the chunk
  int32_t M, N, spans, tiles, reverse;
  int32_t va, vb, vc, vx, vo;   // rows may be read / written 16 bytes at a time
};

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// A matrix operand over 32 contracted indices.  The 16 x 16 matrix instructions
// take an operand as 16 rows (lane % 16) by slots of the contracted index
// (lane / 16 = g and an index within the lane), and give the product with
// column lane % 16 and rows 4 g + i.  The contracted index may be dealt to the
// slots in any order as long as both operands agree: here lane group g holds
// indices 4 g + i and 16 + 4 g + i (i = 0..3).  So a product, read as an
// operand over its row index, is already in place: scores and states go from
// one product into the next without crossing lanes.
template <typename T>
struct Operand;

template <>
struct Operand<bf16_t> {
  bf16x8 v;   // [half][i]
  __device__ __forceinline__ void set(const f32x4& lo, const f32x4& hi) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = static_cast<__bf16>(lo[i]);
      v[4 + i] = static_cast<__bf16>(hi[i]);
    }
  }
};

template <>
struct Operand<float> {
  f32x4 v[2];
  __device__ __forceinline__ void set(const f32x4& lo, const f32x4& hi) {
    v[0] = lo;
    v[1] = hi;
  }
};

__device__ __forceinline__ f32x4 mma(const Operand<bf16_t>& a, const Operand<bf16_t>& b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Operand<float>& a, const Operand<float>& b, f32x4 c) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[h][i], b.v[h][i], c, 0, 0, 0);
  return c;
}

// x as SP operands that sum to it: bf16 keeps 8 bits in each, fp32 all in one.
template <int SP>
__device__ __forceinline__ void split(Operand<bf16_t> (&o)[SP], f32x4 lo, f32x4 hi) {
#pragma unroll
  for (int s = 0; s < SP; ++s) {
    o[s].set(lo, hi);
    if (s + 1 < SP) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        lo[i] -= static_cast<float>(o[s].v[i]);
        hi[i] -= static_cast<float>(o[s].v[4 + i]);
      }
    }
  }
}
template <int SP>
__device__ __forceinline__ void split(Operand<float> (&o)[SP], f32x4 lo, f32x4 hi) {
  static_assert(SP == 1, "");
  o[0].set(lo, hi);
}

// Rows in LDS.  bf16 rows that are read along the row hold the columns of each
// block of 32 in the operands' order (g, half, i), so that an operand is one
// 16-byte read; bf16 operands down the rows come from the transposing LDS read
// (16 lanes name 4 rows x 16 columns, each lane gets one column of them).
template <typename T>
struct Lds;

template <>
struct Lds<bf16_t> {
  static constexpr int kVec = 8;         // elements in 16 bytes
  static constexpr int kPad = 24;        // 12 words: rows fall on different banks
  static constexpr int kPadC = 16;
  __device__ static __forceinline__ int pos(int col) {   // col a multiple of 4
    return (col & ~31) + 2 * (col & 12) + ((col & 16) >> 2);
  }
  __device__ static __forceinline__ void put(bf16_t* row, int col, u32x4 v) {
    *reinterpret_cast<u32x2*>(row + pos(col)) = u32x2{v[0], v[1]};
    *reinterpret_cast<u32x2*>(row + pos(col + 4)) = u32x2{v[2], v[3]};
  }
  __device__ static __forceinline__ void put_plain(bf16_t* row, int col, u32x4 v) {
    *reinterpret_cast<u32x4*>(row + col) = v;
  }
  // along the row: block t of 32 columns
  __device__ static __forceinline__ Operand<bf16_t> along(const bf16_t* row, int t, int g) {
    Operand<bf16_t> o;
    o.v = *reinterpret_cast<const bf16x8*>(row + 32 * t + 8 * g);
    return o;
  }
  __device__ static __forceinline__ s16x4 tr(const bf16_t* p) {
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
        (__attribute__((address_space(3))) s16x4*)(p));
  }
  // down block t of 32 rows; col: the lane's own group of 4 columns
  __device__ static __forceinline__ Operand<bf16_t> down(const bf16_t* s, int stride, int t, int g, int r,
                                                         int col) {
    const bf16_t* p = s + (32 * t + 4 * g + (r >> 2)) * stride + col;
    const s16x4 a = tr(p), b = tr(p + 16 * stride);
    Operand<bf16_t> o;
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    o.v = __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    return o;
  }
  // the column group a lane names for the 16 columns of tile m (rows as put())
  __device__ static __forceinline__ int tile_col(int m, int r) { return pos(16 * m + 4 * (r & 3)); }
  // for the out tiles (rows as put_plain()): with two tiles a lane's 4 + 4
  // columns lie side by side, so that it stores 16 bytes
  template <int NT>
  __device__ static __forceinline__ int out_col(int nt, int r) {
    return NT == 2 ? 8 * (r & 3) + 4 * nt : 4 * (r & 3);
  }
  template <int NT>
  __device__ static __forceinline__ int n_of(int nt, int r) {   // column of tile nt, lane r
    return NT == 2 ? 8 * (r >> 2) + 4 * nt + (r & 3) : r;
  }
};

template <>
struct Lds<float> {
  static constexpr int kVec = 4;
  static constexpr int kPad = 4;
  static constexpr int kPadC = 4;
  __device__ static __forceinline__ void put(float* row, int col, u32x4 v) {
    *reinterpret_cast<u32x4*>(row + col) = v;
  }
  __device__ static __forceinline__ void put_plain(float* row, int col, u32x4 v) { put(row, col, v); }
  __device__ static __forceinline__ Operand<float> along(const float* row, int t, int g) {
    Operand<float> o;
    o.v[0] = *reinterpret_cast<const f32x4*>(row + 32 * t + 4 * g);
    o.v[1] = *reinterpret_cast<const f32x4*>(row + 32 * t + 16 + 4 * g);
    return o;
  }
  __device__ static __forceinline__ Operand<float> down(const float* s, int stride, int t, int g, int,
                                                        int col) {
    Operand<float> o;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) o.v[h][i] = s[(32 * t + 16 * h + 4 * g + i) * stride + col];
    return o;
  }
  __device__ static __forceinline__ int tile_col(int m, int r) { return 16 * m + r; }
  template <int NT>
  __device__ static __forceinline__ int out_col(int nt, int r) { return 16 * nt + r; }
  template <int NT>
  __device__ static __forceinline__ int n_of(int nt, int r) { return 16 * nt + r; }
};

// 16 bytes of a row from column col on, zeros past its end.
template <typename T>
__device__ __forceinline__ u32x4 load16(const T* row, int col, int n, bool vec) {
  u32x4 v{0, 0, 0, 0};
  if (vec) {
    if (col < n) v = *reinterpret_cast<const u32x4*>(row + col);
    return v;
  }
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (col + e < n) v[e >> 1] |= static_cast<uint32_t>(row[col + e]) << (16 * (e & 1));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < n) v[e] = __float_as_uint(row[col + e]);
  }
  return v;
}

// The rows of a chunk, on their way from memory to LDS through registers.
template <typename T, int ROWS, int COLS>
struct Stage {
  static constexpr int kPerRow = COLS / Lds<T>::kVec;
  static constexpr int kCount = ROWS * kPerRow / 256;
  static_assert(kCount * 256 == ROWS * kPerRow, "");
  u32x4 v[kCount];
  // first: token of row 0, step its direction; rows at or past live are zeros
  __device__ __forceinline__ void load(const T* base, int64_t st, int64_t first, int step, int64_t live, int col0,
                                       int n, bool vec) {
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const int i = threadIdx.x + 256 * k, row = i / kPerRow, col = i % kPerRow * Lds<T>::kVec + col0;
      const int64_t t = first + int64_t(step) * row;
      v[k] = u32x4{0, 0, 0, 0};
      if (t < live) v[k] = load16<T>(base + t * st, col, n, vec);
    }
  }
  template <bool PLAIN>
  __device__ __forceinline__ void store(T* s, int stride) const {
#pragma unroll
    for (int k = 0; k < kCount; ++k) {
      const int i = threadIdx.x + 256 * k, row = i / kPerRow, col = i % kPerRow * Lds<T>::kVec;
      if (PLAIN)
        Lds<T>::put_plain(s + row * stride, col, v[k]);
      else
        Lds<T>::put(s + row * stride, col, v[k]);
    }
  }
};

// ---------------------------------------------------------------------------
// The sum over a chunk of CT tokens at a time (b_i: running sum of the log
// decays from the chunk's start, S the state entering it):
//
//   out_i = sum_{j <= i} exp(b_i - b_j) (a_i . b_j) c_j + exp(b_i) S^T a_i
//   S'    = exp(b_CT) S + sum_j exp(b_CT - b_j) b_j c_j^T
//
// A workgroup of four waves walks the chunks of one span of one head, for 64 NT
// of the N columns; wave w holds S for its 16 NT columns in registers.  The
// decayed scores of 16 queries are formed by one wave and shared through LDS.
// Log decays are summed in 64 bits and kept as a rounded value and its rest, so
// that differences of long sums stay exact to 2^-24 (a chunk may hold resets).
//
// With bf16 rows the products' operands are bf16: scores and the state as read
// are rounded once (SP = 1), or kept to 16 bits (SP = 2; the gradient of the
// decay sums differences of what they give).  The state itself is fp32: its
// update takes the decayed rows in three parts, 24 bits.
// STATE: only the state, from zero (the first pass over spans).
// ---------------------------------------------------------------------------
template <typename T, int MP, int NT, int CT, int SP, typename OutT, bool STATE>
__global__ __launch_bounds__(256, sizeof(T) == 2 && MP <= 128 ? 2 : 1) void k_mix(MixParams p) {
  using LD = Lds<T>;
  constexpr int NW = 64 * NT, MT = MP / 16, QT = CT / 16, KT = CT / 32;
  constexpr int SU = sizeof(T) == 2 ? 3 : 1;   // parts of the decayed rows in the state's update
  constexpr int kStride = MP + LD::kPad, kStrideC = NW + LD::kPadC;
  __shared__ __align__(16) T sA[STATE ? 1 : CT * kStride];
  __shared__ __align__(16) T sB[CT * kStride];
  __shared__ __align__(16) T sC[CT * kStrideC];
  __shared__ __align__(16) Operand<T> sP[STATE ? 1 : SP * QT * KT * kWave];
  __shared__ __align__(16) float sBh[CT], sBl[CT];

  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, g = lane >> 4, r = lane & 15;
  int64_t id = blockIdx.x;
  const int tile = int(id % p.tiles);
  id /= p.tiles;
  const int span = int(id % p.spans);
  const int64_t bh = id / p.spans, b = bh / p.H, h = bh % p.H;
  const int n0 = tile * NW, nw = n0 + w * 16 * NT;   // the workgroup's and the wave's columns
  const int64_t live = live_tokens(p.lengths, b, p.L);

  const T* pa = STATE ? nullptr : row_base<T>(p.a, b, h);
  const T* pb = row_base<T>(p.b, b, h);
  const T* pc = row_base<T>(p.c, b, h);
  const T* px = !STATE && p.dots ? row_base<T>(p.x, b, h) : nullptr;

  // chunk k of the span covers positions; a position's token counts from the
  // front or, backward, from the end of the last span: boundaries coincide
  const int64_t pos0 = span * p.span, padded = p.span * p.spans;
  const int chunks = int(p.span / CT);
  const int step = p.reverse ? -1 : 1;
  auto first_token = [&](int k) {
    const int64_t pos = pos0 + int64_t(k) * CT;
    return p.reverse ? padded - 1 - pos : pos;
  };
  auto chunk_live = [&](int k) {   // any token of the chunk before the row's end
    const int64_t t = first_token(k);
    return (p.reverse ? t - (CT - 1) : t) < live;
  };

  f32x4 S[MT][NT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int n = nw + LD::template n_of<NT>(nt, r);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = 16 * mt + 4 * g + i;
        float v = 0.0f;
        if (!STATE && m < p.M && n < p.N) {
          if (span > 0)
            v = p.carry[(bh * p.spans + span) * p.M * p.N + m * p.cm + n * p.cn];
          else if (p.s0)
            v = p.s0[bh * p.M * p.N + m * p.sm + n * p.sn];
        }
        S[mt][nt][i] = v;
      }
    }

  Stage<T, CT, MP> qa, qb;
  Stage<T, CT, NW> qc;
  float gl = 0.0f;   // the lane's log decay, base 2
  auto fetch = [&](int k) {
    const int64_t t0 = first_token(k);
    if constexpr (!STATE) qa.load(pa, p.a.st, t0, step, live, 0, p.M, p.va);
    qb.load(pb, p.b.st, t0, step, live, 0, p.M, p.vb);
    qc.load(pc, p.c.st, t0, step, live, n0, p.N, p.vc);
    gl = 0.0f;
    if (lane < CT) {
      const int64_t t = t0 + int64_t(step) * lane;
      const int64_t td = p.reverse ? t + 1 : t;   // backward, the decay stands behind the token
      if (td < live) gl = log_decay(p.g, b, td, h) * kLog2e;
    }
  };

  double all = 0.0;   // sum of the span's log decays (the state pass)
  bool have = false;
  for (int k = 0; k < chunks; ++k) {
    const int64_t t0 = first_token(k);
    if (!chunk_live(k)) {
      if constexpr (!STATE) {   // nothing but zeros
        for (int i = tid; i < CT * NW; i += 256) {
          const int64_t t = t0 + int64_t(step) * (i / NW);
          const int n = n0 + i % NW;
          if (t < p.L && n < p.N) st(static_cast<OutT*>(p.out) + ((b * p.L + t) * p.H + h) * p.N + n, 0.0f);
        }
      }
      have = false;
      continue;
    }
    if (!have) fetch(k);
    __syncthreads();
    if constexpr (!STATE) qa.template store<false>(sA, kStride);
    qb.template store<false>(sB, kStride);
    qc.template store<true>(sC, kStrideC);
    // running sums of the log decays
    double bs = gl;
#pragma unroll
    for (int d = 1; d < CT; d <<= 1) {
      const double o = __shfl_up(bs, d);
      if (lane >= d) bs += o;
    }
    const double tot = __shfl(bs, CT - 1);
    const float toth = float(tot), totl = float(tot - toth);
    if (w == 0 && lane < CT) {
      const float hi = float(bs);
      sBh[lane] = hi;
      sBl[lane] = float(bs - hi);
    }
    if (STATE) all += tot;
    __syncthreads();
    have = k + 1 < chunks && chunk_live(k + 1);
    if (have) fetch(k + 1);

    if constexpr (!STATE) {
      // scores of 16 queries; with 32 tokens the waves share a query tile
      const int qt = CT == 64 ? w : w & 1;
      const float qh = sBh[16 * qt + r], ql = sBl[16 * qt + r];
      f32x4 pr[QT];
#pragma unroll
      for (int kt = 0; kt < QT; ++kt) {
        f32x4 acc{0.0f, 0.0f, 0.0f, 0.0f};
        if (kt <= qt && (CT == 64 || kt == (w >> 1))) {
#pragma unroll
          for (int t = 0; t < MP / 32; ++t)
            acc = mma(LD::along(sB + (16 * kt + r) * kStride, t, g), LD::along(sA + (16 * qt + r) * kStride, t, g),
                      acc);
          const f32x4 kh = *reinterpret_cast<const f32x4*>(sBh + 16 * kt + 4 * g);
          const f32x4 kl = *reinterpret_cast<const f32x4*>(sBl + 16 * kt + 4 * g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float e = exp2_fast((qh - kh[i]) + (ql - kl[i]));
            acc[i] = 16 * kt + 4 * g + i <= 16 * qt + r ? acc[i] * e : 0.0f;
          }
        }
        pr[kt] = acc;
      }
      if constexpr (CT == 64) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          if (2 * t <= qt) {
            Operand<T> o[SP];
            split<SP>(o, pr[2 * t], pr[2 * t + 1]);
#pragma unroll
            for (int s = 0; s < SP; ++s) sP[((s * QT + qt) * KT + t) * kWave + lane] = o[s];
          }
        }
      } else {
        static_assert(sizeof(T) == 4 || CT == 64, "");
        if constexpr (sizeof(T) == 4) sP[qt * kWave + lane].v[w >> 1] = (w >> 1) ? pr[1] : pr[0];
      }
    }

    // what the state gives
    f32x4 acc[QT][NT];
    if constexpr (!STATE) {
#pragma unroll
      for (int qt = 0; qt < QT; ++qt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[qt][nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < MP / 32; ++t) {
        Operand<T> so[NT][SP];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) split<SP>(so[nt], S[2 * t][nt], S[2 * t + 1][nt]);
#pragma unroll
        for (int qt = 0; qt < QT; ++qt) {
          const Operand<T> a = LD::along(sA + (16 * qt + r) * kStride, t, g);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int s = 0; s < SP; ++s) acc[qt][nt] = mma(so[nt][s], a, acc[qt][nt]);
        }
      }
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) {
        const float e = exp2_fast(sBh[16 * qt + r]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[qt][nt][i] *= e;
      }
      __syncthreads();
    }

    Operand<T> c[KT][NT];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        c[t][nt] = LD::down(sC, kStrideC, t, g, r, w * 16 * NT + LD::template out_col<NT>(nt, r));

    if constexpr (!STATE) {
#pragma unroll
      for (int qt = 0; qt < QT; ++qt) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          if (2 * t > qt) continue;
#pragma unroll
          for (int s = 0; s < SP; ++s) {
            const Operand<T> o = sP[((s * QT + qt) * KT + t) * kWave + lane];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[qt][nt] = mma(c[t][nt], o, acc[qt][nt]);
          }
        }
        // the lane's query and its columns nw + n_of(nt, 4 g + i)
        const int64_t t = t0 + int64_t(step) * (16 * qt + r);
        const bool on = t < live;
        if (t < p.L) {
          OutT* out = static_cast<OutT*>(p.out) + ((b * p.L + t) * p.H + h) * p.N;
          if (!on) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[qt][nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
          }
          if (sizeof(OutT) == 2 && NT == 2 && p.vo) {
            Operand<bf16_t> o;
            o.set(acc[qt][0], acc[qt][NT - 1]);
            const int n = nw + 8 * g;
            if (n < p.N) *reinterpret_cast<bf16x8*>(out + n) = o.v;
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const int n = nw + LD::template n_of<NT>(nt, 4 * g);
              if (p.vo) {
                if (n < p.N) {
                  if constexpr (sizeof(OutT) == 2) {
                    Operand<bf16_t> o;
                    o.set(acc[qt][nt], acc[qt][nt]);
                    const u32x4 u = __builtin_bit_cast(u32x4, o.v);
                    *reinterpret_cast<u32x2*>(out + n) = u32x2{u[0], u[1]};
                  } else {
                    *reinterpret_cast<f32x4*>(out + n) = acc[qt][nt];
                  }
                }
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (n + i < p.N) st(out + n + i, acc[qt][nt][i]);
              }
            }
          }
        }
        if (px) {
          float d = 0.0f;
          if (on) {
            const T* xr = px + t * p.x.st;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int n = nw + LD::template n_of<NT>(nt, 4 * g) + i;
                if (n < p.N) d += acc[qt][nt][i] * ld(xr + n);
              }
          }
          d += __shfl_xor(d, 16);
          d += __shfl_xor(d, 32);
          if (g == 0 && t < p.L) p.dots[((int64_t(tile) * 4 + w) * p.B * p.H + bh) * p.L + t] = d;
        }
      }
    }

    // the state's update
    const float etot = exp2_fast(toth);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) S[mt][nt][i] *= etot;
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      f32x4 e[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const f32x4 kh = *reinterpret_cast<const f32x4*>(sBh + 32 * t + 16 * hf + 4 * g);
        const f32x4 kl = *reinterpret_cast<const f32x4*>(sBl + 32 * t + 16 * hf + 4 * g);
#pragma unroll
        for (int i = 0; i < 4; ++i) e[hf][i] = exp2_fast((toth - kh[i]) + (totl - kl[i]));
      }
      Operand<T> cs[NT][SU];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (sizeof(T) == 2) {
            lo[i] = static_cast<float>(c[t][nt].v[i]) * e[0][i];
            hi[i] = static_cast<float>(c[t][nt].v[4 + i]) * e[1][i];
          } else {
            lo[i] = c[t][nt].v[0][i] * e[0][i];
            hi[i] = c[t][nt].v[1][i] * e[1][i];
          }
        }
        split<SU>(cs[nt], lo, hi);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const Operand<T> bo = LD::down(sB, kStride, t, g, r, LD::tile_col(mt, r));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int s = SU - 1; s >= 0; --s) S[mt][nt] = mma(bo, cs[nt][s], S[mt][nt]);
      }
    }
  }

  float* dst = nullptr;
  float f = 1.0f;
  int64_t dm = p.N, dn = 1;
  if (STATE) {
    dst = p.sum + (bh * p.spans + span) * p.M * p.N;
    if (tid == 0 && tile == 0) p.total[bh * p.spans + span] = exp2_fast(float(all));
  } else if (span == p.spans - 1 && p.s_last) {
    dst = p.s_last + bh * p.M * p.N;
    dm = p.sm;
    dn = p.sn;
    // going backward, the first token's own decay stands between G_0 and h0
    if (p.reverse && live > 0) f = exp2_fast(log_decay(p.g, b, 0, h) * kLog2e);
  }
  if (dst) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int n = nw + LD::template n_of<NT>(nt, r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int m = 16 * mt + 4 * g + i;
          if (m < p.M && n < p.N) dst[m * dm + n * dn] = S[mt][nt][i] * f;
        }
      }
  }
}

// Joins the spans: from each span's end state from zero and its decay, the
// state entering every span, in place (the first span's slot takes s0).  A lane
// per element of S; the loads of later spans do not wait for the chain.
struct JoinParams {
  float* sum;            // (B H, spans, M, N)
  const float* total;    // (B H, spans)
  const float* s0;       // or null
  int64_t sm, sn, inner; // strides of s0; M x N
  int32_t N, spans;
};

static __global__ __launch_bounds__(256) void k_join_spans(JoinParams p) {
  const int64_t blocks = (p.inner + 255) / 256, bh = blockIdx.x / blocks;
  const int64_t e = blockIdx.x % blocks * 256 + threadIdx.x;
  if (e >= p.inner) return;
  float* s = p.sum + bh * p.spans * p.inner + e;
  const float* tot = p.total + bh * p.spans;
  float run = p.s0 ? p.s0[bh * p.inner + e / p.N * p.sm + e % p.N * p.sn] : 0.0f;
  constexpr int U = 8;
  float v[U];
  for (int k = 0; k < p.spans; k += U) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u < p.spans - 1) v[u] = s[(k + u) * p.inner];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u < p.spans) {
        s[(k + u) * p.inner] = run;
        if (k + u < p.spans - 1) run = run * tot[k + u] + v[u];
      }
  }
}

struct DecayGradParams {
  const float* u;        // (uslices, B, H, L)
  const float* w;        // (wslices, B, H, L)
  const float* carry;    // (B, H, spans, inner): states entering the spans (dq's layout)
  const float* rcarry;   // same of their gradients, spans counted from the end
  const float* s_last;   // (B, H, dk, dv), with dh_last; null: no flow through the end
  const float* dh_last;
  Decay g;
  const int32_t* lengths;
  void* dg;              // (B, L, H)
  int64_t B, L, H, inner, span;
  int32_t uslices, wslices, spans, bf16;
};

// dg over one span: the flow through its end, then suffix sums of u - w within
// it.  A workgroup per span; sums in 64 bits.
static __global__ __launch_bounds__(256) void k_decay_grad(DecayGradParams p) {
  __shared__ double part[4];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int span = int(blockIdx.x % p.spans);
  const int64_t bh = blockIdx.x / p.spans, b = bh / p.H, h = bh % p.H;
  const int64_t live = live_tokens(p.lengths, b, p.L), n = p.B * p.H * p.L;
  const int64_t t_begin = span * p.span, t_end = t_begin + p.span < p.L ? t_begin + p.span : p.L;

  double flow = 0.0;
  if (span + 1 < p.spans) {
    const float* s = p.carry + (bh * p.spans + span + 1) * p.inner;
    const float* q = p.rcarry + (bh * p.spans + (p.spans - 1 - span)) * p.inner;
    for (int64_t i = tid; i < p.inner; i += 256) flow += double(s[i]) * q[i];
    const int64_t e = t_begin + p.span;   // the decay between the two
    if (e < live) flow *= exp2_fast(log_decay(p.g, b, e, h) * kLog2e);
  } else if (p.s_last) {
    for (int64_t i = tid; i < p.inner; i += 256)
      flow += double(p.s_last[bh * p.inner + i]) * p.dh_last[bh * p.inner + i];
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) flow += __shfl_xor(flow, d);
  if (lane == 0) part[w] = flow;
  __syncthreads();
  double run = part[0] + part[1] + part[2] + part[3];

  for (int64_t base = t_begin + (t_end - 1 - t_begin) / 256 * 256; base >= t_begin; base -= 256) {
    const int64_t t = base + tid;
    double v = 0.0;
    if (t < t_end && t < live) {
      const int64_t i = bh * p.L + t;
      for (int k = 0; k < p.uslices; ++k) v += p.u[k * n + i];
      for (int k = 0; k < p.wslices; ++k) v -= p.w[k * n + i];
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double o = __shfl_down(v, d);
      if (lane + d < 64) v += o;
    }
    __syncthreads();
    if (lane == 0) part[w] = v;
    __syncthreads();
    double behind = run;
    for (int k = w + 1; k < 4; ++k) behind += part[k];
    if (t < t_end) {
      const float out = t < live ? float(v + behind) : 0.0f;
      const int64_t i = (b * p.L + t) * p.H + h;
      if (p.bf16)
        st(static_cast<bf16_t*>(p.dg) + i, out);
      else
        static_cast<float*>(p.dg)[i] = out;
    }
    run += part[0] + part[1] + part[2] + part[3];
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
