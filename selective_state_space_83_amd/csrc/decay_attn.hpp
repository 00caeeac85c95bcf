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
// The decay's gradient dg_t = exp(g_t) <S_{t-1}, G_t> is the sum over all pairs of
// a token j < t that writes and one i >= t that reads.  Within a chunk, with S the
// state entering it, G its gradient behind it and b_i as below,
//
//   dg_t =   sum_{j < t <= i} exp(b_i - b_j) (q_i . k_j) (v_j . dout_i)    both in it
//          + sum_{i >= t} exp(b_i) q_i . (S dout_i)                        j before it
//          + sum_{j < t} exp(b_end - b_j) k_j . (G v_j)                    i behind it
//          + exp(b_end) <S, G>                                             neither.
//
// Every term is one that passes t, with its own decay: no sums cancel (as those of
// dq_i . q_i - dk_i . k_i would, which also count the pairs that do not pass t),
// a reset's gradient is 0, and other segments' sizes and non-finite values stay
// theirs.  The passes for dq and dk leave the second and third terms as dots of
// the state's part of their rows; the first also leaves the state entering each
// chunk, for the other to take its product with G; k_decay_grad adds up the rest.
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
// The most that the log2 decays of a chunk may grow for its products' form to
// hold: every exp then stays below 2^32, so that nothing times it overflows that
// the recurrence keeps, and a clamped reset followed by growth (2^-184 2^32) is
// still 0.  Chunks that grow more are walked token by token.
constexpr float kMaxGrowth = 32.0f;

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
  return static_cast<const T*>(r.p) + b * r.sb + int64_t(uint32_t(h) / uint32_t(r.per)) * r.sh;
}

struct Decay {
  const void* p;
  int64_t sb, st, sh;
  int32_t bf16;
};

// A log decay's bits, and its value from them: read apart, so that the read can
// be in flight while others are made.
__device__ __forceinline__ uint32_t log_decay_bits(const Decay& d, int64_t b, int64_t t, int64_t h) {
  const int64_t i = b * d.sb + t * d.st + h * d.sh;
  return d.bf16 ? static_cast<const bf16_t*>(d.p)[i] : static_cast<const uint32_t*>(d.p)[i];
}
__device__ __forceinline__ float log_decay_of(const Decay& d, uint32_t bits) {
  return __uint_as_float(d.bf16 ? bits << 16 : bits);
}
__device__ __forceinline__ float log_decay(const Decay& d, int64_t b, int64_t t, int64_t h) {
  return log_decay_of(d, log_decay_bits(d, b, t, h));
}

__device__ __forceinline__ int64_t live_tokens(const int32_t* lengths, int64_t b, int64_t L) {
  if (!lengths) return L;
  const int64_t n = lengths[b];
  return n < 0 ? 0 : n > L ? L : n;
}

struct MixParams {
  Rows a, b, c, x;       // x: rows like out, for the dots
  Decay g;
  const int32_t* lengths;
  const float* s0;       // state before the first token, or null
  float* s_last;         // state after the last, or null
  int64_t sm, sn;        // strides of S(m, n) within a head's state (s0, s_last)
  const float* carry;    // (B, H, spans, M x N): slot k, the state entering span k + 1; null with one span
  int64_t cm, cn;        // strides of S(m, n) within a carry
  float* sum;            // (B, H, spans, M, N): a span's end state from zero (the state pass)
  float* total;          // (B, H, spans): the root of a span's decay, exp2_half (the state pass)
  void* out;             // (B, L, H, N)
  float* dots;           // (slices of N, B, H, span x spans): over a wave's slice, x_t . the state's part of out_t
  float* kept;           // (B, H, chunks, slices, tiles of M, lanes, 4): the state entering a chunk as the waves hold
                         // it; forward in time written, backward read
  float* flow;           // (slices, B, H, chunks): <kept, S> (backward in time)
  int32_t kept_slices, kept_tiles;   // those with columns below N, rows below M
  int64_t B, L, H, span; // span: tokens per span, a multiple of the chunk
  int32_t M, N, spans, tiles;
  int32_t walked;        // spans of this launch: all, or (the state pass) all but the last
};

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float exp2_fast(float v) { return __builtin_amdgcn_exp2f(v); }

// 2^(v / 2), at most 2^127: x 2^v is formed as x f f, which keeps a zero zero
// where 2^v overflows, and what 2^v brings into range or out of it in place
// (past 2^254 everything but a zero has overflowed).
__device__ __forceinline__ float exp2_half(float v) {
  return exp2_fast(0.5f * (v > 254.0f && v < __builtin_inff() ? 254.0f : v));
}

// A matrix operand over 32 contracted indices.  The 16 x 16 matrix instructions
// take an operand as 16 rows (lane % 16) by slots of the contracted index
// (lane / 16 = g and an index within the lane), and give the product with
// column lane % 16 and rows 4 g + i.  The contracted index may be dealt to the
// slots in any order as long as both operands agree: here lane group g holds
// indices (tile, 4 g + i), tile = 0, 1 and i = 0..3, of two products of 16 rows.
// So a product, read as an operand over its row index, is already in place:
// scores and states go from one product into the next without crossing lanes.
template <typename T>
struct Operand;

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two values rounded to bf16, in one register; and as floats again.
__device__ __forceinline__ uint32_t round2(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}
__device__ __forceinline__ float low16(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float high16(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

template <>
struct Operand<bf16_t> {
  bf16x8 v;   // [half][i]
  __device__ __forceinline__ void set(const f32x4& lo, const f32x4& hi) {
    v = __builtin_bit_cast(bf16x8, u32x4{round2(lo[0], lo[1]), round2(lo[2], lo[3]), round2(hi[0], hi[1]),
                                         round2(hi[2], hi[3])});
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
      const u32x4 u = __builtin_bit_cast(u32x4, o[s].v);
      lo -= f32x4{low16(u[0]), high16(u[0]), low16(u[1]), high16(u[1])};
      hi -= f32x4{low16(u[2]), high16(u[2]), low16(u[3]), high16(u[3])};
    }
  }
}
template <int SP>
__device__ __forceinline__ void split(Operand<float> (&o)[SP], f32x4 lo, f32x4 hi) {
  static_assert(SP == 1, "");
  o[0].set(lo, hi);
}

// Rows in LDS, read along the row (16 bytes a lane) or, as an operand over the
// rows, down the columns: bf16 with the transposing LDS read (16 lanes name 4
// rows x 16 columns, in any 4 groups of 4, and each lane gets one column).
//
// A product's rows become a contracted index in the order (tile, 4 g + i); read
// along, lane group g holds 8 columns side by side.  Both name the same index
// when the rows of the state's tiles are the columns m_of below.
template <typename T>
struct Lds;

template <>
struct Lds<bf16_t> {
  static constexpr int kVec = 8;         // elements in 16 bytes
  // rows 8 words apart modulo the 64 banks: reads along and down the rows then
  // meet no conflicts (counted: 64 reads along 1792 cycles of conflict without
  // padding, 256 with 24 elements, 0 with 16; down 896, 128-256, 0-128)
  static constexpr int kPad = 16;
  static constexpr int kPadC = 16;
  // block t of 32 columns of a row
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
  // the column of the state's tile mt, row 4 g + i, and the columns a lane names
  // to read down that tile
  __device__ static __forceinline__ int m_of(int mt, int g, int i) {
    return 32 * (mt >> 1) + 8 * g + 4 * (mt & 1) + i;
  }
  __device__ static __forceinline__ int tile_col(int mt, int r) { return m_of(mt, r & 3, 0); }
  __device__ static __forceinline__ int group_col(int r) { return 4 * (r & 3); }   // of 16 in order
};

template <>
struct Lds<float> {
  static constexpr int kVec = 4;
  static constexpr int kPad = 4;
  static constexpr int kPadC = 4;
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
  __device__ static __forceinline__ int m_of(int mt, int g, int i) { return 16 * mt + 4 * g + i; }
  __device__ static __forceinline__ int tile_col(int mt, int r) { return 16 * mt + r; }
  __device__ static __forceinline__ int group_col(int r) { return r; }
};

constexpr int kBufferFlags = 0x00020000;       // gfx9-family raw buffer, 32-bit data
constexpr uint32_t kOutside = 0x80000000u;     // an offset past any buffer: loads 0, stores nothing

// A window of memory: `rows` rows (at most 0: none), `stride` bytes apart, of
// which `width` bytes count.  Reads outside give zeros, writes nothing.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t window(const void* base, int rows, uint32_t stride, int width) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), static_cast<short>(0),
                                           rows > 0 ? int(uint32_t(rows - 1) * stride) + width : 0, kBufferFlags);
}

// The rows of a chunk, on their way from memory to LDS through registers.  Rows
// are taken in the order of their tokens; `first` is the lowest.
//
// FAST: rows start on 16 bytes, hold whole 16 bytes, do not overlap, and a
// chunk's span less than 2^31 bytes (checked by the host): they are read through
// a window that ends with the row's last token.  Otherwise element by element.
template <typename T, int ROWS, int COLS, int THREADS, bool FAST>
struct Stage {
  static constexpr int kPerRow = COLS / Lds<T>::kVec;
  static constexpr int kStep = THREADS / kPerRow;   // rows between a lane's loads
  static constexpr bool kFew = ROWS < kStep;        // fewer loads than lanes
  static constexpr int kCount = kFew ? 1 : ROWS / kStep;
  static_assert(kFew || kCount * kStep == ROWS, "");
  u32x4 v[kCount];
  __device__ __forceinline__ void load(const T* base, int64_t st, int64_t first, int64_t live, int col0, int n) {
    const int row = threadIdx.x / kPerRow, col = threadIdx.x % kPerRow * Lds<T>::kVec + col0;
    if constexpr (FAST) {
      // a window for each load, so that one offset serves them all
      const int left = live - first < ROWS ? int(live - first) : ROWS;
      const uint32_t pitch = uint32_t(st) * uint32_t(sizeof(T));
      const uint32_t off =
          col < n && (!kFew || row < ROWS) ? uint32_t(row) * pitch + uint32_t(col) * uint32_t(sizeof(T)) : kOutside;
#pragma unroll
      for (int k = 0; k < kCount; ++k)
        v[k] = __builtin_amdgcn_raw_buffer_load_b128(
            window(base + (first + k * kStep) * st, left - k * kStep, pitch, n * int(sizeof(T))), off, 0, 0);
    } else {
#pragma unroll 1
      for (int k = 0; k < kCount; ++k) {
        const int64_t t = first + row + k * kStep;
        u32x4 u{0, 0, 0, 0};
        if (t < live && (!kFew || row < ROWS)) {
          const T* p = base + t * st;
          for (int e = 0; e < Lds<T>::kVec; ++e)
            if (col + e < n) {
              if constexpr (sizeof(T) == 2) {
                const uint32_t x = static_cast<uint32_t>(p[col + e]) << (16 * (e & 1));
                u[0] |= e >> 1 == 0 ? x : 0;
                u[1] |= e >> 1 == 1 ? x : 0;
                u[2] |= e >> 1 == 2 ? x : 0;
                u[3] |= e >> 1 == 3 ? x : 0;
              } else {
                const uint32_t x = __float_as_uint(p[col + e]);
                u[0] = e == 0 ? x : u[0];
                u[1] = e == 1 ? x : u[1];
                u[2] = e == 2 ? x : u[2];
                u[3] = e == 3 ? x : u[3];
              }
            }
        }
#pragma unroll
        for (int j = 0; j < kCount; ++j)
          if (j == k) v[j] = u;
      }
    }
  }
  // Whether one of the lane's values is an infinity or a NaN: its exponent, the
  // bits below the sign, is then the largest there is.
  __device__ __forceinline__ bool non_finite() const {
    if constexpr (sizeof(T) == 2) {
      typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
      u16x2 top{0, 0};
#pragma unroll
      for (int k = 0; k < kCount; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[k][i] & 0x7fff7fffu));
      return top[0] >= 0x7f80u || top[1] >= 0x7f80u;
    } else {
      uint32_t top = 0;
#pragma unroll
      for (int k = 0; k < kCount; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) top = v[k][i] << 1 > top ? v[k][i] << 1 : top;
      return top >= 0xff000000u;
    }
  }
  // REV: the last row first
  template <bool REV>
  __device__ __forceinline__ void store(T* s, int stride) const {
    const int row = threadIdx.x / kPerRow, col = threadIdx.x % kPerRow * Lds<T>::kVec;
    if (kFew && row >= ROWS) return;
    T* p = s + (REV ? (kFew ? ROWS : kStep) - 1 - row : row) * stride + col;
#pragma unroll
    for (int k = 0; k < kCount; ++k)
      *reinterpret_cast<u32x4*>(p + (REV ? kCount - 1 - k : k) * kStep * stride) = v[k];
  }
};

// The other way: rows in LDS that lie as a Stage would have stored them, out to
// memory.  A lane takes the places that it would store to, so that it can follow
// with the next rows without another wait.
template <typename T, int ROWS, int COLS, int THREADS, bool REV>
__device__ __forceinline__ void write_rows(T* base, int64_t st, int64_t first, int64_t end, int col0, int n, const T* s,
                                           int stride) {
  typedef Stage<T, ROWS, COLS, THREADS, true> St;
  const int row = threadIdx.x / St::kPerRow, col = threadIdx.x % St::kPerRow * Lds<T>::kVec;
  if (St::kFew && row >= ROWS) return;
  const T* p = s + (REV ? (St::kFew ? ROWS : St::kStep) - 1 - row : row) * stride + col;
  const int left = end - first < ROWS ? int(end - first) : ROWS;
  const uint32_t pitch = uint32_t(st) * uint32_t(sizeof(T));
  const uint32_t off =
      col + col0 < n ? uint32_t(row) * pitch + uint32_t(col + col0) * uint32_t(sizeof(T)) : kOutside;
#pragma unroll
  for (int k = 0; k < St::kCount; ++k) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p + (REV ? St::kCount - 1 - k : k) * St::kStep * stride);
    __builtin_amdgcn_raw_buffer_store_b128(
        v, window(base + (first + k * St::kStep) * st, left - k * St::kStep, pitch, n * int(sizeof(T))), off, 0, 0);
  }
}

// v plus its value in other lanes (0 where there is none), over two registers.
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ double add_lanes(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, uint32_t(u), CTRL, ROW_MASK, 0xf, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, uint32_t(u >> 32), CTRL, ROW_MASK, 0xf, false);
  return v + __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// Running sum over the wave's lanes.
__device__ __forceinline__ double wave_running_sum(double v) {
  v = add_lanes<0x111, 0xf>(v);   // within rows of 16: lanes 1, 2, 4 and 8 below
  v = add_lanes<0x112, 0xf>(v);
  v = add_lanes<0x114, 0xf>(v);
  v = add_lanes<0x118, 0xf>(v);
  v = add_lanes<0x142, 0xa>(v);   // row 0's last lane into row 1, row 2's into row 3
  v = add_lanes<0x143, 0xc>(v);   // lane 31 into rows 2 and 3
  return v;
}

__device__ __forceinline__ double last_lane(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(u), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(uint32_t(u >> 32), 63);
  return __builtin_bit_cast(double, uint64_t(hi) << 32 | lo);
}

// Sum over the 16 lanes of a row, in all of them; over the wave.
template <int CTRL>
__device__ __forceinline__ float add_lane(float v) {
  return v + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float row_sum(float v) {
  v = add_lane<0xB1>(v);      // lane ^ 1
  v = add_lane<0x4E>(v);      // lane ^ 2
  v = add_lane<0x141>(v);     // mirrored within 8
  return add_lane<0x140>(v);  // mirrored within 16
}
__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// What a launch forms: only the state, from zero (the first pass over spans);
// the rows out; the rows out and what the decay's gradient takes from them.
enum Part : int { kState = 0, kOut = 1, kOutDots = 2 };

// ---------------------------------------------------------------------------
// The sum over a chunk of CT tokens at a time (b_i: running sum of the log
// decays from the chunk's start, S the state entering it):
//
//   out_i = sum_{j <= i} exp(b_i - b_j) (a_i . b_j) c_j + exp(b_i) S^T a_i
//   S'    = exp(b_CT) S + sum_j exp(b_CT - b_j) b_j c_j^T
//
// A workgroup walks the chunks of one span of one head, its W waves with 16 of
// the N columns each and S for them in registers.  The decayed scores of a chunk
// are formed once, a query tile by one or two waves, and shared through LDS.
// Log decays are summed in 64 bits and kept as a rounded value and its rest, so
// that differences of long sums stay exact to 2^-24 (a chunk may hold resets);
// wave 0 does it a chunk ahead.
//
// Where the decays of a chunk add up to growth that the exps cannot hold, as they
// may while the state is zero, the workgroup walks from there on token by token,
// as the recurrence does (log decays of at most 0, the usual ones, never do; a
// test of their signs is all they pay).  So it does where a row of c holds an
// infinity or a NaN, which the products would carry, times their zeros above the
// diagonal, to the rows out before it.
//
// With bf16 rows the products' operands are bf16: scores and the state as read
// are rounded once (SP = 1), or kept to 16 bits (SP = 2; the gradient of the
// decay, which may be fp32, is taken from them).  The state itself is fp32: its
// update takes the decayed rows in three parts, 24 bits.
// ---------------------------------------------------------------------------
// Waves a SIMD is to hold: four (128 registers each) where that does not spill,
// since a chunk's steps wait on each other and other waves fill the gaps.  The
// parts of the scores and the state (SP = 2) do spill, and so do 128 rows of S
// with fp32 operands: every reload from scratch also waits for the rows on their
// way (two passes of 4 x 4096 x 20 heads x 128 x 128 with SP = 2: 200 us each
// with four, 150 with two, both without the states kept for the decay's gradient;
// 2048 x 256 heads x 128 x 128 fp32: 453 and 413 us).
template <typename T, int MP, int SP>
constexpr int waves_per_simd() {
  return SP == 1 && MP <= (sizeof(T) == 4 ? 64 : 128) ? 4 : 2;
}

// Measured (one walk over 2048 tokens a head, calls back to back): 512 heads of
// 128 x 128 bf16 288 us (3.7 TB/s), 512 of 64 x 64 bf16 127 us (4.2 TB/s), 512 of
// 64 x 64 fp32 316 us.  bf16 is bound by a chunk's steps waiting on each other and
// on memory (waves wait 48% of the time, the matrix units are busy 29%), more so
// alone on a CU (176 to 184 us for 256 heads); fp32 by its matrix products, which
// are busy half of the time.
template <typename T, int MP, int W, int CT, int SP, typename OutT, Part PART, bool REV, bool FAST>
__global__ __launch_bounds__(64 * W, (waves_per_simd<T, MP, SP>())) void k_mix(MixParams p) {
  using LD = Lds<T>;
  constexpr bool OUT = PART != kState;
  constexpr int NW = 16 * W, MT = MP / 16, QT = CT / 16, KT = CT / 32;
  constexpr int SU = sizeof(T) == 2 ? 3 : 1;   // parts of the decayed rows in the state's update
  constexpr int kStride = MP + LD::kPad, kStrideC = NW + LD::kPadC;
  constexpr int kScores = CT == 64 ? 6 : 2;    // operands of scores: (query tile, 32 keys) on or under the diagonal
  __shared__ __align__(16) T sA[OUT ? CT * kStride : 1];
  __shared__ __align__(16) T sB[CT * kStride];
  __shared__ __align__(16) T sC[CT * kStrideC];
  __shared__ __align__(16) Operand<T> sP[OUT ? SP * kScores * kWave : 1];
  // of the chunk's running sums b: rounded and rest; exp(b), exp(b_CT - b), exp(b_CT)
  __shared__ __align__(16) float sBh[2][CT], sBl[2][CT], sIn[2][CT], sEnd[2][CT], sAll[2];
  // the log decays themselves (the state pass: their sums to the span's end), and
  // whether the chunk is walked token by token
  __shared__ float sG[2][CT];
  __shared__ int sWalk[2];
  // where query tile q's scores with keys 32 t.. lie: 0 0 | 1 1 2 2 and on
  auto score_at = [](int s, int q, int t) { return (s * kScores + (q < 2 ? q : 2 * q - 2 + t)) * kWave; };

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const uint32_t id = blockIdx.x / uint32_t(p.tiles);   // the grid is below 2^31
  const int tile = int(blockIdx.x % uint32_t(p.tiles)), span = int(id % uint32_t(p.walked));
  const uint32_t bh32 = id / uint32_t(p.walked);
  const int64_t bh = bh32, b = bh32 / uint32_t(p.H), h = bh32 % uint32_t(p.H);
  const int n0 = tile * NW, nw = n0 + w * 16;   // the workgroup's and the wave's columns
  const int64_t live = live_tokens(p.lengths, b, p.L);

  const T* pa = OUT ? row_base<T>(p.a, b, h) : nullptr;
  const T* pb = row_base<T>(p.b, b, h);
  const T* pc = row_base<T>(p.c, b, h);
  const T* px = PART == kOutDots ? row_base<T>(p.x, b, h) : nullptr;
  OutT* const po = OUT ? static_cast<OutT*>(p.out) + (b * p.L * p.H + h) * p.N : nullptr;
  const int64_t ost = p.H * p.N;
  float* const dots = PART == kOutDots ? p.dots + ((int64_t(tile) * W + w) * p.B * p.H + bh) * p.span * p.spans : nullptr;

  // the lowest token of the chunk taken k-th; backward, positions count from the
  // end of the last span, so that spans and chunks have the same boundaries
  // either way.  The state pass takes a span's chunks from its end: what it read
  // last is what the next pass reads first, and comes from the caches.
  const int chunks = int(p.span / CT);
  auto lowest = [&](int k) {
    const int64_t pos = span * p.span + int64_t(OUT ? k : chunks - 1 - k) * CT;
    return REV ? p.span * p.spans - CT - pos : pos;
  };

  f32x4 S[MT];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) S[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (OUT && (span > 0 || p.s0)) {
    const float* src = span > 0 ? p.carry + (bh * p.spans + span - 1) * p.M * p.N : p.s0 + bh * p.M * p.N;
    const int64_t sm = span > 0 ? p.cm : p.sm, sn = span > 0 ? p.cn : p.sn;
    const int n = nw + r;
    const float* col = src + n * sn;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = LD::m_of(mt, g, i);
        if (m < p.M && n < p.N) S[mt][i] = col[m * sm];
      }
  }

  Stage<T, CT, MP, 64 * W, FAST> qa, qb;
  Stage<T, CT, NW, 64 * W, FAST> qc;
  auto fetch = [&](int64_t low) {
    if constexpr (OUT) qa.load(pa, p.a.st, low, live, 0, p.M);
    qb.load(pb, p.b.st, low, live, 0, p.M);
    qc.load(pc, p.c.st, low, live, n0, p.N);
  };
  // The decays are the work of one wave, one that has few scores to form: read
  // two chunks ahead and summed one ahead.
  constexpr int DW = W == 8 ? 1 : 0;
  uint32_t gl = 0;    // the lane's log decay (all zeros: none)
  double all = 0.0;   // the state pass: sum of the log decays behind the chunk
  auto fetch_decays = [&](int64_t low) {
    // backward, the decay stands behind the token; the state pass takes the last
    // token's first
    const int64_t first = low + (REV ? 1 : 0);
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));   // one wave's addresses, not to be held by all through the loop
    const int row = REV == OUT ? CT - 1 - lane : lane, left = live - first < CT ? int(live - first) : CT;
    gl = 0;
    if (row >= 0 && row < left && lane < CT) {
      if constexpr (FAST) {
        const uint32_t es = p.g.bf16 ? 2 : 4, pitch = uint32_t(p.g.st) * es;
        const auto win = window(static_cast<const char*>(p.g.p) + (b * p.g.sb + first * p.g.st + h * p.g.sh) * es,
                                left, pitch, int(es));
        const uint32_t off = uint32_t(row) * pitch;
        if (p.g.bf16)
          gl = __builtin_amdgcn_raw_buffer_load_b16(win, off, 0, 0);
        else
          gl = __builtin_amdgcn_raw_buffer_load_b32(win, off, 0, 0);
      } else {
        gl = log_decay_bits(p.g, b, first + row, h);
      }
    }
  };
  auto sum_decays = [&](int buf) {
    int lane = tid & 63;
    asm volatile("" : "+v"(lane));
    const float g = log_decay_of(p.g, gl) * kLog2e;   // -inf and NaN stay what they are
    bool walk;
    if constexpr (OUT) {
      const double bs = wave_running_sum(g < kMinLogDecay * kLog2e ? kMinLogDecay * kLog2e : g), tot = last_lane(bs);
      const float hi = float(bs);
      if (lane < CT) {
        sBh[buf][lane] = hi;
        sBl[buf][lane] = float(bs - hi);
        sIn[buf][lane] = exp2_fast(hi);
        sEnd[buf][lane] = exp2_fast(float(tot - bs));   // to the chunk's end
        sG[buf][lane] = g;
      }
      if (lane == 0) sAll[buf] = exp2_fast(float(tot));
      walk = __any(!(g <= 0.0f));
      if (walk) walk = !(last_lane(wave_running_sum(g <= 0.0f ? 0.0f : g)) <= kMaxGrowth);
    } else {
      // from behind the lane's token to the span's end
      const double bs = wave_running_sum(g), before = __shfl_up(bs, 1), at = all + (lane > 0 ? before : 0.0);
      if (lane < CT) {
        sEnd[buf][CT - 1 - lane] = exp2_fast(float(at));
        sG[buf][CT - 1 - lane] = float(at);
      }
      walk = __any(lane < CT && !(at <= kMaxGrowth));
      all += last_lane(bs);
    }
    if (lane == 0) sWalk[buf] = walk;
  };

  // A chunk's rows out are held until the next chunk's rows go to LDS: loads and
  // stores are waited for in order, and the wait for those rows would otherwise
  // be one for these stores too.  bf16 rows are held in c's place in LDS (a wave
  // has read its columns of c by then, and no other wave reads them) and leave
  // as whole rows; fp32 ones in registers, 64 bytes of a row to a wave (2048 x
  // 512 heads x 64 x 64: bf16 138 us through registers, 130 through LDS; 8 x 2048
  // x 24 x 64 x 64 fp32 178 and 193).
  constexpr bool SWAP = OUT && FAST && sizeof(T) == 2 && sizeof(OutT) == 2;
  constexpr bool HOLD = OUT && FAST && !SWAP;
  u32x4 held[HOLD ? QT : 1];
  int64_t held_low = -1;   // lowest token of the held chunk
  auto write_held = [&]() {
    if (held_low < 0) return;
    if constexpr (SWAP) {
      write_rows<T, CT, NW, 64 * W, REV>(reinterpret_cast<T*>(po), ost, held_low, p.L, n0, p.N, sC, kStrideC);
    } else if constexpr (HOLD) {
      const uint32_t pitch = uint32_t(ost) * uint32_t(sizeof(OutT));
      const int n = nw + 4 * g, left = p.L - held_low < CT ? int(p.L - held_low) : CT;
      const uint32_t off =
          n < p.N ? uint32_t(REV ? 15 - r : r) * pitch + uint32_t(n) * uint32_t(sizeof(OutT)) : kOutside;
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        const int row = REV ? CT - 16 - 16 * q : 16 * q;
        __builtin_amdgcn_raw_buffer_store_b128(
            held[q], window(po + (held_low + row) * ost, left - row, pitch, p.N * int(sizeof(OutT))), off, 0, 0);
      }
    }
    held_low = -1;
  };

  auto write_zeros = [&](int64_t low) {
    if constexpr (OUT) {
      for (int i = tid; i < CT * NW; i += 64 * W) {
        const int64_t t = low + i / NW;
        const int n = n0 + i % NW;
        if (t < p.L && n < p.N) st(po + t * ost + n, 0.0f);
      }
    }
  };

  // The state entering a chunk, kept for its product with the state of the pass
  // the other way, which has the same tiles in the same lanes: KG tiles at a time.
  constexpr int KG = MT < 8 ? MT : 8;
  const int slice = tile * W + w;
  auto kept_window = [&](int64_t low) {
    const int64_t at = ((bh * p.spans * chunks + low / CT) * p.kept_slices + slice) * p.kept_tiles * 256;
    return window(p.kept + at, slice < p.kept_slices, 0, p.kept_tiles * 1024);
  };
  auto write_kept = [&](int64_t low) {
    const auto win = kept_window(low);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, S[mt]), win, (mt * 64 + lane) * 16, 0, 0);
  };
  auto read_kept = [&](f32x4(&to)[KG], int64_t low, int mt0) {
    const auto win = kept_window(low);
#pragma unroll
    for (int mt = 0; mt < KG; ++mt)
      to[mt] = __builtin_bit_cast(
          f32x4, __builtin_amdgcn_raw_buffer_load_b128(win, ((mt0 + mt) * 64 + lane) * 16, 0, 0));
  };
  auto write_flow = [&](f32x4(&first)[KG], int64_t low) {
    f32x4 sum{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int mt0 = 0; mt0 < MT; mt0 += KG) {
      if (mt0 > 0) read_kept(first, low, mt0);
#pragma unroll
      for (int mt = 0; mt < KG; ++mt) sum += first[mt] * S[mt0 + mt];
    }
    const float d = wave_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
    if (lane == 0 && slice < p.kept_slices)
      p.flow[(slice * p.B * p.H + bh) * p.spans * chunks + low / CT] = d;
  };

  bool have = false;
  int k = 0;
  for (; k < chunks; ++k) {
    const int64_t low = lowest(k);
    const int buf = k & 1;
    if (low >= live) {   // no token: zeros
      write_zeros(low);
      have = false;
      continue;
    }
    if (!have) {
      fetch(low);
      if (w == DW) {
        fetch_decays(low);
        sum_decays(buf);
        if (k + 1 < chunks) fetch_decays(lowest(k + 1));
      }
    }
    __syncthreads();
    if constexpr (OUT) qa.template store<REV>(sA, kStride);
    qb.template store<REV>(sB, kStride);
    if constexpr (SWAP) write_held();   // out of c's place first
    qc.template store<REV>(sC, kStrideC);
    if (OUT && __any(qc.non_finite())) sWalk[buf] = 1;
    if constexpr (HOLD) write_held();
    __syncthreads();
    have = k + 1 < chunks && lowest(k + 1) < live;
    u32x4 xr[PART == kOutDots ? QT : 1];
    f32x4 kept[PART == kOutDots && REV ? KG : 1];
    // ahead of the next chunk's rows: waits are in order
    if constexpr (PART == kOutDots) {
      if constexpr (FAST) {
        // the rows the dots are taken with: the lane's query, its 4 columns
        const uint32_t pitch = uint32_t(p.x.st) * uint32_t(sizeof(T));
        const int n = nw + 4 * g, rows = live - low < CT ? int(live - low) : CT;
        const uint32_t off =
            n < p.N ? uint32_t(REV ? 15 - r : r) * pitch + uint32_t(n) * uint32_t(sizeof(T)) : kOutside;
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          const int row = REV ? CT - 16 - 16 * q : 16 * q;
          const auto win = window(px + (low + row) * p.x.st, rows - row, pitch, p.N * int(sizeof(T)));
          if constexpr (sizeof(T) == 4) {
            xr[q] = __builtin_amdgcn_raw_buffer_load_b128(win, off, 0, 0);
          } else {
            const u32x2 u = __builtin_amdgcn_raw_buffer_load_b64(win, off, 0, 0);
            xr[q] = u32x4{u[0], u[1], 0, 0};
          }
        }
      }
      if constexpr (REV) read_kept(kept, low, 0);
    }
    const int walk = sWalk[buf];   // the same for the whole workgroup
    if (have) {
      if (w == DW) {
        sum_decays(buf ^ 1);
        if (k + 2 < chunks) fetch_decays(lowest(k + 2));
      }
      fetch(lowest(k + 1));
    }
    if (__builtin_amdgcn_readfirstlane(walk)) break;
    if constexpr (PART == kOutDots && !REV) write_kept(low);
    const int rows = live - low < CT ? int(live - low) : CT;       // of the chunk, with tokens
    const int orows = p.L - low < CT ? int(p.L - low) : CT;        // with a place in out

    f32x4 acc[OUT ? QT : 1];
    if constexpr (OUT) {
      // scores: the keys kt0.. of query tile qt that the wave takes
      constexpr int PER = CT == 32 ? 1 : W == 8 ? 2 : 4;   // key tiles of a wave
      const int qt = CT == 32 ? w & 1 : W == 8 ? w >> 1 : w;
      const int kt0 = CT == 32 ? w >> 1 : W == 8 ? 2 * (w & 1) : 0;
      if (kt0 < QT && (kt0 <= qt || CT == 32)) {
        const float qh = sBh[buf][16 * qt + r], ql = sBl[buf][16 * qt + r];
        f32x4 pr[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) {
          const int kt = kt0 + j;
          f32x4 d{0.0f, 0.0f, 0.0f, 0.0f};
          if (kt <= qt) {
#pragma unroll
            for (int t = 0; t < MP / 32; ++t)
              d = mma(LD::along(sB + (16 * kt + r) * kStride, t, g), LD::along(sA + (16 * qt + r) * kStride, t, g), d);
            const f32x4 kh = *reinterpret_cast<const f32x4*>(sBh[buf] + 16 * kt + 4 * g);
            const f32x4 kl = *reinterpret_cast<const f32x4*>(sBl[buf] + 16 * kt + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float e = exp2_fast((qh - kh[i]) + (ql - kl[i]));
              d[i] = 16 * kt + 4 * g + i <= 16 * qt + r ? d[i] * e : 0.0f;
            }
          }
          pr[j] = d;
        }
        if constexpr (CT == 64) {
#pragma unroll
          for (int t = 0; t < PER / 2; ++t) {
            if (kt0 + 2 * t <= qt) {
              Operand<T> o[SP];
              split<SP>(o, pr[2 * t], pr[2 * t + 1]);
#pragma unroll
              for (int s = 0; s < SP; ++s) sP[score_at(s, qt, kt0 / 2 + t) + lane] = o[s];
            }
          }
        } else {
          static_assert(sizeof(T) == 4 || CT == 64, "");
          if constexpr (sizeof(T) == 4) sP[score_at(0, qt, 0) + lane].v[kt0] = pr[0];
        }
      }

      // what the state gives
#pragma unroll
      for (int q = 0; q < QT; ++q) acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int t = 0; t < MP / 32; ++t) {
        Operand<T> so[SP];
        split<SP>(so, S[2 * t], S[2 * t + 1]);
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          const Operand<T> a = LD::along(sA + (16 * q + r) * kStride, t, g);
#pragma unroll
          for (int s = 0; s < SP; ++s) acc[q] = mma(so[s], a, acc[q]);
        }
      }
#pragma unroll
      for (int q = 0; q < QT; ++q) acc[q] *= sIn[buf][16 * q + r];
      if constexpr (PART == kOutDots) {
#pragma unroll
        for (int q = 0; q < QT; ++q) {
          const int row = (REV ? CT - 16 - 16 * q : 16 * q) + (REV ? 15 - r : r);
          const int n = nw + 4 * g;
          float d = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float x = 0.0f;
            if constexpr (!FAST) {
              if (row < rows && n + i < p.N) x = ld(px + (low + row) * p.x.st + n + i);
            } else if constexpr (sizeof(T) == 4) {
              x = __uint_as_float(xr[q][i]);
            } else {
              const uint32_t u = xr[q][i >> 1];
              x = __uint_as_float(i & 1 ? u & 0xffff0000u : u << 16);
            }
            d += acc[q][i] * x;
          }
          d += __shfl_xor(d, 16);
          d += __shfl_xor(d, 32);
          if (g == 0 && row < rows) dots[low + row] = d;
        }
        if constexpr (REV) write_flow(kept, low);
      }
      __syncthreads();
    }

    Operand<T> c[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t) c[t] = LD::down(sC, kStrideC, t, g, r, w * 16 + LD::group_col(r));

    if constexpr (OUT) {
      const int n = nw + 4 * g;   // the lane's columns n..n + 3
      if (FAST) held_low = low;
#pragma unroll
      for (int q = 0; q < QT; ++q) {
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          if (2 * t > q) continue;
#pragma unroll
          for (int s = 0; s < SP; ++s) acc[q] = mma(c[t], sP[score_at(s, q, t) + lane], acc[q]);
        }
        const int row = (REV ? CT - 16 - 16 * q : 16 * q) + (REV ? 15 - r : r);   // the lane's query
        const bool on = row < rows;
        if (rows < CT && !on) acc[q] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if constexpr (SWAP) {
          T* to = sC + (16 * q + r) * kStrideC + w * 16 + 4 * g;
          if constexpr (sizeof(T) == 4)
            *reinterpret_cast<f32x4*>(to) = acc[q];
          else
            *reinterpret_cast<u32x2*>(to) = u32x2{round2(acc[q][0], acc[q][1]), round2(acc[q][2], acc[q][3])};
        } else if constexpr (HOLD) {
          held[q] = __builtin_bit_cast(u32x4, acc[q]);
        } else if (row < orows) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (n + i < p.N) st(po + (low + row) * ost + n + i, acc[q][i]);
        }
      }
    }

    // the state's update
    if constexpr (OUT) {
      const float etot = sAll[buf];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) S[mt] *= etot;
    }
#pragma unroll
    for (int t = 0; t < KT; ++t) {
      const f32x4 e[2] = {*reinterpret_cast<const f32x4*>(sEnd[buf] + 32 * t + 4 * g),
                          *reinterpret_cast<const f32x4*>(sEnd[buf] + 32 * t + 16 + 4 * g)};
      f32x4 lo, hi;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
          const u32x4 u = __builtin_bit_cast(u32x4, c[t].v);
          lo[i] = (i & 1 ? high16(u[i >> 1]) : low16(u[i >> 1])) * e[0][i];
          hi[i] = (i & 1 ? high16(u[2 + (i >> 1)]) : low16(u[2 + (i >> 1)])) * e[1][i];
        } else {
          lo[i] = c[t].v[0][i] * e[0][i];
          hi[i] = c[t].v[1][i] * e[1][i];
        }
      }
      Operand<T> cs[SU];
      split<SU>(cs, lo, hi);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const Operand<T> bo = LD::down(sB, kStride, t, g, r, LD::tile_col(mt, r));
#pragma unroll
        for (int s = SU - 1; s >= 0; --s) S[mt] = mma(bo, cs[s], S[mt]);
      }
    }
  }

  if (SWAP) __syncthreads();
  write_held();

  // token by token from the chunk that needs it to the span's end; a loop of its
  // own, since what it holds would cost the usual one registers; the lane's place
  // is hidden for the same reason
  int lane2 = lane;
  asm volatile("" : "+v"(lane2));
  const int g2 = lane2 >> 4, r2 = lane2 & 15;
  for (const int summed = have ? k + 2 : k + 1; k < chunks; ++k) {
    const int64_t low = lowest(k);
    const int buf = k & 1;
    if (low >= live) {
      write_zeros(low);
      continue;
    }
    const int rows = live - low < CT ? int(live - low) : CT, orows = p.L - low < CT ? int(p.L - low) : CT;
    const int n = nw + r2;   // the lane's column; its rows of S as ever
    __syncthreads();
    fetch(low);
    if (w == DW && k >= summed) {
      fetch_decays(low);
      sum_decays(buf);
    }
    if constexpr (OUT) qa.template store<REV>(sA, kStride);
    qb.template store<REV>(sB, kStride);
    qc.template store<REV>(sC, kStrideC);
    __syncthreads();
    if constexpr (PART == kOutDots) {
      if constexpr (REV) {
        f32x4 kept[KG];
        read_kept(kept, low, 0);
        write_flow(kept, low);
      } else {
        write_kept(low);
      }
      double sum = 0.0;   // of the log decays
#pragma unroll 1
      for (int i = 0; i < CT; ++i) {
        float d = 0.0f;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
          for (int e = 0; e < 4; ++e) d += S[mt][e] * ld(sA + i * kStride + LD::m_of(mt, g2, e));
          asm volatile("" ::: "memory");
        }
        sum += sG[buf][i];
        const float f = exp2_half(float(sum));
        const int row = REV ? CT - 1 - i : i;
        const bool on = row < rows;
        d = wave_sum(on && n < p.N ? d * f * f * ld(px + (low + row) * p.x.st + n) : 0.0f);
        if (lane2 == 0 && on) dots[low + row] = d;
      }
    }
#pragma unroll 1
    for (int i = 0; i < CT; ++i) {
      const float f = exp2_half(sG[buf][i]), cv = ld(sC + i * kStrideC + w * 16 + r2);
      float o = 0.0f;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int m = i * kStride + LD::m_of(mt, g2, e);
          if constexpr (OUT) {
            S[mt][e] = S[mt][e] * f * f + ld(sB + m) * cv;
            o += S[mt][e] * ld(sA + m);
          } else {
            S[mt][e] += ld(sB + m) * cv * f * f;
          }
        }
        asm volatile("" ::: "memory");   // a few reads at a time
      }
      if constexpr (OUT) {
        o += __shfl_xor(o, 16);
        o += __shfl_xor(o, 32);
        const int row = REV ? CT - 1 - i : i;
        if (g2 == 0 && row < orows && n < p.N) st(po + (low + row) * ost + n, row < rows ? o : 0.0f);
      }
    }
  }

  float* dst = nullptr;
  float f = 1.0f;   // the root of a last decay
  int64_t dm = p.N, dn = 1;
  if (!OUT) {
    dst = p.sum + (bh * p.spans + span) * p.M * p.N;
    if (w == DW && lane == 0 && tile == 0) p.total[bh * p.spans + span] = exp2_half(float(all));
  } else if (span == p.spans - 1 && p.s_last) {
    dst = p.s_last + bh * p.M * p.N;
    dm = p.sm;
    dn = p.sn;
    // going backward, the first token's own decay stands between G_0 and h0
    if (REV && live > 0) f = exp2_half(log_decay(p.g, b, 0, h) * kLog2e);
  }
  if (dst) {
    const int n = nw + r2;
    float* col = dst + n * dn;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = LD::m_of(mt, g2, i);
        if (m < p.M && n < p.N) col[m * dm] = S[mt][i] * f * f;
      }
  }
}

// Joins the spans: from each span's end state from zero and its decay, the
// state entering the span behind it, in place (slot k: the state entering span
// k + 1).  A lane takes V elements of S through the spans, U of them read ahead
// of the chain at a time (the last ones again where fewer are left).
struct JoinParams {
  float* sum;            // (B H, spans, M, N)
  const float* total;    // (B H, spans): roots of the decays
  const float* s0;       // or null
  int64_t sm, sn;        // strides of s0
  int32_t inner, N, spans;   // M x N
};

template <int V, int U>
__global__ __launch_bounds__(256) void k_join_spans(JoinParams p) {
  typedef float fvec __attribute__((ext_vector_type(V)));
  const uint32_t blocks = (uint32_t(p.inner) + 256 * V - 1) / (256 * V), bh = blockIdx.x / blocks;
  const uint32_t e = (blockIdx.x % blocks * 256 + threadIdx.x) * V;
  if (e >= uint32_t(p.inner)) return;
  float* s = p.sum + int64_t(bh) * p.spans * p.inner + e;
  const float* tot = p.total + int64_t(bh) * p.spans;
  fvec run = fvec(0.0f);
  if (p.s0) {
#pragma unroll
    for (int i = 0; i < V; ++i)
      run[i] = p.s0[int64_t(bh) * p.inner + (e + i) / uint32_t(p.N) * p.sm + (e + i) % uint32_t(p.N) * p.sn];
  }
  const int last = p.spans - 2;   // the last span's end joins nothing
  for (int k = 0; k <= last; k += U) {
    fvec v[U];
    float f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = k + u < last ? k + u : last;
      v[u] = *reinterpret_cast<const fvec*>(s + int64_t(i) * p.inner);
      f[u] = tot[i];
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u <= last) {
        run = run * f[u] * f[u] + v[u];
        v[u] = run;
      }
    // the state entering span k + u + 1: slot k + u of the carries, which start
    // with the second span
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (k + u <= last) *reinterpret_cast<fvec*>(s + int64_t(k + u) * p.inner) = v[u];
  }
}

struct DecayGradParams {
  Rows q, k, v, dout;
  Decay g;
  const float* reads;    // (slices, B, H, padded): exp(b_i) q_i . (S dout_i)
  const float* writes;   // the same: exp(b_end - b_j) k_j . (G v_j), with the decay behind the chunk
  const float* flow;     // (slices, B, H, padded / CT): <S, G>
  const int32_t* lengths;
  void* dg;              // (B, L, H)
  int64_t B, L, H, padded;
  int32_t dk, dv, slices, bf16;
};

// The decay's gradient, a workgroup to a chunk of CT tokens of a head: the two
// score matrices, a query tile to a wave, their product with the decays, its sums
// over keys before and queries from each token, and the sums that the passes left.
// Decays are summed without the resets, which are counted instead: what passes one
// is 0 whatever grows.  Sums over tokens run forward or back from their own end, so
// that no value reaches a token it does not pass.  Bound by the waits of a chunk's
// few steps on each other: 4 x 4096 x 20 heads of 128 x 128 bf16 in 76 us (four
// workgroups to a CU; 90 with three), 4 x 1024 x 24 of 64 x 64 fp32 in 33 us.
template <typename T, int CT, bool FAST>
__global__ __launch_bounds__(256, (FAST ? 4 : 3)) void k_decay_grad(DecayGradParams p) {
  using LD = Lds<T>;
  constexpr int QT = CT / 16, COLS = sizeof(T) == 2 ? 128 : 64, kStride = COLS + LD::kPad;
  __shared__ __align__(16) T sQ[CT * kStride];
  __shared__ __align__(16) T sK[CT * kStride];
  __shared__ __align__(16) float sBh[CT], sBl[CT];
  __shared__ __align__(16) int sResets[CT];
  __shared__ float sPairs[QT][CT], sReads[CT], sWrites[CT], sFlow;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t chunks = p.padded / CT;
  for (int64_t id = blockIdx.x; id < p.B * p.H * chunks; id += gridDim.x) {
    const int64_t bh = id / chunks, b = bh / p.H, h = bh % p.H;
    const int64_t low = id % chunks * CT, live = live_tokens(p.lengths, b, p.L);
    if (low >= p.L) continue;
    const int rows = live - low < CT ? int(live - low) : CT;   // with tokens; at most 0: none
    const int orows = p.L - low < CT ? int(p.L - low) : CT;
    float out = 0.0f;   // token tid's
    if (rows > 0) {
      const T* pq[2] = {row_base<T>(p.q, b, h), row_base<T>(p.dout, b, h)};
      const T* pk[2] = {row_base<T>(p.k, b, h), row_base<T>(p.v, b, h)};
      const int64_t sq[2] = {p.q.st, p.dout.st}, sk[2] = {p.k.st, p.v.st};
      Stage<T, CT, COLS, 256, FAST> rq, rk;
      const int width[2] = {p.dk, p.dv};
      auto fetch = [&](int m, int c0) {
        rq.load(pq[m], sq[m], low, live, c0, width[m]);
        rk.load(pk[m], sk[m], low, live, c0, width[m]);
      };
      fetch(0, 0);
      // what the passes left: a sum each to a wave
      const int64_t n = p.B * p.H * p.padded, at = bh * p.padded + low;
      if (w == 0) {
        const float gr = lane < rows ? log_decay(p.g, b, low + lane, h) : 0.0f;
        const float gn = low + CT < live ? log_decay(p.g, b, low + CT, h) : 0.0f;
        const bool reset = gr < kMinLogDecay;
        const uint64_t resets = __ballot(reset);
        const double bs = wave_running_sum(reset ? 0.0f : gr * kLog2e), tot = last_lane(bs) + gn * kLog2e;
        if (lane < CT) {
          const float hi = float(bs);
          sBh[lane] = hi;
          sBl[lane] = float(bs - hi);
          sResets[lane] = __popcll(resets & (2ull << lane) - 1);
        }
        // at most 16 slices: the first lanes
        const float f = row_sum(lane < p.slices ? p.flow[(lane * p.B * p.H + bh) * chunks + low / CT] : 0.0f);
        const float e = exp2_half(float(tot));
        if (lane == 0) sFlow = resets || gn < kMinLogDecay ? 0.0f : f * e * e;
      } else if (w < 3) {
        // reads: of the lane's token and those behind it; writes: of those before it
        const int t = w == 1 ? CT - 1 - lane : lane;
        const float* from = (w == 1 ? p.reads : p.writes) + at + t;
        float x = 0.0f;
        if (t >= 0 && t < rows)
          for (int k0 = 0; k0 < p.slices; k0 += 8) {   // eight reads in flight, the last again where fewer are left
            float v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = from[(k0 + k < p.slices ? k0 + k : p.slices - 1) * n];
#pragma unroll
            for (int k = 0; k < 8; ++k) x += k0 + k < p.slices ? v[k] : 0.0f;
          }
        const double sum = wave_running_sum(x), before = __shfl_up(sum, 1);
        if (lane < CT) {
          if (w == 1)
            sReads[t] = float(sum);
          else
            sWrites[t] = lane > 0 ? float(before) : 0.0f;
        }
      }
      f32x4 score[2][QT];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
#pragma unroll
        for (int kt = 0; kt < QT; ++kt) score[m][kt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int c0 = 0; c0 < width[m]; c0 += COLS) {
          __syncthreads();
          rq.template store<false>(sQ, kStride);
          rk.template store<false>(sK, kStride);
          __syncthreads();
          if (c0 + COLS < width[m])
            fetch(m, c0 + COLS);
          else if (m == 0)
            fetch(1, 0);
          const int blocks = (width[m] - c0 < COLS ? width[m] - c0 + 31 : COLS) / 32;
          if (w < QT)
            for (int t = 0; t < blocks; ++t) {
              const Operand<T> a = LD::along(sQ + (16 * w + r) * kStride, t, g);
#pragma unroll
              for (int kt = 0; kt < QT; ++kt)
                if (kt <= w) score[m][kt] = mma(LD::along(sK + (16 * kt + r) * kStride, t, g), a, score[m][kt]);
            }
        }
      }
      if (w < QT) {
        const int query = 16 * w + r;
        const float qh = sBh[query], ql = sBl[query];
        const int qr = sResets[query];
        float run = 0.0f;   // of the tiles of keys before
#pragma unroll
        for (int kt = 0; kt < QT; ++kt) {
          if (kt > w) continue;
          float m[4], sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = 16 * kt + 4 * g + i;
            const float f = exp2_half((qh - sBh[key]) + (ql - sBl[key]));
            const float x = score[0][kt][i] * score[1][kt][i] * f * f;
            m[i] = sum;   // of the lane's keys before
            sum += key < query && query < rows && sResets[key] == qr ? x : 0.0f;
          }
          // of the lanes with keys before, then of all four
          float ahead = sum;
          float o = __shfl_up(ahead, 16);
          ahead += g >= 1 ? o : 0.0f;
          o = __shfl_up(ahead, 32);
          ahead += g >= 2 ? o : 0.0f;
          o = __shfl_up(ahead, 16);
          const float all = __shfl(ahead, 48 + r);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int t = 16 * kt + 4 * g + i;
            const float x = row_sum(t <= query ? run + ((g >= 1 ? o : 0.0f) + m[i]) : 0.0f);
            if (r == 0) sPairs[w][t] = x;
          }
          run += all;
        }
      }
      __syncthreads();
      if (tid < rows) {
        out = sFlow + (sReads[tid] + sWrites[tid]);
#pragma unroll
        for (int q = 0; q < QT; ++q)
          if (q >= tid >> 4) out += sPairs[q][tid];
      }
    }
    if (tid < orows) {
      const int64_t i = (b * p.L + low + tid) * p.H + h;
      if (p.bf16)
        st(static_cast<bf16_t*>(p.dg) + i, out);
      else
        static_cast<float*>(p.dg)[i] = out;
    }
    __syncthreads();   // the sums are read before the next chunk writes its own
  }
}

// Sum over the value heads of a key head: (rows, heads, n) fp32 to (rows, key
// heads, n), in the heads' order.  V = 4 where n is a multiple of it.  Bound by
// memory (16384 tokens, 20 heads to 4, n = 128: 31 to 41 us, 4.9 to 6.5 TB/s,
// partly from the caches that the pass before it filled).
template <typename T, int V>
__global__ __launch_bounds__(256) void k_sum_heads(T* out, const float* in, int64_t total, int32_t n, int32_t per) {
  typedef float fvec __attribute__((ext_vector_type(V)));
  const int64_t step = int64_t(gridDim.x) * 256;
  for (int64_t j = int64_t(blockIdx.x) * 256 + threadIdx.x; j * V < total; j += step) {
    const int64_t i = j * V, row = i / n, c = i % n;   // row: (batch, token, key head)
    const float* p = in + row * per * n + c;
    fvec acc = fvec(0.0f);
    int k = 0;
    for (; k + 4 <= per; k += 4) {
      fvec a[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) a[u] = *reinterpret_cast<const fvec*>(p + (k + u) * int64_t(n));
#pragma unroll
      for (int u = 0; u < 4; ++u) acc += a[u];
    }
    for (; k < per; ++k) acc += *reinterpret_cast<const fvec*>(p + k * int64_t(n));
#pragma unroll
    for (int u = 0; u < V; ++u) st(out + i + u, acc[u]);
  }
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
  int32_t per, dk, dv, g_bf16, tiles;
};

// One token: the state streams through once.  A workgroup of 256 takes LC V
// columns of one head's state (V = 4 side by side where rows are on 16 bytes),
// its LC lanes a row at a time, 256 / LC rows at once; a lane has eight reads in
// flight before it needs the first.  The state's lines are used once a step:
// reads and writes pass the caches by.  o joins the rows over lanes, then waves.
// Bound by memory: 256 x 80 heads of 128 x 64 in 213 us, 6.3 TB/s; 4 x 8 heads of
// 64 x 64 take 4 us.
template <typename T, int V, int LC>
__global__ __launch_bounds__(256) void k_attn_step(AttnStepParams p) {
  typedef float fvec __attribute__((ext_vector_type(V)));
  constexpr int RG = 256 / LC, U = 8;
  __shared__ float sk[256], sq[256];
  __shared__ float so[4][LC * V];
  const int tid = threadIdx.x, lc = tid % LC, rg = tid / LC;
  const uint32_t id = blockIdx.x / uint32_t(p.tiles), bh = id;
  const int n = int(blockIdx.x % uint32_t(p.tiles)) * LC * V + lc * V;
  const int64_t b = bh / uint32_t(p.H), h = bh % uint32_t(p.H), hk = int64_t(uint32_t(h) / uint32_t(p.per));
  const bool on = n < p.dv;
  float* S = p.h + int64_t(bh) * p.dk * p.dv + n;
  fvec s[U];
  auto load = [&](int m0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int m = m0 + u * RG + rg;
      s[u] = fvec(0.0f);
      if (on && m < p.dk) s[u] = __builtin_nontemporal_load(reinterpret_cast<const fvec*>(S + int64_t(m) * p.dv));
    }
  };
  load(0);
  const T* q = static_cast<const T*>(p.q) + b * p.qs[0] + hk * p.qs[1];
  const T* k = static_cast<const T*>(p.k) + b * p.ks[0] + hk * p.ks[1];
  const T* v = static_cast<const T*>(p.v) + b * p.vs[0] + h * p.vs[1];
  if (tid < p.dk) {
    sk[tid] = ld(k + tid);
    sq[tid] = ld(q + tid);
  }
  fvec vv = fvec(0.0f);
  if (on) {
#pragma unroll
    for (int i = 0; i < V; ++i) vv[i] = ld(v + n + i);
  }
  const Decay d{p.g, p.gs[0], 0, p.gs[1], p.g_bf16};
  const float f = exp2_half(log_decay(d, b, 0, h) * kLog2e);
  __syncthreads();
  fvec acc = fvec(0.0f);
  for (int m0 = 0; m0 < p.dk; m0 += RG * U) {
    if (m0 > 0) load(m0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int m = m0 + u * RG + rg;
      if (m < p.dk) {
        s[u] = s[u] * f * f + sk[m] * vv;
        acc += s[u] * sq[m];
        if (on) __builtin_nontemporal_store(s[u], reinterpret_cast<fvec*>(S + int64_t(m) * p.dv));
      }
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
#pragma unroll
    for (int w = LC; w < 64; w <<= 1) acc[i] += __shfl_xor(acc[i], w);
    if ((tid & 63) < LC) so[tid >> 6][lc * V + i] = acc[i];
  }
  __syncthreads();
  const int c = int(blockIdx.x % uint32_t(p.tiles)) * LC * V + tid;
  if (tid < LC * V && c < p.dv)
    st(static_cast<T*>(p.o) + int64_t(bh) * p.dv + c, (so[0][tid] + so[1][tid]) + (so[2][tid] + so[3][tid]));
}

static __global__ void k_attn_state_copy(float* dst, const float* src, int64_t n) {
  const int64_t step = int64_t(gridDim.x) * blockDim.x;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) dst[i] = src ? src[i] : 0.0f;
}

}  // namespace ssma
