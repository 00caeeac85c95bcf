// packed_scan.hpp -- gfx950 device code of the selective scan over packed
// sequences: the recurrence and the lane layout of ssm_kernels.hpp (lane = channel
// with its N states in registers, wave = 64 channels of one chunk of tokens, B and C
// rows through scalar loads), with
//
//   * chunks cut from the packed token axis, whatever sequences they meet.  Within
//     a chunk a sequence's first token replaces the state (by its slot's, or 0), its
//     last one hands it to its slot;
//   * the summary pass walking only what reaches past a chunk's end: from the
//     first token of the sequence that goes on, where that lies in the chunk, with
//     its own initial state.  Nothing from before the chunk passes such a
//     token, so the carry walk starts anew there (reset);
//   * states updated in place: of the sequences that begin in a chunk only the
//     last can go on past it, where another workgroup writes its slot.  The
//     summary pass leaves that one's initial state in the workspace, and the output
//     pass takes it from there.
//
// Bound by VALU issue as the scan is: an exp and about five operations for each
// (token, channel, state) and pass.
#pragma once

#include "packed.hpp"

namespace ssmp {

using namespace ssmk;
using ssmq::Seqs;
using ssmq::seq_resumed;
using ssmq::seq_slot;
using ssmq::seq_start;
using ssmq::seqs_before;

struct PackedParams {
  const void* x;
  const void* delta;
  const void* z;         // or null
  const void* Bm;
  const void* Cm;
  const float* A;
  const float* Dskip;    // or null
  const float* dt_bias;  // or null
  const float* h0;       // (slots, D, N) or null
  float* h_last;         // (slots, D, N) or null; may be h0
  float* hsave;          // state before tokens 16, 32, ..., or null
  void* y;
  float* dsum;           // (nc - 1, D)     sums of Delta of the chunks' ends
  float* hsum;           // (nc - 1, D, N)  states the chunks reach, then carries
  float* hstart;         // (nc - 1, D, N)  initial states kept for the output pass, or null
  int32_t* reset;        // (nc - 1)        1: nothing from before the chunk leaves it
  int64_t xs, dls, zs;   // row strides
  uint32_t bs, cs;
  int64_t D;
  Seqs q;
  int32_t T, nc;         // tokens per chunk, chunks
  int32_t dtiles, nwg;
  float exact_thr;
  int32_t dt_mode;
};

// A row of B or C in scalar registers, as it lies in memory; bf16 rows are widened
// when their step comes, so that the row requested ahead takes half the registers
// (the steps of 16 states have none to spare).  A bf16 row of one element is the word
// that holds it, shifted as it is widened (16384 x 2560: 179 us, and 229 read by itself
// through the vector unit).  ODD: longer bf16 rows that may start on an odd element are
// read by elements, which waits for each row (words and shifts spill: 16384 x 2561 with
// rows of 16 769 us, this 536).
template <int N, typename InT, bool ODD>
struct Row {
  static constexpr bool kWide = std::is_same<InT, float>::value;
  static constexpr int W = kWide || N == 1 ? N : N / 2;
  uint32_t w[W];
  uint32_t shift;   // of a bf16 row of one element
  __device__ __forceinline__ void load(const InT* p) {
    if constexpr (!kWide && N == 1) {
      const uint64_t at = reinterpret_cast<uint64_t>(p);
      shift = uint32_t(at & 2) * 8;
      w[0] = *(const_u32_ptr)(at & ~uint64_t(3));
    } else if constexpr (!kWide && ODD) {
      uint32_t v[N];
#pragma unroll
      for (int n = 0; n < N; ++n) v[n] = __builtin_amdgcn_readfirstlane(uint32_t(p[n]));
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = v[2 * k] | v[2 * k + 1] << 16;
    } else {
      const_u32_ptr q = (const_u32_ptr)(p);
#pragma unroll
      for (int k = 0; k < W; ++k) w[k] = q[k];
    }
  }
  __device__ __forceinline__ void widen(float (&r)[N]) const {
    if constexpr (!kWide && N == 1) {
      r[0] = __uint_as_float(w[0] >> shift << 16);
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n)
        r[n] = __uint_as_float(kWide ? w[n] : n % 2 == 0 ? w[n / 2] << 16 : w[n / 2] & 0xffff0000u);
    }
  }
};

// Rows of one array in a chunk: a buffer window at the wave's channels.
struct RowWindow {
  __amdgpu_buffer_rsrc_t r;
  uint32_t row;   // bytes
};
template <typename InT>
__device__ __forceinline__ RowWindow window(const void* p, int64_t stride, int64_t D, int64_t dbase, int32_t from,
                                            int32_t steps) {
  const InT* base = static_cast<const InT*>(p) + int64_t(from) * stride + dbase;
  RowWindow w;
  w.row = uint32_t(stride * sizeof(InT));
  const int64_t wide = (D - dbase < kWave ? D - dbase : kWave) * int64_t(sizeof(InT));
  w.r = make_rsrc(base, steps > 0 ? uint32_t((steps - 1) * int64_t(w.row) + wide) : 0u);
  return w;
}

// The kernel's arguments, read again: what only the ends of sequences need would
// otherwise stay in scalar registers through the steps, which have none to spare.
template <typename P>
__device__ __forceinline__ const P& args_again() {
  typedef const P __attribute__((address_space(4)))* arg_ptr;
  arg_ptr p = (arg_ptr)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const P*)p;
}

template <int N>
__device__ __forceinline__ void load_n(float (&h)[N], const float* p) {
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = p[n];
}
template <int N>
__device__ __forceinline__ void store_n(float* p, const float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) p[n] = h[n];
}
template <int N>
__device__ __forceinline__ void zero_n(float (&h)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) h[n] = 0.0f;
}

// |Delta A| log2(e) below this takes the slow-decay form of its step (see
// ssm_kernels.hpp): the scan's threshold, state by state.
__device__ __forceinline__ bool any_slow(float z2, float limit) {
  return __builtin_amdgcn_ballot_w64(fabsf(z2) < limit) != 0;
}

// One step of a lane's N states.  Where some lane has a decay that slow at all, the
// form is chosen for every GROUP states on their own: with A[n] about -(n + 1) and
// steps down to 1e-3, two of three steps are slow for the first state and none for
// the others (16384 x 1536 x 16 fp32: 88 us for the summaries with one choice for all
// 16 states, 80 so; the output pass 127, 121 so).  GROUP = N makes one choice: for
// bf16, whose limit is an eighth of fp32's and seldom met, the choices' code costs more
// than they save (16384 x 2560 x 16: 305 us a call, 316 by fours).  SCALED carries A h (see
// ssm_step_lane), SELECT is exp_residual's.
template <int N, int DISC, bool SCALED, int GROUP, bool SELECT>
__device__ __forceinline__ void advance(float (&h)[N], const ChanConst<N, DISC>& cc, const float (&Bv)[N], float u,
                                        float dv, float limit) {
  const float du = dv * u;
  auto fast = [&](int n) {
    const float a = exp2_fast(dv * cc.A2[n]);
    if constexpr (SCALED) {
      const float bu = u * Bv[n];
      h[n] = fmaf(a, h[n] + bu, -bu);
    } else if constexpr (DISC == kDeltaB) {
      h[n] = fmaf(a, h[n], du * Bv[n]);
    } else {
      const float q = (u * Bv[n]) * cc.invA[n];
      h[n] = fmaf(a, h[n] + q, -q);
    }
  };
  auto slow = [&](int n) {
    const float z2 = dv * cc.A2[n], a = exp2_fast(z2), r = exp_residual<SELECT>(z2, a);
    if constexpr (SCALED) {
      const float bu = u * Bv[n];
      h[n] = fmaf(a, h[n], fmaf((a - 1.0f) + r, bu, r * h[n]));   // (a - 1) + r = expm1
    } else {
      float gu = du;
      if constexpr (DISC == kZoh)
        gu = (cc.invA[n] != 0.0f) ? (((a - 1.0f) + r) * cc.invA[n]) * u : du;   // A = 0: limit Delta
      h[n] = fmaf(a, h[n], fmaf(gu, Bv[n], r * h[n]));
    }
  };
  if (__builtin_amdgcn_ballot_w64(dv < cc.thr) == 0) {   // wave-uniform, as all these choices
#pragma unroll
    for (int n = 0; n < N; ++n) fast(n);
    return;
  }
  constexpr int G = GROUP < N ? GROUP : N;
  if constexpr (G == N && N > 4) {
#pragma unroll
    for (int n = 0; n < N; ++n) slow(n);
    return;
  }
#pragma unroll
  for (int g = 0; g < N; g += G) {
    float least = fabsf(dv * cc.A2[g]);
#pragma unroll
    for (int n = g + 1; n < g + G; ++n) least = fminf(least, fabsf(dv * cc.A2[n]));
    if (any_slow(least, limit)) {
#pragma unroll
      for (int n = g; n < g + G; ++n) slow(n);
    } else {
#pragma unroll
      for (int n = g; n < g + G; ++n) fast(n);
    }
  }
}

template <int N, typename InT>
constexpr int kGroup = std::is_same<InT, float>::value ? 4 : N;

// Pass 1: what each chunk but the last hands on.
template <int N, typename InT, int DISC, bool ODD>
__global__ void __launch_bounds__(kWave) __attribute__((amdgpu_waves_per_eu(4))) k_packed_summary(const PackedParams p) {
  constexpr int kU = kUnrollSum;
  constexpr bool kScaled = DISC == kZoh;   // carries A h (see ssm_step_lane)
  const int wg = xcd_remap(blockIdx.x, p.nwg);
  const int64_t dbase = int64_t(wg % p.dtiles) * kWave;
  const int32_t chunk = wg / p.dtiles;
  const int32_t t0 = chunk * p.T, t1 = t0 + p.T;
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, p.q.S);
  int32_t from = t1, fresh = 1, open = -1;
  if (t1 > lo && t1 < hi) {
    const int32_t s = seqs_before(p.q, t1);
    if (s > 0 && seq_start(p.q, s) > t1) {   // sequence s - 1 goes on
      const int32_t first = seq_start(p.q, s - 1);
      fresh = first >= t0;
      from = !fresh ? t0 : first < t1 ? first : t1 - 1;
      open = s - 1;
    }
  }
  if (dbase == 0 && threadIdx.x == 0) p.reset[chunk] = fresh;
  if (open < 0) return;

  const uint32_t lo_ch = lane_offset(dbase, p.D);
  const int64_t d = dbase + lo_ch;
  ChanConst<N, DISC> cc;
  load_chan<N, DISC>(cc, p.A + d * N, p.exact_thr);
  const float limit = p.exact_thr * kLog2e;
  float h[N];
  zero_n(h);
  if (fresh && p.h0) {
    const int32_t slot = seq_slot(p.q, open);
    if (slot >= 0 && seq_resumed(p.q, open)) load_n(h, p.h0 + (int64_t(slot) * p.D + d) * N);
    if (p.hstart) store_n(p.hstart + (int64_t(chunk) * p.D + d) * N, h);
  }
  if constexpr (kScaled) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float a = scaled_a(p.A[d * N + n]);
      cc.A2[n] = a * kLog2e;
      h[n] *= a;
    }
  }
  const int dtm = p.dt_mode;
  const float dtb = p.dt_bias ? p.dt_bias[d] : 0.0f;
  const int32_t steps = t1 - from;
  const RowWindow wx = window<InT>(p.x, p.xs, p.D, dbase, from, steps);
  const RowWindow wd = window<InT>(p.delta, p.dls, p.D, dbase, from, steps);
  const uint32_t lane = lo_ch * sizeof(InT);
  constexpr InT* kIn = nullptr;
  const InT* Brow = static_cast<const InT*>(p.Bm) + int64_t(from) * p.bs;
  Row<N, InT, ODD> Bb0, Bb1;
  Bb0.load(Brow);

  float dacc = 0.0f, dcomp = 0.0f;   // Kahan sum of Delta, as in the scan's summaries
  auto sum_add = [&](float v) {
    const float yv = v - dcomp, tv = dacc + yv;
    dcomp = (tv - dacc) - yv;
    dacc = tv;
  };
  // the next row is requested after this step's has been waited for (see chunk_loop)
  auto one_step = [&](float xv, float dv, const Row<N, InT, ODD>& Bcur, Row<N, InT, ODD>& Bnext) {
    const InT* nb = Brow + p.bs;
    asm volatile("" : "+s"(nb) : "s"(Bcur.w[0]));
    Bnext.load(nb);
    float Bv[N];
    Bcur.widen(Bv);
    advance<N, DISC, kScaled, kGroup<N, InT>, false>(h, cc, Bv, xv, dv, limit);
    Brow = nb;
  };
  float xc[kU], dc[kU];
  auto at = [&](int32_t t) { return uint32_t(t < steps ? t : steps - 1); };
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    xc[j] = ldb(wx.r, lane, at(j) * wx.row, kIn);
    dc[j] = ldb(wd.r, lane, at(j) * wd.row, kIn);
  }
  int32_t t = 0;
  for (; t + kU < steps; t += kU) {
    float xn[kU], dn[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      xn[j] = ldb(wx.r, lane, at(t + kU + j) * wx.row, kIn);
      dn[j] = ldb(wd.r, lane, at(t + kU + j) * wd.row, kIn);
    }
    if (dtm != kDtRaw) {
#pragma unroll
      for (int j = 0; j < kU; ++j) dc[j] = dt_transform(dc[j], dtb, dtm);
    }
    float bs = 0.0f;
#pragma unroll
    for (int j = 0; j < kU; j += 2) {
      one_step(xc[j], dc[j], Bb0, Bb1);
      one_step(xc[j + 1], dc[j + 1], Bb1, Bb0);
      bs += dc[j] + dc[j + 1];
    }
    sum_add(bs);
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      xc[j] = xn[j];
      dc[j] = dn[j];
    }
  }
  // the last block, step by step; no row behind its last is read
#pragma unroll 1
  for (; t < steps; ++t) {
    const float xv = ldb(wx.r, lane, uint32_t(t) * wx.row, kIn);
    float dv = ldb(wd.r, lane, uint32_t(t) * wd.row, kIn);
    if (dtm != kDtRaw) dv = dt_transform(dv, dtb, dtm);
    float Bv[N];
    Bb0.widen(Bv);
    advance<N, DISC, kScaled, kGroup<N, InT>, false>(h, cc, Bv, xv, dv, limit);
    sum_add(dv);
    Brow += t + 1 < steps ? p.bs : 0u;
    Bb0.load(Brow);
  }
  if constexpr (kScaled) {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] /= scaled_a(p.A[d * N + n]);
  }
  store_n(p.hsum + (int64_t(chunk) * p.D + d) * N, h);
  p.dsum[int64_t(chunk) * p.D + d] = dacc - dcomp;
}

// Pass 2: carries; hsum of chunk c becomes the state that enters chunk c + 1.  A lane
// per (channel, state); the 16 waves of a workgroup share the chunks of its 64.  Each
// folds its share from zero, takes the state that enters it from the shares
// before (in LDS), and walks it again.  A chunk's fold is 25 instructions, so one wave
// walking 512 chunks alone took 50 us, which nothing else overlaps; 16 share them in 20.
constexpr int kCarryWaves = 16;

template <int N, bool REV>
__device__ __forceinline__ void carry_walk(const float* A, const float* dsum, float* hsum, const int32_t* reset, int64_t D,
                                           int32_t n) {
  constexpr int U = 8;   // chunks whose loads are issued before they are folded
  __shared__ float end[kCarryWaves][kWave];
  __shared__ float span[kCarryWaves][kWave];
  __shared__ int32_t cut[kCarryWaves];
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), lane = threadIdx.x % kWave;
  const int64_t DN = D * N, i0 = int64_t(blockIdx.x) * kWave + lane, i = i0 < DN ? i0 : DN - 1;
  const float a2 = A[i] * kLog2e;
  const float* ds = dsum + i / N;
  float* hs = hsum + i;
  const int32_t share = (n + kCarryWaves - 1) / kCarryWaves;
  const int32_t c0 = w * share < n ? w * share : n, c1 = c0 + share < n ? c0 + share : n;
  auto place = [&](int32_t c) { return int64_t(REV ? n - 1 - c : c); };
  // REV: the chunks from the last to the first
  auto walk = [&](float carry, auto&& each) {
    for (int32_t c = c0; c < c1; c += U) {
      float sv[U], hv[U];
      int32_t rv[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int64_t at = place(c + j < c1 ? c + j : c1 - 1);
        sv[j] = ds[at * D];
        hv[j] = hs[at * DN];
        rv[j] = reset[at];
      }
#pragma unroll
      for (int j = 0; j < U; ++j)
        if (c + j < c1) {
          carry = rv[j] ? hv[j] : decay_add(a2 * sv[j], carry, hv[j]);
          each(c + j, sv[j], rv[j], carry);
        }
    }
    return carry;
  };
  double sum = 0.0;   // of Delta, while no chunk starts anew
  int32_t anew = 0;
  end[w][lane] = walk(0.0f, [&](int32_t, float sv, int32_t rv, float) {
    sum += sv;
    anew |= rv;
  });
  span[w][lane] = float(sum);
  if (lane == 0) cut[w] = anew;
  __syncthreads();
  float carry = 0.0f;
  for (int v = 0; v < w; ++v) carry = cut[v] ? end[v][lane] : decay_add(a2 * span[v][lane], carry, end[v][lane]);
  walk(carry, [&](int32_t c, float, int32_t, float now) {
    if (i0 < DN) hs[place(c) * DN] = now;
  });
}

template <int N>
__global__ void __launch_bounds__(kWave * kCarryWaves) k_packed_carry(const PackedParams p) {
  carry_walk<N, false>(p.A, p.dsum, p.hsum, p.reset, p.D, p.nc - 1);
}

// Pass 3 (or the only one): every chunk from the state that enters it.
template <int N, typename InT, int DISC, bool GATE, bool ODD>
__global__ void __launch_bounds__(kWave) __attribute__((amdgpu_waves_per_eu(4))) k_packed_out(const PackedParams p) {
  constexpr int kU = kUnrollOut;
  const int wg = xcd_remap(blockIdx.x, p.nwg);
  const int64_t dbase = int64_t(wg % p.dtiles) * kWave;
  const int32_t chunk = wg / p.dtiles;
  const int32_t t0 = chunk * p.T, t1 = p.q.tokens - t0 > p.T ? t0 + p.T : p.q.tokens;
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, p.q.S);
  const int32_t from = t0 > lo ? t0 : lo, to = t1 < hi ? t1 : hi;
  const uint32_t lo_ch = lane_offset(dbase, p.D);
  const int64_t d = dbase + lo_ch, DN = p.D * N;
  ChanConst<N, DISC> cc;
  load_chan<N, DISC>(cc, p.A + d * N, p.exact_thr);
  const float limit = p.exact_thr * kLog2e;
  float h[N];
  zero_n(h);

  // s: the first sequence not begun; open: sequence s - 1 holds the tokens walked
  int32_t s = seqs_before(p.q, from);
  bool open = false;
  if (chunk > 0 && s > 0 && from < to && seq_start(p.q, s) > from) {
    open = true;
    load_n(h, p.hsum + (int64_t(chunk) - 1) * DN + d * N);
  }
  // where the open sequence ends, or else the next one begins
  auto next_of = [&](const PackedParams& a) { return open || s < a.q.S ? seq_start(a.q, s) : INT32_MAX; };
  auto finish = [&](const PackedParams& a) {
    if (!open) return;
    const int32_t slot = a.h_last ? seq_slot(a.q, s - 1) : -1;
    if (slot >= 0) store_n(a.h_last + (int64_t(slot) * a.D + d) * N, h);
    open = false;
  };
  // At token t the open sequence has ended; empty ones pass their state on, and the
  // one that holds t is opened.
  auto meet = [&](const PackedParams& a, int32_t t) {
    finish(a);
    const int64_t last = int64_t(chunk + 1) * a.T;   // (past 32 bits in the last chunk)
    while (!open && s < a.q.S && seq_start(a.q, s) <= t) {
      const int32_t end = seq_start(a.q, s + 1), slot = seq_slot(a.q, s);
      const bool given = a.h0 && slot >= 0 && seq_resumed(a.q, s);
      zero_n(h);
      if (given) {
        const float* from_state = end > last && a.hstart ? a.hstart + int64_t(chunk) * a.D * N : a.h0 + int64_t(slot) * a.D * N;
        load_n(h, from_state + d * N);
      }
      open = true;
      ++s;
      if (end <= t) finish(a);
    }
  };

  const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
  const int dtm = p.dt_mode;
  const float dtb = p.dt_bias ? p.dt_bias[d] : 0.0f;
  const int32_t steps = to - from;
  if (steps > 0) {
    const RowWindow wx = window<InT>(p.x, p.xs, p.D, dbase, from, steps);
    const RowWindow wd = window<InT>(p.delta, p.dls, p.D, dbase, from, steps);
    const RowWindow wz = window<InT>(GATE ? p.z : p.x, GATE ? p.zs : p.xs, p.D, dbase, from, GATE ? steps : 0);
    const RowWindow wy = window<InT>(p.y, p.D, p.D, dbase, from, steps);
    const uint32_t lane = lo_ch * sizeof(InT);
    uint32_t yoff = 0;
    constexpr InT* kIn = nullptr;
    const InT* Brow = static_cast<const InT*>(p.Bm) + int64_t(from) * p.bs;
    const InT* Crow = static_cast<const InT*>(p.Cm) + int64_t(from) * p.cs;
    using R = Row<N, InT, ODD>;
    R Bb0, Bb1;
    Bb0.load(Brow);
    // where the walk stops to keep a state (before tokens 16, 32, ...) or to change
    // sequences, and the step before which it goes block by block (the last step's next
    // row is not there to be read)
    int32_t stop, whole;
    auto set_stop = [&](const PackedParams& a, int32_t t) {
      const int32_t keep = a.hsave ? (t / kSaveStride + 1) * kSaveStride : INT32_MAX, next = next_of(a);
      stop = (next < keep ? next : keep) - from;
      whole = stop < steps - 1 ? stop : steps - 1;
    };
    auto halt = [&](int32_t t) {
      const PackedParams& a = args_again<PackedParams>();
      if (a.hsave && t % kSaveStride == 0 && t > 0)
        store_n(a.hsave + ((int64_t(t / kSaveStride) - 1) * a.D + d) * N, h);
      if (next_of(a) <= t) meet(a, t);
      set_stop(a, t);
    };
    halt(from);
    // B's next row and C's own are requested once this step's B has been waited for
    // (scalar loads come back in any order, so a wait is for all of them): the states'
    // update covers both.  (C a step ahead too takes 16 registers more, which spilled:
    // 16384 x 1536 x 16 fp32: the pass took 150 us so, then 127.)
    auto one_step = [&](float xv, float dv, float zv, uint32_t ahead, const R& Bcur, R& Bnext) {
      const InT* nb = Brow + ahead;
      const InT* nc = Crow;
      asm volatile("" : "+s"(nb), "+s"(nc) : "s"(Bcur.w[0]));
      R Ccur;
      Ccur.load(nc);
      Bnext.load(nb);
      float Bv[N], Cv[N];
      Bcur.widen(Bv);
      advance<N, DISC, false, kGroup<N, InT>, false>(h, cc, Bv, xv, dv, limit);
      Ccur.widen(Cv);
      float even = 0.0f, odd = 0.0f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        if (n & 1)
          odd = fmaf(Cv[n], h[n], odd);
        else
          even = fmaf(Cv[n], h[n], even);
      }
      float yv = fmaf(dsk, xv, even + odd);
      if constexpr (GATE) yv *= silu(zv);
      stb(wy.r, lane, yoff, yv, static_cast<InT*>(nullptr));
      yoff += wy.row;
      Brow = nb;
      Crow = nc + p.cs;
    };
    float xc[kU], dc[kU], zc[kU];
    auto at = [&](int32_t t) { return uint32_t(t < steps ? t : steps - 1); };
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      xc[j] = ldb(wx.r, lane, at(j) * wx.row, kIn);
      dc[j] = ldb(wd.r, lane, at(j) * wd.row, kIn);
      zc[j] = GATE ? ldb(wz.r, lane, at(j) * wz.row, kIn) : 0.0f;
    }
    for (int32_t tb = 0; tb < steps; tb += kU) {
      float xn[kU], dn[kU], zn[kU];
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        xn[j] = ldb(wx.r, lane, at(tb + kU + j) * wx.row, kIn);
        dn[j] = ldb(wd.r, lane, at(tb + kU + j) * wd.row, kIn);
        zn[j] = GATE ? ldb(wz.r, lane, at(tb + kU + j) * wz.row, kIn) : 0.0f;
      }
      if (dtm != kDtRaw) {
#pragma unroll
        for (int j = 0; j < kU; ++j) dc[j] = dt_transform(dc[j], dtb, dtm);
      }
      if (tb == stop) halt(from + tb);
      if (tb + kU <= whole) {
#pragma unroll
        for (int j = 0; j < kU; j += 2) {
          one_step(xc[j], dc[j], zc[j], p.bs, Bb0, Bb1);
          one_step(xc[j + 1], dc[j + 1], zc[j + 1], p.bs, Bb1, Bb0);
        }
      } else {
        // a stop within the block, or the last block: step by step
#pragma unroll 1
        for (int32_t t = tb; t < tb + kU && t < steps; ++t) {
          if (t == stop) halt(from + t);
          const float xv = ldb(wx.r, lane, uint32_t(t) * wx.row, kIn);
          float dv = ldb(wd.r, lane, uint32_t(t) * wd.row, kIn);
          const float zv = GATE ? ldb(wz.r, lane, uint32_t(t) * wz.row, kIn) : 0.0f;
          if (dtm != kDtRaw) dv = dt_transform(dv, dtb, dtm);
          one_step(xv, dv, zv, t + 1 < steps ? p.bs : 0u, Bb0, Bb1);
          Bb0 = Bb1;
        }
      }
#pragma unroll
      for (int j = 0; j < kU; ++j) {
        xc[j] = xn[j];
        dc[j] = dn[j];
        zc[j] = zn[j];
      }
    }
  }
  // behind the last token walked: the sequence that ends there, and the empty ones
  // whose place is in this chunk
  const int32_t at = from > to ? from : to;
  const PackedParams& a = args_again<PackedParams>();
  if (at < t1 || t1 == a.q.tokens) {
    if (open || next_of(a) <= at) meet(a, at);
  } else if (open && next_of(a) <= at) {
    finish(a);
  }
}

// One combine of the lane scan (wave_combine) that stops at sequences: ok says whether
// the lane the pair comes from belongs to this lane's sequence.
template <int CTRL, int ROWS, bool RES, int N>
__device__ __forceinline__ void seq_combine(float (&a)[N], float (&r)[N], float (&bb)[N], bool ok) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    float ap = dpp_from<CTRL, ROWS>(a[n], 1.0f), bp = dpp_from<CTRL, ROWS>(bb[n], 0.0f);
    ap = ok ? ap : 1.0f;
    bp = ok ? bp : 0.0f;
    if constexpr (RES) {
      float rp = dpp_from<CTRL, ROWS>(r[n], 0.0f);
      rp = ok ? rp : 0.0f;
      bb[n] = fmaf(a[n], bp, fmaf(r[n], bp, bb[n]));
      const float m = ap * a[n];
      r[n] = fmaf(ap, a[n], -m) + fmaf(ap, r[n], rp * a[n]);
      a[n] = m;
    } else {
      bb[n] = fmaf(a[n], bp, bb[n]);
      a[n] = ap * a[n];
    }
  }
}

// Few tokens of few channels in one launch, with time across the lanes (the scan's
// k_scan_wave): a workgroup to a channel, a wave to four of its states, 64 tokens at a
// time, their pairs (Abar, Bbar u) scanned over the lanes.  A block in which sequences
// begin takes the scan that stops at them (its pairs are chosen, not multiplied by 0,
// which a NaN would pass).  Bound by latency: 128 x 32 x 16 fp32 in three launches
// 19.5 us a call, so 12.
template <int N, typename InT, int DISC, bool GATE>
__global__ void __launch_bounds__(kWave * BwdLayout<N>::NG) k_packed_wave(const PackedParams p) {
  constexpr int NS = BwdLayout<N>::NS, NG = BwdLayout<N>::NG;
  // sequences that begin, and end, at a lane's token (each wave its own)
  __shared__ int32_t first_at[NG][kWave], last_at[NG][kWave];
  __shared__ float part[2][NG][kWave];   // the waves' parts of y, double-buffered by block
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave), lane = threadIdx.x % kWave;
  const int64_t d = blockIdx.x, DN = p.D * N, dn = d * N + w * NS;
  const int32_t tokens = p.q.tokens, S = p.q.S;
  // what the loop needs first is requested at once: a block's rows (of tokens that may
  // belong to no sequence: their values are dropped), and 64 sequences' offsets
  struct Rows {
    InT x, dl, z, B[NS], C[NS];
  };
  auto request = [&](int32_t t0) {
    const int64_t t = tokens - t0 > lane ? t0 + lane : tokens - 1;
    Rows r;
    r.x = static_cast<const InT*>(p.x)[t * p.xs + d];
    r.dl = static_cast<const InT*>(p.delta)[t * p.dls + d];
    if constexpr (GATE) r.z = static_cast<const InT*>(p.z)[t * p.zs + d];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      r.B[n] = static_cast<const InT*>(p.Bm)[t * p.bs + w * NS + n];
      r.C[n] = static_cast<const InT*>(p.Cm)[t * p.cs + w * NS + n];
    }
    return r;
  };
  auto begin_of = [&](int32_t s) { return ssmq::in_tokens(p.q, p.q.offsets[s < S ? s : S]); };
  Rows rows{};
  if (tokens > 0) rows = request(0);
  const bool few = S <= kWave;
  int32_t b0 = begin_of(lane), e0 = begin_of(lane + 1);
  ChanConst<NS, DISC> cc;
  load_chan<NS, DISC>(cc, p.A + dn, p.exact_thr);
  const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
  const int dtm = p.dt_mode;
  const float dtb = p.dt_bias ? p.dt_bias[d] : 0.0f;
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, S);
  // the state sequence s starts from, into h
  auto initial = [&](float (&h)[NS], int32_t s) {
    zero_n(h);
    const int32_t slot = p.q.slot ? p.q.slot[s] : s;
    if (p.h0 && slot >= 0 && slot < p.q.slots && (!p.q.resume || p.q.resume[s])) load_n(h, p.h0 + int64_t(slot) * DN + dn);
  };
  auto keep = [&](const float (&h)[NS], int32_t s) {
    const int32_t slot = p.q.slot ? p.q.slot[s] : s;
    if (p.h_last && slot >= 0 && slot < p.q.slots) store_n(p.h_last + int64_t(slot) * DN + dn, h);
  };
  float hc[NS];   // the state that enters the block (wave-uniform)
  zero_n(hc);
  int32_t t0 = 0;
  do {
    const int32_t t = t0 + lane, limit = tokens - t0 > kWave ? t0 + kWave : tokens + 1;
    first_at[w][lane] = last_at[w][lane] = -1;
    __builtin_amdgcn_wave_barrier();   // (a wave's LDS accesses stay in order)
    for (int32_t s0 = few ? 0 : seqs_before(p.q, t0) - 1; s0 < S; s0 += kWave) {
      const int32_t s = s0 + lane;
      bool more = false;
      if (s >= 0 && s < S) {
        const int32_t b = few ? b0 : begin_of(s), e = few ? e0 : begin_of(s + 1);
        more = b < limit;
        if (e > b) {
          if (b >= t0 && b < t0 + kWave) first_at[w][b - t0] = s;
          if (e > t0 && e <= t0 + kWave) last_at[w][e - 1 - t0] = s;
        } else if (b >= t0 && b < limit) {
          float h[NS];   // a sequence without tokens, whose place is here
          initial(h, s);
          keep(h, s);
        }
      }
      if (!(__builtin_amdgcn_ballot_w64(more) >> (kWave - 1))) break;
    }
    __builtin_amdgcn_wave_barrier();
    Rows next{};
    if (t0 + kWave < tokens) next = request(t0 + kWave);
    if (t0 < hi && t0 + kWave > lo) {
      const int32_t begins = first_at[w][lane], ends = last_at[w][lane];
      const bool in = t >= lo && t < hi;
      float u = ld(&rows.x), dv = ld(&rows.dl);
      if (dtm != kDtRaw) dv = dt_transform(dv, dtb, dtm);
      const float zv = GATE ? ld(&rows.z) : 0.0f;
      float Bv[NS], Cv[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        Bv[n] = ld(&rows.B[n]);
        Cv[n] = ld(&rows.C[n]);
      }
      if (!in) {   // the identity pair: a = exp(0) = 1, b = 0
        u = dv = 0.0f;
        zero_n(Bv);
      }
      float hs[NS];
      zero_n(hs);
      if (begins >= 0) initial(hs, begins);
      // the lane of the last first token at or before this one; -1: before the block
      const uint64_t starts = __builtin_amdgcn_ballot_w64(begins >= 0), at = starts & (~0ull >> (kWave - 1 - lane));
      const int from = at ? kWave - 1 - __builtin_clzll(at) : -1;
      float h[NS];
      auto block = [&](auto form) {
        constexpr bool RES = decltype(form)::value;
        float a[NS], r[NS], bb[NS];
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const float z2 = dv * cc.A2[n];
          a[n] = exp2_fast(z2);
          r[n] = (RES || DISC == kZoh) ? exp_residual<true>(z2, a[n]) : 0.0f;
          float gu;   // the input factor times u
          if constexpr (DISC == kDeltaB) {
            gu = dv * u;
          } else {
            const float e = (a[n] - 1.0f) + r[n];   // expm1(Delta A)
            gu = (cc.invA[n] != 0.0f) ? (e * cc.invA[n]) * u : dv * u;   // A = 0: limit Delta
          }
          bb[n] = gu * Bv[n];
          if (begins >= 0) bb[n] = fmaf(a[n], hs[n], fmaf(RES ? r[n] : 0.0f, hs[n], bb[n]));
        }
        if ((starts & ~1ull) == 0) {   // no sequence begins within the block
          wave_scan<RES>(a, r, bb);
        } else {
          seq_combine<0x111, 0xF, RES>(a, r, bb, lane - 1 >= from);
          seq_combine<0x112, 0xF, RES>(a, r, bb, lane - 2 >= from);
          seq_combine<0x114, 0xF, RES>(a, r, bb, lane - 4 >= from);
          seq_combine<0x118, 0xF, RES>(a, r, bb, lane - 8 >= from);
          seq_combine<0x142, 0xA, RES>(a, r, bb, (lane & ~15) - 1 >= from);
          seq_combine<0x143, 0xC, RES>(a, r, bb, 31 >= from);
        }
#pragma unroll
        for (int n = 0; n < NS; ++n) {
          const float on = RES ? fmaf(a[n], hc[n], fmaf(r[n], hc[n], bb[n])) : fmaf(a[n], hc[n], bb[n]);
          h[n] = from >= 0 ? bb[n] : on;
        }
      };
      if (__builtin_amdgcn_ballot_w64(dv < cc.thr) != 0)
        block(std::true_type{});
      else
        block(std::false_type{});
      float even = 0.0f, odd = 0.0f;
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        if (n & 1)
          odd = fmaf(Cv[n], h[n], odd);
        else
          even = fmaf(Cv[n], h[n], even);
      }
      float sum = even + odd;
      if constexpr (NG > 1) {
        float(&all)[NG][kWave] = part[(t0 / kWave) & 1];
        all[w][lane] = sum;
        __syncthreads();
        sum = all[0][lane];
#pragma unroll
        for (int v = 1; v < NG; ++v) sum += all[v][lane];
      }
      float yv = fmaf(dsk, u, sum);
      if constexpr (GATE) yv *= silu(zv);
      if (in && w == 0) st(static_cast<InT*>(p.y) + int64_t(t) * p.D + d, yv);
      if (ends >= 0) keep(h, ends);
      if (p.hsave && in && t + 1 < tokens && (t + 1) % kSaveStride == 0)
        store_n(p.hsave + (int64_t((t + 1) / kSaveStride) - 1) * DN + dn, h);
#pragma unroll
      for (int n = 0; n < NS; ++n)
        hc[n] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(h[n]), kWave - 1));
    }
    rows = next;
    t0 += kWave;
  } while (t0 < tokens);
}

struct PackedStepParams {
  const void* x;
  const void* delta;
  const void* z;
  const void* Bm;
  const void* Cm;
  const float* A;
  const float* Dskip;
  const float* dt_bias;
  const int32_t* slot;   // or null
  float* h;              // (slots, D, N)
  void* y;
  int64_t xs, dls, zs, bs, cs;
  int64_t Bt, slots, D;
  int32_t dtiles, nwg;
  float exact_thr;
  int32_t dt_mode;
};

// One token per row, in the lane layout of the decode step (StepLayout).  Bound by
// memory: the states once each way.
template <int N, typename InT, int DISC>
__global__ void __launch_bounds__(kWave * StepLayout<N>::WPG) k_packed_step(const PackedStepParams p) {
  constexpr int NL = StepLayout<N>::NL, S = StepLayout<N>::S, CPW = StepLayout<N>::CPW;
  constexpr int ROWS = StepLayout<N>::ROWS, WPG = StepLayout<N>::WPG;
  const int wg = xcd_remap(blockIdx.x, p.nwg);
  const int64_t gtiles = (p.dtiles + WPG - 1) / WPG;
  const int64_t bt = wg / gtiles;
  const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int64_t dtile = (wg - bt * gtiles) * WPG + w;
  if (dtile >= p.dtiles) return;
  const int lane = threadIdx.x % kWave;
  const int j = lane % S;
  // lanes past the last channel repeat it: they read the old state in the same load
  // and store the same values
  int64_t d = dtile * CPW + lane / S;
  if (d > p.D - 1) d = p.D - 1;
  const int n0 = j * NL;
  ChanConst<NL, DISC> cc;
  load_chan<NL, DISC>(cc, p.A + d * N + n0, p.exact_thr);
  const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
  const float dtb = p.dt_bias ? p.dt_bias[d] : 0.0f;
  float h[ROWS][NL], Bv[ROWS][NL], Cv[ROWS][NL], u[ROWS], dv[ROWS], zg[ROWS];
  float* at[ROWS];
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    int64_t b = bt * ROWS + r;
    if (b > p.Bt - 1) b = p.Bt - 1;
    const int64_t slot = p.slot ? ((ssmq::const_i32_ptr)(p.slot))[b] : b;
    at[r] = slot >= 0 && slot < p.slots ? p.h + (slot * p.D + d) * N + n0 : nullptr;
    zero_n(h[r]);
    if (at[r]) load_state<NL>(h[r], at[r]);
    const InT* Bp = static_cast<const InT*>(p.Bm) + b * p.bs + n0;
    const InT* Cp = static_cast<const InT*>(p.Cm) + b * p.cs + n0;
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      Bv[r][n] = ld(Bp + n);
      Cv[r][n] = ld(Cp + n);
    }
    u[r] = ld(static_cast<const InT*>(p.x) + b * p.xs + d);
    dv[r] = ld(static_cast<const InT*>(p.delta) + b * p.dls + d);
    zg[r] = p.z ? ld(static_cast<const InT*>(p.z) + b * p.zs + d) : 0.0f;
  }
#pragma unroll
  for (int r = 0; r < ROWS; ++r) {
    const int64_t b = bt * ROWS + r;
    if (b >= p.Bt) break;
    float dvr = dv[r];
    if (p.dt_mode != kDtRaw) dvr = dt_transform(dvr, dtb, p.dt_mode);
    float acc = ssm_step_any<NL, DISC, true>(h[r], cc, Bv[r], Cv[r], u[r], dvr);
    if constexpr (S >= 2) acc += dpp_quad_xor1(acc);
    if constexpr (S >= 4) acc += dpp_quad_xor2(acc);
    if (at[r]) store_state<NL>(at[r], h[r]);
    if (j == 0) {
      float yv = fmaf(dsk, u[r], acc);
      if (p.z) yv *= silu(zg[r]);
      st(static_cast<InT*>(p.y) + b * p.D + d, yv);
    }
  }
}

}  // namespace ssmp
