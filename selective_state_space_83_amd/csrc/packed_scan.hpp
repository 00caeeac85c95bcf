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
  int64_t xs, dls, zs, bs, cs;   // row strides
  int64_t D;
  Seqs q;
  int32_t T, nc;         // tokens per chunk, chunks
  int32_t dtiles, nwg;
  float exact_thr;
  int32_t dt_mode;
  int32_t rows_ok;       // bf16 rows of B and C start on 4 bytes
};

// A row of B or C into scalar registers.  bf16 rows that start on an odd element
// are read by elements.
template <int N, typename InT>
__device__ __forceinline__ void row_of(float (&r)[N], const InT* p, bool ok) {
  if constexpr (std::is_same<InT, float>::value || N == 1) {
    load_row<N>(r, p);
  } else if (ok) {
    load_row<N>(r, p);
  } else {
#pragma unroll
    for (int n = 0; n < N; ++n)
      r[n] = __uint_as_float(__builtin_amdgcn_readfirstlane(uint32_t(__builtin_bit_cast(uint16_t, p[n])) << 16));
  }
}

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

// Pass 1: what each chunk but the last hands on.
template <int N, typename InT, int DISC>
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
  const bool ok = p.rows_ok != 0;
  float Bb0[N], Bb1[N];
  row_of<N>(Bb0, Brow, ok);

  float dacc = 0.0f, dcomp = 0.0f;   // Kahan sum of Delta, as in the scan's summaries
  auto sum_add = [&](float v) {
    const float yv = v - dcomp, tv = dacc + yv;
    dcomp = (tv - dacc) - yv;
    dacc = tv;
  };
  // the next row is requested after this step's has been waited for (see chunk_loop)
  auto one_step = [&](float xv, float dv, bool has_next, float (&Bcur)[N], float (&Bnext)[N]) {
    const InT* nb = Brow + (has_next ? p.bs : 0);
    if constexpr (N >= 2) asm volatile("" : "+s"(nb) : "s"(Bcur[0]));
    row_of<N>(Bnext, nb, ok);
    ssm_step_any<N, DISC, false, kScaled>(h, cc, Bcur, Bcur, xv, dv);
    Brow = nb;
  };
  float xc[kU], dc[kU];
  auto at = [&](int32_t t) { return uint32_t(t < steps ? t : steps - 1); };
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    xc[j] = ldb(wx.r, lane, at(j) * wx.row, kIn);
    dc[j] = ldb(wd.r, lane, at(j) * wd.row, kIn);
  }
  for (int32_t tb = 0; tb < steps; tb += kU) {
    float xn[kU], dn[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      xn[j] = ldb(wx.r, lane, at(tb + kU + j) * wx.row, kIn);
      dn[j] = ldb(wd.r, lane, at(tb + kU + j) * wd.row, kIn);
    }
    if (dtm != kDtRaw) {
#pragma unroll
      for (int j = 0; j < kU; ++j) dc[j] = dt_transform(dc[j], dtb, dtm);
    }
    if (tb + kU <= steps) {
      float bs = 0.0f;
#pragma unroll
      for (int j = 0; j < kU; j += 2) {
        one_step(xc[j], dc[j], true, Bb0, Bb1);
        one_step(xc[j + 1], dc[j + 1], tb + j + 2 < steps, Bb1, Bb0);
        bs += dc[j] + dc[j + 1];
      }
      sum_add(bs);
    } else {
#pragma unroll
      for (int j = 0; j < kU; j += 2) {
        if (tb + j < steps) {
          one_step(xc[j], dc[j], tb + j + 1 < steps, Bb0, Bb1);
          sum_add(dc[j]);
        }
        if (tb + j + 1 < steps) {
          one_step(xc[j + 1], dc[j + 1], tb + j + 2 < steps, Bb1, Bb0);
          sum_add(dc[j + 1]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      xc[j] = xn[j];
      dc[j] = dn[j];
    }
  }
  if constexpr (kScaled) {
#pragma unroll
    for (int n = 0; n < N; ++n) h[n] /= scaled_a(p.A[d * N + n]);
  }
  store_n(p.hsum + (int64_t(chunk) * p.D + d) * N, h);
  p.dsum[int64_t(chunk) * p.D + d] = dacc - dcomp;
}

// Pass 2: carries.  One lane per (channel, state) walks the chunks; hsum of chunk c
// becomes the state that enters chunk c + 1.
template <int N>
__global__ void __launch_bounds__(kWave) k_packed_carry(const PackedParams p) {
  constexpr int U = 8;
  const int64_t i = int64_t(blockIdx.x) * kWave + threadIdx.x, DN = p.D * N;
  if (i >= DN) return;
  const float a2 = p.A[i] * kLog2e;
  const float* ds = p.dsum + i / N;
  float* hs = p.hsum + i;
  float carry = 0.0f;
  const int32_t n = p.nc - 1;
  int32_t c = 0;
  for (; c + U <= n; c += U) {
    float sv[U], hv[U];
    int32_t rv[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      sv[j] = ds[(c + j) * p.D];
      hv[j] = hs[(c + j) * DN];
      rv[j] = p.reset[c + j];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      carry = rv[j] ? hv[j] : decay_add(a2 * sv[j], carry, hv[j]);
      hs[(c + j) * DN] = carry;
    }
  }
  for (; c < n; ++c) {
    const float hv = hs[c * DN];
    carry = p.reset[c] ? hv : decay_add(a2 * ds[c * p.D], carry, hv);
    hs[c * DN] = carry;
  }
}

// Pass 3 (or the only one): every chunk from the state that enters it.
template <int N, typename InT, int DISC, bool GATE>
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
  float h[N];
  zero_n(h);

  // sequence `open` holds the tokens walked (none: -1), `next` is where it ends or, with
  // none, where sequence s begins
  int32_t s = seqs_before(p.q, from), open = -1;
  int32_t next = s < p.q.S ? seq_start(p.q, s) : INT32_MAX;
  if (chunk > 0 && s > 0 && from < to) {
    const int32_t end = seq_start(p.q, s);
    if (end > from) {
      open = s - 1;
      next = end;
      load_n(h, p.hsum + (int64_t(chunk) - 1) * DN + d * N);
    }
  }
  auto finish = [&] {
    if (open < 0) return;
    const int32_t slot = p.h_last ? seq_slot(p.q, open) : -1;
    if (slot >= 0) store_n(p.h_last + int64_t(slot) * DN + d * N, h);
    open = -1;
  };
  // At token t the open sequence has ended; empty ones pass their state on, and the
  // one that holds t is opened.
  auto meet = [&](int32_t t) {
    finish();
    next = INT32_MAX;
    for (; s < p.q.S && seq_start(p.q, s) <= t; ++s) {
      const int32_t end = seq_start(p.q, s + 1), slot = seq_slot(p.q, s);
      const bool given = p.h0 && slot >= 0 && seq_resumed(p.q, s);
      zero_n(h);
      if (given) load_n(h, end > t1 && p.hstart ? p.hstart + int64_t(chunk) * DN + d * N : p.h0 + int64_t(slot) * DN + d * N);
      open = s;
      if (end > t) {
        ++s;
        next = end;
        return;
      }
      finish();
    }
    if (s < p.q.S) next = seq_start(p.q, s);
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
    const bool ok = p.rows_ok != 0;
    float Bb0[N], Bb1[N], Cb0[N], Cb1[N];
    row_of<N>(Bb0, Brow, ok);
    row_of<N>(Cb0, Crow, ok);
    // where the walk stops to keep a state or to change sequences
    int32_t keep = p.hsave ? (from + kSaveStride - 1) / kSaveStride * kSaveStride : INT32_MAX;
    if (keep == 0) keep = kSaveStride;
    int32_t stop = next < keep ? next : keep;
    auto halt = [&](int32_t t) {
      if (t == keep) {
        store_n(p.hsave + (int64_t(t / kSaveStride) - 1) * DN + d * N, h);
        keep += kSaveStride;
      }
      if (next <= t) meet(t);
      stop = next < keep ? next : keep;
    };
    auto one_step = [&](float xv, float dv, float zv, bool has_next, float (&Bcur)[N], float (&Bnext)[N],
                        float (&Ccur)[N], float (&Cnext)[N]) {
      const InT* nb = Brow + (has_next ? p.bs : 0);
      const InT* nc = Crow + (has_next ? p.cs : 0);
      // the next rows are requested after this step's have been waited for (see chunk_loop)
      if constexpr (N >= 2) asm volatile("" : "+s"(nb), "+s"(nc) : "s"(Bcur[0]), "s"(Ccur[0]));
      row_of<N>(Bnext, nb, ok);
      row_of<N>(Cnext, nc, ok);
      const float acc = ssm_step_any<N, DISC, true>(h, cc, Bcur, Ccur, xv, dv);
      float yv = fmaf(dsk, xv, acc);
      if constexpr (GATE) yv *= silu(zv);
      stb(wy.r, lane, yoff, yv, static_cast<InT*>(nullptr));
      yoff += wy.row;
      Brow = nb;
      Crow = nc;
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
#pragma unroll
      for (int j = 0; j < kU; j += 2) {
        if (tb + j < steps) {
          if (from + tb + j == stop) halt(from + tb + j);
          one_step(xc[j], dc[j], zc[j], tb + j + 1 < steps, Bb0, Bb1, Cb0, Cb1);
        }
        if (tb + j + 1 < steps) {
          if (from + tb + j + 1 == stop) halt(from + tb + j + 1);
          one_step(xc[j + 1], dc[j + 1], zc[j + 1], tb + j + 2 < steps, Bb1, Bb0, Cb1, Cb0);
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
  if (at < t1 || t1 == p.q.tokens) {
    if (next <= at || open >= 0) meet(at);
  } else if (open >= 0 && next <= at) {
    finish();
  }
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
