// packed_bwd.hpp -- gfx950 device code of the packed scan's gradients: the passes of
// ssm_bwd.hpp (a reverse summary per super-chunk of tokens, a walk over their
// carries, and a main pass that recomputes 16 tokens at a time from the states the
// forward kept and walks them back) over a token axis cut wherever it falls, with
//
//   * the state replaced at a sequence's first token in the recompute (what is kept in
//     registers before it is the state after the step before), and the adjoint
//     replaced behind it (by dh_last of the sequence before, or 0) on the way back;
//     what it was there is that sequence's dh0;
//   * summaries walked only from the end of the sequence that reaches back past a
//     super-chunk's first token, where that end lies in it (reset);
//   * tokens of no sequence left unread, their gradients 0.
#pragma once

#include "packed_scan.hpp"

namespace ssmp {

struct PackedBwdParams {
  const void* x;
  const void* delta;
  const void* Bm;
  const void* Cm;
  const void* dy;
  const float* A;
  const float* Dskip;    // or null
  const float* h0;       // (S, D, N) or null
  const float* hsave;
  const float* dh_last;  // (S, D, N) or null
  float* dx;
  float* ddelta;
  float* dA;
  float* dB;
  float* dC;
  float* dD;             // or null
  float* dh0;            // or null
  float* gsum;           // (nc - 1, D, N) adjoints that leave super-chunks 1 .. nc - 1, then carries
  float* dsum;           // (nc - 1, D)
  int32_t* reset;        // (nc - 1)
  float* dAp;            // (nc, D, N) and
  float* dDp;            // (nc, D): the super-chunks' sums
  float* dBCp;           // (tokens, dtiles, 2, N): the channel tiles' sums for dB, then dC
  int64_t xs, dls, ys;   // row strides; ys: of dy
  uint32_t bs, cs;
  int64_t D;
  Seqs q;
  int32_t T, nc;         // tokens per super-chunk (a multiple of 16), super-chunks
  int32_t dtiles, nwg;
  float exact_thr;
};

// The sequence that holds token t (of those with its first token, the one with any).
__device__ __forceinline__ int32_t seq_at(const Seqs& q, int32_t t) { return seqs_before(q, t + 1) - 1; }

// One step back of a lane's NS states: bwd_lane_step, with the slow-decay form chosen
// state by state (see advance).
//
// ZOH's factor f = Delta (e^z - 1) / z and its derivative by A, Delta^2 q with
// q = (z e^z - (e^z - 1)) / z^2, z = Delta A: the direct forms take differences that lose
// 2^-24 / |z| and 2^-22 / z^2 of their values, which a dA of few tokens shows (one token
// of 8 channels, bf16: 9e-5 in norm with the scan's limit of 1/64 for them, and a series of
// three terms below it).  So they are kept to |z| >= 1/2 (1e-6), and below it
//   q = sum_k z^k (k + 1) / (k + 2)!, to k = 7 (the rest is below 3e-8 of q),
//   f = Delta (e^z - z q).
constexpr float kZohSeries = 0.5f;

template <int NS, int DISC, bool SERIES>
__device__ __forceinline__ void retreat(float (&g)[NS], float (&dA)[NS], const ChanConst<NS, DISC>& cc,
                                        const float (&Bv)[NS], const float (&Cv)[NS], const float (&hp)[NS],
                                        const float (&hn)[NS], float u, float dv, float dyv, float limit,
                                        float (&pB)[NS], float (&pC)[NS], float& du, float& ddt) {
  float z2[NS], a[NS], G[NS], ag[NS];
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    z2[n] = dv * cc.A2[n];
    a[n] = exp2_fast(z2[n]);
    G[n] = fmaf(Cv[n], dyv, g[n]);
    ag[n] = a[n] * G[n];
  }
  if (any_exact<NS, DISC>(cc, dv)) {
#pragma unroll
    for (int n = 0; n < NS; ++n)
      // a G plus what rounding took from a (see decay_add)
      if (any_slow(z2[n], limit)) ag[n] = fmaf(a[n], G[n], exp_residual<true>(z2[n], a[n]) * G[n]);
  }
  if constexpr (DISC == kDeltaB) {
    // du and dDelta's input term are Delta and u times sum_n G B (A is held as
    // A log2(e); the ln 2 that restores A is applied to the state sum once)
    const float dvu = dv * u;
    float gb = 0.0f, dt2 = 0.0f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const float agh = ag[n] * hp[n];   // shared by dDelta and dA
      gb = n ? fmaf(G[n], Bv[n], gb) : G[n] * Bv[n];
      dt2 = n ? fmaf(cc.A2[n], agh, dt2) : cc.A2[n] * agh;
      dA[n] = fmaf(dv, agh, dA[n]);
      pB[n] = G[n] * dvu;
    }
    du = dv * gb;
    ddt = fmaf(dt2, kLn2, u * gb);
  } else {
    float su = 0.0f, dt2 = 0.0f, dtb = 0.0f;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      float f = (a[n] - 1.0f) * cc.invA[n];
      float dfda = fmaf(dv, a[n], -f) * cc.invA[n];
      if constexpr (SERIES) {
        const float z = z2[n] * kLn2;
        float q = fmaf(z, 1.0f / 45360.0f, 1.0f / 5760.0f);
        q = fmaf(z, q, 1.0f / 840.0f);
        q = fmaf(z, q, 1.0f / 144.0f);
        q = fmaf(z, q, 1.0f / 30.0f);
        q = fmaf(z, q, 0.125f);
        q = fmaf(z, q, 1.0f / 3.0f);
        q = fmaf(z, q, 0.5f);
        const bool small = fabsf(z) < kZohSeries || cc.invA[n] == 0.0f;
        f = small ? dv * fmaf(-z, q, a[n]) : f;
        dfda = small ? (dv * dv) * q : dfda;
      }
      const float agh = ag[n] * hp[n], Bu = Bv[n] * u, Gf = G[n] * f;
      pB[n] = Gf * u;
      su = fmaf(Gf, Bv[n], su);
      dt2 = fmaf(cc.A2[n], agh, dt2);
      dtb = fmaf(ag[n], Bu, dtb);   // df/dDelta = a
      dA[n] = fmaf(dv, agh, fmaf(G[n] * dfda, Bu, dA[n]));
    }
    du = su;
    ddt = fmaf(dt2, kLn2, dtb);
  }
#pragma unroll
  for (int n = 0; n < NS; ++n) {
    pC[n] = dyv * hn[n];
    g[n] = ag[n];
  }
}

// Reverse summary of super-chunks 1 .. nc - 1.
template <int N, typename InT, int DISC, bool ODD>
__global__ void __launch_bounds__(kWave) __attribute__((amdgpu_waves_per_eu(4))) k_packed_bwd_summary(const PackedBwdParams p) {
  constexpr int kU = 8;
  const int wg = xcd_remap(blockIdx.x, p.nwg);
  const int64_t dbase = int64_t(wg % p.dtiles) * kWave;
  const int32_t slot = wg / p.dtiles, chunk = slot + 1;
  const int32_t t0 = chunk * p.T, t1 = p.q.tokens - t0 > p.T ? t0 + p.T : p.q.tokens;
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, p.q.S);
  int32_t to = t0, fresh = 1, open = -1;
  if (t0 > lo && t0 < hi) {
    const int32_t s = seqs_before(p.q, t0);   // s - 1 begins before t0
    const int32_t end = s > 0 ? seq_start(p.q, s) : t0;
    if (end > t0) {
      fresh = end <= t1;
      to = fresh ? end : t1;
      open = s - 1;
    }
  }
  if (dbase == 0 && threadIdx.x == 0) p.reset[slot] = fresh;
  if (open < 0) return;

  const uint32_t lo_ch = lane_offset(dbase, p.D);
  const int64_t d = dbase + lo_ch;
  ChanConst<N, DISC> cc;
  load_chan<N, DISC>(cc, p.A + d * N, p.exact_thr);
  const float limit = p.exact_thr * kLog2e;
  float g[N];
  zero_n(g);
  if (fresh && p.dh_last) load_n(g, p.dh_last + (int64_t(open) * p.D + d) * N);
  const int32_t steps = to - t0;
  const RowWindow wd = window<InT>(p.delta, p.dls, p.D, dbase, t0, steps);
  const RowWindow wy = window<InT>(p.dy, p.ys, p.D, dbase, t0, steps);
  const uint32_t lane = lo_ch * sizeof(InT);
  constexpr InT* kIn = nullptr;
  const InT* Crow = static_cast<const InT*>(p.Cm) + int64_t(to - 1) * p.cs;
  float dacc = 0.0f, dcomp = 0.0f;
  using R = Row<N, InT, ODD>;
  R Cb0, Cb1;
  Cb0.load(Crow);
  auto one_step = [&](float dv, float dyv, uint32_t behind, const R& Cthis, R& Cnext) {
    const InT* nc = Crow - behind;
    asm volatile("" : "+s"(nc) : "s"(Cthis.w[0]));
    Cnext.load(nc);
    float Ccur[N];
    Cthis.widen(Ccur);
    float z2[N], G[N], a[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      z2[n] = dv * cc.A2[n];
      a[n] = exp2_fast(z2[n]);
      G[n] = fmaf(Ccur[n], dyv, g[n]);
      g[n] = a[n] * G[n];
    }
    if (any_exact<N, DISC>(cc, dv)) {   // the slow-decay form, for four states at a time (see advance)
      constexpr int W = N < 4 ? N : 4;
#pragma unroll
      for (int q = 0; q < N; q += W) {
        float least = fabsf(z2[q]);
#pragma unroll
        for (int n = q + 1; n < q + W; ++n) least = fminf(least, fabsf(z2[n]));
        if (any_slow(least, limit)) {
#pragma unroll
          for (int n = q; n < q + W; ++n) g[n] = fmaf(a[n], G[n], exp_residual<true>(z2[n], a[n]) * G[n]);
        }
      }
    }
    Crow = nc;
    const float yv = dv - dcomp, tv = dacc + yv;
    dcomp = (tv - dacc) - yv;
    dacc = tv;
  };
  // row k of the walk, from the last down
  auto at = [&](int32_t k) { return uint32_t(k < steps ? steps - 1 - k : 0); };
  float dc[kU], yc[kU];
#pragma unroll
  for (int j = 0; j < kU; ++j) {
    dc[j] = ldb(wd.r, lane, at(j) * wd.row, kIn);
    yc[j] = ldb(wy.r, lane, at(j) * wy.row, kIn);
  }
  int32_t t = 0;
  for (; t + kU < steps; t += kU) {
    float dn[kU], yn[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      dn[j] = ldb(wd.r, lane, at(t + kU + j) * wd.row, kIn);
      yn[j] = ldb(wy.r, lane, at(t + kU + j) * wy.row, kIn);
    }
#pragma unroll
    for (int j = 0; j < kU; j += 2) {
      one_step(dc[j], yc[j], p.cs, Cb0, Cb1);
      one_step(dc[j + 1], yc[j + 1], p.cs, Cb1, Cb0);
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      dc[j] = dn[j];
      yc[j] = yn[j];
    }
  }
#pragma unroll 1
  for (; t < steps; ++t) {
    const float dv = ldb(wd.r, lane, at(t) * wd.row, kIn), dyv = ldb(wy.r, lane, at(t) * wy.row, kIn);
    one_step(dv, dyv, t + 1 < steps ? p.cs : 0u, Cb0, Cb1);
    Cb0 = Cb1;
  }
  store_n(p.gsum + (int64_t(slot) * p.D + d) * N, g);
  p.dsum[int64_t(slot) * p.D + d] = dacc - dcomp;
}

// Carries, from the last super-chunk down: gsum[c - 1] becomes the adjoint that
// enters super-chunk c - 1 from behind.
template <int N>
__global__ void __launch_bounds__(kWave * kCarryWaves) k_packed_bwd_carry(const PackedBwdParams p) {
  carry_walk<N, true>(p.A, p.dsum, p.gsum, p.reset, p.D, p.nc - 1);
}

// Main pass; lanes, waves and LDS as in k_bwd_main.  What only some of the steps need is
// read again from the arguments (args_again) every 16 tokens: kept in scalar registers,
// it spilled 276 of them (16384 x 1536 x 16 fp32: 632 us, then 503).  16 tokens of one
// sequence take a copy of the steps without the questions for its ends, whose steps
// overlap; for its registers a SIMD holds three waves rather than four (forward and
// gradients, fp32 798 -> 776 us, bf16 794 -> 711, ZOH bf16 982 -> 897; with four waves
// it spills, 910 and 807; sequences of four tokens 1333 -> 1477; one state, which has
// little to overlap, 305 -> 323 and so keeps the one copy and four waves).
template <int N, typename InT, int DISC>
__global__ void __launch_bounds__(kWave * BwdLayout<N>::NG) __attribute__((amdgpu_waves_per_eu(N > 1 ? 3 : 4)))
k_packed_bwd(const PackedBwdParams p) {
  constexpr int NS = BwdLayout<N>::NS, NG = BwdLayout<N>::NG;
  constexpr int F = kBwdFine, K = kBwdBlock, H = kBwdHalf;
  constexpr int RR = 4 * NS;           // rows summed together
  constexpr int LPR = kWave / RR;      // lanes per row; each sums RR floats
  __shared__ __attribute__((aligned(16))) float red[NG][RR][kRedPitch];
  __shared__ float xch[2][2][NG][K][kWave];
  // of the sequences that begin among 16 tokens, at the place of their first token:
  // which one it is, and which one ends before it (each wave its own)
  __shared__ int32_t ids[NG][2][F];
  // rows of B and C as fp32, double-buffered by 16 tokens
  __shared__ __attribute__((aligned(16))) float rows[2][2][F][N];

  const int wg = xcd_remap(blockIdx.x, p.nwg);
  const int32_t dtile = wg % p.dtiles;
  const int32_t chunk = wg / p.dtiles;
  const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int lane = threadIdx.x % kWave;
  const int64_t dbase = int64_t(dtile) * kWave;
  const int64_t d = dbase + lane_offset(dbase, p.D, static_cast<uint32_t>(lane));
  const bool valid = dbase + lane < p.D;   // lanes past D duplicate D - 1 and add nothing
  if (!valid) {
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) red[w][rr][lane] = 0.0f;
  }
  int xb = 0;
  const int n0 = w * NS;
  const int64_t dn = d * N + n0;   // this lane's states in a (D, N) array

  ChanConst<NS, DISC> cc;
  load_chan<NS, DISC>(cc, p.A + dn, p.exact_thr);
  const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
  const float limit = p.exact_thr * kLog2e;
  float zoh_thr = 0.0f;   // below it ZOH's factor is taken from its series
  if constexpr (DISC == kZoh) {
    float amin = __builtin_inff();
#pragma unroll
    for (int n = 0; n < NS; ++n) amin = fminf(amin, fabsf(cc.A2[n] * kLn2));
    zoh_thr = amin > 0.0f ? kZohSeries / amin : __builtin_inff();
  }

  const int32_t t0 = chunk * p.T, t1 = p.q.tokens - t0 > p.T ? t0 + p.T : p.q.tokens;
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, p.q.S);   // tokens of sequences
  // the sequence whose tokens are walked next, and its first token
  int32_t seq = -1, first = INT32_MIN;
  float g[NS];
  zero_n(g);
  {
    const int32_t from = t0 > lo ? t0 : lo, to = t1 < hi ? t1 : hi;
    if (from < to) {
      seq = seq_at(p.q, to - 1);
      first = seq_start(p.q, seq);
      if (first > to - 1) first = to - 1;
      if (seq_start(p.q, seq + 1) > t1) {
        load_n(g, p.gsum + int64_t(chunk) * p.D * N + dn);
      } else if (p.dh_last) {
        load_n(g, p.dh_last + int64_t(seq) * p.D * N + dn);
      }
    }
  }
  float dAacc[NS];
  zero_n(dAacc);
  float dDacc = 0.0f;

  const uint32_t lane_in = uint32_t(d - dbase) * sizeof(InT), lane_f = uint32_t(d - dbase) * 4u;
  constexpr InT* kIn = nullptr;
  constexpr float* kF = nullptr;
  // where a lane's sums of two steps go, in a token's (dtiles, 2, N) rows: lane's row is
  // [step of the pair][dB or dC][state]; one lane of each LPR stores (the others past
  // the window's end)
  const int rr_ = lane / LPR;
  const uint32_t sums_row = uint32_t(p.dtiles) * (2 * N * 4);
  const uint32_t sums_at = lane % LPR == 0 ? uint32_t(((rr_ / NS) & 1) * N + n0 + rr_ % NS) * 4u + uint32_t(rr_ / (2 * NS)) * sums_row
                                           : 0x80000000u;

  // the rows each thread moves into LDS, loaded 16 tokens ahead (rows of tokens of no
  // sequence as 0)
  constexpr int kRowVals = 2 * F * N;
  constexpr int RV = (kRowVals + kWave * NG - 1) / (kWave * NG);
  float rpre[RV];
  auto rows_load = [&](const PackedBwdParams& a, int32_t f0) {
    const InT* Bp = static_cast<const InT*>(a.Bm);
    const InT* Cp = static_cast<const InT*>(a.Cm);
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      const int e = static_cast<int>(threadIdx.x) + i * kWave * NG;
      const int kind = (e / (F * N)) & 1, j = (e / N) % F, n = e % N;
      const bool in = e < kRowVals && f0 + j >= lo && f0 + j < hi;
      rpre[i] = in ? ld((kind == 0 ? Bp + int64_t(f0 + j) * a.bs : Cp + int64_t(f0 + j) * a.cs) + n) : 0.0f;
    }
  };
  const int32_t f_top = (t1 - 1) / F * F;
  rows_load(p, f_top);
  int rb = 0;

  for (int32_t f0 = f_top; f0 >= t0; f0 -= F) {
    const PackedBwdParams& a = args_again<PackedBwdParams>();
    const int len = a.q.tokens - f0 < F ? a.q.tokens - f0 : F;
    // bit j of live: token j belongs to a sequence; of begins: it is a first one
    const int jlo = lo > f0 ? (lo - f0 < len ? lo - f0 : len) : 0;
    const int jhi = hi - f0 < len ? (hi > f0 ? hi - f0 : 0) : len;
    const uint32_t live = jlo < jhi ? (1u << jhi) - (1u << jlo) : 0u;
    uint32_t begins = 0;
    while (first >= f0) {
      const int32_t before = first > lo ? seq_at(a.q, first - 1) : -1;
      begins |= 1u << (first - f0);
      if (lane < 2) ids[w][lane][first - f0] = lane == 0 ? seq : before;
      const int32_t start = before >= 0 ? seq_start(a.q, before) : INT32_MIN;
      seq = before;
      first = start < first ? start : INT32_MIN;   // (falling offsets end the walk too)
    }
    // gradients of this channel tile's rows, and its sums for dB and dC
    const __amdgpu_buffer_rsrc_t rdx = make_rsrc(a.dx + int64_t(f0) * a.D + dbase, uint32_t(len * a.D * 4));
    const __amdgpu_buffer_rsrc_t rdd = make_rsrc(a.ddelta + int64_t(f0) * a.D + dbase, uint32_t(len * a.D * 4));
    const uint32_t row_f = uint32_t(a.D * 4);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(a.dBCp + (int64_t(f0) * a.dtiles + dtile) * (2 * N),
                                                uint32_t(len - 1) * sums_row + 2 * N * 4);
    if (live == 0) {   // the whole workgroup
      for (int j = w; j < len; j += NG) {
        stb(rdx, lane_f, uint32_t(j) * row_f, 0.0f, kF);
        stb(rdd, lane_f, uint32_t(j) * row_f, 0.0f, kF);
      }
      for (int e = threadIdx.x; e < len * 2 * N; e += kWave * NG)
        stb(rs, uint32_t(e / (2 * N)) * sums_row + uint32_t(e % (2 * N)) * 4u, 0, 0.0f, kF);
      if (f0 > t0) rows_load(a, f0 - F);
      continue;
    }
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      const int e = static_cast<int>(threadIdx.x) + i * kWave * NG;
      if (e < kRowVals) (&rows[rb][0][0][0])[e] = rpre[i];
    }
    __syncthreads();
    if (f0 > t0) rows_load(a, f0 - F);
    const RowWindow wx = window<InT>(a.x, a.xs, a.D, dbase, f0, len);
    const RowWindow wd = window<InT>(a.delta, a.dls, a.D, dbase, f0, len);
    const RowWindow wy = window<InT>(a.dy, a.ys, a.D, dbase, f0, len);
    auto in = [&](int j) { return uint32_t(j < len ? j : len - 1); };   // a row of the tensors
    const float* hin = f0 > 0 ? a.hsave + (int64_t(f0 / F) - 1) * a.D * N + dn : nullptr;
    // the state before the first token of a sequence
    auto initial = [&](float (&h)[NS], int j) {
      const PackedBwdParams& b = args_again<PackedBwdParams>();
      zero_n(h);
      if (b.h0) load_n(h, b.h0 + int64_t(__builtin_amdgcn_readfirstlane(ids[w][0][j])) * b.D * N + dn);
    };
    // The later half first: from the state kept, through the earlier half, its own steps
    // forwards with the states between them in registers, and back.  (A rolled loop:
    // both halves' steps unrolled are 56 KB of instructions.)
    auto half = [&](auto events, int j0) {
      constexpr bool kEvents = decltype(events)::value;
      const uint32_t live_h = live >> j0, begins_h = begins >> j0;
      const float* Brow = &rows[rb][0][j0][n0];
      const float* Crow = &rows[rb][1][j0][n0];
      float h[NS];
      zero_n(h);
      if (hin) load_n(h, hin);
      auto forward = [&](float xv, float dv, const float* row) {
        float Bv[NS];
        lds_row<NS>(Bv, row);
        advance<NS, DISC, false, NS, true>(h, cc, Bv, xv, dv, limit);
      };
      float xa[K], da[K];
      auto rows_of = [&](float (&u)[K], float (&v)[K], int j) {
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          u[jj] = ldb(wx.r, lane_in, in(j + jj) * wx.row, kIn);
          v[jj] = ldb(wd.r, lane_in, in(j + jj) * wd.row, kIn);
        }
      };
      rows_of(xa, da, 0);
#pragma unroll 1
      for (int jb = 0; jb < j0; jb += K) {
        float xn[K], dn_[K];
        rows_of(xn, dn_, jb + K);
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          if (kEvents && (begins >> (jb + jj) & 1)) initial(h, jb + jj);
          if (!kEvents || (live >> (jb + jj) & 1)) forward(xa[jj], da[jj], &rows[rb][0][jb + jj][n0]);
        }
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          xa[jj] = xn[jj];
          da[jj] = dn_[jj];
        }
      }
      auto dy_of = [&](float (&u)[K], int j) {
#pragma unroll
        for (int jj = 0; jj < K; ++jj) u[jj] = ldb(wy.r, lane_in, in(j + jj) * wy.row, kIn);
      };
      // The last rows of x, Delta and dy are the first on the way back, where four more are
      // requested ahead: fp32 776 -> 739 us, bf16 712 -> 675.  (ZOH's steps have no
      // registers for them: 1439 -> 1492, 898 -> 957.)
      constexpr bool kAheadBack = DISC == kDeltaB;
      float ya[K];
      if (kAheadBack) dy_of(ya, j0 + H - K);
      // the state after the step before each step of the half
      float stash[H][NS];
#pragma unroll
      for (int jb = 0; jb < H; jb += K) {
        float xn[K], dn_[K];
        if (jb + K < H) rows_of(xn, dn_, j0 + jb + K);
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          const int js = jb + jj;
#pragma unroll
          for (int n = 0; n < NS; ++n) stash[js][n] = h[n];
          if (kEvents && (begins_h >> js & 1)) initial(h, j0 + js);
          if (!kEvents || (live_h >> js & 1)) forward(xa[jj], da[jj], Brow + js * N);
        }
        if (jb + K < H) {
#pragma unroll
          for (int jj = 0; jj < K; ++jj) {
            xa[jj] = xn[jj];
            da[jj] = dn_[jj];
          }
        }
      }
#pragma unroll
      for (int jb = H - K; jb >= 0; jb -= K) {
        float un[K], vn[K], yn[K];   // the rows before
        if constexpr (!kAheadBack) {
          rows_of(xa, da, j0 + jb);
          dy_of(ya, j0 + jb);
        } else if (jb > 0) {
          rows_of(un, vn, j0 + jb - K);
          dy_of(yn, j0 + jb - K);
        }
        if (!kEvents || j0 + jb < len) {   // wave-uniform
#pragma unroll
          for (int jj = K - 1; jj >= 0; --jj) {
            const int js = jb + jj;
            float pB[NS], pC[NS], du = 0.0f, ddt = 0.0f;
            zero_n(pB);
            zero_n(pC);
            if (!kEvents || (live_h >> js & 1)) {
              const float u = xa[jj], dv = da[jj], dyv = ya[jj];
              float Bv[NS], Cv[NS];
              lds_row<NS>(Bv, Brow + js * N);
              lds_row<NS>(Cv, Crow + js * N);
              float hp[NS], hn[NS];   // the states before and after the step
#pragma unroll
              for (int n = 0; n < NS; ++n) {
                hp[n] = stash[js][n];
                hn[n] = (js + 1 < H) ? stash[js + 1 < H ? js + 1 : js][n] : h[n];
              }
              if (kEvents && (begins_h >> js & 1)) initial(hp, j0 + js);
              const bool series = DISC == kZoh && __builtin_amdgcn_ballot_w64(dv < zoh_thr) != 0;
              if (series)
                retreat<NS, DISC, true>(g, dAacc, cc, Bv, Cv, hp, hn, u, dv, dyv, limit, pB, pC, du, ddt);
              else
                retreat<NS, DISC, false>(g, dAacc, cc, Bv, Cv, hp, hn, u, dv, dyv, limit, pB, pC, du, ddt);
              dDacc = fmaf(dyv, u, dDacc);
              if (kEvents && (begins_h >> js & 1)) {
                const PackedBwdParams& b = args_again<PackedBwdParams>();
                const int32_t s = __builtin_amdgcn_readfirstlane(ids[w][0][j0 + js]);
                const int32_t before = __builtin_amdgcn_readfirstlane(ids[w][1][j0 + js]);
                if (b.dh0) store_n(b.dh0 + int64_t(s) * b.D * N + dn, g);
                zero_n(g);
                // (of a sequence that ends before this super-chunk, g goes no further)
                if (before >= 0 && b.dh_last) load_n(g, b.dh_last + int64_t(before) * b.D * N + dn);
              }
            }
            const int sp = jj & 1;
            if (valid) {
#pragma unroll
              for (int n = 0; n < NS; ++n) {
                red[w][(sp * 2 + 0) * NS + n][lane] = pB[n];
                red[w][(sp * 2 + 1) * NS + n][lane] = pC[n];
              }
            }
            xch[xb][0][w][jj][lane] = du;
            xch[xb][1][w][jj][lane] = ddt;
            if (sp == 0) {
              __builtin_amdgcn_wave_barrier();
              const int rr = lane / LPR, c = lane % LPR;
              const float4* src = reinterpret_cast<const float4*>(&red[w][rr][c * RR]);
              float acc = 0.0f;
#pragma unroll
              for (int i = 0; i < RR / 4; ++i) {
                const float4 v = src[i];
                acc += v.x;
                acc += v.y;
                acc += v.z;
                acc += v.w;
              }
              if constexpr (LPR >= 2)
                acc += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(acc), 0xB1, 0xF, 0xF, false));
              if constexpr (LPR >= 4)
                acc += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(acc), 0x4E, 0xF, 0xF, false));
              if constexpr (LPR >= 8)
                acc += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(acc), 0x141, 0xF, 0xF, false));
              if constexpr (LPR >= 16)
                acc += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(acc), 0x140, 0xF, 0xF, false));
              // rows of tokens past the last end behind the window (the row's offset goes
              // with the lane's, which is what the window is checked against)
              stb(rs, sums_at + uint32_t(j0 + js) * sums_row, 0, acc, kF);
              __builtin_amdgcn_wave_barrier();
            }
          }
          __syncthreads();
#pragma unroll
          for (int jj = w; jj < K; jj += NG) {
            const int j = j0 + jb + jj;
            if (!kEvents || j < len) {
              float su = 0.0f, sd = 0.0f;
#pragma unroll
              for (int v = 0; v < NG; ++v) {
                su += xch[xb][0][v][jj][lane];
                sd += xch[xb][1][v][jj][lane];
              }
              if (!kEvents || (live >> j & 1)) su = fmaf(dsk, ldb(wy.r, lane_in, uint32_t(j) * wy.row, kIn), su);
              stb(rdx, lane_f, uint32_t(j) * row_f, su, kF);
              stb(rdd, lane_f, uint32_t(j) * row_f, sd, kF);
            }
          }
          xb ^= 1;
        }
        if (kAheadBack && jb > 0) {
#pragma unroll
          for (int jj = 0; jj < K; ++jj) {
            xa[jj] = un[jj];
            da[jj] = vn[jj];
            ya[jj] = yn[jj];
          }
        }
      }
    };
    if (N > 1 && begins == 0 && live == (1u << F) - 1) {
#pragma unroll 1
      for (int j0 = F - H; j0 >= 0; j0 -= H) half(std::false_type{}, j0);
    } else {
#pragma unroll 1
      for (int j0 = F - H; j0 >= 0; j0 -= H)
        if (j0 < len) half(std::true_type{}, j0);   // wave-uniform
    }
    rb ^= 1;
  }
  const PackedBwdParams& a = args_again<PackedBwdParams>();
  const int64_t DN = a.D * N;
  store_n(a.dAp + int64_t(chunk) * DN + dn, dAacc);
  if (w == 0) a.dDp[int64_t(chunk) * a.D + d] = dDacc;
  // sequences without tokens: their last state is their first
  if (chunk == 0 && a.dh0) {
    for (int32_t s0 = 0; s0 < a.q.S; s0 += kWave) {
      const int32_t s = s0 + lane;
      bool empty = false;
      if (s < a.q.S) empty = ssmq::in_tokens(a.q, a.q.offsets[s]) >= ssmq::in_tokens(a.q, a.q.offsets[s + 1]);
      uint64_t todo = __builtin_amdgcn_ballot_w64(empty);
      while (todo) {
        const int64_t e = s0 + __builtin_ctzll(todo);
        todo &= todo - 1;
        float v[NS];
        zero_n(v);
        if (a.dh_last) load_n(v, a.dh_last + e * DN + dn);
        store_n(a.dh0 + e * DN + dn, v);
      }
    }
  }
}

// dB, dC: the channel tiles' sums of a (token, dB or dC, state).
template <int N>
__global__ void __launch_bounds__(256) k_packed_bwd_bc(const PackedBwdParams p) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= int64_t(p.q.tokens) * (2 * N)) return;
  const int64_t t = i / (2 * N);
  const int n = int(i % (2 * N));
  const float* src = p.dBCp + t * p.dtiles * (2 * N) + n;
  float sum = 0.0f;
  for (int k = 0; k < p.dtiles; ++k) sum += src[k * (2 * N)];
  (n < N ? p.dB + t * N + n : p.dC + t * N + n - N)[0] = sum;
}

// dA (D, N), then dD (D): the super-chunks' sums in a fixed order; a workgroup covers
// 64 of them, each of its 16 waves every 16th super-chunk.
template <int N>
__global__ void __launch_bounds__(kWave * kRedWaves) k_packed_bwd_ad(const PackedBwdParams p) {
  __shared__ float part[kRedWaves][kWave];
  const int w = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int64_t i = int64_t(blockIdx.x) * kWave + lane, DN = p.D * N;
  const bool isA = i < DN, isD = !isA && i < DN + p.D && p.dD;
  float acc = 0.0f;
  if (isA) {
    for (int32_t k = w; k < p.nc; k += kRedWaves) acc += p.dAp[k * DN + i];
  } else if (isD) {
    for (int32_t k = w; k < p.nc; k += kRedWaves) acc += p.dDp[k * p.D + (i - DN)];
  }
  part[w][lane] = acc;
  __syncthreads();
  if (w == 0) {
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < kRedWaves; ++v) sum += part[v][lane];
    if (isA)
      p.dA[i] = sum;
    else if (isD)
      p.dD[i - DN] = sum;
  }
}

}  // namespace ssmp
