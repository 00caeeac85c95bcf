// packed_bwd.hpp -- gfx950 device code of the packed scan's gradients: the passes of
// ssm_bwd.hpp (a reverse summary per super-chunk of tokens, a walk over their
// carries, and a main pass that recomputes 16 tokens at a time from the states the
// forward kept and walks them back) over a token axis cut wherever it falls, with
//
//   * the state replaced at a sequence's first token in the recompute, and the
//     adjoint replaced behind it (by dh_last of the sequence before, or 0) on the
//     way back; what it was there is that sequence's dh0;
//   * summaries walked only from the end of the sequence that reaches back past a
//     super-chunk's first token, where that end lies in it (reset);
//   * tokens of no sequence left unread, their gradients 0.
//
// The recomputed states before and after a step are neighbours in registers, except
// before a sequence's first token, where the state after the step is formed again.
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
  float* dBp;            // (tokens, dtiles, N) and
  float* dCp;            // (tokens, dtiles, N): the channel tiles' sums
  int64_t xs, dls, bs, cs, ys;   // row strides; ys: of dy
  int64_t D;
  Seqs q;
  int32_t T, nc;         // tokens per super-chunk (a multiple of 16), super-chunks
  int32_t dtiles, nwg;
  float exact_thr;
  int32_t rows_ok;
};

// The sequence that holds token t (of those with its first token, the one with any).
__device__ __forceinline__ int32_t seq_at(const Seqs& q, int32_t t) { return seqs_before(q, t + 1) - 1; }

// Reverse summary of super-chunks 1 .. nc - 1.
template <int N, typename InT, int DISC>
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
  float g[N];
  zero_n(g);
  if (fresh && p.dh_last) load_n(g, p.dh_last + (int64_t(open) * p.D + d) * N);
  const int32_t steps = to - t0;
  const RowWindow wd = window<InT>(p.delta, p.dls, p.D, dbase, t0, steps);
  const RowWindow wy = window<InT>(p.dy, p.ys, p.D, dbase, t0, steps);
  const uint32_t lane = lo_ch * sizeof(InT);
  constexpr InT* kIn = nullptr;
  const InT* Crow = static_cast<const InT*>(p.Cm) + int64_t(to - 1) * p.cs;
  const bool ok = p.rows_ok != 0;
  float dacc = 0.0f, dcomp = 0.0f;
  float Cb0[N], Cb1[N];
  row_of<N>(Cb0, Crow, ok);
  auto one_step = [&](float dv, float dyv, bool has_next, float (&Ccur)[N], float (&Cnext)[N]) {
    const InT* nc = Crow - (has_next ? p.cs : 0);
    if constexpr (N >= 2) asm volatile("" : "+s"(nc) : "s"(Ccur[0]));
    row_of<N>(Cnext, nc, ok);
    if (any_exact<N, DISC>(cc, dv)) {   // wave-uniform
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const float z2 = dv * cc.A2[n];
        const float G = fmaf(Ccur[n], dyv, g[n]);
        const float a = exp2_fast(z2);
        g[n] = fmaf(a, G, exp_residual<true>(z2, a) * G);
      }
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) g[n] = exp2_fast(dv * cc.A2[n]) * fmaf(Ccur[n], dyv, g[n]);
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
  for (int32_t tb = 0; tb < steps; tb += kU) {
    float dn[kU], yn[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      dn[j] = ldb(wd.r, lane, at(tb + kU + j) * wd.row, kIn);
      yn[j] = ldb(wy.r, lane, at(tb + kU + j) * wy.row, kIn);
    }
#pragma unroll
    for (int j = 0; j < kU; j += 2) {
      if (tb + j < steps) one_step(dc[j], yc[j], tb + j + 1 < steps, Cb0, Cb1);
      if (tb + j + 1 < steps) one_step(dc[j + 1], yc[j + 1], tb + j + 2 < steps, Cb1, Cb0);
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      dc[j] = dn[j];
      yc[j] = yn[j];
    }
  }
  store_n(p.gsum + (int64_t(slot) * p.D + d) * N, g);
  p.dsum[int64_t(slot) * p.D + d] = dacc - dcomp;
}

// Carries, from the last super-chunk down: gsum[c - 1] becomes the adjoint that
// enters super-chunk c - 1 from behind.
template <int N>
__global__ void __launch_bounds__(kWave) k_packed_bwd_carry(const PackedBwdParams p) {
  constexpr int U = 8;
  const int64_t i = int64_t(blockIdx.x) * kWave + threadIdx.x, DN = p.D * N;
  if (i >= DN) return;
  const float a2 = p.A[i] * kLog2e;
  const float* ds = p.dsum + i / N;
  float* gs = p.gsum + i;
  float carry = 0.0f;
  int32_t c = p.nc - 2;
  for (; c >= U - 1; c -= U) {
    float sv[U], gv[U];
    int32_t rv[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      sv[j] = ds[(c - j) * p.D];
      gv[j] = gs[(c - j) * DN];
      rv[j] = p.reset[c - j];
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      carry = rv[j] ? gv[j] : decay_add(a2 * sv[j], carry, gv[j]);
      gs[(c - j) * DN] = carry;
    }
  }
  for (; c >= 0; --c) {
    const float gv = gs[c * DN];
    carry = p.reset[c] ? gv : decay_add(a2 * ds[c * p.D], carry, gv);
    gs[c * DN] = carry;
  }
}

// Main pass; lanes, waves and LDS as in k_bwd_main.
template <int N, typename InT, int DISC>
__global__ void __launch_bounds__(kWave * BwdLayout<N>::NG) __attribute__((amdgpu_waves_per_eu(4)))
k_packed_bwd(const PackedBwdParams p) {
  constexpr int NS = BwdLayout<N>::NS, NG = BwdLayout<N>::NG;
  constexpr int F = kBwdFine, K = kBwdBlock, H = kBwdHalf;
  constexpr int RR = 4 * NS;           // rows summed together
  constexpr int LPR = kWave / RR;      // lanes per row; each sums RR floats
  __shared__ __attribute__((aligned(16))) float red[NG][RR][kRedPitch];
  __shared__ float xch[2][2][NG][K][kWave];
  // bf16 rows of B and C, widened once, double-buffered by 16 tokens; fp32 rows go
  // through scalar loads
  constexpr bool kRowsLds = !std::is_same<InT, float>::value;
  __shared__ __attribute__((aligned(16))) float rows[kRowsLds ? 2 : 1][2][kRowsLds ? F : 1][N];

  const int wg = xcd_remap(blockIdx.x, p.nwg);
  const int64_t dtile = wg % p.dtiles;
  const int32_t chunk = wg / p.dtiles;
  const int w = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int lane = threadIdx.x % kWave;
  const int64_t dbase = dtile * kWave;
  const int64_t d = dbase + lane_offset(dbase, p.D, static_cast<uint32_t>(lane));
  const bool valid = dbase + lane < p.D;   // lanes past D duplicate D - 1 and add nothing
  if (!valid) {
#pragma unroll
    for (int rr = 0; rr < RR; ++rr) red[w][rr][lane] = 0.0f;
  }
  int xb = 0;
  const int n0 = w * NS;
  const int64_t dn = d * N + n0, DN = p.D * N;   // this lane's states in a (D, N) array

  ChanConst<NS, DISC> cc;
  load_chan<NS, DISC>(cc, p.A + dn, p.exact_thr);
  const float dsk = p.Dskip ? p.Dskip[d] : 0.0f;
  constexpr bool kShortSeries = kRowsLds;
  float zoh_thr = 0.0f;   // below it ZOH's factor is taken from its series
  if constexpr (DISC == kZoh) {
    float amin = __builtin_inff();
#pragma unroll
    for (int n = 0; n < NS; ++n) amin = fminf(amin, fabsf(cc.A2[n] * kLn2));
    zoh_thr = amin > 0.0f ? series_z<kShortSeries>() / amin : __builtin_inff();
  }

  const int32_t t0 = chunk * p.T, t1 = p.q.tokens - t0 > p.T ? t0 + p.T : p.q.tokens;
  const int32_t lo = seq_start(p.q, 0), hi = seq_start(p.q, p.q.S);
  const int32_t from = t0 > lo ? t0 : lo, to = t1 < hi ? t1 : hi;   // tokens of sequences
  // the first token of the sequence whose tokens are walked next
  int32_t first = INT32_MIN;
  float g[NS];
  zero_n(g);
  if (from < to) {
    const int32_t s = seq_at(p.q, to - 1);
    first = seq_start(p.q, s);
    if (first > to - 1) first = to - 1;
    if (seq_start(p.q, s + 1) > t1) {
      load_n(g, p.gsum + int64_t(chunk) * DN + dn);
    } else if (p.dh_last) {
      load_n(g, p.dh_last + int64_t(s) * DN + dn);
    }
  }
  float dAacc[NS];
  zero_n(dAacc);
  float dDacc = 0.0f;

  const InT* Bp = static_cast<const InT*>(p.Bm);
  const InT* Cp = static_cast<const InT*>(p.Cm);
  const uint32_t lane_in = uint32_t(d - dbase) * sizeof(InT), lane_f = uint32_t(d - dbase) * 4u;
  const uint32_t row_f = uint32_t(p.D * 4);
  constexpr InT* kIn = nullptr;
  constexpr float* kF = nullptr;
  const bool ok = p.rows_ok != 0;

  // the rows each thread moves into LDS, loaded 16 tokens ahead (rows of tokens of no
  // sequence as 0)
  constexpr int kRowVals = kRowsLds ? 2 * F * N : 1;
  constexpr int RV = (kRowVals + kWave * NG - 1) / (kWave * NG);
  float rpre[RV];
  auto rows_load = [&](int32_t f0) {
#pragma unroll
    for (int i = 0; i < RV; ++i) {
      const int e = static_cast<int>(threadIdx.x) + i * kWave * NG;
      const int kind = (e / (F * N)) & 1, j = (e / N) % F, n = e % N;
      const bool in = e < kRowVals && f0 + j >= lo && f0 + j < hi;
      rpre[i] = in ? ld((kind == 0 ? Bp + int64_t(f0 + j) * p.bs : Cp + int64_t(f0 + j) * p.cs) + n) : 0.0f;
    }
  };
  const int32_t f_top = (t1 - 1) / F * F;
  if constexpr (kRowsLds) rows_load(f_top);
  int rb = 0;

  for (int32_t f0 = f_top; f0 >= t0; f0 -= F) {
    const int len = p.q.tokens - f0 < F ? p.q.tokens - f0 : F;
    // tokens jlo .. jhi - 1 of them belong to sequences; bit j of begins: token j is a first one
    const int jlo = lo > f0 ? (lo - f0 < len ? lo - f0 : len) : 0;
    const int jhi = hi - f0 < len ? (hi > f0 ? hi - f0 : 0) : len;
    const bool some = jlo < jhi;
    uint32_t begins = 0;
    while (first >= f0) {
      begins |= 1u << (first - f0);
      const int32_t before = first > lo ? seq_start(p.q, seq_at(p.q, first - 1)) : INT32_MIN;
      first = before < first ? before : INT32_MIN;   // (falling offsets end the walk too)
    }
    if (!some) {   // wave-uniform, and the workgroup's
      for (int j = w; j < len; j += NG) {
        p.dx[int64_t(f0 + j) * p.D + d] = 0.0f;
        p.ddelta[int64_t(f0 + j) * p.D + d] = 0.0f;
      }
      for (int e = threadIdx.x; e < len * N; e += kWave * NG) {
        const int64_t i = (int64_t(f0 + e / N) * p.dtiles + dtile) * N + e % N;
        p.dBp[i] = 0.0f;
        p.dCp[i] = 0.0f;
      }
      if constexpr (kRowsLds) {
        if (f0 > t0) rows_load(f0 - F);
      }
      continue;
    }
    if constexpr (kRowsLds) {
#pragma unroll
      for (int i = 0; i < RV; ++i) {
        const int e = static_cast<int>(threadIdx.x) + i * kWave * NG;
        if (e < kRowVals) (&rows[rb][0][0][0])[e] = rpre[i];
      }
      __syncthreads();
      if (f0 > t0) rows_load(f0 - F);
    }
    const float* Brow = &rows[kRowsLds ? rb : 0][0][0][n0];
    const float* Crow = &rows[kRowsLds ? rb : 0][1][0][n0];
    // every row is read at a token of a sequence: those of others repeat the nearest
    auto near = [&](int j) { return j < jlo ? jlo : j < jhi ? j : jhi - 1; };
    const RowWindow wx = window<InT>(p.x, p.xs, p.D, dbase, f0, jhi);
    const RowWindow wd = window<InT>(p.delta, p.dls, p.D, dbase, f0, jhi);
    const RowWindow wy = window<InT>(p.dy, p.ys, p.D, dbase, f0, jhi);
    const __amdgpu_buffer_rsrc_t rdx = make_rsrc(p.dx + int64_t(f0) * p.D + dbase, uint32_t(len) * row_f);
    const __amdgpu_buffer_rsrc_t rdd = make_rsrc(p.ddelta + int64_t(f0) * p.D + dbase, uint32_t(len) * row_f);
    const InT* Bc = Bp + int64_t(f0) * p.bs + n0;
    const InT* Cc = Cp + int64_t(f0) * p.cs + n0;
    const float* hin = f0 > 0 ? p.hsave + (int64_t(f0 / F) - 1) * DN + dn : nullptr;
    // the state before the first token of a sequence
    auto initial = [&](float (&h)[NS], int32_t t) {
      zero_n(h);
      if (p.h0) load_n(h, p.h0 + int64_t(seq_at(p.q, t)) * DN + dn);
    };
#pragma unroll
    for (int half = F / H - 1; half >= 0; --half) {
      const int j0 = half * H;
      if (j0 >= len) continue;   // wave-uniform
      float h[NS];
      zero_n(h);
      if (hin) load_n(h, hin);
      float stash[H][NS];
      float xa[K], da[K];
#pragma unroll
      for (int jj = 0; jj < K; ++jj) {
        xa[jj] = ldb(wx.r, lane_in, uint32_t(near(jj)) * wx.row, kIn);
        da[jj] = ldb(wd.r, lane_in, uint32_t(near(jj)) * wd.row, kIn);
      }
#pragma unroll
      for (int jb = 0; jb < (j0 + H) / K; ++jb) {
        float xn[K], dn_[K];
        const int nb = (jb + 1 < (j0 + H) / K) ? jb + 1 : jb;
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          xn[jj] = ldb(wx.r, lane_in, uint32_t(near(nb * K + jj)) * wx.row, kIn);
          dn_[jj] = ldb(wd.r, lane_in, uint32_t(near(nb * K + jj)) * wd.row, kIn);
        }
        float Bb[K][NS];
        if constexpr (!kRowsLds) {
#pragma unroll
          for (int jj = 0; jj < K; ++jj) row_of<NS>(Bb[jj], Bc + near(jb * K + jj) * p.bs, ok);
        }
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          const int j = jb * K + jj;
          float Bv[NS];
          if constexpr (kRowsLds) {
            lds_row<NS>(Bv, Brow + j * N);
          } else {
#pragma unroll
            for (int n = 0; n < NS; ++n) Bv[n] = Bb[jj][n];
          }
          if (begins >> j & 1) initial(h, f0 + j);
          if (j >= j0) {
#pragma unroll
            for (int n = 0; n < NS; ++n) stash[j - j0][n] = h[n];
          }
          if (j >= jlo && j < jhi) {
            if (any_exact<NS, DISC>(cc, da[jj]))
              ssm_step_lane<NS, DISC, false, true, true>(h, cc, Bv, Bv, xa[jj], da[jj]);
            else
              ssm_step_lane<NS, DISC, false, false>(h, cc, Bv, Bv, xa[jj], da[jj]);
          }
        }
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          xa[jj] = xn[jj];
          da[jj] = dn_[jj];
        }
      }
#pragma unroll
      for (int jb = (j0 + H) / K - 1; jb >= j0 / K; --jb) {
        if (jb * K >= len) continue;   // wave-uniform
        float ub[K], db[K], yb[K], Bb[K][NS], Cb[K][NS];
#pragma unroll
        for (int jj = 0; jj < K; ++jj) {
          const int j = near(jb * K + jj);
          ub[jj] = ldb(wx.r, lane_in, uint32_t(j) * wx.row, kIn);
          db[jj] = ldb(wd.r, lane_in, uint32_t(j) * wd.row, kIn);
          yb[jj] = ldb(wy.r, lane_in, uint32_t(j) * wy.row, kIn);
          if constexpr (!kRowsLds) {
            row_of<NS>(Bb[jj], Bc + j * p.bs, ok);
            row_of<NS>(Cb[jj], Cc + j * p.cs, ok);
          }
        }
#pragma unroll
        for (int jj = K - 1; jj >= 0; --jj) {
          const int j = jb * K + jj;
          float pB[NS], pC[NS], du = 0.0f, ddt = 0.0f;
          zero_n(pB);
          zero_n(pC);
          const float u = ub[jj], dv = db[jj], dyv = yb[jj];
          float Bv[NS], Cv[NS];
          if constexpr (kRowsLds) {
            lds_row<NS>(Bv, Brow + j * N);
            lds_row<NS>(Cv, Crow + j * N);
          } else {
#pragma unroll
            for (int n = 0; n < NS; ++n) {
              Bv[n] = Bb[jj][n];
              Cv[n] = Cb[jj][n];
            }
          }
          if (j >= jlo && j < jhi) {
            const int js = j - j0;
            const bool exact = any_exact<NS, DISC>(cc, dv);
            // the state after the step: the one before the next, or, before a sequence's
            // first token, formed again
            float hn[NS];
#pragma unroll
            for (int n = 0; n < NS; ++n) hn[n] = (js + 1 < H) ? stash[js + 1 < H ? js + 1 : js][n] : h[n];
            if (js + 1 < H && (begins >> (j + 1) & 1)) {
#pragma unroll
              for (int n = 0; n < NS; ++n) hn[n] = stash[js][n];
              if (exact)
                ssm_step_lane<NS, DISC, false, true, true>(hn, cc, Bv, Bv, u, dv);
              else
                ssm_step_lane<NS, DISC, false, false>(hn, cc, Bv, Bv, u, dv);
            }
            const bool series = DISC == kZoh && __builtin_amdgcn_ballot_w64(dv < zoh_thr) != 0;
            if (series)
              bwd_lane_step<NS, DISC, true, kShortSeries>(g, dAacc, cc, Bv, Cv, stash[js], hn, u, dv, dyv, exact, pB,
                                                          pC, du, ddt);
            else
              bwd_lane_step<NS, DISC, false, kShortSeries>(g, dAacc, cc, Bv, Cv, stash[js], hn, u, dv, dyv, exact, pB,
                                                           pC, du, ddt);
            dDacc = fmaf(dyv, u, dDacc);
            if (begins >> j & 1) {
              const int32_t t = f0 + j;
              if (p.dh0) store_n(p.dh0 + int64_t(seq_at(p.q, t)) * DN + dn, g);
              zero_n(g);
              if (t > lo && p.dh_last) load_n(g, p.dh_last + int64_t(seq_at(p.q, t - 1)) * DN + dn);
              // (where the sequence before ends before this super-chunk, that is another's to take)
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
            const int jr = jj + rr / (2 * NS);
            const int kind = (rr / NS) & 1;
            const int n = rr % NS;
            if (c == 0 && jb * K + jr < len) {
              float* dst = kind == 0 ? p.dBp : p.dCp;
              dst[(int64_t(f0 + jb * K + jr) * p.dtiles + dtile) * N + n0 + n] = acc;
            }
            __builtin_amdgcn_wave_barrier();
          }
        }
        __syncthreads();
#pragma unroll
        for (int jj = w; jj < K; jj += NG) {
          const int j = jb * K + jj;
          if (j < len) {
            float su = 0.0f, sd = 0.0f;
#pragma unroll
            for (int v = 0; v < NG; ++v) {
              su += xch[xb][0][v][jj][lane];
              sd += xch[xb][1][v][jj][lane];
            }
            if (j >= jlo && j < jhi) su = fmaf(dsk, ldb(wy.r, lane_in, uint32_t(j) * wy.row, kIn), su);
            stb(rdx, lane_f, uint32_t(j) * row_f, su, kF);
            stb(rdd, lane_f, uint32_t(j) * row_f, sd, kF);
          }
        }
        xb ^= 1;
      }
    }
    rb ^= 1;
  }
  store_n(p.dAp + int64_t(chunk) * DN + dn, dAacc);
  if (w == 0) p.dDp[int64_t(chunk) * p.D + d] = dDacc;
  // sequences without tokens: their last state is their first
  if (chunk == 0 && p.dh0) {
    for (int32_t s0 = 0; s0 < p.q.S; s0 += kWave) {
      const int32_t s = s0 + lane;
      bool empty = false;
      if (s < p.q.S) empty = ssmq::in_tokens(p.q, p.q.offsets[s]) >= ssmq::in_tokens(p.q, p.q.offsets[s + 1]);
      uint64_t todo = __builtin_amdgcn_ballot_w64(empty);
      while (todo) {
        const int64_t e = s0 + __builtin_ctzll(todo);
        todo &= todo - 1;
        float v[NS];
        zero_n(v);
        if (p.dh_last) load_n(v, p.dh_last + e * DN + dn);
        store_n(p.dh0 + e * DN + dn, v);
      }
    }
  }
}

// dB, dC: the channel tiles' sums of a (token, state).
template <int N>
__global__ void __launch_bounds__(256) k_packed_bwd_bc(const PackedBwdParams p) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  if (i >= int64_t(p.q.tokens) * N) return;
  const int64_t t = i / N, n = i - t * N;
  const float* sb = p.dBp + t * p.dtiles * N + n;
  const float* sc = p.dCp + t * p.dtiles * N + n;
  float ab = 0.0f, ac = 0.0f;
  for (int k = 0; k < p.dtiles; ++k) {
    ab += sb[k * N];
    ac += sc[k * N];
  }
  p.dB[i] = ab;
  p.dC[i] = ac;
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
