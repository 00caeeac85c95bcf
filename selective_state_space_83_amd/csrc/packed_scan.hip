// packed_scan.hip -- host side of the scan over packed sequences: argument checks,
// the chunk plan and launches.  The device code is packed_scan.hpp and
// packed_bwd.hpp; the contract include/ssm_scan.h.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "ssm_scan.h"
#include "ssm_host.hpp"
#include "packed.hpp"

// The scan's device code, for what it shares with this one; in a namespace of this
// file, so that its kernels that are no templates are defined once for each file.
namespace {
#include "ssm_kernels.hpp"
#include "ssm_bwd.hpp"
#include "packed_scan.hpp"
#include "packed_bwd.hpp"
}  // namespace

namespace {

using namespace ssmh;
using namespace ssmp;

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 4096;   // tokens are counted in 32 bits
// A chunk's rows are addressed through buffer windows with 32-bit offsets.
constexpr int64_t kMaxWindow = (int64_t(1) << 31) - 1;

// Waves the plan aims for: four, or where that cuts chunks shorter than kShortChunk
// tokens three, to each of the 1024 SIMDs; chunks of at least kMinChunk tokens, and
// of at most kLongChunk once there are kBalanceChunks of them; no cut for
// kNoSplitTokens or fewer (the scan's plan, whose work a chunk's is).
constexpr int64_t kTargetWaves = 4 * 1024, kShortTargetWaves = 3 * 1024;
constexpr int64_t kShortChunk = 64, kMinChunk = 8, kBalanceChunks = 16, kLongChunk = 256, kNoSplitTokens = 32;

struct Plan {
  bool wave = false;   // one launch, time across the lanes (k_packed_wave)
  int64_t T = 1, nc = 1, dtiles = 0;
  size_t off_dsum = 0, off_hsum = 0, off_hstart = 0, off_reset = 0, total = 0;
};

template <typename Args>
int64_t widest_stride(const Args* a) {
  return std::max(a->x_stride, a->delta_stride);
}

// The chunk length below which the carries cost more than the walks gain: a token of a
// chunk takes about 0.55 us in the two walks, a chunk 0.026 us + 0.05 ns a channel in
// the carries' walk and their traffic.  (bf16, 16 states, without it: 16384 x 100 50 us
// for 76, 16384 x 256 62 for 71, 65536 x 64 86 for 131, 1024 x 1536 37 for 44.)
int64_t chunk_floor(int64_t tokens, int64_t D) { return int64_t(std::sqrt(double(tokens) * double(D + 520) / 11000)); }

// Sizes assumed validated.  kept: with room for the initial states that a cache updated in
// place needs kept; by whether there are states both ways, not by their addresses.
Plan make_plan(int64_t tokens, int64_t D, int64_t N, int64_t chunk_len, int64_t stride, bool kept) {
  Plan pl;
  pl.dtiles = (D + kWave - 1) / kWave;
  if (tokens == 0) return pl;
  int64_t T;
  if (chunk_len > 0) {
    T = std::min(chunk_len, (tokens + 3) / 4 * 4);
  } else {
    auto chunks = [&](int64_t target) {
      return std::max<int64_t>(1, std::min<int64_t>(target / pl.dtiles, tokens / kMinChunk));
    };
    int64_t nc = chunks(kTargetWaves);
    if (nc > 1 && (tokens + nc - 1) / nc < kShortChunk) nc = chunks(kShortTargetWaves);
    if (tokens <= kNoSplitTokens) nc = 1;
    T = ((tokens + nc - 1) / nc + 3) / 4 * 4;
    T = std::max(T, (chunk_floor(tokens, D) + 3) / 4 * 4);
    if (nc >= kBalanceChunks) T = std::min(T, kLongChunk);
  }
  // rows of 4 bytes an element at most; 4 tokens fit (check_sizes)
  const int64_t most = kMaxWindow / (std::max(stride, D) * 4) / 4 * 4;
  pl.T = std::min(T, std::max<int64_t>(4, most));
  pl.nc = (tokens + pl.T - 1) / pl.T;
  if (pl.nc > 1) {
    const size_t n = size_t(pl.nc - 1), d = size_t(D);
    pl.off_hsum = align256(n * d * 4);
    pl.off_hstart = pl.off_hsum + align256(n * d * size_t(N) * 4);
    pl.off_reset = pl.off_hstart + (kept ? align256(n * d * size_t(N) * 4) : 0);
    pl.total = pl.off_reset + align256(n * 4);
  }
  return pl;
}

// Whether the launch with time across the lanes takes the problem: the scan's rule
// (wave_wins in ssm_scan.hip) for one row of its tokens.
bool wave_wins(int64_t tokens, int64_t D) {
  const int64_t blocks = (tokens + kWave - 1) / kWave;
  return tokens <= 512 && D <= std::min<int64_t>(4096, kWave * tokens) / std::max<int64_t>(blocks, 1);
}

Plan plan_of(const ssm_packed_scan_args_t* a) {
  if (a->chunk_len == 0 && wave_wins(a->tokens, a->dim)) {
    Plan pl;
    pl.wave = true;
    return pl;
  }
  int64_t stride = widest_stride(a);
  if (a->z) stride = std::max(stride, a->z_stride);
  return make_plan(a->tokens, a->dim, a->dstate, a->chunk_len, stride, a->h0 && a->h_last);
}

bool supported_n(int64_t n) { return n == 1 || n == 2 || n == 4 || n == 8 || n == 16; }

Range rows_of(const void* p, int64_t rows, int64_t width, int64_t stride, size_t es) {
  if (!p || rows == 0) return Range{nullptr, 0};
  return Range{p, size_t((rows - 1) * stride + width) * es};
}

// What the calls check of their sizes and types; rows: tokens or batch.
template <typename Args>
ssm_status_t check_sizes(const Args* a, int64_t rows, int64_t seqs, int64_t slots,
                         std::initializer_list<int64_t> strides) {
  if (rows < 0 || seqs < 0 || slots < 0 || a->dim < 0 || a->dstate < 0)
    return fail(SSM_ERR_SHAPE, "negative size: tokens=%lld sequences=%lld slots=%lld dim=%lld dstate=%lld",
                (long long)rows, (long long)seqs, (long long)slots, (long long)a->dim, (long long)a->dstate);
  if (!supported_n(a->dstate)) return fail(SSM_ERR_UNSUPPORTED, "dstate %lld not in {1,2,4,8,16}", (long long)a->dstate);
  if (rows > kMaxTokens || seqs > kMaxTokens || slots > kMaxTokens)
    return fail(SSM_ERR_SHAPE, "problem too large (tokens, sequences and slots are counted in 32 bits)");
  int64_t n;
  // per-token sums of every channel tile, and states, in bytes
  if (a->dim > (int64_t(1) << 24) || !mul_ok(std::max({rows, seqs, slots}), std::max<int64_t>(a->dim, 1) * 16, &n) ||
      n > INT64_MAX / 64)
    return fail(SSM_ERR_SHAPE, "sizes overflow");
  for (int64_t s : strides)
    if (s < 0 || s > kMaxWindow / 32)   // a window holds at least 4 rows of 4-byte elements
      return fail(SSM_ERR_SHAPE, "a row stride is negative or too large");
  if (a->dtype != SSM_F32 && a->dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown dtype %d", a->dtype);
  if (a->disc != SSM_DISC_DELTA_B && a->disc != SSM_DISC_ZOH)
    return fail(SSM_ERR_DTYPE, "unknown discretization %d", a->disc);
  return SSM_OK;
}

ssm_status_t check_softplus(int32_t v) {
  return v == 0 || v == 1 ? SSM_OK : fail(SSM_ERR_UNSUPPORTED, "delta_softplus must be 0 or 1");
}

ssm_status_t check_fwd_sizes(const ssm_packed_scan_args_t* a) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_sizes(a, a->tokens, a->seqs, a->slots,
                                    {a->x_stride, a->delta_stride, a->z ? a->z_stride : 0, a->b_stride, a->c_stride}))
    return st;
  if (ssm_status_t st = check_softplus(a->delta_softplus)) return st;
  if (a->chunk_len < 0 || a->chunk_len % 4 != 0)
    return fail(SSM_ERR_UNSUPPORTED, "chunk_len must be a multiple of 4, not negative");
  return SSM_OK;
}

ssm_status_t check_fwd(const ssm_packed_scan_args_t* a) {
  if (ssm_status_t st = check_fwd_sizes(a)) return st;
  if ((a->slot || a->resume) && !a->h0 && !a->h_last)
    return fail(SSM_ERR_UNSUPPORTED, "slot and resume go with h0 or h_last");
  if ((a->h0 || a->h_last) && !a->slot && a->slots != a->seqs)
    return fail(SSM_ERR_SHAPE, "without slot, slots must be seqs");
  const size_t D = size_t(a->dim), N = size_t(a->dstate), T = size_t(a->tokens), S = size_t(a->seqs);
  if (D == 0 || S == 0) return SSM_OK;
  if (!a->A || !a->offsets || (T > 0 && (!a->x || !a->delta || !a->Bm || !a->Cm || !a->y)))
    return fail(SSM_ERR_NULL, "x, delta, A, Bm, Cm, offsets and y are required");
  const size_t es = dtype_size(a->dtype);
  for (const void* p : {a->x, a->delta, a->z, a->Bm, a->Cm, static_cast<const void*>(a->y)})
    if (misaligned(p, es)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  for (const void* p : {static_cast<const void*>(a->A), static_cast<const void*>(a->Dskip),
                        static_cast<const void*>(a->delta_bias), static_cast<const void*>(a->offsets),
                        static_cast<const void*>(a->slot), static_cast<const void*>(a->h0),
                        static_cast<const void*>(a->h_last), static_cast<const void*>(a->h_saved)})
    if (misaligned(p, 4)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const Plan pl = plan_of(a);
  if (misaligned(a->workspace, 256)) return fail(SSM_ERR_UNSUPPORTED, "workspace must be aligned to 256 bytes");
  if (pl.total > 0 && !a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", pl.total);
  if (a->workspace_bytes < pl.total)
    return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, pl.total);
  const size_t states = size_t(a->slots) * D * N * 4, kept = T > 0 ? ((T + 15) / 16 - 1) * D * N * 4 : 0;
  const bool in_place = a->h_last && a->h_last == a->h0;
  const Range outs[] = {{a->y, T * D * es}, {a->h_last, states}, {a->h_saved, kept}, {a->workspace, pl.total}};
  const Range ins[] = {rows_of(a->x, a->tokens, a->dim, a->x_stride, es),
                       rows_of(a->delta, a->tokens, a->dim, a->delta_stride, es),
                       rows_of(a->z, a->tokens, a->dim, a->z_stride, es),
                       rows_of(a->Bm, a->tokens, a->dstate, a->b_stride, es),
                       rows_of(a->Cm, a->tokens, a->dstate, a->c_stride, es),
                       {a->A, D * N * 4},
                       {a->Dskip, D * 4},
                       {a->delta_bias, D * 4},
                       {a->offsets, (S + 1) * 4},
                       {a->slot, S * 4},
                       {a->resume, S},
                       {a->h0, states}};
  for (int i = 0; i < 4; ++i) {
    for (int k = 0; k < 12; ++k)
      if (overlap(outs[i], ins[k]) && !(i == 1 && k == 11 && in_place))
        return fail(SSM_ERR_ALIAS, "an output overlaps an input");
    for (int k = i + 1; k < 4; ++k)
      if (overlap(outs[i], outs[k])) return fail(SSM_ERR_ALIAS, "two outputs overlap");
  }
  return SSM_OK;
}

ssm_status_t check_step(const ssm_packed_step_args_t* a) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_sizes(a, a->batch, a->batch, a->slots,
                                    {a->x_stride, a->delta_stride, a->z ? a->z_stride : 0, a->b_stride, a->c_stride}))
    return st;
  if (ssm_status_t st = check_softplus(a->delta_softplus)) return st;
  if (a->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (!a->slot && a->slots != a->batch) return fail(SSM_ERR_SHAPE, "without slot, slots must be batch");
  const size_t D = size_t(a->dim), N = size_t(a->dstate), B = size_t(a->batch);
  if (D == 0 || B == 0) return SSM_OK;
  if (!a->x || !a->delta || !a->A || !a->Bm || !a->Cm || !a->y || (a->slots > 0 && !a->h))
    return fail(SSM_ERR_NULL, "x, delta, A, Bm, Cm, h and y are required");
  const size_t es = dtype_size(a->dtype);
  for (const void* p : {a->x, a->delta, a->z, a->Bm, a->Cm, static_cast<const void*>(a->y)})
    if (misaligned(p, es)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  for (const void* p : {static_cast<const void*>(a->A), static_cast<const void*>(a->Dskip),
                        static_cast<const void*>(a->delta_bias), static_cast<const void*>(a->slot)})
    if (misaligned(p, 4)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  if (misaligned(a->h, 4 * std::min<size_t>(N, 4)))
    return fail(SSM_ERR_UNSUPPORTED, "h must be aligned to 4 * min(dstate, 4) bytes");
  const Range h{a->h, size_t(a->slots) * D * N * 4}, y{a->y, B * D * es};
  const Range ins[] = {rows_of(a->x, a->batch, a->dim, a->x_stride, es),
                       rows_of(a->delta, a->batch, a->dim, a->delta_stride, es),
                       rows_of(a->z, a->batch, a->dim, a->z_stride, es),
                       rows_of(a->Bm, a->batch, a->dstate, a->b_stride, es),
                       rows_of(a->Cm, a->batch, a->dstate, a->c_stride, es),
                       {a->A, D * N * 4},
                       {a->Dskip, D * 4},
                       {a->delta_bias, D * 4},
                       {a->slot, B * 4}};
  for (const Range& r : ins)
    if (overlap(h, r) || overlap(y, r)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
  if (overlap(h, y)) return fail(SSM_ERR_ALIAS, "y overlaps h");
  return SSM_OK;
}

// Where |Delta A| is below this the decay takes its slow form (see ssm_kernels.hpp),
// the scan's thresholds.
float exact_threshold(int32_t disc, int32_t dtype) {
  if (dtype == SSM_BF16) return 1.0f / 8192.0f;
  return disc == SSM_DISC_ZOH ? 0.03f : 1.0f / 1024.0f;
}

int dt_mode_of(const float* bias, int32_t softplus) { return softplus ? kDtSoftplus : bias ? kDtBias : kDtRaw; }

// bf16 rows that do not all start on 4 bytes
bool odd_rows(const void* p, uint32_t stride) { return misaligned(p, 4) || stride % 2 != 0; }

// a launch holds at most 2^32 - 1 lanes
ssm_status_t grid_ok(int64_t workgroups, int64_t lanes) {
  return workgroups > int64_t(UINT32_MAX) / lanes || workgroups > kMaxGrid
             ? fail(SSM_ERR_SHAPE, "problem too large for one launch")
             : SSM_OK;
}

template <int N, typename InT, int DISC, bool ODD>
ssm_status_t run_chunks(PackedParams p, hipStream_t s) {
  const int64_t out = int64_t(p.nc) * p.dtiles;
  if (ssm_status_t st = grid_ok(out, kWave)) return st;
  if (ssm_status_t st = grid_ok((p.D * N + kWave - 1) / kWave, kWave * kCarryWaves)) return st;
  if (p.nc > 1) {
    p.nwg = (p.nc - 1) * p.dtiles;
    hipLaunchKernelGGL((k_packed_summary<N, InT, DISC, ODD>), dim3(uint32_t(p.nwg)), dim3(kWave), 0, s, p);
    if (ssm_status_t st = launch_status("k_packed_summary")) return st;
    hipLaunchKernelGGL((k_packed_carry<N>), dim3(uint32_t((p.D * N + kWave - 1) / kWave)), dim3(kWave * kCarryWaves), 0,
                       s, p);
    if (ssm_status_t st = launch_status("k_packed_carry")) return st;
  }
  p.nwg = int32_t(out);
  if (p.z)
    hipLaunchKernelGGL((k_packed_out<N, InT, DISC, true, ODD>), dim3(uint32_t(out)), dim3(kWave), 0, s, p);
  else
    hipLaunchKernelGGL((k_packed_out<N, InT, DISC, false, ODD>), dim3(uint32_t(out)), dim3(kWave), 0, s, p);
  return launch_status("k_packed_out");
}

template <int N, typename InT, int DISC>
ssm_status_t run_fwd(const PackedParams& p, hipStream_t s) {
  if (p.nc == 0) {   // the plan with time across the lanes
    if (p.z)
      hipLaunchKernelGGL((k_packed_wave<N, InT, DISC, true>), dim3(uint32_t(p.D)), dim3(kWave * BwdLayout<N>::NG), 0, s, p);
    else
      hipLaunchKernelGGL((k_packed_wave<N, InT, DISC, false>), dim3(uint32_t(p.D)), dim3(kWave * BwdLayout<N>::NG), 0, s, p);
    return launch_status("k_packed_wave");
  }
  if constexpr (!std::is_same<InT, float>::value && N > 1) {
    if (odd_rows(p.Bm, p.bs) || odd_rows(p.Cm, p.cs)) return run_chunks<N, InT, DISC, true>(p, s);
  }
  return run_chunks<N, InT, DISC, false>(p, s);
}

template <int N, typename InT, int DISC>
ssm_status_t run_step(PackedStepParams p, hipStream_t s) {
  using L = StepLayout<N>;
  p.dtiles = int32_t((p.D + L::CPW - 1) / L::CPW);
  const int64_t n = (p.Bt + L::ROWS - 1) / L::ROWS * ((p.dtiles + L::WPG - 1) / L::WPG);
  if (ssm_status_t st = grid_ok(n, kWave * L::WPG)) return st;
  p.nwg = int32_t(n);
  hipLaunchKernelGGL((k_packed_step<N, InT, DISC>), dim3(uint32_t(n)), dim3(kWave * L::WPG), 0, s, p);
  return launch_status("k_packed_step");
}

struct BwdPlan {
  int64_t T = 16, nc = 1, dtiles = 0;
  size_t off_dsum = 0, off_reset = 0, off_dAp = 0, off_dDp = 0, off_dBCp = 0, total = 0;
};

// Super-chunks: enough for the reverse summary's waves, at most kBwdLong tokens each
// (more, shorter waves even out the SIMDs).
constexpr int64_t kBwdLong = 64;

BwdPlan bwd_plan(const ssm_packed_scan_bwd_args_t* a) {
  BwdPlan pl;
  pl.dtiles = (a->dim + kWave - 1) / kWave;
  const int64_t tokens = a->tokens, fine = (tokens + kBwdFine - 1) / kBwdFine;
  if (a->dim == 0) return pl;
  // (without tokens: one super-chunk, whose sums are 0)
  if (a->super_chunk > 0) {
    pl.T = std::min<int64_t>(a->super_chunk, fine * kBwdFine);
  } else {
    const int64_t nc = std::max<int64_t>(1, std::min(kTargetWaves / pl.dtiles, fine));
    // (see chunk_floor; a token takes 0.83 us here, a chunk 0.06 us + 0.1 ns a channel:
    // 16384 x 100 fp32 89 us for 122)
    const int64_t least = int64_t(std::sqrt(double(tokens) * double(a->dim + 600) / 8300)) + kBwdFine / 2;
    pl.T = std::min(std::max((fine + nc - 1) / nc, least / kBwdFine) * kBwdFine, kBwdLong);
  }
  // the reverse summary's windows
  const int64_t stride = std::max({a->x_stride, a->delta_stride, a->dy_stride, a->dim});
  pl.T = std::min(pl.T, std::max<int64_t>(kBwdFine, kMaxWindow / (stride * 4) / kBwdFine * kBwdFine));
  pl.T = std::max<int64_t>(pl.T, kBwdFine);
  pl.nc = std::max<int64_t>(1, (tokens + pl.T - 1) / pl.T);
  const size_t n = size_t(pl.nc), d = size_t(a->dim), N = size_t(a->dstate), t = size_t(tokens);
  size_t off = align256((n - 1) * d * N * 4);   // gsum
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  pl.off_dsum = take((n - 1) * d * 4);
  pl.off_reset = take((n - 1) * 4);
  pl.off_dAp = take(n * d * N * 4);
  pl.off_dDp = take(n * d * 4);
  pl.off_dBCp = take(t * size_t(pl.dtiles) * 2 * N * 4);
  pl.total = off;
  return pl;
}

ssm_status_t check_bwd_sizes(const ssm_packed_scan_bwd_args_t* a) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_sizes(a, a->tokens, a->seqs, 0,
                                    {a->x_stride, a->delta_stride, a->b_stride, a->c_stride, a->dy_stride}))
    return st;
  if (a->super_chunk < 0 || a->super_chunk % 16 != 0)
    return fail(SSM_ERR_UNSUPPORTED, "super_chunk must be a multiple of 16, not negative");
  // a window holds 16 rows
  for (int64_t s : {a->x_stride, a->delta_stride, a->dy_stride})
    if (s > kMaxWindow / 128) return fail(SSM_ERR_SHAPE, "a row stride is too large");
  if (a->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  return SSM_OK;
}

ssm_status_t check_bwd(const ssm_packed_scan_bwd_args_t* a) {
  if (ssm_status_t st = check_bwd_sizes(a)) return st;
  const size_t D = size_t(a->dim), N = size_t(a->dstate), T = size_t(a->tokens), S = size_t(a->seqs);
  if (D == 0) return SSM_OK;
  const size_t kept = T > 0 ? ((T + 15) / 16 - 1) * D * N * 4 : 0;
  if (!a->A || !a->offsets || !a->dA ||
      (T > 0 && (!a->x || !a->delta || !a->Bm || !a->Cm || !a->dy || !a->dx || !a->ddelta || !a->dB || !a->dC)))
    return fail(SSM_ERR_NULL, "x, delta, A, Bm, Cm, offsets, dy, dx, ddelta, dA, dB and dC are required");
  if (kept > 0 && !a->h_saved) return fail(SSM_ERR_NULL, "h_saved is required (the forward call keeps it)");
  const size_t es = dtype_size(a->dtype);
  for (const void* p : {a->x, a->delta, a->Bm, a->Cm, a->dy})
    if (misaligned(p, es)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  for (const void* p :
       {static_cast<const void*>(a->A), static_cast<const void*>(a->Dskip), static_cast<const void*>(a->offsets),
        static_cast<const void*>(a->h0), static_cast<const void*>(a->h_saved), static_cast<const void*>(a->dh_last),
        static_cast<const void*>(a->dx), static_cast<const void*>(a->ddelta), static_cast<const void*>(a->dA),
        static_cast<const void*>(a->dB), static_cast<const void*>(a->dC), static_cast<const void*>(a->dD),
        static_cast<const void*>(a->dh0)})
    if (misaligned(p, 4)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const BwdPlan pl = bwd_plan(a);
  if (misaligned(a->workspace, 256)) return fail(SSM_ERR_UNSUPPORTED, "workspace must be aligned to 256 bytes");
  if (pl.total > 0 && !a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", pl.total);
  if (a->workspace_bytes < pl.total)
    return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, pl.total);
  const size_t states = S * D * N * 4;
  const Range outs[] = {{a->dx, T * D * 4}, {a->ddelta, T * D * 4}, {a->dA, D * N * 4}, {a->dB, T * N * 4},
                        {a->dC, T * N * 4}, {a->dD, D * 4},         {a->dh0, states},   {a->workspace, pl.total}};
  const Range ins[] = {rows_of(a->x, a->tokens, a->dim, a->x_stride, es),
                       rows_of(a->delta, a->tokens, a->dim, a->delta_stride, es),
                       rows_of(a->dy, a->tokens, a->dim, a->dy_stride, es),
                       rows_of(a->Bm, a->tokens, a->dstate, a->b_stride, es),
                       rows_of(a->Cm, a->tokens, a->dstate, a->c_stride, es),
                       {a->A, D * N * 4},
                       {a->Dskip, D * 4},
                       {a->offsets, (S + 1) * 4},
                       {a->h0, states},
                       {a->h_saved, kept},
                       {a->dh_last, states}};
  for (int i = 0; i < 8; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
    for (int k = i + 1; k < 8; ++k)
      if (overlap(outs[i], outs[k])) return fail(SSM_ERR_ALIAS, "two outputs overlap");
  }
  return SSM_OK;
}

template <int N, typename InT, int DISC>
ssm_status_t run_bwd(PackedBwdParams p, hipStream_t s) {
  const int64_t DN = p.D * N;
  if (ssm_status_t st = grid_ok(int64_t(p.nc) * p.dtiles, kWave * BwdLayout<N>::NG)) return st;
  if (ssm_status_t st = grid_ok((int64_t(p.q.tokens) * 2 * N + 255) / 256, 256)) return st;
  if (ssm_status_t st = grid_ok((DN + p.D + kWave - 1) / kWave, kWave * std::max<int>(kCarryWaves, kRedWaves))) return st;
  if (p.nc > 1) {
    p.nwg = (p.nc - 1) * p.dtiles;
    bool odd = false;
    if constexpr (!std::is_same<InT, float>::value && N > 1) {
      odd = odd_rows(p.Cm, p.cs);
      if (odd)
        hipLaunchKernelGGL((k_packed_bwd_summary<N, InT, DISC, true>), dim3(uint32_t(p.nwg)), dim3(kWave), 0, s, p);
    }
    if (!odd)
      hipLaunchKernelGGL((k_packed_bwd_summary<N, InT, DISC, false>), dim3(uint32_t(p.nwg)), dim3(kWave), 0, s, p);
    if (ssm_status_t st = launch_status("k_packed_bwd_summary")) return st;
    hipLaunchKernelGGL((k_packed_bwd_carry<N>), dim3(uint32_t((DN + kWave - 1) / kWave)), dim3(kWave * kCarryWaves), 0, s,
                       p);
    if (ssm_status_t st = launch_status("k_packed_bwd_carry")) return st;
  }
  p.nwg = p.nc * p.dtiles;
  hipLaunchKernelGGL((k_packed_bwd<N, InT, DISC>), dim3(uint32_t(p.nwg)), dim3(kWave * BwdLayout<N>::NG), 0, s, p);
  if (ssm_status_t st = launch_status("k_packed_bwd")) return st;
  if (p.q.tokens > 0) {
    const int64_t n = (int64_t(p.q.tokens) * 2 * N + 255) / 256;
    hipLaunchKernelGGL((k_packed_bwd_bc<N>), dim3(uint32_t(n)), dim3(256), 0, s, p);
    if (ssm_status_t st = launch_status("k_packed_bwd_bc")) return st;
  }
  hipLaunchKernelGGL((k_packed_bwd_ad<N>), dim3(uint32_t((DN + p.D + kWave - 1) / kWave)), dim3(kWave * kRedWaves), 0,
                     s, p);
  return launch_status("k_packed_bwd_ad");
}

enum Call { kFwd, kStep, kBwd };

template <Call CALL, int N, typename InT, int DISC, typename Params>
ssm_status_t run(const Params& p, hipStream_t s) {
  if constexpr (CALL == kFwd)
    return run_fwd<N, InT, DISC>(p, s);
  else if constexpr (CALL == kStep)
    return run_step<N, InT, DISC>(p, s);
  else
    return run_bwd<N, InT, DISC>(p, s);
}

template <Call CALL, int N, typename Params>
ssm_status_t run_n(const Params& p, int32_t dtype, int32_t disc, hipStream_t s) {
  if (dtype == SSM_F32)
    return disc == SSM_DISC_ZOH ? run<CALL, N, float, kZoh>(p, s) : run<CALL, N, float, kDeltaB>(p, s);
  return disc == SSM_DISC_ZOH ? run<CALL, N, bf16_t, kZoh>(p, s) : run<CALL, N, bf16_t, kDeltaB>(p, s);
}

template <Call CALL, typename Params>
ssm_status_t dispatch(const Params& p, int64_t N, int32_t dtype, int32_t disc, hipStream_t s) {
  switch (N) {
    case 1: return run_n<CALL, 1>(p, dtype, disc, s);
    case 2: return run_n<CALL, 2>(p, dtype, disc, s);
    case 4: return run_n<CALL, 4>(p, dtype, disc, s);
    case 8: return run_n<CALL, 8>(p, dtype, disc, s);
    default: return run_n<CALL, 16>(p, dtype, disc, s);
  }
}

}  // namespace

extern "C" {

size_t ssm_packed_scan_workspace_size(const ssm_packed_scan_args_t* a) {
  const bool good = check_fwd_sizes(a) == SSM_OK;
  clear_message();
  return good && a->dim > 0 && a->seqs > 0 ? plan_of(a).total : 0;
}

ssm_status_t ssm_packed_scan_fwd(const ssm_packed_scan_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_fwd(a)) return st;
  if (a->dim == 0 || a->seqs == 0 || (a->tokens == 0 && !a->h_last)) return SSM_OK;
  const Plan pl = plan_of(a);
  char* ws = static_cast<char*>(a->workspace);
  PackedParams p{};
  p.x = a->x;
  p.delta = a->delta;
  p.z = a->z;
  p.Bm = a->Bm;
  p.Cm = a->Cm;
  p.A = a->A;
  p.Dskip = a->Dskip;
  p.dt_bias = a->delta_bias;
  p.h0 = a->h0;
  p.h_last = a->h_last;
  p.hsave = a->h_saved;
  p.y = a->y;
  if (pl.nc > 1) {
    p.dsum = reinterpret_cast<float*>(ws);
    p.hsum = reinterpret_cast<float*>(ws + pl.off_hsum);
    if (a->h0 && a->h0 == a->h_last) p.hstart = reinterpret_cast<float*>(ws + pl.off_hstart);
    p.reset = reinterpret_cast<int32_t*>(ws + pl.off_reset);
  }
  p.xs = a->x_stride;
  p.dls = a->delta_stride;
  p.zs = a->z ? a->z_stride : 0;
  p.bs = uint32_t(a->b_stride);
  p.cs = uint32_t(a->c_stride);
  p.D = a->dim;
  p.q = Seqs{a->offsets, a->slot, a->resume, int32_t(a->tokens), int32_t(a->seqs), 0, int32_t(a->slots)};
  p.T = int32_t(pl.T);
  p.nc = pl.wave ? 0 : int32_t(pl.nc);
  p.dtiles = int32_t(pl.dtiles);
  p.exact_thr = exact_threshold(a->disc, a->dtype);
  p.dt_mode = dt_mode_of(a->delta_bias, a->delta_softplus);
  return dispatch<kFwd>(p, a->dstate, a->dtype, a->disc, static_cast<hipStream_t>(hip_stream));
}

ssm_status_t ssm_packed_step(const ssm_packed_step_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_step(a)) return st;
  if (a->dim == 0 || a->batch == 0) return SSM_OK;
  PackedStepParams p{};
  p.x = a->x;
  p.delta = a->delta;
  p.z = a->z;
  p.Bm = a->Bm;
  p.Cm = a->Cm;
  p.A = a->A;
  p.Dskip = a->Dskip;
  p.dt_bias = a->delta_bias;
  p.slot = a->slot;
  p.h = a->h;
  p.y = a->y;
  p.xs = a->x_stride;
  p.dls = a->delta_stride;
  p.zs = a->z ? a->z_stride : 0;
  p.bs = a->b_stride;
  p.cs = a->c_stride;
  p.Bt = a->batch;
  p.slots = a->slots;
  p.D = a->dim;
  p.exact_thr = exact_threshold(a->disc, a->dtype);
  p.dt_mode = dt_mode_of(a->delta_bias, a->delta_softplus);
  return dispatch<kStep>(p, a->dstate, a->dtype, a->disc, static_cast<hipStream_t>(hip_stream));
}

size_t ssm_packed_scan_bwd_workspace_size(const ssm_packed_scan_bwd_args_t* a) {
  const bool good = check_bwd_sizes(a) == SSM_OK;
  clear_message();
  return good ? bwd_plan(a).total : 0;
}

ssm_status_t ssm_packed_scan_bwd(const ssm_packed_scan_bwd_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_bwd(a)) return st;
  if (a->dim == 0) return SSM_OK;
  const BwdPlan pl = bwd_plan(a);
  char* ws = static_cast<char*>(a->workspace);
  PackedBwdParams p{};
  p.x = a->x;
  p.delta = a->delta;
  p.Bm = a->Bm;
  p.Cm = a->Cm;
  p.dy = a->dy;
  p.A = a->A;
  p.Dskip = a->Dskip;
  p.h0 = a->h0;
  p.hsave = a->h_saved;
  p.dh_last = a->dh_last;
  p.dx = a->dx;
  p.ddelta = a->ddelta;
  p.dA = a->dA;
  p.dB = a->dB;
  p.dC = a->dC;
  p.dD = a->dD;
  p.dh0 = a->dh0;
  p.gsum = reinterpret_cast<float*>(ws);
  p.dsum = reinterpret_cast<float*>(ws + pl.off_dsum);
  p.reset = reinterpret_cast<int32_t*>(ws + pl.off_reset);
  p.dAp = reinterpret_cast<float*>(ws + pl.off_dAp);
  p.dDp = reinterpret_cast<float*>(ws + pl.off_dDp);
  p.dBCp = reinterpret_cast<float*>(ws + pl.off_dBCp);
  p.xs = a->x_stride;
  p.dls = a->delta_stride;
  p.bs = uint32_t(a->b_stride);
  p.cs = uint32_t(a->c_stride);
  p.ys = a->dy_stride;
  p.D = a->dim;
  p.q = Seqs{a->offsets, nullptr, nullptr, int32_t(a->tokens), int32_t(a->seqs), 0, int32_t(a->seqs)};
  p.T = int32_t(pl.T);
  p.nc = int32_t(pl.nc);
  p.dtiles = int32_t(pl.dtiles);
  p.exact_thr = exact_threshold(a->disc, a->dtype);
  return dispatch<kBwd>(p, a->dstate, a->dtype, a->disc, static_cast<hipStream_t>(hip_stream));
}

}  // extern "C"
