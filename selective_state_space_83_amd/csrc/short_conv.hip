// short_conv.hip -- host side of the short causal convolution over packed
// sequences: argument checks and launches.  The device code is short_conv.hpp; the
// contract include/ssm_scan.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ssm_scan.h"
#include "ssm_host.hpp"
#include "short_conv.hpp"

namespace {

using namespace ssmh;
using namespace ssmc;

constexpr int64_t kMaxTokens = (int64_t(1) << 31) - 4096;   // tokens are counted in 32 bits
constexpr int64_t kMaxChannels = int64_t(1) << 24;

Range rows_of(const void* p, int64_t rows, int64_t channels, int64_t stride, size_t es) {
  if (!p || rows == 0) return Range{nullptr, 0};
  return Range{p, size_t((rows - 1) * stride + channels) * es};
}

// What all three calls check of their sizes and types.
template <typename Args>
ssm_status_t check_common(const Args* a, int64_t rows, int64_t seqs, int64_t slots) {
  int64_t n;
  if (rows < 0 || seqs < 0 || slots < 0 || a->channels < 0)
    return fail(SSM_ERR_SHAPE, "negative size: tokens=%lld sequences=%lld slots=%lld channels=%lld", (long long)rows,
                (long long)seqs, (long long)slots, (long long)a->channels);
  if (rows > kMaxTokens || seqs > kMaxTokens || slots > kMaxTokens || a->channels > kMaxChannels)
    return fail(SSM_ERR_SHAPE, "problem too large (tokens, sequences and slots are counted in 32 bits, channels in 24)");
  if (!mul_ok(std::max(rows, slots), std::max<int64_t>(a->channels, 1), &n) || n > INT64_MAX / 64 || a->x_stride < 0 ||
      !mul_ok(rows, a->x_stride, &n) || n > INT64_MAX / 16)
    return fail(SSM_ERR_SHAPE, "sizes overflow, or x_stride is negative");
  if (a->dtype != SSM_F32 && a->dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown dtype %d", a->dtype);
  if (a->act != SSM_ACT_NONE && a->act != SSM_ACT_SILU) return fail(SSM_ERR_DTYPE, "unknown act %d", a->act);
  if (a->taps < 1 || a->taps > 4) return fail(SSM_ERR_UNSUPPORTED, "taps %d not in 1..4", a->taps);
  if (a->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  return SSM_OK;
}

template <typename Args>
ssm_status_t check_seqs(const Args* a) {
  int64_t n;
  if (a->offsets) return misaligned(a->offsets, 4) ? fail(SSM_ERR_UNSUPPORTED, "misaligned offsets") : SSM_OK;
  if (a->seqlen < 0 || !mul_ok(a->seqs, a->seqlen, &n) || n != a->tokens)
    return fail(SSM_ERR_SHAPE, "without offsets tokens must be seqs * seqlen");
  return SSM_OK;
}

ssm_status_t check_fwd(const ssm_short_conv_args_t* a) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_common(a, a->tokens, a->seqs, a->slots)) return st;
  if (ssm_status_t st = check_seqs(a)) return st;
  if ((a->slot || a->resume) && !a->state) return fail(SSM_ERR_UNSUPPORTED, "slot and resume go with state only");
  if (a->state && !a->slot && a->slots != a->seqs)
    return fail(SSM_ERR_SHAPE, "without slot, slots must be seqs");
  if (a->channels == 0 || a->seqs == 0) return SSM_OK;
  if (!a->weight || (a->tokens > 0 && (!a->x || !a->y))) return fail(SSM_ERR_NULL, "x, weight and y are required");
  const size_t es = dtype_size(a->dtype);
  if (misaligned(a->x, es) || misaligned(a->y, es) || misaligned(a->weight, 4) || misaligned(a->bias, 4) ||
      misaligned(a->slot, 4) || misaligned(a->state, 4))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const size_t C = size_t(a->channels);
  const Range y{a->y, size_t(a->tokens) * C * es}, state{a->state, size_t(a->slots) * C * size_t(a->taps - 1) * 4};
  const Range ins[] = {rows_of(a->x, a->tokens, a->channels, a->x_stride, es), {a->weight, C * size_t(a->taps) * 4},
                       {a->bias, C * 4}, {a->offsets, size_t(a->seqs + 1) * 4}, {a->slot, size_t(a->seqs) * 4},
                       {a->resume, size_t(a->seqs)}};
  for (const Range& r : ins)
    if (overlap(y, r) || overlap(state, r)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
  if (overlap(y, state)) return fail(SSM_ERR_ALIAS, "y overlaps state");
  return SSM_OK;
}

ssm_status_t check_step(const ssm_short_conv_step_args_t* a) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_common(a, a->batch, a->batch, a->slots)) return st;
  if (!a->slot && a->slots != a->batch) return fail(SSM_ERR_SHAPE, "without slot, slots must be batch");
  if (a->channels == 0 || a->batch == 0) return SSM_OK;
  if (!a->x || !a->weight || !a->y || (a->taps > 1 && !a->state && a->slots > 0))
    return fail(SSM_ERR_NULL, "x, weight, y and (with more than one tap) state are required");
  const size_t es = dtype_size(a->dtype), C = size_t(a->channels);
  if (misaligned(a->x, es) || misaligned(a->y, es) || misaligned(a->weight, 4) || misaligned(a->bias, 4) ||
      misaligned(a->slot, 4) || misaligned(a->state, 4))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const Range y{a->y, size_t(a->batch) * C * es}, state{a->state, size_t(a->slots) * C * size_t(a->taps - 1) * 4};
  const Range ins[] = {rows_of(a->x, a->batch, a->channels, a->x_stride, es), {a->weight, C * size_t(a->taps) * 4},
                       {a->bias, C * 4}, {a->slot, size_t(a->batch) * 4}};
  for (const Range& r : ins)
    if (overlap(y, r) || overlap(state, r)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
  if (overlap(y, state)) return fail(SSM_ERR_ALIAS, "y overlaps state");
  return SSM_OK;
}

// A lane's channels.  (8 bf16 channels, 16 bytes, take twice the registers: 32768 x 2560
// 84 us for 78.)
constexpr int V = 4;

// Rows that all start on V elements.
bool row_wide(const void* p, int64_t stride, size_t es) { return !misaligned(p, V * es) && stride % V == 0; }

// Tokens per tile: short enough that the tiles fill the GPU with `waves` waves, at
// least 8 (a tile reads up to three rows more than its own).  The forward pass takes 16 at
// most (32768 x 2560 bf16 77 us, 78 with 32, 79 with 64; fp32 141, 142, 147; 4000 x 1027
// bf16, an element at a time, 14, 19, 19), the gradients 64 (16384 x 2560 bf16 after a
// forward pass 117 us, 126 with 32).
int32_t tile_len(int64_t tokens, int64_t cgroups, int64_t waves, int64_t most) {
  int64_t t = most;
  while (t > 8 && (tokens + t - 1) / t * cgroups < waves) t /= 2;
  return int32_t(t);
}

int64_t channel_groups(int64_t C, int64_t v) { return (C + 64 * v - 1) / (64 * v); }

template <typename Args>
Seqs sequences(const Args* a) {
  Seqs q{};
  q.offsets = a->offsets;
  q.tokens = int32_t(a->tokens);
  q.S = int32_t(a->seqs);
  q.seqlen = int32_t(a->offsets ? 0 : a->seqlen);
  return q;
}

ssm_status_t set_tiles(ConvParams* p, int64_t v, int32_t tile, uint32_t* grid) {
  p->tile = tile;
  p->cgroups = int32_t(channel_groups(p->C, v));
  p->tiles = int32_t(std::max<int64_t>(1, (int64_t(p->q.tokens) + tile - 1) / tile));
  const int64_t n = (int64_t(p->tiles) * p->cgroups + 3) / 4;
  if (n > int64_t(UINT32_MAX) / 256) return fail(SSM_ERR_SHAPE, "problem too large for one launch");
  *grid = uint32_t(n);
  return SSM_OK;
}

template <typename T, int W, int K>
ssm_status_t launch_fwd(ConvParams p, hipStream_t s) {
  uint32_t grid;
  if (ssm_status_t st = set_tiles(&p, W, tile_len(p.q.tokens, channel_groups(p.C, W), 2048, 16), &grid)) return st;
  hipLaunchKernelGGL((k_short_conv<T, W, K>), dim3(grid), dim3(256), 0, s, p);
  return launch_status("k_short_conv");
}

template <typename T, int W, int K>
ssm_status_t launch_step(const ConvParams& p, hipStream_t s) {
  const int64_t rows = (p.q.S + kStepRows - 1) / kStepRows, y = std::min<int64_t>(rows, 32768);
  const dim3 grid(uint32_t((p.C + 256 * W - 1) / (256 * W)), uint32_t(y));
  hipLaunchKernelGGL((k_short_conv_step<T, W, K>), grid, dim3(256), 0, s, p);
  return launch_status("k_short_conv_step");
}

template <typename T, int W, int K>
ssm_status_t launch_bwd(ConvParams p, int32_t tile, hipStream_t s) {
  uint32_t grid;
  if (ssm_status_t st = set_tiles(&p, W, tile, &grid)) return st;
  hipLaunchKernelGGL((k_short_conv_bwd<T, W, K>), dim3(grid), dim3(256), 0, s, p);
  return launch_status("k_short_conv_bwd");
}

// One instance for each type, width and number of taps.
#define SSM_CONV_CASES(RUN, ...)                                                         \
  switch (taps) {                                                                        \
    case 1: return vec ? RUN<T, V, 1>(__VA_ARGS__) : RUN<T, 1, 1>(__VA_ARGS__);          \
    case 2: return vec ? RUN<T, V, 2>(__VA_ARGS__) : RUN<T, 1, 2>(__VA_ARGS__);          \
    case 3: return vec ? RUN<T, V, 3>(__VA_ARGS__) : RUN<T, 1, 3>(__VA_ARGS__);          \
    default: return vec ? RUN<T, V, 4>(__VA_ARGS__) : RUN<T, 1, 4>(__VA_ARGS__);         \
  }

template <typename T>
ssm_status_t run_fwd(const ConvParams& p, int taps, bool vec, hipStream_t s) {
  SSM_CONV_CASES(launch_fwd, p, s)
}
template <typename T>
ssm_status_t run_step(const ConvParams& p, int taps, bool vec, hipStream_t s) {
  SSM_CONV_CASES(launch_step, p, s)
}
template <typename T>
ssm_status_t run_bwd(const ConvParams& p, int taps, bool vec, int32_t tile, hipStream_t s) {
  SSM_CONV_CASES(launch_bwd, p, tile, s)
}
#undef SSM_CONV_CASES

// Tokens per tile of the backward pass: the tiles' sums for dweight and dbias are
// written once a tile.  By sizes alone, as the workspace is.
int32_t bwd_tile(const ssm_short_conv_bwd_args_t* a) {
  return tile_len(a->tokens, channel_groups(a->channels, V), 1536, 64);
}

size_t bwd_workspace(const ssm_short_conv_bwd_args_t* a) {
  if ((!a->dweight && !a->dbias) || a->tokens * a->channels == 0) return 0;
  const int64_t tile = bwd_tile(a), tiles = (a->tokens + tile - 1) / tile;
  return align256(size_t(tiles) * size_t(a->channels) * size_t(a->taps + 1) * 4);
}

ssm_status_t check_bwd_sizes(const ssm_short_conv_bwd_args_t* a) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_common(a, a->tokens, a->seqs, 0)) return st;
  int64_t n;
  if (a->dy_stride < 0 || !mul_ok(a->tokens, a->dy_stride, &n) || n > INT64_MAX / 16)
    return fail(SSM_ERR_SHAPE, "dy_stride is negative or overflows");
  return check_seqs(a);
}

ssm_status_t check_bwd(const ssm_short_conv_bwd_args_t* a) {
  if (ssm_status_t st = check_bwd_sizes(a)) return st;
  if (misaligned(a->dweight, 4) || misaligned(a->dbias, 4))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const size_t C = size_t(a->channels), es = dtype_size(a->dtype);
  const Range dw{a->dweight, C * size_t(a->taps) * 4}, db{a->dbias, C * 4};
  if (overlap(dw, db)) return fail(SSM_ERR_ALIAS, "two gradients overlap");
  if (a->tokens * a->channels == 0) return SSM_OK;
  if (!a->x || !a->weight || !a->dy || !a->dx) return fail(SSM_ERR_NULL, "x, weight, dy and dx are required");
  const size_t need = bwd_workspace(a);
  if (misaligned(a->x, es) || misaligned(a->dy, es) || misaligned(a->dx, es) || misaligned(a->weight, 4) ||
      misaligned(a->bias, 4) || misaligned(a->workspace, 256))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment; workspace 256 bytes)");
  if (need > 0 && !a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
  if (a->workspace_bytes < need)
    return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, need);
  const Range outs[] = {{a->dx, size_t(a->tokens) * C * es}, dw, db, {a->workspace, need}};
  const Range ins[] = {rows_of(a->x, a->tokens, a->channels, a->x_stride, es),
                       rows_of(a->dy, a->tokens, a->channels, a->dy_stride, es), {a->weight, C * size_t(a->taps) * 4},
                       {a->bias, C * 4}, {a->offsets, size_t(a->seqs + 1) * 4}};
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
    for (int k = i + 1; k < 4; ++k)
      if (overlap(outs[i], outs[k])) return fail(SSM_ERR_ALIAS, "two outputs overlap");
  }
  return SSM_OK;
}

template <typename Args>
ConvParams params(const Args* a) {
  ConvParams p{};
  p.x = a->x;
  p.w = a->weight;
  p.b = a->bias;
  p.C = a->channels;
  p.xs = a->x_stride;
  p.silu = a->act == SSM_ACT_SILU;
  return p;
}

}  // namespace

extern "C" {

ssm_status_t ssm_short_conv_fwd(const ssm_short_conv_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_fwd(a)) return st;
  if (a->channels == 0 || a->seqs == 0 || (a->tokens == 0 && !a->state)) return SSM_OK;
  ConvParams p = params(a);
  p.q = sequences(a);
  p.q.slot = a->slot;
  p.q.resume = a->resume;
  p.q.slots = int32_t(a->slots);
  p.state = a->taps > 1 ? a->state : nullptr;
  p.y = a->y;
  const size_t es = dtype_size(a->dtype);
  const bool vec = a->channels % V == 0 && row_wide(a->x, a->x_stride, es) && !misaligned(a->y, V * es) &&
                   !misaligned(a->weight, 16) && !misaligned(a->bias, 16) && !misaligned(a->state, 16);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return a->dtype == SSM_F32 ? run_fwd<float>(p, a->taps, vec, s) : run_fwd<bf16_t>(p, a->taps, vec, s);
}

ssm_status_t ssm_short_conv_step(const ssm_short_conv_step_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_step(a)) return st;
  if (a->channels == 0 || a->batch == 0) return SSM_OK;
  ConvParams p = params(a);
  p.q.slot = a->slot;
  p.q.S = int32_t(a->batch);
  p.q.slots = int32_t(a->slots);
  p.state = a->state;
  p.y = a->y;
  const size_t es = dtype_size(a->dtype);
  const bool vec = a->channels % V == 0 && row_wide(a->x, a->x_stride, es) && !misaligned(a->y, V * es) &&
                   !misaligned(a->weight, 16) && !misaligned(a->bias, 16) && !misaligned(a->state, 16);
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return a->dtype == SSM_F32 ? run_step<float>(p, a->taps, vec, s) : run_step<bf16_t>(p, a->taps, vec, s);
}

size_t ssm_short_conv_bwd_workspace_size(const ssm_short_conv_bwd_args_t* a) {
  if (!a) return 0;
  if (a->tokens < 0 || a->channels < 0 || a->tokens > kMaxTokens || a->channels > kMaxChannels || a->taps < 1 || a->taps > 4)
    return 0;
  int64_t n;
  return mul_ok(a->tokens, a->channels, &n) && n <= INT64_MAX / 64 ? bwd_workspace(a) : 0;
}

ssm_status_t ssm_short_conv_bwd(const ssm_short_conv_bwd_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_bwd(a)) return st;
  if (a->channels == 0) return SSM_OK;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  int64_t tiles = 0;
  if (a->tokens > 0) {
    ConvParams p = params(a);
    p.q = sequences(a);
    p.dy = a->dy;
    p.ds = a->dy_stride;
    p.y = a->dx;
    p.part = a->dweight || a->dbias ? static_cast<float*>(a->workspace) : nullptr;
    const size_t es = dtype_size(a->dtype);
    const bool vec = a->channels % V == 0 && row_wide(a->x, a->x_stride, es) && row_wide(a->dy, a->dy_stride, es) &&
                     !misaligned(a->dx, V * es) && !misaligned(a->weight, 16) && !misaligned(a->bias, 16);
    const int32_t tile = bwd_tile(a);
    tiles = (a->tokens + tile - 1) / tile;
    if (ssm_status_t st = a->dtype == SSM_F32 ? run_bwd<float>(p, a->taps, vec, tile, s)
                                              : run_bwd<bf16_t>(p, a->taps, vec, tile, s))
      return st;
  }
  if (!a->dweight && !a->dbias) return SSM_OK;
  const ConvSumParams c{static_cast<const float*>(a->workspace), a->dweight, a->dbias, tiles, a->channels, a->taps};
  const int64_t cols = a->channels * (a->taps + 1);
  hipLaunchKernelGGL(k_conv_sums, dim3(uint32_t((cols + 15) / 16)), dim3(256), 0, s, c);
  return launch_status("k_conv_sums");
}

}  // extern "C"
