// decay_attn.hip -- host side of decay attention: argument checks, plans and
// launches.  The device code is decay_attn.hpp; the contract include/ssm_scan.h.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "ssm_scan.h"
#include "ssm_host.hpp"
#include "decay_attn.hpp"

namespace {

using namespace ssmh;
using namespace ssma;

constexpr int64_t kMaxDim = 256;
// A launch holds at most 2^32 - 1 lanes; workgroups have up to 512.
constexpr int64_t kMaxGroups = int64_t(UINT32_MAX) / 512;
constexpr int64_t kSpanAlign = 64;

// Sizes common to the three calls; `tokens` is batch * seqlen.
struct Sizes {
  int64_t B, L, H, Hk, dk, dv;
  int64_t tokens, state;   // state: batch * heads * dk * dv
};

ssm_status_t check_sizes(Sizes* z) {
  if (z->B < 0 || z->L < 0 || z->H < 0 || z->Hk < 0)
    return fail(SSM_ERR_SHAPE, "negative size: batch=%lld seqlen=%lld heads=%lld key_heads=%lld",
                (long long)z->B, (long long)z->L, (long long)z->H, (long long)z->Hk);
  if (z->dk < 1 || z->dv < 1)
    return fail(SSM_ERR_SHAPE, "key_dim and value_dim must be >= 1 (got %lld, %lld)",
                (long long)z->dk, (long long)z->dv);
  if (z->dk > kMaxDim || z->dv > kMaxDim)
    return fail(SSM_ERR_UNSUPPORTED, "key_dim %lld and value_dim %lld must be <= %lld",
                (long long)z->dk, (long long)z->dv, (long long)kMaxDim);
  if (z->H > 0 && (z->Hk < 1 || z->H % z->Hk != 0))
    return fail(SSM_ERR_SHAPE, "heads %lld is not a multiple of key_heads %lld", (long long)z->H,
                (long long)z->Hk);
  // the largest arrays: per token and value head up to kMaxDim fp32 values
  int64_t bh, n;
  if (!mul_ok(z->B, z->L, &z->tokens) || !mul_ok(z->B, z->H, &bh) ||
      !mul_ok(bh, z->dk * z->dv, &z->state) || !mul_ok(z->tokens, z->H, &n) ||
      !mul_ok(n, kMaxDim, &n) || n > INT64_MAX / 64 || z->state > INT64_MAX / 64)
    return fail(SSM_ERR_SHAPE, "sizes overflow");
  if (bh > kMaxGrid) return fail(SSM_ERR_SHAPE, "problem too large for one launch");
  return SSM_OK;
}

ssm_status_t check_dtypes(int32_t dtype, int32_t decay_dtype) {
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown dtype %d", dtype);
  if (decay_dtype != SSM_F32 && decay_dtype != SSM_BF16)
    return fail(SSM_ERR_DTYPE, "unknown decay_dtype %d", decay_dtype);
  return SSM_OK;
}

// The bytes from p on that a strided array of `rank` outer dimensions spans.
bool extent(const void* p, const int64_t* size, const int64_t* stride, int rank, int64_t inner,
            size_t elem, Range* r) {
  int64_t last = inner - 1;
  bool empty = false;
  for (int i = 0; i < rank; ++i) {
    int64_t n;
    if (stride[i] < 0) return false;
    if (size[i] == 0) empty = true;
    if (size[i] > 0 && (!mul_ok(size[i] - 1, stride[i], &n) || last > INT64_MAX / 16 - n)) return false;
    if (size[i] > 0) last += n;
  }
  if (last > INT64_MAX / 16) return false;
  *r = Range{p, empty ? 0 : size_t(last + 1) * elem};
  return true;
}

ssm_status_t check_rows(const char* name, const void* p, const int64_t* size, const int64_t* stride,
                        int rank, int64_t inner, int32_t dtype, Range* r) {
  if (!extent(p, size, stride, rank, inner, dtype_size(dtype), r))
    return fail(SSM_ERR_SHAPE, "%s has a negative or overflowing stride", name);
  if (misaligned(p, dtype_size(dtype))) return fail(SSM_ERR_UNSUPPORTED, "misaligned %s", name);
  return SSM_OK;
}

struct Named {
  const char* name;
  Range r;
};

ssm_status_t check_alias(const Named* outs, int nout, const Named* ins, int nin) {
  for (int i = 0; i < nout; ++i) {
    for (int k = 0; k < nin; ++k)
      if (overlap(outs[i].r, ins[k].r))
        return fail(SSM_ERR_ALIAS, "%s overlaps %s", outs[i].name, ins[k].name);
    for (int k = i + 1; k < nout; ++k)
      if (overlap(outs[i].r, outs[k].r))
        return fail(SSM_ERR_ALIAS, "%s overlaps %s", outs[i].name, outs[k].name);
  }
  return SSM_OK;
}

ssm_status_t check_step(const ssm_decay_attn_step_args_t* a, Sizes* z) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  *z = Sizes{a->batch, 1, a->heads, a->key_heads, a->key_dim, a->value_dim, 0, 0};
  if (ssm_status_t st = check_sizes(z)) return st;
  if (ssm_status_t st = check_dtypes(a->dtype, a->decay_dtype)) return st;
  if (z->B * z->H == 0) return SSM_OK;
  if (!a->q || !a->k || !a->v || !a->log_decay || !a->h || !a->o)
    return fail(SSM_ERR_NULL, "q, k, v, log_decay, h and o are required");
  if (misaligned(a->h, 4) || misaligned(a->o, dtype_size(a->dtype)))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const int64_t kn[] = {z->B, z->Hk}, vn[] = {z->B, z->H};
  Range q, k, v, g;
  if (ssm_status_t st = check_rows("q", a->q, kn, a->q_stride, 2, z->dk, a->dtype, &q)) return st;
  if (ssm_status_t st = check_rows("k", a->k, kn, a->k_stride, 2, z->dk, a->dtype, &k)) return st;
  if (ssm_status_t st = check_rows("v", a->v, vn, a->v_stride, 2, z->dv, a->dtype, &v)) return st;
  if (ssm_status_t st = check_rows("log_decay", a->log_decay, vn, a->decay_stride, 2, 1, a->decay_dtype, &g))
    return st;
  const Named outs[] = {{"o", {a->o, size_t(z->B * z->H * z->dv) * dtype_size(a->dtype)}},
                        {"h", {a->h, size_t(z->state) * 4}}};
  const Named ins[] = {{"q", q}, {"k", k}, {"v", v}, {"log_decay", g}};
  return check_alias(outs, 2, ins, 4);
}

// Columns a workgroup takes, 16 for each of its 4 or 8 waves.
int64_t tile_width(int64_t N) { return N > 64 ? 128 : 64; }
int64_t tiles_of(int64_t N) { return (N + tile_width(N) - 1) / tile_width(N); }

// Tokens of a chunk.  fp32 takes 32: its products are the bound, and those of the
// scores grow with the chunk.
constexpr int chunk_tokens(int32_t dtype) { return dtype == SSM_BF16 ? 64 : 32; }

// How the time axis is cut: `spans` spans of `span` tokens (a multiple of
// kSpanAlign), each walked by workgroups of its own.
struct Cut {
  int64_t span = kSpanAlign, spans = 1;
};

int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// The plan's cut, the cheapest by this count.  `walkers` workgroups walk a span
// of n chunks in n + 1 steps (one to fill).  m workgroups on a CU take 1 + slope
// (m - 1) times as long as one: slope 0.7 for those of eight waves, 0.6 for those
// of four (2048 tokens, us for 1, 2, 4 on a CU of 128 x 128 bf16: 163, 278, 540;
// 1, 2, 3 of 64 x 64 fp32: 201, 320, 424).  More than one span costs the first
// pass over all but the last (`state`, its share of a step), two launches (two
// steps), and reading and writing the spans' states (32 MB a step); the backward's
// three passes share two such first passes and joins (two thirds of a pass's).
// The shares are counted from the chunk's products and bytes, one for both types.
// Measured, us by number of spans, the plan's marked: 80 walkers of 128 chunks,
// 128 x 128 bf16: 3 298, *6 246, 12 285, 24 325; 4 walkers of 2048 chunks: 64
// 223, *128 192, 256 231; 320 walkers of 32 chunks: *1 214, 2 259, 3 265; 192
// walkers of 32 chunks, 64 x 64 fp32: 1 181, 3 170, *4 143, 8 151; bf16 85, 74,
// *67, 77.  Backward, all its launches: 80 walkers of 64 chunks, 128 x 128 bf16: 1
// 1322, 3 723, 4 856, 5 795, *6 728, 11 832, 16 834; 320 walkers of 32 chunks: 1
// 1372, 2 1298, 3 1310, *4 1325, 8 1542; 8 walkers of 256 chunks, 64 x 64: 8 431, 32
// 169, *64 149; 96 walkers of 16 chunks, 64 x 64 fp32: 1 373, 2 276, 4 227, *8 189,
// 16 215; 192 walkers of 32 chunks: 1 822, 3 706, *4 624, 8 661, 16 687.
Cut cut_time(int64_t L, int64_t walkers, int64_t inner, double slope, double state, double join, int32_t span) {
  constexpr int64_t kCus = 256, kMaxSpans = 1024;
  Cut c;
  if (L == 0 || walkers == 0) return c;
  const int64_t chunks = (L + kSpanAlign - 1) / kSpanAlign;
  int64_t best = chunks;   // chunks of a span
  if (span > 0) {
    best = std::min<int64_t>(span / kSpanAlign, chunks);
  } else {
    const int64_t most = std::min({chunks, kMaxSpans, 1 + 8 * kCus / walkers});
    double least = 0.0;
    auto step = [&](int64_t groups) { return 1.0 + slope * double((groups - 1) / kCus); };
    for (int64_t want = 1; want <= most; ++want) {
      const int64_t per = (chunks + want - 1) / want, n = (chunks + per - 1) / per;
      if (n != want) continue;
      double cost = double(per + 1) * step(walkers * n);
      if (n > 1)
        cost += state * double(per + 1) * step(walkers * (n - 1)) +
                join * (2.0 + double(n * walkers) * double(inner) / 1.6e6);
      if (want == 1 || cost < least) {
        least = cost;
        best = per;
      }
    }
  }
  c.span = best * kSpanAlign;
  c.spans = (chunks + best - 1) / best;
  return c;
}

// Workspace of the forward pass: the states entering the spans and their decays.
struct FwdPlan {
  Cut cut;
  size_t off_total = 0, total = 0;
};

FwdPlan make_fwd_plan(const Sizes& z, int32_t span) {
  FwdPlan pl;
  pl.cut = cut_time(z.L, z.B * z.H * tiles_of(z.dv), z.dk * z.dv, tile_width(z.dv) == 128 ? 0.7 : 0.6, 0.35, 1.0,
                    span);
  if (pl.cut.spans > 1) {
    pl.off_total = align256(size_t(z.state) * size_t(pl.cut.spans) * 4);
    pl.total = pl.off_total + align256(size_t(z.B * z.H) * size_t(pl.cut.spans) * 4);
  }
  return pl;
}

// Workspace of the backward pass.
struct BwdPlan {
  Cut cut;
  int64_t slices = 0, tiles = 0;   // of 16 columns of key_dim, whose dots are kept apart, and of 16 rows of value_dim
  size_t off_carry = 0, off_rcarry = 0, off_total = 0, off_u = 0, off_w = 0, off_kept = 0, off_flow = 0, off_heads = 0,
         total = 0;
};

BwdPlan make_bwd_plan(const Sizes& z, int32_t span, int32_t dtype) {
  BwdPlan pl;
  if (z.tokens == 0 || z.H == 0) return pl;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += align256(bytes);
    return o;
  };
  pl.cut = cut_time(z.L, z.B * z.H * tiles_of(z.dk), z.dk * z.dv, tile_width(z.dk) == 128 ? 0.7 : 0.6, 0.35 * 2 / 3,
                    2.0 / 3, span);
  pl.slices = (z.dk + 15) / 16;
  pl.tiles = round_up(z.dv, 32) / 16;
  const int64_t chunks = pl.cut.span * pl.cut.spans / chunk_tokens(dtype);
  const size_t th = size_t(z.tokens) * size_t(z.H);
  const size_t dots = size_t(z.B * z.H) * size_t(pl.cut.span * pl.cut.spans) *
                      size_t(tile_width(z.dk) / 16 * tiles_of(z.dk)) * 4;
  const size_t spans = pl.cut.spans > 1 ? size_t(pl.cut.spans) : 0;
  pl.off_carry = take(size_t(z.state) * spans * 4);
  pl.off_rcarry = take(size_t(z.state) * spans * 4);
  pl.off_total = take(size_t(z.B * z.H) * spans * 4);
  pl.off_u = take(dots);
  pl.off_w = take(dots);
  pl.off_kept = take(size_t(z.B * z.H) * size_t(chunks) * size_t(pl.slices * pl.tiles) * 1024);
  pl.off_flow = take(size_t(z.B * z.H) * size_t(chunks) * size_t(pl.slices) * 4);
  const bool shared = z.H != z.Hk;
  pl.off_heads = take(shared ? th * size_t(z.dk) * 4 : 0);
  pl.total = off;
  return pl;
}

// Launches of a plan stay within one grid: workgroups of 512 lanes, two for a
// head's span at most, and with spans to join a lane for an element of a state.
ssm_status_t check_grid(const Sizes& z, const Cut& c) {
  int64_t n, m;
  if (!mul_ok(z.B * z.H * 4, c.spans, &n) || n > kMaxGroups || !mul_ok(z.state, c.spans, &m) ||
      m > INT64_MAX / 16 || (c.spans > 1 && z.B * z.H * round_up(z.dk * z.dv, 256) > int64_t(UINT32_MAX)))
    return fail(SSM_ERR_SHAPE, "problem too large for one launch");
  return SSM_OK;
}

ssm_status_t check_fwd(const ssm_decay_attn_args_t* a, Sizes* z, FwdPlan* pl) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  *z = Sizes{a->batch, a->seqlen, a->heads, a->key_heads, a->key_dim, a->value_dim, 0, 0};
  if (ssm_status_t st = check_sizes(z)) return st;
  if (ssm_status_t st = check_dtypes(a->dtype, a->decay_dtype)) return st;
  if (a->span < 0 || a->span % kSpanAlign != 0)
    return fail(SSM_ERR_UNSUPPORTED, "span must be a non-negative multiple of %lld", (long long)kSpanAlign);
  if (a->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved field must be 0");
  *pl = make_fwd_plan(*z, a->span);
  if (ssm_status_t st = check_grid(*z, pl->cut)) return st;
  if (z->B * z->H == 0) return SSM_OK;
  if (z->L > 0 && (!a->q || !a->k || !a->v || !a->log_decay || !a->o))
    return fail(SSM_ERR_NULL, "q, k, v, log_decay and o are required");
  if (misaligned(a->lengths, 4) || misaligned(a->h0, 4) || misaligned(a->h_last, 4) ||
      misaligned(a->o, dtype_size(a->dtype)) || misaligned(a->workspace, 256))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment; workspace 256 bytes)");
  const int64_t kn[] = {z->B, z->L, z->Hk}, vn[] = {z->B, z->L, z->H};
  Range q, k, v, g;
  if (ssm_status_t st = check_rows("q", a->q, kn, a->q_stride, 3, z->dk, a->dtype, &q)) return st;
  if (ssm_status_t st = check_rows("k", a->k, kn, a->k_stride, 3, z->dk, a->dtype, &k)) return st;
  if (ssm_status_t st = check_rows("v", a->v, vn, a->v_stride, 3, z->dv, a->dtype, &v)) return st;
  if (ssm_status_t st = check_rows("log_decay", a->log_decay, vn, a->decay_stride, 3, 1, a->decay_dtype, &g))
    return st;
  const size_t state = size_t(z->state) * 4;
  const Named outs[] = {
      {"o", {a->o, size_t(z->tokens) * size_t(z->H * z->dv) * dtype_size(a->dtype)}},
      {"h_last", {a->h_last, state}},
      {"workspace", {a->workspace, pl->total}}};
  const Named ins[] = {{"q", q}, {"k", k}, {"v", v}, {"log_decay", g}, {"h0", {a->h0, state}},
                       {"lengths", {a->lengths, size_t(z->B) * 4}}};
  if (pl->total > 0) {
    if (!a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", pl->total);
    if (a->workspace_bytes < pl->total)
      return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes,
                  pl->total);
  }
  return check_alias(outs, 3, ins, 6);
}

ssm_status_t check_bwd(const ssm_decay_attn_bwd_args_t* a, Sizes* z, BwdPlan* pl) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  *z = Sizes{a->batch, a->seqlen, a->heads, a->key_heads, a->key_dim, a->value_dim, 0, 0};
  if (ssm_status_t st = check_sizes(z)) return st;
  if (ssm_status_t st = check_dtypes(a->dtype, a->decay_dtype)) return st;
  if (a->span < 0 || a->span % kSpanAlign != 0)
    return fail(SSM_ERR_UNSUPPORTED, "span must be a non-negative multiple of %lld", (long long)kSpanAlign);
  if (a->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved field must be 0");
  *pl = make_bwd_plan(*z, a->span, a->dtype);
  if (ssm_status_t st = check_grid(*z, pl->cut)) return st;
  if (z->B * z->H == 0) return SSM_OK;
  if (z->L > 0 && (!a->q || !a->k || !a->v || !a->log_decay || !a->dout || !a->dq || !a->dk ||
                   !a->dv || !a->dlog_decay))
    return fail(SSM_ERR_NULL, "q, k, v, log_decay, dout, dq, dk, dv and dlog_decay are required");
  const size_t es = dtype_size(a->dtype), gs = dtype_size(a->decay_dtype);
  if (misaligned(a->lengths, 4) || misaligned(a->h0, 4) || misaligned(a->dh_last, 4) ||
      misaligned(a->dh0, 4) || misaligned(a->dq, es) || misaligned(a->dk, es) ||
      misaligned(a->dv, es) || misaligned(a->dlog_decay, gs) || misaligned(a->workspace, 256))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment; workspace 256 bytes)");
  const int64_t kn[] = {z->B, z->L, z->Hk}, vn[] = {z->B, z->L, z->H};
  Range q, k, v, g, d;
  if (ssm_status_t st = check_rows("q", a->q, kn, a->q_stride, 3, z->dk, a->dtype, &q)) return st;
  if (ssm_status_t st = check_rows("k", a->k, kn, a->k_stride, 3, z->dk, a->dtype, &k)) return st;
  if (ssm_status_t st = check_rows("v", a->v, vn, a->v_stride, 3, z->dv, a->dtype, &v)) return st;
  if (ssm_status_t st = check_rows("log_decay", a->log_decay, vn, a->decay_stride, 3, 1, a->decay_dtype, &g))
    return st;
  if (ssm_status_t st = check_rows("dout", a->dout, vn, a->dout_stride, 3, z->dv, a->dtype, &d)) return st;
  const size_t state = size_t(z->state) * 4, tok = size_t(z->tokens);
  const Named ins[] = {{"q", q}, {"k", k}, {"v", v}, {"log_decay", g}, {"dout", d},
                       {"h0", {a->h0, state}}, {"dh_last", {a->dh_last, state}},
                       {"lengths", {a->lengths, size_t(z->B) * 4}}};
  const Named outs[] = {{"dq", {a->dq, tok * size_t(z->Hk * z->dk) * es}},
                        {"dk", {a->dk, tok * size_t(z->Hk * z->dk) * es}},
                        {"dv", {a->dv, tok * size_t(z->H * z->dv) * es}},
                        {"dlog_decay", {a->dlog_decay, tok * size_t(z->H) * gs}},
                        {"dh0", {a->dh0, state}},
                        {"workspace", {a->workspace, pl->total}}};
  if (pl->total > 0) {
    if (!a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", pl->total);
    if (a->workspace_bytes < pl->total)
      return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes,
                  pl->total);
  }
  return check_alias(outs, 6, ins, 8);
}

// ---------------------------------------------------------------------------
// launches
// ---------------------------------------------------------------------------

// Whether rows can be read through windows (Stage in decay_attn.hpp): they
// start on 16 bytes, hold whole 16 bytes, do not overlap, and 64 of them lie
// within 2^31 bytes.
bool fast_rows(const Rows& r, int64_t n, size_t elem) {
  const int64_t k = int64_t(16 / elem);
  return !misaligned(r.p, 16) && n % k == 0 && r.sb % k == 0 && r.st % k == 0 && r.sh % k == 0 && r.st >= n &&
         r.st < (int64_t(1) << 31) / 64 / int64_t(elem);
}

template <typename T, int MP, int W, int SP, typename OutT, Part PART, bool REV, bool FAST>
ssm_status_t launch_mix(const MixParams& p, hipStream_t s) {
  constexpr int CT = chunk_tokens(sizeof(T) == 2 ? SSM_BF16 : SSM_F32);
  hipLaunchKernelGGL((k_mix<T, MP, W, CT, sizeof(T) == 2 ? SP : 1, OutT, PART, REV, FAST>),
                     dim3(uint32_t(p.B * p.H * p.tiles * p.walked)), dim3(64 * W), 0, s, p);
  return launch_status("k_mix");
}

template <typename T, int MP, int SP, typename OutT, Part PART, bool REV, bool FAST>
ssm_status_t tile_mix(const MixParams& p, hipStream_t s) {
  return tile_width(p.N) == 128 ? launch_mix<T, MP, 8, SP, OutT, PART, REV, FAST>(p, s)
                                : launch_mix<T, MP, 4, SP, OutT, PART, REV, FAST>(p, s);
}

template <typename T, int SP, typename OutT, Part PART, bool REV, bool FAST>
ssm_status_t size_mix(const MixParams& p, hipStream_t s) {
  if (p.M <= 32) return tile_mix<T, 32, SP, OutT, PART, REV, FAST>(p, s);
  if (p.M <= 64) return tile_mix<T, 64, SP, OutT, PART, REV, FAST>(p, s);
  if (p.M <= 128) return tile_mix<T, 128, SP, OutT, PART, REV, FAST>(p, s);
  return tile_mix<T, 256, SP, OutT, PART, REV, FAST>(p, s);
}

template <typename T, int SP, typename OutT, Part PART, bool REV>
ssm_status_t run_mix(MixParams p, hipStream_t s) {
  const size_t e = sizeof(T);
  const int64_t k = int64_t(16 / sizeof(OutT));
  p.tiles = int32_t(tiles_of(p.N));
  p.walked = PART == kState ? p.spans - 1 : p.spans;
  bool fast = fast_rows(p.b, p.M, e) && fast_rows(p.c, p.N, e) && p.g.st < (int64_t(1) << 31) / 64 / 4;
  if (PART != kState)
    fast = fast && fast_rows(p.a, p.M, e) && !misaligned(p.out, 16) && p.N % k == 0 &&
           p.H * p.N < (int64_t(1) << 31) / 64 / int64_t(sizeof(OutT));
  if (PART == kOutDots) fast = fast && fast_rows(p.x, p.N, e);
  return fast ? size_mix<T, SP, OutT, PART, REV, true>(p, s) : size_mix<T, SP, OutT, PART, REV, false>(p, s);
}

// The states entering the spans of p (which has its b, c, s0 and span set): the
// state pass into `carry`, then the join.
template <typename T, bool REV>
ssm_status_t run_carries(MixParams p, float* carry, float* total, hipStream_t s) {
  p.sum = carry;
  p.total = total;
  p.dots = nullptr;
  p.out = nullptr;
  p.s_last = nullptr;
  if (ssm_status_t st = run_mix<T, 1, T, kState, REV>(p, s)) return st;
  const JoinParams j{carry, total, p.s0, p.sm, p.sn, p.M * p.N, p.N, p.spans};
  // four elements to a lane where that leaves enough lanes; few heads with many
  // spans want the lanes, and the reads in flight (4 heads of 128 x 128, 128
  // spans: 29 us with 8, 17 with 32; 96 heads of 64 x 64, 8 spans: 13 us with 32)
  const int64_t heads = p.B * p.H;
  const dim3 ones(uint32_t(heads * ((j.inner + 255) / 256)));
  if (j.inner % 4 == 0 && heads * j.inner >= int64_t(1) << 19)
    hipLaunchKernelGGL((k_join_spans<4, 8>), dim3(uint32_t(heads * ((j.inner + 1023) / 1024))), dim3(256), 0, s, j);
  else if (p.spans <= 16)
    hipLaunchKernelGGL((k_join_spans<1, 8>), ones, dim3(256), 0, s, j);
  else
    hipLaunchKernelGGL((k_join_spans<1, 32>), ones, dim3(256), 0, s, j);
  return launch_status("k_join_spans");
}

ssm_status_t copy_state(float* dst, const float* src, int64_t n, hipStream_t s) {
  if (!dst || n == 0) return SSM_OK;
  const uint32_t groups = uint32_t(std::min<int64_t>((n + 255) / 256, 1 << 20));
  hipLaunchKernelGGL(k_attn_state_copy, dim3(groups), dim3(256), 0, s, dst, src, n);
  return launch_status("k_attn_state_copy");
}

Rows rows(const void* p, const int64_t* st, int64_t per) {
  return Rows{p, st[0], st[1], st[2], int32_t(per)};
}

Decay decay(const void* p, const int64_t* st, int32_t dtype) {
  return Decay{p, st[0], st[1], st[2], dtype == SSM_BF16};
}

template <typename T>
ssm_status_t run_fwd(const ssm_decay_attn_args_t* a, const Sizes& z, const FwdPlan& pl, hipStream_t s) {
  MixParams p{};
  const int64_t per = z.H / z.Hk;
  p.a = rows(a->q, a->q_stride, per);
  p.b = rows(a->k, a->k_stride, per);
  p.c = rows(a->v, a->v_stride, 1);
  p.g = decay(a->log_decay, a->decay_stride, a->decay_dtype);
  p.lengths = a->lengths;
  p.s0 = a->h0;
  p.sm = z.dv;
  p.sn = 1;
  p.B = z.B;
  p.L = z.L;
  p.H = z.H;
  p.M = int32_t(z.dk);
  p.N = int32_t(z.dv);
  p.span = pl.cut.span;
  p.spans = int32_t(pl.cut.spans);
  if (p.spans > 1) {
    char* ws = static_cast<char*>(a->workspace);
    float* carry = reinterpret_cast<float*>(ws);
    if (ssm_status_t st = run_carries<T, false>(p, carry, reinterpret_cast<float*>(ws + pl.off_total), s)) return st;
    p.carry = carry;
    p.cm = z.dv;
    p.cn = 1;
  }
  p.s_last = a->h_last;
  p.out = a->o;
  return run_mix<T, 1, T, kOut, false>(p, s);
}

// (tokens, heads, dk) fp32 to (tokens, key heads, dk).
template <typename T>
ssm_status_t sum_heads(void* out, const void* in, const Sizes& z, hipStream_t s) {
  const int64_t n = z.tokens * z.Hk * z.dk;
  const int32_t per = int32_t(z.H / z.Hk);
  const bool four = z.dk % 4 == 0;
  const dim3 grid(uint32_t(std::min<int64_t>((n / (four ? 4 : 1) + 255) / 256, 1 << 20)));
  if (four)
    hipLaunchKernelGGL((k_sum_heads<T, 4>), grid, dim3(256), 0, s, static_cast<T*>(out),
                       static_cast<const float*>(in), n, int32_t(z.dk), per);
  else
    hipLaunchKernelGGL((k_sum_heads<T, 1>), grid, dim3(256), 0, s, static_cast<T*>(out),
                       static_cast<const float*>(in), n, int32_t(z.dk), per);
  return launch_status("k_sum_heads");
}

template <typename T>
ssm_status_t run_bwd(const ssm_decay_attn_bwd_args_t* a, const Sizes& z, const BwdPlan& pl,
                     hipStream_t s) {
  char* ws = static_cast<char*>(a->workspace);
  const int64_t per = z.H / z.Hk;
  const bool shared = per > 1;
  const Rows q = rows(a->q, a->q_stride, per), k = rows(a->k, a->k_stride, per);
  const Rows v = rows(a->v, a->v_stride, 1), d = rows(a->dout, a->dout_stride, 1);
  float* carry = reinterpret_cast<float*>(ws + pl.off_carry);
  float* rcarry = reinterpret_cast<float*>(ws + pl.off_rcarry);
  float* total = reinterpret_cast<float*>(ws + pl.off_total);
  MixParams p{};
  p.g = decay(a->log_decay, a->decay_stride, a->decay_dtype);
  p.lengths = a->lengths;
  p.B = z.B;
  p.L = z.L;
  p.H = z.H;
  p.span = pl.cut.span;
  p.spans = int32_t(pl.cut.spans);
  // dq, with the state transposed: S(m, n) at row n of the stored state
  MixParams dq = p;
  dq.a = d;
  dq.b = v;
  dq.c = k;
  dq.x = q;
  dq.s0 = a->h0;
  dq.sm = 1;
  dq.sn = z.dv;
  dq.M = int32_t(z.dv);
  dq.N = int32_t(z.dk);
  dq.cm = z.dk;
  dq.cn = 1;
  // dk, backward in time, G transposed
  MixParams dk = dq;
  dk.a = v;
  dk.b = d;
  dk.c = q;
  dk.x = k;
  dk.s0 = a->dh_last;
  // dv, backward in time, the same G
  MixParams dv = p;
  dv.a = k;
  dv.b = q;
  dv.c = d;
  dv.s0 = a->dh_last;
  dv.s_last = a->dh0;
  dv.sm = z.dv;
  dv.sn = 1;
  dv.M = int32_t(z.dk);
  dv.N = int32_t(z.dv);
  dv.cm = 1;
  dv.cn = z.dk;
  dv.out = a->dv;
  if (p.spans > 1) {
    if (ssm_status_t st = run_carries<T, false>(dq, carry, total, s)) return st;
    if (ssm_status_t st = run_carries<T, true>(dk, rcarry, total, s)) return st;
    dq.carry = carry;
    dk.carry = dv.carry = rcarry;
  }
  dq.dots = reinterpret_cast<float*>(ws + pl.off_u);
  dk.dots = reinterpret_cast<float*>(ws + pl.off_w);
  dq.kept = dk.kept = reinterpret_cast<float*>(ws + pl.off_kept);
  dk.flow = reinterpret_cast<float*>(ws + pl.off_flow);
  dq.kept_slices = dk.kept_slices = int32_t(pl.slices);
  dq.kept_tiles = dk.kept_tiles = int32_t(pl.tiles);
  dq.out = shared ? ws + pl.off_heads : a->dq;
  dk.out = shared ? ws + pl.off_heads : a->dk;
  if (ssm_status_t st = run_mix<T, 1, T, kOut, true>(dv, s)) return st;
  if (shared) {
    // per value head into one buffer, each summed while the caches still hold it
    if (ssm_status_t st = run_mix<T, 2, float, kOutDots, false>(dq, s)) return st;
    if (ssm_status_t st = sum_heads<T>(a->dq, dq.out, z, s)) return st;
    if (ssm_status_t st = run_mix<T, 2, float, kOutDots, true>(dk, s)) return st;
    if (ssm_status_t st = sum_heads<T>(a->dk, dk.out, z, s)) return st;
  } else {
    if (ssm_status_t st = run_mix<T, 2, T, kOutDots, false>(dq, s)) return st;
    if (ssm_status_t st = run_mix<T, 2, T, kOutDots, true>(dk, s)) return st;
  }
  DecayGradParams gp{};
  gp.q = q;
  gp.k = k;
  gp.v = v;
  gp.dout = d;
  gp.g = p.g;
  gp.reads = dq.dots;
  gp.writes = dk.dots;
  gp.flow = dk.flow;
  gp.lengths = a->lengths;
  gp.dg = a->dlog_decay;
  gp.B = z.B;
  gp.L = z.L;
  gp.H = z.H;
  gp.padded = pl.cut.span * pl.cut.spans;
  gp.dk = int32_t(z.dk);
  gp.dv = int32_t(z.dv);
  gp.slices = int32_t(pl.slices);
  gp.bf16 = a->decay_dtype == SSM_BF16;
  constexpr int CT = chunk_tokens(sizeof(T) == 2 ? SSM_BF16 : SSM_F32);
  const dim3 grid(uint32_t(std::min<int64_t>(z.B * z.H * (gp.padded / CT), kMaxGroups)));
  if (fast_rows(q, z.dk, sizeof(T)) && fast_rows(k, z.dk, sizeof(T)) && fast_rows(v, z.dv, sizeof(T)) &&
      fast_rows(d, z.dv, sizeof(T)))
    hipLaunchKernelGGL((k_decay_grad<T, CT, true>), grid, dim3(256), 0, s, gp);
  else
    hipLaunchKernelGGL((k_decay_grad<T, CT, false>), grid, dim3(256), 0, s, gp);
  return launch_status("k_decay_grad");
}

template <typename T, int V, int LC>
ssm_status_t launch_step(AttnStepParams p, hipStream_t s) {
  p.tiles = (p.dv + LC * V - 1) / (LC * V);
  const int64_t groups = p.B * p.H * p.tiles;
  if (groups > kMaxGroups) return fail(SSM_ERR_SHAPE, "problem too large for one launch");
  hipLaunchKernelGGL((k_attn_step<T, V, LC>), dim3(uint32_t(groups)), dim3(256), 0, s, p);
  return launch_status("k_attn_step");
}

template <typename T>
ssm_status_t run_step(const AttnStepParams& p, hipStream_t s) {
  if (p.dv % 4 == 0 && !misaligned(p.h, 16)) {
    if (p.dv <= 16) return launch_step<T, 4, 4>(p, s);
    if (p.dv <= 32) return launch_step<T, 4, 8>(p, s);
    return launch_step<T, 4, 16>(p, s);
  }
  return p.dv <= 16 ? launch_step<T, 1, 16>(p, s) : launch_step<T, 1, 64>(p, s);
}

}  // namespace

extern "C" {

size_t ssm_decay_attn_workspace_size(const ssm_decay_attn_args_t* a) {
  if (!a || a->span < 0 || a->span % kSpanAlign != 0) return 0;
  Sizes z{a->batch, a->seqlen, a->heads, a->key_heads, a->key_dim, a->value_dim, 0, 0};
  if (check_sizes(&z)) return 0;
  return make_fwd_plan(z, a->span).total;
}

size_t ssm_decay_attn_bwd_workspace_size(const ssm_decay_attn_bwd_args_t* a) {
  if (!a || a->span < 0 || a->span % kSpanAlign != 0) return 0;
  Sizes z{a->batch, a->seqlen, a->heads, a->key_heads, a->key_dim, a->value_dim, 0, 0};
  if (check_sizes(&z)) return 0;
  return make_bwd_plan(z, a->span, a->dtype).total;
}

ssm_status_t ssm_decay_attn_fwd(const ssm_decay_attn_args_t* a, void* hip_stream) {
  clear_message();
  Sizes z;
  FwdPlan pl;
  if (ssm_status_t st = check_fwd(a, &z, &pl)) return st;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (z.B * z.H == 0) return SSM_OK;
  if (z.L == 0) return copy_state(a->h_last, a->h0, z.state, s);
  return a->dtype == SSM_F32 ? run_fwd<float>(a, z, pl, s) : run_fwd<bf16_t>(a, z, pl, s);
}

ssm_status_t ssm_decay_attn_step(const ssm_decay_attn_step_args_t* a, void* hip_stream) {
  clear_message();
  Sizes z;
  if (ssm_status_t st = check_step(a, &z)) return st;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (z.B * z.H == 0) return SSM_OK;
  AttnStepParams p{};
  p.q = a->q;
  p.k = a->k;
  p.v = a->v;
  p.g = a->log_decay;
  for (int i = 0; i < 2; ++i) {
    p.qs[i] = a->q_stride[i];
    p.ks[i] = a->k_stride[i];
    p.vs[i] = a->v_stride[i];
    p.gs[i] = a->decay_stride[i];
  }
  p.h = a->h;
  p.o = a->o;
  p.B = z.B;
  p.H = z.H;
  p.per = int32_t(z.H / z.Hk);
  p.dk = int32_t(z.dk);
  p.dv = int32_t(z.dv);
  p.g_bf16 = a->decay_dtype == SSM_BF16;
  return a->dtype == SSM_F32 ? run_step<float>(p, s) : run_step<bf16_t>(p, s);
}

ssm_status_t ssm_decay_attn_bwd(const ssm_decay_attn_bwd_args_t* a, void* hip_stream) {
  clear_message();
  Sizes z;
  BwdPlan pl;
  if (ssm_status_t st = check_bwd(a, &z, &pl)) return st;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (z.B * z.H == 0) return SSM_OK;
  if (z.L == 0) return copy_state(a->dh0, a->dh_last, z.state, s);
  return a->dtype == SSM_F32 ? run_bwd<float>(a, z, pl, s) : run_bwd<bf16_t>(a, z, pl, s);
}

}  // extern "C"
