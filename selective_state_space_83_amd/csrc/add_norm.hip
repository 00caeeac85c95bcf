// add_norm.hip -- host side of the residual's addition with the root-mean-square
// norm: argument checks and launches.  The device code is add_norm.hpp; the
// contract include/ssm_scan.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ssm_scan.h"
#include "ssm_host.hpp"
#include "add_norm.hpp"

namespace {

using namespace ssmh;
using namespace ssma;

bool known(int32_t dt) { return dt == SSM_F32 || dt == SSM_BF16; }

// rows x channels with a row stride: sizes that addresses and counts hold.
ssm_status_t check_sizes(int64_t rows, int64_t channels, std::initializer_list<int64_t> strides) {
  int64_t n;
  if (rows < 0 || channels < 0)
    return fail(SSM_ERR_SHAPE, "negative size: rows=%lld channels=%lld", (long long)rows, (long long)channels);
  if (!mul_ok(rows, channels, &n) || n > INT64_MAX / 16) return fail(SSM_ERR_SHAPE, "sizes overflow");
  if (rows > kMaxGrid || channels > (int64_t(1) << 27)) return fail(SSM_ERR_SHAPE, "problem too large for one launch");
  for (int64_t s : strides)
    if (s < 0 || !mul_ok(rows, s, &n) || n > INT64_MAX / 16)
      return fail(SSM_ERR_SHAPE, "a row stride is negative or overflows");
  return SSM_OK;
}

Range rows_of(const void* p, int64_t rows, int64_t channels, int64_t stride, size_t es) {
  if (!p || rows == 0) return Range{nullptr, 0};
  return Range{p, size_t((rows - 1) * stride + channels) * es};
}

bool power_of_two_block(int64_t b) { return b == 32 || b == 64 || b == 128 || b == 256; }

ssm_status_t check_fwd(const ssm_add_norm_args_t* a) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_sizes(a->rows, a->channels, {a->x_stride, a->residual ? a->residual_stride : 0})) return st;
  if (!known(a->dtype)) return fail(SSM_ERR_DTYPE, "unknown dtype %d", a->dtype);
  if (a->residual_dtype != a->dtype && a->residual_dtype != SSM_F32)
    return fail(SSM_ERR_DTYPE, "residual_dtype must be dtype or SSM_F32");
  if (a->y_dtype != a->dtype && a->y_dtype != SSM_E4M3) return fail(SSM_ERR_DTYPE, "y_dtype must be dtype or SSM_E4M3");
  if (!(a->eps >= 0.0f) || std::isinf(a->eps))
    return fail(SSM_ERR_UNSUPPORTED, "eps must be finite and not negative");
  const bool quant = a->y_dtype == SSM_E4M3;
  if (a->block != 0 && (!quant || !power_of_two_block(a->block)))
    return fail(SSM_ERR_UNSUPPORTED, "block must be 0, or with SSM_E4M3 32, 64, 128 or 256");
  if (!quant && a->scale) return fail(SSM_ERR_UNSUPPORTED, "scale goes with SSM_E4M3 only");
  if (a->rows * a->channels == 0) return SSM_OK;
  if (!a->x || !a->y || (quant && !a->scale)) return fail(SSM_ERR_NULL, "x, y and (with SSM_E4M3) scale are required");
  const size_t es = dtype_size(a->dtype), rs = dtype_size(a->residual_dtype), ys = quant ? 1 : es;
  if (misaligned(a->x, es) || misaligned(a->residual, rs) || misaligned(a->sum, rs) || misaligned(a->y, ys) ||
      misaligned(a->weight, 4) || misaligned(a->scale, 4))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const size_t n = size_t(a->rows * a->channels);
  const Range sum{a->sum, n * rs}, y{a->y, n * ys}, w{a->weight, size_t(a->channels) * 4};
  const int64_t nblk = a->block ? (a->channels + a->block - 1) / a->block : 1;
  const Range scale{a->scale, size_t(a->rows) * size_t(nblk) * 4};
  const Range x = rows_of(a->x, a->rows, a->channels, a->x_stride, es);
  const Range res = rows_of(a->residual, a->rows, a->channels, a->residual_stride, rs);
  for (const Range& out : {sum, y, scale})
    if (overlap(out, x) || overlap(out, w)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
  // the sum may take the residual's place
  const bool in_place = a->sum == a->residual && (a->residual_stride == a->channels || a->rows == 1);
  if (overlap(y, res) || overlap(scale, res) || (overlap(sum, res) && !in_place))
    return fail(SSM_ERR_ALIAS, "an output overlaps the residual");
  if (overlap(sum, y) || overlap(sum, scale) || overlap(y, scale)) return fail(SSM_ERR_ALIAS, "two outputs overlap");
  return SSM_OK;
}

constexpr int64_t kL2Bytes = int64_t(32) << 20;   // of the eight XCDs

// Neighbouring channels of a lane where every row allows it: 16 bytes of the row's
// widest type, so that a wave's loads and stores have no gaps.  (8 channels of bf16 x
// beside an fp32 residual: two loads 32 bytes apart, 32768 x 2560 to 8 bits 181 us for 161.)
constexpr int kWide16 = 8, kWide32 = 4;
template <typename A, typename B>
constexpr int wide() { return sizeof(A) == 2 && sizeof(B) == 2 ? kWide16 : kWide32; }

// How the lanes are dealt: TG lanes to a row, R times V channels each (V = 1 or as
// above), and in the backward pass `per` rows to a lane.  TG = 0: the row is too long
// for registers.
struct Deal {
  int TG = 0, R = 0;
  bool vec = false;
  int64_t per = 1, blocks = 0;
};

Deal deal_row(int64_t C, bool vec, int64_t v, bool bwd) {
  Deal d;
  d.vec = vec;
  const int64_t n = vec ? C / v : C;   // turns of the lanes
  if (vec && n <= 16) {
    d.TG = n <= 4 ? 4 : 16;
    d.R = 1;
  } else if (n <= 64) {
    d.TG = 64;
    d.R = 1;
  } else if (n <= 128 || (n <= 256 && !(vec && bwd))) {
    d.TG = 64;
    d.R = vec && n <= 128 ? 2 : 4;
  } else {
    // at most 64 channels to a lane, and 32 in the backward pass, which holds more of a
    // row; beyond, registers would spill
    const int64_t turns = (n + 255) / 256, most = (bwd && vec ? 32 : 64) / (vec ? v : 1);
    if (vec ? turns <= most : turns <= 16) {
      d.TG = 256;
      d.R = !vec ? 16 : turns <= 4 ? int(turns) : turns <= 8 ? 8 : 16;
    }
  }
  return d;
}

// Rows to a lane in the backward pass, at most 64, and no more than leaves the GPU 2^17
// lanes (two waves a SIMD, what its registers allow): the weights are read once for
// them, and the sums for dweight leave registers once.
void deal_rows(Deal* d, int64_t rows) {
  const int64_t lanes = rows * (d->TG ? d->TG : 256);
  d->per = std::max<int64_t>(1, std::min<int64_t>(64, lanes >> 17));
  d->blocks = (rows + d->per - 1) / d->per;
}

// A launch holds at most 2^32 - 1 lanes; n: groups of them.
ssm_status_t lanes_ok(const Deal& d, int64_t n) {
  return n > (int64_t(UINT32_MAX) - 255) / (d.TG ? d.TG : 256) ? fail(SSM_ERR_SHAPE, "problem too large for one launch") : SSM_OK;
}

// Workgroups for n groups of TG lanes.
uint32_t workgroups(int64_t n, int TG) { return uint32_t((n * TG + 255) / 256); }

template <typename InT, typename ResT, typename OutT, int V, int TG, int R>
ssm_status_t launch(const AddNormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((k_add_norm<InT, ResT, OutT, V, TG, R>), dim3(workgroups(p.rows, TG)), dim3(256), 0, s, p);
  return launch_status("k_add_norm");
}

template <typename InT, typename ResT, typename OutT>
ssm_status_t run_fwd(AddNormParams p, const Deal& d, hipStream_t s) {
  constexpr int V = wide<InT, ResT>();
  if (d.TG == 0) {
    if (d.vec)
      hipLaunchKernelGGL((k_add_norm_long<InT, ResT, OutT, V>), dim3(uint32_t(p.rows)), dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_add_norm_long<InT, ResT, OutT, 1>), dim3(uint32_t(p.rows)), dim3(256), 0, s, p);
    return launch_status("k_add_norm_long");
  }
  if (!d.vec) {
    if (d.TG == 256) return launch<InT, ResT, OutT, 1, 256, 16>(p, s);
    return d.R == 1 ? launch<InT, ResT, OutT, 1, 64, 1>(p, s) : launch<InT, ResT, OutT, 1, 64, 4>(p, s);
  }
  switch (d.TG) {
    case 4: return launch<InT, ResT, OutT, V, 4, 1>(p, s);
    case 16: return launch<InT, ResT, OutT, V, 16, 1>(p, s);
    case 64:
      return d.R == 1 ? launch<InT, ResT, OutT, V, 64, 1>(p, s)
                      : d.R == 2 ? launch<InT, ResT, OutT, V, 64, 2>(p, s) : launch<InT, ResT, OutT, V, 64, 4>(p, s);
    default:
      if (d.R == 1) return launch<InT, ResT, OutT, V, 256, 1>(p, s);
      if (d.R == 3) return launch<InT, ResT, OutT, V, 256, 3>(p, s);
      if constexpr (V == kWide32)
        if (d.R == 16) return launch<InT, ResT, OutT, V, 256, 16>(p, s);
      return d.R == 2 ? launch<InT, ResT, OutT, V, 256, 2>(p, s)
                      : d.R == 4 ? launch<InT, ResT, OutT, V, 256, 4>(p, s) : launch<InT, ResT, OutT, V, 256, 8>(p, s);
  }
}

template <typename InT, typename SumT, bool RES, int V, int TG, int R>
ssm_status_t launch_bwd(const AddNormBwdParams& p, const Deal& d, hipStream_t s) {
  hipLaunchKernelGGL((k_add_norm_bwd<InT, SumT, RES, V, TG, R>), dim3(workgroups(d.blocks, TG)), dim3(256), 0, s, p);
  return launch_status("k_add_norm_bwd");
}

template <typename InT, typename SumT, bool RES>
ssm_status_t run_bwd_of(AddNormBwdParams p, const Deal& d, hipStream_t s) {
  p.per = d.per;
  constexpr int V = wide<InT, SumT>();
  if (d.TG == 0) {
    if (d.vec)
      hipLaunchKernelGGL((k_add_norm_bwd_long<InT, SumT, RES, V>), dim3(uint32_t(d.blocks)), dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_add_norm_bwd_long<InT, SumT, RES, 1>), dim3(uint32_t(d.blocks)), dim3(256), 0, s, p);
    return launch_status("k_add_norm_bwd_long");
  }
  if (!d.vec) {
    if (d.TG == 256) return launch_bwd<InT, SumT, RES, 1, 256, 16>(p, d, s);
    return d.R == 1 ? launch_bwd<InT, SumT, RES, 1, 64, 1>(p, d, s) : launch_bwd<InT, SumT, RES, 1, 64, 4>(p, d, s);
  }
  switch (d.TG) {
    case 4: return launch_bwd<InT, SumT, RES, V, 4, 1>(p, d, s);
    case 16: return launch_bwd<InT, SumT, RES, V, 16, 1>(p, d, s);
    case 64:
      return d.R == 1 ? launch_bwd<InT, SumT, RES, V, 64, 1>(p, d, s)
                      : d.R == 2 ? launch_bwd<InT, SumT, RES, V, 64, 2>(p, d, s) : launch_bwd<InT, SumT, RES, V, 64, 4>(p, d, s);
    default:
      if (d.R == 1) return launch_bwd<InT, SumT, RES, V, 256, 1>(p, d, s);
      if (d.R == 3) return launch_bwd<InT, SumT, RES, V, 256, 3>(p, d, s);
      if constexpr (V == kWide32)
        if (d.R == 8) return launch_bwd<InT, SumT, RES, V, 256, 8>(p, d, s);
      return d.R == 2 ? launch_bwd<InT, SumT, RES, V, 256, 2>(p, d, s) : launch_bwd<InT, SumT, RES, V, 256, 4>(p, d, s);
  }
}

template <typename InT, typename SumT>
ssm_status_t run_bwd(const AddNormBwdParams& p, const Deal& d, hipStream_t s) {
  return p.res ? run_bwd_of<InT, SumT, true>(p, d, s) : run_bwd_of<InT, SumT, false>(p, d, s);
}

// Rows that all start on v elements.
bool row_wide(const void* p, int64_t stride, int64_t v, size_t es) { return !misaligned(p, size_t(v) * es) && stride % v == 0; }

int64_t wide_of(int32_t dtype, int32_t other) { return dtype == SSM_BF16 && other == SSM_BF16 ? kWide16 : kWide32; }

Deal bwd_deal(const ssm_add_norm_bwd_args_t* a, bool vec) {
  Deal d = deal_row(a->channels, vec, wide_of(a->dtype, a->sum_dtype), true);
  deal_rows(&d, a->rows);
  return d;
}

// The workspace must not depend on addresses, which a caller that asks for its size
// may not have filled in: it holds the most blocks any dealing makes.
size_t bwd_workspace(const ssm_add_norm_bwd_args_t* a) {
  if (!a->dweight || a->rows * a->channels == 0) return 0;
  const int64_t blocks = std::max(bwd_deal(a, false).blocks, bwd_deal(a, true).blocks);
  return align256(size_t(blocks) * size_t(a->channels) * 4);
}

// residual: null for the gradients from the kept sum.
ssm_status_t check_bwd(const ssm_add_norm_bwd_args_t* a, const void* residual, int64_t residual_stride) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (ssm_status_t st = check_sizes(a->rows, a->channels,
                                    {a->sum_stride, residual ? residual_stride : 0, a->dy_stride,
                                     a->dsum ? a->dsum_stride : 0}))
    return st;
  if (!known(a->dtype)) return fail(SSM_ERR_DTYPE, "unknown dtype %d", a->dtype);
  if (a->sum_dtype != a->dtype && a->sum_dtype != SSM_F32)
    return fail(SSM_ERR_DTYPE, "sum_dtype must be dtype or SSM_F32");
  if (a->reserved != 0) return fail(SSM_ERR_UNSUPPORTED, "reserved must be 0");
  if (!(a->eps >= 0.0f) || std::isinf(a->eps))
    return fail(SSM_ERR_UNSUPPORTED, "eps must be finite and not negative");
  if (a->dresidual && a->sum_dtype == a->dtype)
    return fail(SSM_ERR_UNSUPPORTED, "with one type dx is the residual's gradient too: dresidual must be NULL");
  if (misaligned(a->dweight, 4)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  if (a->rows * a->channels == 0) return SSM_OK;
  if (!a->sum || !a->dy || !a->dx) return fail(SSM_ERR_NULL, "sum, dy and dx are required");
  const size_t es = dtype_size(a->dtype), ss = dtype_size(a->sum_dtype), need = bwd_workspace(a);
  const size_t first = residual ? es : ss;   // of x, or of the kept sum
  if (misaligned(a->sum, first) || misaligned(residual, ss) || misaligned(a->dsum, ss) ||
      misaligned(a->dresidual, ss) || misaligned(a->dy, es) || misaligned(a->dx, es) ||
      misaligned(a->weight, 4) || misaligned(a->workspace, 256))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment; workspace 256 bytes)");
  if (need > 0 && !a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
  if (a->workspace_bytes < need)
    return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, need);
  const size_t n = size_t(a->rows * a->channels), c4 = size_t(a->channels) * 4;
  const Range outs[] = {{a->dx, n * es}, {a->dresidual, n * ss}, {a->dweight, c4}, {a->workspace, need}};
  const Range ins[] = {rows_of(a->sum, a->rows, a->channels, a->sum_stride, first),
                       rows_of(residual, a->rows, a->channels, residual_stride, ss),
                       rows_of(a->dy, a->rows, a->channels, a->dy_stride, es),
                       rows_of(a->dsum, a->rows, a->channels, a->dsum_stride, ss), {a->weight, c4}};
  for (int i = 0; i < 4; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
    for (int k = i + 1; k < 4; ++k)
      if (overlap(outs[i], outs[k])) return fail(SSM_ERR_ALIAS, "two outputs overlap");
  }
  return SSM_OK;
}

ssm_status_t add_norm_bwd(const ssm_add_norm_bwd_args_t* a, const void* residual, int64_t residual_stride, void* hip_stream) {
  if (ssm_status_t st = check_bwd(a, residual, residual_stride)) return st;
  if (a->channels == 0) return SSM_OK;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  int64_t blocks = 0;
  if (a->rows > 0) {
    AddNormBwdParams p{};
    p.sum = a->sum;
    p.res = residual;
    p.dy = a->dy;
    p.dsum = a->dsum;
    p.w = a->weight;
    p.dx = a->dx;
    p.dres = a->dresidual;
    p.dw = a->dweight ? static_cast<float*>(a->workspace) : nullptr;
    p.rows = a->rows;
    p.C = a->channels;
    p.ss = a->sum_stride;
    p.rs = residual ? residual_stride : 0;
    p.ds = a->dy_stride;
    p.gs = a->dsum ? a->dsum_stride : 0;
    p.eps = a->eps;
    const int64_t v = wide_of(a->dtype, a->sum_dtype);
    const size_t es = dtype_size(a->dtype), ss = dtype_size(a->sum_dtype);
    p.stream = a->rows * a->channels * int64_t(es + (a->dresidual ? ss : 0)) > kL2Bytes;
    const bool vec = a->channels % v == 0 && row_wide(a->sum, p.ss, v, residual ? es : ss) &&
                     row_wide(residual, p.rs, v, ss) && row_wide(a->dy, p.ds, v, es) &&
                     row_wide(a->dsum, p.gs, v, ss) && !misaligned(a->weight, 16) && !misaligned(a->dx, size_t(v) * es) &&
                     !misaligned(a->dresidual, size_t(v) * ss);
    const Deal d = bwd_deal(a, vec);
    blocks = d.blocks;
    ssm_status_t st = lanes_ok(d, blocks);
    if (st) return st;
    if (a->dtype == SSM_F32)
      st = run_bwd<float, float>(p, d, s);
    else if (a->sum_dtype == SSM_F32)
      st = run_bwd<bf16_t, float>(p, d, s);
    else
      st = run_bwd<bf16_t, bf16_t>(p, d, s);
    if (st) return st;
  }
  if (!a->dweight) return SSM_OK;
  const ssmn::ColsParams c{{static_cast<const float*>(a->workspace), nullptr}, {a->dweight, nullptr}, blocks, a->channels};
  hipLaunchKernelGGL(ssmn::k_norm_cols, dim3(uint32_t((a->channels + 15) / 16), 1), dim3(256), 0, s, c);
  return launch_status("k_norm_cols");
}

}  // namespace

extern "C" {

ssm_status_t ssm_add_norm_fwd(const ssm_add_norm_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_fwd(a)) return st;
  if (a->rows * a->channels == 0) return SSM_OK;
  AddNormParams p{};
  p.x = a->x;
  p.res = a->residual;
  p.w = a->weight;
  p.sum = a->sum;
  p.y = a->y;
  p.scale = a->scale;
  p.rows = a->rows;
  p.C = a->channels;
  p.xs = a->x_stride;
  p.rs = a->residual ? a->residual_stride : 0;
  p.eps = a->eps;
  p.block = a->block && a->block < a->channels ? int32_t(a->block) : int32_t(a->channels);
  p.nblk = int32_t((a->channels + p.block - 1) / p.block);
  const int64_t v = wide_of(a->dtype, a->residual_dtype);
  const size_t es = dtype_size(a->dtype), rs = dtype_size(a->residual_dtype);
  const bool quant = a->y_dtype == SSM_E4M3;
  const bool vec = a->channels % v == 0 && row_wide(a->x, a->x_stride, v, es) && row_wide(a->residual, p.rs, v, rs) &&
                   !misaligned(a->weight, 16) && !misaligned(a->sum, size_t(v) * rs) &&
                   !misaligned(a->y, size_t(v) * (quant ? 1 : es));
  p.stream = a->rows * a->channels * int64_t((quant ? 1 : es) + (a->sum ? rs : 0)) > kL2Bytes;
  Deal d = deal_row(a->channels, vec, v, false);
  // blocks are formed within a wave's turn, side by side
  if (p.nblk > 1 && !(vec && d.TG * v >= p.block)) d.TG = d.R = 0;
  if (ssm_status_t st = lanes_ok(d, p.rows)) return st;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  if (a->dtype == SSM_F32)
    return quant ? run_fwd<float, float, fp8_t>(p, d, s) : run_fwd<float, float, float>(p, d, s);
  if (a->residual_dtype == SSM_F32)
    return quant ? run_fwd<bf16_t, float, fp8_t>(p, d, s) : run_fwd<bf16_t, float, bf16_t>(p, d, s);
  return quant ? run_fwd<bf16_t, bf16_t, fp8_t>(p, d, s) : run_fwd<bf16_t, bf16_t, bf16_t>(p, d, s);
}

size_t ssm_add_norm_bwd_workspace_size(const ssm_add_norm_bwd_args_t* a) {
  int64_t n;
  if (!a || a->rows < 0 || a->channels < 0 || !mul_ok(a->rows, a->channels, &n) || n > INT64_MAX / 16) return 0;
  return bwd_workspace(a);
}

ssm_status_t ssm_add_norm_bwd(const ssm_add_norm_bwd_args_t* a, void* hip_stream) {
  clear_message();
  return add_norm_bwd(a, nullptr, 0, hip_stream);
}

ssm_status_t ssm_add_norm_bwd_residual(const ssm_add_norm_bwd_args_t* a, const void* residual, int64_t residual_stride,
                                       void* hip_stream) {
  clear_message();
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (!residual && a->rows > 0 && a->channels > 0) return fail(SSM_ERR_NULL, "residual is required");
  return add_norm_bwd(a, residual, residual_stride, hip_stream);
}

}  // extern "C"
