// group_norm.hip -- host side of the group norm: argument checks and launches.
// The device code is group_norm.hpp; the contract include/ssm_scan.h.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "ssm_scan.h"
#include "ssm_host.hpp"
#include "group_norm.hpp"

namespace {

using namespace ssmh;
using namespace ssmn;

// What both calls check; the ranges of x and z on success.
template <typename Args>
ssm_status_t check_norm(const Args* a, Range* x, Range* z) {
  if (!a) return fail(SSM_ERR_NULL, "args is NULL");
  if (a->rows < 0 || a->channels < 0)
    return fail(SSM_ERR_SHAPE, "negative size: rows=%lld channels=%lld", (long long)a->rows,
                (long long)a->channels);
  if (a->groups < 1 || a->channels % a->groups != 0)
    return fail(SSM_ERR_SHAPE, "channels %lld is not a multiple of groups %lld",
                (long long)a->channels, (long long)a->groups);
  if (a->dtype != SSM_F32 && a->dtype != SSM_BF16) return fail(SSM_ERR_DTYPE, "unknown dtype %d", a->dtype);
  if (a->mode < SSM_NORM_PLAIN || a->mode > SSM_NORM_GATE_FIRST)
    return fail(SSM_ERR_DTYPE, "unknown mode %d", a->mode);
  if (a->rms != 0 && a->rms != 1) return fail(SSM_ERR_UNSUPPORTED, "rms must be 0 or 1");
  if (!(a->eps >= 0.0f) || std::isinf(a->eps))
    return fail(SSM_ERR_UNSUPPORTED, "eps must be finite and not negative");
  const bool gated = a->mode >= SSM_NORM_GATE;
  if (!gated && a->z) return fail(SSM_ERR_UNSUPPORTED, "z goes with the gate modes only");
  int64_t n, e;
  if (!mul_ok(a->rows, a->channels, &n) || n > INT64_MAX / 16)
    return fail(SSM_ERR_SHAPE, "sizes overflow");
  if (a->x_stride < 0 || (gated && a->z_stride < 0) || !mul_ok(a->rows, a->x_stride, &e) ||
      e > INT64_MAX / 16 || (gated && (!mul_ok(a->rows, a->z_stride, &e) || e > INT64_MAX / 16)))
    return fail(SSM_ERR_SHAPE, "a row stride is negative or overflows");
  // rows times groups, and a row's channels, are counted in 32 bits
  if (!mul_ok(a->rows, a->groups, &e) || e > kMaxGrid || a->channels > kMaxGrid) return fail(SSM_ERR_SHAPE, "problem too large for one launch");
  const size_t es = dtype_size(a->dtype);
  *x = *z = Range{nullptr, 0};
  if (n == 0) return SSM_OK;
  if (!a->x) return fail(SSM_ERR_NULL, "x is required");
  if (gated && !a->z) return fail(SSM_ERR_NULL, "z is required with the gate modes");
  if (misaligned(a->x, es) || misaligned(a->z, es) || misaligned(a->weight, 4) || misaligned(a->bias, 4))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  *x = Range{a->x, size_t((a->rows - 1) * a->x_stride + a->channels) * es};
  if (gated) *z = Range{a->z, size_t((a->rows - 1) * a->z_stride + a->channels) * es};
  return SSM_OK;
}

ssm_status_t check_fwd(const ssm_group_norm_args_t* a) {
  Range x, z;
  if (ssm_status_t st = check_norm(a, &x, &z)) return st;
  if (a->rows * a->channels == 0) return SSM_OK;
  if (!a->y) return fail(SSM_ERR_NULL, "y is required");
  const size_t es = dtype_size(a->dtype), c4 = size_t(a->channels) * 4;
  if (misaligned(a->y, es)) return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const Range y{a->y, size_t(a->rows * a->channels) * es};
  for (const Range& r : {x, z, Range{a->weight, c4}, Range{a->bias, c4}})
    if (overlap(y, r)) return fail(SSM_ERR_ALIAS, "y overlaps an input");
  return SSM_OK;
}

// How the lanes are dealt: TG lanes to a group, R times V channels each (V = 1,
// or 16 bytes' worth where every row and group starts on 16 bytes), and `per`
// rows to a lane.  TG = 0: the group is too long for registers.
struct Deal {
  int TG = 0, R = 0;
  bool vec = false;
  int64_t per = 1, blocks = 0;
};

// The backward pass holds more of a row: past 1024 turns its registers would spill
// (at 1024 bf16 takes up to 440 of them, one wave a SIMD: 4096 rows of 8192
// channels 98 us without dweight and dbias, 3.4 TB/s, the long form would read the
// rows again for each pass over them).
Deal deal_groups(int64_t gs, bool vec, int elem, bool bwd) {
  Deal d;
  d.vec = vec;
  const int64_t n = vec ? gs / (16 / elem) : gs;   // turns of the lanes
  if (n <= 64) {
    d.R = 1;
    for (d.TG = vec ? 1 : 4; d.TG < n; d.TG *= vec ? 2 : 4) {
    }
  } else if (n <= 256) {
    d.TG = 64;
    d.R = n <= 128 ? 2 : 4;
  } else if (n <= (!vec ? 4096 : bwd ? 1024 : 2048)) {
    d.TG = 256;
    d.R = vec ? (n <= 1024 ? 4 : 8) : 16;
  }
  return d;
}

// Rows to a lane, at most `most`: the weights are read once for them, and the
// sums for dweight and dbias leave registers once.  No more than leaves the GPU
// 2^18 lanes (four waves a SIMD).
void deal_rows(Deal* d, int64_t rows, int64_t groups, int64_t most) {
  const int64_t lanes = rows * groups * (d->TG ? d->TG : 256);
  d->per = std::max<int64_t>(1, std::min(most, lanes >> 18));
  d->blocks = (rows + d->per - 1) / d->per;
}

template <typename Args>
bool rows_wide(const Args* a) {
  const int64_t k = a->dtype == SSM_BF16 ? 8 : 4, gs = a->channels / a->groups;
  const bool gated = a->mode >= SSM_NORM_GATE;
  return gs % k == 0 && !misaligned(a->weight, 16) && !misaligned(a->bias, 16) && a->x_stride % k == 0 && !misaligned(a->x, 16) &&
         (!gated || (a->z_stride % k == 0 && !misaligned(a->z, 16)));
}

Deal bwd_deal(const ssm_group_norm_bwd_args_t* a) {
  const int64_t k = a->dtype == SSM_BF16 ? 8 : 4;
  const bool vec = rows_wide(a) && a->dy_stride % k == 0 && !misaligned(a->dy, 16) && !misaligned(a->dx, 16) &&
                   !misaligned(a->dz, 16);
  Deal d = deal_groups(a->channels / a->groups, vec, a->dtype == SSM_BF16 ? 2 : 4, true);
  deal_rows(&d, a->rows, a->groups, 64);
  return d;
}

// The workspace must not depend on addresses, which a caller that asks for its
// size may not have filled in: it holds the most blocks any dealing makes (one
// with the most lanes, and so rows, to a group has the fewest).
size_t bwd_workspace(const ssm_group_norm_bwd_args_t* a) {
  const int want = (a->dweight ? 1 : 0) + (a->dbias ? 1 : 0);
  if (want == 0 || a->rows * a->channels == 0) return 0;
  const int64_t gs = a->channels / a->groups;
  int64_t blocks = 0;
  for (int vec = 0; vec < 2; ++vec) {
    Deal d = deal_groups(gs, vec != 0, a->dtype == SSM_BF16 ? 2 : 4, true);
    deal_rows(&d, a->rows, a->groups, 64);
    blocks = std::max(blocks, d.blocks);
  }
  return size_t(want) * align256(size_t(blocks) * size_t(a->channels) * 4);
}

ssm_status_t check_bwd(const ssm_group_norm_bwd_args_t* a) {
  Range x, z;
  if (ssm_status_t st = check_norm(a, &x, &z)) return st;
  int64_t e;
  if (a->dy_stride < 0 || !mul_ok(a->rows, a->dy_stride, &e) || e > INT64_MAX / 16)
    return fail(SSM_ERR_SHAPE, "a row stride is negative or overflows");
  if (misaligned(a->dweight, 4) || misaligned(a->dbias, 4))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment)");
  const bool gated = a->mode >= SSM_NORM_GATE;
  if (!gated && a->dz) return fail(SSM_ERR_UNSUPPORTED, "dz goes with the gate modes only");
  const size_t c4 = size_t(a->channels) * 4;
  const Range dw{a->dweight, c4}, db{a->dbias, c4};
  if (overlap(dw, db)) return fail(SSM_ERR_ALIAS, "two gradients overlap");
  if (a->rows * a->channels == 0) return SSM_OK;
  if (!a->dy || !a->dx) return fail(SSM_ERR_NULL, "dy and dx are required");
  if (gated && !a->dz) return fail(SSM_ERR_NULL, "dz is required with the gate modes");
  const size_t es = dtype_size(a->dtype), need = bwd_workspace(a);
  if (misaligned(a->dy, es) || misaligned(a->dx, es) || misaligned(a->dz, es) || misaligned(a->workspace, 256))
    return fail(SSM_ERR_UNSUPPORTED, "misaligned pointer (element alignment; workspace 256 bytes)");
  if (need > 0 && !a->workspace) return fail(SSM_ERR_WORKSPACE, "workspace of %zu bytes required", need);
  if (a->workspace_bytes < need)
    return fail(SSM_ERR_WORKSPACE, "workspace has %zu bytes, %zu required", a->workspace_bytes, need);
  const size_t n = size_t(a->rows * a->channels) * es;
  const Range dy{a->dy, size_t((a->rows - 1) * a->dy_stride + a->channels) * es};
  const Range outs[] = {{a->dx, n}, {a->dz, n}, dw, db, {a->workspace, need}};
  const Range ins[] = {x, z, dy, {a->weight, c4}, {a->bias, c4}};
  for (int i = 0; i < 5; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return fail(SSM_ERR_ALIAS, "an output overlaps an input");
    for (int k = i + 1; k < 5; ++k)
      if (overlap(outs[i], outs[k])) return fail(SSM_ERR_ALIAS, "two outputs overlap");
  }
  return SSM_OK;
}

template <typename Args>
NormParams params(const Args* a) {
  NormParams p{};
  p.x = a->x;
  p.z = a->z;
  p.w = a->weight;
  p.b = a->bias;
  p.rows = a->rows;
  p.C = a->channels;
  p.G = a->groups;
  p.gs = a->channels / a->groups;
  p.xs = a->x_stride;
  p.zs = a->z_stride;
  p.mode = a->mode;
  p.rms = a->rms;
  p.eps = a->eps;
  return p;
}

template <typename T, bool BWD, int V, int TG, int R>
ssm_status_t launch(const NormParams& p, int64_t blocks, hipStream_t s) {
  const dim3 grid(uint32_t((blocks * p.G * TG + 255) / 256));
  const bool z = p.mode >= kGate;
  if constexpr (BWD) {
    if (z)
      hipLaunchKernelGGL((k_norm_bwd<T, V, TG, R, true>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_norm_bwd<T, V, TG, R, false>), grid, dim3(256), 0, s, p);
  } else {
    if (z)
      hipLaunchKernelGGL((k_norm<T, V, TG, R, true>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_norm<T, V, TG, R, false>), grid, dim3(256), 0, s, p);
  }
  return launch_status(BWD ? "k_norm_bwd" : "k_norm");
}

template <typename T, bool BWD>
ssm_status_t run_norm(NormParams p, const Deal& d, hipStream_t s) {
  // a launch holds at most 2^32 - 1 lanes
  if (d.blocks * p.G > int64_t(UINT32_MAX) / (d.TG ? d.TG : 256))
    return fail(SSM_ERR_SHAPE, "problem too large for one launch");
  p.per = d.per;
  constexpr int V = 16 / int(sizeof(T));
  const int64_t n = d.blocks;
  if (d.TG == 0) {
    const dim3 grid(uint32_t(n * p.G));
    if constexpr (BWD)
      hipLaunchKernelGGL((k_norm_bwd_long<T>), grid, dim3(256), 0, s, p);
    else
      hipLaunchKernelGGL((k_norm_long<T>), grid, dim3(256), 0, s, p);
    return launch_status(BWD ? "k_norm_bwd_long" : "k_norm_long");
  }
  if (d.vec) {
    switch (d.TG) {
      case 1: return launch<T, BWD, V, 1, 1>(p, n, s);
      case 2: return launch<T, BWD, V, 2, 1>(p, n, s);
      case 4: return launch<T, BWD, V, 4, 1>(p, n, s);
      case 8: return launch<T, BWD, V, 8, 1>(p, n, s);
      case 16: return launch<T, BWD, V, 16, 1>(p, n, s);
      case 32: return launch<T, BWD, V, 32, 1>(p, n, s);
      case 64:
        return d.R == 1 ? launch<T, BWD, V, 64, 1>(p, n, s)
                        : d.R == 2 ? launch<T, BWD, V, 64, 2>(p, n, s) : launch<T, BWD, V, 64, 4>(p, n, s);
      default:
        if constexpr (!BWD)
          if (d.R == 8) return launch<T, BWD, V, 256, 8>(p, n, s);
        return launch<T, BWD, V, 256, 4>(p, n, s);
    }
  }
  switch (d.TG) {
    case 4: return launch<T, BWD, 1, 4, 1>(p, n, s);
    case 16: return launch<T, BWD, 1, 16, 1>(p, n, s);
    case 64:
      return d.R == 1 ? launch<T, BWD, 1, 64, 1>(p, n, s)
                      : d.R == 2 ? launch<T, BWD, 1, 64, 2>(p, n, s) : launch<T, BWD, 1, 64, 4>(p, n, s);
    default: return launch<T, BWD, 1, 256, 16>(p, n, s);
  }
}

template <typename T>
ssm_status_t run_bwd(const ssm_group_norm_bwd_args_t* a, NormParams p, hipStream_t s) {
  char* ws = static_cast<char*>(a->workspace);
  int64_t blocks = 0;
  if (a->rows > 0) {
    const Deal d = bwd_deal(a);
    blocks = d.blocks;
    p.dw = a->dweight ? reinterpret_cast<float*>(ws) : nullptr;
    p.db = a->dbias ? reinterpret_cast<float*>(ws + (a->dweight ? align256(size_t(blocks) * size_t(p.C) * 4) : 0))
                    : nullptr;
    if (ssm_status_t st = run_norm<T, true>(p, d, s)) return st;
  }
  if (!a->dweight && !a->dbias) return SSM_OK;
  const ColsParams c{{p.dw, p.db}, {a->dweight, a->dbias}, blocks, p.C};
  hipLaunchKernelGGL(k_norm_cols, dim3(uint32_t((p.C + 15) / 16), 2), dim3(256), 0, s, c);
  return launch_status("k_norm_cols");
}

}  // namespace

extern "C" {

ssm_status_t ssm_group_norm_fwd(const ssm_group_norm_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_fwd(a)) return st;
  if (a->rows * a->channels == 0) return SSM_OK;
  NormParams p = params(a);
  p.y = a->y;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  Deal d = deal_groups(p.gs, rows_wide(a) && !misaligned(a->y, 16), a->dtype == SSM_BF16 ? 2 : 4,
                       false);
  deal_rows(&d, a->rows, a->groups, d.TG ? 8 : 1);
  return a->dtype == SSM_F32 ? run_norm<float, false>(p, d, s) : run_norm<bf16_t, false>(p, d, s);
}

size_t ssm_group_norm_bwd_workspace_size(const ssm_group_norm_bwd_args_t* a) {
  int64_t n;
  if (!a || a->rows < 0 || a->channels < 0 || a->groups < 1 || a->channels % a->groups != 0 ||
      !mul_ok(a->rows, a->channels, &n) || n > INT64_MAX / 16)
    return 0;
  return n == 0 ? 0 : bwd_workspace(a);
}

ssm_status_t ssm_group_norm_bwd(const ssm_group_norm_bwd_args_t* a, void* hip_stream) {
  clear_message();
  if (ssm_status_t st = check_bwd(a)) return st;
  if (a->channels == 0) return SSM_OK;
  NormParams p = params(a);
  p.dy = a->dy;
  p.ds = a->dy_stride;
  p.y = a->dx;
  p.dz = a->dz;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return a->dtype == SSM_F32 ? run_bwd<float>(a, p, s) : run_bwd<bf16_t>(a, p, s);
}

}  // extern "C"
