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
  if (a->rows * a->groups > kMaxGrid) return fail(SSM_ERR_SHAPE, "problem too large for one launch");
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

size_t bwd_workspace(const ssm_group_norm_bwd_args_t* a) {
  if (!a->dweight && !a->dbias) return 0;
  return size_t(a->rows * a->groups) * 8;
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

template <typename T>
ssm_status_t run_fwd(const NormParams& p, hipStream_t s) {
  hipLaunchKernelGGL((k_norm_simple<T>), dim3(uint32_t(p.rows * p.G)), dim3(kWave), 0, s, p);
  return launch_status("k_norm_simple");
}

template <typename T>
ssm_status_t run_bwd(const NormParams& p, hipStream_t s) {
  if (p.rows > 0) {
    hipLaunchKernelGGL((k_norm_bwd_simple<T>), dim3(uint32_t(p.rows * p.G)), dim3(kWave), 0, s, p);
    if (ssm_status_t st = launch_status("k_norm_bwd_simple")) return st;
  }
  if (!p.dw && !p.db) return SSM_OK;
  hipLaunchKernelGGL((k_norm_cols_simple<T>), dim3(uint32_t((p.C + kWave - 1) / kWave)), dim3(kWave), 0, s, p);
  return launch_status("k_norm_cols_simple");
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
  return a->dtype == SSM_F32 ? run_fwd<float>(p, s) : run_fwd<bf16_t>(p, s);
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
  p.dw = a->dweight;
  p.db = a->dbias;
  p.stats = a->dweight || a->dbias ? static_cast<float*>(a->workspace) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(hip_stream);
  return a->dtype == SSM_F32 ? run_bwd<float>(p, s) : run_bwd<bf16_t>(p, s);
}

}  // extern "C"
