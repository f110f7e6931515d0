// Host side of the gated norm's and the linear layer's entry points
// (include/ssm_scan.h): argument checks, all before any HIP call, and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "capi_common.h"
#include "ssm_kernels.h"
#include "ssm_scan.h"

using namespace ssm::capi;

namespace {

// a launch has fewer than 2^32 threads, here in workgroups of 256
constexpr int64_t kMaxWorkgroups = int64_t(1) << 24;

int check_norm(ssm::NormArgs* a, const void* x, const void* z, const float* weight, int64_t rows, int64_t channels,
               int64_t groups, float eps, int center, int gate_first, int dtype) {
  if (!x) return fail(SSM_EINVAL, "x must not be NULL");
  if (rows <= 0 || channels <= 0 || groups <= 0)
    return fail(SSM_EINVAL, "sizes must be positive (rows=%lld channels=%lld groups=%lld)", (long long)rows,
                (long long)channels, (long long)groups);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_EUNSUPPORTED, "dtype %d is not supported", dtype);
  if (channels % groups != 0)
    return fail(SSM_EINVAL, "channels=%lld must be a multiple of groups=%lld", (long long)channels, (long long)groups);
  if (channels / groups > ssm::kNormMaxGroup)
    return fail(SSM_EUNSUPPORTED, "%lld channels per group, at most %lld are supported", (long long)(channels / groups),
                (long long)ssm::kNormMaxGroup);
  if (!(eps >= 0) || !std::isfinite(eps)) return fail(SSM_EINVAL, "eps must be finite and not negative");
  if ((center != 0 && center != 1) || (gate_first != 0 && gate_first != 1))
    return fail(SSM_EINVAL, "center and gate_first must be 0 or 1");
  int64_t n;
  if (!mul_ok(rows, channels, &n) || n > (int64_t(1) << 58)) return fail(SSM_EINVAL, "tensor sizes overflow");
  a->x = x; a->z = z; a->w = weight;
  a->rows = rows; a->channels = channels; a->groups = groups;
  a->eps = eps; a->center = center; a->gate_first = gate_first;
  if (ssm::norm_workgroups(*a, dtype == SSM_BF16) >= kMaxWorkgroups)
    return fail(SSM_EUNSUPPORTED, "too many workgroups for one launch");
  return SSM_OK;
}

int check_ranges(std::initializer_list<Range> ins, std::initializer_list<Range> outs) {
  for (const Range& r : ins)
    if (r.valid && r.lo % 16 != 0) return fail(SSM_EINVAL, "every pointer must be 16-byte aligned");
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    if (o->valid && o->lo % 16 != 0) return fail(SSM_EINVAL, "every pointer must be 16-byte aligned");
    for (const Range& r : ins)
      if (overlap(*o, r)) return fail(SSM_EINVAL, "outputs must not overlap inputs");
    for (const Range* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return fail(SSM_EINVAL, "outputs overlap each other");
  }
  return SSM_OK;
}

int check_workspace(const void* workspace, int64_t have, int64_t need) {
  if (need > 0 && (!workspace || have < need))
    return fail(SSM_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)(workspace ? have : 0), (long long)need);
  return SSM_OK;
}

int check_linear(ssm::LinearArgs* a, int64_t rows, int64_t k, int64_t m, int act, int dtype) {
  if (rows <= 0 || k <= 0 || m <= 0)
    return fail(SSM_EINVAL, "sizes must be positive (rows=%lld d_in=%lld d_out=%lld)", (long long)rows, (long long)k,
                (long long)m);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_EUNSUPPORTED, "dtype %d is not supported", dtype);
  if (act != ssm::kActNone && act != ssm::kActSilu && act != ssm::kActGelu)
    return fail(SSM_EINVAL, "unknown activation %d", act);
  // a tile's rows are addressed with 32-bit byte offsets
  if (k >= (int64_t(1) << 21) || m >= (int64_t(1) << 21))
    return fail(SSM_EUNSUPPORTED, "d_in=%lld and d_out=%lld must be under 2^21", (long long)k, (long long)m);
  if (rows > (int64_t(1) << 36)) return fail(SSM_EUNSUPPORTED, "rows=%lld is too large", (long long)rows);
  a->rows = rows; a->k = k; a->m = m; a->act = act;
  if (ssm::linear_workgroups(*a, dtype == SSM_BF16) >= kMaxWorkgroups)
    return fail(SSM_EUNSUPPORTED, "too many output tiles for one launch");
  return SSM_OK;
}

}  // namespace

extern "C" {

int ssm_gate_norm(const void* x, const void* z, const float* weight, void* y, int64_t rows, int64_t channels,
                  int64_t groups, float eps, int center, int gate_first, int dtype, void* stream) {
  g_err.clear();
  ssm::NormArgs a{};
  if (!y) return fail(SSM_EINVAL, "y must not be NULL");
  if (int rc = check_norm(&a, x, z, weight, rows, channels, groups, eps, center, gate_first, dtype)) return rc;
  const uint64_t n = uint64_t(rows) * channels * (dtype == SSM_BF16 ? 2 : 4);
  if (int rc = check_ranges({range_of(x, n), range_of(z, n), range_of(weight, uint64_t(channels) * 4)}, {range_of(y, n)}))
    return rc;
  a.y = y;
  const hipError_t e = ssm::launch_gate_norm(a, dtype == SSM_BF16, false, nullptr, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "gated norm launch");
  return SSM_OK;
}

int ssm_gate_norm_workspace(int64_t rows, int64_t channels, int64_t groups, int dtype, int64_t* bytes) {
  g_err.clear();
  if (!bytes) return fail(SSM_EINVAL, "bytes must not be NULL");
  ssm::NormArgs a{};
  float dummy = 0;
  if (int rc = check_norm(&a, &dummy, nullptr, nullptr, rows, channels, groups, 0.f, 0, 0, dtype)) return rc;
  a.dw = &dummy;
  *bytes = ssm::norm_workspace_bytes(a, dtype == SSM_BF16);
  return SSM_OK;
}

int ssm_gate_norm_bwd(const void* x, const void* z, const float* weight, const void* dy, void* dx, void* dz,
                      float* dweight, void* workspace, int64_t workspace_bytes, int64_t rows, int64_t channels,
                      int64_t groups, float eps, int center, int gate_first, int dtype, void* stream) {
  g_err.clear();
  ssm::NormArgs a{};
  if (!dy || !dx) return fail(SSM_EINVAL, "dy and dx must not be NULL");
  if ((z != nullptr) != (dz != nullptr)) return fail(SSM_EINVAL, "dz must be given if and only if z is");
  if (int rc = check_norm(&a, x, z, weight, rows, channels, groups, eps, center, gate_first, dtype)) return rc;
  a.dy = dy; a.dx = dx; a.dz = dz; a.dw = dweight;
  const int64_t need = ssm::norm_workspace_bytes(a, dtype == SSM_BF16);
  if (int rc = check_workspace(workspace, workspace_bytes, need)) return rc;
  const uint64_t n = uint64_t(rows) * channels * (dtype == SSM_BF16 ? 2 : 4), nw = uint64_t(channels) * 4;
  if (int rc = check_ranges({range_of(x, n), range_of(z, n), range_of(weight, nw), range_of(dy, n)},
                            {range_of(dx, n), range_of(dz, n), range_of(dweight, nw), range_of(workspace, uint64_t(need))}))
    return rc;
  const hipError_t e = ssm::launch_gate_norm(a, dtype == SSM_BF16, true, static_cast<float*>(workspace),
                                             static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "gated norm backward launch");
  return SSM_OK;
}

int ssm_linear_workspace(int64_t rows, int64_t d_in, int64_t d_out, int act, int dtype, int backward, int64_t* bytes) {
  g_err.clear();
  if (!bytes) return fail(SSM_EINVAL, "bytes must not be NULL");
  ssm::LinearArgs a{};
  if (int rc = check_linear(&a, rows, d_in, d_out, act, dtype)) return rc;
  a.dx = a.dw = a.dbias = bytes;  // all of them
  *bytes = ssm::linear_workspace_bytes(a, dtype == SSM_BF16, backward != 0);
  return SSM_OK;
}

int ssm_linear(const void* x, const void* W, const void* bias, const void* residual, int act, void* out, void* pre,
               void* workspace, int64_t workspace_bytes, int64_t rows, int64_t d_in, int64_t d_out, int dtype,
               void* stream) {
  g_err.clear();
  if (!x || !W || !out) return fail(SSM_EINVAL, "x, W and out must not be NULL");
  ssm::LinearArgs a{};
  if (int rc = check_linear(&a, rows, d_in, d_out, act, dtype)) return rc;
  a.x = x; a.w = W; a.bias = bias; a.residual = residual; a.out = out; a.pre = pre;
  const int64_t need = ssm::linear_workspace_bytes(a, dtype == SSM_BF16, false);
  if (int rc = check_workspace(workspace, workspace_bytes, need)) return rc;
  const uint64_t es = dtype == SSM_BF16 ? 2 : 4, nx = uint64_t(rows) * d_in * es, no = uint64_t(rows) * d_out * es;
  if (int rc = check_ranges({range_of(x, nx), range_of(W, uint64_t(d_in) * d_out * es), range_of(bias, uint64_t(d_out) * es),
                             range_of(residual, no)},
                            {range_of(out, no), range_of(pre, no), range_of(workspace, uint64_t(need))}))
    return rc;
  const hipError_t e = ssm::launch_linear(a, dtype == SSM_BF16, static_cast<char*>(workspace),
                                          static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "linear layer launch");
  return SSM_OK;
}

int ssm_linear_bwd(const void* x, const void* W, const void* pre, int act, const void* dout, void* dx, void* dW,
                   void* dbias, void* workspace, int64_t workspace_bytes, int64_t rows, int64_t d_in, int64_t d_out,
                   int dtype, void* stream) {
  g_err.clear();
  if (!x || !W || !dout) return fail(SSM_EINVAL, "x, W and dout must not be NULL");
  if (!dx && !dW && !dbias) return fail(SSM_EINVAL, "at least one of dx, dW and dbias must be given");
  ssm::LinearArgs a{};
  if (int rc = check_linear(&a, rows, d_in, d_out, act, dtype)) return rc;
  if (act != ssm::kActNone && !pre) return fail(SSM_EINVAL, "pre must be given with an activation");
  a.x = x; a.w = W; a.pre = const_cast<void*>(pre); a.dout = dout; a.dx = dx; a.dw = dW; a.dbias = dbias;
  const int64_t need = ssm::linear_workspace_bytes(a, dtype == SSM_BF16, true);
  if (int rc = check_workspace(workspace, workspace_bytes, need)) return rc;
  const uint64_t es = dtype == SSM_BF16 ? 2 : 4, nx = uint64_t(rows) * d_in * es, no = uint64_t(rows) * d_out * es;
  const uint64_t nw = uint64_t(d_in) * d_out * es;
  if (int rc = check_ranges({range_of(x, nx), range_of(W, nw), range_of(pre, no), range_of(dout, no)},
                            {range_of(dx, nx), range_of(dW, nw), range_of(dbias, uint64_t(d_out) * es),
                             range_of(workspace, uint64_t(need))}))
    return rc;
  const hipError_t e = ssm::launch_linear_bwd(a, dtype == SSM_BF16, static_cast<char*>(workspace),
                                              static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "linear layer backward launch");
  return SSM_OK;
}

}  // extern "C"
