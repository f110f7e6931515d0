// Host-side argument checks that the head scan's and the delta scan's entry
// points share (include/ssm_scan.h).
#pragma once

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "capi_common.h"
#include "ssm_kernels.h"
#include "ssm_scan.h"

namespace ssm {
namespace capi {

constexpr int64_t kLim31 = int64_t(1) << 31;
// a launch has fewer than 2^32 threads; 256 for every 64 columns of a head
constexpr int64_t kMaxWorkgroups = int64_t(1) << 24;

inline int check_head_sizes(int64_t batch, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv, int dtype) {
  if (batch <= 0 || L <= 0 || H <= 0 || Hk <= 0 || dk <= 0 || dv <= 0)
    return fail(SSM_EINVAL, "sizes must be positive (batch=%lld L=%lld n_heads=%lld n_qk_heads=%lld d_key=%lld d_value=%lld)",
                (long long)batch, (long long)L, (long long)H, (long long)Hk, (long long)dk, (long long)dv);
  if (dtype != SSM_F32 && dtype != SSM_BF16) return fail(SSM_EUNSUPPORTED, "dtype %d is not supported", dtype);
  if (H % Hk != 0)
    return fail(SSM_EINVAL, "n_heads=%lld must be a multiple of n_qk_heads=%lld", (long long)H, (long long)Hk);
  if (dk > kHeadMaxDim || dv > kHeadMaxDim)
    return fail(SSM_EUNSUPPORTED, "d_key=%lld and d_value=%lld must be at most %lld", (long long)dk, (long long)dv,
                (long long)kHeadMaxDim);
  int64_t bh, n;
  if (!mul_ok(batch, H, &bh) || !mul_ok(bh, L, &n) || !mul_ok(n, kHeadMaxDim, &n) || n > (int64_t(1) << 58))
    return fail(SSM_EINVAL, "tensor sizes overflow");
  if (L > (int64_t(1) << 30)) return fail(SSM_EUNSUPPORTED, "L=%lld > 2^30 is not supported", (long long)L);
  return SSM_OK;
}

inline int check_scan_sizes(int64_t batch, int64_t L, int64_t H, int64_t Hk, int64_t dk, int64_t dv, int dtype) {
  if (int rc = check_head_sizes(batch, L, H, Hk, dk, dv, dtype)) return rc;
  if (batch * H > 65535)
    return fail(SSM_EUNSUPPORTED, "batch * n_heads = %lld > 65535 is not supported", (long long)(batch * H));
  return SSM_OK;
}

// One token of every sequence: a workgroup for 32 columns of a head
inline int check_step_sizes(int64_t batch, int64_t H, int64_t Hk, int64_t dk, int64_t dv, int dtype) {
  if (int rc = check_head_sizes(batch, 1, H, Hk, dk, dv, dtype)) return rc;
  if (batch * H * ((dv + 31) / 32) >= kMaxWorkgroups) return fail(SSM_EUNSUPPORTED, "too many workgroups for one launch");
  return SSM_OK;
}

// A token-strided operand [batch][L][heads * width]: its strides, and the bytes it spans.  A stride over a size of one
// addresses nothing, but the kernels bound their loads by tokens times stride: it is replaced by the dense one.
inline int check_strides(const char* name, int64_t& b, int64_t& t, int64_t batch, int64_t L, int64_t row, int64_t es,
                  uint64_t* bytes) {
  if (L == 1) t = row;
  if (t < row) return fail(SSM_EINVAL, "%s: a token stride of %lld is less than its row of %lld", name, (long long)t,
                           (long long)row);
  // a chunk's rows are addressed with 32-bit byte offsets
  if (t >= kLim31 / 128 / es) return fail(SSM_EUNSUPPORTED, "%s: a token stride of %lld is too large", name, (long long)t);
  int64_t span, bspan;
  if (!mul_ok(L - 1, t, &span)) return fail(SSM_EINVAL, "tensor sizes overflow");
  span += row;
  if (batch == 1) b = L * t;
  if (batch > 1 && b < span) return fail(SSM_EINVAL, "%s: a batch stride of %lld is less than its %lld values", name,
                                         (long long)b, (long long)span);
  if (b < 0 || !mul_ok(batch - 1, b, &bspan) || !mul_ok(bspan + span, es, &bspan))
    return fail(SSM_EINVAL, "%s: strides overflow", name);
  *bytes = uint64_t(bspan);
  return SSM_OK;
}

inline int check_overlaps(std::initializer_list<Range> ins, std::initializer_list<Range> outs) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range& r : ins)
      if (overlap(*o, r)) return fail(SSM_EINVAL, "outputs must not overlap inputs");
    for (const Range* q = o + 1; q != outs.end(); ++q)
      if (overlap(*o, *q)) return fail(SSM_EINVAL, "outputs overlap each other");
  }
  return SSM_OK;
}

struct Spans {
  uint64_t q, k, v;
};

inline int check_operands(HeadArgs& a, int64_t es, Spans* s) {
  for (const void* q : {a.q, a.k, a.v, a.g})
    if (q && reinterpret_cast<uintptr_t>(q) % es != 0) return fail(SSM_EINVAL, "q, k, v and g must be aligned to their type");
  if (int rc = check_strides("q", a.q_b, a.q_t, a.batch, a.L, a.Hk * a.dk, es, &s->q)) return rc;
  if (int rc = check_strides("k", a.k_b, a.k_t, a.batch, a.L, a.Hk * a.dk, es, &s->k)) return rc;
  if (int rc = check_strides("v", a.v_b, a.v_t, a.batch, a.L, a.H * a.dv, es, &s->v)) return rc;
  if (a.H * (a.dv > a.dk ? a.dv : a.dk) * 4 >= kLim31 / 128)
    return fail(SSM_EUNSUPPORTED, "a token's row of %lld heads is too large", (long long)a.H);
  if (a.g && a.g_head) return fail(SSM_EINVAL, "give g or g_head, not both");
  if (!std::isfinite(a.scale)) return fail(SSM_EINVAL, "scale must be finite");
  return SSM_OK;
}

}  // namespace capi
}  // namespace ssm
