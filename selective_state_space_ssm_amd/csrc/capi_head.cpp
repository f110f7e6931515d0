// Host side of the head scan's entry points (include/ssm_scan.h): argument
// checks, all before any HIP call, and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "capi_head.h"
#include "ssm_kernels.h"
#include "ssm_scan.h"

using namespace ssm::capi;

extern "C" {

int ssm_head_scan_workspace(int64_t batch, int64_t L, int64_t n_heads, int64_t n_qk_heads, int64_t d_key,
                            int64_t d_value, int dtype, int backward, int64_t* bytes) {
  g_err.clear();
  if (!bytes) return fail(SSM_EINVAL, "bytes must not be NULL");
  if (int rc = check_scan_sizes(batch, L, n_heads, n_qk_heads, d_key, d_value, dtype)) return rc;
  ssm::HeadArgs a{};
  a.batch = batch; a.L = L; a.H = n_heads; a.Hk = n_qk_heads; a.dk = d_key; a.dv = d_value;
  *bytes = ssm::head_workspace_bytes(a, dtype == SSM_BF16, backward != 0);
  return SSM_OK;
}

int ssm_head_scan_fwd(const void* q, int64_t q_batch, int64_t q_token, const void* k, int64_t k_batch, int64_t k_token,
                      const void* v, int64_t v_batch, int64_t v_token, const void* g, const float* g_head,
                      const float* h0, const int32_t* lengths, float scale, void* o, float* last_state,
                      void* workspace, int64_t workspace_bytes, int64_t batch, int64_t L, int64_t n_heads,
                      int64_t n_qk_heads, int64_t d_key, int64_t d_value, int dtype, void* stream) {
  g_err.clear();
  if (!q || !k || !v || !o) return fail(SSM_EINVAL, "q, k, v and o must not be NULL");
  if (int rc = check_scan_sizes(batch, L, n_heads, n_qk_heads, d_key, d_value, dtype)) return rc;
  ssm::HeadArgs a{};
  a.q = q; a.q_b = q_batch; a.q_t = q_token; a.k = k; a.k_b = k_batch; a.k_t = k_token;
  a.v = v; a.v_b = v_batch; a.v_t = v_token;
  a.g = g; a.g_head = g_head; a.lengths = lengths; a.h0 = h0; a.o = o; a.last = last_state;
  a.batch = batch; a.L = L; a.H = n_heads; a.Hk = n_qk_heads; a.dk = d_key; a.dv = d_value; a.scale = scale;
  const bool bf16 = dtype == SSM_BF16;
  const int64_t es = bf16 ? 2 : 4;
  Spans s;
  if (int rc = check_operands(a, es, &s)) return rc;
  for (const void* r : {(const void*)g_head, (const void*)h0, (const void*)lengths, (const void*)o,
                        (const void*)last_state, (const void*)workspace})
    if (r && !aligned16(r)) return fail(SSM_EINVAL, "every dense pointer must be 16-byte aligned");
  const uint64_t nstate = uint64_t(batch) * n_heads * d_key * d_value * 4, nt = uint64_t(batch) * L * n_heads;
  const int64_t need = ssm::head_workspace_bytes(a, bf16, false);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(SSM_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)(workspace ? workspace_bytes : 0),
                (long long)need);
  if (ssm::head_workgroups(a, bf16, false) >= kMaxWorkgroups) return fail(SSM_EUNSUPPORTED, "too many workgroups for one launch");
  if (int rc = check_overlaps({range_of(q, s.q), range_of(k, s.k), range_of(v, s.v), range_of(g, nt * es),
                               range_of(g_head, uint64_t(n_heads) * 4), range_of(h0, nstate),
                               range_of(lengths, uint64_t(batch) * 4)},
                              {range_of(o, nt * d_value * es), range_of(last_state, nstate),
                               range_of(workspace, uint64_t(need))}))
    return rc;
  const hipError_t e = ssm::launch_head_fwd(a, bf16, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "head scan launch");
  return SSM_OK;
}

int ssm_head_scan_bwd(const void* q, int64_t q_batch, int64_t q_token, const void* k, int64_t k_batch, int64_t k_token,
                      const void* v, int64_t v_batch, int64_t v_token, const void* g, const float* g_head,
                      const float* h0, const int32_t* lengths, float scale, const void* dout, const float* dlast,
                      void* dq, void* dk, void* dv, void* dg, float* dh0, void* workspace, int64_t workspace_bytes,
                      int64_t batch, int64_t L, int64_t n_heads, int64_t n_qk_heads, int64_t d_key, int64_t d_value,
                      int dtype, void* stream) {
  g_err.clear();
  if (!q || !k || !v || !dout || !dq || !dk || !dv) return fail(SSM_EINVAL, "q, k, v, do, dq, dk and dv must not be NULL");
  if (int rc = check_scan_sizes(batch, L, n_heads, n_qk_heads, d_key, d_value, dtype)) return rc;
  if (dg && !g) return fail(SSM_EINVAL, "dg needs g");
  ssm::HeadArgs a{};
  a.q = q; a.q_b = q_batch; a.q_t = q_token; a.k = k; a.k_b = k_batch; a.k_t = k_token;
  a.v = v; a.v_b = v_batch; a.v_t = v_token;
  a.g = g; a.g_head = g_head; a.lengths = lengths; a.h0 = h0; a.dout = dout; a.dlast = dlast;
  a.dq = dq; a.dk_out = dk; a.dv_out = dv; a.dg = dg; a.dh0 = dh0;
  a.batch = batch; a.L = L; a.H = n_heads; a.Hk = n_qk_heads; a.dk = d_key; a.dv = d_value; a.scale = scale;
  const bool bf16 = dtype == SSM_BF16;
  const int64_t es = bf16 ? 2 : 4;
  Spans s;
  if (int rc = check_operands(a, es, &s)) return rc;
  for (const void* r : {(const void*)g_head, (const void*)h0, (const void*)lengths, dout, (const void*)dlast,
                        (const void*)dq, (const void*)dk, (const void*)dv, (const void*)dg, (const void*)dh0,
                        (const void*)workspace})
    if (r && !aligned16(r)) return fail(SSM_EINVAL, "every dense pointer must be 16-byte aligned");
  const uint64_t nstate = uint64_t(batch) * n_heads * d_key * d_value * 4, nt = uint64_t(batch) * L * n_heads;
  const uint64_t nqk = uint64_t(batch) * L * n_qk_heads * d_key * es, nv = nt * d_value * es;
  const int64_t need = ssm::head_workspace_bytes(a, bf16, true);
  if (!workspace || workspace_bytes < need)
    return fail(SSM_EINVAL, "workspace of %lld bytes, %lld are needed", (long long)(workspace ? workspace_bytes : 0),
                (long long)need);
  if (ssm::head_workgroups(a, bf16, true) >= kMaxWorkgroups) return fail(SSM_EUNSUPPORTED, "too many workgroups for one launch");
  if (int rc = check_overlaps({range_of(q, s.q), range_of(k, s.k), range_of(v, s.v), range_of(g, nt * es),
                               range_of(g_head, uint64_t(n_heads) * 4), range_of(h0, nstate),
                               range_of(lengths, uint64_t(batch) * 4), range_of(dout, nv), range_of(dlast, nstate)},
                              {range_of(dq, nqk), range_of(dk, nqk), range_of(dv, nv), range_of(dg, nt * es),
                               range_of(dh0, nstate), range_of(workspace, uint64_t(need))}))
    return rc;
  const hipError_t e = ssm::launch_head_bwd(a, bf16, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "head scan backward launch");
  return SSM_OK;
}

int ssm_head_step(const void* q, const void* k, const void* v, const void* g, const float* g_head, float scale,
                  const float* state_in, float* state_out, void* o, int64_t batch, int64_t n_heads, int64_t n_qk_heads,
                  int64_t d_key, int64_t d_value, int dtype, void* stream) {
  g_err.clear();
  if (!q || !k || !v || !state_in || !state_out || !o)
    return fail(SSM_EINVAL, "q, k, v, state_in, state_out and o must not be NULL");
  if (int rc = check_step_sizes(batch, n_heads, n_qk_heads, d_key, d_value, dtype)) return rc;
  if (g && g_head) return fail(SSM_EINVAL, "give g or g_head, not both");
  if (!std::isfinite(scale)) return fail(SSM_EINVAL, "scale must be finite");
  for (const void* r : {q, k, v, g, (const void*)g_head, (const void*)state_in, (const void*)state_out, (const void*)o})
    if (r && !aligned16(r)) return fail(SSM_EINVAL, "every pointer must be 16-byte aligned");
  const uint64_t es = dtype == SSM_BF16 ? 2 : 4, bh = uint64_t(batch) * n_heads;
  const uint64_t nqk = uint64_t(batch) * n_qk_heads * d_key * es, nstate = bh * d_key * d_value * 4;
  const Range rsi = range_of(state_in, nstate), rso = range_of(state_out, nstate), ro = range_of(o, bh * d_value * es);
  if (state_in != state_out && overlap(rsi, rso))
    return fail(SSM_EINVAL, "state_out must equal state_in or be disjoint from it");
  if (overlap(ro, rsi)) return fail(SSM_EINVAL, "o overlaps the state");
  if (int rc = check_overlaps({range_of(q, nqk), range_of(k, nqk), range_of(v, bh * d_value * es), range_of(g, bh * es),
                               range_of(g_head, uint64_t(n_heads) * 4)}, {ro, rso}))
    return rc;
  ssm::HeadStepArgs a{};
  a.q = q; a.k = k; a.v = v; a.g = g; a.g_head = g_head; a.state_in = state_in; a.state_out = state_out; a.o = o;
  a.batch = batch; a.H = n_heads; a.Hk = n_qk_heads; a.dk = d_key; a.dv = d_value; a.scale = scale;
  const hipError_t e = ssm::launch_head_step(a, dtype == SSM_BF16, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e, "head step launch");
  return SSM_OK;
}

}  // extern "C"
