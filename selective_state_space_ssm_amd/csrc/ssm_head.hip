// The head scan: a selective scan whose decay is one number per head and
// whose state is a matrix [d_key][d_value] (linear attention with a decay),
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t,
//
// its gradients and its step for single tokens.  With R_t = dLoss/dS_t,
//
//   R_t = scale q_t do_t^T + e^{g_{t+1}} R_{t+1}          (R_L += dlast)
//   dq_t = scale S_t do_t,  dk_t = R_t v_t,  dv_t = R_t^T k_t,  dh0 = e^{g_1} R_1
//
// each of which is the chunk kernel of ssm_head_kernel.h with other operands:
//
//            x    y    z    state           time
//   o        q    k    v    S   [dk][dv]    forwards
//   dq       do   v    k    S^T [dv][dk]    forwards
//   dk       v    do   q    R^T [dv][dk]    backwards
//   dv       k    q    do   R   [dk][dv]    backwards
//
// The gradient of the decays needs no pass of its own: <R_t, S_t> taken with
// either recurrence gives dg_t = dg_{t+1} + q_t . dq_t - k_t . dk_t, a sum
// from the end.  Both dots hold scale (q_t . k_t)(do_t . v_t), a token's own
// pair, which is all there is to them where little of the state outlasts a
// token: it is left out of both (with it in, its rounding was a tenth of dg at
// e^-12 a token).  The dq and dk passes hand out those dots in float32; the
// sum starts anew at every segment's end from <R, S> there, so that its
// rounding does not grow with the length, and from zero where the state does.
//
// Long sequences with few heads are cut into segments: every segment's own
// end state first (kState), then the states are carried over the segments
// (ssm_head_carry_kernel), then all segments at once from their start states.
//
// Page cited: [Mamba-2 page] "Mamba (part 2): parallel scan and
// hardware-aware optimisation" (scwacadex.pages.dev, blog8_mamba_parallel_scan)
// §4.3 on chunked recomputation, §7 on the constant-time step.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ssm_device.h"
#include "ssm_head_kernel.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

using namespace dev;
using headk::HeadDev;

// The length is split where there are fewer workgroups than CUs, into as many
// segments as give every CU two.  A split costs a second pass over y and z for
// the segments' states: 256 heads of 128 x 128 (8 x 2048 ragged tokens, bfloat16)
// take 151 us whole and 180 us in two segments; 16 heads over 65536 tokens 438 us
// in 32 segments, 489 in 48.  The backward's three passes share the segments'
// states: it is split for two workgroups per CU in any case (gradients of 4 x 2048
// tokens, 64 heads of 128 x 64: 737 us whole, 551 in two, 672 in three; float32,
// 4 x 1999, 24 heads of 64: 457 whole, 295 in five).
// How short a segment may be: its states take two passes whatever its length,
// and they are carried over the segments one after the other, so that the best
// number of segments grows like the root of the length (4 heads, 8000 tokens:
// bfloat16, 128 x 128, 47 us with the root's 42 segments, 55 with 31, 66 with
// 125).  Below that 64 tokens: float32, 100 x 48, 300 tokens 31 us, whole 51, 2757
// tokens 40, in segments of 256 73 (their gradients 114, 213).  bfloat16
// with more than 64 heads or fewer than six chunks is better off with 256
// (128 heads, 500 tokens 46 us, in segments of 64 or 128 tokens 53; few heads:
// 4, 500 tokens 27, 43).
constexpr int64_t kHeadCUs = 256;
constexpr int64_t kHeadSlots = 512;
constexpr int64_t kHeadSumWorkgroups = 8192;  // of the sums over shared heads, which go on from there
constexpr int64_t kHeadMinSegment = 64;       // tokens
constexpr int64_t kHeadMinSegmentMany = 256;
// Tokens that the running sum of dg covers: its terms are off by 2^-24 (float32)
// or 2^-17 (bfloat16, where dg itself is rounded to 2^-8) of themselves, and the
// sum's error grows like the root of their number.
constexpr int64_t kHeadMaxDgSegmentF32 = 1024;
constexpr int64_t kHeadMaxDgSegmentBf16 = 4096;

// States carried over the segments, in order: state <- decay * (carried) + own,
// or own alone where the state starts anew in the segment (a decay of -0; what
// was carried may not be finite).  Segment `first` holds its final state already.
__global__ void __launch_bounds__(256) ssm_head_carry_kernel(float* state, const float* decay, int64_t nseg, int64_t n,
                                                            int64_t ssize, int rev) {
  const int64_t bh = blockIdx.y, e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (e >= ssize) return;
  const int64_t step = rev ? -1 : 1, first = rev ? nseg - 1 : 0;
  float* s = state + bh * nseg * ssize + e;
  const float* d = decay + bh * nseg;
  float c = s[first * ssize];
#pragma unroll 4
  for (int64_t i = 1; i < n; ++i) {
    const int64_t at = first + i * step;
    const float own = s[at * ssize], dec = d[at];
    c = __float_as_uint(dec) == 0x80000000u ? own : __builtin_fmaf(dec, c, own);
    s[at * ssize] = c;
  }
}

// dg of one segment: <R, S> at its end, then the sum of q . dq - k . dk from the end.  Where the state starts anew
// (a decay of -inf) dg is zero, and so is what the tokens before it take over: their sum is begun there, so that no
// rounding of a packed sequence's dots enters those of the sequences before it.
template <typename IO>
__global__ void __launch_bounds__(256) ssm_head_dg_kernel(const float* s_seg, const float* r_seg, const float* s_last,
                                                         const float* dlast, const float* rq, const float* rk,
                                                         int64_t ntile, HeadDev p, int64_t seg_len, void* dg) {
  __shared__ double sh[4];
  __shared__ int sh_anew[4];
  const int64_t bh = blockIdx.y, k = blockIdx.x, b = bh / p.H, h = bh % p.H, ssize = static_cast<int64_t>(p.rows) * p.cols;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int64_t len = p.L;
  if (p.lengths != nullptr) {
    const int64_t n = p.lengths[b];
    len = n < 0 ? 0 : (n < p.L ? n : p.L);
  }
  const int64_t t0 = k * seg_len, t1 = t0 + seg_len < p.L ? t0 + seg_len : p.L;
  auto decay = [&](int64_t t) { return headk::decay_at<IO>(p, static_cast<int>(b), static_cast<int>(h), static_cast<int>(t)); };
  auto starts = [&](int64_t t) { return t < len && decay(t) == headk::kMinLog2Decay; };
  const float* S = k + 1 < p.nseg ? s_seg + (bh * p.nseg + k) * ssize : s_last + bh * ssize;
  const float* R = k + 1 < p.nseg ? r_seg + (bh * p.nseg + k + 1) * ssize : (dlast ? dlast + bh * ssize : nullptr);
  double x = 0;
  if (R != nullptr)
    for (int64_t i = tid; i < ssize; i += 256) x += static_cast<double>(R[i]) * S[i];
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  if (lane == 0) sh[wave] = x;
  __syncthreads();
  double carry = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  if (k + 1 < p.nseg && t1 < len) carry = starts(t1) ? 0. : carry * __builtin_amdgcn_exp2f(decay(t1));
  const int64_t nbh = static_cast<int64_t>(p.batch) * p.H;
  for (int64_t e = t1; e > t0; e -= 256) {
    const int64_t t = e - 1 - tid;  // thread 0 has the last token
    double v = 0;
    int anew = 0;  // the sum up to here begins at a token of these, not with what was carried
    if (t >= t0) {
      for (int64_t c = 0; c < ntile; ++c)
        v += static_cast<double>(rq[(c * nbh + bh) * p.L + t]) - rk[(c * nbh + bh) * p.L + t];
      anew = starts(t + 1);
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double o = __shfl_up(v, d);
      const int a = __shfl_up(anew, d);
      if (lane >= d) {
        if (!anew) v += o;
        anew |= a;
      }
    }
    __syncthreads();
    if (lane == 63) {
      sh[wave] = v;
      sh_anew[wave] = anew;
    }
    __syncthreads();
    double before = carry;
    for (int w = 0; w < wave; ++w) before = sh_anew[w] ? sh[w] : before + sh[w];
    for (int w = 0; w < 4; ++w) carry = sh_anew[w] ? sh[w] : carry + sh[w];
    if (t >= t0) {
      // nothing is decayed at the first token of a sequence that starts from zero, or where the state starts anew
      const bool none = t >= len || (t == 0 && p.h0 == nullptr) || starts(t);
      const float out = none ? 0.f : static_cast<float>(anew ? v : before + v);
      IO::template st<1>(static_cast<typename IO::T*>(dg) + (b * p.L + t) * p.H + h, &out);
    }
  }
}

// out[t][hk][e] = sum over the heads that share hk of part[t][h][e], V values a
// thread and turn.  The parts stay float32: 32 pairs of heads of 128 over 4 x 2048 tokens are
// 134 MB, 30 us to read (4.4 TB/s).
template <typename IO, int V>
__global__ void __launch_bounds__(256) ssm_head_group_sum_kernel(const float* part, void* out, int64_t n, int64_t d,
                                                                int64_t rep) {
  for (int64_t i = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V; i < n; i += static_cast<int64_t>(gridDim.x) * 256 * V) {
    const float* src = part + (i / d) * rep * d + i % d;
    float s[V] = {}, x[V];
#pragma unroll 8
    for (int64_t r = 0; r < rep; ++r) {
      F32::ld<V>(src + r * d, x);
#pragma unroll
      for (int e = 0; e < V; ++e) s[e] += x[e];
    }
    IO::template st<V>(static_cast<typename IO::T*>(out) + i, s);
  }
}

// One token.  A workgroup owns one (batch row, head) and 32 columns of the
// state: thread (rg, c) takes rows rg + 32 i, columns 4 c .. 4 c + 3.  Every
// load is issued before the first store (the update may be in place); the
// bound is the state's traffic, 8 bytes per value: 256 rows of 32 heads of 128 x
// 128 take 191 us, 5.6 TB/s.
struct HeadStepDev {
  const char* q;
  const char* k;
  const char* v;
  const char* g;
  const float* g_head;
  const float* in;
  float* out;
  char* o;
  int64_t H, Hk, dk, dv, ntile;
  float scale;
};

template <typename IO, bool VEC>
__global__ void __launch_bounds__(256) ssm_head_step_kernel(HeadStepDev p) {
  using T = typename IO::T;
  constexpr int kRows = 8;  // rows per thread: d_key <= 256
  __shared__ float sh[4][32];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t ct = blockIdx.x % p.ntile, bh = blockIdx.x / p.ntile, b = bh / p.H, h = bh % p.H;
  const int64_t c = ct * 32 + 4 * (tid & 7);
  const int rg = tid >> 3;
  const T* q = reinterpret_cast<const T*>(p.q) + (b * p.Hk + h / (p.H / p.Hk)) * p.dk;
  const T* k = reinterpret_cast<const T*>(p.k) + (b * p.Hk + h / (p.H / p.Hk)) * p.dk;
  const T* v = reinterpret_cast<const T*>(p.v) + bh * p.dv;
  float s[kRows][4], kk[kRows], qq[kRows], vv[4];
  const int64_t base = bh * p.dk * p.dv + c;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = rg + 32 * i;
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
    kk[i] = qq[i] = 0.f;
    if (r < p.dk) {
      if constexpr (VEC) {
        if (c < p.dv) {
          const headk::f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const headk::f32x4*>(p.in + base + r * p.dv));
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][e] = x[e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.dv) s[i][e] = p.in[base + r * p.dv + e];
      }
      IO::template ld<1>(k + r, &kk[i]);
      IO::template ld<1>(q + r, &qq[i]);
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    vv[e] = 0.f;
    if (c + e < p.dv) IO::template ld<1>(v + c + e, &vv[e]);
  }
  float a = 0.f;
  if (p.g != nullptr) {
    IO::template ld<1>(reinterpret_cast<const T*>(p.g) + bh, &a);
  } else if (p.g_head != nullptr) {
    a = p.g_head[h];
  }
  a = __builtin_amdgcn_exp2f(headk::clamp_decay(a * kLog2e));
  if (a == 0.f) {  // what is forgotten may not be finite
#pragma unroll
    for (int i = 0; i < kRows; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
  }
  float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t r = rg + 32 * i;
    if (r < p.dk) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[i][e] = __builtin_fmaf(a, s[i][e], kk[i] * vv[e]);
        o[e] = __builtin_fmaf(qq[i], s[i][e], o[e]);
      }
      if constexpr (VEC) {
        if (c < p.dv) {
          const headk::f32x4 x = {s[i][0], s[i][1], s[i][2], s[i][3]};
          __builtin_nontemporal_store(x, reinterpret_cast<headk::f32x4*>(p.out + base + r * p.dv));
        }
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c + e < p.dv) p.out[base + r * p.dv + e] = s[i][e];
      }
    }
  }
  // over the wavefront's 8 row groups, then over the wavefronts
#pragma unroll
  for (int e = 0; e < 4; ++e) {
#pragma unroll
    for (int d = 8; d < 64; d *= 2) o[e] += __shfl_xor(o[e], d);
    if (lane < 8) sh[wave][4 * lane + e] = o[e];
  }
  __syncthreads();
  if (tid < 32 && ct * 32 + tid < p.dv) {
    const float y = p.scale * ((sh[0][tid] + sh[1][tid]) + (sh[2][tid] + sh[3][tid]));
    IO::template st<1>(reinterpret_cast<T*>(p.o) + bh * p.dv + ct * 32 + tid, &y);
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

// Columns of a workgroup's tile: 128 where there are more than 64 and every
// operand row is whole vectors, else 64.
bool wide_for(int64_t cols, bool vec) { return cols > 64 && vec; }
int64_t tiles_for(int64_t cols, bool vec) { return cdiv(cols, wide_for(cols, vec) ? 128 : 64); }

struct Plan {
  int64_t C, nch, cps, nseg;
  bool vec;
};
Plan plan_of(int64_t batch, int64_t H, int64_t tiles, int64_t L, bool bf16, bool backward, bool vec) {
  Plan p;
  p.vec = vec;
  p.C = bf16 ? headk::HeadCfg<BF16>::C : headk::HeadCfg<F32>::C;
  p.nch = cdiv(L, p.C);
  const int64_t wgs = batch * H * tiles;
  int64_t want = backward || wgs < kHeadCUs ? kHeadSlots / wgs : 1;
  const int64_t least = bf16 && (want < 8 || p.nch < 6) ? kHeadMinSegmentMany : kHeadMinSegment;
  const int64_t most = std::min(L / least, static_cast<int64_t>(std::sqrt(static_cast<double>(L)) / 1.5));
  if (want > most) want = most;
  if (want < 1) want = 1;
  p.cps = cdiv(p.nch, want);
  const int64_t span = bf16 ? kHeadMaxDgSegmentBf16 : kHeadMaxDgSegmentF32;
  if (backward && p.cps * p.C > span) p.cps = span / p.C;
  p.nseg = cdiv(p.nch, p.cps);
  return p;
}

struct Operand {
  const void* p;
  int64_t b, t;
  int rep;
};

hipError_t launch_pass(const HeadDev& p, bool bf16, int mode, bool vec, hipStream_t st) {
  const bool wide = wide_for(p.cols, vec);
  return bf16 ? launch_head_bf16(p, mode, wide, vec, st) : launch_head_f32(p, mode, wide, vec, st);
}

// Every row of every operand is whole, aligned 16-byte vectors.
bool vec16(const void* p, int64_t b, int64_t t, int64_t es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && b * es % 16 == 0 && t * es % 16 == 0;
}
bool all_vec(const HeadArgs& a, bool bf16) {
  const int64_t es = bf16 ? 2 : 4;
  return a.dk * es % 16 == 0 && a.dv * es % 16 == 0 && vec16(a.q, a.q_b, a.q_t, es) && vec16(a.k, a.k_b, a.k_t, es) &&
         vec16(a.v, a.v_b, a.v_t, es);
}

// A pass' operands: x and y of width `rows`, z and the output of width `cols`.
HeadDev pass_of(const HeadArgs& a, const Plan& pl, const Operand& x, const Operand& y, const Operand& z, void* o,
                int64_t rows, int64_t cols, bool bf16) {
  const int64_t es = bf16 ? 2 : 4;
  HeadDev d{};
  d.x = static_cast<const char*>(x.p); d.y = static_cast<const char*>(y.p); d.z = static_cast<const char*>(z.p);
  d.o = static_cast<char*>(o);
  d.x_b = x.b * es; d.y_b = y.b * es; d.z_b = z.b * es;
  d.x_t = static_cast<uint32_t>(x.t * es); d.y_t = static_cast<uint32_t>(y.t * es); d.z_t = static_cast<uint32_t>(z.t * es);
  d.x_rep = x.rep; d.y_rep = y.rep; d.z_rep = z.rep;
  d.g = static_cast<const char*>(a.g); d.g_head = a.g_head; d.lengths = a.lengths;
  d.batch = static_cast<int>(a.batch); d.H = static_cast<int>(a.H); d.L = static_cast<int>(a.L);
  d.rows = static_cast<int>(rows); d.cols = static_cast<int>(cols);
  d.nch = static_cast<int>(pl.nch); d.cps = static_cast<int>(pl.cps); d.nseg = static_cast<int>(pl.nseg);
  d.ntile = static_cast<int>(tiles_for(cols, pl.vec));
  d.ps = d.ss = d.us = 1.f;
  return d;
}

hipError_t launch_carry(const HeadDev& d, hipStream_t st) {
  if (d.nseg <= 2) return hipSuccess;
  const int64_t ssize = static_cast<int64_t>(d.rows) * d.cols;
  hipLaunchKernelGGL(ssm_head_carry_kernel, dim3(static_cast<unsigned>(cdiv(ssize, 256)),
                                                 static_cast<unsigned>(d.batch * d.H)), dim3(256), 0, st, d.seg_state,
                     d.seg_decay, static_cast<int64_t>(d.nseg), static_cast<int64_t>(d.nseg - 1), ssize, d.rev);
  return hipGetLastError();
}

// Where the workspace's parts are, in bytes from its start.
struct FwdSpace {
  int64_t state, decay, total;
};
FwdSpace fwd_space(const HeadArgs& a, const Plan& pl) {
  FwdSpace w{};
  if (pl.nseg > 1) {
    w.decay = up16(4 * a.batch * a.H * pl.nseg * a.dk * a.dv);
    w.total = w.decay + up16(4 * a.batch * a.H * pl.nseg);
  }
  return w;
}
struct BwdSpace {
  int64_t s, r, sdec, rdec, slast, rq, rk, pq, pk, total;
};
BwdSpace bwd_space(const HeadArgs& a, const Plan& pl) {
  BwdSpace w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t r = at;
    at += up16(bytes);
    return r;
  };
  const int64_t bh = a.batch * a.H, ss = a.dk * a.dv, nt = tiles_for(a.dk, false);  // the narrower tiles: enough for both
  if (pl.nseg > 1) {
    w.s = take(4 * bh * pl.nseg * ss);
    w.r = take(4 * bh * pl.nseg * ss);
    w.sdec = take(4 * bh * pl.nseg);
    w.rdec = take(4 * bh * pl.nseg);
  }
  w.slast = take(4 * bh * ss);
  w.rq = take(4 * nt * bh * a.L);
  w.rk = take(4 * nt * bh * a.L);
  if (a.Hk != a.H) {
    w.pq = take(4 * bh * a.L * a.dk);
    w.pk = take(4 * bh * a.L * a.dk);
  }
  w.total = at;
  return w;
}
// The segments go by the sizes alone (the workspace's size is asked for without the operands).
Plan fwd_plan(const HeadArgs& a, bool bf16) {
  return plan_of(a.batch, a.H, tiles_for(a.dv, true), a.L, bf16, false, all_vec(a, bf16));
}
Plan bwd_plan(const HeadArgs& a, bool bf16) {
  const int64_t t1 = tiles_for(a.dv, true), t2 = tiles_for(a.dk, true);
  return plan_of(a.batch, a.H, t1 < t2 ? t1 : t2, a.L, bf16, true, all_vec(a, bf16));
}

// Heads whose parts of dq and dk a workgroup adds (kOutPair) where q and k are
// shared: two if that leaves every CU a workgroup.  Gradients of 4 x 2048 tokens,
// 64 heads of 128 x 64, bfloat16: 551 us (the two passes 147 each, their sums 30),
// one head a workgroup 619.
int64_t part_heads(const HeadArgs& a, const Plan& pl, bool bf16) {
  return bf16 && pl.vec && a.dv <= headk::kPairRows && a.H / a.Hk % 2 == 0 &&
                 a.batch * a.H / 2 * tiles_for(a.dk, true) * pl.nseg >= kHeadCUs
             ? 2
             : 1;
}

template <typename IO>
hipError_t launch_group_sum(const float* part, void* out, const HeadArgs& a, int64_t heads, hipStream_t st) {
  const int64_t n = a.batch * a.L * a.Hk * a.dk;
  const bool four = a.dk % 4 == 0;
  auto kern = four ? ssm_head_group_sum_kernel<IO, 4> : ssm_head_group_sum_kernel<IO, 1>;
  const int64_t wgs = std::min(cdiv(n, four ? 1024 : 256), kHeadSumWorkgroups);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(wgs)), dim3(256), 0, st, part, out, n, a.dk, a.H / a.Hk / heads);
  return hipGetLastError();
}

}  // namespace

int64_t head_workspace_bytes(const HeadArgs& a, bool bf16, bool backward) {
  return backward ? bwd_space(a, bwd_plan(a, bf16)).total : fwd_space(a, fwd_plan(a, bf16)).total;
}

int64_t head_workgroups(const HeadArgs& a, bool bf16, bool backward) {
  // a tile of 128 columns counts as two of 64
  auto tiles = [](int64_t cols) { return std::max(tiles_for(cols, false), cols > 64 ? 2 * tiles_for(cols, true) : 1); };
  return backward ? a.batch * a.H * std::max(tiles(a.dv), tiles(a.dk)) * bwd_plan(a, bf16).nseg
                  : a.batch * a.H * tiles(a.dv) * fwd_plan(a, bf16).nseg;
}

hipError_t launch_head_fwd(const HeadArgs& a, bool bf16, char* work, hipStream_t st) {
  const Plan pl = fwd_plan(a, bf16);
  const FwdSpace w = fwd_space(a, pl);
  const int rep = static_cast<int>(a.H / a.Hk);
  HeadDev d = pass_of(a, pl, {a.q, a.q_b, a.q_t, rep}, {a.k, a.k_b, a.k_t, rep}, {a.v, a.v_b, a.v_t, 1}, a.o, a.dk, a.dv,
                      bf16);
  d.ps = d.ss = a.scale;
  d.s_r = static_cast<int>(a.dv); d.s_c = 1;
  d.h0 = a.h0;
  d.last = a.last;
  d.seg_state = reinterpret_cast<float*>(work + w.state);
  d.seg_decay = reinterpret_cast<float*>(work + w.decay);
  if (pl.nseg > 1) {
    hipError_t e = launch_pass(d, bf16, headk::kState, pl.vec, st);
    if (e == hipSuccess) e = launch_carry(d, st);
    if (e != hipSuccess) return e;
  }
  return launch_pass(d, bf16, headk::kOut, pl.vec, st);
}

hipError_t launch_head_bwd(const HeadArgs& a, bool bf16, char* work, hipStream_t st) {
  const Plan pl = bwd_plan(a, bf16);
  const BwdSpace w = bwd_space(a, pl);
  const int rep = static_cast<int>(a.H / a.Hk);
  const bool shared = rep > 1, dg = a.dg != nullptr;
  const int64_t es = bf16 ? 2 : 4;
  const Operand q{a.q, a.q_b, a.q_t, rep}, k{a.k, a.k_b, a.k_t, rep}, v{a.v, a.v_b, a.v_t, 1};
  const Operand go{a.dout, a.L * a.H * a.dv, a.H * a.dv, 1};
  float* s_seg = reinterpret_cast<float*>(work + w.s);
  float* r_seg = reinterpret_cast<float*>(work + w.r);
  float* s_last = reinterpret_cast<float*>(work + w.slast);
  float* rq = reinterpret_cast<float*>(work + w.rq);
  float* rk = reinterpret_cast<float*>(work + w.rk);
  void* pq = shared ? static_cast<void*>(work + w.pq) : a.dq;
  void* pk = shared ? static_cast<void*>(work + w.pk) : a.dk_out;

  HeadDev dq = pass_of(a, pl, go, v, k, pq, a.dv, a.dk, bf16);
  dq.ps = dq.ss = a.scale;
  dq.s_r = 1; dq.s_c = static_cast<int>(a.dv);
  dq.h0 = a.h0;
  dq.seg_state = s_seg; dq.seg_decay = reinterpret_cast<float*>(work + w.sdec);
  dq.last = dg ? s_last : nullptr;

  HeadDev dv = pass_of(a, pl, k, q, go, a.dv_out, a.dk, a.dv, bf16);
  dv.ps = dv.us = a.scale;
  dv.s_r = static_cast<int>(a.dv); dv.s_c = 1;
  dv.rev = 1;
  dv.h0 = a.dlast;
  dv.seg_state = r_seg; dv.seg_decay = reinterpret_cast<float*>(work + w.rdec);
  dv.last = a.dh0; dv.end_decay = 1;

  HeadDev dk = pass_of(a, pl, v, go, q, pk, a.dv, a.dk, bf16);
  dk.ps = dk.us = a.scale;
  dk.s_r = 1; dk.s_c = static_cast<int>(a.dv);
  dk.rev = 1;
  dk.h0 = a.dlast;
  dk.seg_state = r_seg; dk.seg_decay = dv.seg_decay;

  // the float32 parts of shared heads come with their dots, wanted or not
  const int64_t heads = shared ? part_heads(a, pl, bf16) : 1;
  const int mode = !shared || !bf16 ? headk::kOut : (heads == 2 ? headk::kOutPair : headk::kOutF32);
  if (dg || mode != headk::kOut) {
    dq.dotv = static_cast<const char*>(a.q); dq.dot_b = a.q_b * es; dq.dot_t = static_cast<uint32_t>(a.q_t * es);
    dq.dot_rep = rep; dq.dot_out = rq;
    dk.dotv = static_cast<const char*>(a.k); dk.dot_b = a.k_b * es; dk.dot_t = static_cast<uint32_t>(a.k_t * es);
    dk.dot_rep = rep; dk.dot_out = rk;
  }
  hipError_t e = hipSuccess;
  if (pl.nseg > 1) {
    e = launch_pass(dq, bf16, headk::kState, pl.vec, st);
    if (e == hipSuccess) e = launch_carry(dq, st);
    if (e == hipSuccess) e = launch_pass(dv, bf16, headk::kState, pl.vec, st);
    if (e == hipSuccess) e = launch_carry(dv, st);
  }
  if (e == hipSuccess) e = launch_pass(dq, bf16, mode, pl.vec, st);
  if (e == hipSuccess) e = launch_pass(dk, bf16, mode, pl.vec, st);
  if (e == hipSuccess) e = launch_pass(dv, bf16, headk::kOut, pl.vec, st);
  if (e != hipSuccess) return e;
  if (dg) {
    auto kern = bf16 ? ssm_head_dg_kernel<BF16> : ssm_head_dg_kernel<F32>;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(pl.nseg), static_cast<unsigned>(a.batch * a.H)), dim3(256), 0, st,
                       s_seg, r_seg, s_last, a.dlast, rq, rk, static_cast<int64_t>(dq.ntile), dq, pl.cps * pl.C, a.dg);
    e = hipGetLastError();
  }
  if (e == hipSuccess && shared) {
    e = bf16 ? launch_group_sum<BF16>(static_cast<const float*>(pq), a.dq, a, heads, st)
             : launch_group_sum<F32>(static_cast<const float*>(pq), a.dq, a, heads, st);
    if (e == hipSuccess)
      e = bf16 ? launch_group_sum<BF16>(static_cast<const float*>(pk), a.dk_out, a, heads, st)
               : launch_group_sum<F32>(static_cast<const float*>(pk), a.dk_out, a, heads, st);
  }
  return e;
}

hipError_t launch_head_step(const HeadStepArgs& a, bool bf16, hipStream_t st) {
  HeadStepDev d{};
  d.q = static_cast<const char*>(a.q); d.k = static_cast<const char*>(a.k); d.v = static_cast<const char*>(a.v);
  d.g = static_cast<const char*>(a.g); d.g_head = a.g_head;
  d.in = a.state_in; d.out = a.state_out; d.o = static_cast<char*>(a.o);
  d.H = a.H; d.Hk = a.Hk; d.dk = a.dk; d.dv = a.dv; d.ntile = cdiv(a.dv, 32); d.scale = a.scale;
  const bool vec = a.dv % 4 == 0;
  auto kern = bf16 ? (vec ? ssm_head_step_kernel<BF16, true> : ssm_head_step_kernel<BF16, false>)
                   : (vec ? ssm_head_step_kernel<F32, true> : ssm_head_step_kernel<F32, false>);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(a.batch * a.H * d.ntile)), dim3(256), 0, st, d);
  return hipGetLastError();
}

}  // namespace ssm
