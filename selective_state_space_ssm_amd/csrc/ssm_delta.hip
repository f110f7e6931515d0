// The delta scan: the head scan whose update takes out what the state holds
// under the key first,
//
//   S~_t = e^{g_t} S_{t-1},  r_t = v_t - S~_t^T k_t,  S_t = S~_t + b_t k_t r_t^T,  o_t = scale S_t^T q_t,
//
// its gradients and its step for single tokens.  The chunk kernels and their
// mathematics are in ssm_delta_kernel.h; here are the order of the passes, the
// carry over segments of the length and the step.
//
//   forwards   M of all chunks | [segments' own ends and transitions, carry] | the walk with the outputs
//   backwards  M, P | [segments, from the start and from the end, carries] | the walk that keeps the states and r beside
//              the one from the end that keeps R and e | all other gradients, all chunks at once | [sums over shared
//              heads]
//
// The walk is a chain of chunks; where batch rows, heads and column tiles leave
// CUs idle the length is cut into segments.  A segment makes A S + B of the state
// S before it: B is the walk from zero, A the walk from the identity without v,
// so that both come from the same kernel, and R before it is A^T R + B'.
//
// Page cited: [Mamba-2 page] "Mamba (part 2): parallel scan and
// hardware-aware optimisation" (scwacadex.pages.dev, blog8_mamba_parallel_scan)
// §4.3 on chunked recomputation, §7 on the constant-time step.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "ssm_delta_kernel.h"
#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

using namespace dev;
using deltak::DeltaDev;
using headk::f32x4;
using deltak::DeltaGradDev;

constexpr int64_t kDeltaCUs = 256;
constexpr int64_t kDeltaMinSegment = 3;   // chunks
constexpr int64_t kDeltaMaxSegments = 64;  // the carry's wavefronts hold something of each in a lane

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up(int64_t a, int64_t b) { return cdiv(a, b) * b; }
// Columns of a workgroup's tile: 128 in bfloat16 past 128 keys, where every operand row is whole vectors and tiles of 64
// are more than the CUs (LDS holds one workgroup either way, and with tiles of 64 a second round would be needed: 8 x 2048
// tokens, 32 heads of 192 x 128, forward and backward 499 and 2518 us, with tiles of 64 563 and 2706; 8 x 2048, 16 heads of
// 256 x 256 429 and 2398, 505 and 2584; 4 x 2048, 32 heads of 192 x 128 373 and 1422, 296 and 1381; 2 x 2048, 16 heads of
// 256 x 256 244 and 994, 229 and 710), else 64 (float32, the latter 538 and 1220, with 128 596 and 1811).
bool wide_for(int64_t rows, int64_t cols, int64_t bh, bool vec, bool bf16) {
  return bf16 && rows > 128 && cols > 64 && vec && bh * cdiv(cols, 64) > kDeltaCUs;
}
int64_t tiles_for(int64_t rows, int64_t cols, int64_t bh, bool vec, bool bf16) {
  return cdiv(cols, wide_for(rows, cols, bh, vec, bf16) ? 128 : 64);
}

// States carried over the segments, in order, 16 columns a workgroup: state <- A carried + own, or A^T carried + own
// from the end.  Float32 matrix instructions, 16 rows a wavefront; the carried columns are in LDS.  A segment's rows of
// A are asked for while the segment before is worked on: each operand takes its successor once it is used.  The column
// tiles of a head are a multiple of the heads apart, so that with 8 or more heads they share an XCD's L2 for A.  16 heads
// of 128 x 128 in 16 segments: 56 us, 4 a segment, from load to load.  A segment in which the state starts anew, or which
// has no tokens, takes no product (see kSegWhole).
template <int NW, bool REV>
__global__ void __launch_bounds__(64 * NW) ssm_delta_carry_kernel(float* state, const float* trans, const int* kinds, int nseg,
                                                                  int rp, int cp) {
  __shared__ float carried[16 * NW][17];
  const int64_t bh = blockIdx.x;
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = blockIdx.y * 16 + li, tiles = rp / 16, row = 16 * wave;
  const int64_t ws = static_cast<int64_t>(rp) * cp, ts = static_cast<int64_t>(rp) * rp;
  float* const s = state + bh * nseg * ws;
  const float* const m = trans + bh * nseg * ts;
  const int first = REV ? nseg - 1 : 0, step = REV ? -1 : 1;
  const bool mine = wave < tiles;
  const int kind_of_lane = lane < nseg ? kinds[bh * nseg + lane] : 0;  // of segment `lane`
  float4 f[NW];  // operand steps of 16 of A's columns
  auto load_a = [&](int at, int k) {
    if (!mine || k >= tiles) return;
    const Rsrc a = make_rsrc(m + at * ts, static_cast<uint32_t>(4 * ts));
    float* const o = reinterpret_cast<float*>(&f[k]);
    if constexpr (REV) {
#pragma unroll
      for (int e = 0; e < 4; ++e) BufF32::ld<1>(a, 4 * ((4 * g + e) * rp + row + li) + 64 * k * rp, o + e);
    } else {
      BufF32::ld<4>(a, 4 * ((row + li) * rp + 4 * g) + 64 * k, o);
    }
  };
  for (int i = tid; i < rp * 16; i += 64 * NW)
    carried[i / 16][i % 16] = s[first * ws + static_cast<int64_t>(i / 16) * cp + blockIdx.y * 16 + i % 16];
#pragma unroll
  for (int k = 0; k < NW; ++k) load_a(first + step, k);
  __syncthreads();
  for (int i = 1; i < nseg - 1; ++i) {
    const int at = first + i * step, next = i + 2 < nseg ? at + step : at;
    float* const own = s + at * ws;
    const int kind = __builtin_amdgcn_readlane(kind_of_lane, at);
    f32x4 acc = {0.f, 0.f, 0.f, 0.f}, sum[2] = {acc, acc};
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (mine) acc[v] = own[static_cast<int64_t>(row + 4 * g + v) * cp + c];
#pragma unroll
    for (int k = 0; k < NW; ++k) {
      if (k >= tiles) continue;
      const float4 x = make_float4(carried[16 * k + 4 * g][li], carried[16 * k + 4 * g + 1][li], carried[16 * k + 4 * g + 2][li],
                                   carried[16 * k + 4 * g + 3][li]);
      if (mine) sum[k & 1] = headk::mma<F32>(__builtin_bit_cast(uint4, f[k]), __builtin_bit_cast(uint4, x), sum[k & 1]);
      load_a(next, k);
    }
    __syncthreads();
    if (mine) {
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = row + 4 * g + v;
        float x = acc[v] + (sum[0][v] + sum[1][v]);
        if (kind == deltak::kSegAnew) x = acc[v];
        else if (kind == deltak::kSegEmpty) x = carried[r][li];
        carried[r][li] = x;
        own[static_cast<int64_t>(r) * cp + c] = x;
      }
    }
    __syncthreads();
  }
}

// One token.  A workgroup owns one (batch row, head) and 32 columns of the
// state: thread (rg, c) takes rows rg + 32 i, columns 4 c .. 4 c + 3.  With
// S~ = e^g S, both S~^T k and S~^T q come from one pass over the state's
// registers, with q . k: o = scale (S~^T q + (q . k) u), u = b (v - S~^T k), so
// that one exchange between the wavefronts serves both.  Every load is issued
// before the first store (the update may be in place).  Bound by the state's
// traffic: 256 sequences, 32 heads of 128 x 128 196 us, 5.5 TB/s, past what a
// copy reaches (4.9); eight workgroups a CU, whose registers allow it up to 128
// rows (with four 222 us).
struct DeltaStepDev {
  const char* q;
  const char* k;
  const char* v;
  const char* g;
  const char* beta;
  const float* in;
  float* out;
  char* o;
  int64_t H, Hk, dk, dv, ntile;
  float scale;
};

template <typename IO, int ROWS, bool VEC>
__global__ void __launch_bounds__(256, (ROWS == 256 || !VEC ? 4 : 8)) ssm_delta_step_kernel(DeltaStepDev p) {
  using B = typename BufOf<IO>::type;
  constexpr int N = ROWS / 32, ES = sizeof(typename IO::T);  // rows per thread
  constexpr uint32_t kOOB = headk::kOOB;
  __shared__ float sh[4][2][32], shq[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int dk = static_cast<int>(p.dk), dv = static_cast<int>(p.dv);
  const int64_t ct = blockIdx.x % p.ntile, bh = blockIdx.x / p.ntile, b = bh / p.H, h = bh % p.H;
  const int64_t hk = b * p.Hk + h / (p.H / p.Hk);
  const int c = static_cast<int>(ct) * 32 + 4 * (tid & 7), rg = tid >> 3;
  // resources bound the rows: nothing past them is read (it is zero) or written
  const Rsrc rin = make_rsrc(p.in + bh * p.dk * p.dv, static_cast<uint32_t>(dk * dv * 4));
  const Rsrc rq = make_rsrc(p.q + hk * p.dk * ES, static_cast<uint32_t>(dk * ES));
  const Rsrc rk = make_rsrc(p.k + hk * p.dk * ES, static_cast<uint32_t>(dk * ES));
  const Rsrc rv = make_rsrc(p.v + bh * p.dv * ES, static_cast<uint32_t>(dv * ES));
  const uint32_t off = static_cast<uint32_t>(rg * dv + c) * 4, step = static_cast<uint32_t>(32 * dv) * 4;
  float s[N][4], kk[N], qq[N], vv[4];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if constexpr (VEC) {
      const u32x4 x = __builtin_amdgcn_raw_buffer_load_b128(rin, c < dv ? off + i * step : kOOB, 0, kCacheNT);
      s[i][0] = __uint_as_float(x.x); s[i][1] = __uint_as_float(x.y);
      s[i][2] = __uint_as_float(x.z); s[i][3] = __uint_as_float(x.w);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) BufF32::ld<1>(rin, c + e < dv ? off + i * step + 4 * e : kOOB, &s[i][e]);
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    B::template ld<1>(rk, (rg + 32 * i) * ES, &kk[i]);
    B::template ld<1>(rq, (rg + 32 * i) * ES, &qq[i]);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) B::template ld<1>(rv, (c + e) * ES, &vv[e]);
  float a = 0.f, bt = 1.f;
  if (p.g != nullptr) IO::template ld<1>(reinterpret_cast<const typename IO::T*>(p.g) + bh, &a);
  if (p.beta != nullptr) IO::template ld<1>(reinterpret_cast<const typename IO::T*>(p.beta) + bh, &bt);
  a = __builtin_amdgcn_exp2f(headk::clamp_decay(a * kLog2e));
  float pk[4] = {0.f, 0.f, 0.f, 0.f}, pq[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    qk = __builtin_fmaf(qq[i], kk[i], qk);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s[i][e] = headk::times(a, s[i][e]);  // what is forgotten may not be finite
      pk[e] = __builtin_fmaf(kk[i], s[i][e], pk[e]);
      pq[e] = __builtin_fmaf(qq[i], s[i][e], pq[e]);
    }
  }
  // over the wavefront's 8 row groups, then over the wavefronts
#pragma unroll
  for (int d = 8; d < 64; d *= 2) {
    qk += __shfl_xor(qk, d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      pk[e] += __shfl_xor(pk[e], d);
      pq[e] += __shfl_xor(pq[e], d);
    }
  }
  if (lane < 8) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      sh[wave][0][4 * lane + e] = pk[e];
      sh[wave][1][4 * lane + e] = pq[e];
    }
    if (lane == 0) shq[wave] = qk;
  }
  __syncthreads();
  float u[4], y[4];
  qk = (shq[0] + shq[1]) + (shq[2] + shq[3]);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int x = 4 * (tid & 7) + e;
    u[e] = bt * (vv[e] - ((sh[0][0][x] + sh[1][0][x]) + (sh[2][0][x] + sh[3][0][x])));
    y[e] = p.scale * __builtin_fmaf(qk, u[e], (sh[0][1][x] + sh[1][1][x]) + (sh[2][1][x] + sh[3][1][x]));
  }
  const Rsrc rout = make_rsrc(p.out + bh * p.dk * p.dv, static_cast<uint32_t>(dk * dv * 4));
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int e = 0; e < 4; ++e) s[i][e] = __builtin_fmaf(kk[i], u[e], s[i][e]);
    if constexpr (VEC) {
      u32x4 x;
      x.x = __float_as_uint(s[i][0]); x.y = __float_as_uint(s[i][1]);
      x.z = __float_as_uint(s[i][2]); x.w = __float_as_uint(s[i][3]);
      __builtin_amdgcn_raw_buffer_store_b128(x, rout, c < dv ? off + i * step : kOOB, 0, kCacheNT);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) BufF32::st<1>(rout, c + e < dv ? off + i * step + 4 * e : kOOB, &s[i][e]);
    }
  }
  if (rg == 0) {
    const Rsrc ro = make_rsrc(p.o + bh * p.dv * ES, static_cast<uint32_t>(dv * ES));
#pragma unroll
    for (int e = 0; e < 4; ++e) B::template st<1>(ro, (c + e) * ES, &y[e]);
  }
}

struct Plan {
  int64_t C, nch, cps, nseg, rp, cp;
};
Plan plan_of(const DeltaArgs& a, bool bf16) {
  Plan p;
  p.C = bf16 ? headk::HeadCfg<BF16>::C : headk::HeadCfg<F32>::C;
  p.nch = cdiv(a.L, p.C);
  p.rp = up(a.dk, 16);
  p.cp = up(a.dv, deltak::kSlab);
  // The number of segments that the model below finds shortest, in chunks of a workgroup alone on its CU (4.2 us,
  // bfloat16, 128 x 128, M in two parts): two workgroups a CU take 1.75 of that (float32: 2, the matrix instructions bound it), the
  // segments' own walk 0.8, with the transitions' tiles beside the state's in all but the first, a step of the carry
  // 0.8, two more launches 3.  16 heads of 128 x 128 over 32768 tokens: 634 us in 16 segments, 637 in 8, 712
  // in 24, whole some 2.2 ms; 128 heads of 128 x 128 over 2048 tokens are better off whole.  A tenth has to be gained.
  const int64_t bh = a.batch * a.H, tv = tiles_for(a.dk, a.dv, bh, true, bf16);
  const int64_t tt = cdiv(p.rp, wide_for(a.dk, a.dv, bh, true, bf16) ? 128 : 64);
  const double pair = bf16 ? 1.75 : 2.;
  auto rate = [pair](double wgs) { return wgs <= kDeltaCUs ? 1. : std::max(pair, wgs * pair / (2 * kDeltaCUs)); };
  double best = 0.9 * p.nch * rate(bh * tv);
  int64_t want = 1;
  for (int64_t n = 2; n <= kDeltaMaxSegments && n * kDeltaMinSegment <= p.nch; ++n) {
    const double own = bh * ((n - 1) * tv + (n - 2) * tt);
    const double t = cdiv(p.nch, n) * (0.8 * rate(own) + rate(bh * n * tv)) + 0.8 * (n - 2) + 3;
    if (t < best) {
      best = t;
      want = n;
    }
  }
  p.cps = cdiv(p.nch, want);
  p.nseg = cdiv(p.nch, p.cps);
  return p;
}

// Every row of every operand is whole, aligned 16-byte vectors.
bool vec16(const void* p, int64_t b, int64_t t, int64_t es) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && b * es % 16 == 0 && t * es % 16 == 0;
}
bool all_vec(const DeltaArgs& a, bool bf16) {
  const int64_t es = bf16 ? 2 : 4;
  return a.dk * es % 16 == 0 && a.dv * es % 16 == 0 && vec16(a.q, a.q_b, a.q_t, es) && vec16(a.k, a.k_b, a.k_t, es) &&
         vec16(a.v, a.v_b, a.v_t, es);
}

// M (and, backwards, P) of every chunk, or forwards P
int64_t square_bytes(const DeltaArgs& a, const Plan& pl, bool bf16, bool query) {
  using deltak::Square;
  return a.batch * a.H * pl.nch * (bf16 ? (query ? Square<BF16, 2>::BYTES : Square<BF16, 3>::BYTES) : Square<F32, 1>::BYTES);
}

// Heads whose parts of dq and dk a workgroup adds: all that share a key head, unless that leaves CUs idle (4 x 2048
// tokens, 32 heads of 128 x 128 on 16 key heads, bfloat16: backward 583 us, with parts for every head 778, since
// float32 states 673; 2048 tokens,
// 16 heads of 64 x 64 on one: 105 us, with all in a workgroup 262), and one past 128 keys, where the sums do not fit the
// registers.
int64_t grad_heads(const DeltaArgs& a, const Plan& pl) {
  const int64_t rep = a.H / a.Hk;
  int64_t n = a.dk > 128 ? 1 : rep;
  while (n > 1 && a.batch * (a.H / n) * pl.nch < 2 * kDeltaCUs) {
    --n;
    while (rep % n != 0) --n;
  }
  return n;
}

// Where the workspace's parts are, in bytes from its start.
struct Space {
  int64_t m, s, rates, ss, rs, trans, kind, kept, pq, pk, total;
};
Space space_of(const DeltaArgs& a, const Plan& pl, bool bf16, bool backward) {
  Space w{};
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t r = at;
    at += up(bytes, 16);
    return r;
  };
  const int64_t bh = a.batch * a.H;
  w.m = take(square_bytes(a, pl, bf16, false));
  w.s = take(square_bytes(a, pl, bf16, !backward));
  w.rates = take(bh * pl.nch * pl.C * deltak::kRates * 4);
  if (pl.nseg > 1) {
    w.ss = take(4 * bh * pl.nseg * pl.rp * pl.cp);
    w.trans = take(4 * bh * pl.nseg * pl.rp * pl.rp);
    w.kind = take(4 * bh * pl.nseg);
    if (backward) w.rs = take(4 * bh * pl.nseg * pl.rp * pl.cp);
  }
  if (backward) {
    const int rp = static_cast<int>(pl.rp), cp = static_cast<int>(pl.cp);
    w.kept = take(bh * pl.nch * (bf16 ? deltak::Kept<BF16>(rp, cp).bytes() : deltak::Kept<F32>(rp, cp).bytes()));
    const int64_t hn = grad_heads(a, pl);
    if (hn < a.H / a.Hk) {
      w.pq = take(4 * bh / hn * a.L * a.dk);
      w.pk = take(4 * bh / hn * a.L * a.dk);
    }
  }
  w.total = at;
  return w;
}

DeltaDev dev_of(const DeltaArgs& a, const Plan& pl, const Space& w, char* work, bool bf16, bool vec) {
  const int64_t es = bf16 ? 2 : 4;
  DeltaDev d{};
  d.q = static_cast<const char*>(a.q); d.k = static_cast<const char*>(a.k); d.v = static_cast<const char*>(a.v);
  d.o = static_cast<char*>(a.o);
  d.q_b = a.q_b * es; d.k_b = a.k_b * es; d.v_b = a.v_b * es;
  d.q_t = static_cast<uint32_t>(a.q_t * es); d.k_t = static_cast<uint32_t>(a.k_t * es); d.v_t = static_cast<uint32_t>(a.v_t * es);
  d.rep = static_cast<int>(a.H / a.Hk);
  d.g = static_cast<const char*>(a.g); d.beta = static_cast<const char*>(a.beta); d.lengths = a.lengths;
  d.h0 = a.h0; d.last = a.last;
  d.m = work + w.m;
  d.s = work + w.s;
  d.rates = reinterpret_cast<float*>(work + w.rates);
  d.seg_state = reinterpret_cast<float*>(work + w.ss);
  d.seg_trans = reinterpret_cast<float*>(work + w.trans);
  d.seg_kind = reinterpret_cast<int*>(work + w.kind);
  d.kept = work + w.kept;
  d.batch = static_cast<int>(a.batch); d.H = static_cast<int>(a.H); d.L = static_cast<int>(a.L);
  d.rows = static_cast<int>(a.dk); d.cols = static_cast<int>(a.dv);
  d.rp = static_cast<int>(pl.rp); d.cp = static_cast<int>(pl.cp);
  d.nch = static_cast<int>(pl.nch); d.cps = static_cast<int>(pl.cps); d.nseg = static_cast<int>(pl.nseg);
  d.nvt = d.ntile = static_cast<int>(tiles_for(a.dk, a.dv, a.batch * a.H, vec, bf16));
  d.places = static_cast<int>(a.dk > 128 ? kDeltaCUs : 2 * kDeltaCUs);  // past 128 keys LDS has room for one a CU
  d.scale = a.scale;
  return d;
}

hipError_t launch_pass(const DeltaDev& d, const DeltaDev& r, bool bf16, int pass, bool vec, hipStream_t st) {
  return bf16 ? launch_delta_bf16(d, r, pass, wide_for(d.rows, d.cols, int64_t(d.batch) * d.H, vec, true), vec, st) : launch_delta_f32(d, r, pass, vec, st);
}

hipError_t launch_carry(const DeltaDev& d, bool rev, hipStream_t st) {
  if (d.nseg <= 2) return hipSuccess;
  const bool wide = d.rp > 128;
  auto kern = wide ? (rev ? ssm_delta_carry_kernel<16, true> : ssm_delta_carry_kernel<16, false>)
                   : (rev ? ssm_delta_carry_kernel<8, true> : ssm_delta_carry_kernel<8, false>);
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(d.batch * d.H), static_cast<unsigned>(d.cp / 16)), dim3(wide ? 1024 : 512),
                     0, st, d.seg_state, d.seg_trans, d.seg_kind, d.nseg, d.rp, d.cp);
  return hipGetLastError();
}

// with the tiles of the transitions
DeltaDev with_transitions(DeltaDev d, bool vec, bool bf16) {
  d.ntile = d.nvt + static_cast<int>(cdiv(d.rp, wide_for(d.rows, d.cols, int64_t(d.batch) * d.H, vec, bf16) ? 128 : 64));
  return d;
}

}  // namespace

int64_t delta_workspace_bytes(const DeltaArgs& a, bool bf16, bool backward) {
  return space_of(a, plan_of(a, bf16), bf16, backward).total;
}

int64_t delta_workgroups(const DeltaArgs& a, bool bf16, bool backward) {
  const Plan pl = plan_of(a, bf16);
  const int64_t bh = a.batch * a.H, tiles = cdiv(a.dv, 64) + cdiv(pl.rp, 64);
  return std::max(2 * bh * pl.nch, 4 * bh * tiles * pl.nseg);  // the larger workgroups have 512 threads
}

hipError_t launch_delta_fwd(const DeltaArgs& a, bool bf16, char* work, hipStream_t st) {
  const Plan pl = plan_of(a, bf16);
  const bool vec = all_vec(a, bf16);
  const DeltaDev d = dev_of(a, pl, space_of(a, pl, bf16, false), work, bf16, vec);
  if (pl.nch == 1 && d.ntile == 1 && !wide_for(d.rows, d.cols, a.batch * a.H, vec, bf16))  // that kernel's tile has 64 columns
    return launch_pass(d, d, bf16, deltak::kPassOne, vec, st);
  hipError_t e = launch_pass(d, d, bf16, deltak::kPassPrep, vec, st);
  if (e == hipSuccess && pl.nseg > 1) {
    e = launch_pass(with_transitions(d, vec, bf16), d, bf16, deltak::kPassSeg, vec, st);
    if (e == hipSuccess) e = launch_carry(d, false, st);
  }
  return e == hipSuccess ? launch_pass(d, d, bf16, deltak::kPassOut, vec, st) : e;
}

hipError_t launch_delta_bwd(const DeltaArgs& a, bool bf16, char* work, hipStream_t st) {
  const Plan pl = plan_of(a, bf16);
  const bool vec = all_vec(a, bf16);
  const Space w = space_of(a, pl, bf16, true);
  const int64_t es = bf16 ? 2 : 4;
  DeltaDev d = dev_of(a, pl, w, work, bf16, vec);
  d.last = nullptr;
  d.back = 1;
  DeltaDev r = d;
  r.v = static_cast<const char*>(a.dout);
  r.v_b = a.L * a.H * a.dv * es;
  r.v_t = static_cast<uint32_t>(a.H * a.dv * es);
  r.h0 = a.dlast;
  r.last = a.dh0;
  r.seg_state = reinterpret_cast<float*>(work + w.rs);
  hipError_t e = launch_pass(d, d, bf16, deltak::kPassPrep, vec, st);
  if (e == hipSuccess && pl.nseg > 1) {
    e = launch_pass(with_transitions(d, vec, bf16), r, bf16, deltak::kPassBothSeg, vec, st);
    if (e == hipSuccess) e = launch_carry(d, false, st);
    if (e == hipSuccess) e = launch_carry(r, true, st);
  }
  if (e == hipSuccess) e = launch_pass(d, r, bf16, deltak::kPassBoth, vec, st);
  if (e != hipSuccess) return e;

  const int64_t rep = a.H / a.Hk, hn = grad_heads(a, pl);
  DeltaGradDev gd{};
  gd.f = d;
  gd.f.v = r.v; gd.f.v_b = r.v_b; gd.f.v_t = r.v_t;
  gd.hn = static_cast<int>(hn);
  gd.parts = hn < rep;
  gd.dq = gd.parts ? work + w.pq : static_cast<char*>(a.dq);
  gd.dk = gd.parts ? work + w.pk : static_cast<char*>(a.dk_out);
  gd.dv = static_cast<char*>(a.dv_out);
  gd.dg = static_cast<char*>(a.dg);
  gd.db = static_cast<char*>(a.dbeta);
  e = bf16 ? launch_delta_grad_bf16(gd, vec, st) : launch_delta_grad_f32(gd, vec, st);
  if (e != hipSuccess || !gd.parts) return e;
  e = launch_head_group_sum(reinterpret_cast<const float*>(gd.dq), a.dq, a, hn, bf16, st);
  return e == hipSuccess ? launch_head_group_sum(reinterpret_cast<const float*>(gd.dk), a.dk_out, a, hn, bf16, st) : e;
}

namespace {

template <typename IO, bool VEC>
auto step_kernel(int64_t dk) {
  return dk <= 64 ? ssm_delta_step_kernel<IO, 64, VEC> : dk <= 128 ? ssm_delta_step_kernel<IO, 128, VEC>
                                                                   : ssm_delta_step_kernel<IO, 256, VEC>;
}

}  // namespace

hipError_t launch_delta_step(const DeltaStepArgs& a, bool bf16, hipStream_t st) {
  DeltaStepDev d{};
  d.q = static_cast<const char*>(a.q); d.k = static_cast<const char*>(a.k); d.v = static_cast<const char*>(a.v);
  d.g = static_cast<const char*>(a.g); d.beta = static_cast<const char*>(a.beta);
  d.in = a.state_in; d.out = a.state_out; d.o = static_cast<char*>(a.o);
  d.H = a.H; d.Hk = a.Hk; d.dk = a.dk; d.dv = a.dv; d.ntile = cdiv(a.dv, 32); d.scale = a.scale;
  const bool vec = a.dv % 4 == 0;
  auto kern = bf16 ? (vec ? step_kernel<BF16, true>(a.dk) : step_kernel<BF16, false>(a.dk))
                   : (vec ? step_kernel<F32, true>(a.dk) : step_kernel<F32, false>(a.dk));
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(a.batch * a.H * d.ntile)), dim3(256), 0, st, d);
  return hipGetLastError();
}

}  // namespace ssm
