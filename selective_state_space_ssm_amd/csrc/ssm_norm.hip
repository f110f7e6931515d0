// Grouped norm of token rows with a SiLU gate (channels last), and its
// gradients.  A row of C channels is cut into `groups` groups of n channels;
// with mu the group's mean (0 without `center`), n^ the normalised values,
//
//   u = x            or x silu(z)  (gate first)
//   n^ = (u - mu) / sqrt(mean((u - mu)^2) + eps)
//   y = w n^ silu(z) or w n^
//
// Backward, with p = dy w (silu(z)) the gradient of n^ and r = 1 / sqrt(...):
//
//   du = r (p - [center] mean(p) - n^ mean(p n^))
//   gate last:   dx = du,          dz = dy w n^ silu'(z),   dw += dy n^ silu(z)
//   gate first:  dx = du silu(z),  dz = du x silu'(z),      dw += dy n^
//
// Bound by the memory traffic (one read of each input, one write of each
// output): a group's values stay in registers between the passes over them.
// Token rows being dense, group u of the flattened rows * groups is the n
// values from u n on.  LANES lanes share a group: the smallest power of two
// that covers it with one 16-byte vector per lane, a wavefront with two, a
// workgroup of 256 with up to eight beyond that (few registers a lane, so
// that many wavefronts' loads are in flight).  In the forward small groups are
// taken several at a time by the same lanes, for the same reason.  Groups that
// are no whole vectors take single values in the same shapes.
//
// Measured: 16384 x 4096 in 32 groups, bfloat16, 100 us (4.0 TB/s; one group at
// a time 142); 8191 x 1536 in one group, float32, forward 24 us and backward
// 44 (the backward with 64 lanes and eight vectors each: 124).  Single values are
// slower, 4096 rows of 5001 with the gate first 134 us in bfloat16 and 47 in
// float32 (5000: 29 and 37), backward 318 and 125 (110 and 108); above 4096 of
// them without a gate or with it last the forward's registers spill by the
// thousand: 3.1 and 4.1 ms.
//
// dw is a sum over rows: every workgroup of the backward walks rows of one
// group, keeps its sum in registers and leaves one float32 partial; a second
// launch adds the partials in order (the same bits on every call).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int64_t kBwdWorkgroups = 1024;  // four workgroups per CU

enum { kNoGate = 0, kGateLast = 1, kGateFirst = 2 };

struct NormDev {
  const char* x;
  const char* z;
  const float* w;
  const char* dy;
  char* y;          // y, or dx
  char* dz;
  float* part;      // [nsplit][C], nullable
  int64_t rows, groups, n;
  int64_t nsplit;   // workgroups that share a set of groups' rows (backward)
  float eps;
  int center;
};

// The E NV values of lane `l` of a group: vectors l, l + LANES, ... or, where rows are not 16-byte aligned, single
// values in the same manner.
template <typename IO, int LANES, int NV, bool VEC>
struct Group {
  static constexpr int E = 16 / static_cast<int>(sizeof(typename IO::T)), CNT = NV * E;
  static __device__ __forceinline__ int at(int l, int i) {
    return VEC ? ((i / E) * LANES + l) * E + i % E : i * LANES + l;
  }
  static __device__ __forceinline__ void load(const void* base, int64_t off, int l, int64_t n, float* o) {
    const typename IO::T* p = static_cast<const typename IO::T*>(base) + off;
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int c = (v * LANES + l) * E;
        if (c < n) {
          IO::template ld<E>(p + c, o + v * E);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) o[v * E + e] = 0.f;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < CNT; ++i) {
        o[i] = 0.f;
        if (at(l, i) < n) IO::template ld<1>(p + at(l, i), o + i);
      }
    }
  }
  // float32 values (16-byte aligned with VEC) at the same places
  static __device__ __forceinline__ void load_f32(const float* p, int l, int64_t n, float* o) {
    if constexpr (VEC) {
#pragma unroll
      for (int e = 0; e < CNT; e += 4) {
        const float4 v = at(l, e) < n ? *reinterpret_cast<const float4*>(p + at(l, e)) : make_float4(0.f, 0.f, 0.f, 0.f);
        o[e] = v.x; o[e + 1] = v.y; o[e + 2] = v.z; o[e + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < CNT; ++e) o[e] = at(l, e) < n ? p[at(l, e)] : 0.f;
    }
  }
  static __device__ __forceinline__ void store(void* base, int64_t off, int l, int64_t n, const float* o) {
    typename IO::T* p = static_cast<typename IO::T*>(base) + off;
    if constexpr (VEC) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if ((v * LANES + l) * E < n) IO::template st<E>(p + (v * LANES + l) * E, o + v * E);
    } else {
#pragma unroll
      for (int i = 0; i < CNT; ++i)
        if (at(l, i) < n) IO::template st<1>(p + at(l, i), o + i);
    }
  }
};

__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * z));
}

// Sum over the group's lanes; every lane gets it.
template <int LANES>
__device__ __forceinline__ float group_sum(float v, float* sh) {
#pragma unroll
  for (int d = 1; d < (LANES < 64 ? LANES : 64); d *= 2) v += __shfl_xor(v, d);
  if constexpr (LANES == 256) {
    __syncthreads();
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  }
  return v;
}

// u, its normalised values and 1 / sqrt(...): lanes past n hold zeros and stay out of the sums
template <typename IO, int LANES, int NV, bool VEC, int GATE>
__device__ __forceinline__ float normalise(const NormDev& p, int l, float* u, const float* s, float* sh) {
  using Gr = Group<IO, LANES, NV, VEC>;
  const float inv = 1.f / static_cast<float>(p.n);
  if constexpr (GATE == kGateFirst) {
#pragma unroll
    for (int i = 0; i < Gr::CNT; ++i) u[i] *= s[i];
  }
  if (p.center) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < Gr::CNT; ++i) m += u[i];
    m = group_sum<LANES>(m, sh) * inv;
#pragma unroll
    for (int i = 0; i < Gr::CNT; ++i) u[i] = Gr::at(l, i) < p.n ? u[i] - m : 0.f;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < Gr::CNT; ++i) q = __builtin_fmaf(u[i], u[i], q);
  q = group_sum<LANES>(q, sh) * inv;
  const float r = 1.f / __builtin_sqrtf(q + p.eps);
#pragma unroll
  for (int i = 0; i < Gr::CNT; ++i) u[i] *= r;
  return r;
}

// Groups that the same lanes take one after the other in the forward.
constexpr int norm_units(int lanes, int nv) { return lanes < 256 ? 4 / nv : 1; }

template <typename IO, int LANES, int NV, bool VEC, int GATE>
__global__ void __launch_bounds__(256) ssm_gate_norm_kernel(NormDev p) {
  using Gr = Group<IO, LANES, NV, VEC>;
  constexpr int U = norm_units(LANES, NV), PER = 256 / LANES;
  __shared__ float sh[4];
  const int l = threadIdx.x % LANES;
  const int64_t total = p.rows * p.groups;
  const int64_t u0 = static_cast<int64_t>(blockIdx.x) * (PER * U) + threadIdx.x / LANES;
  float x[U][Gr::CNT], s[U][Gr::CNT], w[Gr::CNT];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t u = u0 + i * PER;
    const int64_t n = u < total ? p.n : 0;  // nothing is read or written past the last group
    Gr::load(p.x, u * p.n, l, n, x[i]);
    if constexpr (GATE != kNoGate) Gr::load(p.z, u * p.n, l, n, s[i]);
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const int64_t u = u0 + i * PER, wo = (u % p.groups) * p.n;
    if (p.w != nullptr) Gr::load_f32(p.w + wo, l, p.n, w);
    if constexpr (GATE != kNoGate) {
#pragma unroll
      for (int e = 0; e < Gr::CNT; ++e) s[i][e] *= sigmoid(s[i][e]);
    }
    normalise<IO, LANES, NV, VEC, GATE>(p, l, x[i], s[i], sh);
    if (p.w != nullptr) {
#pragma unroll
      for (int e = 0; e < Gr::CNT; ++e) x[i][e] *= w[e];
    }
    if constexpr (GATE == kGateLast) {
#pragma unroll
      for (int e = 0; e < Gr::CNT; ++e) x[i][e] *= s[i][e];
    }
    Gr::store(p.y, u * p.n, l, u < total ? p.n : 0, x[i]);
  }
}

template <typename IO, int LANES, int NV, bool VEC, int GATE>
__global__ void __launch_bounds__(256) ssm_gate_norm_bwd_kernel(NormDev p) {
  using Gr = Group<IO, LANES, NV, VEC>;
  constexpr int PER = 256 / LANES;  // groups side by side in a workgroup
  __shared__ float sh[4];
  const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES;
  // workgroup (split, g0): groups g0 PER .. of rows split, split + nsplit, ...
  const int64_t ng = (p.groups + PER - 1) / PER;
  const int64_t g = (blockIdx.x % ng) * PER + sub, split = blockIdx.x / ng;
  const bool ok = g < p.groups;
  if (LANES < 256 && !ok) return;
  float w[Gr::CNT], dw[Gr::CNT];
#pragma unroll
  for (int i = 0; i < Gr::CNT; ++i) {
    w[i] = Gr::at(l, i) < p.n ? (p.w != nullptr ? p.w[g * p.n + Gr::at(l, i)] : 1.f) : 0.f;
    dw[i] = 0.f;
  }
  const float inv = 1.f / static_cast<float>(p.n);
  for (int64_t t = split; t < p.rows; t += p.nsplit) {
    const int64_t off = (t * p.groups + g) * p.n;
    float x[Gr::CNT], u[Gr::CNT], s[Gr::CNT], ds[Gr::CNT], dy[Gr::CNT];
    Gr::load(p.x, off, l, p.n, x);
    Gr::load(p.dy, off, l, p.n, dy);
    if constexpr (GATE != kNoGate) {
      float z[Gr::CNT];
      Gr::load(p.z, off, l, p.n, z);
#pragma unroll
      for (int i = 0; i < Gr::CNT; ++i) {
        const float sg = sigmoid(z[i]);
        s[i] = z[i] * sg;
        ds[i] = __builtin_fmaf(s[i], 1.f - sg, sg);
      }
    }
#pragma unroll
    for (int i = 0; i < Gr::CNT; ++i) u[i] = x[i];
    const float r = normalise<IO, LANES, NV, VEC, GATE>(p, l, u, s, sh);
    float m = 0.f, q = 0.f;
    float pn[Gr::CNT];
#pragma unroll
    for (int i = 0; i < Gr::CNT; ++i) {
      float d = dy[i];
      if constexpr (GATE == kGateLast) {
        ds[i] *= d * w[i] * u[i];  // dz
        d *= s[i];
      }
      dw[i] = __builtin_fmaf(d, u[i], dw[i]);
      pn[i] = d * w[i];
      m += pn[i];
      q = __builtin_fmaf(pn[i], u[i], q);
    }
    m = p.center ? group_sum<LANES>(m, sh) * inv : 0.f;
    q = group_sum<LANES>(q, sh) * inv;
#pragma unroll
    for (int i = 0; i < Gr::CNT; ++i) {
      float d = r * (pn[i] - m - u[i] * q);
      if constexpr (GATE == kGateFirst) {
        ds[i] *= d * x[i];  // dz
        d *= s[i];
      }
      pn[i] = d;
    }
    Gr::store(p.y, off, l, p.n, pn);
    if constexpr (GATE != kNoGate) Gr::store(p.dz, off, l, p.n, ds);
  }
  if (p.part != nullptr) {
#pragma unroll
    for (int i = 0; i < Gr::CNT; ++i)
      if (Gr::at(l, i) < p.n) p.part[(split * p.groups + g) * p.n + Gr::at(l, i)] = dw[i];
  }
}

// out[c] = sum over k of part[k][c], in order: 64 columns and 16 strands of k per workgroup
template <typename IO>
__global__ void __launch_bounds__(1024) ssm_column_sum_kernel(const float* part, int64_t count, int64_t cols, void* out) {
  __shared__ float sh[16][64];
  const int lane = threadIdx.x & 63, strand = threadIdx.x >> 6;
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 64 + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int64_t k = strand; k < count; k += 16) s += part[k * cols + c];
  }
  sh[strand][lane] = s;
  __syncthreads();
  if (strand == 0 && c < cols) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += sh[i][lane];
    IO::template st<1>(static_cast<typename IO::T*>(out) + c, &v);
  }
}

template <typename IO, int LANES, int NV, bool VEC>
hipError_t launch_norm_t(NormDev p, bool backward, int gate, hipStream_t st) {
  constexpr int PER = 256 / LANES;
  constexpr int64_t fwd = PER * norm_units(LANES, NV);
  const int64_t blocks = backward ? (p.groups + PER - 1) / PER * p.nsplit : (p.rows * p.groups + fwd - 1) / fwd;
  auto run = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, p);
    return hipGetLastError();
  };
  if (backward) {
    if (gate == kNoGate) return run(ssm_gate_norm_bwd_kernel<IO, LANES, NV, VEC, kNoGate>);
    if (gate == kGateLast) return run(ssm_gate_norm_bwd_kernel<IO, LANES, NV, VEC, kGateLast>);
    return run(ssm_gate_norm_bwd_kernel<IO, LANES, NV, VEC, kGateFirst>);
  }
  if (gate == kNoGate) return run(ssm_gate_norm_kernel<IO, LANES, NV, VEC, kNoGate>);
  if (gate == kGateLast) return run(ssm_gate_norm_kernel<IO, LANES, NV, VEC, kGateLast>);
  return run(ssm_gate_norm_kernel<IO, LANES, NV, VEC, kGateFirst>);
}

// Lanes per group and vectors per lane for n values of `es` bytes.
struct Shape {
  int lanes, nv;
};
Shape shape_of(int64_t n, int64_t es) {
  const int64_t vecs = (n * es + 15) / 16;
  Shape s{8, 1};
  while (s.lanes < 64 && s.lanes < vecs) s.lanes *= 2;
  if (s.lanes * 2 < vecs) s.lanes = 256;
  while (static_cast<int64_t>(s.lanes) * s.nv < vecs) s.nv *= 2;
  return s;
}

template <typename IO, bool VEC>
hipError_t launch_norm_v(const NormDev& p, Shape s, bool backward, int gate, hipStream_t st) {
  if (s.nv == 1) {
    if (s.lanes == 8) return launch_norm_t<IO, 8, 1, VEC>(p, backward, gate, st);
    if (s.lanes == 16) return launch_norm_t<IO, 16, 1, VEC>(p, backward, gate, st);
    if (s.lanes == 32) return launch_norm_t<IO, 32, 1, VEC>(p, backward, gate, st);
    if (s.lanes == 64) return launch_norm_t<IO, 64, 1, VEC>(p, backward, gate, st);
    return launch_norm_t<IO, 256, 1, VEC>(p, backward, gate, st);
  }
  if (s.lanes == 64) return launch_norm_t<IO, 64, 2, VEC>(p, backward, gate, st);
  if (s.nv == 2) return launch_norm_t<IO, 256, 2, VEC>(p, backward, gate, st);
  if (s.nv == 4) return launch_norm_t<IO, 256, 4, VEC>(p, backward, gate, st);
  // float32 only: 8192 values of bfloat16 are four vectors a lane
  if constexpr (std::is_same<IO, F32>::value) return launch_norm_t<IO, 256, 8, VEC>(p, backward, gate, st);
  return hipErrorInvalidValue;
}

int64_t bwd_splits(const NormArgs& a, int64_t es) {
  const Shape s = shape_of(a.channels / a.groups, es);
  const int64_t per = 256 / s.lanes, ng = (a.groups + per - 1) / per;
  int64_t n = kBwdWorkgroups / ng;
  if (n > a.rows) n = a.rows;
  return n < 1 ? 1 : n;
}

}  // namespace

int64_t norm_workspace_bytes(const NormArgs& a, bool bf16) {
  return a.dw == nullptr ? 0 : 4 * bwd_splits(a, bf16 ? 2 : 4) * a.channels;
}

int64_t norm_workgroups(const NormArgs& a, bool bf16) {
  const int64_t es = bf16 ? 2 : 4;
  const Shape s = shape_of(a.channels / a.groups, es);
  const int64_t per = 256 / s.lanes, fwd = per * norm_units(s.lanes, s.nv);
  const int64_t f = (a.rows * a.groups + fwd - 1) / fwd, b = (a.groups + per - 1) / per * bwd_splits(a, es);
  return f > b ? f : b;
}

hipError_t launch_column_sum(const float* part, int64_t count, int64_t cols, void* out, bool bf16, hipStream_t st) {
  auto kern = bf16 ? ssm_column_sum_kernel<BF16> : ssm_column_sum_kernel<F32>;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>((cols + 63) / 64)), dim3(1024), 0, st, part, count, cols, out);
  return hipGetLastError();
}

hipError_t launch_gate_norm(const NormArgs& a, bool bf16, bool backward, float* work, hipStream_t st) {
  const int64_t es = bf16 ? 2 : 4;
  NormDev p{};
  p.x = static_cast<const char*>(a.x); p.z = static_cast<const char*>(a.z); p.w = a.w;
  p.dy = static_cast<const char*>(a.dy);
  p.y = static_cast<char*>(backward ? a.dx : a.y); p.dz = static_cast<char*>(a.dz);
  p.rows = a.rows; p.groups = a.groups; p.n = a.channels / a.groups; p.eps = a.eps; p.center = a.center;
  p.nsplit = backward ? bwd_splits(a, es) : 1;
  p.part = backward && a.dw != nullptr ? work : nullptr;
  const int gate = a.z == nullptr ? kNoGate : (a.gate_first ? kGateFirst : kGateLast);
  const Shape s = shape_of(p.n, es);
  const bool vec = p.n * es % 16 == 0;
  hipError_t e = bf16 ? (vec ? launch_norm_v<BF16, true>(p, s, backward, gate, st)
                             : launch_norm_v<BF16, false>(p, s, backward, gate, st))
                      : (vec ? launch_norm_v<F32, true>(p, s, backward, gate, st)
                             : launch_norm_v<F32, false>(p, s, backward, gate, st));
  if (e == hipSuccess && p.part != nullptr) e = launch_column_sum(work, p.nsplit, a.channels, a.dw, false, st);
  return e;
}

}  // namespace ssm
