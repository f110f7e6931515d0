// Root-mean-square norm of token rows with the residual's addition in front of
// it, its output in the storage type or in 8 bits with scales, and its gradients:
//
//   h = x + residual                       (in the residual's type: the stream that goes on to the next block)
//   y = w h n,   n = 1 / sqrt(mean(h^2) + eps)
//   8 bits (e4m3): a scale s = amax |y| / 448 for each row or group of channels, y / s rounded
//
//   dx = dresidual = dh + n (p - h n mean(p h n)),  p = dy w;     dw = sum over rows of dy h n
//
// The norm acts on h as it is stored, so that the backward, which reads h, sees
// what the forward saw.  Sums and statistics are float32.
//
// Bound by the memory traffic: a row's values stay in registers between the pass
// that sums and the pass that writes.  LANES lanes share a row, each with up to
// four vectors of eight values (rows that are no whole vectors: single values in
// the same shapes).  16384 rows of 2048, bfloat16 with a float32 residual, to e4m3:
// 68 us, 5.4 TB/s, where a copy of 2 GiB reaches 4.9; forward and gradients 177 us,
// 4.5 TB/s.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

using namespace dev;

constexpr int E = 8;                      // values of a vector
constexpr float kE4m3Max = 448.f;

struct AddNormDev {
  const char* x;       // backward: dy
  const char* res;     // nullable; backward: h
  const float* w;      // nullable (ones)
  char* y;             // backward: dx, nullable
  char* h;             // nullable; backward: dresidual, nullable
  const char* dh;      // backward, nullable
  float* scale;        // 8 bits: [rows][n / group]
  float* part;         // backward: [workgroups][n], nullable
  int64_t rows, n;
  float eps;
  int group;           // channels per scale, n for a row's
};

// The rows that a workgroup works on side by side, as a buffer resource that bounds them; an offset past it for what is
// no channel.
constexpr uint32_t kOOB = 0x80000000u;
template <typename IO>
__device__ __forceinline__ Rsrc rows_of(const void* base, int64_t row, int64_t left, int per, int64_t n) {
  const int64_t es = sizeof(typename IO::T);
  return make_rsrc(static_cast<const char*>(base) + row * n * es,
                   static_cast<uint32_t>((left < per ? left : per) * n * es));
}

// The CNT values of lane l of a row that starts `off` values into the resource: vectors l, l + LANES, ..., or single
// values in the same manner.
template <int LANES, int NV, bool VEC>
struct Row {
  static constexpr int CNT = NV * E;
  static __device__ __forceinline__ int at(int l, int i) { return VEC ? ((i / E) * LANES + l) * E + i % E : i * LANES + l; }
  template <typename IO>
  static __device__ __forceinline__ void load(Rsrc r, uint32_t off, int l, int n, float* o) {
    constexpr int ES = sizeof(typename IO::T), V = VEC ? 16 / ES : 1;
#pragma unroll
    for (int i = 0; i < CNT; i += V) {
      const uint32_t to = at(l, i) < n ? (off + at(l, i)) * ES : kOOB;
      BufOf<IO>::type::template ld<V>(r, to, o + i);
    }
  }
  template <typename IO>
  static __device__ __forceinline__ void store(Rsrc r, uint32_t off, int l, int n, const float* o) {
    constexpr int ES = sizeof(typename IO::T), V = VEC ? 16 / ES : 1;
#pragma unroll
    for (int i = 0; i < CNT; i += V) {
      const uint32_t to = at(l, i) < n ? (off + at(l, i)) * ES : kOOB;
      BufOf<IO>::type::template st<V>(r, to, o + i);
    }
  }
};

// Reductions over a row's lanes, the result in every lane; sh is this reduction's own.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* sh) {
#pragma unroll
  for (int d = 1; d < (LANES < 64 ? LANES : 64); d *= 2) v += __shfl_xor(v, d);
  if constexpr (LANES == 256) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = (sh[0] + sh[1]) + (sh[2] + sh[3]);
  }
  return v;
}
template <int LANES>
__device__ __forceinline__ void row_sums(float& u, float& v, float (*sh)[4]) {
#pragma unroll
  for (int d = 1; d < (LANES < 64 ? LANES : 64); d *= 2) {
    u += __shfl_xor(u, d);
    v += __shfl_xor(v, d);
  }
  if constexpr (LANES == 256) {
    if ((threadIdx.x & 63) == 0) {
      sh[0][threadIdx.x >> 6] = u;
      sh[1][threadIdx.x >> 6] = v;
    }
    __syncthreads();
    u = (sh[0][0] + sh[0][1]) + (sh[0][2] + sh[0][3]);
    v = (sh[1][0] + sh[1][1]) + (sh[1][2] + sh[1][3]);
  }
}
// the larger, or no number where one of them is none
__device__ __forceinline__ float larger(float a, float b) { return a > b || a != a ? a : b; }
template <int LANES>
__device__ __forceinline__ float row_max(float v, float* sh) {
#pragma unroll
  for (int d = 1; d < (LANES < 64 ? LANES : 64); d *= 2) v = larger(v, __shfl_xor(v, d));
  if constexpr (LANES == 256) {
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = larger(larger(sh[0], sh[1]), larger(sh[2], sh[3]));
  }
  return v;
}

// Values up to amax to e4m3: what they are multiplied with, in two steps where 448 / amax would not be finite.
struct Quant {
  float up, by;
  __device__ __forceinline__ explicit Quant(float amax) {
    up = amax < 1e-30f ? 0x1p64f : 1.f;
    by = amax == 0.f ? 0.f : kE4m3Max / (amax * up);
  }
  __device__ __forceinline__ float operator()(float v) const { return v * up * by; }
};

template <typename XT, typename HT, int LANES, int NV, bool VEC, bool OUT8>
__global__ void __launch_bounds__(256) ssm_add_norm_kernel(AddNormDev p) {
  using R = Row<LANES, NV, VEC>;
  __shared__ float sh[2][4];
  constexpr int PER = 256 / LANES;
  const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES, n = static_cast<int>(p.n);
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * PER, left = p.rows - row0;
  const uint32_t off = static_cast<uint32_t>(sub * n);
  float h[R::CNT], w[R::CNT];
  R::template load<XT>(rows_of<XT>(p.x, row0, left, PER, n), off, l, n, h);
  if (p.res != nullptr) {
    R::template load<HT>(rows_of<HT>(p.res, row0, left, PER, n), off, l, n, w);
#pragma unroll
    for (int i = 0; i < R::CNT; ++i) h[i] += w[i];
  }
  if constexpr (std::is_same<HT, BF16>::value) {  // as it is stored
#pragma unroll
    for (int i = 0; i < R::CNT; i += 2) {
      const uint32_t u = BF16::cvt2(h[i], h[i + 1]);
      h[i] = bf_lo(u);
      h[i + 1] = bf_hi(u);
    }
  }
  if (p.h != nullptr) R::template store<HT>(rows_of<HT>(p.h, row0, left, PER, n), off, l, n, h);
  if (p.w != nullptr) R::template load<F32>(rows_of<F32>(p.w, 0, 1, 1, n), 0, l, n, w);
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < R::CNT; ++i) q = __builtin_fmaf(h[i], h[i], q);
  q = row_sum<LANES>(q, sh[0]) / static_cast<float>(p.n);
  const float r = 1.f / __builtin_sqrtf(q + p.eps);
#pragma unroll
  for (int i = 0; i < R::CNT; ++i) h[i] *= p.w != nullptr ? r * w[i] : r;
  if constexpr (!OUT8) {
    R::template store<XT>(rows_of<XT>(p.y, row0, left, PER, n), off, l, n, h);
  } else {
    const int64_t row = row0 + sub;
    const bool there = sub < left;
    float amax[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      amax[v] = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) amax[v] = larger(__builtin_fabsf(h[v * E + e]), amax[v]);
    }
    const Rsrc ry = make_rsrc(p.y + row0 * p.n, static_cast<uint32_t>((left < PER ? left : PER) * p.n));
    if (p.group == n) {
#pragma unroll
      for (int v = 1; v < NV; ++v) amax[0] = larger(amax[0], amax[v]);
      amax[0] = row_max<LANES>(amax[0], sh[1]);
      if (l == 0 && there) p.scale[row] = amax[0] / kE4m3Max;
#pragma unroll
      for (int v = 1; v < NV; ++v) amax[v] = amax[0];
    } else {
      // whole vectors (n is a multiple of the group): a group is four, eight or sixteen lanes side by side
      const int lanes = p.group / E;
      const int64_t per = n / p.group;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        for (int d = 1; d < lanes; d *= 2) amax[v] = larger(amax[v], __shfl_xor(amax[v], d));
        const int c = (v * LANES + l) * E;
        if (c < n && there && l % lanes == 0) p.scale[row * per + c / p.group] = amax[v] / kE4m3Max;
      }
    }
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const Quant f(amax[v]);
      if constexpr (VEC) {
        uint32_t u[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float* s = h + v * E + 4 * e;
          int t = __builtin_amdgcn_cvt_pk_fp8_f32(f(s[0]), f(s[1]), 0, false);
          u[e] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(f(s[2]), f(s[3]), t, true));
        }
        const int c = (v * LANES + l) * E;
        u32x2 w2;
        w2.x = u[0];
        w2.y = u[1];
        __builtin_amdgcn_raw_buffer_store_b64(w2, ry, c < n ? off + c : kOOB, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = R::at(l, v * E + e);
          __builtin_amdgcn_raw_buffer_store_b8(
              static_cast<uint8_t>(__builtin_amdgcn_cvt_pk_fp8_f32(f(h[v * E + e]), 0.f, 0, false)), ry, c < n ? off + c : kOOB, 0, 0);
        }
      }
    }
  }
}

// Rows blockIdx.x PER + sub, + gridDim.x PER, ...: the next row's values are asked for before the present one's sums.
template <typename XT, typename HT, int LANES, int NV, bool VEC>
__global__ void __launch_bounds__(256) ssm_add_norm_bwd_kernel(AddNormDev p) {
  using R = Row<LANES, NV, VEC>;
  constexpr int PER = 256 / LANES;
  __shared__ float sh[2][2][4];
  __shared__ float cols[LANES < 256 ? 256 * R::CNT : 1];
  const int l = threadIdx.x % LANES, sub = threadIdx.x / LANES, n = static_cast<int>(p.n);
  const uint32_t off = static_cast<uint32_t>(sub * n);
  float w[R::CNT], dw[R::CNT];
#pragma unroll
  for (int i = 0; i < R::CNT; ++i) {
    w[i] = 1.f;
    dw[i] = 0.f;
  }
  if (p.w != nullptr) R::template load<F32>(rows_of<F32>(p.w, 0, 1, 1, n), 0, l, n, w);
  const float inv = 1.f / static_cast<float>(p.n);
  float h[R::CNT], dy[R::CNT];
  const int64_t step = static_cast<int64_t>(gridDim.x) * PER, row0 = static_cast<int64_t>(blockIdx.x) * PER;
  auto load = [&](int64_t row) {
    R::template load<HT>(rows_of<HT>(p.res, row, p.rows - row, PER, n), off, l, n, h);
    R::template load<XT>(rows_of<XT>(p.x, row, p.rows - row, PER, n), off, l, n, dy);
  };
  load(row0);
  int turn = 0;
  for (int64_t first = row0; first < p.rows; first += step, turn ^= 1) {  // the same number of turns for all lanes
    const int64_t left = p.rows - first;
    float d[R::CNT], a[R::CNT], q = 0.f, m = 0.f;
    if (p.dh != nullptr) R::template load<HT>(rows_of<HT>(p.dh, first, left, PER, n), off, l, n, d);
#pragma unroll
    for (int i = 0; i < R::CNT; ++i) {
      if (p.dh == nullptr) d[i] = 0.f;
      a[i] = dy[i] * w[i];
      q = __builtin_fmaf(h[i], h[i], q);
      m = __builtin_fmaf(a[i], h[i], m);
    }
    row_sums<LANES>(q, m, sh[turn]);
    // lanes without a row give nothing to dw, with eps = 0 either
    const float r = sub < left ? 1.f / __builtin_sqrtf(q * inv + p.eps) : 0.f, by = r * r * (m * inv);
#pragma unroll
    for (int i = 0; i < R::CNT; ++i) {
      dw[i] = __builtin_fmaf(dy[i] * r, h[i], dw[i]);
      d[i] = __builtin_fmaf(r, __builtin_fmaf(-by, h[i], a[i]), d[i]);
    }
    if (first + step < p.rows) load(first + step);
    if (p.y != nullptr) R::template store<XT>(rows_of<XT>(p.y, first, left, PER, n), off, l, n, d);
    if (p.h != nullptr) R::template store<HT>(rows_of<HT>(p.h, first, left, PER, n), off, l, n, d);
  }
  if (p.part == nullptr) return;
  float* const part = p.part + blockIdx.x * p.n;
  if constexpr (LANES < 256) {
    // the rows side by side are added in order
#pragma unroll
    for (int i = 0; i < R::CNT; ++i) cols[i * 256 + threadIdx.x] = dw[i];
    __syncthreads();
    for (int i = threadIdx.x; i < R::CNT * LANES; i += 256) {
      const int e = i / LANES, k = i % LANES;
      float s = 0.f;
#pragma unroll
      for (int u = 0; u < PER; ++u) s += cols[e * 256 + u * LANES + k];
      if (R::at(k, e) < p.n) part[R::at(k, e)] = s;
    }
  } else {
#pragma unroll
    for (int i = 0; i < R::CNT; ++i)
      if (R::at(l, i) < p.n) part[R::at(l, i)] = dw[i];
  }
}

struct Shape {
  int lanes, nv;
};
// A wavefront takes up to 1024 values (no exchange through LDS), a workgroup more.  16384 rows of bfloat16 with a float32
// residual, 1024 channels: backward 53 us, with workgroups 57; 2048 channels: forward 78 and backward 106, with
// wavefronts 81 and 109; 4096 rows of 1536 in float32 17.3 and 24.8, 18.0 and 29.7.
Shape shape_of(int64_t n) {
  const int64_t vecs = (n + E - 1) / E;
  Shape s{8, 1};
  while (s.lanes < 64 && s.lanes < vecs) s.lanes *= 2;
  if (vecs > 128) s.lanes = 256;
  while (static_cast<int64_t>(s.lanes) * s.nv < vecs) s.nv *= 2;
  return s;
}

template <typename XT, typename HT, bool VEC>
hipError_t launch_fwd(const AddNormDev& p, bool out8, hipStream_t st) {
  const Shape s = shape_of(p.n);
  const int64_t blocks = (p.rows + 256 / s.lanes - 1) / (256 / s.lanes);
  auto run = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, st, p);
    return hipGetLastError();
  };
#define SSM_ADD_NORM(L, N)                                                                        \
  if (s.lanes == L && s.nv == N)                                                                  \
    return out8 ? run(ssm_add_norm_kernel<XT, HT, L, N, VEC, true>) : run(ssm_add_norm_kernel<XT, HT, L, N, VEC, false>);
  SSM_ADD_NORM(8, 1)
  SSM_ADD_NORM(16, 1)
  SSM_ADD_NORM(32, 1)
  SSM_ADD_NORM(64, 1)
  SSM_ADD_NORM(64, 2)
  SSM_ADD_NORM(256, 1)
  SSM_ADD_NORM(256, 2)
  SSM_ADD_NORM(256, 4)
#undef SSM_ADD_NORM
  return hipErrorInvalidValue;
}

// Three workgroups a CU: 16384 rows of 2048 in bfloat16 with a float32 residual 103 us, with two 109, four 106, eight 116;
// of 1024 50, 48, 53, 57; of 4096 without it 105, 104, 121, 122; 8191 of 768 in float32 21, 20, 23, 28.
int64_t bwd_blocks(int64_t rows, int64_t n) {
  const int64_t per = 256 / shape_of(n).lanes, need = (rows + per - 1) / per;
  return need < 768 ? need : 768;
}

template <typename XT, typename HT, bool VEC>
hipError_t launch_bwd(const AddNormDev& p, hipStream_t st) {
  const Shape s = shape_of(p.n);
  auto run = [&](auto kern) {
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(bwd_blocks(p.rows, p.n))), dim3(256), 0, st, p);
    return hipGetLastError();
  };
  if (s.lanes == 8) return run(ssm_add_norm_bwd_kernel<XT, HT, 8, 1, VEC>);
  if (s.lanes == 16) return run(ssm_add_norm_bwd_kernel<XT, HT, 16, 1, VEC>);
  if (s.lanes == 32) return run(ssm_add_norm_bwd_kernel<XT, HT, 32, 1, VEC>);
  if (s.lanes == 64 && s.nv == 1) return run(ssm_add_norm_bwd_kernel<XT, HT, 64, 1, VEC>);
  if (s.lanes == 64) return run(ssm_add_norm_bwd_kernel<XT, HT, 64, 2, VEC>);
  if (s.nv == 1) return run(ssm_add_norm_bwd_kernel<XT, HT, 256, 1, VEC>);
  if (s.nv == 2) return run(ssm_add_norm_bwd_kernel<XT, HT, 256, 2, VEC>);
  return run(ssm_add_norm_bwd_kernel<XT, HT, 256, 4, VEC>);
}

template <bool VEC>
hipError_t launch_types(const AddNormDev& p, bool bf16, bool res32, bool backward, bool out8, hipStream_t st) {
  if (!bf16) return backward ? launch_bwd<F32, F32, VEC>(p, st) : launch_fwd<F32, F32, VEC>(p, out8, st);
  if (res32) return backward ? launch_bwd<BF16, F32, VEC>(p, st) : launch_fwd<BF16, F32, VEC>(p, out8, st);
  return backward ? launch_bwd<BF16, BF16, VEC>(p, st) : launch_fwd<BF16, BF16, VEC>(p, out8, st);
}

}  // namespace

int64_t add_norm_workspace_bytes(int64_t rows, int64_t n) { return 4 * bwd_blocks(rows, n) * n; }

int64_t add_norm_workgroups(int64_t rows, int64_t n) {
  const int64_t per = 256 / shape_of(n).lanes;
  return (rows + per - 1) / per;
}

hipError_t launch_add_norm(const AddNormArgs& a, bool bf16, bool res32, bool out8, hipStream_t st) {
  AddNormDev p{};
  p.x = static_cast<const char*>(a.x); p.res = static_cast<const char*>(a.residual); p.w = a.w;
  p.y = static_cast<char*>(a.y); p.h = static_cast<char*>(a.h); p.scale = a.scale;
  p.rows = a.rows; p.n = a.n; p.eps = a.eps; p.group = static_cast<int>(a.group > 0 ? a.group : a.n);
  return a.n % E == 0 ? launch_types<true>(p, bf16, res32, false, out8, st)
                      : launch_types<false>(p, bf16, res32, false, out8, st);
}

hipError_t launch_add_norm_bwd(const AddNormArgs& a, bool bf16, bool res32, float* work, hipStream_t st) {
  AddNormDev p{};
  p.x = static_cast<const char*>(a.dy); p.res = static_cast<const char*>(a.h); p.w = a.w;
  p.dh = static_cast<const char*>(a.dh);
  p.y = static_cast<char*>(a.dx); p.h = static_cast<char*>(a.dres);
  p.part = a.dw != nullptr ? work : nullptr;
  p.rows = a.rows; p.n = a.n; p.eps = a.eps;
  hipError_t e = a.n % E == 0 ? launch_types<true>(p, bf16, res32, true, false, st)
                              : launch_types<false>(p, bf16, res32, true, false, st);
  if (e == hipSuccess && a.dw != nullptr) e = launch_column_sum(work, bwd_blocks(a.rows, a.n), a.n, a.dw, false, st);
  return e;
}

}  // namespace ssm
