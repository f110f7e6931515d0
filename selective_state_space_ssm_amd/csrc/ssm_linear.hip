// Linear layer on token rows with bias, activation and residual in its
// epilogue, and its gradients, on the matrix cores:
//
//   pre = x W^T + bias,  out = act(pre) + residual       x [T][K], W [M][K]
//   dpre = dout act'(pre)                                 (elementwise, with the column sums for dbias)
//   dx = dpre W,   dW = dpre^T x,   dbias = sum_t dpre
//
// All three products are one kernel: out[r][c] = sum_k R[r][k] C[c][k], each
// operand stored either with k contiguous or (template flags) with its rows
// contiguous:
//
//            r      c      k      R             C
//   out      token  m      k      x             W
//   dx       token  k      m      dpre          W, rows contiguous
//   dW       m      k      token  dpre, rows c. x, rows contiguous
//
// 16384 x 4096 -> 2048 in bfloat16 with gelu and residual: 289 us forward (950
// TFLOP/s; the epilogue's 200 MB come after the products, nothing covers them),
// dx 237, dW 222 (1240), dpre 43.  8192 x 4096 -> 2048 in float32: 131 TFLOP/s.
// Both are bound by the matrix instructions and what stands between them.
//
// The c side is the first operand of the matrix instruction, so that a lane
// holds four consecutive c of one r and the epilogue reads and writes them as
// one vector.
//
// A sum over k with few output tiles (dW over all tokens; few rows) is split
// over workgroups: float32 partials, added in a fixed order by a second launch
// that then holds the epilogue.
//
// Rows that are no whole number of 16-byte chunks are first copied to rows that
// are, zeros behind them (one small launch for both operands; dpre is written
// that way at once), and an odd number of outputs leaves through that second
// launch, so that every product reads aligned vectors and one set of tiles
// serves all sizes: 414 us for the forward and gradients of 8192 x 1001 -> 4096
// in bfloat16, against 1330 with element loads in the tiles and 790 with
// unaligned vector loads there.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "ssm_device.h"
#include "ssm_dma.h"
#include "ssm_kernels.h"

namespace ssm {
namespace {

using namespace dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kOOB = 0x80000000u;     // an offset past every resource
constexpr uint32_t kRecords = 0x7fffffffu;  // resources are bounded by the offsets' own checks
constexpr int64_t kCUs = 256;

template <typename IO>
struct LinCfg;
template <>
struct LinCfg<F32> {
  static constexpr int ES = 4, E = 4;  // bytes per value, values per 16 bytes
};
template <>
struct LinCfg<BF16> {
  static constexpr int ES = 2, E = 8;
};

constexpr float kLog2eLo = 1.9259629911e-8f;  // log2(e) - kLog2e

struct LinDev {
  const char* c;
  const char* r;
  char* out;                 // [nr][nc], or float32 partials [nsplit][nr][nc]
  int64_t nc, nr, K;
  int64_t ldc, ldr;          // elements between rows (k contiguous) or between k (rows contiguous)
  int64_t ldo;               // columns between rows of the partials
  int64_t kpart, nsplit;     // k per split (a multiple of the step)
  const char* bias;          // [nc], nullable
  const char* residual;      // [nr][nc], nullable
  char* pre;                 // [nr][nc], nullable
  int act;
};

// exp(-p^2 / 2).  An absolute error of the exponent is a relative one of the
// result, so that p^2 / 2 and its product with log2(e) are taken as hi + lo and
// the lo parts applied to the result (the plain float32 form is off by 1e-5 at p =
// -12).
__device__ __forceinline__ float gauss(float p) {
  const float h = 0.5f * p, q = h * p, ql = __builtin_fmaf(h, p, -q);
  const float e = q * kLog2e, el = __builtin_fmaf(q, kLog2eLo, __builtin_fmaf(q, kLog2e, -e));
  return __builtin_amdgcn_exp2f(-e) * (1.f - __builtin_fmaf(el, kLn2, ql));
}

// The normal distribution function, erfc(-p / sqrt 2) / 2, and exp(-p^2 / 2).
// Relative error below 1e-6 for every p (so that gelu keeps its digits in the
// tail): Chebyshev fit of log(erfc(z) exp(z^2) / t) in t = 1 / (1 + z / 2), z >= 0,
// to 1.2e-7 (W. H. Press et al., Numerical Recipes, "Incomplete Gamma Function,
// Error Function"), mirrored for p > 0; the rest are the roundings.
// For bfloat16, rounded to 2^-8 next, the plain exponential does: below 2e-5 down
// to p = -12 (forward of 16384 x 4096 -> 2048 with gelu and residual 270 us, with
// the other 278; dpre 36 and 38).
template <typename IO>
__device__ __forceinline__ float normal_cdf(float p, float* g) {
  // exp(-24^2 / 2) is far below the smallest float; further out p^2 is infinite and its lo part no number
  const float a = __builtin_fminf(__builtin_fabsf(p), 24.f);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.5f, 0.70710678118654752f * a, 1.f));
  float s = 0.17087277f;
  s = __builtin_fmaf(s, t, -0.82215223f);
  s = __builtin_fmaf(s, t, 1.48851587f);
  s = __builtin_fmaf(s, t, -1.13520398f);
  s = __builtin_fmaf(s, t, 0.27886807f);
  s = __builtin_fmaf(s, t, -0.18628806f);
  s = __builtin_fmaf(s, t, 0.09678418f);
  s = __builtin_fmaf(s, t, 0.37409196f);
  s = __builtin_fmaf(s, t, 1.00002368f);
  s = __builtin_fmaf(s, t, -1.26551223f);
  float e;
  if constexpr (std::is_same<IO, F32>::value) {
    *g = gauss(a);
    e = 0.5f * (t * __builtin_amdgcn_exp2f(kLog2e * s) * *g);
  } else {
    const float q = 0.5f * a * a;
    *g = __builtin_amdgcn_exp2f(-kLog2e * q);
    e = 0.5f * (t * __builtin_amdgcn_exp2f(kLog2e * (s - q)));
  }
  return p <= 0.f ? e : 1.f - e;
}

template <typename IO>
__device__ __forceinline__ float act_of(float p, int act) {
  if (act == kActSilu) return p * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * p));
  if (act == kActGelu) {
    float g;
    return p * normal_cdf<IO>(p, &g);
  }
  return p;
}

template <typename IO>
__device__ __forceinline__ float act_grad(float p, int act) {
  if (act == kActSilu) {
    const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * p));
    return s * __builtin_fmaf(p, 1.f - s, 1.f);
  }
  if (act == kActGelu) {
    float g;
    const float c = normal_cdf<IO>(p, &g);
    return __builtin_fmaf(p, 0.3989422804014327f * g, c);
  }
  return 1.f;
}

// CNT values of row r from column c on: bias, act, residual, rounding.
template <typename IO, int CNT>
__device__ __forceinline__ void epilogue(const LinDev& p, int64_t r, int64_t c, float* v) {
  using T = typename IO::T;
  const int64_t at = r * p.nc + c;
  float t[CNT];
  if (p.bias != nullptr) {
    IO::template ld<CNT>(reinterpret_cast<const T*>(p.bias) + c, t);
#pragma unroll
    for (int e = 0; e < CNT; ++e) v[e] += t[e];
  }
  if (p.pre != nullptr) IO::template st<CNT>(reinterpret_cast<T*>(p.pre) + at, v);
  if (p.act != kActNone) {
#pragma unroll
    for (int e = 0; e < CNT; ++e) v[e] = act_of<IO>(v[e], p.act);
  }
  if (p.residual != nullptr) {
    IO::template ld<CNT>(reinterpret_cast<const T*>(p.residual) + at, t);
#pragma unroll
    for (int e = 0; e < CNT; ++e) v[e] += t[e];
  }
  IO::template st<CNT>(reinterpret_cast<T*>(p.out) + at, v);
}

// ------------------------------------------------------------------------
// Tiles staged through registers, both types.  A workgroup of four
// wavefronts (2 x 2) owns 32 TC columns x 32 TR rows and walks k in steps of
// 128 bytes; LDS holds both operands with k contiguous (the rows-contiguous
// ones are transposed on the way in), double buffered, 16-byte chunk q of row
// r at q ^ swz(r).
// ------------------------------------------------------------------------
__device__ __forceinline__ int swz(int r) { return (r ^ (r >> 3)) & 7; }

template <typename IO, int ROWS, bool TR>
struct Stage {
  using C = LinCfg<IO>;
  static constexpr int E = C::E, ES = C::ES;
  static constexpr int N = TR ? E : ROWS / 32;  // 16-byte registers per thread
  uint4 reg[N];

  // rows row0 .. of `base` (nrows in all), k from k0, krem of them exist
  __device__ __forceinline__ void load(const char* base, int64_t ld, int64_t row0, int64_t nrows, int64_t k0, int krem,
                                       int tid) {
    if constexpr (!TR) {
      const int q = tid & 7, r0 = tid >> 3;
      const Rsrc rs = make_rsrc(base + (row0 * ld + k0) * ES, kRecords);
      const uint32_t rb = static_cast<uint32_t>(ld * ES);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = r0 + 32 * i;
        fetch(rs, static_cast<uint32_t>(r) * rb + q * 16, row0 + r < nrows && q * E < krem, reg[i]);
      }
    } else {
      constexpr int G = ROWS / E;  // row groups; 8 k groups
      const int tg = tid % G, kg = tid / G;
      const Rsrc rs = make_rsrc(base + (k0 * ld + row0) * ES, kRecords);
      const uint32_t kb = static_cast<uint32_t>(ld * ES);
      const bool rok = kg < 8 && row0 + tg * E < nrows;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int k = kg * E + i;
        fetch(rs, static_cast<uint32_t>(k) * kb + tg * 16, rok && k < krem, reg[i]);
      }
    }
  }
  static __device__ __forceinline__ void fetch(Rsrc rs, uint32_t off, bool ok, uint4& o) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, ok ? off : kOOB, 0, 0);
    o = make_uint4(v.x, v.y, v.z, v.w);
  }
  __device__ __forceinline__ void store(uint4* tile, int tid) const {
    if constexpr (!TR) {
      const int q = tid & 7, r0 = tid >> 3;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = r0 + 32 * i;
        tile[r * 8 + (q ^ swz(r))] = reg[i];
      }
    } else {
      constexpr int G = ROWS / E;
      const int tg = tid % G, kg = tid / G;
      if (kg >= 8) return;
#pragma unroll
      for (int j = 0; j < E; ++j) {
        uint32_t o[4];
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          if constexpr (ES == 2) {
            const uint32_t lo = reinterpret_cast<const uint32_t*>(&reg[2 * d])[j >> 1];
            const uint32_t hi = reinterpret_cast<const uint32_t*>(&reg[2 * d + 1])[j >> 1];
            o[d] = (j & 1) ? ((lo >> 16) | (hi & 0xffff0000u)) : ((lo & 0xffffu) | (hi << 16));
          } else {
            o[d] = reinterpret_cast<const uint32_t*>(&reg[d])[j];
          }
        }
        const int r = tg * E + j;
        tile[r * 8 + (kg ^ swz(r))] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
};

template <typename IO, int TC, int TR, bool CTR, bool RTR, bool PART>
__global__ void __launch_bounds__(256, 2) ssm_linear_tile_kernel(LinDev p) {
  using C = LinCfg<IO>;
  constexpr int E = C::E, ES = C::ES, BC = 32 * TC, BR = 32 * TR, BK = 8 * E;
  extern __shared__ uint4 lds[];  // [2][BC + BR][8]
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wc = wave & 1, wr = wave >> 1;

  const int64_t mc = (p.nc + BC - 1) / BC, mr = (p.nr + BR - 1) / BR;
  // XCD-contiguous order, c tiles fastest: the workgroups of an XCD share rows of R
  const int64_t G = gridDim.x, pid = blockIdx.x, q8 = G / 8, r8 = G % 8, xcd = pid % 8;
  int64_t idx = xcd * q8 + (xcd < r8 ? xcd : r8) + pid / 8;
  const int64_t c0 = idx % mc * BC;
  idx /= mc;
  const int64_t r0 = idx % mr * BR, split = idx / mr;
  const int64_t kb = split * p.kpart, ke = kb + p.kpart < p.K ? kb + p.kpart : p.K;

  Stage<IO, BC, CTR> sc;
  Stage<IO, BR, RTR> sr;
  auto load = [&](int64_t k0) {
    const int krem = ke - k0 > BK ? BK : static_cast<int>(ke - k0);
    sc.load(p.c, p.ldc, c0, p.nc, k0, krem, tid);
    sr.load(p.r, p.ldr, r0, p.nr, k0, krem, tid);
  };
  f32x4 acc[TC][TR];
#pragma unroll
  for (int i = 0; i < TC; ++i)
#pragma unroll
    for (int j = 0; j < TR; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int64_t steps = (ke - kb + BK - 1) / BK;
  if (steps > 0) {
    load(kb);
    sc.store(lds, tid);
    sr.store(lds + BC * 8, tid);
  }
  __syncthreads();
  for (int64_t s = 0; s < steps; ++s) {
    const uint4* tc = lds + (s & 1) * (BC + BR) * 8 + wc * (BC / 2) * 8;
    const uint4* tr = lds + (s & 1) * (BC + BR) * 8 + (BC + wr * (BR / 2)) * 8;
    if (s + 1 < steps) load(kb + (s + 1) * BK);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 fc[TC], fr[TR];
#pragma unroll
      for (int i = 0; i < TC; ++i) fc[i] = tc[(16 * i + li) * 8 + ((4 * h + g) ^ swz(16 * i + li + wc * (BC / 2)))];
#pragma unroll
      for (int j = 0; j < TR; ++j) fr[j] = tr[(16 * j + li) * 8 + ((4 * h + g) ^ swz(16 * j + li + wr * (BR / 2)))];
      if constexpr (ES == 2) {
#pragma unroll
        for (int i = 0; i < TC; ++i)
#pragma unroll
          for (int j = 0; j < TR; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fc[i]),
                                                                __builtin_bit_cast(bf16x8, fr[j]), acc[i][j], 0, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int i = 0; i < TC; ++i)
#pragma unroll
            for (int j = 0; j < TR; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                  __uint_as_float(reinterpret_cast<const uint32_t*>(&fc[i])[e]),
                  __uint_as_float(reinterpret_cast<const uint32_t*>(&fr[j])[e]), acc[i][j], 0, 0, 0);
      }
    }
    if (s + 1 < steps) {
      uint4* n = lds + ((s + 1) & 1) * (BC + BR) * 8;
      sc.store(n, tid);
      sr.store(n + BC * 8, tid);
    }
    __syncthreads();
  }

#pragma unroll
  for (int i = 0; i < TC; ++i) {
    const int64_t c = c0 + wc * (BC / 2) + 16 * i + 4 * g;
#pragma unroll
    for (int j = 0; j < TR; ++j) {
      const int64_t r = r0 + wr * (BR / 2) + 16 * j + li;
      if (r >= p.nr || c >= p.nc) continue;
      float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
      if constexpr (PART) {
        F32::st<4>(reinterpret_cast<float*>(p.out) + (split * p.nr + r) * p.ldo + c, v);
      } else {
        epilogue<IO, 4>(p, r, c, v);
      }
    }
  }
}

// ------------------------------------------------------------------------
// bfloat16, whole 16-byte chunks, large products: 256 x 256 tiles whose
// operands go from memory straight into LDS, four stages of 32 k, three of
// them in flight.
//
// A stage holds each operand as it is stored: k contiguous as [256 rows][32 k]
// (64-byte rows, chunk q of row r at q ^ ((r >> 1) & 3), read as they are), or
// rows contiguous as [32 k][256 rows] (512-byte rows, chunk q of row k at
// q ^ swz_kn(k), read with the transposing LDS read).  Both swizzles keep the
// reads free of bank conflicts, and are applied by choosing which chunk a lane
// fetches.
// ------------------------------------------------------------------------
constexpr int kStageK = 32;
constexpr int kStages = 4;
constexpr int kOperand = 256 * kStageK * 2;  // bytes of one operand's stage
constexpr int kStage = 2 * kOperand;
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

__device__ __forceinline__ int swz_kn(int k) { return 2 * ((k & 3) | (((k >> 3) & 1) << 2)); }

// One operand's share of the loads and reads of a workgroup of four wavefronts.
template <bool TR>
struct DmaSide {
  uint32_t voff[4];  // byte offset of this lane's chunk in block `wave` + 4 i of a stage, kOOB outside the rows
  int k[4];          // its first k in the stage
  uint64_t addr;     // the next stage's start
  uint64_t step;     // bytes to the one after
  int frag[TR ? 8 : 1];

  // rows row0 .. (nrows in all) from k0 on; the wavefront reads rows half * 128 .. of the tile
  __device__ __forceinline__ void init(const char* base, int64_t ld, int64_t row0, int64_t nrows, int64_t k0, int wave,
                                       int lane, int half) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = wave + 4 * i;  // 1 KB block
      if constexpr (!TR) {
        const int r = 16 * q + (lane >> 2), c = (lane & 3) ^ ((r >> 1) & 3);
        k[i] = 8 * c;
        voff[i] = row0 + r < nrows ? static_cast<uint32_t>(r * ld * 2 + 16 * c) : kOOB;
      } else {
        const int r = 2 * q + (lane >> 5), c = (lane & 31) ^ swz_kn(r);
        k[i] = r;
        voff[i] = row0 + 8 * c < nrows ? static_cast<uint32_t>(r * ld * 2 + 16 * c) : kOOB;
      }
    }
    addr = reinterpret_cast<uint64_t>(base) + static_cast<uint64_t>((TR ? k0 * ld + row0 : row0 * ld + k0) * 2);
    step = static_cast<uint64_t>(TR ? kStageK * ld * 2 : kStageK * 2);
    if constexpr (!TR) {
      frag[0] = (half * 128 + (lane & 15)) * 64 + 16 * ((lane >> 4) ^ (((lane & 15) >> 1) & 3));
    } else {
      const int kk = 8 * (lane >> 4) + ((lane & 15) >> 2);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        frag[j] = kk * 512 + 16 * (half * 16 + ((2 * j) ^ swz_kn(kk)) + ((lane >> 1) & 1)) + 8 * (lane & 1);
    }
  }
  // i-th of the four loads of the next stage into LDS at `lds`
  __device__ __forceinline__ void load(uint32_t lds, int wave, int i) const {
    dma16(dma_desc(reinterpret_cast<const void*>(addr), kRecords), voff[i], lds + (wave + 4 * i) * 1024);
  }
  // only krem k of the next stage exist, and none of those after it: what is past them reads zeros from here on
  __device__ __forceinline__ void end(int krem) {
#pragma unroll
    for (int i = 0; i < 4; ++i) voff[i] = k[i] < krem ? voff[i] : kOOB;
  }
  __device__ __forceinline__ uint4 read(const char* stage, int j) const {
    if constexpr (!TR) {
      return *reinterpret_cast<const uint4*>(stage + frag[0] + 1024 * j);
    } else {
      const v4i16 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(stage + frag[j]));
      const v4i16 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)(stage + frag[j] + 4 * 512));
      const uint2 l = __builtin_bit_cast(uint2, lo), h = __builtin_bit_cast(uint2, hi);
      return make_uint4(l.x, l.y, h.x, h.y);
    }
  }
};

// How a tile leaves: float32 partials, rounded values, or through the epilogue.
enum { kPart = 0, kPlain = 1, kFull = 2 };

template <bool CTR, bool RTR, int OUT>
__global__ void __launch_bounds__(256, 1) ssm_linear_dma_kernel(LinDev p) {
  __shared__ __attribute__((aligned(1024))) char stg[kStages][kStage];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wc = wave & 1, wr = wave >> 1;
  const int64_t mc = (p.nc + 255) / 256, mr = (p.nr + 255) / 256;
  const int64_t G = gridDim.x, pid = blockIdx.x, q8 = G / 8, r8 = G % 8, xcd = pid % 8;
  int64_t idx = xcd * q8 + (xcd < r8 ? xcd : r8) + pid / 8;
  const int64_t c0 = idx % mc * 256;
  idx /= mc;
  const int64_t r0 = idx % mr * 256, split = idx / mr;
  const int64_t kb = split * p.kpart, ke = kb + p.kpart < p.K ? kb + p.kpart : p.K;
  const int64_t nsteps = (ke - kb + kStageK - 1) / kStageK;

  DmaSide<CTR> sc;
  DmaSide<RTR> sr;
  sc.init(p.c, p.ldc, c0, p.nc, kb, wave, lane, wc);
  sr.init(p.r, p.ldr, r0, p.nr, kb, wave, lane, wr);
  int64_t left = ke - kb;  // k from the next stage on
  // a stage past the end is still issued (its loads read zeros), so that one count serves every wait
  auto before = [&]() {
    if (left < kStageK) {
      const int krem = left > 0 ? static_cast<int>(left) : 0;
      sc.end(krem);
      sr.end(krem);
    }
  };
  auto next = [&]() {
    left -= kStageK;
    sc.addr += sc.step;
    sr.addr += sr.step;
  };
  auto lds_of = [&](auto KS) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((lds_void*)stg[decltype(KS)::value]));
  };
  auto issue = [&](auto KS) {
    before();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      sc.load(lds_of(KS), wave, i);
      sr.load(lds_of(KS) + kOperand, wave, i);
    }
    next();
  };
  struct Frag {
    uint4 c[8], r[8];
  };
  auto read_c = [&](auto KS, Frag& f) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f.c[i] = sc.read(stg[decltype(KS)::value], i);
  };
  auto read_r = [&](auto KS, Frag& f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f.r[j] = sr.read(stg[decltype(KS)::value] + kOperand, j);
  };
  f32x4 acc[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // Step s: wait until stage s + 1 has landed (8 loads a wavefront and stage: vmcnt(8) leaves stage s + 2 in flight)
  // and this wavefront's reads of step s - 1 are done; barrier; then step s's 64 products.  What else the step issues,
  // the reads of step s + 1's operands and the refill of the stage read at step s - 1, stands between the first 32 of
  // them, so that it goes out while the matrix unit is busy and the reads have the other 32 to arrive: forward, dx and
  // dW of 16384 x 4096 -> 2048 take 0.87, 0.84 and 0.85 of the time that they took in four blocks between groups of 16
  // products, spread over 24 or all 32 pairs 0.88, 0.88 and 0.88.
  using S0 = std::integral_constant<int, 0>;
  using S1 = std::integral_constant<int, 1>;
  using S2 = std::integral_constant<int, 2>;
  using S3 = std::integral_constant<int, 3>;
  constexpr int kWait16 = 0 | (7 << 4) | (0 << 8) | (1 << 14);  // vmcnt(16) lgkmcnt(0)
  constexpr int kWait8 = 8 | (7 << 4) | (0 << 8);               // vmcnt(8) lgkmcnt(0)
  Frag F0, F1;
  issue(S0{});
  issue(S1{});
  issue(S2{});
  __builtin_amdgcn_s_waitcnt(kWait16);
  asm volatile("s_barrier" ::: "memory");
  read_c(S0{}, F0);
  read_r(S0{}, F0);
  auto step = [&](auto KR, auto KN, Frag& cur, Frag& nxt) {
    __builtin_amdgcn_s_waitcnt(kWait8);
    asm volatile("s_barrier" ::: "memory");
    before();
    const char* const from = stg[decltype(KN)::value];
#pragma unroll
    for (int t = 0; t < 32; ++t) {
#pragma unroll
      for (int m = 2 * t; m < 2 * t + 2; ++m)
        acc[m / 8][m % 8] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, cur.c[m / 8]),
                                                                    __builtin_bit_cast(bf16x8, cur.r[m % 8]),
                                                                    acc[m / 8][m % 8], 0, 0, 0);
      if (t < 16) {
        const int u = t;
        if (u < 8) nxt.c[u] = sc.read(from, u);
        else nxt.r[u - 8] = sr.read(from + kOperand, u - 8);
      }
      if (t < 16 && t % 2 == 0) {
        const int u = t / 2;
        if (u < 4) sc.load(lds_of(KR), wave, u);
        else sr.load(lds_of(KR) + kOperand, wave, u - 4);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    next();
  };
  for (int64_t s = 0; s < nsteps; s += 4) {
    step(S3{}, S1{}, F0, F1);
    if (s + 1 < nsteps) step(S0{}, S2{}, F1, F0);
    if (s + 2 < nsteps) step(S1{}, S3{}, F0, F1);
    if (s + 3 < nsteps) step(S2{}, S0{}, F1, F0);
  }
  // no load into LDS may still be in flight when the workgroup ends
  __builtin_amdgcn_s_waitcnt(0);

  if constexpr (OUT == kFull) {
    // The epilogue reads and writes whole 128-byte runs of a row: every wavefront passes its 128 x 128 sums through
    // its quarter of the LDS in two halves of 64 columns ([128 rows][16 chunks of 4 columns], chunk q of row r at
    // q ^ (r & 15)).  Straight from the accumulators it is 64 copies of the epilogue's code (the forward of 16384 x
    // 4096 -> 2048 with gelu and residual half as long again).
    // The residuals of eight rows a lane are in flight together.
    __syncthreads();
    float4* own = reinterpret_cast<float4*>(&stg[0][0]) + wave * 128 * 16;
    const int64_t rw = r0 + wr * 128, cwv = c0 + wc * 128, base = (rw * p.nc + cwv) * 2;
    const Rsrc rres = make_rsrc(p.residual + base, kRecords), rout = make_rsrc(p.out + base, kRecords);
    const Rsrc rpre = make_rsrc(p.pre + base, kRecords);
    const uint32_t row_bytes = static_cast<uint32_t>(p.nc * 2);
    const int rows = p.nr - rw > 128 ? 128 : static_cast<int>(p.nr - rw), lr = lane >> 3, lc = 8 * (lane & 7);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int r = 16 * j + (lane & 15);
          const f32x4 v = acc[4 * half + i][j];
          own[r * 16 + ((4 * i + (lane >> 4)) ^ (r & 15))] = make_float4(v[0], v[1], v[2], v[3]);
        }
      const bool cok = cwv + 64 * half + lc < p.nc;
      float bias[8] = {};
      if (p.bias != nullptr && cok) BF16::ld<8>(reinterpret_cast<const uint16_t*>(p.bias) + cwv + 64 * half + lc, bias);
#pragma unroll 1
      for (int k0 = 0; k0 < 128; k0 += 64) {
        u32x4 res[8];
        uint32_t off[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rl = k0 + 8 * k + lr;
          off[k] = cok && rl < rows ? static_cast<uint32_t>(rl) * row_bytes + 2 * (64 * half + lc) : kOOB;
          if (p.residual != nullptr) res[k] = __builtin_amdgcn_raw_buffer_load_b128(rres, off[k], 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rl = k0 + 8 * k + lr, q = 2 * (lane & 7);
          const float4 x = own[rl * 16 + (q ^ (rl & 15))], y = own[rl * 16 + ((q + 1) ^ (rl & 15))];
          float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] += bias[e];
          if (p.pre != nullptr) BufBF16::st<8>(rpre, off[k], v);
          if (p.act != kActNone) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = act_of<BF16>(v[e], p.act);
          }
          if (p.residual != nullptr) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] += e & 1 ? bf_hi(res[k][e >> 1]) : bf_lo(res[k][e >> 1]);
          }
          BufBF16::st<8>(rout, off[k], v);
        }
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t c = c0 + wc * 128 + 16 * i + 4 * (lane >> 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t r = r0 + wr * 128 + 16 * j + (lane & 15);
        if (r >= p.nr || c >= p.nc) continue;
        const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
        if constexpr (OUT == kPart) F32::st<4>(reinterpret_cast<float*>(p.out) + (split * p.nr + r) * p.ldo + c, v);
        else BF16::st<4>(reinterpret_cast<uint16_t*>(p.out) + r * p.nc + c, v);
      }
    }
  }
}

// Partials added in order, then the epilogue: a workgroup takes 64 CNT columns,
// one row a wavefront.
template <typename IO, int CNT>
__global__ void __launch_bounds__(256) ssm_linear_sum_kernel(const float* part, LinDev p) {
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63)) * CNT;
  if (c >= p.nc) return;
  for (int64_t r = static_cast<int64_t>(blockIdx.y) * 4 + (threadIdx.x >> 6); r < p.nr; r += 4 * gridDim.y) {
    float v[CNT], t[CNT];
    F32::ld<CNT>(part + r * p.ldo + c, v);
    for (int64_t s = 1; s < p.nsplit; ++s) {
      F32::ld<CNT>(part + (s * p.nr + r) * p.ldo + c, t);
#pragma unroll
      for (int e = 0; e < CNT; ++e) v[e] += t[e];
    }
    epilogue<IO, CNT>(p, r, c, v);
  }
}

// Rows of n values copied to rows of ld, whole chunks, zeros behind the n:
// blockIdx.z picks the operand, a thread writes 16 bytes of a row.
struct PackDev {
  const char* src[2];
  char* dst[2];
  int64_t rows[2], n[2], ld[2];
};
template <typename IO>
__global__ void __launch_bounds__(256) ssm_linear_pack_kernel(PackDev p) {
  using T = typename IO::T;
  constexpr int E = LinCfg<IO>::E;
  const int z = blockIdx.z;
  const int64_t n = p.n[z], c = (static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63)) * E;
  if (c >= p.ld[z]) return;
  for (int64_t r = static_cast<int64_t>(blockIdx.y) * 4 + (threadIdx.x >> 6); r < p.rows[z]; r += 4 * gridDim.y) {
    const T* const from = reinterpret_cast<const T*>(p.src[z]) + r * n + c;
    T v[E];
    if (c + E <= n) {
      __builtin_memcpy(v, from, 16);  // aligned to an element
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = c + e < n ? from[e] : T(0);
    }
    uint4 w;
    __builtin_memcpy(&w, v, 16);
    *reinterpret_cast<uint4*>(p.dst[z] + (r * p.ld[z] + c) * LinCfg<IO>::ES) = w;
  }
}

// Few rows (up to 16): one launch whose traffic is W's.  A workgroup of eight
// wavefronts owns COLS columns; wavefront w takes every eighth run of DEPTH steps of k, reads
// both operands straight from memory (a lane reads 16 bytes of one row of W and
// of x), and the eight partial 16 x 16 tiles meet in LDS.
// COLS = 8 (up to 8 rows): lanes 8 to 15 of a group of 16 hold the same columns
// and rows, one instruction's k further on, so that two diagonal quarters of
// the tile are halves of the sum and there are twice the workgroups: where 16
// columns give no more than every CU one, 8 x 4096 -> 2048 in bfloat16 takes 6.7
// us with 8 columns and 9.0 with 16 (W alone at the rate of a large copy: 3.5;
// the rest is the launch, one trip to memory and the sum through LDS).  With
// more columns 16 are at that rate: 8 x 4096 -> 8192 14.9 us, 4.5 TB/s.
template <typename IO, int COLS, bool VEC>
__global__ void __launch_bounds__(512) ssm_linear_rows_kernel(LinDev p) {
  using C = LinCfg<IO>;
  constexpr int E = C::E, ES = C::ES, BK = 4 * E, DEPTH = 8;  // k per instruction (chunk of four lanes), steps in flight
  using T = typename IO::T;
  constexpr int STEP = BK * 16 / COLS;
  __shared__ float part[8][16][17];
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = li / COLS, mine = li % COLS;
  const int64_t c0 = static_cast<int64_t>(blockIdx.x) * COLS;
  const char* const cbase = p.c + c0 * p.ldc * ES;
  const Rsrc rc = make_rsrc(cbase, kRecords), rr = make_rsrc(p.r, kRecords);
  const bool cok = c0 + mine < p.nc, rok = mine < p.nr;
  const uint32_t cb = static_cast<uint32_t>(mine * p.ldc * ES), rb = static_cast<uint32_t>(mine * p.ldr * ES);
  // what the epilogue adds is on its way during the products
  const int er = tid / COLS, ec = tid % COLS;
  const bool eok = er < COLS && er < p.nr && c0 + ec < p.nc;
  float bias = 0.f, res = 0.f;
  if (eok && p.bias != nullptr) IO::template ld<1>(reinterpret_cast<const T*>(p.bias) + c0 + ec, &bias);
  if (eok && p.residual != nullptr) IO::template ld<1>(reinterpret_cast<const T*>(p.residual) + er * p.nc + c0 + ec, &res);
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  // 16 bytes from p on, the first `have` values of them
  auto fetch = [&](Rsrc rs, const char* base, uint32_t off, int have) {
    uint4 o = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, have > 0 ? off : kOOB, 0, 0);
      o = make_uint4(v.x, v.y, v.z, v.w);
    } else if (have == E) {
      __builtin_memcpy(&o, base + off, 16);  // aligned to an element
    } else if (have > 0) {
      T v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = e < have ? reinterpret_cast<const T*>(base + off)[e] : T(0);
      __builtin_memcpy(&o, v, 16);
    }
    return o;
  };
  for (int64_t k0 = wave * STEP * DEPTH; k0 < p.K; k0 += 8 * STEP * DEPTH) {
    uint4 fc[DEPTH], fr[DEPTH];
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      const int64_t k = k0 + d * STEP + half * BK + g * E, left = p.K - k;
      const int have = left > E ? E : (left > 0 ? static_cast<int>(left) : 0);
      fc[d] = fetch(rc, cbase, cb + static_cast<uint32_t>(k * ES), cok ? have : 0);
      fr[d] = fetch(rr, p.r, rb + static_cast<uint32_t>(k * ES), rok ? have : 0);
    }
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if constexpr (ES == 2) {
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fc[d]), __builtin_bit_cast(bf16x8, fr[d]),
                                                      acc, 0, 0, 0);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(reinterpret_cast<const uint32_t*>(&fc[d])[e]),
                                                     __uint_as_float(reinterpret_cast<const uint32_t*>(&fr[d])[e]), acc, 0,
                                                     0, 0);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < 4; ++v) part[wave][li][4 * g + v] = acc[v];
  __syncthreads();
  if (eok) {
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w)
      v += COLS == 16 ? part[w][er][ec] : part[w][er][ec] + part[w][8 + er][8 + ec];
    v += bias;
    const int64_t at = er * p.nc + c0 + ec;
    if (p.pre != nullptr) IO::template st<1>(reinterpret_cast<T*>(p.pre) + at, &v);
    v = act_of<IO>(v, p.act) + res;
    IO::template st<1>(reinterpret_cast<T*>(p.out) + at, &v);
  }
}

// dpre = dout act'(pre), and its column sums over this workgroup's rows (into
// dbias where it has them all): thread (cv, rr) takes CNT columns of rows rr,
// rr + 8, ...  dpre's rows (none: it is not kept) are ld long, zeros behind m.
template <typename IO, int CNT>
__global__ void __launch_bounds__(256) ssm_linear_dpre_kernel(const void* dout, const void* pre, void* dpre, float* part,
                                                             void* dbias, int64_t rows, int64_t m, int64_t ld,
                                                             int64_t per, int act) {
  using T = typename IO::T;
  __shared__ float sh[8][32 * CNT];
  const int cv = threadIdx.x & 31, rr = threadIdx.x >> 5;
  const int64_t c = (static_cast<int64_t>(blockIdx.x) * 32 + cv) * CNT;
  const int64_t t0 = blockIdx.y * per, t1 = t0 + per < rows ? t0 + per : rows;
  float s[CNT];
#pragma unroll
  for (int e = 0; e < CNT; ++e) s[e] = 0.f;
  if (c < m) {
    for (int64_t t = t0 + rr; t < t1; t += 8) {
      float d[CNT], q[CNT];
      IO::template ld<CNT>(static_cast<const T*>(dout) + t * m + c, d);
      if (act != kActNone) {
        IO::template ld<CNT>(static_cast<const T*>(pre) + t * m + c, q);
#pragma unroll
        for (int e = 0; e < CNT; ++e) d[e] *= act_grad<IO>(q[e], act);
      }
      if (dpre != nullptr) IO::template st<CNT>(static_cast<T*>(dpre) + t * ld + c, d);
#pragma unroll
      for (int e = 0; e < CNT; ++e) s[e] += d[e];
    }
  } else if (c < ld && dpre != nullptr) {
    for (int64_t t = t0 + rr; t < t1; t += 8) IO::template st<CNT>(static_cast<T*>(dpre) + t * ld + c, s);
  }
  if (part == nullptr && dbias == nullptr) return;
#pragma unroll
  for (int e = 0; e < CNT; ++e) sh[rr][cv * CNT + e] = s[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * CNT; i += 256) {
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 32 * CNT + i;
    if (col < m) {
      float v = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) v += sh[k][i];
      if (dbias != nullptr) IO::template st<1>(static_cast<T*>(dbias) + col, &v);
      else part[blockIdx.y * m + col] = v;
    }
  }
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up16(int64_t bytes) { return (bytes + 15) / 16 * 16; }

int64_t up(int64_t n, int64_t to) { return cdiv(n, to) * to; }

// One product's tile (32 t x 32 t) and split of k.
//   bfloat16 takes 256 x 256 tiles (t = 8) where they, with k in parts of at
//   least 1024, give three quarters of the CUs a workgroup (products of 16384 x
//   4096 x 2048: 222 to 289 us, 128 x 128 tiles 1.6 to 1.9 times that).
//   Else 128 x 128 where they, with k in parts of at least 16 steps, give as
//   many (300 x 4096 -> 2048: bfloat16 25 us, float32 73; 64 x 64: 40 and 103;
//   forward and gradients of 4099 x 768 -> 1536 in float32: 339, 64 x 64 where
//   there are fewer tiles than CUs: 431).  k is split for one or for two
//   workgroups a CU, whichever leaves a CU less to do, two where it is the same
//   (1024 x 4096 -> 1024 in float32: 82 us, one: 89; 2048 x 768 -> 1536, where
//   two do not come out even: 247, one: 215).
//   float32, which the matrix instructions bound, takes 96 x 96 where the last of
//   them leave fewer CUs idle (4099 x 768 -> 1536: 107 us, 128 x 128: 118; 6000 x
//   2048 -> 1024: 232, 265).
//   Below that 64 x 64, k in parts of at least four steps, split for one
//   workgroup a CU (64 x 4096 -> 2048: bfloat16 15.3 us, float32 22.7; for two:
//   19.4 and 24.5).
struct Tiling {
  int t;
  int64_t kpart, nsplit;
};
template <typename IO>
Tiling tiling(int64_t nc, int64_t nr, int64_t K) {
  constexpr int64_t BK = 8 * LinCfg<IO>::E;
  Tiling w{2, 0, 1};
  auto tiles = [&](int t) { return cdiv(nc, 32 * t) * cdiv(nr, 32 * t); };
  const int64_t steps = cdiv(K, BK);
  int64_t split = 1;
  if (std::is_same<IO, BF16>::value) {
    split = tiles(8) < kCUs ? kCUs / tiles(8) : 1;
    if (split > K / 1024) split = K / 1024;
    if (split < 1) split = 1;
    if (4 * tiles(8) * split >= 3 * kCUs) w.t = 8;
  }
  if (w.t != 8) {
    if (4 * tiles(4) * (steps >= 16 ? steps / 16 : 1) >= 3 * kCUs) w.t = 4;
    auto parts = [&](int t, int64_t wgs, int64_t least) {
      const int64_t s = wgs / tiles(t) < steps / least ? wgs / tiles(t) : steps / least;
      return s < 1 ? 1 : s;
    };
    // what the fullest CU has to do, in 32 x 32 tiles times s
    auto load = [&](int t, int64_t s) { return cdiv(tiles(t) * s, kCUs) * t * t; };
    if (w.t == 4) {
      const int64_t one = parts(4, kCUs, 16), two = parts(4, 2 * kCUs, 16);
      split = load(4, two) * one <= load(4, one) * two ? two : one;
      if (std::is_same<IO, F32>::value && load(3, 1) * split < load(4, split)) {
        w.t = 3;
        split = 1;
      }
    } else {
      split = parts(2, kCUs, 4);
    }
  }
  w.kpart = cdiv(steps, split) * BK;
  w.nsplit = cdiv(K, w.kpart);
  return w;
}

// A product's tiles, whether its outputs go through partials, and its workspace.
struct Plan {
  Tiling w;
  bool part;
  int64_t ldo;
  int64_t c, r, sums, total;  // the copies of the operands and the partials in the workspace
};
template <typename IO, bool CTR, bool RTR>
Plan plan_of(int64_t nc, int64_t nr, int64_t K, int64_t ldc, int64_t ldr) {
  constexpr int64_t E = LinCfg<IO>::E, ES = LinCfg<IO>::ES;
  Plan q{tiling<IO>(nc, nr, K), false, up(nc, 4), 0, 0, 0, 0};
  q.part = q.w.nsplit > 1 || nc % (q.w.t == 8 ? 8 : 4) != 0;
  if (ldc % E != 0) q.total += (CTR ? K : nc) * up(ldc, E) * ES;
  q.r = q.total;
  if (ldr % E != 0) q.total += (RTR ? K : nr) * up(ldr, E) * ES;
  q.sums = q.total;
  if (q.part) q.total += up16(4 * q.w.nsplit * nr * q.ldo);
  return q;
}

// Blocks of four rows, a bounded number of them (the kernels go on from there).
dim3 row_grid(int64_t chunks, int64_t rows, int z) {
  const int64_t x = cdiv(chunks, 64), y = cdiv(rows, 4), most = x < 16384 ? cdiv(16384, x) : 1;
  return dim3(static_cast<unsigned>(x), static_cast<unsigned>(y < most ? y : most), z);
}

template <typename IO, int T, bool CTR, bool RTR, bool PART>
hipError_t launch_tile_t(const LinDev& p, hipStream_t st) {
  const int64_t wgs = cdiv(p.nc, 32 * T) * cdiv(p.nr, 32 * T) * p.nsplit;
  if constexpr (T == 8) {
    // the backward's products have no epilogue
    constexpr int OUT = PART ? kPart : (CTR ? kPlain : kFull);
    hipLaunchKernelGGL((ssm_linear_dma_kernel<CTR, RTR, OUT>), dim3(static_cast<unsigned>(wgs)), dim3(256), 0, st, p);
  } else {
    constexpr size_t smem = size_t(2) * 2 * 32 * T * 128;
    hipLaunchKernelGGL((ssm_linear_tile_kernel<IO, T, T, CTR, RTR, PART>), dim3(static_cast<unsigned>(wgs)), dim3(256),
                       smem, st, p);
  }
  return hipGetLastError();
}

template <typename IO, bool CTR, bool RTR>
hipError_t product(LinDev p, char* work, hipStream_t st) {
  constexpr int64_t E = LinCfg<IO>::E;
  const Plan q = plan_of<IO, CTR, RTR>(p.nc, p.nr, p.K, p.ldc, p.ldr);
  hipError_t e = hipSuccess;
  if (q.sums > 0) {
    PackDev k{};
    int z = 0;
    int64_t chunks = 0, rows = 0;
    auto add = [&](const char*& at, int64_t& ld, char* to, int64_t n) {
      if (ld % E == 0) return;
      k.src[z] = at; k.dst[z] = to; k.rows[z] = n; k.n[z] = ld; k.ld[z] = up(ld, E);
      at = to; ld = k.ld[z];
      if (ld / E > chunks) chunks = ld / E;
      if (n > rows) rows = n;
      ++z;
    };
    add(p.c, p.ldc, work + q.c, CTR ? p.K : p.nc);
    add(p.r, p.ldr, work + q.r, RTR ? p.K : p.nr);
    hipLaunchKernelGGL((ssm_linear_pack_kernel<IO>), row_grid(chunks, rows, z), dim3(256), 0, st, k);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  p.kpart = q.w.kpart;
  p.nsplit = q.w.nsplit;
  p.ldo = q.ldo;
  const LinDev whole = p;
  if (q.part) {
    p.out = work + q.sums;
    p.bias = p.residual = nullptr;
    p.pre = nullptr;
  }
  auto run = [&](auto t) {
    constexpr int T = decltype(t)::value;
    return q.part ? launch_tile_t<IO, T, CTR, RTR, true>(p, st) : launch_tile_t<IO, T, CTR, RTR, false>(p, st);
  };
  if (q.w.t == 8) {
    if constexpr (std::is_same<IO, BF16>::value) e = run(std::integral_constant<int, 8>{});
  } else {
    if constexpr (std::is_same<IO, F32>::value)
      if (q.w.t == 3) e = run(std::integral_constant<int, 3>{});
    if (q.w.t == 4) e = run(std::integral_constant<int, 4>{});
    if (q.w.t == 2) e = run(std::integral_constant<int, 2>{});
  }
  if (e != hipSuccess || !q.part) return e;
  const bool four = p.nc % 4 == 0;
  auto sum = four ? ssm_linear_sum_kernel<IO, 4> : ssm_linear_sum_kernel<IO, 1>;
  hipLaunchKernelGGL(sum, row_grid(cdiv(p.nc, four ? 4 : 1), p.nr, 1), dim3(256), 0, st,
                     reinterpret_cast<const float*>(work + q.sums), whole);
  return hipGetLastError();
}

// Rows of the one-launch kernel; W's row offsets are 32-bit there (16 rows of under 2^21 values).
constexpr int64_t kFewRows = 16;

template <typename IO>
hipError_t forward_io(const LinearArgs& a, char* work, hipStream_t st) {
  LinDev p{};
  p.c = static_cast<const char*>(a.w); p.r = static_cast<const char*>(a.x); p.out = static_cast<char*>(a.out);
  p.nc = a.m; p.nr = a.rows; p.K = a.k; p.ldc = a.k; p.ldr = a.k;
  p.bias = static_cast<const char*>(a.bias); p.residual = static_cast<const char*>(a.residual);
  p.pre = static_cast<char*>(a.pre); p.act = a.act;
  if (a.rows <= kFewRows) {
    const bool vec = a.k % LinCfg<IO>::E == 0, few = a.rows <= 8 && cdiv(a.m, 16) <= kCUs;
    auto kern = few ? (vec ? ssm_linear_rows_kernel<IO, 8, true> : ssm_linear_rows_kernel<IO, 8, false>)
                    : (vec ? ssm_linear_rows_kernel<IO, 16, true> : ssm_linear_rows_kernel<IO, 16, false>);
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(cdiv(a.m, few ? 8 : 16))), dim3(512), 0, st, p);
    return hipGetLastError();
  }
  return product<IO, false, false>(p, work, st);
}

// Rows per workgroup of the dpre kernel: about 2048 workgroups, 64 rows at least.
int64_t dpre_rows(const LinearArgs& a, int64_t cols_per) {
  const int64_t n = cdiv(2048, cdiv(a.m, cols_per));
  const int64_t per = cdiv(a.rows, n);
  return per < 64 ? 64 : per;
}

struct BwdSpace {
  bool keep;    // dpre is written, with rows of ld values (else it is dout)
  int64_t ld;
  int64_t colsum, part, total;
};
template <typename IO>
BwdSpace bwd_space(const LinearArgs& a) {
  constexpr int64_t E = LinCfg<IO>::E;
  BwdSpace w{};
  int64_t at = 0;
  w.ld = up(a.m, E);
  w.keep = (a.dx != nullptr || a.dw != nullptr) && (a.act != kActNone || a.m % E != 0);
  if (w.keep) at += a.rows * w.ld * LinCfg<IO>::ES;
  w.colsum = at;
  if (a.dbias != nullptr) at += up16(4 * cdiv(a.rows, dpre_rows(a, 32 * (a.m % E == 0 ? E : 1))) * a.m);
  w.part = at;
  const int64_t px = a.dx ? plan_of<IO, true, false>(a.k, a.rows, a.m, a.k, w.ld).total : 0;
  const int64_t pw = a.dw ? plan_of<IO, true, true>(a.k, a.m, a.rows, a.k, w.ld).total : 0;
  w.total = at + (px > pw ? px : pw);
  return w;
}

template <typename IO>
hipError_t backward_io(const LinearArgs& a, char* work, hipStream_t st) {
  constexpr int E = LinCfg<IO>::E;
  const BwdSpace w = bwd_space<IO>(a);
  void* const kept = w.keep ? work : nullptr;
  const void* const dpre = w.keep ? kept : a.dout;
  hipError_t e = hipSuccess;
  if (w.keep || a.dbias != nullptr) {
    const bool vec = a.m % E == 0;
    const int64_t per = dpre_rows(a, 32 * (vec ? E : 1)), nblk = cdiv(a.rows, per);
    float* part = a.dbias != nullptr && nblk > 1 ? reinterpret_cast<float*>(work + w.colsum) : nullptr;
    void* dbias = nblk > 1 ? nullptr : a.dbias;
    auto kern = vec ? ssm_linear_dpre_kernel<IO, E> : ssm_linear_dpre_kernel<IO, 1>;
    hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(cdiv(w.ld, 32 * (vec ? E : 1))), static_cast<unsigned>(nblk)),
                       dim3(256), 0, st, a.dout, a.pre, kept, part, dbias, a.rows, a.m, w.ld, per, a.act);
    e = hipGetLastError();
    if (e == hipSuccess && part != nullptr)
      e = launch_column_sum(part, nblk, a.m, a.dbias, std::is_same<IO, BF16>::value, st);
  }
  if (e == hipSuccess && a.dx != nullptr) {
    LinDev p{};
    p.c = static_cast<const char*>(a.w); p.r = static_cast<const char*>(dpre); p.out = static_cast<char*>(a.dx);
    p.nc = a.k; p.nr = a.rows; p.K = a.m; p.ldc = a.k; p.ldr = w.ld;
    e = product<IO, true, false>(p, work + w.part, st);
  }
  if (e == hipSuccess && a.dw != nullptr) {
    LinDev p{};
    p.c = static_cast<const char*>(a.x); p.r = static_cast<const char*>(dpre); p.out = static_cast<char*>(a.dw);
    p.nc = a.k; p.nr = a.m; p.K = a.rows; p.ldc = a.k; p.ldr = w.ld;
    e = product<IO, true, true>(p, work + w.part, st);
  }
  return e;
}

}  // namespace

int64_t linear_workspace_bytes(const LinearArgs& a, bool bf16, bool backward) {
  if (backward) return bf16 ? bwd_space<BF16>(a).total : bwd_space<F32>(a).total;
  if (a.rows <= kFewRows) return 0;
  return bf16 ? plan_of<BF16, false, false>(a.m, a.rows, a.k, a.k, a.k).total
              : plan_of<F32, false, false>(a.m, a.rows, a.k, a.k, a.k).total;
}

int64_t linear_workgroups(const LinearArgs& a, bool bf16) {
  auto count = [&](int64_t nc, int64_t nr, int64_t K) {
    const Tiling w = bf16 ? tiling<BF16>(nc, nr, K) : tiling<F32>(nc, nr, K);
    return cdiv(nc, 32 * w.t) * cdiv(nr, 32 * w.t) * w.nsplit;
  };
  const int64_t f = count(a.m, a.rows, a.k), x = count(a.k, a.rows, a.m), w = count(a.k, a.m, a.rows);
  const int64_t most = f > x ? f : x;
  return most > w ? most : w;
}

hipError_t launch_linear(const LinearArgs& a, bool bf16, char* work, hipStream_t st) {
  return bf16 ? forward_io<BF16>(a, work, st) : forward_io<F32>(a, work, st);
}

hipError_t launch_linear_bwd(const LinearArgs& a, bool bf16, char* work, hipStream_t st) {
  return bf16 ? backward_io<BF16>(a, work, st) : backward_io<F32>(a, work, st);
}

}  // namespace ssm
