// The head scan's chunk kernel: a linear recurrence with one decay per head
// and a matrix state, computed chunk by chunk on the matrix cores (gfx950).
//
//   S_t = e^{g_t} S_{t-1} + u y_t z_t^T          S [rows][cols]
//   o_t = S_t^T x_t  (with the scales below)
//
// x and y have `rows` values per token and head, z and o `cols`.  For a
// chunk of C tokens with the running decay G_i = g_1 + ... + g_i and the
// state S_0 before it,
//
//   o_i   = ps sum_{j <= i} e^{G_i - G_j} (x_i . y_j) z_j + ss e^{G_i} S_0^T x_i
//   S_C   = e^{G_C} S_0 + us sum_j e^{G_C - G_j} y_j z_j^T
//
// The same kernel, with the operands in other roles and the time reversed,
// gives every gradient (ssm_head.hip).
//
// Mapping.  A workgroup of NW wavefronts owns one (batch row, head), a tile of
// 16 NW columns and one segment of the length; it walks its segment's chunks
// with the state in accumulators.  Wavefront w owns all rows and the columns
// [16 w, 16 w + 16) of the tile, so that the state never leaves its registers:
// the accumulator layout of a 16 x 16 tile (lane l holds rows 4 (l / 16) .. + 3
// of column l % 16) is also the layout in which a matrix instruction takes that
// tile as an operand contracted over the rows, when the other operand is read
// in the matching order of k.  Only the C x C score matrix is shared by the
// wavefronts, through LDS.  The next chunk's tiles are loaded into registers
// while the present one is worked on.
//
// Roundings.  bfloat16 storage: scores and the state enter their products as
// hi + lo pairs of bfloat16 (error 2^-17), and the decayed z of the state's
// update as hi + mid + lo, which is exact to float32: the state is a float32
// output.  Accumulators, decays and sums are float32; the running decay is a
// pair of float32, since differences of it are exponentiated.  float32
// storage: float32 matrix instructions, nothing is rounded further.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_device.h"
#include "ssm_kernels.h"

namespace ssm {
namespace headk {

using namespace dev;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short v4i16 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) v4i16 lds_v4i16;

constexpr uint32_t kOOB = 0x80000000u;  // an offset past every resource (sizes are < 2^31)
constexpr float kMinLog2Decay = -2000.f;  // 2^-2000 is 0 in float32: a decay of -inf becomes this

template <typename IO>
struct HeadCfg;
template <>
struct HeadCfg<BF16> {
  static constexpr int ES = 2, E = 8, KS = 32, C = 64;  // bytes, values per 16 bytes, k per product step, tokens per chunk
};
template <>
struct HeadCfg<F32> {
  static constexpr int ES = 4, E = 4, KS = 16, C = 32;
};

// Position of 16-byte chunk c of row r in a row of N chunks: the 16 rows of an
// operand read (one chunk each) fall on different banks.
template <int N>
__device__ __forceinline__ int swz(int r, int c) {
  if constexpr (N >= 16) return c ^ (r & 15);
  else if constexpr (N == 8) return c ^ ((r ^ (r >> 3)) & 7);
  else return c ^ (((r >> 1) ^ (r >> 3)) & 3);
}

template <typename IO>
__device__ __forceinline__ f32x4 mma(const uint4& a, const uint4& b, f32x4 acc) {
  if constexpr (HeadCfg<IO>::ES == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), acc, 0,
                                                   0, 0);
  } else {
    const float* pa = reinterpret_cast<const float*>(&a);
    const float* pb = reinterpret_cast<const float*>(&b);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(pa[e], pb[e], acc, 0, 0, 0);
    return acc;
  }
}

// 16 bytes of row r, k = KS s + E g ..
template <int N>
__device__ __forceinline__ uint4 frag_row(const char* tile, int r, int s, int g) {
  return *reinterpret_cast<const uint4*>(tile + (r * N + swz<N>(r, 4 * s + g)) * 16);
}

// row r, k = 32 s + 4 g .. + 3 and 32 s + 16 + 4 g .. + 3 (bfloat16): the order
// in which two 16-row accumulator tiles hold their rows
template <int N>
__device__ __forceinline__ uint4 frag_acc_order(const char* tile, int r, int s, int g) {
  const int u0 = 8 * s + g, u1 = u0 + 4;
  const uint2 a = *reinterpret_cast<const uint2*>(tile + (r * N + swz<N>(r, u0 >> 1)) * 16 + (u0 & 1) * 8);
  const uint2 b = *reinterpret_cast<const uint2*>(tile + (r * N + swz<N>(r, u1 >> 1)) * 16 + (u1 & 1) * 8);
  return make_uint4(a.x, a.y, b.x, b.y);
}

// column 16 ct + (lane & 15) of the tile, k = rows KS s + E g .. (transposed read)
template <typename IO, int N>
__device__ __forceinline__ uint4 frag_col(const char* tile, int ct, int s, int lane) {
  const int g = lane >> 4;
  if constexpr (HeadCfg<IO>::ES == 2) {
    const int i = lane & 15, r = 32 * s + 8 * g + (i >> 2), u = 4 * ct + (i & 3);
    const char* p0 = tile + (r * N + swz<N>(r, u >> 1)) * 16 + (u & 1) * 8;
    const char* p1 = tile + ((r + 4) * N + swz<N>(r + 4, u >> 1)) * 16 + (u & 1) * 8;
    const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p0));
    const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p1));
    return make_uint4(a.x, a.y, b.x, b.y);
  } else {
    const int c = 16 * ct + (lane & 15), r = 16 * s + 4 * g;
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = *reinterpret_cast<const uint32_t*>(tile + ((r + e) * N + swz<N>(r + e, c >> 2)) * 16 + (c & 3) * 4);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The lane's place, opaque to the compiler: addresses and bounds derived from
// it are worked out where they are used.  Derived from threadIdx they are all
// loop invariants (or common to prologue and epilogue) and kept in registers
// across the loop, which then spills (measured: 40 to 400 spilled registers).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// 8 values as a sum of bfloat16 parts: hi takes the leading 8 bits; what is
// left stays in v
__device__ __forceinline__ uint4 take_bf16(float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    w[e] = BF16::cvt2(v[2 * e], v[2 * e + 1]);
    v[2 * e] -= bf_lo(w[e]);
    v[2 * e + 1] -= bf_hi(w[e]);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct HeadDev {
  const char* x;
  const char* y;
  const char* z;
  char* o;
  int64_t x_b, y_b, z_b;       // byte strides of batch rows
  uint32_t x_t, y_t, z_t;      // byte strides of tokens
  int x_rep, y_rep, z_rep;     // head h reads head h / rep of the operand
  const char* g;               // [b][L][H], nullable
  const float* g_head;         // [H], nullable
  const int32_t* lengths;      // [b], nullable
  const float* h0;             // start state [b][H][rows cols], nullable
  float* last;                 // last state, nullable
  int s_r, s_c;                // state strides of rows and columns
  float* seg_state;            // [b][H][nseg][rows cols]
  float* seg_decay;            // [b][H][nseg]
  const char* dotv;            // [b][L][H / dot_rep][cols]: the dot of o_t with it goes to dot_out (DOT)
  int64_t dot_b;
  uint32_t dot_t;
  int dot_rep;
  float* dot_out;              // [ctile][b][H][L]
  int batch, H, L, rows, cols;
  int nch, cps, nseg, ntile;   // chunks, chunks per segment, segments, column tiles
  float ps, ss, us;
  int rev;                     // time reversed; a token's decay then acts on the step after it
  int out_f32;                 // o is float32 whatever the storage type
  int end_decay;               // the last state is decayed by the first token's g
  int vec_o;                   // four outputs of a row are one aligned store
};

// NaN stays NaN; -inf becomes kMinLog2Decay
__device__ __forceinline__ float clamp_decay(float x) { return x < kMinLog2Decay ? kMinLog2Decay : x; }

template <typename IO>
__device__ __forceinline__ float decay_at(const HeadDev& p, int b, int h, int t) {
  float v = 0.f;
  if (p.g != nullptr) {
    const int64_t i = (static_cast<int64_t>(b) * p.L + t) * p.H + h;
    if constexpr (HeadCfg<IO>::ES == 2)
      v = __uint_as_float(static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p.g)[i]) << 16);
    else
      v = reinterpret_cast<const float*>(p.g)[i];
  } else if (p.g_head != nullptr) {
    v = p.g_head[h];
  }
  return clamp_decay(v * kLog2e);
}

// MODE: kOut writes o (and the last state), kState only the segment's own end
// state (from zero, or from the start state for the first segment) and decay.
constexpr int kOut = 0, kState = 1;

// Bytes of LDS: y and z tiles, x tile, scores (bfloat16: hi and lo), the
// chunk's decays, and the wavefronts' dots.
template <typename IO, int ROWS, int NW, int MODE, bool DOT>
constexpr size_t head_lds_bytes() {
  using K = HeadCfg<IO>;
  constexpr size_t xy = size_t(K::C) * ROWS * K::ES, z = size_t(K::C) * 16 * NW * K::ES;
  constexpr size_t sc = size_t(K::C) * K::C * K::ES * (K::ES == 2 ? 2 : 1);
  return xy + z + 4 * K::C * 4 + (MODE == kOut ? xy + sc : 0) + (DOT ? size_t(NW) * K::C * 4 : 0);
}

template <typename IO, int ROWS, int NW, int MODE, bool DOT, bool VEC>
__global__ void __launch_bounds__(64 * NW, 2) ssm_head_kernel(const HeadDev p) {
  using K = HeadCfg<IO>;
  constexpr int ES = K::ES, E = K::E, KS = K::KS, C = K::C, T = 64 * NW, COLS = 16 * NW;
  constexpr int NK = ROWS * ES / 16, NZ = COLS * ES / 16, NP = C * ES / 16;  // 16-byte chunks per LDS row
  constexpr int RT = ROWS / 16, IB = C / 16, JS = C / KS, RS = ROWS / KS;
  // 16-byte chunks per thread and tile; a small tile leaves threads without one
  constexpr int LX = (C * NK + T - 1) / T, LZ = C * NZ / T;
  static_assert(LZ >= 1 && C * NZ % T == 0, "the z tile has the same share for every thread");

  extern __shared__ __attribute__((aligned(16))) char lds[];
  char* const ty = lds;
  char* const tz = ty + C * ROWS * ES;
  char* const tx = tz + C * COLS * ES;
  char* const tp = tx + C * ROWS * ES;
  char* const tpl = tp + C * C * ES;
  float* const ghi = reinterpret_cast<float*>(MODE == kState ? tx : (ES == 2 ? tpl + C * C * ES : tpl));
  float* const glo = ghi + C;
  float* const eg = glo + C;    // ss e^{G_i}
  float* const we = eg + C;     // us e^{G_C - G_j}
  float* const red = we + C;    // [NW][C]

  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // XCD-contiguous order, column tiles fastest: tiles that share x and y share an L2
  int ct, seg, h, b;
  {
    const uint32_t G = gridDim.x, pid = blockIdx.x, q8 = G / 8, r8 = G % 8, xcd = pid % 8;
    uint32_t idx = xcd * q8 + (xcd < r8 ? xcd : r8) + pid / 8;
    ct = idx % p.ntile;
    idx /= p.ntile;
    const uint32_t nrun = MODE == kState ? p.nseg - 1 : p.nseg;
    seg = idx % nrun;
    idx /= nrun;
    h = idx % p.H;
    b = idx / p.H;
  }
  const int pseg = p.rev ? p.nseg - 1 - seg : seg;
  const int c0 = pseg * p.cps, c1 = c0 + p.cps < p.nch ? c0 + p.cps : p.nch;
  int len = p.L;
  if (p.lengths != nullptr) {
    const int n = p.lengths[b];
    len = n < 0 ? 0 : (n < p.L ? n : p.L);
  }
  const int col0 = ct * COLS, cw = col0 + wave * 16;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h, ssize = static_cast<int64_t>(p.rows) * p.cols;

  // ---- the state: lane holds rows 16 rt + 4 g + v, column cw + li
  f32x4 S[RT];
  {
    const float* src = nullptr;
    if (seg == 0) {
      if (p.h0 != nullptr) src = p.h0 + bh * ssize;
    } else if (MODE == kOut) {
      src = p.seg_state + (bh * p.nseg + (p.rev ? pseg + 1 : pseg - 1)) * ssize;
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * rt + 4 * ((tid & 63) >> 4) + v, c = cw + (tid & 15);
        S[rt][v] = src != nullptr && r < p.rows && c < p.cols ? src[r * p.s_r + c * p.s_c] : 0.f;
      }
  }
  if constexpr (MODE == kOut) {
    // the score tiles above the diagonal that a product step covers are never written again
    for (int i = tid; i < (ES == 2 ? 2 : 1) * C * C * ES / 16; i += T)
      reinterpret_cast<uint4*>(tp)[i] = make_uint4(0, 0, 0, 0);
  }

  const char* const xb = p.x + b * p.x_b + static_cast<int64_t>(h / p.x_rep) * p.rows * ES;
  const char* const yb = p.y + b * p.y_b + static_cast<int64_t>(h / p.y_rep) * p.rows * ES;
  const char* const zb = p.z + b * p.z_b + static_cast<int64_t>(h / p.z_rep) * p.cols * ES;

  // one [C][N 16-byte chunks] tile of tokens t0 .. (those below len; the rest zero) into registers: `width` values
  // of a token from value w0 on
  auto load_tile = [&](const char* base, uint32_t ts, int width, int w0, int t0, auto nchunk, uint4* reg, auto count) {
    constexpr int N = decltype(nchunk)::value, CNT = decltype(count)::value;
    const Rsrc r = make_rsrc(base + static_cast<int64_t>(t0) * ts, 0x7fffffffu);
    const int live = len - t0;  // rows
    const int me = opaque(threadIdx.x);
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int id = me + T * i, row = id / N, c = w0 + id % N * E;
      const uint32_t off = static_cast<uint32_t>(row) * ts + static_cast<uint32_t>(c * ES);
      const int lim = row < live ? (C * N % T != 0 && row >= C ? 0 : width) : 0;
      if constexpr (VEC) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, c < lim ? off : kOOB, 0, 0);
        reg[i] = make_uint4(v.x, v.y, v.z, v.w);
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t oe = c + e < lim ? off + e * ES : kOOB;
          if constexpr (ES == 4) {
            w[e] = __builtin_amdgcn_raw_buffer_load_b32(r, oe, 0, 0);
          } else {
            const uint32_t hv = __builtin_amdgcn_raw_buffer_load_b16(r, oe, 0, 0);
            w[e >> 1] |= (e & 1) ? (hv << 16) : hv;
          }
        }
        reg[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  };
  auto store_tile = [&](char* tile, auto nchunk, const uint4* reg, auto count) {
    constexpr int N = decltype(nchunk)::value, CNT = decltype(count)::value;
    const int me = opaque(threadIdx.x);
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int id = me + T * i, ph = id / N;
      if (C * N % T != 0 && ph >= C) break;
      const int row = p.rev ? C - 1 - ph : ph;
      *reinterpret_cast<uint4*>(tile + (row * N + swz<N>(row, id % N)) * 16) = reg[i];
    }
  };
  using KN = std::integral_constant<int, NK>;
  using ZN = std::integral_constant<int, NZ>;
  using XC = std::integral_constant<int, LX>;
  using ZC = std::integral_constant<int, LZ>;

  float seg_dec = 1.f;
  uint4 rx[LX], ry[LX], rz[LZ];
  float rg = 0.f;
  auto load_chunk = [&](int pc) {
    const int t0 = pc * C;
    if constexpr (MODE == kOut) load_tile(xb, p.x_t, p.rows, 0, t0, KN{}, rx, XC{});
    load_tile(yb, p.y_t, p.rows, 0, t0, KN{}, ry, XC{});
    load_tile(zb, p.z_t, p.cols, col0, t0, ZN{}, rz, ZC{});
    if (wave == NW - 1) {
      // the decay that acts on logical row `lane` of the chunk
      rg = 0.f;
      const int lane = tid & 63;
      if (lane < C) {
        const int t = p.rev ? t0 + C - lane : t0 + lane;  // reversed: the token after it
        if (t < len) rg = decay_at<IO>(p, b, h, t);
      }
    }
  };

  const int n = c1 - c0;
  if (n > 0) load_chunk(p.rev ? c1 - 1 : c0);
  for (int k = 0; k < n; ++k) {
    const int pc = p.rev ? c1 - 1 - k : c0 + k, t0 = pc * C;
    const int lane = opaque(tid) & 63, g = lane >> 4, li = lane & 15;
    __syncthreads();  // the chunk before is done with the tiles
    if constexpr (MODE == kOut) store_tile(tx, KN{}, rx, XC{});
    store_tile(ty, KN{}, ry, XC{});
    store_tile(tz, ZN{}, rz, ZC{});
    if (wave == NW - 1) {
      // running sum over the chunk as a pair of floats (two-sum at every step)
      const int lane = tid & 63;
      float hi = rg, lo = 0.f;
#pragma unroll
      for (int d = 1; d < C; d *= 2) {
        const float ph = __shfl_up(hi, d), pl = __shfl_up(lo, d);
        if (lane >= d) {
          const float s = ph + hi, bb = s - ph;
          lo = (pl + lo) + ((ph - (s - bb)) + (hi - bb));
          hi = s;
        }
      }
      const float eh = __shfl(hi, C - 1), el = __shfl(lo, C - 1);
      if (lane < C) {
        ghi[lane] = hi;
        glo[lane] = lo;
        eg[lane] = p.ss * __builtin_amdgcn_exp2f(hi + lo);
        we[lane] = p.us * __builtin_amdgcn_exp2f((eh - hi) + (el - lo));
      }
    }
    __syncthreads();
    const float end_dec = __builtin_amdgcn_exp2f(ghi[C - 1] + glo[C - 1]);
    if constexpr (MODE == kState) seg_dec *= end_dec;
    if (k + 1 < n) load_chunk(p.rev ? pc - 1 : pc + 1);

    f32x4 O[IB];  // transposed: lane holds columns cw + 4 g + v of logical token 16 ib + li
    if constexpr (MODE == kOut) {
      // ---- scores, 16 x 16 tiles on and below the diagonal dealt to the wavefronts: lane holds j = 4 g + v of i = li
#pragma unroll
      for (int tile = 0; tile < IB * (IB + 1) / 2; ++tile) {
        if (tile % NW != wave) continue;
        int ib = 0, jb = tile;
#pragma unroll
        for (int q = 0; q < IB; ++q)
          if (jb > ib) {
            jb -= ib + 1;
            ++ib;
          }
        const int i = 16 * ib + li, j0 = 16 * jb + 4 * g;
        f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < RS; ++s) a = mma<IO>(frag_row<NK>(ty, 16 * jb + li, s, g), frag_row<NK>(tx, i, s, g), a);
        const float gi = ghi[i], gl = glo[i];
        float w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float d = __builtin_amdgcn_exp2f((gi - ghi[j0 + v]) + (gl - glo[j0 + v]));
          w[v] = j0 + v <= i ? p.ps * d * a[v] : 0.f;
        }
        if constexpr (ES == 2) {
          const int u = 4 * jb + g;
          const int at = (i * NP + swz<NP>(i, u >> 1)) * 16 + (u & 1) * 8;
          const uint2 hi2 = make_uint2(BF16::cvt2(w[0], w[1]), BF16::cvt2(w[2], w[3]));
          *reinterpret_cast<uint2*>(tp + at) = hi2;
          *reinterpret_cast<uint2*>(tpl + at) = make_uint2(BF16::cvt2(w[0] - bf_lo(hi2.x), w[1] - bf_hi(hi2.x)),
                                                           BF16::cvt2(w[2] - bf_lo(hi2.y), w[3] - bf_hi(hi2.y)));
        } else {
          *reinterpret_cast<float4*>(tp + (i * NP + swz<NP>(i, 4 * jb + g)) * 16) = make_float4(w[0], w[1], w[2], w[3]);
        }
      }
      // ---- what the state before the chunk gives
#pragma unroll
      for (int ib = 0; ib < IB; ++ib) O[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        if constexpr (ES == 2) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = S[2 * s + (e >> 2)][e & 3];
          const uint4 hi = take_bf16(v), lo = take_bf16(v);
#pragma unroll
          for (int ib = 0; ib < IB; ++ib) {
            const uint4 fx = frag_acc_order<NK>(tx, 16 * ib + li, s, g);
            O[ib] = mma<IO>(hi, fx, O[ib]);
            O[ib] = mma<IO>(lo, fx, O[ib]);
          }
        } else {
#pragma unroll
          for (int ib = 0; ib < IB; ++ib)
            O[ib] = mma<IO>(__builtin_bit_cast(uint4, S[s]), frag_row<NK>(tx, 16 * ib + li, s, g), O[ib]);
        }
      }
#pragma unroll
      for (int ib = 0; ib < IB; ++ib) O[ib] *= eg[16 * ib + li];
      __syncthreads();  // scores
    }

    // ---- z as an operand: column li, tokens KS js + E g ..
    uint4 fz[JS];
#pragma unroll
    for (int js = 0; js < JS; ++js) fz[js] = frag_col<IO, NZ>(tz, wave, js, lane);

    if constexpr (MODE == kOut) {
#pragma unroll
      for (int ib = 0; ib < IB; ++ib)
#pragma unroll
        for (int js = 0; js * KS < 16 * (ib + 1); ++js) {
          O[ib] = mma<IO>(fz[js], frag_row<NP>(tp, 16 * ib + li, js, g), O[ib]);
          if constexpr (ES == 2) O[ib] = mma<IO>(fz[js], frag_row<NP>(tpl, 16 * ib + li, js, g), O[ib]);
        }
    }

    // ---- the state after the chunk
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) S[rt] *= end_dec;
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      float w[E];
#pragma unroll
      for (int e = 0; e < E; ++e) w[e] = we[KS * js + E * g + e];
      if constexpr (ES == 2) {
        float v[8];
        const uint32_t* pw = reinterpret_cast<const uint32_t*>(&fz[js]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = w[e] * (e & 1 ? bf_hi(pw[e >> 1]) : bf_lo(pw[e >> 1]));
        const uint4 hi = take_bf16(v), mid = take_bf16(v), lo = take_bf16(v);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const uint4 fy = frag_col<IO, NK>(ty, rt, js, lane);
          S[rt] = mma<IO>(fy, hi, S[rt]);
          S[rt] = mma<IO>(fy, mid, S[rt]);
          S[rt] = mma<IO>(fy, lo, S[rt]);
        }
      } else {
        const float* pf = reinterpret_cast<const float*>(&fz[js]);
        const float4 v = make_float4(w[0] * pf[0], w[1] * pf[1], w[2] * pf[2], w[3] * pf[3]);
        const uint4 hz = __builtin_bit_cast(uint4, v);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) S[rt] = mma<IO>(frag_col<IO, NK>(ty, rt, js, lane), hz, S[rt]);
      }
    }

    // ---- outputs, zero in rows past the length
    if constexpr (MODE == kOut) {
      const int oes = p.out_f32 ? 4 : ES;
      const uint32_t ts = static_cast<uint32_t>(p.H * p.cols * oes);
      const Rsrc ro = make_rsrc(p.o + ((static_cast<int64_t>(b) * p.L + t0) * p.H + h) * p.cols * oes, 0x7fffffffu);
      const int c = cw + 4 * g;
#pragma unroll
      for (int ib = 0; ib < IB; ++ib) {
        const int i = 16 * ib + li, ph = p.rev ? C - 1 - i : i;
        const bool ok = t0 + ph < p.L, live = t0 + ph < len;
        const f32x4 v = live ? O[ib] : f32x4{0.f, 0.f, 0.f, 0.f};
        const uint32_t off = static_cast<uint32_t>(ph) * ts + static_cast<uint32_t>(c * oes);
        if (p.vec_o) {
          const uint32_t at = ok && c < p.cols ? off : kOOB;
          if (ES == 4 || p.out_f32) {
            u32x4 w;
            w.x = __float_as_uint(v[0]); w.y = __float_as_uint(v[1]);
            w.z = __float_as_uint(v[2]); w.w = __float_as_uint(v[3]);
            __builtin_amdgcn_raw_buffer_store_b128(w, ro, at, 0, 0);
          } else {
            u32x2 w;
            w.x = BF16::cvt2(v[0], v[1]);
            w.y = BF16::cvt2(v[2], v[3]);
            __builtin_amdgcn_raw_buffer_store_b64(w, ro, at, 0, 0);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t at = ok && c + e < p.cols ? off + e * oes : kOOB;
            if (ES == 4 || p.out_f32)
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), ro, at, 0, 0);
            else
              __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(BF16::cvt(v[e])), ro, at, 0, 0);
          }
        }
        if constexpr (DOT) {
          float dot = 0.f;
          const Rsrc rd = make_rsrc(p.dotv + b * p.dot_b + static_cast<int64_t>(t0) * p.dot_t +
                                        static_cast<int64_t>(h / p.dot_rep) * p.cols * ES, 0x7fffffffu);
          const uint32_t doff = static_cast<uint32_t>(ph) * p.dot_t + static_cast<uint32_t>(c * ES);
          float d[4];
          if constexpr (VEC) {
            BufOf<IO>::type::template ld<4>(rd, live && c < p.cols ? doff : kOOB, d);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              BufOf<IO>::type::template ld<1>(rd, live && c + e < p.cols ? doff + e * ES : kOOB, d + e);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(d[e], v[e], dot);
          dot += __shfl_xor(dot, 16);
          dot += __shfl_xor(dot, 32);
          if (g == 0) red[wave * C + i] = dot;
        }
      }
      if constexpr (DOT) {
        __syncthreads();
        if (tid < C) {
          const int t = t0 + (p.rev ? C - 1 - tid : tid);
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < NW; ++w) sum += red[w * C + tid];
          if (t < p.L) p.dot_out[(static_cast<int64_t>(ct) * p.batch * p.H + bh) * p.L + t] = sum;
        }
      }
    }
  }

  // ---- the segment's own state and decay, or the last state
  float* dst = nullptr;
  float dec = 1.f;
  if constexpr (MODE == kState) {
    dst = p.seg_state + (bh * p.nseg + pseg) * ssize;
    if (ct == 0 && tid == 0) p.seg_decay[bh * p.nseg + pseg] = seg_dec;
  } else if (p.last != nullptr && seg == p.nseg - 1) {
    dst = p.last + bh * ssize;
    if (p.end_decay && len > 0) dec = __builtin_amdgcn_exp2f(decay_at<IO>(p, b, h, 0));
  }
  if (dst != nullptr) {
    const int lane = opaque(tid) & 63, g = lane >> 4, li = lane & 15;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * rt + 4 * g + v, c = cw + li;
        if (r < p.rows && c < p.cols) dst[r * p.s_r + c * p.s_c] = dec * S[rt][v];
      }
  }
}

template <typename IO, int ROWS, int NW, int MODE, bool DOT, bool VEC>
hipError_t launch_head_t(const HeadDev& p, hipStream_t st) {
  const int64_t nrun = MODE == kState ? p.nseg - 1 : p.nseg;
  const int64_t wgs = nrun * p.ntile * p.H * p.batch;
  constexpr size_t smem = head_lds_bytes<IO, ROWS, NW, MODE, DOT>();
  auto kern = ssm_head_kernel<IO, ROWS, NW, MODE, DOT, VEC>;
  if (smem > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(wgs)), dim3(64 * NW), smem, st, p);
  return hipGetLastError();
}

// ROWS: rows rounded up to 32, 64, 128 or 256.  Eight wavefronts (128 columns)
// only where every operand row is whole 16-byte vectors.
template <typename IO, int MODE, bool DOT, int ROWS>
hipError_t launch_head_r(const HeadDev& p, int nw, bool vec, hipStream_t st) {
  if (!vec) return launch_head_t<IO, ROWS, 4, MODE, DOT, false>(p, st);
  if (nw == 8) return launch_head_t<IO, ROWS, 8, MODE, DOT, true>(p, st);
  return launch_head_t<IO, ROWS, 4, MODE, DOT, true>(p, st);
}

template <typename IO, int MODE, bool DOT>
hipError_t launch_head_m(const HeadDev& p, int nw, bool vec, hipStream_t st) {
  if (p.rows <= 32) return launch_head_r<IO, MODE, DOT, 32>(p, nw, vec, st);
  if (p.rows <= 64) return launch_head_r<IO, MODE, DOT, 64>(p, nw, vec, st);
  if (p.rows <= 128) return launch_head_r<IO, MODE, DOT, 128>(p, nw, vec, st);
  return launch_head_r<IO, MODE, DOT, 256>(p, nw, vec, st);
}

// One pass: mode kOut (with the dot if p.dotv is set) or kState.
template <typename IO>
hipError_t launch_head_io(const HeadDev& p, int mode, int nw, bool vec, hipStream_t st) {
  if (mode == kState) return launch_head_m<IO, kState, false>(p, nw, vec, st);
  if (p.dotv != nullptr) return launch_head_m<IO, kOut, true>(p, nw, vec, st);
  return launch_head_m<IO, kOut, false>(p, nw, vec, st);
}

}  // namespace headk

hipError_t launch_head_bf16(const headk::HeadDev& p, int mode, int nw, bool vec, hipStream_t st);
hipError_t launch_head_f32(const headk::HeadDev& p, int mode, int nw, bool vec, hipStream_t st);

}  // namespace ssm
