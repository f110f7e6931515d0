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
// 16 NW NC columns and one segment of the length; it walks its segment's
// chunks with the state in accumulators.  Wavefront w owns all rows and 16 NC
// columns of the tile, so that the state never leaves its registers:
// the accumulator layout of a 16 x 16 tile (lane l holds rows 4 (l / 16) .. + 3
// of column l % 16) is also the layout in which a matrix instruction takes that
// tile as an operand contracted over the rows (see state_row).  Only the C x C
// score matrix is shared by the wavefronts, through LDS.  The next chunk's
// tiles are loaded into registers while the present one is worked on.  Eight
// wavefronts take 128 columns, four 64 or fewer: with four for 128 the state and
// the tiles in flight do not fit the registers (twice the time in the case
// below).
//
// Roundings.  bfloat16 storage: scores and the state enter their products as
// hi + lo pairs of bfloat16 (error 2^-17), and the decayed z of the state's
// update as hi + mid + lo, which is exact to float32: the state is a float32
// output.  Accumulators, decays and sums are float32; the running decay is a
// pair of float32, since differences of it are exponentiated.  float32
// storage: float32 matrix instructions, nothing is rounded further.
//
// What bounds it.  8 x 2048 ragged tokens (some five eighths of them there), 32
// heads of 128 x 128, bfloat16: 150 us where the longest row has 1630 tokens, 171
// where it has 2029 (a row's workgroups walk it whole), 2.2 TB/s of q, k, v, o and
// the last states; the loads and stores alone are three quarters of it, the
// scores a sixth (each left out by itself).  A head's
// chunks follow each other, 256 heads are one workgroup a CU, and a chunk's
// 5 us are vector work (some 560 instructions a wavefront: decays, splits into
// bfloat16 parts) and then matrix work (97 instructions of 16 cycles) between
// three barriers, with little of one under the other.  Tried and no faster: two
// column tiles a wavefront, loads further ahead, scores in two accumulation
// chains, a prescribed order of vector and matrix instructions.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

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
constexpr float kMinLog2Decay = -2000.f;  // 2^-2000 is 0 in float32: a decay of -inf becomes this, a start of the state

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

// LDS tiles have rows of N 16-byte chunks; chunk c of row r sits at position
// c ^ swz(r).  Both kinds of operand read then spread over the banks: 16 bytes a
// lane, which go by 16 lanes, four chunks of 16 rows (a sixteen holds rows 0 to
// 3 and 12 to 15 of one chunk and rows 4 to 11 of its neighbour: with a swizzle
// made for 16 rows of one chunk every such read took half as long again, 9.1
// instead of 3.0 million cycles of bank conflicts in the case above, 3 % of its
// time), and (bfloat16) two chunks of four rows from each of two eights;
// four half chunks of them, the state's update, are two to a bank at best.
// (float32: four chunks of rows four apart.)  swz goes by r % 16, so that an
// address is a lane's base, XORed with a constant for the chunk and offset by
// whole rows: for row 16 R + i and chunk c | j (j the lane's, on other bits),
//   16 N (16 R + i) + 16 ((c | j) ^ swz(i)) = (base(i, j) ^ 16 c) + 256 N R.
template <typename IO, int N>
__device__ __forceinline__ constexpr int swz(int r) {
  const int r0 = r & 1, r1 = (r >> 1) & 1, r2 = (r >> 2) & 1, r3 = (r >> 3) & 1;
  if constexpr (HeadCfg<IO>::ES == 2) {
    if constexpr (N >= 16) return r1 << 3 | r0 << 2 | (r1 ^ r3) << 1;
    else if constexpr (N == 8) return r1 << 2 | (r2 ^ r3) << 1 | r3;
    else return (r1 ^ r3) << 1;
  } else {
    if constexpr (N >= 16) return r & 15;
    else return (r & 7) ^ r3;
  }
}
template <typename IO, int N>
__device__ __forceinline__ int lane_base(int i, int j) {
  return 16 * (N * i + (j ^ swz<IO, N>(i)));
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

// Row 16 R + li, k = KS s + E g .. (16 bytes); base = lane_base(li, g).
template <int N>
__device__ __forceinline__ uint4 frag_row(const char* tile, int base, int R, int s) {
  return *reinterpret_cast<const uint4*>(tile + ((base ^ (64 * s)) + 256 * N * R));
}

// Rows of the state.  An operand read gives lane group g the k of E g .. of a
// step; the accumulator tiles hold four rows a group each.  With float32 that
// is the same; with bfloat16 the two tiles of a step hold rows 8 g .. + 3 and
// 8 g + 4 .. + 7 of its 32, so that they are its operand as they stand.
template <typename IO>
__device__ __forceinline__ constexpr int state_row(int rt, int g, int v) {
  return HeadCfg<IO>::ES == 2 ? 32 * (rt >> 1) + 8 * g + 4 * (rt & 1) + v : 16 * rt + 4 * g + v;
}

// Transposed reads: for k = rows KS s + E g .. of a tile, one column a lane.
// frag_col: column 16 ct + li.  frag_state_col: the column that is row li of
// accumulator tile rt (state_row).  bfloat16: the transposing read takes four
// columns of four rows from every group of 16 lanes (rows 8 g + li / 4, then
// those four further on), lane li % 4 naming the columns.
template <typename IO, int N>
__device__ __forceinline__ int col_base(int li, int g) {
  if constexpr (HeadCfg<IO>::ES == 2) {
    const int r = 8 * g + (li >> 2);
    return 16 * (N * r + (((li & 3) >> 1) ^ swz<IO, N>(r))) + 8 * (li & 1);
  } else {
    return 16 * (N * 4 * g + ((li >> 2) ^ swz<IO, N>(4 * g))) + 4 * (li & 3);
  }
}
template <typename IO, int N>
__device__ __forceinline__ int state_col_base(int li, int g) {
  if constexpr (HeadCfg<IO>::ES == 2) return lane_base<IO, N>(8 * g + (li >> 2), li & 3);
  else return col_base<IO, N>(li, g);
}
// `flip`: 16-byte chunk that the constant part of the columns adds
template <typename IO, int N>
__device__ __forceinline__ uint4 frag_transposed(const char* tile, int base, int flip, int s) {
  if constexpr (HeadCfg<IO>::ES == 2) {
    const char* p0 = tile + ((base ^ (16 * flip)) + 16 * N * 32 * s);
    const char* p1 = tile + ((base ^ (16 * (flip ^ swz<IO, N>(4)))) + 16 * N * (32 * s + 4));
    const uint2 a = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p0));
    const uint2 b = __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4i16*)p1));
    return make_uint4(a.x, a.y, b.x, b.y);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = *reinterpret_cast<const uint32_t*>(tile + ((base ^ (16 * (flip ^ swz<IO, N>(e)))) + 16 * N * (16 * s + e)));
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}
template <typename IO, int N>
__device__ __forceinline__ uint4 frag_col(const char* tile, int base, int ct, int s) {
  return frag_transposed<IO, N>(tile, base, HeadCfg<IO>::ES == 2 ? 2 * ct : 4 * ct, s);
}
template <typename IO, int N>
__device__ __forceinline__ uint4 frag_state_col(const char* tile, int base, int rt, int s) {
  if constexpr (HeadCfg<IO>::ES == 2) return frag_transposed<IO, N>(tile, base + 8 * (rt & 1), 4 * (rt >> 1), s);
  else return frag_transposed<IO, N>(tile, base, 4 * rt, s);
}

// A lane's place or base address, opaque to the compiler: what is derived from
// it is worked out where it is used.  Derived from threadIdx, every LDS address
// is a loop invariant (or common to prologue and epilogue) and is kept in a
// register across the loop, which then spills (measured: 40 to 400 registers).
__device__ __forceinline__ int opaque(int v) {
  asm volatile("" : "+v"(v));
  return v;
}

// 8 values as a sum of bfloat16 parts: returns the leading 8 bits; what is
// left stays in v (exact).
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

// A value that is the same in every lane, for buffer resources: the compiler
// clamps such values in a vector instruction and then takes them for divergent
// (a loop over the lanes round every access).
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
// n rows of ts bytes, n clamped to 0 .. most
__device__ __forceinline__ uint32_t row_bytes(int n, int most, uint32_t ts) {
  return static_cast<uint32_t>(uniform(n < 0 ? 0 : (n < most ? n : most))) * ts;
}

// Running sum over the wavefront's 64 lanes as a pair of floats (hi, lo): a
// two-sum at every step of a scan on cross-lane operands; lanes that a step
// does not reach add zero.
template <int CTRL, int ROWS>
__device__ __forceinline__ void scan_step(float& hi, float& lo) {
  const float ph = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(hi), CTRL, ROWS, 0xf, false));
  const float pl = __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(lo), CTRL, ROWS, 0xf, false));
  const float s = ph + hi, bb = s - ph;
  lo = (pl + lo) + ((ph - (s - bb)) + (hi - bb));
  hi = s;
}
__device__ __forceinline__ void scan_pair(float& hi, float& lo) {
  lo = 0.f;
  scan_step<0x111, 0xf>(hi, lo);  // one lane up within a row of 16
  scan_step<0x112, 0xf>(hi, lo);
  scan_step<0x114, 0xf>(hi, lo);
  scan_step<0x118, 0xf>(hi, lo);
  scan_step<0x142, 0xa>(hi, lo);  // the row before's total to rows 1 and 3
  scan_step<0x143, 0xc>(hi, lo);  // the lower half's to rows 2 and 3
}

// A decay times a value: where the decay is zero so is this, whatever the
// value.  What a state held before it starts anew (g = -inf), and what tokens
// before that gave, is gone, infinities and NaN too.  (Operands of a matrix
// product cannot be left out that way: see `cut` for y.)  The instruction for it
// has no builtin of its own: the intrinsic is named.
extern "C" __device__ __attribute__((const)) float ssm_mul_legacy(float, float) __asm("llvm.amdgcn.fmul.legacy");
__device__ __forceinline__ float times(float decay, float v) { return ssm_mul_legacy(decay, v); }
__device__ __forceinline__ void scale(f32x4& v, float decay) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = times(decay, v[i]);
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
  float* seg_decay;            // [b][H][nseg], -0 where nothing is left of the state before one of the chunks
  const char* dotv;            // [b][L][H / dot_rep][cols]: its dot with o_t, the token's own part of that left out,
                               // goes to dot_out (DOT)
  int64_t dot_b;
  uint32_t dot_t;
  int dot_rep;
  float* dot_out;              // [ctile][b][H][L]
  int batch, H, L, rows, cols;
  int nch, cps, nseg, ntile;   // chunks, chunks per segment, segments, column tiles
  float ps, ss, us;
  int rev;                     // time reversed; a token's decay then acts on the step after it
  int end_decay;               // the last state is decayed by the first token's g
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

// MODE: kOut writes o (and the last state), kOutF32 writes it in float32
// whatever the storage type (per-head parts of a shared head's gradient),
// kState only the segment's own end state (from zero, or from the start state
// for the first segment) and decay.  kOutPair is kOutF32 with two neighbouring
// heads, whose outputs it adds, in a workgroup of twice the wavefronts: half
// the parts to write and to read again.
constexpr int kOut = 0, kState = 1, kOutF32 = 2, kOutPair = 3;
template <int MODE>
constexpr int heads_of() { return MODE == kOutPair ? 2 : 1; }

// Bytes of LDS: y and z tiles, x tile, scores (bfloat16: hi and lo), the
// chunk's decays and last start, and (DOT) the tokens' own scores and the
// wavefronts' dots.
template <typename IO, int ROWS, int NW, int NC, int MODE, bool DOT>
constexpr size_t head_lds_bytes() {
  using K = HeadCfg<IO>;
  constexpr size_t xy = size_t(K::C) * ROWS * K::ES, z = size_t(K::C) * 16 * NW * NC * K::ES;
  constexpr size_t sc = size_t(K::C) * K::C * K::ES * (K::ES == 2 ? 2 : 1);
  return xy + z + 4 * K::C * 4 + 16 + (MODE != kState ? xy + sc : 0) + (DOT ? size_t(NW + 1) * K::C * 4 : 0);
}
// The outputs that the two heads of kOutPair exchange.
template <typename IO, int NW, int NC, int MODE>
constexpr size_t pair_lds_bytes() { return MODE == kOutPair ? size_t(HeadCfg<IO>::C) * 16 * NW * NC * 4 : 0; }

// Wavefronts per SIMD the registers have to leave room for: what fits without
// spills.  One size does not: float32, more than 128 rows, four wavefronts, 131 to
// 156 registers of 256 and their traffic in the chunk loop (4 x 2048 tokens, 32
// heads of 192 x 48: 456 us, bfloat16 188).
template <typename IO, int ROWS, int NW, bool DOT, bool VEC>
constexpr int head_waves() {
  if (!VEC || ROWS == 256) return 2;
  if (ROWS == 128) return HeadCfg<IO>::ES == 2 && !DOT ? (NW == 8 ? 4 : 3) : 2;
  return 4;
}

template <typename IO, int ROWS, int NW, int NC, int MODE, bool DOT, bool VEC>
__global__ void __launch_bounds__((64 * NW * heads_of<MODE>()), (head_waves<IO, ROWS, NW, DOT, VEC>()))
ssm_head_kernel(const HeadDev p) {
  using K = HeadCfg<IO>;
  constexpr bool F32OUT = K::ES == 4 || MODE == kOutF32 || MODE == kOutPair;
  constexpr int HEADS = heads_of<MODE>();
  constexpr int OES = F32OUT ? 4 : 2;  // bytes per output
  constexpr int ES = K::ES, E = K::E, KS = K::KS, C = K::C, T = 64 * NW, COLS = 16 * NW * NC;
  constexpr int NK = ROWS * ES / 16, NZ = COLS * ES / 16, NP = C * ES / 16;  // 16-byte chunks per LDS row
  constexpr int RT = ROWS / 16, IB = C / 16, JS = C / KS, RS = ROWS / KS;
  // 16-byte chunks per thread and tile; a small tile leaves threads without one
  constexpr int LX = (C * NK + T - 1) / T, LZ = C * NZ / T;
  static_assert(LZ >= 1 && C * NZ % T == 0, "the z tile has the same share for every thread");

  extern __shared__ __attribute__((aligned(16))) char lds[];
  // with two heads the threads and all of LDS but the exchange are halved: below, everything is one head's
  const int half = HEADS == 1 ? 0 : __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / T);
  char* const ty = lds + half * static_cast<int>(head_lds_bytes<IO, ROWS, NW, NC, MODE, DOT>());
  char* const tz = ty + C * ROWS * ES;
  char* const tx = tz + C * COLS * ES;
  char* const tp = tx + C * ROWS * ES;
  char* const tpl = tp + C * C * ES;
  float* const ghi = reinterpret_cast<float*>(MODE == kState ? tx : (ES == 2 ? tpl + C * C * ES : tpl));
  float* const glo = ghi + C;
  float* const eg = glo + C;    // ss e^{G_i}
  float* const we = eg + C;     // us e^{G_C - G_j}
  int* const start = reinterpret_cast<int*>(we + C);  // the chunk's last token where the state starts anew (0: none)
  float* const own = we + C + 4;  // scores of tokens with themselves
  float* const red = own + C;   // [NW][C]

  const int tid = static_cast<int>(threadIdx.x) - half * T;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Workgroups go to the 8 XCDs in turn.  The column tiles of a (batch row, head, segment), which share x and y, stay
  // on one XCD and follow each other there; the heads and batch rows are dealt out in turn, so that rows of different
  // lengths load the XCDs alike.
  int ct, seg, h, b;
  {
    const uint32_t pid = blockIdx.x, nt = p.ntile, whole = gridDim.x / nt / 8 * 8 * nt;
    uint32_t idx = pid / nt;
    ct = pid % nt;
    if (pid < whole) {
      const uint32_t slot = pid / 8;
      idx = slot / nt * 8 + pid % 8;
      ct = slot % nt;
    }
    const uint32_t nrun = MODE == kState ? p.nseg - 1 : p.nseg;
    seg = idx % nrun;
    idx /= nrun;
    h = idx % (p.H / HEADS) * HEADS + half;
    b = idx / (p.H / HEADS);
  }
  const int pseg = p.rev ? p.nseg - 1 - seg : seg;
  const int c0 = pseg * p.cps, c1 = c0 + p.cps < p.nch ? c0 + p.cps : p.nch;
  int len = p.L;
  if (p.lengths != nullptr) {
    const int n = p.lengths[b];
    len = n < 0 ? 0 : (n < p.L ? n : p.L);
  }
  const int col0 = ct * COLS, cw = col0 + wave * 16 * NC;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h, ssize = static_cast<int64_t>(p.rows) * p.cols;

  // ---- the state: lane holds rows state_row(rt, g, v), columns cw + 16 nc + li
  f32x4 S[RT][NC];
  {
    const float* src = nullptr;
    if (seg == 0) {
      if (p.h0 != nullptr) src = p.h0 + bh * ssize;
    } else if (MODE != kState) {
      src = p.seg_state + (bh * p.nseg + (p.rev ? pseg + 1 : pseg - 1)) * ssize;
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int i = 0; i < 4 * NC; ++i) {
        const int nc = i / 4, v = i % 4, r = state_row<IO>(rt, (tid & 63) >> 4, v), c = cw + 16 * nc + (tid & 15);
        S[rt][nc][v] = src != nullptr && r < p.rows && c < p.cols ? src[r * p.s_r + c * p.s_c] : 0.f;
      }
  }
  if constexpr (MODE != kState) {
    // the score tiles above the diagonal that a product step covers are never written again
    for (int i = tid; i < (ES == 2 ? 2 : 1) * C * C * ES / 16; i += T)
      reinterpret_cast<uint4*>(tp)[i] = make_uint4(0, 0, 0, 0);
  }

  const char* const xb = p.x + b * p.x_b + static_cast<int64_t>(h / p.x_rep) * p.rows * ES;
  const char* const yb = p.y + b * p.y_b + static_cast<int64_t>(h / p.y_rep) * p.rows * ES;
  const char* const zb = p.z + b * p.z_b + static_cast<int64_t>(h / p.z_rep) * p.cols * ES;

  // Staging.  Thread t holds the 16-byte chunk t % N of rows t / N + i T / N of a [C][N chunks] tile, i counted
  // backwards when the time is reversed, so that register i always goes to the same place after register i - 1.  A
  // resource of its own for every i bounds the rows by the length: what is past it reads zero.
  auto load_tile = [&](const char* base, uint32_t ts, uint32_t voff, int left, int t0, auto nchunk, uint4* reg,
                       auto count) {
    constexpr int N = decltype(nchunk)::value, CNT = decltype(count)::value, STEP = T / N;
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int r0 = STEP * (p.rev ? CNT - 1 - i : i);
      const Rsrc r = make_rsrc(base + static_cast<int64_t>(t0 + r0) * ts, row_bytes(len - t0 - r0, C, ts));
      if constexpr (VEC) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, left > 0 ? voff : kOOB, 0, 0);
        reg[i] = make_uint4(v.x, v.y, v.z, v.w);
      } else {
        uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const uint32_t oe = e < left ? voff + e * ES : kOOB;
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
  auto store_tile = [&](char* tile, int row, int ch, auto nchunk, const uint4* reg, auto count) {
    constexpr int N = decltype(nchunk)::value, CNT = decltype(count)::value, STEP = T / N;
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int r = row + STEP * i;
      *reinterpret_cast<uint4*>(tile + 16 * (N * r + (ch ^ swz<IO, N>(STEP % 16 == 0 ? row : r)))) = reg[i];
    }
  };
  using KN = std::integral_constant<int, NK>;
  using ZN = std::integral_constant<int, NZ>;
  using XC = std::integral_constant<int, LX>;
  using ZC = std::integral_constant<int, LZ>;
  // this thread's chunk and first row of the x and y tiles and of the z tile; threads past a small tile have none
  const int kr = tid / NK, kc = tid % NK, zr = tid / NZ, zc = tid % NZ;
  const int left_k = C * NK % T == 0 || kr < C ? p.rows - kc * E : 0, left_z = p.cols - col0 - zc * E;
  const uint32_t vx = kr * p.x_t + kc * 16, vy = kr * p.y_t + kc * 16, vz = zr * p.z_t + (col0 + zc * E) * ES;

  float seg_dec = 1.f;
  uint4 rx[LX], ry[LX], rz[LZ];
  // The decay that acts on logical row `lane` of a chunk (reversed: that of the token after it), as stored; nothing
  // past the length.  Asked for by every wavefront and first, so that no branch and no later load is waited for with
  // it; scanned by the wavefront with the fewest score tiles, ahead of the barrier.
  uint32_t raw_g = 0;
  float rg = 0.f, rlo = 0.f;
  int last_start = 0;
  const char* const gb = p.g != nullptr ? p.g + (static_cast<int64_t>(b) * p.L * p.H + h) * ES : p.y;
  const uint32_t g_t = p.g != nullptr ? p.H * ES : 0;
  const float fixed = p.g == nullptr && p.g_head != nullptr ? clamp_decay(p.g_head[h] * kLog2e) : 0.f;
  auto scan_decay = [&](int pc) {
    if (wave != NW - 1) return;
    if (p.g != nullptr)
      rg = clamp_decay((ES == 2 ? __uint_as_float(raw_g << 16) : __uint_as_float(raw_g)) * kLog2e);
    else
      rg = (tid & 63) < C && pc * C + (p.rev ? C - (tid & 63) : tid & 63) < len ? fixed : 0.f;
    const uint64_t at = __builtin_amdgcn_ballot_w64(rg == kMinLog2Decay);
    last_start = at != 0 ? 63 - __builtin_clzll(at) : 0;
    scan_pair(rg, rlo);
  };
  auto load_chunk = [&](int pc) {
    const int t0 = pc * C;
    {
      const Rsrc r = make_rsrc(gb + static_cast<int64_t>(t0) * g_t, row_bytes(len - t0, C + 1, g_t));
      const int lane = opaque(tid) & 63;
      const uint32_t off = lane < C ? (p.rev ? C - lane : lane) * g_t : kOOB;
      if constexpr (ES == 2) raw_g = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
      else raw_g = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
    }
    if constexpr (MODE != kState) load_tile(xb, p.x_t, vx, left_k, t0, KN{}, rx, XC{});
    load_tile(yb, p.y_t, vy, left_k, t0, KN{}, ry, XC{});
    load_tile(zb, p.z_t, vz, left_z, t0, ZN{}, rz, ZC{});
  };

  // One chunk's outputs (physical chunk at t0; nothing is written with rows = 0), columns cw + 16 nc + 4 g + v.  Of two
  // heads each writes half of the blocks.
  constexpr int OB = IB / HEADS;
  const int oh = p.H / HEADS, ho = h / HEADS;
  auto store_out = [&](const f32x4 (&O)[OB][NC], int t0, int rows, int li, int g) {
    const int lr = p.rev ? 15 - li : li;  // the lane's token in its block of 16
    const uint32_t ts = static_cast<uint32_t>(oh * p.cols * OES);
    const char* const ob = p.o + ((static_cast<int64_t>(b) * p.L + t0) * oh + ho) * p.cols * OES;
#pragma unroll
    for (int ob_ = 0; ob_ < OB; ++ob_) {
      const int ib = half * OB + ob_, r0 = 16 * (p.rev ? IB - 1 - ib : ib);
      const Rsrc ro = make_rsrc(ob + static_cast<int64_t>(r0) * ts, row_bytes(rows - r0, 16, ts));
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        const int c = cw + 16 * nc + 4 * g;
        const uint32_t off = lr * ts + static_cast<uint32_t>(c * OES);
        const f32x4 v = O[ob_][nc];
        if constexpr (VEC) {
          const uint32_t to = c < p.cols ? off : kOOB;
          if constexpr (F32OUT) {
            u32x4 w;
            w.x = __float_as_uint(v[0]); w.y = __float_as_uint(v[1]);
            w.z = __float_as_uint(v[2]); w.w = __float_as_uint(v[3]);
            __builtin_amdgcn_raw_buffer_store_b128(w, ro, to, 0, 0);
          } else {
            u32x2 w;
            w.x = BF16::cvt2(v[0], v[1]);
            w.y = BF16::cvt2(v[2], v[3]);
            __builtin_amdgcn_raw_buffer_store_b64(w, ro, to, 0, 0);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t to = c + e < p.cols ? off + e * OES : kOOB;
            if constexpr (F32OUT)
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), ro, to, 0, 0);
            else
              __builtin_amdgcn_raw_buffer_store_b16(static_cast<uint16_t>(BF16::cvt(v[e])), ro, to, 0, 0);
          }
        }
      }
    }
  };

  // chunks wholly past the length leave the state alone (their rows are zeroed at the end): they come last forwards,
  // first backwards
  const int cl = (len + C - 1) / C, ce = c1 < cl ? c1 : cl, n = ce - c0;
  if (n > 0) {
    load_chunk(p.rev ? ce - 1 : c0);
    scan_decay(p.rev ? ce - 1 : c0);
    if constexpr (MODE != kState) {
      // Loads and stores are counted together and in order.  With as many stores behind the first loads as the loop
      // has behind its own (these write nothing), the wait for a chunk's loads leaves the stores behind them in
      // flight on either way into the loop; without them it waits for every store to arrive.
      const f32x4 none[OB][NC] = {};
      store_out(none, 0, 0, tid & 15, (tid & 63) >> 4);
    }
  }
  for (int k = 0; k < n; ++k) {
    const int pc = p.rev ? ce - 1 - k : c0 + k, t0 = pc * C;
    __syncthreads();  // the chunk before is done with the tiles
    {
      const int me = opaque(tid), rk = me / NK, rz0 = me / NZ;
      const int kl = p.rev ? C - 1 - rk - (T / NK) * (LX - 1) : rk;   // logical row of register 0
      const int zl = p.rev ? C - 1 - rz0 - (T / NZ) * (LZ - 1) : rz0;
      if (C * NK % T == 0 || rk < C) {
        if constexpr (MODE != kState) store_tile(tx, kl, me % NK, KN{}, rx, XC{});
        store_tile(ty, kl, me % NK, KN{}, ry, XC{});
      }
      store_tile(tz, zl, me % NZ, ZN{}, rz, ZC{});
    }
    if (wave == NW - 1) {
      const float eh = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rg), C - 1));
      const float el = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(rlo), C - 1));
      const int lane = tid & 63;
      if (lane < C) {
        ghi[lane] = rg;
        glo[lane] = rlo;
        eg[lane] = p.ss * __builtin_amdgcn_exp2f(rg + rlo);
        we[lane] = p.us * __builtin_amdgcn_exp2f((eh - rg) + (el - rlo));
      }
      if (lane == 0) *start = last_start;
    }
    __syncthreads();
    const float end_dec = __builtin_amdgcn_exp2f(ghi[C - 1] + glo[C - 1]);
    if constexpr (MODE == kState) seg_dec = end_dec == 0.f ? -0.f : seg_dec * end_dec;

    const int lane = opaque(tid) & 63, g = lane >> 4, li = lane & 15;
    f32x4 O[IB][NC];  // transposed: lane holds columns cw + 16 nc + 4 g + v of logical token 16 ib + li
    if constexpr (MODE != kState) {
      // ---- scores, 16 x 16 tiles on and below the diagonal dealt to the wavefronts: lane holds j = 4 g + v of i = li
      const int rb = lane_base<IO, NK>(li, g);
      for (int tile = wave; tile < IB * (IB + 1) / 2; tile += NW) {
        const int ib = (tile >= 1) + (IB > 2 && tile >= 3) + (IB > 2 && tile >= 6), jb = tile - ib * (ib + 1) / 2;
        const int i = 16 * ib + li, j0 = 16 * jb + 4 * g;
        f32x4 a = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int s = 0; s < RS; ++s) a = mma<IO>(frag_row<NK>(ty, rb, jb, s), frag_row<NK>(tx, rb, ib, s), a);
        const float gi = ghi[i], gl = glo[i];
        const float4 gj = *reinterpret_cast<const float4*>(ghi + j0), gk = *reinterpret_cast<const float4*>(glo + j0);
        float w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float d = __builtin_amdgcn_exp2f((gi - get(gj, v)) + (gl - get(gk, v)));
          w[v] = (DOT ? j0 + v < i : j0 + v <= i) ? times(p.ps * d, a[v]) : 0.f;
        }
        if constexpr (DOT) {
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (j0 + v == i) own[i] = p.ps * a[v];
        }
        if constexpr (ES == 2) {
          const int u = 4 * jb + g;
          const int to = (i * NP + ((u >> 1) ^ swz<IO, NP>(i))) * 16 + (u & 1) * 8;
          const uint2 hi2 = make_uint2(BF16::cvt2(w[0], w[1]), BF16::cvt2(w[2], w[3]));
          *reinterpret_cast<uint2*>(tp + to) = hi2;
          *reinterpret_cast<uint2*>(tpl + to) = make_uint2(BF16::cvt2(w[0] - bf_lo(hi2.x), w[1] - bf_hi(hi2.x)),
                                                           BF16::cvt2(w[2] - bf_lo(hi2.y), w[3] - bf_hi(hi2.y)));
        } else {
          *reinterpret_cast<float4*>(tp + (i * NP + ((4 * jb + g) ^ swz<IO, NP>(i))) * 16) = make_float4(w[0], w[1], w[2], w[3]);
        }
      }
      // ---- what the state before the chunk gives
#pragma unroll
      for (int ib = 0; ib < IB; ++ib)
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) O[ib][nc] = f32x4{0.f, 0.f, 0.f, 0.f};
      const int ab = opaque(rb);
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        uint4 hi[NC], lo[NC];
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) {
          if constexpr (ES == 2) {
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = S[2 * s + (e >> 2)][nc][e & 3];
            hi[nc] = take_bf16(v);
            lo[nc] = take_bf16(v);
          } else {
            hi[nc] = __builtin_bit_cast(uint4, S[s][nc]);
          }
        }
#pragma unroll
        for (int ib = 0; ib < IB; ++ib) {
          const uint4 fx = frag_row<NK>(tx, ab, ib, s);
#pragma unroll
          for (int nc = 0; nc < NC; ++nc) {
            O[ib][nc] = mma<IO>(hi[nc], fx, O[ib][nc]);
            if constexpr (ES == 2) O[ib][nc] = mma<IO>(lo[nc], fx, O[ib][nc]);
          }
        }
      }
#pragma unroll
      for (int ib = 0; ib < IB; ++ib) {
        const float e = eg[16 * ib + li];
#pragma unroll
        for (int nc = 0; nc < NC; ++nc) scale(O[ib][nc], e);
      }
      __syncthreads();  // scores
    }
    const int from = uniform(*start);
    bool cut = from > 0;  // in either head: the barriers are common
    if constexpr (HEADS == 2)
      cut |= uniform(start[(half ? -1 : 1) * static_cast<int>(head_lds_bytes<IO, ROWS, NW, NC, MODE, DOT>() / 4)]) > 0;
    // What comes before the chunk's last start is left out of the state after it: y's rows here (they are done with
    // but for that), z's by its decays of zero.
    if (cut) {
      for (int i = opaque(tid); i < from * NK; i += T) reinterpret_cast<uint4*>(ty)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
    }
    if (k + 1 < n) load_chunk(p.rev ? pc - 1 : pc + 1);

    // ---- z as an operand: column li, tokens KS js + E g ..
    uint4 fz[JS][NC];
    const int zb0 = opaque(col_base<IO, NZ>(li, g));
#pragma unroll
    for (int js = 0; js < JS; ++js)
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) fz[js][nc] = frag_col<IO, NZ>(tz, zb0, wave * NC + nc, js);

    if constexpr (MODE != kState) {
      const int pb = opaque(lane_base<IO, NP>(li, g));
#pragma unroll
      for (int ib = 0; ib < IB; ++ib)
#pragma unroll
        for (int js = 0; js * KS < 16 * (ib + 1); ++js) {
          const uint4 fp = frag_row<NP>(tp, pb, ib, js);
#pragma unroll
          for (int nc = 0; nc < NC; ++nc) O[ib][nc] = mma<IO>(fz[js][nc], fp, O[ib][nc]);
          if constexpr (ES == 2) {
            const uint4 fl = frag_row<NP>(tpl, pb, ib, js);
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) O[ib][nc] = mma<IO>(fz[js][nc], fl, O[ib][nc]);
          }
        }
    }

    // ---- the state after the chunk
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) scale(S[rt][nc], end_dec);
    const int yb0 = opaque(state_col_base<IO, NK>(li, g));
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      float w[E];
      F32::ld<E>(we + KS * js + E * g, w);
      constexpr int TERMS = ES == 2 ? 3 : 1;
      uint4 hz[NC][TERMS];
#pragma unroll
      for (int nc = 0; nc < NC; ++nc) {
        if constexpr (ES == 2) {
          float v[8];
          const uint32_t* pw = reinterpret_cast<const uint32_t*>(&fz[js][nc]);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = times(w[e], e & 1 ? bf_hi(pw[e >> 1]) : bf_lo(pw[e >> 1]));
#pragma unroll
          for (int q = 0; q < TERMS; ++q) hz[nc][q] = take_bf16(v);
        } else {
          const float* pf = reinterpret_cast<const float*>(&fz[js][nc]);
          const float4 v = make_float4(times(w[0], pf[0]), times(w[1], pf[1]), times(w[2], pf[2]), times(w[3], pf[3]));
          hz[nc][0] = __builtin_bit_cast(uint4, v);
        }
      }
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const uint4 fy = frag_state_col<IO, NK>(ty, yb0, rt, js);
#pragma unroll
        for (int q = 0; q < TERMS; ++q)
#pragma unroll
          for (int nc = 0; nc < NC; ++nc) S[rt][nc] = mma<IO>(fy, hz[nc][q], S[rt][nc]);
      }
    }

    if (k + 1 < n) scan_decay(p.rev ? pc - 1 : pc + 1);

    // ---- outputs, zero in rows past the length
    if constexpr (MODE != kState) {
      const int lr = p.rev ? 15 - li : li;  // the lane's token in physical block pb
      if (t0 + C > len) {
#pragma unroll
        for (int ib = 0; ib < IB; ++ib)
          if (t0 + 16 * (p.rev ? IB - 1 - ib : ib) + lr >= len) {
#pragma unroll
            for (int nc = 0; nc < NC; ++nc) O[ib][nc] = f32x4{0.f, 0.f, 0.f, 0.f};
          }
      }
      if constexpr (DOT) {
#pragma unroll
        for (int ib = 0; ib < IB; ++ib) {
          const int r0 = 16 * (p.rev ? IB - 1 - ib : ib);
          const Rsrc rd = make_rsrc(p.dotv + b * p.dot_b + static_cast<int64_t>(t0 + r0) * p.dot_t +
                                        static_cast<int64_t>(h / p.dot_rep) * p.cols * ES, row_bytes(len - t0 - r0, 16, p.dot_t));
          float dot = 0.f;
#pragma unroll
          for (int nc = 0; nc < NC; ++nc) {
            const int c = cw + 16 * nc + 4 * g;
            const uint32_t off = lr * p.dot_t + static_cast<uint32_t>(c * ES);
            float d[4];
            if constexpr (VEC) {
              BufOf<IO>::type::template ld<4>(rd, c < p.cols ? off : kOOB, d);
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e) BufOf<IO>::type::template ld<1>(rd, c + e < p.cols ? off + e * ES : kOOB, d + e);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) dot = __builtin_fmaf(d[e], O[ib][nc][e], dot);
          }
          dot += __shfl_xor(dot, 16);
          dot += __shfl_xor(dot, 32);
          if (g == 0) red[wave * C + 16 * ib + li] = dot;
        }
        // what a token's own y and z give
#pragma unroll
        for (int ib = 0; ib < IB; ++ib) {
          const int r = 16 * ib + li;
          const float e = own[r];
#pragma unroll
          for (int nc = 0; nc < NC; ++nc) {
            const int c = 16 * (wave * NC + nc) + 4 * g;  // column in the tile
            float zv[4];
            IO::template ld<4>(reinterpret_cast<const typename IO::T*>(
                                   tz + 16 * (NZ * r + (c / E ^ swz<IO, NZ>(li))) + c % E * ES), zv);
#pragma unroll
            for (int v = 0; v < 4; ++v) O[ib][nc][v] = __builtin_fmaf(e, zv[v], O[ib][nc][v]);
          }
        }
      }
      if constexpr (HEADS == 1) {
        store_out(O, t0, p.L - t0, li, g);
      } else {
        f32x4* const ex = reinterpret_cast<f32x4*>(lds + 2 * head_lds_bytes<IO, ROWS, NW, NC, MODE, DOT>());
        f32x4 mine[OB][NC];
#pragma unroll
        for (int ob = 0; ob < OB; ++ob)
#pragma unroll
          for (int nc = 0; nc < NC; ++nc) {
            ex[((half * OB + ob) * NC + nc) * T + tid] = half == 0 ? O[OB + ob][nc] : O[ob][nc];
            mine[ob][nc] = half == 0 ? O[ob][nc] : O[OB + ob][nc];
          }
        __syncthreads();
#pragma unroll
        for (int ob = 0; ob < OB; ++ob)
#pragma unroll
          for (int nc = 0; nc < NC; ++nc) mine[ob][nc] += ex[(((1 - half) * OB + ob) * NC + nc) * T + tid];
        store_out(mine, t0, p.L - t0, li, g);
      }
      if constexpr (DOT) {
        if constexpr (HEADS == 1) __syncthreads();
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

  if constexpr (MODE != kState) {
    // outputs (and dots) of the chunks past the length
    const int t1 = c1 * C < p.L ? c1 * C : p.L;
    for (int t = (ce > c0 ? ce : c0) * C + wave; t < t1; t += NW) {
      char* const row = p.o + ((static_cast<int64_t>(b) * p.L + t) * oh + ho) * p.cols * OES;
      for (int c = col0 + (tid & 63); half == 0 && c < col0 + COLS && c < p.cols; c += 64) {
        if constexpr (F32OUT) reinterpret_cast<float*>(row)[c] = 0.f;
        else reinterpret_cast<uint16_t*>(row)[c] = 0;
      }
      if (DOT && (tid & 63) == 0) p.dot_out[(static_cast<int64_t>(ct) * p.batch * p.H + bh) * p.L + t] = 0.f;
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
      for (int i = 0; i < 4 * NC; ++i) {
        const int nc = i / 4, v = i % 4, r = state_row<IO>(rt, g, v), c = cw + 16 * nc + li;
        if (r < p.rows && c < p.cols) dst[r * p.s_r + c * p.s_c] = times(dec, S[rt][nc][v]);
      }
  }
}

template <typename IO, int ROWS, int NW, int NC, int MODE, bool DOT, bool VEC>
hipError_t launch_head_t(const HeadDev& p, hipStream_t st) {
  const int64_t nrun = MODE == kState ? p.nseg - 1 : p.nseg;
  constexpr int HEADS = heads_of<MODE>();
  const int64_t wgs = nrun * p.ntile * (p.H / HEADS) * p.batch;
  constexpr size_t smem = HEADS * head_lds_bytes<IO, ROWS, NW, NC, MODE, DOT>() + pair_lds_bytes<IO, NW, NC, MODE>();
  auto kern = ssm_head_kernel<IO, ROWS, NW, NC, MODE, DOT, VEC>;
  if constexpr (smem > 65536) {
    // asked for once per device (the call costs as much as a launch)
    static std::atomic<uint64_t> allowed{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev > 63 || (allowed.load(std::memory_order_relaxed) & bit) == 0) {
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(smem));
      if (e != hipSuccess) return e;
      if (dev <= 63) allowed.fetch_or(bit, std::memory_order_relaxed);
    }
  }
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(wgs)), dim3(64 * NW * HEADS), smem, st, p);
  return hipGetLastError();
}

// ROWS: rows rounded up to 32, 64, 128 or 256.  `wide` is a tile of 128
// columns, eight wavefronts of 16, else 64 and four.
template <typename IO, int MODE, bool DOT, int ROWS>
hipError_t launch_head_r(const HeadDev& p, bool wide, bool vec, hipStream_t st) {
  if (!vec) return launch_head_t<IO, ROWS, 4, 1, MODE, DOT, false>(p, st);
  if (wide) return launch_head_t<IO, ROWS, 8, 1, MODE, DOT, true>(p, st);
  return launch_head_t<IO, ROWS, 4, 1, MODE, DOT, true>(p, st);
}

template <typename IO, int MODE, bool DOT>
hipError_t launch_head_m(const HeadDev& p, bool wide, bool vec, hipStream_t st) {
  if (p.rows <= 32) return launch_head_r<IO, MODE, DOT, 32>(p, wide, vec, st);
  if (p.rows <= 64) return launch_head_r<IO, MODE, DOT, 64>(p, wide, vec, st);
  if (p.rows <= 128) return launch_head_r<IO, MODE, DOT, 128>(p, wide, vec, st);
  return launch_head_r<IO, MODE, DOT, 256>(p, wide, vec, st);
}

// Whether kOutPair is there for a size: two heads' state and tiles have to fit the registers and LDS.
constexpr int kPairRows = 64;

// One pass: mode kOut (with the dot if p.dotv is set), kOutF32 and kOutPair (with the dot) or kState.
template <typename IO>
hipError_t launch_head_io(const HeadDev& p, int mode, bool wide, bool vec, hipStream_t st) {
  if (mode == kState) return launch_head_m<IO, kState, false>(p, wide, vec, st);
  if constexpr (HeadCfg<IO>::ES == 2) {
    if (mode == kOutF32) return launch_head_m<IO, kOutF32, true>(p, wide, vec, st);
    if (mode == kOutPair) {
      if (!vec || p.rows > kPairRows || p.H % 2 != 0) return hipErrorInvalidValue;
      if (p.rows <= 32)
        return wide ? launch_head_t<IO, 32, 8, 1, kOutPair, true, true>(p, st)
                    : launch_head_t<IO, 32, 4, 1, kOutPair, true, true>(p, st);
      return wide ? launch_head_t<IO, 64, 8, 1, kOutPair, true, true>(p, st)
                  : launch_head_t<IO, 64, 4, 1, kOutPair, true, true>(p, st);
    }
  }
  if (p.dotv != nullptr) return launch_head_m<IO, kOut, true>(p, wide, vec, st);
  return launch_head_m<IO, kOut, false>(p, wide, vec, st);
}

}  // namespace headk

hipError_t launch_head_bf16(const headk::HeadDev& p, int mode, bool wide, bool vec, hipStream_t st);
hipError_t launch_head_f32(const headk::HeadDev& p, int mode, bool wide, bool vec, hipStream_t st);

}  // namespace ssm
