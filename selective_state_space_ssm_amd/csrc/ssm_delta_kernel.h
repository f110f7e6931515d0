// The delta scan's chunk kernels: a linear recurrence with one decay per head
// and a matrix state that first takes out what it holds under the key, computed
// chunk by chunk on the matrix cores (gfx950).
//
//   S~_t = e^{g_t} S_{t-1},  r_t = v_t - S~_t^T k_t,  S_t = S~_t + b_t k_t r_t^T
//   o_t = scale S_t^T q_t                          S [rows = d_key][cols = d_value]
//
// For a chunk of C tokens with the running decay G_i, the state S_0 before it,
// D_ij = e^{G_i - G_j}, N = the part of (D . K K^T) below the diagonal and
// P = scale (D . Q K^T) on and below it:
//
//   x = V - e^G (K S_0),   r = x - M (b x),   M = N (I + diag(b) N)^-1
//   o = scale e^G (Q S_0) + P (b r)
//   S_C = e^{G_C} S_0 + K^T (e^{G_C - G} b r)
//
// Backwards, with R_C = dLoss/dS_C and e_t = R_t^T k_t (so that dv = b e):
//
//   y = P^T dO + e^{G_C - G} (K R_C),   e = y - M^T (b y)
//   R_0 = e^{G_C} R_C + Q^T (scale e^G dO) - K^T (e^G b e)
//
// M needs neither the state nor b on its outside (b = 0 divides nothing) and is
// the same in both directions: ssm_delta_prep_kernel makes it, P and the decays
// for all chunks at once, and what is left of a chunk in the walk over the
// length is products.
// With S_0 and R_C of every chunk kept, and r and e, the other gradients are
// again all chunks at once (ssm_delta_grad_kernel):
//
//   dP = dO (b r)^T,  dN = -(b e)(b r)^T, each times D below the diagonal
//   dq = scale e^G (dO S_0^T) + dP K
//   dk = e^{G_C - G} (b r) R_C^T + dP^T Q + dN^T K - e^G (b e) S_0^T + dN K
//   db = e . r,   dg: see there
//
// The kernels' tiles, swizzles and operand layouts are those of the head scan's
// chunk kernel: a wavefront owns 16 columns of the state and all rows, in
// accumulators, and an accumulator tile is an operand contracted over its rows
// as it stands (state_row), so that x, r and the state pass from product to
// product without leaving the wavefront.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ssm_device.h"
#include "ssm_head_kernel.h"
#include "ssm_kernels.h"

namespace ssm {
namespace deltak {

using namespace headk;

constexpr int kSlab = 64;  // columns of d_value that the gradient kernel takes at a time; padded widths go by it

struct DeltaDev {
  const char* q;
  const char* k;
  const char* v;               // backwards dO
  char* o;
  int64_t q_b, k_b, v_b;       // byte strides of batch rows
  uint32_t q_t, k_t, v_t;      // byte strides of tokens
  int rep;                     // head h reads head h / rep of q and k
  const char* g;               // [b][L][H], nullable
  const char* beta;            // [b][L][H], nullable (ones)
  const int32_t* lengths;      // [b], nullable
  const float* h0;             // state at the first token (backwards: after the last), nullable
  float* last;                 // state after the last token (backwards: at the first), nullable
  char* m;                     // -M of every chunk, [b][H][nch] (see Square)
  char* s;                     // P of every chunk, as m
  float* rates;                // [b][H][nch][kRates][C]
  float* seg_state;            // [b][H][nseg][rp][cp]
  float* seg_trans;            // [b][H][nseg][rp][rp]: what a segment makes of the state before it
  int* seg_kind;               // [b][H][nseg]: see kSegWhole
  char* kept;                  // [b][H][nch] records of what the walks leave for the gradients (see Kept)
  int batch, H, L, rows, cols;
  int rp, cp;                  // rows and columns of states in the workspace: multiples of 16 and of kSlab
  int nch, cps, nseg;          // chunks, chunks per segment, segments
  int ntile, nvt;              // column tiles, those of the state (the others: of the transition)
  int back;                    // P is for the walk backwards
  int places;                  // workgroups of the walk that the CUs hold at once
  float scale;
};

// Parts that a float32 value enters a product in (bfloat16 storage): the state,
// what is added to it and the corrections among a chunk's tokens in three, which
// is exact to float32 at any size; what ends in a bfloat16 result in two (2^-17
// of themselves).  Of the nine products of M's parts with (b x)'s the six of
// 2^-16 and more are made.  (Two parts of each leave the last state off by 1.4e-6
// after 1114 tokens with keys of 16, three by 1.3e-7.  Two of float16 over a power
// of two do not, with half the products, but lose what is 2^-39 of the largest
// among the 64 tokens.)
template <typename IO>
struct DeltaCfg {
  static constexpr int STATE = HeadCfg<IO>::ES == 2 ? 3 : 1;
  static constexpr int PAIR = HeadCfg<IO>::ES == 2 ? 2 : 1;
};

// E values (one operand register of a lane) as N parts
template <typename IO, int N>
__device__ __forceinline__ void split(float* v, uint4* out) {
  if constexpr (HeadCfg<IO>::ES == 2) {
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = v[e];
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = take_bf16(w);
  } else {
    static_assert(N == 1, "float32 is one part");
    out[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
  }
}
// storage values of one operand register as float32
template <typename IO>
__device__ __forceinline__ void unpack(const uint4& r, float* v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&r);
#pragma unroll
  for (int e = 0; e < HeadCfg<IO>::E; ++e) {
    if constexpr (HeadCfg<IO>::ES == 2) v[e] = e & 1 ? bf_hi(w[e >> 1]) : bf_lo(w[e >> 1]);
    else v[e] = __uint_as_float(w[e]);
  }
}

// The row that is row li of accumulator tile rt (state_row), k = KS s + E g ..
template <typename IO, int N>
__device__ __forceinline__ int state_row_base(int li, int g) {
  return HeadCfg<IO>::ES == 2 ? lane_base<IO, N>(8 * (li >> 2) + (li & 3), g) : lane_base<IO, N>(li, g);
}
template <typename IO, int N>
__device__ __forceinline__ uint4 frag_state_row(const char* tile, int base, int rt, int s) {
  if constexpr (HeadCfg<IO>::ES == 2) {
    const int up = rt & 1;
    return *reinterpret_cast<const uint4*>(tile + ((base ^ (64 * s) ^ (up ? 16 * swz<IO, N>(4) : 0)) +
                                                   16 * N * (32 * (rt >> 1) + 4 * up)));
  } else {
    return frag_row<N>(tile, base, rt, s);
  }
}

// The order of what lies between two scheduling barriers: N matrix instructions with V vector instructions after each
template <int N, int V>
__device__ __forceinline__ void mix() {
  if constexpr (N > 0) {
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
    mix<N - 1, V>();
  }
}

// Accumulator tile and register of value e of operand step s
template <typename IO>
__device__ __forceinline__ constexpr int tile_of(int s, int e) { return s * (HeadCfg<IO>::E / 4) + (e >> 2); }

// 16 bytes at byte offset off of a row bounded by the resource; `left` values of the row remain there
template <typename IO, bool VEC>
__device__ __forceinline__ uint4 load16(Rsrc r, uint32_t off, int left) {
  constexpr int E = HeadCfg<IO>::E, ES = HeadCfg<IO>::ES;
  if constexpr (VEC) {
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, left > 0 ? off : kOOB, 0, 0);
    return make_uint4(v.x, v.y, v.z, v.w);
  } else {
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t oe = e < left ? off + e * ES : kOOB;
      if constexpr (ES == 4) {
        w[e] = __builtin_amdgcn_raw_buffer_load_b32(r, oe, 0, 0);
      } else {
        const uint32_t hv = __builtin_amdgcn_raw_buffer_load_b16(r, oe, 0, 0);
        w[e >> 1] |= (e & 1) ? (hv << 16) : hv;
      }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// A tile of C tokens, N chunks of 16 bytes each, dealt to T threads: thread t
// has chunk t % N of rows t / N + i T / N.
template <typename IO, int N, int T>
struct Tile {
  static constexpr int C = HeadCfg<IO>::C, CNT = (C * N + T - 1) / T, STEP = T / N;
  template <bool VEC>
  static __device__ __forceinline__ void load(const char* base, uint32_t ts, int t0, int len, int width, int tid, uint4* reg) {
    const int row = tid / N, c = tid % N;
    const int left = C * N % T == 0 || row < C ? width - c * HeadCfg<IO>::E : 0;
    const uint32_t off = row * ts + c * 16;
    const Rsrc r = make_rsrc(base + static_cast<int64_t>(t0) * ts, row_bytes(len - t0, C, ts));
#pragma unroll
    for (int i = 0; i < CNT; ++i) reg[i] = load16<IO, VEC>(r, off + STEP * i * ts, left);
  }
  static __device__ __forceinline__ void store(char* tile, int tid, const uint4* reg) {
    const int row = tid / N, c = tid % N;
    if (C * N % T != 0 && row >= C) return;
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int r = row + STEP * i;
      *reinterpret_cast<uint4*>(tile + 16 * (N * r + (c ^ swz<IO, N>(STEP % 16 == 0 ? row : r)))) = reg[i];
    }
  }
};

// BYTES as they stand, dealt to T threads
template <int BYTES, int T>
struct Flat {
  static constexpr int CNT = (BYTES / 16 + T - 1) / T;
  static __device__ __forceinline__ void load(const char* base, int tid, uint4* reg) {
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int at = tid + i * T;
      reg[i] = make_uint4(0, 0, 0, 0);
      if (at < BYTES / 16) reg[i] = reinterpret_cast<const uint4*>(base)[at];
    }
  }
  static __device__ __forceinline__ void store(char* to, int tid, const uint4* reg) {
#pragma unroll
    for (int i = 0; i < CNT; ++i)
      if (tid + i * T < BYTES / 16) reinterpret_cast<uint4*>(to)[tid + i * T] = reg[i];
  }
};

// A chunk's M or P in the workspace: of a [C][C] matrix the 16-byte chunks of the 16 x 16 blocks on and below the
// diagonal, block row by block row (five eighths of it for 64 tokens), a part after the other.  In LDS (bfloat16) the upper
// half of the rows holds the left half of the columns only, which is what product steps of 32 read of them.
template <typename IO, int PARTS>
struct Square {
  using K = HeadCfg<IO>;
  static constexpr bool HALVES = K::ES == 2;
  static constexpr int PER = 16 / K::E, IB = K::C / 16, CHUNKS = 8 * PER * IB * (IB + 1), N = K::C / K::E;
  static constexpr int TOP = HALVES ? K::C / 2 * (N / 2) * 16 : 0;  // bytes of the upper half
  static constexpr int PART = HALVES ? TOP + K::C / 2 * N * 16 : K::C * N * 16;
  static constexpr int BYTES = 16 * CHUNKS * PARTS, LDS = PARTS * PART;
  static __device__ __forceinline__ void place(int i, int& row, int& c) {
    const int rb = (i >= 16 * PER) + (IB > 2 && i >= 48 * PER) + (IB > 2 && i >= 96 * PER), at = i - 8 * PER * rb * (rb + 1);
    row = 16 * rb + at / (PER * (rb + 1));
    c = at % (PER * (rb + 1));
  }
  static __device__ __forceinline__ int in_lds(int part, int row, int c) {
    if (HALVES && row < K::C / 2) return part * PART + 16 * (N / 2 * row + (c ^ swz<IO, N / 2>(row)));
    return part * PART + TOP + 16 * (N * (row - (HALVES ? K::C / 2 : 0)) + (c ^ swz<IO, N>(row)));
  }
};

// The same dealt to T threads for LDS tiles; where a thread's chunks go there is worked out once.
template <typename IO, int T, int PARTS>
struct TileM {
  using S = Square<IO, PARTS>;
  static constexpr int CNT = (S::CHUNKS * PARTS + T - 1) / T;
  int to[CNT];
  __device__ __forceinline__ explicit TileM(int tid) {
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const int at = tid + i * T, part = at / S::CHUNKS;
      int row, c;
      S::place(at % S::CHUNKS, row, c);
      to[i] = part < PARTS ? S::in_lds(part, row, c) : -1;
    }
  }
  static __device__ __forceinline__ void load(const char* base, int tid, uint4* reg) {
    const Rsrc r = make_rsrc(base, S::BYTES);
#pragma unroll
    for (int i = 0; i < CNT; ++i) {
      const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, 16 * (tid + i * T), 0, 0);
      reg[i] = make_uint4(v.x, v.y, v.z, v.w);
    }
  }
  __device__ __forceinline__ void store(char* tile, const uint4* reg) const {
#pragma unroll
    for (int i = 0; i < CNT; ++i)
      if (S::CHUNKS * PARTS % T == 0 || to[i] >= 0) *reinterpret_cast<uint4*>(tile + to[i]) = reg[i];
  }
  // what lies above the blocks is never written again
  static __device__ __forceinline__ void clear(char* tile, int tid) {
    for (int i = tid; i < S::LDS / 16; i += T) reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
  }
};

// Operands from such a tile (a part of it): rows by state_row, rows as they follow each other, and columns by state_row;
// block i and product step s on or below the diagonal.
template <typename IO>
struct SquareFrag {
  using S = Square<IO, 1>;
  static constexpr int N = S::N, H = S::HALVES ? N / 2 : N, IH = S::HALVES ? S::IB / 2 : 0;
  enum { kStateRow, kRow, kStateCol };
  int top, low;  // the lane's bases
  __device__ __forceinline__ SquareFrag(int kind, int li, int g)
      : top(kind == kStateRow ? state_row_base<IO, H>(li, g) : kind == kRow ? lane_base<IO, H>(li, g) : state_col_base<IO, H>(li, g)),
        low(kind == kStateRow ? state_row_base<IO, N>(li, g) : kind == kRow ? lane_base<IO, N>(li, g) : state_col_base<IO, N>(li, g)) {}
  __device__ __forceinline__ uint4 state_row_of(const char* tile, int i, int s) const {
    return i < IH ? frag_state_row<IO, H>(tile, top, i, s) : frag_state_row<IO, N>(tile + S::TOP, low, i - IH, s);
  }
  __device__ __forceinline__ uint4 row_of(const char* tile, int i, int s) const {
    return i < IH ? frag_row<H>(tile, top, i, s) : frag_row<N>(tile + S::TOP, low, i - IH, s);
  }
  __device__ __forceinline__ uint4 state_col_of(const char* tile, int i, int s) const {
    if (!S::HALVES) return frag_state_col<IO, N>(tile, low, i, s);
    return s == 0 ? frag_state_col<IO, H>(tile, top, i, 0) : frag_state_col<IO, N>(tile + S::TOP, low, i, 0);
  }
};

// What is kept of a chunk's decays and b, a row of C floats each: G_i as a pair (log2 units), e^{G_i}, e^{G_C - G_i},
// b_i, and 1 where the state starts anew.
enum { kGHi, kGLo, kEk, kWe, kBeta, kAnew, kRates };

// A chunk's decays and b, one token a lane of one wavefront: asked for, then scanned.  A token past the length has
// neither decay nor b.
template <typename IO>
struct Rates {
  static constexpr int C = HeadCfg<IO>::C, ES = HeadCfg<IO>::ES;
  uint32_t raw_g = 0, raw_b = 0;
  static __device__ __forceinline__ uint32_t one(const char* p, const DeltaDev& d, int b, int h, int t0, int len, int lane) {
    const uint32_t ts = d.H * ES;
    const Rsrc r = make_rsrc(p + ((static_cast<int64_t>(b) * d.L + t0) * d.H + h) * ES, row_bytes(len - t0, C, ts));
    const uint32_t off = lane < C ? lane * ts : kOOB;
    if constexpr (ES == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else return __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
  }
  __device__ __forceinline__ void load(const DeltaDev& d, int b, int h, int t0, int len, int lane) {
    if (d.g != nullptr) raw_g = one(d.g, d, b, h, t0, len, lane);
    if (d.beta != nullptr) raw_b = one(d.beta, d, b, h, t0, len, lane);
  }
  static __device__ __forceinline__ float value(uint32_t raw) { return __uint_as_float(ES == 2 ? raw << 16 : raw); }
  // G as a pair of floats (log2 units), lanes past C hold the chunk's sum
  __device__ __forceinline__ void scan(float& hi, float& lo) const {
    hi = clamp_decay(value(raw_g) * kLog2e);
    scan_pair(hi, lo);
  }
  __device__ __forceinline__ float beta(const DeltaDev& d, int t0, int len, int lane) const {
    return d.beta != nullptr ? value(raw_b) : (t0 + lane < len ? 1.f : 0.f);
  }
};

__device__ __forceinline__ int length_of(const DeltaDev& p, int b) {
  if (p.lengths == nullptr) return p.L;
  const int n = p.lengths[b];
  return n < 0 ? 0 : (n < p.L ? n : p.L);
}

// ---------------------------------------------------------------- M of every chunk

template <typename IO, int ROWS>
constexpr size_t prep_lds_bytes() {
  using K = HeadCfg<IO>;
  constexpr size_t tiles = 2 * size_t(K::C) * ROWS * K::ES;
  constexpr size_t square = size_t(K::C) * (K::C + 4) * 4 + size_t(K::C / 16) * 16 * 20 * 4;
  return kRates * K::C * 4 + (tiles > square ? tiles : square);
}

// Score tiles, 16 x 16 on and below the diagonal, dealt to wavefronts
template <int IB>
__device__ __forceinline__ void score_tile(int tile, int& ib, int& jb) {
  ib = (tile >= 1) + (IB > 2 && tile >= 3) + (IB > 2 && tile >= 6);
  jb = tile - ib * (ib + 1) / 2;
}

// A float32 matrix [C][LD] in LDS to global memory as parts
template <typename IO, int LD, int T, int PARTS>
__device__ __forceinline__ void store_parts(const float* n, char* dst, int tid) {
  using S = Square<IO, PARTS>;
  constexpr int E = HeadCfg<IO>::E;
  for (int i = tid; i < S::CHUNKS; i += T) {
    int r, c;
    S::place(i, r, c);
    float v[E];
    F32::ld<E>(n + r * LD + c * E, v);
    uint4 w[PARTS];
    split<IO, PARTS>(v, w);
#pragma unroll
    for (int q = 0; q < PARTS; ++q) *reinterpret_cast<uint4*>(dst + 16 * (q * S::CHUNKS + i)) = w[q];
  }
}

// One (batch row, head, chunk) a workgroup of four wavefronts.  N and P on the
// matrix cores; the 16 x 16 blocks on the diagonal of I + N diag(b) inverted by
// substitution, all of them by one wavefront, a block a group of 16 lanes and a
// column a lane; then, a block column a wavefront, by block rows
//   M_IK = (I + N_II b_I)^-1 (N_IK - sum_{K <= J < I} N_IJ b_J M_JK)
// in float32 matrix instructions, the tiles M_JK staying in registers.
// (Substitution, not powers of N b: keys alike make those grow past float32
// where the inverse does not.)
// A chunk needs nothing of the others, and a workgroup's steps wait for each
// other: what counts is how many share a CU, hence the scores in the place of the
// tiles.  It reads k and q and writes five eighths of M and P: 8 x 2048 ragged
// tokens, 32 heads of 128, bfloat16, 58 us (chunks of a head one after the other,
// each its own rows apart: 84), 4 x 2048 tokens 48.
template <typename IO, int ROWS, bool VEC>
__device__ __forceinline__ void delta_prep(const DeltaDev& p, uint32_t pid, char* lds) {
  using K = HeadCfg<IO>;
  constexpr int ES = K::ES, C = K::C, T = 256, IB = C / 16, NK = ROWS * ES / 16, RS = ROWS / K::KS;
  constexpr int LD = C + 4, TILES = IB * (IB + 1) / 2, MINE = (TILES + 3) / 4;
  constexpr int PP = DeltaCfg<IO>::PAIR, PS = DeltaCfg<IO>::STATE;
  using TK = Tile<IO, NK, T>;
  float* const rt = reinterpret_cast<float*>(lds);  // [kRates][C]
  char* const ty = reinterpret_cast<char*>(rt + kRates * C);
  char* const tx = ty + C * ROWS * ES;
  // in the place of the tiles once the scores are there: with half the LDS twice the workgroups share a CU
  float* const n = reinterpret_cast<float*>(ty);    // [C][LD]: N, then M, then P
  float* const inv = n + C * LD;                    // [IB][16][20]
  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int h = pid % p.H, pc = pid / p.H % p.nch, b = pid / p.H / p.nch, bh = b * p.H + h, t0 = pc * C;
  const int len = length_of(p, b);
  if (t0 >= len) return;
  const int64_t chunk = static_cast<int64_t>(bh) * p.nch + pc;

  uint4 ry[TK::CNT], rx[TK::CNT];
  Rates<IO> rates;
  if (wave == 3) rates.load(p, b, h, t0, len, lane);
  TK::template load<VEC>(p.k + b * p.k_b + static_cast<int64_t>(h / p.rep) * p.rows * ES, p.k_t, t0, len, p.rows, tid, ry);
  TK::template load<VEC>(p.q + b * p.q_b + static_cast<int64_t>(h / p.rep) * p.rows * ES, p.q_t, t0, len, p.rows, tid, rx);
  if (wave == 3) {
    float hi, lo;
    rates.scan(hi, lo);
    const float eh = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(hi), C - 1));
    const float el = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lo), C - 1));
    if (lane < C) {
      rt[kGHi * C + lane] = hi;
      rt[kGLo * C + lane] = lo;
      rt[kEk * C + lane] = __builtin_amdgcn_exp2f(hi + lo);
      rt[kWe * C + lane] = __builtin_amdgcn_exp2f((eh - hi) + (el - lo));
      rt[kBeta * C + lane] = rates.beta(p, t0, len, lane);
      rt[kAnew * C + lane] = clamp_decay(Rates<IO>::value(rates.raw_g) * kLog2e) == kMinLog2Decay ? 1.f : 0.f;
    }
  }
  TK::store(ty, tid, ry);
  TK::store(tx, tid, rx);
  __syncthreads();
  if (tid < kRates * C / 4)
    reinterpret_cast<float4*>(p.rates + chunk * kRates * C)[tid] = reinterpret_cast<const float4*>(rt)[tid];

  // lane holds j = 4 g + v of i = li
  const int rb = lane_base<IO, NK>(li, g);
  f32x4 sc[MINE], sq[MINE];
#pragma unroll
  for (int m = 0; m < MINE; ++m) {
    const int tile = wave + 4 * m;
    sc[m] = sq[m] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (tile >= TILES) continue;
    int ib, jb;
    score_tile<IB>(tile, ib, jb);
    const int i = 16 * ib + li, j0 = 16 * jb + 4 * g;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int s = 0; s < RS; ++s) {
      const uint4 fy = frag_row<NK>(ty, rb, jb, s);
      a = mma<IO>(fy, frag_row<NK>(ty, rb, ib, s), a);
      c = mma<IO>(fy, frag_row<NK>(tx, rb, ib, s), c);
    }
    const float gi = rt[kGHi * C + i], gl = rt[kGLo * C + i];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float d = __builtin_amdgcn_exp2f((gi - rt[kGHi * C + j0 + v]) + (gl - rt[kGLo * C + j0 + v]));
      sc[m][v] = j0 + v < i ? times(d, a[v]) : 0.f;
      sq[m][v] = j0 + v <= i ? times(p.scale * d, c[v]) : 0.f;
    }
  }
  auto put_scores = [&](const f32x4 (&x)[MINE]) {
#pragma unroll
    for (int m = 0; m < MINE; ++m) {
      const int tile = wave + 4 * m;
      if (tile >= TILES) continue;
      int ib, jb;
      score_tile<IB>(tile, ib, jb);
      *reinterpret_cast<f32x4*>(n + (16 * ib + li) * LD + 16 * jb + 4 * g) = x[m];
    }
  };
  __syncthreads();
  put_scores(sc);
  __syncthreads();

  if (wave == 0 && g < IB) {
    // column li of block g's inverse, each value times its row's b as it is needed further down
    const float* const nb = n + 16 * g * LD + 16 * g;
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float s = i == li ? 1.f : 0.f;
#pragma unroll
      for (int k = 0; k < i; ++k) s = __builtin_fmaf(-nb[i * LD + k], t[k], s);
      inv[(g * 16 + i) * 20 + li] = s;
      t[i] = s * rt[kBeta * C + 16 * g + i];
    }
  }
  __syncthreads();

  f32x4 M[IB];
  if (wave < IB) {
    f32x4 mb[IB];  // -b M
#pragma unroll
    for (int I = 0; I < IB; ++I) {
      M[I] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (I < wave) continue;
      f32x4 a;
#pragma unroll
      for (int v = 0; v < 4; ++v) a[v] = n[(16 * I + 4 * g + v) * LD + 16 * wave + li];
#pragma unroll
      for (int J = 0; J < I; ++J) {
        if (J < wave) continue;
        const float4 f = *reinterpret_cast<const float4*>(n + (16 * I + li) * LD + 16 * J + 4 * g);
        a = mma<F32>(__builtin_bit_cast(uint4, f), __builtin_bit_cast(uint4, mb[J]), a);
      }
      const float4 f = *reinterpret_cast<const float4*>(inv + (I * 16 + li) * 20 + 4 * g);
      M[I] = mma<F32>(__builtin_bit_cast(uint4, f), __builtin_bit_cast(uint4, a), M[I]);
#pragma unroll
      for (int v = 0; v < 4; ++v) mb[I][v] = -rt[kBeta * C + 16 * I + 4 * g + v] * M[I][v];
    }
  }
  __syncthreads();
  if (wave < IB) {
#pragma unroll
    for (int I = 0; I < IB; ++I)
#pragma unroll
      for (int v = 0; v < 4; ++v) n[(16 * I + 4 * g + v) * LD + 16 * wave + li] = -M[I][v];
  }
  __syncthreads();
  store_parts<IO, LD, T, PS>(n, p.m + chunk * Square<IO, PS>::BYTES, tid);
  __syncthreads();
  put_scores(sq);  // above the diagonal -M holds zeros, and so does P
  __syncthreads();
  if (p.back) store_parts<IO, LD, T, PS>(n, p.s + chunk * Square<IO, PS>::BYTES, tid);
  else store_parts<IO, LD, T, PP>(n, p.s + chunk * Square<IO, PP>::BYTES, tid);
}

template <typename IO, int ROWS, bool VEC>
__global__ void __launch_bounds__(256) ssm_delta_prep_kernel(const DeltaDev p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // Heads follow each other, so that workgroups of one time read neighbouring parts of the same tokens' rows, eighths of
  // them on an XCD each, where they share a key head's lines.
  const uint32_t per = p.H / 8, slot = blockIdx.x / 8;
  delta_prep<IO, ROWS, VEC>(p, p.H % 8 != 0 ? blockIdx.x : slot / per * p.H + blockIdx.x % 8 * per + slot % per, lds);
}

// ---------------------------------------------------------------- the walk over the length, forwards

// kOut writes o (and the last state); kSeg a segment's own end state (from zero,
// or from the start state for the first segment) and, in the tiles past nvt, what
// it makes of the state before it (the walk from the identity without v); kStates
// the state before every chunk and r.
constexpr int kDeltaOut = 0, kDeltaSeg = 1, kDeltaStates = 2;

// What a segment leaves of the state before it: what its transition makes of it; nothing, since the state starts anew in
// it; all, since it has no tokens.  A product with that transition of zeros or ones would not be that where the state is
// not finite.
constexpr int kSegWhole = 0, kSegAnew = 1, kSegEmpty = 2;

// KIND: 0 without queries, 1 with those of o, 2 with those of the walk backwards
template <typename IO, int ROWS, int NW, int KIND>
constexpr size_t delta_lds_bytes() {
  using K = HeadCfg<IO>;
  constexpr size_t xy = size_t(K::C) * ROWS * K::ES, z = size_t(K::C) * 16 * NW * K::ES;
  constexpr size_t m = Square<IO, DeltaCfg<IO>::STATE>::LDS, s = Square<IO, KIND == 1 ? DeltaCfg<IO>::PAIR : DeltaCfg<IO>::STATE>::LDS;
  return xy + z + m + kRates * K::C * 4 + (KIND != 0 ? xy + s : 0);
}

// The batch row of place b: the longest first, and where all workgroups are on the CUs at once the second half of the places
// from the shortest on, so that of two on a CU a long row is beside a short one (8 ragged rows of up to 2048 tokens, 32
// heads of 128 x 128, the mean of eight draws: 205 us, 208 with the longest first throughout, 217 in the rows' own order;
// where they are not, float32, 8 rows of up to 1024 tokens, 16 heads of 256 x 256, the mean of six: longest first 398, the
// other order 432).  Up to 64 rows, a lane each.
__device__ __forceinline__ int by_length(const DeltaDev& p, int b, int workgroups) {
  const int lane = threadIdx.x & 63, n = lane < p.batch ? length_of(p, lane) : -1;
  int rank = 0;  // of the lane's row
  for (int j = 0; j < p.batch; ++j) {
    const int o = __builtin_amdgcn_readlane(n, j);
    rank += o > n || (o == n && j < lane);
  }
  const int half = (p.batch + 1) / 2;
  if (b >= half && workgroups <= p.places) b = p.batch - 1 - (b - half);
  return __builtin_ctzll(__builtin_amdgcn_ballot_w64(rank == b && lane < p.batch));
}

// Workgroups are dealt to the XCDs as the head scan's: the column tiles of a (batch row, head, segment) follow each
// other on one XCD.
__device__ __forceinline__ void place(const DeltaDev& p, uint32_t pid, int nrun, int& ct, int& seg, int& h, int& b) {
  const uint32_t nt = p.ntile, whole = static_cast<uint32_t>(nrun) * p.H * p.batch / 8 * 8 * nt;
  uint32_t idx = pid / nt;
  ct = pid % nt;
  if (pid < whole) {
    const uint32_t slot = pid / 8;
    idx = slot / nt * 8 + pid % 8;
    ct = slot % nt;
  }
  seg = idx % nrun;
  idx /= nrun;
  h = idx % p.H;
  b = idx / p.H;
  if (p.lengths != nullptr && p.batch <= 64) b = by_length(p, b, p.ntile * nrun * p.H * p.batch);
}

template <typename IO, int RT>
__device__ __forceinline__ void load_state(const float* src, int rows, int cols, int ld, int c, int g, f32x4 (&S)[RT]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = state_row<IO>(rt, g, v);
      S[rt][v] = src != nullptr && r < rows && c < cols ? src[r * ld + c] : 0.f;
    }
}
template <typename IO, int RT>
__device__ __forceinline__ void store_state(float* dst, int rows, int cols, int ld, int c, int g, const f32x4 (&S)[RT]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int r = state_row<IO>(rt, g, v);
      if (r < rows && c < cols) dst[r * ld + c] = S[rt][v];
    }
}

// What the walks leave of a chunk for the gradients, one piece of memory so that one resource reaches all of it: S_0, R_C
// ([rp][cp] each), r, e ([C][cp]), float32 as they hold them.  (Float16 over powers of two moves half the bytes; dg, a sum
// of many products that cancel, is then off by 3e-3 of its norm where its own rounding is 1.7e-3, and an e far below the
// largest of its chunk is lost.)
template <typename IO>
struct Kept {
  uint32_t w, t;  // bytes of a state, of tokens' rows
  __host__ __device__ __forceinline__ Kept(int rp, int cp) : w(rp * cp * 4), t(HeadCfg<IO>::C * cp * 4) {}
  __host__ __device__ __forceinline__ uint32_t state(int back) const { return back * w; }
  __host__ __device__ __forceinline__ uint32_t rows(int back) const { return 2 * w + back * t; }
  __host__ __device__ __forceinline__ uint32_t bytes() const { return 2 * (w + t); }
};

// Accumulator tiles to `rows` rows of cp floats in the workspace (a resource, which bounds the rows; none of it with
// rows = 0), by instructions whose number does not depend on the sizes: loads and stores are counted together and in
// order, and the wait for the next chunk's loads can leave these in flight only if their number is known.
template <typename IO, int N>
__device__ __forceinline__ void keep(char* dst, int rows, int cp, int c, int g, const f32x4 (&X)[N]) {
  const Rsrc r = make_rsrc(dst, static_cast<uint32_t>(rows * cp * 4));
  const uint32_t off = c < cp ? c * 4 : kOOB;
#pragma unroll
  for (int rt = 0; rt < N; ++rt)
#pragma unroll
    for (int v = 0; v < 4; ++v)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(X[rt][v]), r, off + state_row<IO>(rt, g, v) * cp * 4, 0, 0);
}

// A chunk at a time, a workgroup for a (batch row, head, segment) and 16 NW columns of d_value: its chunks follow each
// other, and every wavefront's products too (S into x, x into r, r into S), so that a chunk takes what its longest chain
// takes.  The next chunk's operands are under way meanwhile, those of a product are read and split under the product
// before.  Two workgroups share a CU (80 KB of LDS, 256 registers): alone a chunk takes 4.2 us, two 7.3 (128 x 128,
// bfloat16, M in two parts).  A wavefront's priority falls from product to product of a chunk, so that two on a SIMD are
// in different ones: 8 x 2048 ragged tokens, 32 heads, 163 us, all alike 175 (rising priorities 174; backwards no order
// gains anything).  With M in three parts 168, of the busy CUs' time the matrix unit's 39 %.
template <typename IO, int ROWS, int NW, int MODE, bool VEC>
__device__ __forceinline__ void delta_walk(const DeltaDev& p, uint32_t pid, char* lds) {
  using K = HeadCfg<IO>;
  constexpr bool QUERY = MODE == kDeltaOut;
  constexpr int ES = K::ES, E = K::E, KS = K::KS, C = K::C, T = 64 * NW, COLS = 16 * NW;
  constexpr int NK = ROWS * ES / 16, NZ = COLS * ES / 16;
  constexpr int RT = ROWS / 16, IB = C / 16, JS = C / KS, RS = ROWS / KS;
  constexpr int PP = DeltaCfg<IO>::PAIR, PS = DeltaCfg<IO>::STATE;
  constexpr int MPART = Square<IO, 1>::PART;  // bytes of a part of M or P in LDS
  using TK = Tile<IO, NK, T>;
  using TZ = Tile<IO, NZ, T>;
  using TM = TileM<IO, T, PS>;
  using TP = TileM<IO, T, PP>;
  using TR = Flat<kRates * C * 4, T>;

  char* const ty = lds;
  char* const tz = ty + C * ROWS * ES;
  char* const tm = tz + C * COLS * ES;
  float* const rt = reinterpret_cast<float*>(tm + PS * MPART);  // [kRates][C]
  const float* const ek = rt + kEk * C;
  const float* const we = rt + kWe * C;
  const float* const bt = rt + kBeta * C;
  char* const tx = reinterpret_cast<char*>(rt + kRates * C);
  char* const tp = tx + C * ROWS * ES;

  const int tid = static_cast<int>(threadIdx.x);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int ct, seg, h, b;
  place(p, pid, MODE == kDeltaSeg ? p.nseg - 1 : p.nseg, ct, seg, h, b);
  const bool trans = MODE == kDeltaSeg && ct >= p.nvt;
  if (trans) {
    if (seg == 0) return;  // its state before is the start state
    ct -= p.nvt;
  }
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nch ? c0 + p.cps : p.nch;
  const int len = length_of(p, b);
  const int col0 = ct * COLS, cw = col0 + wave * 16;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h, wsize = static_cast<int64_t>(p.rp) * p.cp;

  f32x4 S[RT];
  {
    const int g = (tid & 63) >> 4, c = cw + (tid & 15);
    if (trans) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int v = 0; v < 4; ++v) S[rt][v] = state_row<IO>(rt, g, v) == c ? 1.f : 0.f;
    } else if (seg == 0) {
      load_state<IO, RT>(p.h0 != nullptr ? p.h0 + bh * p.rows * p.cols : nullptr, p.rows, p.cols, p.cols, c, g, S);
    } else {
      load_state<IO, RT>(MODE == kDeltaSeg ? nullptr : p.seg_state + (bh * p.nseg + seg - 1) * wsize, p.rp, p.cp, p.cp, c, g, S);
    }
  }
  const char* const xb = p.q + b * p.q_b + static_cast<int64_t>(h / p.rep) * p.rows * ES;
  const char* const yb = p.k + b * p.k_b + static_cast<int64_t>(h / p.rep) * p.rows * ES;
  const char* const zb = p.v + b * p.v_b + (static_cast<int64_t>(h) * p.cols + col0) * ES;

  const TM square(tid);
  const TP query_square(tid);
  TM::clear(tm, tid);
  if constexpr (QUERY) TP::clear(tp, tid);
  uint4 rx[TK::CNT], ry[TK::CNT], rz[TZ::CNT], rm[TM::CNT], rp[TP::CNT], rr[TR::CNT];
  auto load_chunk = [&](int pc) {
    const int t0 = pc * C, me = ROWS == 256 || !VEC ? opaque(tid) : tid;
    const int64_t chunk = bh * p.nch + pc;
    TK::template load<VEC>(yb, p.k_t, t0, len, p.rows, me, ry);
    TR::load(reinterpret_cast<const char*>(p.rates + chunk * kRates * C), me, rr);
    if (!trans) TZ::template load<VEC>(zb, p.v_t, t0, len, p.cols - col0, me, rz);
    TM::load(p.m + chunk * TM::S::BYTES, me, rm);
  };
  // these are asked for half a chunk later: with them the registers do not hold the products' operands
  auto load_queries = [&](int pc) {
    const int t0 = pc * C, me = ROWS == 256 || !VEC ? opaque(tid) : tid;
    TK::template load<VEC>(xb, p.q_t, t0, len, p.rows, me, rx);
    TP::load(p.s + (bh * p.nch + pc) * TP::S::BYTES, me, rp);
  };

  // A chunk's outputs: lane holds columns cw + 4 g + v of token 16 ib + li; nothing is written with rows = 0.
  auto store_out = [&](const f32x4 (&O)[IB], int t0, int rows, int li, int g) {
    const uint32_t ts = static_cast<uint32_t>(p.H * p.cols * ES);
    const char* const ob = p.o + ((static_cast<int64_t>(b) * p.L + t0) * p.H + h) * p.cols * ES;
    const Rsrc ro = make_rsrc(ob, row_bytes(rows, C, ts));
    const int c = cw + 4 * g;
    const uint32_t off = li * ts + static_cast<uint32_t>(c * ES);
#pragma unroll
    for (int ib = 0; ib < IB; ++ib) {
      const float w[4] = {O[ib][0], O[ib][1], O[ib][2], O[ib][3]};
      const uint32_t at = off + 16 * ib * ts;
      if constexpr (VEC) {
        BufOf<IO>::type::template st<4>(ro, c < p.cols ? at : kOOB, w);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) BufOf<IO>::type::template st<1>(ro, c + e < p.cols ? at + e * ES : kOOB, w + e);
      }
    }
  };

  const Kept<IO> kept(p.rp, p.cp);
  const int cl = (len + C - 1) / C, ce = c1 < cl ? c1 : cl, nc = ce - c0;
  int kind = nc > 0 ? kSegWhole : kSegEmpty;
  if (nc > 0) {
    load_chunk(c0);
    if constexpr (QUERY) load_queries(c0);
    // as many stores behind the first loads as the loop has behind its own (see keep)
    const f32x4 none[RT > IB ? RT : IB] = {};
    const int li = tid & 15, g = (tid & 63) >> 4;
    if constexpr (QUERY) {
      store_out(reinterpret_cast<const f32x4(&)[IB]>(none), 0, 0, li, g);
    } else if constexpr (MODE == kDeltaStates) {
      keep<IO, RT>(p.kept, 0, p.cp, cw + li, g, reinterpret_cast<const f32x4(&)[RT]>(none));
      keep<IO, IB>(p.kept, 0, p.cp, cw + li, g, reinterpret_cast<const f32x4(&)[IB]>(none));
    }
  }
  for (int kk = 0; kk < nc; ++kk) {
    const int pc = c0 + kk, t0 = pc * C;
    char* const record = p.kept + (bh * p.nch + pc) * static_cast<int64_t>(kept.bytes());
    __syncthreads();  // the chunk before is done with the tiles
    {
      const int me = ROWS == 256 || !VEC ? opaque(tid) : tid;
      TK::store(ty, me, ry);
      if (!trans) TZ::store(tz, me, rz);
      square.store(tm, rm);
      TR::store(reinterpret_cast<char*>(rt), me, rr);
      if constexpr (QUERY) {
        TK::store(tx, me, rx);
        query_square.store(tp, rp);
      }
    }
    __syncthreads();
    const float end_dec = ek[C - 1];
    const int lane = opaque(tid) & 63, g = lane >> 4, li = lane & 15;
    if (kk + 1 < nc) load_chunk(pc + 1);
    if constexpr (MODE == kDeltaSeg)
      if (trans && end_dec == 0.f && __builtin_amdgcn_ballot_w64(lane < C && rt[kAnew * C + lane % C] != 0.f) != 0) kind = kSegAnew;

    if constexpr (MODE == kDeltaStates)
      keep<IO, RT>(record + kept.state(0), p.rp, p.cp, cw + li, g, S);

    __builtin_amdgcn_s_setprio(3);
    // ---- what the state before the chunk gives: X = K S (rows are tokens, by state_row), O = Q S (transposed).  The
    // operands of step s + 1 are read and split under the matrix instructions of step s.
    f32x4 X[IB], O[IB];
#pragma unroll
    for (int i = 0; i < IB; ++i) X[i] = O[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint4 fz[JS];
    float e[JS][E];
    {
      const int sb = state_row_base<IO, NK>(li, g), qb = lane_base<IO, NK>(li, g), zb0 = col_base<IO, NZ>(li, g);
      uint4 fk[IB], fq[QUERY ? IB : 1], sp[2][PS];
      auto read_keys = [&](int s) {
#pragma unroll
        for (int i = 0; i < IB; ++i) fk[i] = frag_state_row<IO, NK>(ty, sb, i, s);
      };
      auto parts = [&](int s) {
        float v[E];
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = S[tile_of<IO>(s, i)][i & 3];
        split<IO, PS>(v, sp[s & 1]);
      };
      read_keys(0);
      parts(0);
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        if constexpr (QUERY) {
#pragma unroll
          for (int i = 0; i < IB; ++i) fq[i] = frag_row<NK>(tx, qb, i, s);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 < RS) parts(s + 1);
#pragma unroll
        for (int q = 0; q < PS; ++q)
#pragma unroll
          for (int i = 0; i < IB; ++i) X[i] = mma<IO>(fk[i], sp[s & 1][q], X[i]);
        mix<IB * PS, 4>();
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 < RS) {
          read_keys(s + 1);
        } else {
#pragma unroll
          for (int js = 0; js < JS; ++js) {
            if (!trans) fz[js] = frag_col<IO, NZ>(tz, zb0, wave, js);
            F32::ld<E>(ek + KS * js + E * g, e[js]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (QUERY) {
#pragma unroll
          for (int q = 0; q < PP; ++q)
#pragma unroll
            for (int i = 0; i < IB; ++i) O[i] = mma<IO>(sp[s & 1][q], fq[i], O[i]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    __builtin_amdgcn_s_setprio(2);
    // ---- x, then r = x - M (b x)
    constexpr int LOW = IB == 2 ? 3 : 6;  // operand steps on and below the diagonal
    uint4 bx[JS][PS], fm[LOW], fl[LOW];
    using Frag = SquareFrag<IO>;
    const Frag mb0(Frag::kStateRow, li, g);
    auto read_m = [&](int part, uint4 (&f)[LOW]) {
#pragma unroll
      for (int i = 0, n = 0; i < IB; ++i)
#pragma unroll
        for (int js = 0; js * KS < 16 * (i + 1); ++js, ++n) f[n] = mb0.state_row_of(tm + part * MPART, i, js);
    };
    read_m(0, fm);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      float v[E] = {}, w[E];
      F32::ld<E>(bt + KS * js + E * g, w);
      if (!trans) unpack<IO>(fz[js], v);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int t = tile_of<IO>(js, i);
        v[i] -= times(e[js][i], X[t][i & 3]);
        X[t][i & 3] = v[i];
        w[i] *= v[i];
      }
      split<IO, PS>(w, bx[js]);
    }
    if constexpr (PS == 3) read_m(1, fl);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) scale(S[rt], end_dec);
    if constexpr (QUERY) {
#pragma unroll
      for (int ib = 0; ib < IB; ++ib) scale(O[ib], p.scale * ek[16 * ib + li]);
    }
    auto times_m = [&](const uint4 (&f)[LOW], int part) {
#pragma unroll
      for (int i = 0, n = 0; i < IB; ++i)
#pragma unroll
        for (int js = 0; js * KS < 16 * (i + 1); ++js, ++n) X[i] = mma<IO>(f[n], bx[js][part], X[i]);
    };
    if constexpr (PS == 3) {
#pragma unroll
      for (int q = 2; q >= 0; --q) times_m(fm, q);
      mix<LOW * 3, 3>();
      __builtin_amdgcn_sched_barrier(0);
      read_m(2, fm);
      __builtin_amdgcn_sched_barrier(0);
      times_m(fl, 1);
      times_m(fl, 0);
      __builtin_amdgcn_sched_barrier(0);
      times_m(fm, 0);
    } else {
      times_m(fm, 0);
      mix<LOW, 2>();
    }
    __builtin_amdgcn_sched_barrier(0);
    if (QUERY && kk + 1 < nc) load_queries(pc + 1);
    const Frag pb(Frag::kRow, li, g);
    if constexpr (QUERY) {
#pragma unroll
      for (int i = 0, n = 0; i < IB; ++i)
#pragma unroll
        for (int js = 0; js * KS < 16 * (i + 1); ++js, ++n) fm[n] = pb.row_of(tp, i, js);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (MODE == kDeltaStates)
      keep<IO, IB>(record + kept.rows(0), C, p.cp, cw + li, g, X);

    __builtin_amdgcn_s_setprio(1);
    // ---- u = b r as an operand of o, e^{G_C - G} u as one of the state's update
    const int yb0 = state_col_base<IO, NK>(li, g);
    uint4 fu[JS][PP], fw[2][PS];
    auto update_parts = [&](int js) {
      float v[E], w[E];
      F32::ld<E>(we + KS * js + E * g, w);
      F32::ld<E>(bt + KS * js + E * g, v);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        v[i] *= X[tile_of<IO>(js, i)][i & 3];
        w[i] = times(w[i], v[i]);
      }
      if constexpr (QUERY) split<IO, PP>(v, fu[js]);
      split<IO, PS>(w, fw[js & 1]);
    };
    update_parts(0);
    if constexpr (QUERY) {
#pragma unroll
      for (int js = 1; js < JS; ++js) update_parts(js);
      if constexpr (PP == 2) {
#pragma unroll
        for (int i = 0, n = 0; i < IB; ++i)
#pragma unroll
          for (int js = 0; js * KS < 16 * (i + 1); ++js, ++n) fl[n] = pb.row_of(tp + MPART, i, js);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int q = 0; q < 2 * PP - 1; ++q)
#pragma unroll
        for (int i = 0, n = 0; i < IB; ++i)
#pragma unroll
          for (int js = 0; js * KS < 16 * (i + 1); ++js, ++n)
            O[i] = q < PP ? mma<IO>(fu[js][q], fm[n], O[i]) : mma<IO>(fu[js][0], fl[n], O[i]);
    }
    __builtin_amdgcn_s_setprio(0);
    // ---- the state after the chunk; under its products the next operand
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      constexpr int GR = ROWS == 256 ? 2 : 4;  // rows' operands read together
      uint4 fy[2][GR];
#pragma unroll
      for (int i = 0; i < GR; ++i) fy[0][i] = frag_state_col<IO, NK>(ty, yb0, i, js);
#pragma unroll
      for (int r = 0; r < RT / GR; ++r) {
        if (r + 1 < RT / GR) {
#pragma unroll
          for (int i = 0; i < GR; ++i) fy[(r + 1) & 1][i] = frag_state_col<IO, NK>(ty, yb0, GR * (r + 1) + i, js);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (!QUERY && r == 0 && js + 1 < JS) update_parts(js + 1);
#pragma unroll
        for (int q = 0; q < PS; ++q)
#pragma unroll
          for (int i = 0; i < GR; ++i) S[GR * r + i] = mma<IO>(fy[r & 1][i], fw[js & 1][q], S[GR * r + i]);
        mix<GR * PS, 6>();
        __builtin_amdgcn_sched_barrier(0);
      }
    }

    // ---- outputs, zero in rows past the length
    if constexpr (QUERY) {
#pragma unroll
      for (int ib = 0; ib < IB; ++ib)
        if (t0 + 16 * ib + li >= len) O[ib] = f32x4{0.f, 0.f, 0.f, 0.f};
      store_out(O, t0, p.L - t0, li, g);
    }
  }

  if constexpr (QUERY) {
    // outputs of the chunks past the length
    const int t1 = c1 * C < p.L ? c1 * C : p.L;
    for (int t = (ce > c0 ? ce : c0) * C + wave; t < t1; t += NW) {
      char* const row = p.o + ((static_cast<int64_t>(b) * p.L + t) * p.H + h) * p.cols * ES;
      for (int c = col0 + (tid & 63); c < col0 + COLS && c < p.cols; c += 64) {
        if constexpr (ES == 4) reinterpret_cast<float*>(row)[c] = 0.f;
        else reinterpret_cast<uint16_t*>(row)[c] = 0;
      }
    }
  }
  const int g = (tid & 63) >> 4, c = cw + (tid & 15);
  if constexpr (MODE == kDeltaSeg) {
    if (trans) {
      store_state<IO, RT>(p.seg_trans + (bh * p.nseg + seg) * p.rp * p.rp, p.rp, p.rp, p.rp, c, g, S);
      if (ct == 0 && tid == 0) p.seg_kind[bh * p.nseg + seg] = kind;
    } else {
      store_state<IO, RT>(p.seg_state + (bh * p.nseg + seg) * wsize, p.rp, p.cp, p.cp, c, g, S);
    }
  } else if (p.last != nullptr && seg == p.nseg - 1) {
    store_state<IO, RT>(p.last + bh * p.rows * p.cols, p.rows, p.cols, p.cols, c, g, S);
  }
}

// Wavefronts per SIMD that the registers leave room for: two workgroups of four or one of eight; one of four in bfloat16
// past 128 keys, of which LDS holds no second.
template <typename IO, int ROWS, int NW>
constexpr int walk_waves() { return HeadCfg<IO>::ES == 2 && ROWS == 256 && NW == 4 ? 1 : 2; }

template <typename IO, int ROWS, int NW, int MODE, bool VEC>
__global__ void __launch_bounds__((64 * NW), (walk_waves<IO, ROWS, NW>())) ssm_delta_kernel(const DeltaDev p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  delta_walk<IO, ROWS, NW, MODE, VEC>(p, blockIdx.x, lds);
}

// One chunk and one column tile: a launch for both (17 tokens, 4 heads of 32 x 32: 12.7 us, two launches 15.6).
template <typename IO, int ROWS, bool VEC>
__global__ void __launch_bounds__(256, (walk_waves<IO, ROWS, 4>())) ssm_delta_one_kernel(const DeltaDev p) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  // the walk's workgroup of a (batch row, head) makes that one's M
  int ct, seg, h, b;
  place(p, blockIdx.x, 1, ct, seg, h, b);
  delta_prep<IO, ROWS, VEC>(p, b * p.H + h, lds);
  __syncthreads();  // what it wrote, the walk reads back
  delta_walk<IO, ROWS, 4, kDeltaOut, VEC>(p, blockIdx.x, lds);
}

// ---------------------------------------------------------------- the walk over the length, backwards

// v is dO, h0 dlast, last dh0.  SEG: a segment's own R at its first token, from zero (the last segment: from dlast);
// else R after every chunk and e are written.
template <typename IO, int ROWS, int NW, bool SEG, bool VEC>
__device__ __forceinline__ void delta_walk_back(const DeltaDev& p, uint32_t pid, char* lds) {
  using K = HeadCfg<IO>;
  constexpr int ES = K::ES, E = K::E, KS = K::KS, C = K::C, T = 64 * NW, COLS = 16 * NW;
  constexpr int NK = ROWS * ES / 16, NZ = COLS * ES / 16;
  constexpr int RT = ROWS / 16, IB = C / 16, JS = C / KS, RS = ROWS / KS;
  constexpr int PS = DeltaCfg<IO>::STATE;
  constexpr int MPART = Square<IO, 1>::PART;
  using TK = Tile<IO, NK, T>;
  using TZ = Tile<IO, NZ, T>;
  using TM = TileM<IO, T, PS>;
  using TR = Flat<kRates * C * 4, T>;

  char* const ty = lds;
  char* const tz = ty + C * ROWS * ES;
  char* const tm = tz + C * COLS * ES;
  float* const rt = reinterpret_cast<float*>(tm + PS * MPART);  // [kRates][C]
  const float* const ek = rt + kEk * C;
  const float* const we = rt + kWe * C;
  const float* const bt = rt + kBeta * C;
  char* const tx = reinterpret_cast<char*>(rt + kRates * C);
  char* const tp = tx + C * ROWS * ES;

  const int tid = static_cast<int>(threadIdx.x);
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int ct, seg, h, b;
  place(p, pid, SEG ? p.nseg - 1 : p.nseg, ct, seg, h, b);
  if constexpr (SEG) ++seg;
  const int c0 = seg * p.cps, c1 = c0 + p.cps < p.nch ? c0 + p.cps : p.nch;
  const int len = length_of(p, b);
  const int col0 = ct * COLS, cw = col0 + wave * 16;
  const int64_t bh = static_cast<int64_t>(b) * p.H + h, wsize = static_cast<int64_t>(p.rp) * p.cp;

  f32x4 R[RT];
  {
    const int g = (tid & 63) >> 4, c = cw + (tid & 15);
    if (seg == p.nseg - 1)
      load_state<IO, RT>(p.h0 != nullptr ? p.h0 + bh * p.rows * p.cols : nullptr, p.rows, p.cols, p.cols, c, g, R);
    else
      load_state<IO, RT>(SEG ? nullptr : p.seg_state + (bh * p.nseg + seg + 1) * wsize, p.rp, p.cp, p.cp, c, g, R);
  }

  const char* const xb = p.q + b * p.q_b + static_cast<int64_t>(h / p.rep) * p.rows * ES;
  const char* const yb = p.k + b * p.k_b + static_cast<int64_t>(h / p.rep) * p.rows * ES;
  const char* const zb = p.v + b * p.v_b + (static_cast<int64_t>(h) * p.cols + col0) * ES;

  const TM square(tid);
  TM::clear(tm, tid);
  TM::clear(tp, tid);
  uint4 rx[TK::CNT], ry[TK::CNT], rz[TZ::CNT], rm[TM::CNT], rp[TM::CNT], rr[TR::CNT];
  auto load_chunk = [&](int pc) {
    const int t0 = pc * C, me = ROWS >= 128 || !VEC ? opaque(tid) : tid;
    const int64_t chunk = bh * p.nch + pc;
    TK::template load<VEC>(yb, p.k_t, t0, len, p.rows, me, ry);
    TR::load(reinterpret_cast<const char*>(p.rates + chunk * kRates * C), me, rr);
    TM::load(p.s + chunk * TM::S::BYTES, me, rp);
    TZ::template load<VEC>(zb, p.v_t, t0, len, p.cols - col0, me, rz);
  };
  // these are asked for half a chunk later: with them the registers do not hold the products' operands
  auto load_late = [&](int pc) {
    const int t0 = pc * C, me = ROWS >= 128 || !VEC ? opaque(tid) : tid;
    TM::load(p.m + (bh * p.nch + pc) * TM::S::BYTES, me, rm);
    TK::template load<VEC>(xb, p.q_t, t0, len, p.rows, me, rx);
  };

  const Kept<IO> kept(p.rp, p.cp);
  const int cl = (len + C - 1) / C, ce = c1 < cl ? c1 : cl, nc = ce - c0;
  if (nc > 0) {
    load_chunk(ce - 1);
    load_late(ce - 1);
    if constexpr (!SEG) {
      // as many stores behind the first loads as the loop has behind its own (see keep)
      const f32x4 none[RT > IB ? RT : IB] = {};
      const int li = tid & 15, g = (tid & 63) >> 4;
      keep<IO, RT>(p.kept, 0, p.cp, cw + li, g, reinterpret_cast<const f32x4(&)[RT]>(none));
      keep<IO, IB>(p.kept, 0, p.cp, cw + li, g, reinterpret_cast<const f32x4(&)[IB]>(none));
    }
  }
  for (int kk = 0; kk < nc; ++kk) {
    const int pc = ce - 1 - kk;
    char* const record = p.kept + (bh * p.nch + pc) * static_cast<int64_t>(kept.bytes());
    __syncthreads();
    {
      const int me = ROWS >= 128 || !VEC ? opaque(tid) : tid;
      TK::store(ty, me, ry);
      TK::store(tx, me, rx);
      TZ::store(tz, me, rz);
      square.store(tm, rm);
      square.store(tp, rp);
      TR::store(reinterpret_cast<char*>(rt), me, rr);
    }
    __syncthreads();
    const float end_dec = ek[C - 1];
    const int lane = opaque(tid) & 63, g = lane >> 4, li = lane & 15;
    if (kk + 1 < nc) load_chunk(pc - 1);
    if constexpr (!SEG) keep<IO, RT>(record + kept.state(1), p.rp, p.cp, cw + li, g, R);

    // ---- X = K R (rows are tokens); the operands of step s + 1 are read and split under the matrix instructions of step s
    constexpr int LOW = IB == 2 ? 3 : 6;  // operand steps on and below the diagonal
    f32x4 X[IB], Y[IB];
#pragma unroll
    for (int i = 0; i < IB; ++i) X[i] = Y[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    uint4 fz[JS], ft[LOW], fl[LOW];
    const SquareFrag<IO> mc0(SquareFrag<IO>::kStateCol, li, g);
    // columns of a square matrix, its rows as the contraction: what lies below the diagonal of the transposed
    auto read_square = [&](const char* tile, uint4 (&f)[LOW]) {
#pragma unroll
      for (int i = 0, n = 0; i < IB; ++i)
#pragma unroll
        for (int js = 0; js < JS; ++js)
          if (KS * (js + 1) > 16 * i) f[n++] = mc0.state_col_of(tile, i, js);
    };
    auto times_square = [&](const uint4 (&f)[LOW], const uint4 (&by)[JS], f32x4 (&acc)[IB]) {
#pragma unroll
      for (int i = 0, n = 0; i < IB; ++i)
#pragma unroll
        for (int js = 0; js < JS; ++js)
          if (KS * (js + 1) > 16 * i) acc[i] = mma<IO>(f[n++], by[js], acc[i]);
    };
    {
      const int sb = state_row_base<IO, NK>(li, g), zb0 = col_base<IO, NZ>(li, g);
      constexpr int NB = ROWS == 256 ? 1 : 2;  // what fits the registers
      uint4 fk[NB][IB], sp[2][PS];
      auto read_keys = [&](int s) {
#pragma unroll
        for (int i = 0; i < IB; ++i) fk[s % NB][i] = frag_state_row<IO, NK>(ty, sb, i, s);
      };
      auto parts = [&](int s) {
        float v[E];
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = R[tile_of<IO>(s, i)][i & 3];
        split<IO, PS>(v, sp[s & 1]);
      };
      if (NB == 2) read_keys(0);
      parts(0);
#pragma unroll
      for (int s = 0; s < RS; ++s) {
        if (NB == 1) read_keys(s);
        if (s + 1 < RS) {
          if (NB == 2) read_keys(s + 1);
        } else {
#pragma unroll
          for (int js = 0; js < JS; ++js) fz[js] = frag_col<IO, NZ>(tz, zb0, wave, js);
          read_square(tp, ft);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (s + 1 < RS) parts(s + 1);
#pragma unroll
        for (int q = 0; q < PS; ++q)
#pragma unroll
          for (int i = 0; i < IB; ++i) X[i] = mma<IO>(fk[s % NB][i], sp[s & 1][q], X[i]);
        mix<IB * PS, 4>();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // ---- y = P^T dO + e^{G_C - G} X
    if constexpr (PS == 3) read_square(tp + MPART, fl);
    __builtin_amdgcn_sched_barrier(0);
    times_square(ft, fz, Y);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (PS == 3) {
      read_square(tp + 2 * MPART, ft);
      __builtin_amdgcn_sched_barrier(0);
      times_square(fl, fz, Y);
      __builtin_amdgcn_sched_barrier(0);
      read_square(tm + MPART, fl);
      __builtin_amdgcn_sched_barrier(0);
      times_square(ft, fz, Y);
      __builtin_amdgcn_sched_barrier(0);
    }
    read_square(tm, ft);
    __builtin_amdgcn_sched_barrier(0);
    // ---- e = y - M^T (b y)
    uint4 by[PS][JS];
#pragma unroll
    for (int js = 0; js < JS; ++js) {
      float w[E], b[E];
      F32::ld<E>(we + KS * js + E * g, w);
      F32::ld<E>(bt + KS * js + E * g, b);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int t = tile_of<IO>(js, i);
        X[t][i & 3] = Y[t][i & 3] + times(w[i], X[t][i & 3]);
        b[i] *= X[t][i & 3];
      }
      uint4 f[PS];
      split<IO, PS>(b, f);
#pragma unroll
      for (int q = 0; q < PS; ++q) by[q][js] = f[q];
    }
    __builtin_amdgcn_sched_barrier(0);
    // What the state before the chunk is made of, one operand after the other: scale e^G dO (with Q's rows), then
    // -e^G b e (with K's); each is split under the products of the one before, the first under those of M.
    uint4 fw[2][PS];
    auto parts = [&](int n) {
      const int js = n % JS;
      float e[E], v[E];
      F32::ld<E>(ek + KS * js + E * g, e);
      if (n < JS) {
        unpack<IO>(fz[js], v);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = times(p.scale * e[i], v[i]);
      } else {
        F32::ld<E>(bt + KS * js + E * g, v);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = -times(e[i], v[i] * X[tile_of<IO>(js, i)][i & 3]);
      }
      split<IO, PS>(v, fw[n & 1]);
    };
    parts(0);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) scale(R[rt], end_dec);
    if constexpr (PS == 3) {
#pragma unroll
      for (int q = 2; q >= 0; --q) times_square(ft, by[q], X);
      mix<LOW * 3, 3>();
      __builtin_amdgcn_sched_barrier(0);
      read_square(tm + 2 * MPART, ft);
      __builtin_amdgcn_sched_barrier(0);
      times_square(fl, by[1], X);
      times_square(fl, by[0], X);
      __builtin_amdgcn_sched_barrier(0);
      times_square(ft, by[0], X);
    } else {
      times_square(ft, by[0], X);
      mix<LOW, 3>();
    }
    __builtin_amdgcn_sched_barrier(0);
    if (kk + 1 < nc) load_late(pc - 1);
    if constexpr (!SEG) keep<IO, IB>(record + kept.rows(1), C, p.cp, cw + li, g, X);

    const int yb0 = state_col_base<IO, NK>(li, g);
#pragma unroll
    for (int n = 0; n < 2 * JS; ++n) {
      const char* const tile = n < JS ? tx : ty;
      constexpr int GR = ROWS == 256 ? 2 : 4;  // rows' operands read together
      uint4 fx[2][GR];
#pragma unroll
      for (int i = 0; i < GR; ++i) fx[0][i] = frag_state_col<IO, NK>(tile, yb0, i, n % JS);
#pragma unroll
      for (int r = 0; r < RT / GR; ++r) {
        if (r + 1 < RT / GR) {
#pragma unroll
          for (int i = 0; i < GR; ++i) fx[(r + 1) & 1][i] = frag_state_col<IO, NK>(tile, yb0, GR * (r + 1) + i, n % JS);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (r == 0 && n + 1 < 2 * JS) parts(n + 1);
#pragma unroll
        for (int q = 0; q < PS; ++q)
#pragma unroll
          for (int i = 0; i < GR; ++i) R[GR * r + i] = mma<IO>(fx[r & 1][i], fw[n & 1][q], R[GR * r + i]);
        mix<GR * PS, 5>();
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  const int g = (tid & 63) >> 4, c = cw + (tid & 15);
  if constexpr (SEG) store_state<IO, RT>(p.seg_state + (bh * p.nseg + seg) * wsize, p.rp, p.cp, p.cp, c, g, R);
  else if (p.last != nullptr && seg == 0) store_state<IO, RT>(p.last + bh * p.rows * p.cols, p.rows, p.cols, p.cols, c, g, R);
}

// The backward's two walks need nothing of each other: the first half of the workgroups walks forwards, the second half
// backwards, so that the stores of one lie under the products of the other (forward and backward of 4 x 2048 tokens, 32
// heads of 128 x 128, bfloat16, 903 us for 983 with a launch each; of 4 x 1999 ragged tokens, 24 heads of 64, float32, 571
// for 706).  Now 306 and 213 of it.  SEG: the segments' own ends.
template <typename IO, int ROWS, int NW, bool SEG, bool VEC>
__global__ void __launch_bounds__((64 * NW), (walk_waves<IO, ROWS, NW>())) ssm_delta_both_kernel(const DeltaDev p, const DeltaDev r, uint32_t first) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  if (blockIdx.x < first) delta_walk<IO, ROWS, NW, SEG ? kDeltaSeg : kDeltaStates, VEC>(p, blockIdx.x, lds);
  else delta_walk_back<IO, ROWS, NW, SEG, VEC>(r, blockIdx.x - first, lds);
}

// ---------------------------------------------------------------- the gradients, all chunks at once

struct DeltaGradDev {
  DeltaDev f;                  // q, k, rates, kept, sizes; v is dO
  char* dq;                    // [b][L][H / hn][rows]; float32 parts with `parts`
  char* dk;
  char* dv;                    // [b][L][H][cols]
  char* dg;                    // [b][L][H], nullable
  char* db;                    // [b][L][H], nullable
  int hn;                      // heads of a group that a workgroup adds up
  int parts;
};

// The scores' gradients take the place of the slab once it is done with.
// The sums over the heads of a key head lie in LDS where the registers do not hold them and it has room.
template <typename IO, int ROWS, bool MULTI>
constexpr bool sums_in_lds() { return MULTI && ROWS == 128 && HeadCfg<IO>::ES == 2; }
template <typename IO, int ROWS, int NW, bool MULTI>
constexpr size_t grad_lds_bytes() {
  using K = HeadCfg<IO>;
  constexpr size_t slab = size_t(K::C) * kSlab * K::ES * (1 + 2 * DeltaCfg<IO>::PAIR);
  constexpr size_t sc = size_t(2) * K::C * K::C * K::ES * DeltaCfg<IO>::PAIR;
  constexpr size_t sums = sums_in_lds<IO, ROWS, MULTI>() ? 2 * size_t(K::C) * ROWS * 4 : 0;
  return 2 * size_t(K::C) * ROWS * K::ES + (slab > sc ? slab : sc) + (size_t(2) * NW + kRates + 1) * K::C * 4 + NW * 4 + sums;
}

// Running sum from the last lane as a pair of floats (scan_pair's, the other way round)
__device__ __forceinline__ void scan_back(float& hi, float& lo) {
  lo = 0.f;
  scan_step<0x101, 0xf>(hi, lo);  // one lane down within a row of 16
  scan_step<0x102, 0xf>(hi, lo);
  scan_step<0x104, 0xf>(hi, lo);
  scan_step<0x108, 0xf>(hi, lo);
  const int row = (threadIdx.x & 63) >> 4;
  float h = 0.f, l = 0.f;  // what the rows further on hold together
#pragma unroll
  for (int r = 3; r > 0; --r) {
    const float th = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(hi), 16 * r));
    const float tl = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(lo), 16 * r));
    const float s = h + (row < r ? th : 0.f), bb = s - h;
    l += ((h - (s - bb)) + ((row < r ? th : 0.f) - bb)) + (row < r ? tl : 0.f);
    h = s;
  }
  const float s = h + hi, bb = s - h;
  lo = (l + lo) + ((h - (s - bb)) + (hi - bb));
  hi = s;
}

// dg_t = <dLoss/dS~_t, S~_t> telescopes within the chunk:
//   dg_t = sum_{i >= t} (q_i . dq_i - k_i . dk^+_i + k_i . dk^-_i) + e^{G_C} <R_C, S_0> + sum_i k_i . w_i R_C u_i
// with dk^+ the key's gradient as what is written (first three terms of dk above), dk^- as what is taken out (the
// last two), each without a token's own pair scale (q . k)(do . u), which is in both and cancels.  Where the state
// starts anew (a decay of -inf) dg is zero and the sum of the tokens before begins there.
//
// In bfloat16 the states, r and e are two bfloat16 parts each, off by 2^-17 at most: dg cancels, and with one part of float16
// (261 us for 330, 4 x 2048 tokens, 32 heads of 128 x 128 on 16 key heads) its error is twice its own rounding.  <R_C, S_0>
// is of the float32 values.  A workgroup a CU, so that nothing covers what it waits for at its start and between its
// barriers; 3.0 TB/s.  Loads are one or two steps of states and, where the registers hold it, a slab ahead.
//
// MULTI adds up the heads of a key head in the workgroup: 4 x 2048 tokens, 32 heads of 128 x 128 on 8 key heads, bfloat16,
// 637 us for the whole backward, 709 with key heads of their own (more loads and stores of keys' gradients).  The next
// slab's loads then go out behind the products (64 keys, M in two parts: 304 us, ahead of them, with 42 spilled registers, 347).
// A workgroup is on its CU alone in bfloat16 past 64 keys (its registers), two or three in float32 with one head (4 x 2048
// tokens, 32 heads of 64 x 64: the backward 468 us; bfloat16 335 with two).
template <typename IO, int ROWS, int NW, bool MULTI>
constexpr int grad_waves() { return HeadCfg<IO>::ES == 4 && !MULTI ? (ROWS == 128 ? 4 : ROWS == 64 ? 3 : 2) : 2; }

template <typename IO, int ROWS, int NW, bool MULTI, bool VEC>
__global__ void __launch_bounds__((64 * NW), (grad_waves<IO, ROWS, NW, MULTI>())) ssm_delta_grad_kernel(const DeltaGradDev d) {
  using K = HeadCfg<IO>;
  const DeltaDev& p = d.f;
  constexpr int ES = K::ES, E = K::E, KS = K::KS, C = K::C, T = 64 * NW;
  constexpr int NK = ROWS * ES / 16, NS = kSlab * ES / 16, NP = C * ES / 16;
  constexpr int IB = C / 16, JS = C / KS, SS = kSlab / KS, CT = ROWS / 16 / NW;
  constexpr int PP = DeltaCfg<IO>::PAIR, SB = C * kSlab * ES, PB = C * C * ES, GAP = KS == 32 ? IB / 2 : 0;  // tiles above the diagonal that a product step covers
  constexpr int TILES = IB * (IB + 1) / 2, MINE = (2 * TILES + NW - 1) / NW;
  // loads of states under way, and operands of blocks and of scores read ahead: two where the registers hold them
  constexpr int AHEAD = PP == 1 || (!MULTI && ROWS <= 128) ? 2 : 1, NB = AHEAD, NT = AHEAD;
  constexpr bool LATE = MULTI && PP == 2;  // the next slab's loads behind the products, for their registers
  constexpr bool SUMS = sums_in_lds<IO, ROWS, MULTI>();
  constexpr int TASKS = C * NS / T;  // staging tasks a thread, rows tid / NS + i T / NS
  static_assert(C * NS % T == 0 && CT >= 1 && SS % 2 == 0, "shares are even");
  using TK = Tile<IO, NK, T>;
  using TR = Flat<kRates * C * 4, T>;

  extern __shared__ __attribute__((aligned(16))) char lds[];
  char* const tx = lds;
  char* const ty = tx + C * ROWS * ES;
  char* const tdo = ty + C * ROWS * ES;  // dO, b r, b e of kSlab columns
  char* const tu = tdo + SB;
  char* const te = tu + PP * SB;
  char* const tp = tdo;                  // in their place dP, then dN
  char* const tn = tp + PP * PB;
  float* const rt = reinterpret_cast<float*>(tdo + ((1 + 2 * PP) * SB > 2 * PP * PB ? (1 + 2 * PP) * SB : 2 * PP * PB));  // [kRates][C]
  const float* const ghi = rt + kGHi * C;
  const float* const glo = rt + kGLo * C;
  const float* const ek = rt + kEk * C;
  const float* const we = rt + kWe * C;
  const float* const bt = rt + kBeta * C;
  const float* const anew = rt + kAnew * C;
  float* const own = rt + kRates * C;  // scale do . u of a token's own
  float* const red = own + C;       // [NW][C]
  float* const redc = red + NW * C;
  float* const rs = redc + NW * C;  // [NW]
  f32x4* const sums = reinterpret_cast<f32x4*>(rs + NW) + threadIdx.x;  // [CT][IB][2][T]: the thread's DQ and DK

  const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int heads = MULTI ? d.hn : 1;  // of a key head that the workgroup adds up
  const int groups = p.H / heads;
  const int pc = blockIdx.x % p.nch, bg = blockIdx.x / p.nch, hg = bg % groups, b = bg / groups, t0 = pc * C;
  const int len = length_of(p, b);
  const int oes = d.parts ? 4 : ES;
  const uint32_t ots = static_cast<uint32_t>(groups * p.rows * oes), vts = p.H * p.cols * ES;
  const int64_t row0 = static_cast<int64_t>(b) * p.L + t0;

  // the head's, and the sums over the heads that share a key head (one head: none)
  f32x4 dq[CT][IB], ur[CT][IB], DQ[MULTI && !SUMS ? CT : 1][IB], DK[MULTI && !SUMS ? CT : 1][IB];
#pragma unroll
  for (int c = 0; c < CT; ++c)
#pragma unroll
    for (int i = 0; i < IB; ++i) {
      dq[c][i] = ur[c][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (SUMS) sums[2 * (c * IB + i) * T] = sums[(2 * (c * IB + i) + 1) * T] = f32x4{0.f, 0.f, 0.f, 0.f};
      else if (MULTI) DQ[c][i] = DK[c][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

  if (t0 < len) {
    constexpr int KW = E / 4;  // 16-byte loads for the E kept values of an operand
    const int hk = hg * heads / p.rep, nslab = p.cp / kSlab;
    const Kept<IO> kept(p.rp, p.cp);
    const int64_t chunk0 = (static_cast<int64_t>(b) * p.H + hg * heads) * p.nch + pc;  // of head hh: hh nch further
    // What a thread has in flight: its part of a slab's dO, r and e, and the operands S_0 and R_C of its wavefront for
    // the next two steps.
    uint4 go[TASKS], gr[TASKS][KW], ge[TASKS][KW], s0[AHEAD][CT][KW], r1[AHEAD][CT][KW], rr[TR::CNT];
    auto record = [&](int hh) {
      return make_rsrc(p.kept + (chunk0 + static_cast<int64_t>(hh) * p.nch) * kept.bytes(), kept.bytes());
    };
    auto values_at = [](Rsrc r, uint32_t off, uint32_t part, uint4* to) {
#pragma unroll
      for (int i = 0; i < KW; ++i) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, part, 0);
        to[i] = make_uint4(v.x, v.y, v.z, v.w);
      }
    };
    auto load_slab = [&](Rsrc rec, int hh, int v0) {
      const Rsrc rdo = make_rsrc(p.v + b * p.v_b + static_cast<int64_t>(t0) * p.v_t + static_cast<int64_t>(hg * heads + hh) * p.cols * ES,
                                 row_bytes(len - t0, C, p.v_t));
#pragma unroll
      for (int i = 0; i < TASKS; ++i) {
        const int me = opaque(tid), r = me / NS + i * (T / NS), col = v0 + me % NS * E;
        go[i] = load16<IO, VEC>(rdo, r * p.v_t + col * ES, p.cols - col);
        values_at(rec, (r * p.cp + col) * 4, kept.rows(0), gr[i]);
        values_at(rec, (r * p.cp + col) * 4, kept.rows(1), ge[i]);
      }
    };
    // rows' block c of step n of a head
    auto load_states = [&](Rsrc rec, int n, int to, int c) {
      const int me = opaque(lane), col = KS * n + E * (me >> 4), row = (wave * CT + c) * 16;
      const uint32_t off = row < p.rp ? static_cast<uint32_t>((row + (me & 15)) * p.cp + col) * 4 : kOOB;
      values_at(rec, off, kept.state(0), s0[to][c]);
      values_at(rec, off, kept.state(1), r1[to][c]);
    };
    {
      uint4 rx[TK::CNT], ry[TK::CNT];
      TK::template load<VEC>(p.q + b * p.q_b + static_cast<int64_t>(hk) * p.rows * ES, p.q_t, t0, len, p.rows, tid, rx);
      TK::template load<VEC>(p.k + b * p.k_b + static_cast<int64_t>(hk) * p.rows * ES, p.k_t, t0, len, p.rows, tid, ry);
      TR::load(reinterpret_cast<const char*>(p.rates + chunk0 * kRates * C), tid, rr);
      load_slab(record(0), 0, 0);
#pragma unroll
      for (int n = 0; n < AHEAD; ++n)
#pragma unroll
        for (int c = 0; c < CT; ++c) load_states(record(0), n, n, c);
      TK::store(tx, tid, rx);
      TK::store(ty, tid, ry);
    }
    for (int hh = 0; hh < heads; ++hh) {
      const int h = hg * heads + hh;
      __syncthreads();  // the head before is done with the rates
      TR::store(reinterpret_cast<char*>(rt), tid, rr);
      __syncthreads();
      if (hh + 1 < heads) TR::load(reinterpret_cast<const char*>(p.rates + (chunk0 + (hh + 1) * static_cast<int64_t>(p.nch)) * kRates * C), tid, rr);

      f32x4 vs[CT][IB], sc[MINE];
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < IB; ++i) dq[c][i] = ur[c][i] = vs[c][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < MINE; ++i) sc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      float dot_rs = 0.f, dot_b[TASKS] = {};

      for (int v = 0; v < nslab; ++v) {
        const int v0 = v * kSlab;
        if (v > 0) __syncthreads();  // the slab before is done with
        auto floats = [](const uint4* r, float* v) {
          for (int i = 0; i < E; ++i) v[i] = reinterpret_cast<const float*>(r)[i];
        };
        // ---- dO, b r and b e of 64 columns, as parts; dv and the sums of db on the way
        const Rsrc rdv = make_rsrc(d.dv + row0 * vts + static_cast<int64_t>(h) * p.cols * ES, row_bytes(p.L - t0, C, vts));
#pragma unroll
        for (int i = 0; i < TASKS; ++i) {
          const int me = opaque(tid), r = me / NS + i * (T / NS), c = me % NS, col = v0 + c * E;
          const float bb = bt[r];
          float x[E], y[E];
          floats(gr[i], x);
          floats(ge[i], y);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            dot_b[i] = __builtin_fmaf(x[e], y[e], dot_b[i]);
            x[e] *= bb;
            y[e] *= bb;
          }
          const uint32_t off = r * vts + col * ES;
          if constexpr (VEC) {
            BufOf<IO>::type::template st<E>(rdv, col < p.cols ? off : kOOB, y);
          } else {
#pragma unroll
            for (int e = 0; e < E; ++e) BufOf<IO>::type::template st<1>(rdv, col + e < p.cols ? off + e * ES : kOOB, y + e);
          }
          const int to = 16 * (NS * r + (c ^ swz<IO, NS>(r)));
          uint4 w[PP];
          *reinterpret_cast<uint4*>(tdo + to) = go[i];
          split<IO, PP>(x, w);
#pragma unroll
          for (int q = 0; q < PP; ++q) *reinterpret_cast<uint4*>(tu + q * SB + to) = w[q];
          split<IO, PP>(y, w);
#pragma unroll
          for (int q = 0; q < PP; ++q) *reinterpret_cast<uint4*>(te + q * SB + to) = w[q];
        }
        __syncthreads();
        // the next slab is this head's or the next one's
        const bool more = v + 1 < nslab, any = more || hh + 1 < heads;
        const int hn = more ? hh : hh + 1, vn = more ? v + 1 : 0;
        const Rsrc rec = record(hn);
        if (!LATE && any) load_slab(rec, hn, vn * kSlab);
        const int fb = opaque(lane_base<IO, NS>(li, g));
#pragma unroll
        for (int s = 0; s < SS; ++s) {
          // the next block's operands are read before the present one's products
          uint4 fo[NB], fu[NB][PP], fe[NB][PP], fx[NT][PP], fy[NT][PP];
          auto read = [&](int ib) {
            fo[ib % NB] = frag_row<NS>(tdo, fb, ib, s);
#pragma unroll
            for (int q = 0; q < PP; ++q) {
              fu[ib % NB][q] = frag_row<NS>(tu + q * SB, fb, ib, s);
              fe[ib % NB][q] = frag_row<NS>(te + q * SB, fb, ib, s);
            }
          };
          // tiles of dP, then of dN, dealt to the wavefronts: lane holds j = 4 g + v of i = li.  dO is one part: its second
          // is b e's, which is not multiplied.
          auto read_scores = [&](int m) {
            const int job = wave + m * NW < 2 * TILES ? wave + m * NW : 0;
            int ib, jb;
            score_tile<IB>(job < TILES ? job : job - TILES, ib, jb);
#pragma unroll
            for (int q = 0; q < PP; ++q) {
              fx[m % NT][q] = frag_row<NS>(tu + q * SB, fb, jb, s);
              fy[m % NT][q] = frag_row<NS>(job < TILES && q == 0 ? tdo : te + q * SB, fb, ib, s);
            }
          };
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            uint4 fs[PP], fr[PP];
            {
              float x[E], y[E];
              floats(s0[s % AHEAD][c], x);
              floats(r1[s % AHEAD][c], y);
#pragma unroll
              for (int e = 0; e < E; ++e) dot_rs = __builtin_fmaf(x[e], y[e], dot_rs);
              split<IO, PP>(x, fs);
              split<IO, PP>(y, fr);
            }
            if (s + AHEAD < SS) load_states(record(hh), v * SS + s + AHEAD, s % AHEAD, c);
            else if (any) load_states(rec, vn * SS + s + AHEAD - SS, s % AHEAD, c);
            if (NB == 2) read(0);
#pragma unroll
            for (int ib = 0; ib < IB; ++ib) {
              if (NB == 1) read(ib);
              else if (ib + 1 < IB) read(ib + 1);
              if (c + 1 == CT && ib + 1 == IB && NT == 2) read_scores(0);
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int q = 0; q < PP; ++q) {
                dq[c][ib] = mma<IO>(fs[q], fo[ib % NB], dq[c][ib]);
                ur[c][ib] = mma<IO>(fr[q], fu[ib % NB][0], ur[c][ib]);
                vs[c][ib] = mma<IO>(fs[q], fe[ib % NB][0], vs[c][ib]);
                if (q > 0) {
                  ur[c][ib] = mma<IO>(fr[0], fu[ib % NB][q], ur[c][ib]);
                  vs[c][ib] = mma<IO>(fs[0], fe[ib % NB][q], vs[c][ib]);
                }
              }
              __builtin_amdgcn_sched_barrier(0);
            }
          }
#pragma unroll
          for (int m = 0; m < MINE; ++m) {
            if (NT == 1) read_scores(m);
            else if (m + 1 < MINE) read_scores(m + 1);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int q = 0; q < PP; ++q) sc[m] = mma<IO>(fx[m % NT][q], fy[m % NT][0], sc[m]);
            if (PP == 2 && wave + m * NW >= TILES) sc[m] = mma<IO>(fx[m % NT][0], fy[m % NT][PP - 1], sc[m]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
        if (LATE && any) load_slab(rec, hn, vn * kSlab);
      }

      // ---- the scores' gradients to LDS, below the diagonal, and zeros in the tiles above it that a product step covers
      __syncthreads();
      if constexpr (GAP > 0) {
        for (int i = tid; i < 2 * PP * GAP * 16 * (16 / E); i += T) {
          const int part = i / (GAP * 16 * (16 / E)), at = i % (GAP * 16 * (16 / E)), r = at / (16 / E), c = at % (16 / E);
          const int row = (r / 16) * 32 + r % 16, col = ((r / 16) * 32 + 16) / E + c;
          *reinterpret_cast<uint4*>(tp + part * PB + 16 * (NP * row + (col ^ swz<IO, NP>(row)))) = make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int m = 0; m < MINE; ++m) {
        __builtin_amdgcn_sched_barrier(0);
        const int job = wave + m * NW;
        if (job >= 2 * TILES) continue;
        int ib, jb;
        score_tile<IB>(job < TILES ? job : job - TILES, ib, jb);
        const int me = opaque(lane), g = me >> 4, i = 16 * ib + (me & 15), j0 = 16 * jb + 4 * g;
        const float by = job < TILES ? p.scale : -1.f;
        float w[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float dd = __builtin_amdgcn_exp2f((ghi[i] - ghi[j0 + v]) + (glo[i] - glo[j0 + v]));
          w[v] = j0 + v < i ? times(by * dd, sc[m][v]) : 0.f;
          if (job < TILES && j0 + v == i) own[i] = by * sc[m][v];
        }
        char* const to = job < TILES ? tp : tn;
        if constexpr (ES == 2) {
          const int u = 4 * jb + g, at = (i * NP + ((u >> 1) ^ swz<IO, NP>(i))) * 16 + (u & 1) * 8;
          const uint2 hi2 = make_uint2(BF16::cvt2(w[0], w[1]), BF16::cvt2(w[2], w[3]));
          *reinterpret_cast<uint2*>(to + at) = hi2;
          *reinterpret_cast<uint2*>(to + PB + at) = make_uint2(BF16::cvt2(w[0] - bf_lo(hi2.x), w[1] - bf_hi(hi2.x)),
                                                               BF16::cvt2(w[2] - bf_lo(hi2.y), w[3] - bf_hi(hi2.y)));
        } else {
          *reinterpret_cast<float4*>(to + (i * NP + ((4 * jb + g) ^ swz<IO, NP>(i))) * 16) = make_float4(w[0], w[1], w[2], w[3]);
        }
      }
      // <R_C, S_0> of the wavefront
#pragma unroll
      for (int x = 1; x < 64; x *= 2) dot_rs += __shfl_xor(dot_rs, x);
      if (lane == 0) rs[wave] = dot_rs;
      // db: the NS lanes of a row
      if (d.db != nullptr) {
#pragma unroll
        for (int i = 0; i < TASKS; ++i) {
          float x = dot_b[i];
#pragma unroll
          for (int s = 1; s < NS; s *= 2) x += __shfl_xor(x, s);
          const int r = tid / NS + i * (T / NS);
          if (tid % NS == 0 && t0 + r < p.L) {
            IO::template st<1>(reinterpret_cast<typename IO::T*>(d.db) + (row0 + r) * p.H + h, &x);
          }
        }
      }
      // ---- the state's parts scaled: lane holds rows (d_key) 16 (wave CT + c) + 4 g + v of token 16 ib + li
      auto values = [&](const char* tile, int c, int ib, float* v) {
        const int me = opaque(lane), r = 16 * ib + (me & 15), col = 16 * (wave * CT + c) + 4 * (me >> 4);
        IO::template ld<4>(reinterpret_cast<const typename IO::T*>(
                               tile + 16 * (NK * r + (col / E ^ swz<IO, NK>(r))) + col % E * ES), v);
      };
#pragma unroll
      for (int ib = 0; ib < IB; ++ib) {
        __builtin_amdgcn_sched_barrier(0);
        const float fe = ek[16 * ib + li], fw = we[16 * ib + li];
        float dot = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          scale(dq[c][ib], p.scale * fe);
          scale(vs[c][ib], -fe);
          scale(ur[c][ib], fw);
          float kv[4];
          values(ty, c, ib, kv);
#pragma unroll
          for (int v = 0; v < 4; ++v) dot = __builtin_fmaf(kv[v], ur[c][ib][v], dot);
        }
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        if (g == 0) redc[wave * C + 16 * ib + li] = dot;
      }
      __syncthreads();  // scores
      // ---- what the chunk's tokens give each other
      const int pb = opaque(lane_base<IO, NP>(li, g)), pcb = opaque(col_base<IO, NP>(li, g));
      const int kb = opaque(col_base<IO, NK>(li, g));
#pragma unroll
      for (int js = 0; js < JS; ++js) {
        uint4 fk[CT], fq[CT];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          fk[c] = frag_col<IO, NK>(ty, kb, wave * CT + c, js);
          fq[c] = frag_col<IO, NK>(tx, kb, wave * CT + c, js);
        }
#pragma unroll
        for (int ib = 0; ib < IB; ++ib) {
          if (js * KS < 16 * (ib + 1)) {
#pragma unroll
            for (int q = 0; q < PP; ++q) {
              const uint4 fp = frag_row<NP>(tp + q * PB, pb, ib, js), fn = frag_row<NP>(tn + q * PB, pb, ib, js);
#pragma unroll
              for (int c = 0; c < CT; ++c) {
                dq[c][ib] = mma<IO>(fk[c], fp, dq[c][ib]);
                vs[c][ib] = mma<IO>(fk[c], fn, vs[c][ib]);
              }
            }
          }
          if (KS * (js + 1) > 16 * ib) {
#pragma unroll
            for (int q = 0; q < PP; ++q) {
              const uint4 fp = frag_col<IO, NP>(tp + q * PB, pcb, ib, js), fn = frag_col<IO, NP>(tn + q * PB, pcb, ib, js);
#pragma unroll
              for (int c = 0; c < CT; ++c) {
                ur[c][ib] = mma<IO>(fq[c], fp, ur[c][ib]);
                ur[c][ib] = mma<IO>(fk[c], fn, ur[c][ib]);
              }
            }
          }
        }
      }
      // ---- the dots for dg, then a token's own pair
#pragma unroll
      for (int ib = 0; ib < IB; ++ib) {
        __builtin_amdgcn_sched_barrier(0);
        float dot = 0.f;
        const float o = own[16 * ib + li];
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          float qv[4], kv[4];
          values(tx, c, ib, qv);
          values(ty, c, ib, kv);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            dot = __builtin_fmaf(qv[v], dq[c][ib][v], dot);
            dot = __builtin_fmaf(kv[v], vs[c][ib][v] - ur[c][ib][v], dot);
            dq[c][ib][v] = __builtin_fmaf(o, kv[v], dq[c][ib][v]);
            ur[c][ib][v] = __builtin_fmaf(o, qv[v], ur[c][ib][v] + vs[c][ib][v]);
            if (MULTI && !SUMS) {
              DQ[c][ib][v] += dq[c][ib][v];
              DK[c][ib][v] += ur[c][ib][v];
            }
          }
          if (SUMS) {
            sums[2 * (c * IB + ib) * T] += dq[c][ib];
            sums[(2 * (c * IB + ib) + 1) * T] += ur[c][ib];
          }
        }
        dot += __shfl_xor(dot, 16);
        dot += __shfl_xor(dot, 32);
        if (g == 0) red[wave * C + 16 * ib + li] = dot;
      }
      if (d.dg != nullptr) {
        __syncthreads();
        if (wave == 0) {
          float v = 0.f, end = 0.f, edge = 0.f;
          int cut = 0;
          if (lane < C) {
            for (int w = 0; w < NW; ++w) {
              v += red[w * C + lane];
              end += redc[w * C + lane];
            }
            cut = lane + 1 < C && anew[lane + 1] != 0.f;
          }
          for (int w = 0; w < NW; ++w) edge += rs[w];
          float lo, end_lo;
          scan_back(end, end_lo);  // lane 0 has the sum
          end = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(end), 0)) +
                __int_as_float(__builtin_amdgcn_readlane(__float_as_int(end_lo), 0));
          if (lane == C - 1) v += end + times(ek[C - 1], edge);
          // sums from the end
          if (__builtin_amdgcn_ballot_w64(cut) == 0) {
            scan_back(v, lo);
            v += lo;
          } else {
            // lane l takes over those further on unless the state starts anew between
#pragma unroll
            for (int x = 1; x < 64; x *= 2) {
              const float o = __shfl_down(v, x);
              const int a = __shfl_down(cut, x);
              if (lane + x < 64) {
                if (!cut) v += o;
                cut |= a;
              }
            }
          }
          const int t = t0 + lane;
          if (lane < C && t < p.L) {
            const bool none = t >= len || (t == 0 && p.h0 == nullptr) || anew[lane] != 0.f;
            const float out = none ? 0.f : v;
            IO::template st<1>(reinterpret_cast<typename IO::T*>(d.dg) + (row0 + lane) * p.H + h, &out);
          }
        }
      }
    }
  } else {
    // nothing of the chunk exists
    for (int r = wave; r < C && t0 + r < p.L; r += NW) {
      for (int hh = 0; hh < heads; ++hh) {
        const int64_t at = (row0 + r) * p.H + hg * heads + hh;
        const float z = 0.f;
        for (int c = lane; c < p.cols; c += 64) IO::template st<1>(reinterpret_cast<typename IO::T*>(d.dv) + at * p.cols + c, &z);
        if (lane == 0 && d.dg != nullptr) IO::template st<1>(reinterpret_cast<typename IO::T*>(d.dg) + at, &z);
        if (lane == 0 && d.db != nullptr) IO::template st<1>(reinterpret_cast<typename IO::T*>(d.db) + at, &z);
      }
    }
  }

  // ---- dq and dk
  const int64_t out0 = row0 * ots + static_cast<int64_t>(hg) * p.rows * oes;
#pragma unroll
  for (int ib = 0; ib < IB; ++ib) {
    const uint32_t nb = row_bytes(p.L - t0 - 16 * ib, 16, ots);
    const Rsrc rq = make_rsrc(d.dq + out0 + static_cast<int64_t>(16 * ib) * ots, nb);
    const Rsrc rk = make_rsrc(d.dk + out0 + static_cast<int64_t>(16 * ib) * ots, nb);
#pragma unroll
    for (int c = 0; c < CT; ++c) {
      const int col = 16 * (wave * CT + c) + 4 * g;
      const uint32_t off = li * ots + col * oes;
      constexpr bool IN = MULTI && !SUMS;
      const f32x4 xq = SUMS ? sums[2 * (c * IB + ib) * T] : IN ? DQ[IN ? c : 0][ib] : dq[c][ib];
      const f32x4 xk = SUMS ? sums[(2 * (c * IB + ib) + 1) * T] : IN ? DK[IN ? c : 0][ib] : ur[c][ib];
      const float vq[4] = {xq[0], xq[1], xq[2], xq[3]}, vk[4] = {xk[0], xk[1], xk[2], xk[3]};
      if (VEC && !d.parts) {
        BufOf<IO>::type::template st<4>(rq, col < p.rows ? off : kOOB, vq);
        BufOf<IO>::type::template st<4>(rk, col < p.rows ? off : kOOB, vk);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t oe = col + e < p.rows ? off + e * oes : kOOB;
          if (d.parts) {
            BufF32::st<1>(rq, oe, vq + e);
            BufF32::st<1>(rk, oe, vk + e);
          } else {
            BufOf<IO>::type::template st<1>(rq, oe, vq + e);
            BufOf<IO>::type::template st<1>(rk, oe, vk + e);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------- launches

template <typename IO, int ROWS, bool VEC>
hipError_t launch_prep_t(const DeltaDev& p, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  constexpr size_t smem = prep_lds_bytes<IO, ROWS>();
  auto kern = ssm_delta_prep_kernel<IO, ROWS, VEC>;
  if (hipError_t e = allow_lds(kern, smem, allowed); e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(p.batch * p.H * p.nch)), dim3(256), smem, st, p);
  return hipGetLastError();
}

template <typename IO, int ROWS, bool VEC>
hipError_t launch_one_t(const DeltaDev& p, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  constexpr size_t prep = prep_lds_bytes<IO, ROWS>(), walk = delta_lds_bytes<IO, ROWS, 4, 1>();
  constexpr size_t smem = prep > walk ? prep : walk;
  auto kern = ssm_delta_one_kernel<IO, ROWS, VEC>;
  if (hipError_t e = allow_lds(kern, smem, allowed); e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(p.H * p.batch)), dim3(256), smem, st, p);
  return hipGetLastError();
}

template <typename IO, int ROWS, int NW, int MODE, bool VEC>
hipError_t launch_walk_t(const DeltaDev& p, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  constexpr size_t smem = delta_lds_bytes<IO, ROWS, NW, MODE == kDeltaOut ? 1 : 0>();
  const int64_t nrun = MODE == kDeltaSeg ? p.nseg - 1 : p.nseg;
  auto kern = ssm_delta_kernel<IO, ROWS, NW, MODE, VEC>;
  if (hipError_t e = allow_lds(kern, smem, allowed); e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(nrun * p.ntile * p.H * p.batch)), dim3(64 * NW), smem, st, p);
  return hipGetLastError();
}

template <typename IO, int ROWS, int NW, bool SEG, bool VEC>
hipError_t launch_both_t(const DeltaDev& p, const DeltaDev& r, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  constexpr size_t smem = delta_lds_bytes<IO, ROWS, NW, 2>();
  const int64_t runs = (SEG ? p.nseg - 1 : p.nseg) * static_cast<int64_t>(p.H) * p.batch;
  auto kern = ssm_delta_both_kernel<IO, ROWS, NW, SEG, VEC>;
  if (hipError_t e = allow_lds(kern, smem, allowed); e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(runs * (p.ntile + r.ntile))), dim3(64 * NW), smem, st, p, r,
                     static_cast<uint32_t>(runs * p.ntile));
  return hipGetLastError();
}

template <typename IO, int ROWS, int NW, bool MULTI, bool VEC>
hipError_t launch_grad_t(const DeltaGradDev& d, hipStream_t st) {
  static std::atomic<uint64_t> allowed{0};
  constexpr size_t smem = grad_lds_bytes<IO, ROWS, NW, MULTI>();
  auto kern = ssm_delta_grad_kernel<IO, ROWS, NW, MULTI, VEC>;
  if (hipError_t e = allow_lds(kern, smem, allowed); e != hipSuccess) return e;
  const int64_t wgs = static_cast<int64_t>(d.f.batch) * (d.f.H / d.hn) * d.f.nch;
  hipLaunchKernelGGL(kern, dim3(static_cast<unsigned>(wgs)), dim3(64 * NW), smem, st, d);
  return hipGetLastError();
}

template <typename IO, bool VEC>
hipError_t launch_grad_v(const DeltaGradDev& d, hipStream_t st) {
  if (d.hn > 1) return d.f.rows <= 64 ? launch_grad_t<IO, 64, 4, true, VEC>(d, st) : launch_grad_t<IO, 128, 8, true, VEC>(d, st);
  return d.f.rows <= 64    ? launch_grad_t<IO, 64, 4, false, VEC>(d, st)
         : d.f.rows <= 128 ? launch_grad_t<IO, 128, 8, false, VEC>(d, st)
                           : launch_grad_t<IO, 256, 8, false, VEC>(d, st);
}

// Four wavefronts of 16 columns: with eight for 128 the prompts of 8 x 2048 ragged tokens take as long and the training's
// 256 walks of 4 x 2048 tokens, 32 heads of 128 x 128, half as long again.  `wide` is eight, see
// wide_for.
enum { kPassPrep, kPassOne, kPassOut, kPassSeg, kPassBoth, kPassBothSeg };

template <typename IO, int ROWS, int NW, bool VEC>
hipError_t launch_pass_n(const DeltaDev& p, const DeltaDev& r, int pass, hipStream_t st) {
  if (pass == kPassOut) return launch_walk_t<IO, ROWS, NW, kDeltaOut, VEC>(p, st);
  if (pass == kPassSeg) return launch_walk_t<IO, ROWS, NW, kDeltaSeg, VEC>(p, st);
  if (pass == kPassBoth) return launch_both_t<IO, ROWS, NW, false, VEC>(p, r, st);
  return launch_both_t<IO, ROWS, NW, true, VEC>(p, r, st);
}

template <typename IO, int ROWS, bool VEC>
hipError_t launch_pass_r(const DeltaDev& p, const DeltaDev& r, int pass, bool wide, hipStream_t st) {
  if (pass == kPassPrep) return launch_prep_t<IO, ROWS, VEC>(p, st);
  if (pass == kPassOne) return launch_one_t<IO, ROWS, VEC>(p, st);
  if constexpr (VEC && ROWS == 256 && HeadCfg<IO>::ES == 2)
    if (wide) return launch_pass_n<IO, ROWS, 8, VEC>(p, r, pass, st);
  return launch_pass_n<IO, ROWS, 4, VEC>(p, r, pass, st);
}

template <typename IO>
hipError_t launch_pass_io(const DeltaDev& p, const DeltaDev& r, int pass, bool wide, bool vec, hipStream_t st) {
  if (p.rows <= 64) return vec ? launch_pass_r<IO, 64, true>(p, r, pass, wide, st) : launch_pass_r<IO, 64, false>(p, r, pass, wide, st);
  if (p.rows <= 128)
    return vec ? launch_pass_r<IO, 128, true>(p, r, pass, wide, st) : launch_pass_r<IO, 128, false>(p, r, pass, wide, st);
  return vec ? launch_pass_r<IO, 256, true>(p, r, pass, wide, st) : launch_pass_r<IO, 256, false>(p, r, pass, wide, st);
}

template <typename IO>
hipError_t launch_grad_io(const DeltaGradDev& d, bool vec, hipStream_t st) {
  return vec ? launch_grad_v<IO, true>(d, st) : launch_grad_v<IO, false>(d, st);
}

}  // namespace deltak

// One pass (r: the walk backwards, where the pass has one); ROWS is d_key rounded up to 64, 128 or 256.
hipError_t launch_delta_bf16(const deltak::DeltaDev& p, const deltak::DeltaDev& r, int pass, bool wide, bool vec, hipStream_t st);
hipError_t launch_delta_f32(const deltak::DeltaDev& p, const deltak::DeltaDev& r, int pass, bool vec, hipStream_t st);
hipError_t launch_delta_grad_bf16(const deltak::DeltaGradDev& d, bool vec, hipStream_t st);
hipError_t launch_delta_grad_f32(const deltak::DeltaGradDev& d, bool vec, hipStream_t st);

}  // namespace ssm
