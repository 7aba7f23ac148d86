// What the chunked delta kernels share (device code only): fp32 values as
// sums of bf16 planes, matrix-core tiles over them, and the matrices of one
// chunk of 32 tokens.
//
// Chunk form.  With a_t = 1 - alpha_t, G_t = a_1..a_t within the chunk and
// D[t,j] = G_t / G_j, the token recurrence
//   f_t = v_t - a_t W_{t-1} k_t,  W_t = a_t W_{t-1} + theta_t f_t k_t^T
// over a chunk that starts at W is
//   (I + B) F = V - diag(G) K W^T,   B[t,j] = D[t,j] (k_t.k_j) theta_j,  j < t
//   Y = diag(G) Q W^T + P F,         P[t,j] = D[t,j] (q_t.k_j) theta_j,  j <= t
//   W' = G_C W + (diag(E theta) F)^T K,  E_j = G_C / G_j.
// F holds the residuals themselves, so theta = 0 divides nothing.
//
// Decays.  D is exp2 of a difference of prefix sums of log2 a, taken in fp64
// and kept as a pair of floats, so a difference carries no more error than
// its own rounding however far the sums have run.  a = 0 (alpha = 1) counts
// as log2 a = -2000: every product over it is exactly 0.
//
// Precision.  A float is the exact sum of three bf16 numbers (8 bits each,
// by truncation).  A product of two floats keeps the six partial products
// down to 2^-16 (the three dropped ones are below 2^-24 of it), a product
// with a bf16 input, which is its own first plane, the three that exist: so
// the bf16 matrix cores (16 times the fp32 ones' rate) give fp32 results.
// That holds for bf16 outputs too: where a large old association is
// overwritten, y is a small difference of terms of the old one's size, and
// factors of two planes would leave it 2^-17 of that size off.
#pragma once

#include "tm_internal.h"

namespace titans {
namespace {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

constexpr int kC = 32;          // tokens per chunk
// (unsigned: n may be 2^31 - 1)
__host__ __device__ inline int chunks_of(int n) { return (int)(((unsigned)n + kC - 1) / kC); }
constexpr int kCS = kC + 8;     // row stride of a [32][32] plane, in bf16
constexpr int kBS = kC + 4;     // row stride of the fp32 scratch

__device__ __forceinline__ uint32_t bits(float x) { return __builtin_bit_cast(uint32_t, x); }
__device__ __forceinline__ float flt(uint32_t x) { return __builtin_bit_cast(float, x); }
__device__ __forceinline__ float top(float x) { return flt(bits(x) & 0xffff0000u); }
// the bf16 halves of two floats side by side
__device__ __forceinline__ uint32_t tops(float a, float b) { return __builtin_amdgcn_perm(bits(b), bits(a), 0x07060302u); }

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// A 16x16 accumulator tile has column l % 16 and rows 4 (l / 16) + 0..3 in
// lane l; an operand has 8 contraction indices a lane.  Two stacked tiles are
// therefore an operand over 32 rows without a move, if both operands run
// through those rows in the order 4g..4g+3, 16+4g..16+4g+3 for lane group g.
// Every 32-long contraction axis in LDS is stored in that order, so that an
// operand is one 16-byte read: element e of the axis lies at perm32(e).
__device__ __forceinline__ constexpr int perm32(int e) { return ((e & 15) >> 2) * 8 + (e >> 4) * 4 + (e & 3); }

// Two stacked tiles as NP planes of one operand.
template <int NP>
__device__ __forceinline__ void split8(const f32x4& a, const f32x4& b, bf16x8 (&out)[NP]) {
  float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    const u32x4 u = {tops(x[0], x[1]), tops(x[2], x[3]), tops(x[4], x[5]), tops(x[6], x[7])};
    out[p] = __builtin_bit_cast(bf16x8, u);
    if (p + 1 < NP) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] -= top(x[i]);
    }
  }
}

// Four consecutive values of one row to NP planes in LDS.
template <int NP>
__device__ __forceinline__ void put4(uint16_t* at, int plane, float x0, float x1, float x2, float x3) {
#pragma unroll
  for (int p = 0; p < NP; ++p) {
    *(uint2*)(at + p * plane) = make_uint2(tops(x0, x1), tops(x2, x3));
    x0 -= top(x0), x1 -= top(x1), x2 -= top(x2), x3 -= top(x3);
  }
}

// Both row tiles (the second `step` further on) of one 32-long step of A from
// LDS, in NA planes `plane` apart.
template <int NA>
__device__ __forceinline__ void read2(const uint16_t* a, int plane, int step, bf16x8 (&av)[2][NA]) {
#pragma unroll
  for (int i = NA - 1; i >= 0; --i)
#pragma unroll
    for (int t = 0; t < 2; ++t) av[t][i] = *(const bf16x8*)(a + i * plane + t * step);
}

// The products of planes kept for operands of NA and NB planes, those with
// i + j < max(NA, NB), smallest first.
struct Planes {
  int i, j;
};
template <int NA, int NB>
constexpr int products() {
  int n = 0;
  for (int i = 0; i < NA; ++i)
    for (int j = 0; j < NB; ++j) n += i + j < (NA > NB ? NA : NB);
  return n;
}
template <int NA, int NB>
constexpr Planes product(int which) {
  for (int o = (NA > NB ? NA : NB) - 1; o >= 0; --o)
    for (int i = NA - 1; i >= 0; --i)
      if (o - i >= 0 && o - i < NB && which-- == 0) return {i, o - i};
  return {0, 0};
}

// c += A B for the two tiles, by the which-th of these products.  SWAP: the
// product's transpose (an operand's lanes hold the same values on either side).
template <bool SWAP, int NB, int NA, int MB>
__device__ __forceinline__ void mul2_one(int which, const bf16x8 (&av)[2][NA], const bf16x8 (&b)[MB], f32x4 (&c)[2]) {
  static_assert(NB <= MB, "planes of B");
  const Planes x = product<NA, NB>(which);
#pragma unroll
  for (int t = 0; t < 2; ++t) c[t] = SWAP ? mfma(b[x.j], av[t][x.i], c[t]) : mfma(av[t][x.i], b[x.j], c[t]);
}

// All of them, the two tiles' accumulation chains in turn.  B may have more
// planes than the NB that take part.
template <bool SWAP, int NB, int NA, int MB>
__device__ __forceinline__ void mul2(const bf16x8 (&av)[2][NA], const bf16x8 (&b)[MB], f32x4 (&c)[2]) {
#pragma unroll
  for (int which = 0; which < products<NA, NB>(); ++which) mul2_one<SWAP, NB>(which, av, b, c);
}

// Keeps what is written before it ahead of what is written after it.
__device__ __forceinline__ void in_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The operand A[m][k] of a [k][m] array (row stride rs in bf16, k = 32 tokens in their natural row order, m0 the tile's
// first column; PERM: its rows
// are permuted): the hardware's transposing read gives a group of 16 lanes 4 rows by 16 columns, a column per lane.
template <bool PERM>
__device__ __forceinline__ bf16x8 read_transposed(const uint16_t* base, int rs, int m0, int lane) {
  typedef __attribute__((address_space(3))) bf16x4 lds4;
  // columns 4c..4c+3 of a permuted row are contiguous, at perm32
  const int col = m0 + 4 * (lane & 3), at = PERM ? (col & ~31) + perm32(col & 31) : col;
  const uint16_t* p0 = base + (4 * (lane >> 4) + ((lane & 15) >> 2)) * rs + at;
  const bf16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)p0);
  const bf16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(p0 + 16 * rs));
  return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Orders a wave's own LDS traffic between lanes.
__device__ __forceinline__ void wave_fence() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// 2^x in one instruction, 0 below 2^-126
__device__ __forceinline__ float exp2_of(float x) { return __builtin_amdgcn_exp2f(x); }

// a double moved by a DPP control (0 where no lane supplies it), and one lane's
template <int CTRL>
__device__ __forceinline__ double dpp_f64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xf, 0xf, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double lane_f64(double x, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane((int)(uint32_t)u, lane);
  const uint32_t hi = __builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), lane);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// log2(1 - alpha), at least `floor` (-2000: alpha = 1 gives exact zeros); NaN
// for alpha above 1.  1 - alpha is rounded, by
// u; log2 u (-alpha) / (u - 1) is log2(1 - alpha) to a few units in the last
// place, as log x / (x - 1) hardly changes over one rounding of x.
constexpr float kForget = -2000.f;
__device__ __forceinline__ float log2_keep(float alpha, float floor = kForget) {
  const float u = 1.f - alpha, x = u - 1.f;
  const float l = x == 0.f ? -alpha * 1.44269504088896f : __builtin_amdgcn_logf(u) * (-alpha * __builtin_amdgcn_rcpf(x));
  return l < floor ? floor : l;
}

// LDS of one chunk: NP planes of K and Q, three of T = (I + B)^-1 and of P,
// per-token factors, and VC columns of V.  T's upper right block is zeroed once.
template <int DP, int NP, int VC>
struct ChunkLds {
  static constexpr int RS = DP + 8;                 // row stride of K and Q in bf16
  static constexpr int KP = kC * RS, CP = kC * kCS; // plane sizes
  static constexpr int OFF_K = 0, OFF_Q = OFF_K + NP * KP * 2, OFF_T = OFF_Q + NP * KP * 2, OFF_P = OFF_T + 3 * CP * 2,
                       OFF_G = OFF_P + 3 * CP * 2, OFF_V = OFF_G + (2 * kC + 4) * 4,
                       VS = VC + 4,   // row stride of V: bf16, or fp32 where NP is 3
                       BYTES = OFF_V + kC * VS * (NP == 1 ? 2 : 4);
  static_assert(3 * CP * 2 >= kC * kBS * 4, "the fp32 scratch lies where P comes to lie");
  static_assert(16 * kCS * 2 >= 3 * kC * 4, "the gates' scratch lies in T's lower half");
  unsigned char* base;
  __device__ uint16_t* k() const { return (uint16_t*)(base + OFF_K); }
  __device__ uint16_t* q() const { return (uint16_t*)(base + OFF_Q); }
  __device__ uint16_t* t() const { return (uint16_t*)(base + OFF_T); }
  __device__ uint16_t* p() const { return (uint16_t*)(base + OFF_P); }
  __device__ float* g() const { return (float*)(base + OFF_G); }          // G_t
  __device__ float* eth() const { return (float*)(base + OFF_G) + kC; }   // E_j theta_j over theta's scale
  __device__ float* gc() const { return (float*)(base + OFF_G) + 2 * kC; }   // G_C, and theta's scale (a power of two)
  __device__ unsigned char* v() const { return base + OFF_V; }
  __device__ float* scratch() const { return (float*)(base + OFF_P); }    // [32][kBS]
  __device__ float* gates() const { return (float*)(base + OFF_T + 16 * kCS * 2); }   // log2 G (hi, lo), theta
};

// Raw rows of a chunk's K or Q on their way from global memory to LDS: the
// loads of a later chunk are in flight while this one is computed.
// F32: fp32 input.  VB: bytes of the pieces that rows consist of and are
// aligned for (16 or 8); 0: any row, element by element and not ahead of
// time (such rows are rare, and their registers would be many).
template <int DP, int COLS, bool F32, int VB>
struct RowLoad {
  static constexpr int PER = VB ? VB / (F32 ? 4 : 2) : 4;    // elements per piece
  static constexpr int PIECES = kC * COLS / PER / 64;        // per lane
  // a lane's i-th piece is at row r, column c; the offsets repeat every P pieces, ROWS rows further down
  static constexpr int ROW = COLS / PER, P = ROW % 3 ? 1 : 3, ROWS = P * 64 / ROW;
  static_assert(P * 64 % ROW == 0 && PIECES % P == 0, "whole rows");
  static __device__ __forceinline__ void place(int i, int lane, int& r, int& c) {
    const int e = i % P * 64 + lane;
    r = e / ROW + i / P * ROWS, c = e % ROW * PER;
  }
  uint32_t raw[VB ? PIECES : 1][VB ? VB / 4 : 1];
  const char* src;
  int n, d, cols;
  // `rows` rows of `real` columns at `from`, d elements apart; the other rows and columns are zero
  __device__ __forceinline__ void load(const char* from, int rows, int width, int real, int lane) {
    src = from, n = rows, d = width, cols = real;
    if constexpr (VB > 0) {
      if (n == kC && d == DP && cols >= COLS) {   // offsets that no chunk changes
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          int r, c;
          place(i, lane, r, c);
          take(i, (r * DP + c) * (F32 ? 4 : 2));
        }
      } else {   // clamped addresses: no branch between the loads
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          int r, c;
          place(i, lane, r, c);
          take(i, (min(r, n - 1) * d + max(min(c, cols - PER), 0)) * (F32 ? 4 : 2));
        }
      }
    }
  }
  __device__ __forceinline__ void take(int i, int at) {
    if constexpr (VB == 16) {
      const u32x4 x = *(const u32x4*)(src + (uint32_t)at);
#pragma unroll
      for (int j = 0; j < 4; ++j) raw[i][j] = x[j];
    } else {
      const uint2 x = *(const uint2*)(src + (uint32_t)at);
      raw[i][0] = x.x, raw[i][1] = x.y;
    }
  }
  // put(row, column, 4 values in order, as stored bits) for every 4 columns
  template <class Put>
  __device__ __forceinline__ void store(int lane, Put put) {
    if constexpr (VB > 0) {
      if (n != kC || cols < COLS) {
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          int r, c;
          place(i, lane, r, c);
#pragma unroll
          for (int j = 0; j < VB / 4; ++j) raw[i][j] = r < n && c < cols ? raw[i][j] : 0u;
        }
      }
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        int r, c;
        place(i, lane, r, c);
#pragma unroll
        for (int j = 0; j < PER; j += 4) put(r, c + j, raw[i] + (F32 ? j : j / 2));
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < PIECES; ++i) {
        int r, c;
        place(i, lane, r, c);
        uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r < n && c + j < cols) {
            if (F32)
              x[j] = ((const uint32_t*)src)[r * d + c + j];
            else
              x[j / 2] |= (uint32_t)((const uint16_t*)src)[r * d + c + j] << (j % 2 * 16);
          }
        put(r, c, x);
      }
    }
  }
};

// Rows of K or Q (from column col0 on) into their permuted planes.
template <int DP, bool F32, class Load>
__device__ __forceinline__ void store_planes(Load& rows, uint16_t* dst, int lane, int col0 = 0) {
  constexpr int RS = DP + 8, KP = kC * RS;
  rows.store(lane, [&](int r, int c, const uint32_t* x) {
    c += col0;
    uint16_t* at = dst + r * RS + (c & ~31) + perm32(c & 31);
    if constexpr (F32)
      put4<3>(at, KP, flt(x[0]), flt(x[1]), flt(x[2]), flt(x[3]));
    else
      *(uint2*)at = make_uint2(x[0], x[1]);
  });
}

// Prefix sums over lanes 0..31 and their total, in fp64, by DPP (16 lanes a row).
__device__ __forceinline__ double prefix_sums(float x, int lane, double& all) {
  double sum = x;
  sum += dpp_f64<0x111>(sum);
  sum += dpp_f64<0x112>(sum);
  sum += dpp_f64<0x114>(sum);
  sum += dpp_f64<0x118>(sum);
  const double half = lane_f64(sum, 15);
  if (lane >= 16) sum += half;
  all = lane_f64(sum, kC - 1);
  return sum;
}

// One wave builds a chunk's matrices in LDS from its K and Q (already stored)
// and its gates (lane t < 32: token t's log2 a and theta; 0 past the end).
// WITH_Q: P too.
template <bool WITH_Q, int DP, int NP, int VC>
__device__ __forceinline__ void build_chunk(const ChunkLds<DP, NP, VC>& L, float la, float th, int lane) {
  using Lds = ChunkLds<DP, NP, VC>;
  const int g = lane >> 4, li = lane & 15;
  double all;
  const double sum = prefix_sums(la, lane, all);
  const float hi = (float)sum;
  // E theta f is split into planes, whose last bits lie 2^-24 below it: where theta alone would bring them near the
  // least fp32 exponent (or theta f near the largest), a power of two is taken out of theta
  float scale = 1.f;
  const float size = lane < kC ? fabsf(th) : 0.f;
  if (__ballot(size > 0x1p40f) || (!__ballot(size >= 0x1p-40f) && __ballot(size > 0.f))) {
    float most = size;
#pragma unroll
    for (int m = 1; m < 64; m *= 2) most = fmaxf(most, __shfl_xor(most, m, 64));
    scale = most < 3.0e38f ? ldexpf(1.f, min(max(ilogbf(most), -100), 100)) : 1.f;
  }
  float* gs = L.gates();
  if (lane < kC) {
    gs[lane] = hi;
    gs[kC + lane] = (float)(sum - (double)hi);
    gs[2 * kC + lane] = th;
    L.g()[lane] = exp2_of(hi);
    L.eth()[lane] = exp2_of((float)(all - sum)) * (th * (1.f / scale));
    if (lane == 0) L.gc()[0] = exp2_of((float)all), L.gc()[1] = scale;
  }
  wave_fence();
  // K K^T and K Q^T by 16x16 tiles (j rows, t columns), j tile <= t tile:
  // 0: j 0 t 0, 1: j 0 t 1, 2: j 1 t 1
  f32x4 kk[3], qk[3];
#pragma unroll
  for (int x = 0; x < 3; ++x) kk[x] = qk[x] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int s = 0; s < DP / 32; ++s) {
    const int at = li * Lds::RS + 32 * s + 8 * g;
    bf16x8 k1[NP], q0[NP], q1[NP], k0[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      k0[i] = *(const bf16x8*)(L.k() + i * Lds::KP + at);
      k1[i] = *(const bf16x8*)(L.k() + i * Lds::KP + 16 * Lds::RS + at);
      if (WITH_Q) {
        q0[i] = *(const bf16x8*)(L.q() + i * Lds::KP + at);
        q1[i] = *(const bf16x8*)(L.q() + i * Lds::KP + 16 * Lds::RS + at);
      }
    }
#pragma unroll
    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
      for (int i = o; i >= 0; --i) {
        kk[0] = mfma(k0[i], k0[o - i], kk[0]);
        kk[1] = mfma(k0[i], k1[o - i], kk[1]);
        kk[2] = mfma(k1[i], k1[o - i], kk[2]);
        if (WITH_Q) {
          qk[0] = mfma(k0[i], q0[o - i], qk[0]);
          qk[1] = mfma(k0[i], q1[o - i], qk[1]);
          qk[2] = mfma(k1[i], q1[o - i], qk[2]);
        }
      }
  }
  // lane: token t = 16 tt + li, tokens j = 16 jt + 4 g + 0..3
  float* sc = L.scratch();
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int tt = x > 0, jt = x > 1, t = 16 * tt + li, j0 = 16 * jt + 4 * g;
    const float th_ = gs[t], tl = gs[kC + t];
    const f32x4 jh = *(const f32x4*)(gs + j0), jl = *(const f32x4*)(gs + kC + j0), tj = *(const f32x4*)(gs + 2 * kC + j0);
    f32x4 b;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float D = exp2_of((th_ - jh[r]) + (tl - jl[r])) * tj[r];
      b[r] = x == 1 || t > j0 + r ? D * kk[x][r] : 0.f;
      qk[x][r] = x == 1 || t >= j0 + r ? D * qk[x][r] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) sc[(j0 + r) * kBS + t] = b[r];
  }
  wave_fence();
  // the two diagonal blocks' inverses: lane (block, column) by forward
  // substitution (stable for any B), a solved row taken out of all later ones
  // at once; B's columns are read two ahead
  {
    const float* Bt = sc + 16 * (g & 1) * (kBS + 1);   // this block of B^T
    f32x4 col[15][4];
    auto read = [&](int j) {
#pragma unroll
      for (int e = (j + 1) / 4; e < 4; ++e) col[j][e] = *(const f32x4*)(Bt + j * kBS + 4 * e);
    };
    float T[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) T[r] = r == li ? 1.f : 0.f;
    read(0);
    read(1);
#pragma unroll
    for (int j = 0; j < 15; ++j) {
      if (j % 2 == 0) {
        // (tied to the sums, so that the reads stay two columns ahead and no more)
        asm volatile("" : "+v"(T[j]), "+v"(T[(j + 16) / 2]), "+v"(T[15]) : : "memory");
        in_order();
        if (j + 2 < 15) read(j + 2);
        if (j + 3 < 15) read(j + 3);
      }
#pragma unroll
      for (int r = j + 1; r < 16; ++r) T[r] = fmaf(-col[j][r / 4][r % 4], T[j], T[r]);
    }
    wave_fence();
    if (lane < 32) {   // in B^T's place, transposed too
#pragma unroll
      for (int e = 0; e < 4; ++e)
        *(f32x4*)(sc + (16 * (g & 1) + li) * kBS + 16 * (g & 1) + 4 * e) = f32x4{T[4 * e], T[4 * e + 1], T[4 * e + 2], T[4 * e + 3]};
    }
  }
  wave_fence();
  // T10^T = -T00^T (B10^T T11^T) in fp32 matrix instructions; the inner
  // product's tile is the second one's operand over rows 4 g + r
  f32x4 x = {0.f, 0.f, 0.f, 0.f}, t10 = x, t00, t11;
  const f32x4 left = *(const f32x4*)(sc + li * kBS + 4 * g);
#pragma unroll
  for (int s = 0; s < 4; ++s)
    x = __builtin_amdgcn_mfma_f32_16x16x4f32(sc[li * kBS + 16 + 4 * s + g], sc[(16 + 4 * s + g) * kBS + 16 + li], x, 0, 0, 0);
#pragma unroll
  for (int r = 0; r < 4; ++r) t00[r] = sc[(4 * g + r) * kBS + li], t11[r] = sc[(16 + 4 * g + r) * kBS + 16 + li];
#pragma unroll
  for (int r = 0; r < 4; ++r) t10 = __builtin_amdgcn_mfma_f32_16x16x4f32(left[r], x[r], t10, 0, 0, 0);
  wave_fence();
  uint16_t* T = L.t() + li * kCS + 8 * g;
  put4<3>(T, Lds::CP, t00[0], t00[1], t00[2], t00[3]);
  put4<3>(T + 16 * kCS, Lds::CP, -t10[0], -t10[1], -t10[2], -t10[3]);
  put4<3>(T + 16 * kCS + 4, Lds::CP, t11[0], t11[1], t11[2], t11[3]);
  if (!WITH_Q) return;
  uint16_t* P = L.p() + li * kCS + 8 * g;
  put4<3>(P, Lds::CP, qk[0][0], qk[0][1], qk[0][2], qk[0][3]);
  put4<3>(P + 4, Lds::CP, 0.f, 0.f, 0.f, 0.f);
  put4<3>(P + 16 * kCS, Lds::CP, qk[1][0], qk[1][1], qk[1][2], qk[1][3]);
  put4<3>(P + 16 * kCS + 4, Lds::CP, qk[2][0], qk[2][1], qk[2][2], qk[2][3]);
}

// A counter in LDS that one wave raises and others wait for.
__device__ __forceinline__ int seen(const int* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP); }
__device__ __forceinline__ void acquire() { __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local"); }
__device__ __forceinline__ void wait_for(const int* p, int value) {
  while (seen(p) < value) __builtin_amdgcn_s_sleep(1);
  acquire();
}
__device__ __forceinline__ void raise_to(int* p, int value, int lane) {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  if (lane == 0) __hip_atomic_store(p, value, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
}


// A workgroup's waves around a ring of NB chunk buffers: CW chain waves, PB
// builders and, for fp32 inputs, a helper for every builder, which splits and
// stores Q and V (a third of a builder's time, and half of its registers).
// Their counters, after the buffers: chunks that a builder has finished, that
// a chain wave has, that a helper has.
template <class Lds, int CW, int PB, int NB, bool HELP>
struct Ring {
  static_assert(NB > PB, "a chunk is consumed while PB are built");
  static constexpr int WAVES = CW + PB * (HELP ? 2 : 1), COUNTERS = CW + 2 * PB,
                       BYTES = NB * Lds::BYTES + COUNTERS * 4;
  unsigned char* smem;
  __device__ int* built() const { return (int*)(smem + NB * Lds::BYTES); }
  __device__ int* used() const { return built() + PB; }
  __device__ int* stored() const { return used() + CW; }
  __device__ Lds buffer(int i) const { return Lds{smem + i % NB * Lds::BYTES}; }
  // counters to zero, and the blocks of T that stay zero; every wave calls it
  __device__ __forceinline__ void init(int wave, int lane) const {
    if (threadIdx.x < COUNTERS) built()[threadIdx.x] = 0;
    for (int x = wave; x < 3 * NB; x += WAVES)
      *(uint2*)(buffer(x / 3).t() + x % 3 * Lds::CP + (lane & 15) * kCS + 8 * (lane >> 4) + 4) = make_uint2(0, 0);
    __syncthreads();
  }
};

// A stream's (or a segment's) rows and gates, for its builders.
struct Rows {
  const char *k, *q, *v;
  const float *alpha, *theta;
  int chunks, n, d, vcols;   // vcols: real columns of v from its address on
};

// Wave `wave` >= CW of a ring: builder pw builds the chunks pw, pw + PB, ...
// (BACK: counted from the sequence's end).  WITH_Q: Q and P too.
template <int DP, bool F32, int VB, int VC, bool WITH_Q, bool BACK, class Lds, int CW, int PB, int NB, bool HELP>
__device__ __forceinline__ void run_builder(const Ring<Lds, CW, PB, NB, HELP>& ring, int wave, int lane, const Rows& in) {
  constexpr int kE = F32 ? 4 : 2;
  const bool helps = HELP && wave >= CW + PB;
  const int pw = wave - CW - (helps ? PB : 0);
  auto first = [&](int i) { return (BACK ? in.chunks - 1 - i : i) * kC; };
  auto wait_free = [&](int i) {
#pragma unroll
    for (int w = 0; w < CW; ++w) wait_for(ring.used() + w, i - NB + 1);
  };
  RowLoad<DP, DP, F32, VB> qr;
  RowLoad<DP, VC, F32, VB> vr;
  auto fetch_qv = [&](int i) {
    if (i >= in.chunks) return;
    const int t0 = first(i), m = min(kC, in.n - t0);
    const int64_t at = (int64_t)t0 * in.d * kE;
    if (WITH_Q) qr.load(in.q + at, m, in.d, in.d, lane);
    vr.load(in.v + at, m, in.d, in.vcols, lane);
  };
  auto store_qv = [&](const Lds& L) {
    if (WITH_Q) store_planes<DP, F32>(qr, L.q(), lane);
    vr.store(lane, [&](int r, int c, const uint32_t* x) {
      if constexpr (F32)
        *(uint4*)((float*)L.v() + r * Lds::VS + c) = make_uint4(x[0], x[1], x[2], x[3]);
      else
        *(uint2*)((uint16_t*)L.v() + r * Lds::VS + c) = make_uint2(x[0], x[1]);
    });
  };
  if (helps) {
    fetch_qv(pw);
    for (int i = pw; i < in.chunks; i += PB) {
      wait_free(i);
      store_qv(ring.buffer(i));
      fetch_qv(i + PB);
      raise_to(ring.stored() + pw, i + 1, lane);
    }
    return;
  }
  RowLoad<DP, DP, F32, VB> kr;
  float al = 0.f, th = 0.f;
  auto fetch = [&](int i) {
    if (i >= in.chunks) return;
    const int t0 = first(i), m = min(kC, in.n - t0);
    kr.load(in.k + (int64_t)t0 * in.d * kE, m, in.d, in.d, lane);
    al = in.alpha[t0 + min(lane, m - 1)];   // (zeroed when used: nothing here waits)
    th = in.theta[t0 + min(lane, m - 1)];
  };
  fetch(pw);
  if (!HELP) fetch_qv(pw);
  for (int i = pw; i < in.chunks; i += PB) {
    const Lds L = ring.buffer(i);
    const bool real = lane < in.n - first(i);
    const float la = real ? log2_keep(al) : 0.f, th0 = real ? th : 0.f;
    wait_free(i);
    store_planes<DP, F32>(kr, L.k(), lane);
    if (!HELP) store_qv(L);
    fetch(i + PB);
    if (HELP)
      wait_for(ring.stored() + pw, i + 1);
    else
      fetch_qv(i + PB);
    wave_fence();
    build_chunk<WITH_Q>(L, la, th0, lane);
    raise_to(ring.built() + pw, i + 1, lane);
  }
}

// A chain wave's 16 columns of W^T from and to the [d x d] state of stream s:
// lane's column `col`, tile i's rows 16 i + 4 g + 0..3.
template <int NT, int VB>
__device__ __forceinline__ void load_state(f32x4 (&S)[NT], const float* W, int s, int col, int d, int g) {
  const bool live = col < d;
  const int64_t at = (int64_t)s * d * d + (int64_t)col * d;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int c = 16 * i + 4 * g;
    S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (VB) {
      if (live && c < d) S[i] = *(const f32x4*)(W + at + c);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool in = live && c + r < d;
        const float w = W[in ? at + c + r : 0];
        S[i][r] = in ? w : 0.f;
      }
    }
  }
}
// Waits for the state's loads here.  Left to its first use, in the chain's
// loop, the wait would be taken every time round, for the loop's own stores.
template <int NT>
__device__ __forceinline__ void arrived(f32x4 (&S)[NT]) {
#pragma unroll
  for (int i = 0; i < NT; ++i) asm volatile("" : "+v"(S[i]));
}
template <int NT, int VB>
__device__ __forceinline__ void store_state(const f32x4 (&S)[NT], float* W, int s, int col, int d, int g) {
  if (col >= d) return;
  float* to = W + (int64_t)s * d * d + (int64_t)col * d;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int c = 16 * i + 4 * g;
    if (VB) {
      if (c < d) *(f32x4*)(to + c) = S[i];
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (c + r < d) to[c + r] = S[i][r];
    }
  }
}

}  // namespace
}  // namespace titans
