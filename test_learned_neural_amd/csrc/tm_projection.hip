// The projection that closes a block ("Titans: Learning to Memorize at Test
// Time", mer.dev notes, section 4.4, "Architectural Details": the output
// projection behind normalization and gating, and the residual connection),
// and its gradient:
//
//   z = x W^T + bias,  out = act(z) + residual
//   dz = dout act'(z),  dx = dz W,  dW = dz^T x,  dbias = sum over rows of dz
//
// All three products are out[r][c] = sum_t P(c, t) Q(r, t), c being contiguous
// in memory: P is an operand's first and Q its second factor, and each lies in
// memory either along t (rows of t) or across it (t counts rows).  A workgroup
// has a tile of out, whose operands go through LDS in slices of 32 or 64 steps of t,
// loaded straight to it kStages - 1 slices ahead.  Accumulators have c in
// registers and r in lanes; they go through LDS once more, so that bias,
// residual and out are met in whole rows.
//
// fp32 factors go through the bf16 matrix cores as three planes each
// (tm_attention.h).
//
// Measured, bf16, 1024 to 1024: 131072 rows with a residual 347 us (a copy of what
// is read and written: 157; the product by the library alone: 213 to 263); the
// gradient of 16384 rows with SiLU 160: slope 26 (at a copy's rate), dx 43, dweight 75
// (twice the work: two planes), its parts 20.  8192^3: 903 to 925 us, 1190 TFLOP/s.  fp32,
// 1001 rows of 500 to 777: 14 to 15 us, the gradient 41: slope 4, dx 21, dweight 18, parts 4;
// 4096 rows, 1024 to 1024, 59 us, 145 TFLOP/s.
#include "tm_attention.h"

namespace titans {
namespace {

using att::bf16x4;
using att::bf16x8;
using att::f32x2;
using att::factor;
using att::f32x4;
using att::f32x8;
using att::f32x16;
using att::lds_bf16x4;
using att::lds_void_ptr;
using att::u32x2;

constexpr int kT = 32;           // steps of t in a slice
// Rows up to which the narrow kernel runs.  bf16, 1024 to 1024, in us, 64 x 64
// tiles second: 16 rows 11.6, 20.9; 64 rows 11.5, 22.7 (4096 to 4096: 27.6, 70.1).
constexpr int kNarrowRows = 64;

// what a slice's end past t is made of
__device__ const float4 kZeros[1] = {};

struct Gemm {
  const void *P, *Q, *Q2;    // Q2: what Q was rounded by, for the parts behind the first half (or null)
  int64_t p_row, q_row;      // elements from one row to the next
  int64_t R, T;              // rows of out, length of the sum
  int C;                     // columns of out
  int64_t per;               // steps of t in a part (a multiple of kT)
  int row_tiles, col_tiles, parts;
  const float* bias;
  const void* residual;
  void *out, *pre;           // out: io type, or fp32 (parts of R C)
  int silu;
};

__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

// ---------------------------------------------------------------- operands
// How rows lie in memory: as whole 16-byte pieces, or as anything.
constexpr int kPieces = 0, kOdd = 1;

// One operand's slice in LDS, and its fragments: EXTENT values of c (or r) by
// KT of t; ALONG: rows are values, else rows are steps of t.
template <bool BF16, bool ALONG, int EXTENT, int THREADS, int KT = kT>
struct Slice {
  typedef typename att::Types<BF16>::elem elem;
  typedef typename att::Types<BF16>::frag frag;
  static constexpr int kSize = BF16 ? 2 : 4;
  static constexpr int PC = 16 / kSize;
  static constexpr int ROWS = ALONG ? EXTENT : KT, COLS = ALONG ? KT : EXTENT;
  static constexpr int RB = COLS * kSize, NC = RB / 16;
  static constexpr int kBytes = ROWS * RB;
  static constexpr int kLoads = kBytes / 16 / THREADS;   // of a thread
  static_assert(kBytes % (16 * THREADS) == 0, "");

  static __device__ __forceinline__ int swz(int r) { return att::swizzle<NC>(r); }

  // A thread's pieces of a slice: their distances from the slice's start (32
  // bits: 256 rows of 2^22 elements), which is the wave's.  Values past the
  // end are some other value (their results are not stored).
  struct Loads {
    uint32_t off[kLoads];

    // values v0 .. `values` - 1 of rows `row` elements apart
    __device__ __forceinline__ Loads(int64_t row, int64_t v0, int64_t values, int tid) {
      const int most = (int)(values - v0 < EXTENT ? values - v0 : EXTENT);
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        const int at = i * THREADS + tid, r = at / NC, c = ((at % NC) ^ swz(r)) * PC;
        const int v = ALONG ? min(r, most - 1) : min(c, max(most - PC, 0));
        off[i] = (uint32_t)((ALONG ? v : r) * (uint32_t)row + (ALONG ? c : v)) * kSize;
      }
    }
    // the slice at step t of the sum straight to LDS; steps from `end` on are zero
    __device__ __forceinline__ void wide(unsigned char* s, const elem* src, int64_t row, int64_t v0, int64_t t, int64_t end,
                                         int tid) const {
      const elem* start = src + (ALONG ? v0 * row + t : t * row + v0);
      const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
      if (t + KT <= end) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          __builtin_amdgcn_global_load_lds((const void*)((const char*)start + off[i]),
                                           (lds_void_ptr)(s + (i * THREADS + wave * 64) * 16), 16, 0, 0);
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int at = i * THREADS + tid, r = at / NC, c = ((at % NC) ^ swz(r)) * PC;
          const void* p = t + (ALONG ? c : r) < end ? (const void*)((const char*)start + off[i]) : (const void*)kZeros;
          __builtin_amdgcn_global_load_lds(p, (lds_void_ptr)(s + (i * THREADS + wave * 64) * 16), 16, 0, 0);
        }
        asm volatile("; the last slice");   // (or the compiler joins the two, and the whole one pays for it)
      }
    }
    // piece i of them alone, without a branch: `left` steps are there
    __device__ __forceinline__ void one(unsigned char* s, const elem* start, int left, int i, int tid) const {
      const int at = i * THREADS + tid, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
      const int t = ALONG ? ((at % NC) ^ swz(at / NC)) * PC : at / NC;
      const void* p = t < left ? (const void*)((const char*)start + off[i]) : (const void*)kZeros;
      __builtin_amdgcn_global_load_lds(p, (lds_void_ptr)(s + (i * THREADS + wave * 64) * 16), 16, 0, 0);
    }
    static __device__ __forceinline__ const elem* start(const elem* src, int64_t row, int64_t v0, int64_t t) {
      return src + (ALONG ? v0 * row + t : t * row + v0);
    }
    // The same into registers, then to LDS, where rows are not made of whole
    // pieces: 16 bytes from any address.  Across, the last piece of a row ends
    // with it, and is shifted into its place on the way to LDS.
    typedef elem Held[kLoads][PC];
    __device__ __forceinline__ void fetch(Held& x, const elem* src, int64_t row, int64_t v0, int64_t values, int64_t t,
                                          int64_t end, int tid) const {
      const elem* from = start(src, row, v0, t);
      const int left = end - t < KT ? (int)(end - t) : KT;
      if (ALONG ? left == KT : values - v0 >= PC) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const void* p = ALONG || (i * THREADS + tid) / NC < left ? (const void*)((const char*)from + off[i]) : (const void*)kZeros;
          __builtin_memcpy(x[i], p, 16);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int at = i * THREADS + tid, r = at / NC, c = ((at % NC) ^ swz(r)) * PC;
#pragma unroll
          for (int e = 0; e < PC; ++e) {   // (across: fewer than PC values)
            const bool there = ALONG ? c + e < left : r < left && c + e < values - v0;
            x[i][e] = there ? *(const elem*)((const char*)from + off[i] + (ALONG || c == 0 ? e * kSize : 0)) : (elem)0.f;
          }
        }
      }
    }
    static __device__ __forceinline__ void put(unsigned char* s, Held& x, int64_t v0, int64_t values, int tid) {
      typedef __attribute__((ext_vector_type(PC))) elem piece;
      if (!ALONG && values - v0 < EXTENT && values - v0 >= PC)
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int at = i * THREADS + tid, by = ((at % NC) ^ swz(at / NC)) * PC + PC - (int)(values - v0);
#pragma unroll
          for (int n = 1; n < PC; n *= 2)
#pragma unroll
            for (int e = 0; e + n < PC; ++e) x[i][e] = by > 0 && (by & n) ? x[i][e + n] : x[i][e];
        }
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        piece v;
#pragma unroll
        for (int e = 0; e < PC; ++e) v[e] = x[i][e];
        *(piece*)(s + (i * THREADS + tid) * 16) = v;
      }
    }
  };

  // value v0 + lane % 32, steps 16 k + 8 (lane / 32) + 0..7
  static __device__ __forceinline__ frag get(const unsigned char* s, int v0, int k, int lane) {
    const int half = lane >> 5;
    if constexpr (ALONG) {
      const int r = v0 + (lane & 31);
      if constexpr (BF16) {
        return *(const frag*)(s + r * RB + ((2 * k + half) ^ swz(r)) * 16);
      } else {
        const f32x4 a = *(const f32x4*)(s + r * RB + ((4 * k + 2 * half) ^ swz(r)) * 16);
        const f32x4 b = *(const f32x4*)(s + r * RB + ((4 * k + 2 * half + 1) ^ swz(r)) * 16);
        return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
      }
    } else if constexpr (BF16) {
      const int l = lane & 15, c = (v0 + (lane & 16)) / 8 + ((l >> 1) & 1), r = 16 * k + 8 * half + (l >> 2);
      const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(s + r * RB + (c ^ swz(r)) * 16 + (l & 1) * 8));
      const bf16x4 b =
          __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(s + (r + 4) * RB + (c ^ swz(r + 4)) * 16 + (l & 1) * 8));
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      frag f;
      const int c = v0 + (lane & 31);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = 16 * k + 8 * half + j;
        f[j] = *(const float*)(s + r * RB + ((c / 4) ^ swz(r)) * 16 + (c & 3) * 4);
      }
      return f;
    }
  }
};

// 8 neighbouring elements of a row, n of which are there; whole: as pieces of 16 bytes
__device__ __forceinline__ f32x8 load8(const __bf16* p, int n, bool whole) {
  if (whole) return __builtin_convertvector(*(const bf16x8*)p, f32x8);
  f32x8 x = {};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) x[e] = (float)p[e];
  return x;
}
__device__ __forceinline__ f32x8 load8(const float* p, int n, bool whole) {
  f32x8 x = {};
  if (whole) {
    const f32x4 a = *(const f32x4*)p;
    f32x4 b = {};
    if (n > 4) b = *(const f32x4*)(p + 4);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) x[e] = p[e];
  return x;
}
__device__ __forceinline__ void store8(__bf16* p, f32x8 x, int n, bool whole) {
  if (whole) {
    *(bf16x8*)p = __builtin_convertvector(x, bf16x8);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e] = (__bf16)x[e];
}
__device__ __forceinline__ void store8(float* p, f32x8 x, int n, bool whole) {
  if (whole) {
    *(f32x4*)p = __builtin_shufflevector(x, x, 0, 1, 2, 3);
    if (n > 4) *(f32x4*)(p + 4) = __builtin_shufflevector(x, x, 4, 5, 6, 7);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) p[e] = x[e];
}

// A wave's accumulators, 32 NR rows from r0 on by 32 NCOL columns from c0 on,
// to memory: 32 rows by W columns at a time through LDS, so that bias, residual
// and out are met in pieces of rows, lines of 128 bytes where NCOL is even.  (A
// wave's LDS operations stay in their order: only the compiler has to keep it.)
template <int NCOL>
constexpr int piece_of() { return NCOL % 2 ? 4096 : 8192; }   // of LDS, a wave's

template <bool BF16, bool F32_OUT, int NR, int NCOL>
__device__ __forceinline__ void finish(const Gemm& g, f32x16 (&acc)[NR][NCOL], unsigned char* mine, int64_t r0, int c0,
                                       int part, int lane) {
  typedef typename att::Types<BF16>::elem elem;
  typedef __attribute__((ext_vector_type(8), aligned(16))) elem elem8;   // (8 floats, too: rows begin at 16 bytes, not 32)
  constexpr int E = NCOL % 2 ? 1 : 2, W = 32 * E, L = W / 8, TURNS = 32 * L / 64;   // lanes of a row, rows' turns
  const bool whole = g.C % (F32_OUT || !BF16 ? 4 : 8) == 0;   // rows of 16-byte pieces
  // The residual may be out, so that no piece of it could pass a store: where
  // pieces are whole, those of 32 rows are sent for ahead of the rows before.
  const bool ahead = !F32_OUT && g.residual && g.C % 8 == 0;
  constexpr int NB = NCOL / E;
  elem8 res[2][F32_OUT ? 1 : NB][TURNS];
  auto send = [&](int a) __attribute__((always_inline)) {
    if constexpr (!F32_OUT) {
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int i = 0; i < TURNS; ++i) {
          const int64_t r = r0 + 32 * a + 64 / L * i + lane / L;
          const int c = c0 + W * b + lane % L * 8;
          if (r < g.R && c < g.C) res[a & 1][b][i] = *(const elem8*)((const elem*)g.residual + r * g.C + c);
        }
    }
  };
  if (ahead) send(0);
#pragma unroll
  for (int a = 0; a < NR; ++a) {
    if (ahead && a + 1 < NR) send(a + 1);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      asm volatile("" ::: "memory");
#pragma unroll
      for (int u = 0; u < 4 * E; ++u) {   // 16-byte chunk c of row r at c ^ (r % chunks)
        const f32x16& x = acc[a][E * b + u / 4];
        const int v = u % 4;
        *(f32x4*)(mine + (lane & 31) * W * 4 + ((2 * u + (lane >> 5)) ^ (lane & (8 * E - 1))) * 16) =
            f32x4{x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]};
      }
      asm volatile("" ::: "memory");
      const int l = lane % L * 2, c = c0 + W * b + 4 * l, n = g.C - c < 8 ? g.C - c : 8;
#pragma unroll
      for (int i = 0; i < TURNS; ++i) {
        const int row = 64 / L * i + lane / L;
        const int64_t r = r0 + 32 * a + row;
        if (r >= g.R || n <= 0) continue;
        const f32x4 x0 = *(const f32x4*)(mine + row * W * 4 + (l ^ (row & (8 * E - 1))) * 16);
        const f32x4 x1 = *(const f32x4*)(mine + row * W * 4 + ((l + 1) ^ (row & (8 * E - 1))) * 16);
        f32x8 x = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
        const int64_t o = r * g.C + c;
        if constexpr (F32_OUT) {
          store8((float*)g.out + (int64_t)part * g.R * g.C + o, x, n, whole);
        } else {
          if (g.bias) x += load8(g.bias + c, n, false);
          if (g.pre) store8((elem*)g.pre + o, x, n, whole);
          if (g.silu)
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] *= sigmoid(x[e]);
          if (ahead)
            x += __builtin_convertvector(res[a & 1][b][i], f32x8);
          else if (g.residual)
            x += load8((const elem*)g.residual + o, n, whole);
          store8((elem*)g.out + o, x, n, whole);
        }
      }
    }
  }
}

// The same of 32 x 32 fp32 sums that SETS waves hold a share of each: every
// wave writes its share to LDS, and stores 32 / SETS rows of the total.  Bias
// and residual are sent for ahead of the product (an element's place in out is
// written by the lane that read its residual).
template <int SETS>
struct Shared {
  static constexpr int ROWS = 32 / SETS, kBytes = 4096;   // of LDS, a wave's
  static_assert(ROWS == 8, "");
  f32x4 bias = {}, res = {};
  int64_t o[4];    // places in out (or -1)
  int at[4];       // in a wave's 32 x 32 sums

  // 4 neighbours a lane where rows are whole pieces, else one each of 4 pairs of rows
  __device__ __forceinline__ Shared(const Gemm& g, int64_t r0, int c0, int set, int lane) {
    const bool whole = g.C % 4 == 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = set * ROWS + (whole ? lane >> 3 : 2 * e + (lane >> 5)), c = whole ? 4 * (lane & 7) + e : lane & 31;
      at[e] = row * 32 + ((c >> 2) ^ (row & 7)) * 4 + (c & 3);
      o[e] = r0 + row < g.R && c0 + c < g.C ? (r0 + row) * g.C + c0 + c : -1;
      if (g.bias && o[e] >= 0) bias[e] = g.bias[c0 + c];
    }
    if (g.residual) {
      if (whole) {
        if (o[0] >= 0) res = *(const f32x4*)((const float*)g.residual + o[0]);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (o[e] >= 0) res[e] = ((const float*)g.residual)[o[e]];
      }
    }
  }
  __device__ __forceinline__ void put(unsigned char* mine, const f32x16& x, int lane) const {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      *(f32x4*)(mine + (lane & 31) * 128 + ((2 * u + (lane >> 5)) ^ (lane & 7)) * 16) =
          f32x4{x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]};
  }
  // shares of the tile lie `apart` bytes from each other
  __device__ __forceinline__ void store(const Gemm& g, const unsigned char* shares, int apart, int part) const {
    f32x4 x = {};
    const bool whole = g.C % 4 == 0;
#pragma unroll
    for (int h = 0; h < SETS; ++h) {
      const float* s = (const float*)(shares + h * apart);
      if (whole)
        x += *(const f32x4*)(s + at[0]);
      else
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] += s[at[e]];
    }
    x += bias;
    f32x4 y = x;
    if (g.silu)
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] *= sigmoid(y[e]);
    y += res;
    float* out = (float*)g.out + (int64_t)part * g.R * g.C;
    if (whole) {
      if (o[0] < 0) return;
      if (g.pre) *(f32x4*)((float*)g.pre + o[0]) = x;
      *(f32x4*)(out + o[0]) = y;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (o[e] >= 0) {
          if (g.pre) ((float*)g.pre)[o[e]] = x[e];
          out[o[e]] = y[e];
        }
    }
  }
};

struct Nothing {
  __device__ __forceinline__ Nothing(const Gemm&, int64_t, int, int, int) {}
};

// Tile `id` of all, part by part: an XCD's tiles run one after the other, and
// walk the columns of 8 row tiles at a time, so that both factors stay in its
// L2.
template <int TR, int TC>
__device__ __forceinline__ void tile_of(const Gemm& g, unsigned id, int& part, int64_t& r0, int& c0) {
  const unsigned tiles = (unsigned)g.row_tiles * g.col_tiles;
  part = id / tiles;
  id -= part * tiles;
  const int group = id / (8 * g.col_tiles), rows = min(8, g.row_tiles - 8 * group);
  id -= group * 8 * g.col_tiles;
  r0 = (int64_t)(8 * group + id % rows) * TR;
  c0 = id / rows * TC;
}

// ---------------------------------------------------------------- the tile kernel
// TR x TC of out by WR x WC waves; by SETS times as many, each set of which
// takes its share of a slice's steps, and whose sums are joined in the end.
// fp32 factors are split where they are used, which takes a SIMD as long as their
// products: with four sets a wave's splitting runs beside others' products
// (two sets and slices of 32 steps: 22 us for 1001 x 777 to 500; this 16 to 17).
template <bool BF16_, int TR_, int TC_, int WR_, int WC_, int STAGES_, int SETS_ = 1, int KT_ = kT>
struct Form {
  static constexpr bool BF16 = BF16_;
  static constexpr int TR = TR_, TC = TC_, WR = WR_, WC = WC_, STAGES = STAGES_, SETS = SETS_, KT = KT_;
  static constexpr int kThreads = 64 * WR * WC * SETS;
};

template <typename S, bool P_ALONG, bool Q_ALONG, int KIND, bool F32_OUT>
__global__ void __launch_bounds__(S::kThreads, 2) gemm_kernel(Gemm g) {
  constexpr bool BF16 = S::BF16;
  constexpr int NR = S::TR / S::WR / 32, NCOL = S::TC / S::WC / 32;
  typedef Slice<BF16, P_ALONG, S::TC, S::kThreads, S::KT> SP;
  typedef Slice<BF16, Q_ALONG, S::TR, S::kThreads, S::KT> SQ;
  typedef typename SP::elem elem;
  typedef typename att::Types<BF16>::op Op;
  constexpr int kStage = SP::kBytes + SQ::kBytes, kLoads = (SP::kLoads + SQ::kLoads);
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  constexpr int kSteps = S::KT / 16 / S::SETS;   // of a wave, in a slice
  const int wr = wave / S::WC % S::WR, wc = wave % S::WC, k0 = S::SETS == 1 ? 0 : wave / (S::WC * S::WR) * kSteps;
  // blocks go round the 8 XCDs
  const unsigned all = (unsigned)g.row_tiles * g.col_tiles * g.parts, share = (all + 7) / 8;
  const unsigned id = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
  if (id >= all || (blockIdx.x >> 3) >= share) return;
  int part, c0;
  int64_t r0;
  tile_of<S::TR, S::TC>(g, id, part, r0, c0);
  const bool second = g.Q2 && part >= g.parts / 2;
  const elem *P = (const elem*)g.P, *Q = (const elem*)(second ? g.Q2 : g.Q);
  const int64_t t0 = (second ? part - g.parts / 2 : part) * g.per, t1 = t0 + g.per < g.T ? t0 + g.per : g.T;
  const int slices = t1 > t0 ? (int)((t1 - t0 + S::KT - 1) / S::KT) : 0;
  const typename SP::Loads load_p(g.p_row, c0, g.C, tid);
  const typename SQ::Loads load_q(g.q_row, r0, g.R, tid);
  typename std::conditional<(S::SETS > 1), Shared<4>, Nothing>::type shared(g, r0 + 32 * wr, c0 + 32 * wc, wave / (S::WR * S::WC), lane);
  // Pieces on their way through registers, of several slices where they are
  // few.  They are held as long, so that memory has as many steps to answer as
  // in the other kinds; kept in one set, it has one.
  constexpr int kSets = KIND == kOdd && kLoads <= 4 ? S::STAGES : 1;
  typename SP::Loads::Held hp[kSets];
  typename SQ::Loads::Held hq[kSets];
  auto issue = [&](unsigned char* s, int i, int set) __attribute__((always_inline)) {
    const int64_t t = t0 + (int64_t)i * S::KT;
    if constexpr (KIND == kPieces) {
      load_p.wide(s, P, g.p_row, c0, t, t1, tid);
      load_q.wide(s + SP::kBytes, Q, g.q_row, r0, t, t1, tid);
    } else {
      load_p.fetch(hp[set % kSets], P, g.p_row, c0, g.C, t, t1, tid);
      load_q.fetch(hq[set % kSets], Q, g.q_row, r0, g.R, t, t1, tid);
    }
  };
  auto put = [&](unsigned char* s, int set) __attribute__((always_inline)) {
    if constexpr (KIND == kOdd) {
      SP::Loads::put(s, hp[set % kSets], c0, g.C, tid);
      SQ::Loads::put(s + SP::kBytes, hq[set % kSets], r0, g.R, tid);
    }
  };
  f32x16 acc[NR][NCOL] = {};
  // slice i + STAGES - 1 goes to `next` (restrict: the transposing reads of
  // this one do not wait for it)
  auto step = [&](const unsigned char* __restrict__ cur, unsigned char* __restrict__ next, int i, int st)
                  __attribute__((always_inline)) {
    const bool more = i + S::STAGES - 1 < slices;
    Op q[kSteps][NR], p[kSteps][NCOL];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
#pragma unroll
      for (int a = 0; a < NR; ++a) q[k][a] = factor(SQ::get(cur + SP::kBytes, 32 * (NR * wr + a), k0 + k, lane));
#pragma unroll
      for (int b = 0; b < NCOL; ++b) p[k][b] = factor(SP::get(cur, 32 * (NCOL * wc + b), k0 + k, lane));
    }
    if (more) issue(next, i + S::STAGES - 1, st + S::STAGES - 1);   // (while the operands come)
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int k = 0; k < kSteps; ++k)
#pragma unroll
      for (int b = 0; b < NCOL; ++b)
#pragma unroll
        for (int a = 0; a < NR; ++a) att::mma(acc[a][b], p[k][b], q[k][a]);
    __builtin_amdgcn_s_setprio(0);
    if (kSets == 1 && more) put(next, 0);
  };
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i)
    if (i < slices) {
      issue(smem + i * kStage, i, i);
      if (kSets == 1 || i == 0) put(smem + i * kStage, i);
    }
  for (int i = 0; i < slices;) {
#pragma unroll
    for (int st = 0; st < S::STAGES; ++st) {   // (places in LDS that are constant)
      // this slice has landed; those issued after it may still be under way
      if (KIND == kOdd)   // (only LDS is waited for)
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
      else if (S::STAGES == 2 || i + S::STAGES - 2 >= slices)
        att::landed();
      else
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S::STAGES - 2) * kLoads) : "memory");
      step(smem + st * kStage, smem + (st + S::STAGES - 1) % S::STAGES * kStage, i, st);
      if (++i >= slices) break;
      if (kSets > 1) put(smem + (st + 1) % S::STAGES * kStage, st + 1);
    }
  }
  __syncthreads();
  if constexpr (S::SETS > 1) {
    static_assert(NR == 1 && NCOL == 1 && !BF16, "");
    constexpr int kPiece = decltype(shared)::kBytes, kWaves = S::WR * S::WC;
    static_assert(kPiece * kWaves * S::SETS <= S::STAGES * kStage, "");
    shared.put(smem + wave * kPiece, acc[0][0], lane);
    __syncthreads();
    shared.store(g, smem + wave % kWaves * kPiece, kWaves * kPiece, part);
  } else {
    constexpr int kPiece = piece_of<NCOL>();
    static_assert(kPiece * S::WR * S::WC <= S::STAGES * kStage, "");
    finish<BF16, F32_OUT>(g, acc, smem + wave * kPiece, r0 + 32 * NR * wr, c0 + 32 * NCOL * wc, part, lane);
  }
}

// ---------------------------------------------------------------- the wide tile kernel
// 256 x 256 of out by 4 waves of 128 x 128, bf16 in whole pieces.  A slice's
// operands are read from LDS by 16 KB a wave for 2^20 products: three quarters
// of the matrix cores' time (waves of 64 x 128, eight of them: all of it).  With
// one wave a SIMD, a step's operands are fetched while the step before it is
// multiplied, and the next slice is on its way.  A slice has 64 steps, so that a
// row's piece is a whole line of the caches (with 32, every line passed from L2
// twice: 0.95 us for 32 steps instead of 0.88).  A workgroup takes tile after
// tile; the next one's first slice is sent for before a tile is written.
constexpr int kWide = 256, kWideT = 64, kWideBlocks = 256;

__global__ void __launch_bounds__(256, 1) wide_kernel(Gemm g) {
  typedef Slice<true, true, kWide, 256, kWideT> SP, SQ;
  constexpr int NR = 4, NCOL = 4, kStage = SP::kBytes + SQ::kBytes;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];   // [2 slices], then a piece for every wave
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave >> 1, wc = wave & 1;
  // blocks go round the 8 XCDs; a block's tiles are gridDim / 8 apart in its XCD's run
  const unsigned all = (unsigned)g.row_tiles * g.col_tiles, share = (all + 7) / 8, stride = gridDim.x >> 3;
  const unsigned first = (blockIdx.x & 7) * share, end = min(first + share, all);
  unsigned id = first + (blockIdx.x >> 3);
  int part, c0;   // (one part)
  int64_t r0;
  const int slices = (int)((g.T + kWideT - 1) / kWideT);
  const __bf16 *P = (const __bf16*)g.P, *Q = (const __bf16*)g.Q;
  typename SP::Loads load_p(g.p_row, 0, kWide, tid);
  typename SQ::Loads load_q(g.q_row, 0, kWide, tid);
  constexpr int kLoads = SP::kLoads + SQ::kLoads;
  // pieces from .. to - 1 of the slice at step t
  auto issue = [&](unsigned char* s, int64_t t, int from, int to) __attribute__((always_inline)) {
    const int left = (int)(g.T - t < kWideT ? g.T - t : kWideT);   // (zero or less behind the last slice)
    const __bf16 *sp = SP::Loads::start(P, g.p_row, c0, t), *sq = SQ::Loads::start(Q, g.q_row, r0, t);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      if (i >= from && i < to) {
        if (i < SP::kLoads)
          load_p.one(s, sp, left, i, tid);
        else
          load_q.one(s + SP::kBytes, sq, left, i - SP::kLoads, tid);
      }
  };
  auto begin = [&]() __attribute__((always_inline)) {   // tile `id`, and its first slice
    tile_of<kWide, kWide>(g, id, part, r0, c0);
    load_p = typename SP::Loads(g.p_row, c0, g.C, tid);
    load_q = typename SQ::Loads(g.q_row, r0, g.R, tid);
    issue(smem, 0, 0, kLoads);
  };
  if (id >= end) return;
  begin();
  bool stores = false;   // 32 of them, at least, were issued behind the slice that is waited for
  for (;;) {
    f32x16 acc[NR][NCOL] = {};
    bf16x8 q[2][NR], p[2][NCOL];
    auto fetch = [&](const unsigned char* cur, int k) __attribute__((always_inline)) {
#pragma unroll
      for (int a = 0; a < NR; ++a) q[k % 2][a] = SQ::get(cur + SP::kBytes, 32 * (NR * wr + a), k, lane);
#pragma unroll
      for (int b = 0; b < NCOL; ++b) p[k % 2][b] = SP::get(cur, 32 * (NCOL * wc + b), k, lane);
    };
    auto multiply = [&](int k) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < NCOL; ++b)
#pragma unroll
        for (int a = 0; a < NR; ++a) att::mma(acc[a][b], p[k % 2][b], q[k % 2][a]);
    };
    // The next step's operands come while one is multiplied, and the next
    // slice's pieces are sent for one by one between the products: together
    // they would hold the wave up for as long as 16 products take.  (restrict:
    // the transposing reads do not wait for the loads under way)
    auto step = [&](const unsigned char* __restrict__ cur, unsigned char* __restrict__ next, int64_t t)
                    __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k + 1 < kWideT / 16; ++k) {
        constexpr int each = kLoads / 2;   // (in the first two steps: they have the third to arrive in)
        fetch(cur, k + 1);
        issue(next, t, each * k, each * (k + 1));
        multiply(k);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);              // a read of LDS,
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);              // a product,
          if (k < 2) __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);   // a load,
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);              // a product
        }
      }
    };
    if (stores)
      asm volatile("s_waitcnt vmcnt(32) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
      att::landed();
    fetch(smem, 0);
#pragma unroll 1
    for (int i = 0; i < slices; ++i) {
      unsigned char* next = smem + (i + 1) % 2 * kStage;
      step(smem + i % 2 * kStage, next, (int64_t)(i + 1) * kWideT);
      att::landed();     // the next slice is there for everyone, and nobody reads this one any more
      fetch(next, 0);    // (behind the last slice: not used)
      multiply(kWideT / 16 - 1);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      }
    }
    const int was_c = c0;
    const int64_t was_r = r0;
    id += stride;
    const bool more = id < end;
    // (the last slice was read before the last barrier; what was fetched behind it is not used)
    if (more) begin();
    finish<true, false>(g, acc, smem + 2 * kStage + wave * piece_of<NCOL>(), was_r + 32 * NR * wr, was_c + 32 * NCOL * wc, 0, lane);
    if (!more) return;
    stores = was_r + kWide <= g.R && was_c + kWide <= g.C && g.C % 8 == 0;
  }
}

// ---------------------------------------------------------------- few rows
// A workgroup has 16 columns and all rows (in blocks of 16) of out; its waves
// share t, every wave taking 32 of each 256 steps, from memory straight to the
// operands, and meet in LDS.  Bound by reading W once: one row, 1024 to 1024, 3.6 us
// (a call: 8.8), 64 rows, 4096 to 4096, 27.6.
template <bool BF16, int BLOCKS, bool VEC>
__global__ void __launch_bounds__(512) narrow_kernel(Gemm g) {
  typedef typename att::Types<BF16>::elem elem;
  typedef typename att::Types<BF16>::frag frag;
  typedef typename att::Types<BF16>::op Op;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c0 = blockIdx.x * 16, v = lane & 15;
  const elem* p = (const elem*)g.P + (int64_t)min(c0 + v, g.C - 1) * g.p_row;
  f32x4 acc[BLOCKS] = {};
  auto get = [&](const elem* row, int t) __attribute__((always_inline)) {
    frag f = {};
    if (VEC) {
      if (t < g.T) {
        if constexpr (BF16) {
          f = *(const frag*)(row + t);
        } else {
          const f32x4 a = *(const f32x4*)(row + t);
          f32x4 b = {};
          if (t + 4 < g.T) b = *(const f32x4*)(row + t + 4);
          f = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = t + e < g.T ? row[t + e] : (elem)0.f;
    }
    return f;
  };
#pragma unroll 4
  for (int t0 = wave * 32; t0 < g.T; t0 += 256) {
    const int t = t0 + 8 * (lane >> 4);
    const Op a = factor(get(p, t));
#pragma unroll
    for (int b = 0; b < BLOCKS; ++b) {
      const int64_t r = 16 * b + v < g.R ? 16 * b + v : g.R - 1;
      const Op x = factor(get((const elem*)g.Q + r * g.q_row, t));
      att::products(a, x, [&](bf16x8 y, bf16x8 z) {
        acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y, z, acc[b], 0, 0, 0);
      });
    }
  }
  __shared__ float red[8][16 * BLOCKS][17];   // [wave][row][column]
#pragma unroll
  for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
    for (int e = 0; e < 4; ++e) red[wave][16 * b + v][4 * (lane >> 4) + e] = acc[b][e];
  __syncthreads();
  for (int i = tid; i < 256 * BLOCKS; i += 512) {
    const int r = i / 16, c = c0 + i % 16;
    if (r >= g.R || c >= g.C) continue;
    float x = g.bias ? g.bias[c] : 0.f, sum = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) sum += red[w][r][i % 16];
    x += sum;
    const int64_t o = (int64_t)r * g.C + c;
    if (g.pre) ((elem*)g.pre)[o] = (elem)x;
    if (g.silu) x *= sigmoid(x);
    if (g.residual) x += (float)((const elem*)g.residual)[o];
    ((elem*)g.out)[o] = (elem)x;
  }
}

// ---------------------------------------------------------------- dz and dbias
// dz = dout act'(pre) and its column sums.  The products read it in the io
// type; dx is of that type too, but dweight is fp32, for which a bf16 dz comes
// with what it was rounded by (dz2: together 16 bits, 2^-16 off at most), the
// second half of a sum twice as long (dweight is 2.5e-6 off; by one plane it would
// be 1.7e-3).  dx, 2.3e-3 off where its own rounding is 1.7e-3, takes one plane: two
// would be its product twice, 43 us of 160 for 16384 rows.  A workgroup has 64
// lanes x PC columns and `per` rows, which its 4 waves share.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) slope_kernel(const void* dout_, const void* pre_, void* dz_, void* dz2_, float* sums,
                                                    int64_t R, int C, int64_t per) {
  typedef typename att::Types<BF16>::elem elem;
  constexpr int PC = VEC ? (BF16 ? 8 : 4) : 1;
  typedef __attribute__((ext_vector_type(PC))) elem piece;
  const elem *dout = (const elem*)dout_, *pre = (const elem*)pre_;
  elem *dz = (elem*)dz_, *dz2 = (elem*)dz2_;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = ((int)blockIdx.x * 64 + lane) * PC;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < R ? r0 + per : R;
  float sum[PC] = {};
  if (c < C)
#pragma unroll 4
    for (int64_t r = r0 + wave; r < r1; r += 4) {
      const int64_t o = r * C + c;
      const piece x = *(const piece*)(dout + o);
      float y[PC];
#pragma unroll
      for (int e = 0; e < PC; ++e) y[e] = (float)x[e];
      if (pre) {
        const piece z = *(const piece*)(pre + o);
        piece hi, lo;
#pragma unroll
        for (int e = 0; e < PC; ++e) {
          const float a = (float)z[e], sg = sigmoid(a);
          y[e] *= sg * fmaf(a, 1.f - sg, 1.f);
          hi[e] = (elem)y[e];
          lo[e] = (elem)(__builtin_isinf((float)hi[e]) ? 0.f : y[e] - (float)hi[e]);   // (an infinity leaves nothing)
        }
        *(piece*)(dz + o) = hi;
        if (BF16) *(piece*)(dz2 + o) = lo;
      }
#pragma unroll
      for (int e = 0; e < PC; ++e) sum[e] += y[e];
    }
  __shared__ float red[4][64 * PC];
#pragma unroll
  for (int e = 0; e < PC; ++e) red[wave][lane * PC + e] = sum[e];
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * PC; i += 256) {
    const int col = (int)blockIdx.x * 64 * PC + i;
    if (col < C) sums[(int64_t)blockIdx.y * C + col] = red[0][i] + red[1][i] + red[2][i] + red[3][i];
  }
}

// out[i] = sum over parts of in[part][i], parts in order; the bias's sums behind the weight's
__global__ void __launch_bounds__(256) parts_kernel(const float* in, int parts, int64_t n, float* out, const float* in2,
                                                    int parts2, int n2, float* out2, unsigned blocks) {
  if (blockIdx.x < blocks) {
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (n % 4 == 0) {
      if (i >= n) return;
      f32x4 s = *(const f32x4*)(in + i);
#pragma unroll 4
      for (int p = 1; p < parts; ++p) s += *(const f32x4*)(in + p * n + i);
      *(f32x4*)(out + i) = s;
    } else {
      for (int64_t j = i; j < n && j < i + 4; ++j) {
        float s = in[j];
        for (int p = 1; p < parts; ++p) s += in[p * n + j];
        out[j] = s;
      }
    }
    return;
  }
  // 16 columns a workgroup, 16 threads a column
  __shared__ float red[16][17];
  const int c = (int)(blockIdx.x - blocks) * 16 + (threadIdx.x & 15), k = threadIdx.x >> 4;
  float s = 0.f;
  if (c < n2)
    for (int p = k; p < parts2; p += 16) s += in2[(int64_t)p * n2 + c];
  red[k][threadIdx.x & 15] = s;
  __syncthreads();
  if (k || c >= n2) return;
  s = 0.f;
  for (int i = 0; i < 16; ++i) s += red[i][threadIdx.x & 15];
  out2[c] = s;
}

// ---------------------------------------------------------------- launches
template <typename S, bool P_ALONG, bool Q_ALONG, int KIND, bool F32_OUT>
hipError_t launch_tiles(Gemm g, hipStream_t stream) {
  constexpr int lds = S::STAGES * (Slice<S::BF16, P_ALONG, S::TC, S::kThreads, S::KT>::kBytes +
                                   Slice<S::BF16, Q_ALONG, S::TR, S::kThreads, S::KT>::kBytes);
  g.row_tiles = (int)((g.R + S::TR - 1) / S::TR), g.col_tiles = (g.C + S::TC - 1) / S::TC;
  const int64_t all = (int64_t)g.row_tiles * g.col_tiles * g.parts;
  auto kernel = gemm_kernel<S, P_ALONG, Q_ALONG, KIND, F32_OUT>;
  hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  kernel<<<(unsigned)((all + 7) / 8 * 8), S::kThreads, lds, stream>>>(g);
  return hipGetLastError();
}

hipError_t launch_wide(Gemm g, hipStream_t stream) {
  constexpr int lds = 2 * 2 * kWide * kWideT * 2 + 4 * piece_of<4>();
  g.row_tiles = (int)((g.R + kWide - 1) / kWide), g.col_tiles = (g.C + kWide - 1) / kWide;
  const int64_t all = (int64_t)g.row_tiles * g.col_tiles;
  hipError_t e = hipFuncSetAttribute((const void*)wide_kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  wide_kernel<<<all < kWideBlocks ? (unsigned)((all + 7) / 8 * 8) : kWideBlocks, 256, lds, stream>>>(g);
  return hipGetLastError();
}

template <bool BF16>
using Large = Form<BF16, BF16 ? 256 : 128, 128, BF16 ? 4 : 2, BF16 ? 1 : 2, BF16 ? 3 : 2>;
template <bool BF16>
using Small = Form<BF16, 64, 64, 2, 2, BF16 ? 6 : 2, BF16 ? 1 : 4, BF16 ? 32 : 64>;   // (a slice is short: more of them on their way)

// Large tiles from three for every four CUs on, small ones below.  1024 to 1024,
// in us, large tiles first: bf16 4096 rows (128 tiles) 25.1, 24.2; 6144 rows 25.9,
// 31.2; 8192 rows 26.9, 38.9; fp32 1536 rows (96 tiles) 55, 43; 3000 rows (192)
// 57, 63; 4096 rows 59, 82.
bool large(int64_t R, int64_t C, int io) {
  const int64_t tr = io == TM_IO_BF16 ? 256 : 128;
  return (R + tr - 1) / tr * ((C + 127) / 128) >= 192;
}

template <bool P_ALONG, bool Q_ALONG, bool F32_OUT, bool BF16, int KIND>
hipError_t launch_sized(const Gemm& g, bool big, hipStream_t stream) {
  return big ? launch_tiles<Large<BF16>, P_ALONG, Q_ALONG, KIND, F32_OUT>(g, stream)
             : launch_tiles<Small<BF16>, P_ALONG, Q_ALONG, KIND, F32_OUT>(g, stream);
}

// Rows made of whole 16-byte pieces, in both factors.
bool whole_pieces(const Gemm& g, int io) {
  const int pc = io == TM_IO_BF16 ? 8 : 4;
  return g.p_row % pc == 0 && g.q_row % pc == 0;
}

// The tiles that a product is made by.
// Wide tiles from two rounds of the device on, bf16 along in whole pieces only.  1024 to
// 1024, in us, large tiles first: 20480 rows 60, 68; 24576 rows 63, 70; 65536
// rows 146, 144; 131072 rows with a residual 380, 347.  Across, the
// transposing reads' addresses do not fit beside the tile: dx and dweight
// of 60000 rows 302, wide 350.
// Rows on their way through registers leave few to large tiles of operands
// across, and neither is always faster (fp32, the gradient in us, large tiles
// first: 5387 rows, 641 to 1165 254, 222; 4100 rows, 1023 to 1025 302, 294; 20000
// rows, 643 to 1160 715, 765; 30001 rows, 255 to 257 120, 144): small ones are
// taken.  Along, 20000 rows, 643 to 1160: 237, by small tiles 330.
enum Tiles { kSmallTiles, kLargeTiles, kWideTiles };
Tiles tiles_by(const Gemm& g, int io, bool big, bool p_along, bool q_along) {
  const bool whole = whole_pieces(g, io);
  if (io == TM_IO_BF16 && whole && p_along && q_along &&
      (g.R + kWide - 1) / kWide * ((g.C + kWide - 1) / kWide) >= 2 * kWideBlocks)
    return kWideTiles;
  return big && (whole || p_along) ? kLargeTiles : kSmallTiles;
}

template <typename S>
bool fits(const Gemm& g) {   // fewer than 2^32 threads, tiles in eights
  const int64_t all = (g.R + S::TR - 1) / S::TR * ((g.C + S::TC - 1) / S::TC) * g.parts;
  return (all + 7) / 8 * 8 < ((int64_t)1 << 32) / S::kThreads;
}
// whether one launch can hold them
bool one_launch(const Gemm& g, int io, bool big, bool p_along, bool q_along) {
  const Tiles by = tiles_by(g, io, big, p_along, q_along);
  if (by == kWideTiles)   // (always 256 workgroups: counted in 32 bits)
    return (g.R + kWide - 1) / kWide * ((g.C + kWide - 1) / kWide) < ((int64_t)1 << 31);
  if (io == TM_IO_BF16) return by == kLargeTiles ? fits<Large<true>>(g) : fits<Small<true>>(g);
  return by == kLargeTiles ? fits<Large<false>>(g) : fits<Small<false>>(g);
}

template <bool P_ALONG, bool Q_ALONG, bool F32_OUT>
hipError_t launch_gemm(const Gemm& g, int io, bool big, hipStream_t stream) {
  const Tiles by = tiles_by(g, io, big, P_ALONG, Q_ALONG);
  const bool large = by == kLargeTiles;
  if constexpr (P_ALONG && Q_ALONG)
    if (by == kWideTiles) return launch_wide(g, stream);
  if (whole_pieces(g, io))
    return io == TM_IO_BF16 ? launch_sized<P_ALONG, Q_ALONG, F32_OUT, true, kPieces>(g, large, stream)
                            : launch_sized<P_ALONG, Q_ALONG, F32_OUT, false, kPieces>(g, large, stream);
  if constexpr (P_ALONG)
    return io == TM_IO_BF16 ? launch_sized<P_ALONG, Q_ALONG, F32_OUT, true, kOdd>(g, large, stream)
                            : launch_sized<P_ALONG, Q_ALONG, F32_OUT, false, kOdd>(g, large, stream);
  else
    return io == TM_IO_BF16 ? launch_tiles<Small<true>, P_ALONG, Q_ALONG, kOdd, F32_OUT>(g, stream)
                            : launch_tiles<Small<false>, P_ALONG, Q_ALONG, kOdd, F32_OUT>(g, stream);
}

template <bool BF16, bool VEC>
hipError_t launch_narrow(const Gemm& g, hipStream_t stream) {
  const unsigned grid = (unsigned)(((int64_t)g.C + 15) / 16);
  if (g.R <= 16)
    narrow_kernel<BF16, 1, VEC><<<grid, 512, 0, stream>>>(g);
  else if (g.R <= 32)
    narrow_kernel<BF16, 2, VEC><<<grid, 512, 0, stream>>>(g);
  else
    narrow_kernel<BF16, 4, VEC><<<grid, 512, 0, stream>>>(g);
  return hipGetLastError();
}

// The weight's gradient: parts of the rows that together fill the device, a
// part with 128 rows at least; large tiles where there are enough of them.
// With two planes of dz half of the parts belong to each.  Small fp32 tiles
// have a CU each: a part more than fits at once costs a round of the device
// (1001 rows, 500 to 777, 104 tiles: 2 parts 41 us for the whole gradient, 5 parts 54).
int weight_parts(const ProjectionShape& s, bool* big) {
  const int pc = s.io == TM_IO_BF16 ? 8 : 4;
  const int planes = s.silu && s.io == TM_IO_BF16 ? 2 : 1;
  int64_t parts = 1;
  for (int pass = s.O % pc || s.K % pc; pass < 2; ++pass) {   // (odd rows: small tiles only)
    *big = pass == 0;
    const int64_t tr = *big ? (s.io == TM_IO_BF16 ? 256 : 128) : 64, tc = *big ? 128 : 64;
    const int64_t tiles = (s.O + tr - 1) / tr * ((s.K + tc - 1) / tc), most = s.M / 128 > 1 ? s.M / 128 : 1;
    parts = *big || s.io == TM_IO_BF16 ? (512 / planes + tiles - 1) / tiles : tiles < 256 ? 256 / tiles : 1;
    if (parts > most) parts = most;
    if (parts > 64) parts = 64;
    if (tiles * parts * planes >= 192) break;
  }
  return (int)parts * planes;
}

int slope_parts(const ProjectionShape& s) {
  const int64_t pc = s.io == TM_IO_BF16 ? (s.O % 8 ? 1 : 8) : s.O % 4 ? 1 : 4;
  const int64_t cols = (s.O + 64 * pc - 1) / (64 * pc);
  int64_t parts = (1024 + cols - 1) / cols, most = (s.M + 15) / 16;
  if (parts > most) parts = most;
  return parts < 1 ? 1 : parts > 1024 ? 1024 : (int)parts;
}

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }
int64_t round_t(int64_t x) { return (x + 63) / 64 * 64; }   // (slices of either length)

}  // namespace

namespace {

// The three products, without their pointers.
Gemm forward_product(const ProjectionShape& s) {
  Gemm g = {};
  g.p_row = g.q_row = s.K, g.R = s.M, g.C = s.O, g.T = s.K, g.per = round_t(s.K), g.parts = 1;
  return g;
}
Gemm dx_product(const ProjectionShape& s) {
  Gemm g = {};
  g.p_row = s.K, g.q_row = s.O, g.R = s.M, g.C = s.K, g.T = s.O, g.per = round_t(s.O), g.parts = 1;
  return g;
}
Gemm dweight_product(const ProjectionShape& s, int parts) {
  Gemm g = {};
  const int64_t each = s.silu && s.io == TM_IO_BF16 ? parts / 2 : parts;
  g.p_row = s.K, g.q_row = s.O, g.R = s.O, g.C = s.K, g.T = s.M, g.per = round_t((s.M + each - 1) / each), g.parts = parts;
  return g;
}

}  // namespace

bool projection_supported(const ProjectionShape& s, bool backward) {
  if (s.K > 1 << 22 || s.O > 1 << 22) return false;   // (Loads' distances)
  if (!backward)   // (few rows: a workgroup for 16 columns)
    return s.M <= kNarrowRows || one_launch(forward_product(s), s.io, large(s.M, s.O, s.io), true, true);
  bool big;
  const int parts = weight_parts(s, &big);
  return one_launch(dx_product(s), s.io, large(s.M, s.K, s.io), false, true) &&
         one_launch(dweight_product(s, parts), s.io, big, false, false) &&
         (int64_t)s.O * s.K / 1024 < kMostBlocks;   // (the parts' sums)
}

hipError_t launch_projection(const ProjectionShape& s, const void* x, const void* weight, const float* bias,
                             const void* residual, void* out, void* pre, hipStream_t stream) {
  if (s.M == 0) return hipSuccess;
  Gemm g = forward_product(s);
  g.P = weight, g.Q = x, g.bias = bias, g.residual = residual, g.out = out, g.pre = pre, g.silu = s.silu;
  if (s.M <= kNarrowRows) {
    const bool vec = s.K % (s.io == TM_IO_BF16 ? 8 : 4) == 0;
    if (s.io == TM_IO_BF16) return vec ? launch_narrow<true, true>(g, stream) : launch_narrow<true, false>(g, stream);
    return vec ? launch_narrow<false, true>(g, stream) : launch_narrow<false, false>(g, stream);
  }
  return launch_gemm<true, true, false>(g, s.io, large(s.M, s.O, s.io), stream);
}

// dz (where there is an activation) and what a bf16 one was rounded by, the weight's parts, the bias's sums
int64_t projection_backward_ws_bytes(const ProjectionShape& s) {
  bool big;
  const int parts = weight_parts(s, &big);
  return (s.silu ? (s.io == TM_IO_BF16 ? 2 * round16(s.M * s.O * 2) : round16(s.M * s.O * 4)) : 0) +
         (parts > 1 ? round16((int64_t)parts * s.O * s.K * 4) : 0) + round16((int64_t)slope_parts(s) * s.O * 4);
}

hipError_t launch_projection_backward(const ProjectionShape& s, const void* x, const void* weight, const void* pre,
                                      const void* dout, void* dx, float* dweight, float* dbias, void* ws,
                                      hipStream_t stream) {
  const int64_t esz = s.io == TM_IO_BF16 ? 2 : 4;
  bool big;
  const int parts = weight_parts(s, &big), sparts = slope_parts(s);
  char* at = (char*)ws;
  void *dz = nullptr, *dz2 = nullptr;
  if (s.silu) {
    dz = at, at += round16(s.M * s.O * esz);
    if (s.io == TM_IO_BF16) dz2 = at, at += round16(s.M * s.O * esz);
  }
  float* wparts = parts > 1 ? (float*)at : nullptr;
  if (wparts) at += round16((int64_t)parts * s.O * s.K * 4);
  float* bparts = (float*)at;
  const bool whole = s.O % (16 / esz) == 0;
  const int pc = whole ? (int)(16 / esz) : 1;
  const dim3 grid((s.O + 64 * pc - 1) / (64 * pc), sparts);
  const int64_t per = (s.M + sparts - 1) / sparts;
  auto slope = s.io == TM_IO_BF16 ? (whole ? slope_kernel<true, true> : slope_kernel<true, false>)
                                  : (whole ? slope_kernel<false, true> : slope_kernel<false, false>);
  slope<<<grid, 256, 0, stream>>>(dout, s.silu ? pre : nullptr, dz, dz2, sparts > 1 ? bparts : dbias, s.M, s.O, per);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const void* z = s.silu ? dz : dout;
  Gemm g;
  if (s.M > 0) {
    g = dx_product(s);
    g.P = weight, g.Q = z, g.out = dx;
    err = launch_gemm<false, true, false>(g, s.io, large(s.M, s.K, s.io), stream);
    if (err != hipSuccess) return err;
  }
  g = dweight_product(s, parts);
  g.P = x, g.Q = z, g.out = parts > 1 ? wparts : dweight;
  if (s.silu && s.io == TM_IO_BF16) g.Q2 = dz2;
  err = launch_gemm<false, false, true>(g, s.io, big, stream);
  if (err != hipSuccess || (parts == 1 && sparts == 1)) return err;
  const int64_t n = (int64_t)s.O * s.K;
  const unsigned blocks = parts > 1 ? (unsigned)((n + 1023) / 1024) : 0;
  parts_kernel<<<blocks + (sparts > 1 ? (unsigned)((s.O + 15) / 16) : 0), 256, 0, stream>>>(
      wparts, parts, n, dweight, bparts, sparts, s.O, dbias, blocks);
  return hipGetLastError();
}

}  // namespace titans
