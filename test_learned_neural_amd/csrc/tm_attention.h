// What the attention kernels share: the call's parameters, how a workgroup
// finds its rows, tiles in LDS and the operands that the matrix cores take
// from them.
//
// Matrix products are 32x32 tiles with a contraction in steps of 16, bf16 in
// one instruction (v_mfma_f32_32x32x16_bf16) and fp32 in six of them (Planes).
// Either way a lane holds 8 elements of its row (or
// column) lane % 32 a step, the lower half of the wave the first 8 of a step's
// 16 and the upper half the others; any order will do that both operands keep.
// An accumulator has its column in lane % 32 and its rows 8 (r / 4) + 4 (lane /
// 32) + r % 4 in registers r = 0..15.  So a tile of scores, keys in rows and
// queries in columns, is by itself the second operand of the product over the
// keys: registers 8 s .. 8 s + 7 are step s, whose keys are 16 s + 4 (lane /
// 32) + {0..3, 8..11}, and no lane hands anything to another.
#pragma once

#include <limits.h>

#include <type_traits>

#include "tm_internal.h"

namespace titans {
namespace att {

typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) __bf16 bf16x4;
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) float f32x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) float f32x8;
typedef __attribute__((ext_vector_type(16))) float f32x16;
typedef __attribute__((address_space(3))) void* lds_void_ptr;
typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
typedef __attribute__((ext_vector_type(2))) unsigned u32x2;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLowest = -1e30f;   // a running maximum before its first score

struct Params {
  const void *q, *k, *v, *dout;
  void *out, *dq, *dk, *dv;
  float *parts_k, *parts_v;   // the gradient's parts of dk and dv, where there are several
  int64_t part_size;
  int parts, ahead;
  float *lse, *stats;       // stats: the gradient's two fp32 values a query and head, stat_rows apart
  int64_t stat_rows;
  const int32_t *offsets, *lengths;
  // elements from one sequence, head and token to the next (offsets: one row of N tokens, no sequence stride)
  int64_t q_seq, q_head, q_tok, k_seq, k_head, k_tok, o_seq, o_tok;
  int B, H, Hk, N, d, window, prefix;
  float scale;
  int streams, units;   // key heads by sequences (offsets: key heads), tiles of each
};

// How rows lie in memory: as whole 16-byte pieces that fill the padded width
// DP, as whole pieces, or as anything.
constexpr int kOdd = 0, kPieces = 1, kFull = 2;

// An fp32 factor as three bf16 numbers that add up to it: the first cut off (so
// that the largest numbers stay finite), the second rounded to nearest, the
// third exact.  Six of the nine products are kept: m l, l m and l l are left
// out, at most 2^-22 of a product together, of either sign, as the third number
// has either, so that a long sum does not drift (0.36 2^-24 on the average;
// with the second cut off too, 2^-21 and always towards zero).  Six bf16
// instructions take 192 cycles for a step where the fp32 ones take 512.  An
// infinity becomes NaN on the way.  (bf16 numbers end at 2^-133, and so do the
// planes of factors below 2^-110.)
// The first rounded as well would keep 2^-24, and has to be held below the
// largest bf16 number: 6 to 15% of the fp32 kernels' time (4096 tokens, 16
// heads, d 128: 530 us, 574; 1001 rows, 500 to 777: 14.7, 15.6).
struct Planes {
  bf16x8 h, m, l;
};

template <bool BF16>
struct Types;
template <>
struct Types<true> {
  typedef __bf16 elem;
  typedef bf16x8 frag;   // 8 elements
  typedef bf16x8 op;     // the same as a factor
};
template <>
struct Types<false> {
  typedef float elem;
  typedef f32x8 frag;
  typedef Planes op;
};

__device__ __forceinline__ bf16x8 factor(bf16x8 f) { return f; }
__device__ __forceinline__ Planes factor(f32x8 f) {
  typedef __attribute__((ext_vector_type(4))) unsigned u32x4;
  u32x4 a, b, c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // (floats of their own: a bit cast of a vector's element would take its first one)
    const float y0 = f[2 * i], y1 = f[2 * i + 1];
    const unsigned u0 = __builtin_bit_cast(unsigned, y0), u1 = __builtin_bit_cast(unsigned, y1);
    const f32x2 r = {y0 - __builtin_bit_cast(float, u0 & 0xffff0000u), y1 - __builtin_bit_cast(float, u1 & 0xffff0000u)};
    const unsigned m = __builtin_bit_cast(unsigned, __builtin_convertvector(r, bf16x2));
    const float z0 = r[0] - __builtin_bit_cast(float, m << 16), z1 = r[1] - __builtin_bit_cast(float, m & 0xffff0000u);
    a[i] = __builtin_amdgcn_perm(u1, u0, 0x07060302u);   // the upper halves of both
    b[i] = m;
    c[i] = __builtin_amdgcn_perm(__builtin_bit_cast(unsigned, z1), __builtin_bit_cast(unsigned, z0), 0x07060302u);
  }
  return {__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, c)};
}

// f(x, y) for the products that a b is made of, the small ones first
template <typename F>
__device__ __forceinline__ void products(const bf16x8& a, const bf16x8& b, F f) {
  f(a, b);
}
template <typename F>
__device__ __forceinline__ void products(const Planes& a, const Planes& b, F f) {
  f(a.l, b.h), f(a.h, b.l), f(a.m, b.m), f(a.m, b.h), f(a.h, b.m), f(a.h, b.h);
}
template <typename Op>
__device__ __forceinline__ void mma(f32x16& acc, const Op& a, const Op& b) {
  products(a, b, [&](bf16x8 x, bf16x8 y) { acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x, y, acc, 0, 0, 0); });
}

// registers 8 s .. 8 s + 7 of an accumulator as a factor, rounded to bf16 for
// bf16 tensors: a weight keeps 8 bits, as the values that it multiplies
template <typename Op>
__device__ __forceinline__ Op operand(const f32x16& x, int s) {
  f32x8 t;
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = x[8 * s + j];
  if constexpr (sizeof(Op) == sizeof(bf16x8))
    return __builtin_convertvector(t, bf16x8);
  else
    return factor(t);
}

// what operand() has rounded them by, rounded itself: with it a weight keeps 16 bits
__device__ __forceinline__ bf16x8 remainder(const f32x16& x, int s, const bf16x8& rounded) {
  f32x8 t;
#pragma unroll
  for (int j = 0; j < 8; ++j) t[j] = x[8 * s + j] - (float)rounded[j];
  return __builtin_convertvector(t, bf16x8);
}

// the other half wave's value
__device__ __forceinline__ float other_half(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const u32x2 r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __builtin_bit_cast(float, (threadIdx.x & 32) ? r[0] : r[1]);
}

// LDS has 64 banks of 4 bytes.  Reads of 16 bytes a lane go 16 lanes at a time,
// transposing ones of 8 bytes 32 lanes at a time: 16 rows of one chunk, or 4
// rows of 4 neighbouring chunks, have to fall on 16 different places of 16
// bytes in 256.  Rows of NC chunks fill those 256 bytes by 16 / NC; chunk c of
// row r lies at c ^ swizzle(r).
template <int NC>
__device__ __forceinline__ int swizzle(int r) {
  if (NC == 4) return (r >> 2) & 3;
  if (NC == 8) return ((r >> 1) & 1) << 2 | ((r >> 2) & 3);
  return (r & 3) << 2 | ((r >> 2) & 3);
}

// A tile's rows in LDS: LS elements each (the padded width up to the next
// power of two), 16-byte chunk c of row r at c ^ swz(r).
template <bool BF16, int DP>
struct Tile {
  typedef typename Types<BF16>::elem elem;
  typedef typename Types<BF16>::frag frag;
  typedef typename Types<BF16>::op op;
  static constexpr int kSize = BF16 ? 2 : 4;
  static constexpr int LS = DP == 96 ? 128 : DP;
  static constexpr int RB = LS * kSize;       // bytes of a row
  static constexpr int NC = RB / 16;          // its chunks
  static constexpr int PC = 16 / kSize;       // elements of a chunk

  static __device__ __forceinline__ int swz(int r) {
    return swizzle<NC>(r);
  }

  // step s of row r, contraction along the row
  static __device__ __forceinline__ op along(const unsigned char* t, int r, int s, int half) {
    if constexpr (BF16) {
      return *(const frag*)(t + r * RB + ((2 * s + half) ^ swz(r)) * 16);
    } else {
      const f32x4 a = *(const f32x4*)(t + r * RB + ((4 * s + 2 * half) ^ swz(r)) * 16);
      const f32x4 b = *(const f32x4*)(t + r * RB + ((4 * s + 2 * half + 1) ^ swz(r)) * 16);
      return factor(__builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
    }
  }

  // step s of column c0 + lane % 32, contraction over rows r0 + 16 s + .. in an accumulator's order
  static __device__ __forceinline__ op across(const unsigned char* t, int r0, int s, int c0, int lane) {
    const int half = lane >> 5;
    if constexpr (BF16) {
      const int l = lane & 15, col = c0 + (lane & 16) + 4 * (l & 3);
      const int r = r0 + 16 * s + 4 * half + (l >> 2);
      const unsigned char* p0 = t + r * RB + ((col / 8) ^ swz(r)) * 16 + (l & 1) * 8;
      const unsigned char* p1 = t + (r + 8) * RB + ((col / 8) ^ swz(r + 8)) * 16 + (l & 1) * 8;
      const bf16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)p0);
      const bf16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)p1);
      return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
    } else {
      frag f;
      const int col = c0 + (lane & 31);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int r = r0 + 16 * s + 4 * half + (j & 3) + 8 * (j >> 2);
        f[j] = *(const float*)(t + r * RB + ((col / 4) ^ swz(r)) * 16 + (col & 3) * 4);
      }
      return factor(f);
    }
  }

  // The elements from c on of a row of d, a chunk of them, from any address, zero
  // behind the row's end: 16 bytes that end with the row where the chunk
  // passes it, shifted into place.
  typedef __attribute__((ext_vector_type(PC))) elem piece;
  static __device__ __forceinline__ piece odd(const elem* row, int c, int d) {
    piece x = {};
    if (d >= PC) {
      const int from = min(c, d - PC), by = c - from;
      __builtin_memcpy(&x, row + from, 16);
      if (by) {
#pragma unroll
        for (int n = 1; n < PC; n *= 2)
#pragma unroll
          for (int e = 0; e + n < PC; ++e) x[e] = by & n ? x[e + n] : x[e];
#pragma unroll
        for (int e = 0; e < PC; ++e) x[e] = c + e < d ? x[e] : (elem)0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < PC; ++e)
        if (c + e < d) x[e] = row[c + e];
    }
    return x;
  }

  // Rows j0 .. j0 + ROWS - 1 of a tensor (rows `tok` elements apart, rows past
  // `last` as row `last`) into LDS by THREADS threads: wide pieces straight to
  // LDS, or through registers where rows are not made of 16-byte pieces.
  // Columns from d on are zero: cleared once (clear()) where pieces go straight
  // to LDS, which then leaves them alone.  A thread's places within a tile are
  // the same in every whole tile, so it keeps their distances from the tile's
  // first row (32 bits: 64 rows of 2^22 elements), which is the wave's.
  template <int ROWS, int THREADS, int VEC>
  struct Loads {
    static constexpr int kCount = ROWS * NC / THREADS;
    uint32_t off[kCount];

    __device__ __forceinline__ Loads(int64_t tok, int tid) {
      static_assert(ROWS * NC % THREADS == 0, "");
#pragma unroll
      for (int i = 0; i < kCount; ++i) {
        const int at = i * THREADS + tid, r = at / NC, c = (at % NC) ^ swz(r);
        off[i] = (uint32_t)(r * (int)tok + c * PC) * kSize;
      }
    }

    __device__ __forceinline__ void operator()(unsigned char* t, const elem* src, int64_t tok, int j0, int last, int d,
                                               int tid) const {
      const elem* row0 = src + (int64_t)j0 * tok;
      const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
      for (int i = 0; i < kCount; ++i) {
        const int base = i * THREADS + wave * 64, at = i * THREADS + tid;
        const int r = at / NC, c = (at % NC) ^ swz(r);
        if constexpr (VEC != kOdd) {
          uint32_t o = off[i];
          if (j0 + ROWS - 1 > last) o = (uint32_t)(min(r, last - j0) * (int)tok + c * PC) * kSize;
          if (VEC == kFull && DP == LS ? true : c * PC < d)
            __builtin_amdgcn_global_load_lds((const void*)((const char*)row0 + o), (lds_void_ptr)(t + base * 16), 16, 0, 0);
        } else {
          *(piece*)(t + at * 16) = odd(row0 + (int64_t)min(r, last - j0) * tok, c * PC, d);
        }
      }
    }
  };

  // row j (clamped) of a tensor as an operand's DP / 16 steps, straight from memory
  template <int VEC>
  static __device__ __forceinline__ void row(frag (&f)[DP / 16], const elem* src, int d, int half) {
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
      const int c = 16 * s + 8 * half;
      if (VEC != kOdd) {
        frag z = {};
        if constexpr (BF16) {
          if (VEC == kFull || c < d) z = *(const frag*)(src + c);
        } else {
          f32x4 a = {}, b = {};
          if (VEC == kFull || c < d) a = *(const f32x4*)(src + c);
          if (VEC == kFull || c + 4 < d) b = *(const f32x4*)(src + c + 4);
          z = __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        f[s] = z;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[s][e] = c + e < d ? src[c + e] : (elem)0.f;
      }
    }
  }

  // an accumulator's four rows 8 g + 4 half + 0..3 (columns c.. of a row in memory)
  template <int VEC>
  static __device__ __forceinline__ void store4(elem* dst, int c, int d, const f32x4 x) {
    if (VEC != kOdd) {
      if (VEC != kFull && c >= d) return;
      if constexpr (BF16)
        *(bf16x4*)(dst + c) = __builtin_convertvector(x, bf16x4);
      else
        *(f32x4*)(dst + c) = x;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < d) dst[c + e] = (elem)x[e];
    }
  }
};

// A barrier behind which every wave's LDS writes are there, the loads straight
// to LDS among them: a plain barrier does not wait for those.
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// The same for what this wave alone reads.  (vmcnt and lgkmcnt zero; as a
// builtin, so that the compiler knows too that its own loads have come.)
__device__ __forceinline__ void landed_in_wave() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ void clear(unsigned char* t, int bytes, int tid, int threads) {
  for (int i = tid * 16; i < bytes; i += threads * 16) *(f32x4*)(t + i) = f32x4{0.f, 0.f, 0.f, 0.f};
}

// The tile of rows that unit `unit` of stream `stream` stands for.
struct Place {
  int seq, head0, key_head;   // the sequence's row of the tensors, first query head, key head
  int t0, n, tile;            // its first token, its tokens, the tile
};

// Sequences packed one behind the other: sequence s has the units from
// offsets[s] / ROWS + s on, as many as it needs at least, so that a unit's
// sequence is found by comparing the starts that the lanes hold.  The rest
// are empty.  Offsets are clamped to what memory holds.
template <int ROWS>
__device__ __forceinline__ bool find(const Params& p, int stream, int unit, Place& at) {
  const int G = p.H / p.Hk;
  if (p.offsets) {
    at.key_head = stream;
    at.seq = 0;
    int lo = 0, hi = p.B;    // the last sequence in [lo, hi) that starts at or before the unit
    const int lane = threadIdx.x & 63;
    while (hi - lo > 1) {
      const int step = (hi - lo + 63) / 64, s = lo + lane * step;
      bool before = false;
      if (s < hi) {
        const int o = min(max(p.offsets[s], 0), p.N);
        before = o / ROWS + s <= unit;
      }
      const int c = max(__popcll(__ballot(before)), 1);
      lo += (c - 1) * step;
      hi = min(hi, lo + step);
    }
    const int a = min(max(p.offsets[lo], 0), p.N);
    at.t0 = __builtin_amdgcn_readfirstlane(a);
    at.n = __builtin_amdgcn_readfirstlane(min(max(p.offsets[lo + 1], a), p.N)) - at.t0;
    unit -= at.t0 / ROWS + __builtin_amdgcn_readfirstlane(lo);
  } else {
    at.key_head = stream % p.Hk;
    at.seq = stream / p.Hk;
    at.t0 = 0;
    at.n = p.N;
    if (p.lengths) at.n = __builtin_amdgcn_readfirstlane(min(max(p.lengths[at.seq], 0), p.N));
  }
  at.head0 = at.key_head * G;
  const int tiles = (at.n + ROWS - 1) / ROWS;
  at.tile = unit;
  return unit >= 0 && unit < tiles;
}

// Block -> (stream, unit, head of the group).  Blocks go round the 8 XCDs.
// With streams in eights every XCD takes whole streams, one after the other,
// so that their keys stay in its L2; otherwise units go round the XCDs.  The
// heads that share keys are neighbours on one XCD in both.  The first `ahead`
// units of every stream (much longer ones) come before all others.
__device__ __forceinline__ bool place_of(const Params& p, int heads, int& stream, int& unit, int& head) {
  const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
  head = slot % heads;
  const int u = slot / heads;
  if (p.streams % 8 == 0) {
    const int each = p.streams / 8, v = u - each * p.ahead;
    if (v < 0) {
      stream = xcd + 8 * (u % each);
      unit = u / each;
    } else {
      stream = xcd + 8 * (v / (p.units - p.ahead));
      unit = p.ahead + v % (p.units - p.ahead);
    }
    return true;
  }
  const int64_t v = (int64_t)u * 8 + xcd;
  stream = (int)(v % p.streams);
  unit = (int)(v / p.streams);
  return unit < p.units;
}

// Scores that the mask takes away, registers of one 32 x 32 tile: keys in rows
// and queries in columns, or the other way round.  row0: the row of register 0
// in this lane; col: the lane's column; some keys are below the prefix or none.
// Behind the prefix j <= i and i - j < window are one unsigned comparison.
template <bool KEYS_IN_ROWS>
__device__ __forceinline__ void mask_tile(f32x16& x, int row0, int col, int window, int prefix, bool some_below) {
  const int far = KEYS_IN_ROWS ? col - row0 : row0 - col;
  if (!some_below) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int c = 8 * (r >> 2) + (r & 3);
      x[r] = (unsigned)(KEYS_IN_ROWS ? far - c : far + c) < (unsigned)window ? x[r] : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int c = 8 * (r >> 2) + (r & 3), apart = KEYS_IN_ROWS ? far - c : far + c, j = KEYS_IN_ROWS ? row0 + c : col;
      const int reach = j < prefix ? INT_MAX : window;
      x[r] = (unsigned)apart < (unsigned)reach ? x[r] : -__builtin_inff();
    }
  }
}

// DP and the rows' kind for a width, f(integral constants BF16, DP, VEC)
template <bool BF16, int DP, typename F>
hipError_t by_rows(int d, F f) {
  typedef std::integral_constant<bool, BF16> B;
  typedef std::integral_constant<int, DP> W;
  if constexpr (DP != 96)
    if (d == DP) return f(B(), W(), std::integral_constant<int, kFull>());
  return d % (BF16 ? 8 : 4) == 0 ? f(B(), W(), std::integral_constant<int, kPieces>())
                                 : f(B(), W(), std::integral_constant<int, kOdd>());
}
template <bool BF16, typename F>
hipError_t by_width(int d, F f) {
  return d <= 32   ? by_rows<BF16, 32>(d, f)
         : d <= 64 ? by_rows<BF16, 64>(d, f)
         : d <= 96 ? by_rows<BF16, 96>(d, f)
                   : by_rows<BF16, 128>(d, f);
}
template <typename F>
hipError_t by_type(int io, int d, F f) {
  return io == TM_IO_BF16 ? by_width<true>(d, f) : by_width<false>(d, f);
}

}  // namespace att

att::Params attention_params(const AttentionShape& s);
int64_t attention_units(const AttentionShape& s, int rows);
int64_t attention_blocks(const AttentionShape& s, int rows, int heads);

}  // namespace titans
