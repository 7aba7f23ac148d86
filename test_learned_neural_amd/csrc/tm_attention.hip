// Causal attention over whole prompts: the short-term memory beside the
// neural one ("Titans: Learning to Memorize at Test Time", mer.dev notes,
// section 2.1 for the formula, 4.2 and 4.3 for the sliding window with
// persistent tokens before it).  Token i of a sequence sees token j where
// j <= i and (window == 0 or i - j < window or j < prefix):
//
//   x_ij = scale q_i . k_j,  lse_i = log sum_j exp(x_ij)
//   out_i = sum_j exp(x_ij - lse_i) v_j
//
// One pass over the keys with a running maximum m and sum l: the scores of a
// tile are exp2(x log2 e - m), and where a tile's maximum passes m by more
// than kSlack, l and the output so far are scaled to the new one.  Until then
// weights may reach 2^kSlack, which costs nothing in floating point.
//
// A workgroup has kWaves x 32 queries of one head, each wave 32 of them in the
// lanes: scores are formed transposed (keys in rows), so a query's maximum and
// sum are taken along a lane's registers and one exchange between the halves,
// and the scores' registers are an operand of the second product as they lie.
// Keys and values go through LDS in tiles, loaded straight to it one tile
// ahead.
//
// Weights are rounded to bf16 before they meet v for bf16 tensors, which puts out
// 2.0e-3 off where its own rounding is 1.6e-3.  As two bf16 numbers (what the
// step's kernel does, where memory is waited for) they would take a third more: the
// two cases below 1061 us instead of 804, and 2338 instead of 1720.
//
// Measured: 8 x 16 sequences of 16384, d 64, bf16, a window of 1024: 777 us, 697
// TFLOP/s of scores seen (a product of 8192^3 by the library: 1137).  Its
// exponentials, maxima, sums and roundings bound it: 5 vector instructions a
// score are as long as its two products.  32768 packed tokens in 12 sequences, 16
// query heads, 4 key heads, d 128: 1745 us, 1004 TFLOP/s, matrix cores 52% busy
// at the clock that they leave.  LDS is read without bank conflicts.  fp32, 2 x 8
// sequences of 4096, d 128: 550 us, 125 TFLOP/s with a wave a SIMD, whose registers
// hold all planes; two waves of half the registers spill and took 1.9 times as
// long.  d 64: 365 us, 94 TFLOP/s.
#include "tm_attention.h"

namespace titans {
namespace {

using namespace att;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;     // queries of a workgroup
constexpr float kSlack = 8.f;          // in powers of two

template <bool BF16>
constexpr int keys_of() { return BF16 ? 64 : 32; }

template <bool BF16, int DP, int VEC>
__global__ void __launch_bounds__(kThreads, BF16 && DP <= 64 ? 3 : BF16 || DP <= 96 ? 2 : 1) attention_kernel(Params p) {
  typedef Tile<BF16, DP> T;
  typedef typename T::elem elem;
  typedef typename T::op op;
  constexpr int KT = keys_of<BF16>(), kBytes = KT * T::RB;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];   // [2][K, V]
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int stream, unit, head;
  if (!place_of(p, p.H / p.Hk, stream, unit, head)) return;
  Place at;
  if (!find<kRows>(p, stream, unit, at)) return;
  const int tile = (at.n + kRows - 1) / kRows - 1 - at.tile;   // the longest first
  const int h = at.head0 + head;
  const int i0 = tile * kRows, w0 = i0 + 32 * wave, qi = w0 + (lane & 31), last = at.n - 1;
  const elem* qp = (const elem*)p.q + at.seq * p.q_seq + h * p.q_head + (int64_t)(at.t0 + min(qi, last)) * p.q_tok;
  const elem* kp = (const elem*)p.k + at.seq * p.k_seq + at.key_head * p.k_head + (int64_t)at.t0 * p.k_tok;
  const elem* vp = (const elem*)p.v + at.seq * p.k_seq + at.key_head * p.k_head + (int64_t)at.t0 * p.k_tok;

  // tiles of keys: those of the prefix, then those in reach of the first query
  const int top = min(i0 + kRows - 1, last) / KT;
  const int lo = p.window ? max(0, i0 - p.window + 1) / KT : 0;
  const int pre = min((p.prefix + KT - 1) / KT, lo);
  int t = pre > 0 ? 0 : lo;
  // (of the prefix's tiles only the persistent tokens are read: a NaN behind them is not met by a weight of 0)
  auto end_of = [&](int t) __attribute__((always_inline)) { return t < pre ? min(last, p.prefix - 1) : last; };

  if (VEC == kPieces && p.d < DP) {
    clear(smem, 4 * kBytes, tid, kThreads);
    __syncthreads();
  }
  const typename T::template Loads<KT, kThreads, VEC> load(p.k_tok, tid);
  load(smem, kp, p.k_tok, t * KT, end_of(t), p.d, tid);
  load(smem + kBytes, vp, p.k_tok, t * KT, end_of(t), p.d, tid);
  op q[DP / 16];
  {
    typename T::frag f[DP / 16];
    T::template row<VEC>(f, qp, p.d, half);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) q[s] = factor(f[s]);
  }

  const int window = p.window ? p.window : INT_MAX;
  const float c = p.scale * kLog2e;
  float m = kLowest, l = 0.f;
  f32x16 o[DP / 32] = {};
  // The tile in kb, while tile t goes to nb.  That the two are apart is said to
  // the compiler (restrict): its transposing reads would wait for the loads
  // under way otherwise.
  auto step = [&](const unsigned char* __restrict__ kb, unsigned char* __restrict__ nb, int t, int k0) __attribute__((always_inline)) {
    const unsigned char* vb = kb + kBytes;
    if (t <= top) {
      load(nb, kp, p.k_tok, t * KT, end_of(t), p.d, tid);
      load(nb + kBytes, vp, p.k_tok, t * KT, end_of(t), p.d, tid);
    }
    // nothing of the tile is seen by this wave's queries
    if (w0 > last || k0 > w0 + 31 || (p.window && w0 - (k0 + KT - 1) >= p.window && k0 >= p.prefix)) return;
    f32x16 x[KT / 32] = {};
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s)
#pragma unroll
      for (int g = 0; g < KT / 32; ++g) mma(x[g], T::along(kb, 32 * g + (lane & 31), s, half), q[s]);
    __builtin_amdgcn_s_setprio(0);
    if (k0 + KT - 1 > w0 || (p.window && w0 + 31 - k0 >= p.window)) {
#pragma unroll
      for (int g = 0; g < KT / 32; ++g) mask_tile<true>(x[g], k0 + 32 * g + 4 * half, qi, window, p.prefix, k0 < p.prefix);
    }
    float mx = x[0][0];
#pragma unroll
    for (int g = 0; g < KT / 32; ++g)
#pragma unroll
      for (int r = 0; r < 16; ++r) mx = fmaxf(mx, x[g][r]);
    mx = fmaxf(mx, other_half(mx)) * c;
    if (__any(mx > m + kSlack)) {
      const float to = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= f;
#pragma unroll
      for (int e = 0; e < DP / 32; ++e)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[e][r] *= f;
    }
    float sum = 0.f;
#pragma unroll
    for (int g = 0; g < KT / 32; ++g)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        x[g][r] = __builtin_amdgcn_exp2f(fmaf(x[g][r], c, -m));
        sum += x[g][r];
      }
    l += sum;
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int s = 0; s < KT / 16; ++s) {
      const op w = operand<op>(x[s / 2], s % 2);
#pragma unroll
      for (int e = 0; e < DP / 32; ++e) mma(o[e], T::across(vb, 0, s, 32 * e, lane), w);
    }
    __builtin_amdgcn_s_setprio(0);
    };
  auto turn = [&](int buf) __attribute__((always_inline)) {
    const int k0 = t * KT;
    t = t + 1 == pre ? lo : t + 1;
    landed();   // this tile is there, and nobody reads the other any more
    step(smem + buf * 2 * kBytes, smem + (buf ^ 1) * 2 * kBytes, t, k0);
  };
  while (t <= top) {   // (both buffers in turn, their places in LDS constant)
    turn(0);
    if (t <= top) turn(1);
  }
  if (qi > last) return;
  l += other_half(l);
  const float inv = 1.f / l;
  elem* to = (elem*)p.out + at.seq * p.o_seq + (int64_t)(at.t0 + qi) * p.o_tok + h * p.d;
#pragma unroll
  for (int e = 0; e < DP / 32; ++e)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      T::template store4<VEC>(to, 32 * e + 8 * g + 4 * half, p.d,
                              f32x4{o[e][4 * g] * inv, o[e][4 * g + 1] * inv, o[e][4 * g + 2] * inv, o[e][4 * g + 3] * inv});
  if (p.lse && half == 0)
    p.lse[((int64_t)at.seq * p.H + h) * p.N + at.t0 + qi] = kLn2 * (m + __builtin_amdgcn_logf(l));
}

}  // namespace

att::Params attention_params(const AttentionShape& s) {
  att::Params p = {};
  p.B = s.B, p.H = s.H, p.Hk = s.Hk, p.N = s.N, p.d = s.d, p.window = s.window, p.prefix = s.prefix, p.scale = s.scale;
  const int64_t rows = s.N, d = s.d;
  p.q_head = s.last ? d : rows * d, p.q_tok = s.last ? s.H * d : d, p.q_seq = s.packed ? 0 : rows * s.H * d;
  p.k_head = s.last ? d : rows * d, p.k_tok = s.last ? s.Hk * d : d, p.k_seq = s.packed ? 0 : rows * s.Hk * d;
  p.o_tok = s.H * d, p.o_seq = s.packed ? 0 : rows * s.H * d;
  return p;
}

int64_t attention_units(const AttentionShape& s, int rows) {
  return s.packed ? (int64_t)s.N / rows + s.B : ((int64_t)s.N + rows - 1) / rows;
}

int64_t attention_blocks(const AttentionShape& s, int rows, int heads) {
  const int64_t streams = s.packed ? s.Hk : (int64_t)s.B * s.Hk, units = attention_units(s, rows);
  return (streams * units + 7) / 8 * 8 * heads;
}

bool attention_supported(const AttentionShape& s) {
  return attention_blocks(s, 32, s.H / s.Hk) < kMostBlocks && (int64_t)s.H * s.d <= 1 << 22;   // (Loads' distances)
}

hipError_t launch_attention(const AttentionShape& s, const void* q, const void* k, const void* v,
                            const int32_t* offsets, const int32_t* lengths, void* out, float* lse,
                            hipStream_t stream) {
  if (s.N == 0) return hipSuccess;
  Params p = attention_params(s);
  p.q = q, p.k = k, p.v = v, p.out = out, p.lse = lse, p.offsets = offsets, p.lengths = lengths;
  p.streams = s.packed ? s.Hk : s.B * s.Hk, p.units = (int)attention_units(s, kRows);
  const unsigned grid = (unsigned)attention_blocks(s, kRows, s.H / s.Hk);
  return by_type(s.io, s.d, [&](auto bf16, auto dp, auto vec) {
    constexpr bool BF16 = decltype(bf16)::value;
    constexpr int DP = decltype(dp)::value, lds = 4 * keys_of<BF16>() * Tile<BF16, DP>::RB;
    attention_kernel<BF16, DP, decltype(vec)::value><<<grid, kThreads, lds, stream>>>(p);
    return hipGetLastError();
  });
}

}  // namespace titans
