// Gradient of the causal attention (tm_attention.hip has the forward pass and
// the mask).  With P_ij = exp(scale q_i . k_j - lse_i) where j is seen:
//
//   D_i = dout_i . out_i,  dS_ij = P_ij (dout_i . v_j - D_i)
//   dq_i = scale sum_j dS_ij k_j,  dk_j = scale sum_i dS_ij q_i,  dv_j = sum_i P_ij dout_i
//
// dk_j and dv_j are sums over the query heads that share the key head, too.
//
// Two kernels, so that every sum stays in one workgroup's registers, in a
// fixed order, with no atomics: one owns queries and runs over keys (D, dq),
// the other owns keys and runs over queries and heads (dk, dv).  Scores and
// dout . v are formed in both: seven products a tile instead of five, against
// an fp32 copy of dq in memory and an order of its sums that changes from call
// to call.
//
// Either kernel forms its scores so that what it owns lies in the lanes, and
// what it sums over in the registers, where P and dS are operands as they lie
// (tm_attention.h).  P and dS are rounded to bf16 there for bf16 tensors: each
// meets factors that have 8 bits themselves.  Gradients are 2.4e-3 off by that; as
// two bf16 numbers each they would be 1.8e-3 off, for 161 us instead of 127 (the
// case below), and 445 instead of 373 at d 128, 2 x 8 x 4096.
//
// Measured, 8 x 16 sequences of 1024, d 64, bf16: 54 us and 82 us, 130 for the call;
// matrix cores 30% busy, the rest is the exponentials' and masks' vector work and
// tiles of the diagonal, half of which the mask takes.  Registers decide the other
// kernel's waves a SIMD: d 128, one 373 us for 2 x 8 x 4096, two (which spill) 602;
// d 64, two 201 us for 4 x 16 x 2048, three 210.
#include "tm_attention.h"

namespace titans {
namespace {

using namespace att;

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kRows = 32 * kWaves;     // queries, or keys, of a workgroup

// rows of a tile in LDS
template <bool BF16, int DP>
constexpr int tile_of() { return BF16 ? 64 : 32; }

// Packed rows before the first sequence and behind the last: the gradient is
// zero.  Workgroup `unit` has rows unit * kRows .. of one head.
template <typename elem>
__device__ __forceinline__ void zero_rows(const Params& p, int unit, elem* a, elem* b, int64_t tok) {
  const int first = min(max(p.offsets[0], 0), p.N), end = min(max(p.offsets[p.B], 0), p.N);
  const int64_t r0 = (int64_t)unit * kRows;
  if (r0 >= first && r0 + kRows <= end) return;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = wave; i < kRows; i += kWaves) {
    const int64_t r = r0 + i;
    if (r >= p.N || (r >= first && r < end)) continue;
    for (int c = lane; c < p.d; c += 64) {
      a[r * tok + c] = (elem)0.f;
      if (b) b[r * tok + c] = (elem)0.f;
    }
  }
}

// Padded rows past a sequence's length.
template <typename elem>
__device__ __forceinline__ void zero_past(const Params& p, int row0, int n, elem* a, elem* b, int64_t tok) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int r = max(row0, n) + wave; r < min(row0 + kRows, p.N); r += kWaves)
    for (int c = lane; c < p.d; c += 64) {
      a[(int64_t)r * tok + c] = (elem)0.f;
      if (b) b[(int64_t)r * tok + c] = (elem)0.f;
    }
}

// dq, and per query lse log2 e and D for the other kernel.
template <bool BF16, int DP, int VEC>
__global__ void __launch_bounds__(kThreads, (BF16 ? (DP <= 64 ? 3 : 2) : DP < 96 ? 2 : 1)) attention_dq_kernel(Params p) {
  typedef Tile<BF16, DP> T;
  typedef typename T::elem elem;
  typedef typename T::frag frag;
  typedef typename T::op op;
  constexpr int KT = tile_of<BF16, DP>(), kBytes = KT * T::RB;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];   // [2][K, V]
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int stream, unit, head;
  if (!place_of(p, p.H / p.Hk, stream, unit, head)) return;
  Place at;
  const bool found = find<kRows>(p, stream, unit, at);
  const int h = at.head0 + head;
  if (p.offsets) zero_rows(p, unit, (elem*)p.dq + h * p.q_head, (elem*)nullptr, p.q_tok);
  // units of a padded row count tiles from its end; those past the length are all padding
  const int tiles = (at.n + kRows - 1) / kRows, tile = found ? tiles - 1 - at.tile : at.tile;
  elem* dq = (elem*)p.dq + at.seq * p.q_seq + h * p.q_head + (int64_t)at.t0 * p.q_tok;
  if (p.lengths) zero_past(p, tile * kRows, at.n, dq, (elem*)nullptr, p.q_tok);
  if (!found) return;
  const int i0 = tile * kRows, w0 = i0 + 32 * wave, qi = w0 + (lane & 31), last = at.n - 1;
  const int64_t qt = at.t0 + min(qi, last), kv = at.seq * p.k_seq + at.key_head * p.k_head + (int64_t)at.t0 * p.k_tok;
  const elem* kp = (const elem*)p.k + kv;
  const elem* vp = (const elem*)p.v + kv;

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

  op q[DP / 16], go[DP / 16];
  const int64_t ot = at.seq * p.o_seq + qt * p.o_tok + h * p.d, stat = ((int64_t)at.seq * p.H + h) * p.N + qt;
  float D = 0.f;
  {
    frag x[DP / 16], y[DP / 16];
    T::template row<VEC>(x, (const elem*)p.dout + ot, p.d, half);
    T::template row<VEC>(y, (const elem*)p.out + ot, p.d, half);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) {
#pragma unroll
      for (int e = 0; e < 8; ++e) D = fmaf((float)x[s][e], (float)y[s][e], D);
      go[s] = factor(x[s]);
    }
    T::template row<VEC>(x, (const elem*)p.q + at.seq * p.q_seq + h * p.q_head + qt * p.q_tok, p.d, half);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) q[s] = factor(x[s]);
  }
  D += other_half(D);
  const float lse = p.lse[stat] * kLog2e;
  if (half == 0 && qi <= last) {
    p.stats[stat] = lse;
    p.stats[p.stat_rows + stat] = D;
  }

  const int window = p.window ? p.window : INT_MAX;
  const float c = p.scale * kLog2e;
  f32x16 acc[DP / 32] = {};
  // (restrict: the transposing reads do not wait for the loads under way)
  auto step = [&](const unsigned char* __restrict__ kb, unsigned char* __restrict__ nb, int t, int k0) __attribute__((always_inline)) {
    const unsigned char* vb = kb + kBytes;
    if (t <= top) {
      load(nb, kp, p.k_tok, t * KT, end_of(t), p.d, tid);
      load(nb + kBytes, vp, p.k_tok, t * KT, end_of(t), p.d, tid);
    }
#pragma unroll
    for (int g = 0; g < KT / 32; ++g) {
      const int g0 = k0 + 32 * g;
      if (w0 > last || g0 > w0 + 31 || (w0 - (g0 + 31) >= window && g0 >= p.prefix)) continue;
      f32x16 x = {}, y = {};
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        mma(x, T::along(kb, 32 * g + (lane & 31), s, half), q[s]);
        mma(y, T::along(vb, 32 * g + (lane & 31), s, half), go[s]);
      }
      if (g0 + 31 > w0 || w0 + 31 - g0 >= window) mask_tile<true>(x, g0 + 4 * half, qi, window, p.prefix, g0 < p.prefix);
#pragma unroll
      for (int r = 0; r < 16; ++r) x[r] = __builtin_amdgcn_exp2f(fmaf(x[r], c, -lse)) * (y[r] - D);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const op w = operand<op>(x, s);
#pragma unroll
        for (int e = 0; e < DP / 32; ++e) mma(acc[e], T::across(kb, 32 * g, s, 32 * e, lane), w);
      }
    }
    };
  auto turn = [&](int buf) __attribute__((always_inline)) {
    const int k0 = t * KT;
    t = t + 1 == pre ? lo : t + 1;
    landed();
    step(smem + buf * 2 * kBytes, smem + (buf ^ 1) * 2 * kBytes, t, k0);
  };
  while (t <= top) {
    turn(0);
    if (t <= top) turn(1);
  }
  if (qi > last) return;
  dq += (int64_t)qi * p.q_tok;
#pragma unroll
  for (int e = 0; e < DP / 32; ++e)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      T::template store4<VEC>(dq, 32 * e + 8 * g + 4 * half, p.d,
                              f32x4{acc[e][4 * g], acc[e][4 * g + 1], acc[e][4 * g + 2], acc[e][4 * g + 3]} * p.scale);
}

// dk and dv of one key head.
template <bool BF16, int DP, int VEC>
__global__ void __launch_bounds__(kThreads, (BF16 ? (DP <= 64 ? 2 : 1) : DP < 64 ? 2 : 1)) attention_dkv_kernel(Params p) {
  typedef Tile<BF16, DP> T;
  typedef typename T::elem elem;
  typedef typename T::frag frag;
  typedef typename T::op op;
  constexpr int QT = tile_of<BF16, DP>(), kBytes = QT * T::RB, kStage = 2 * kBytes + 2 * 64 * 4;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];   // [2][Q, dout, lse[64], D[64]]
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int stream, unit, head;
  if (!place_of(p, 1, stream, unit, head)) return;
  Place at;
  const bool found = find<kRows>(p, stream, unit, at);
  const int part = blockIdx.y;
  const int64_t kv = at.seq * p.k_seq + at.key_head * p.k_head + (int64_t)at.t0 * p.k_tok;
  // where there are several parts, each leaves its sums in fp32
  float *pk = p.parts_k + part * p.part_size, *pv = p.parts_v + part * p.part_size;
  elem* dk = (elem*)p.dk + kv;
  elem* dv = (elem*)p.dv + kv;
  if (p.offsets) {
    if (p.parts == 1)
      zero_rows(p, unit, (elem*)p.dk + at.key_head * p.k_head, (elem*)p.dv + at.key_head * p.k_head, p.k_tok);
    else
      zero_rows(p, unit, pk + at.key_head * p.k_head, pv + at.key_head * p.k_head, p.k_tok);
  }
  if (p.lengths) {
    if (p.parts == 1)
      zero_past(p, at.tile * kRows, at.n, dk, dv, p.k_tok);
    else
      zero_past(p, at.tile * kRows, at.n, pk + kv, pv + kv, p.k_tok);
  }
  if (!found) return;
  const int j0 = at.tile * kRows, w0 = j0 + 32 * wave, kj = w0 + (lane & 31), last = at.n - 1, G = p.H / p.Hk;
  const int window = p.window ? p.window : INT_MAX;

  // tiles of queries: from the workgroup's first key to the last query in reach of its last one
  const int lo = j0 / QT;
  const int end = p.window && j0 >= p.prefix ? (int)min((int64_t)last, (int64_t)j0 + kRows - 1 + p.window - 1) : last;
  const int per = end / QT - lo + 1, share = (per * G + p.parts - 1) / p.parts;
  const int from = part * share, all = min(per * G, from + share);   // this part's
  if (VEC == kPieces && p.d < DP) {
    clear(smem, 2 * kStage, tid, kThreads);
    __syncthreads();
  }
  // tile number n of all: head n / per, query tile lo + n % per
  const int lt0 = lo + from % per;
  int lh = from / per, lt = lt0;
  const typename T::template Loads<QT, kThreads, VEC> load_q(p.q_tok, tid), load_o(p.o_tok, tid);
  auto issue = [&](unsigned char* b) __attribute__((always_inline)) {
    const int h = at.head0 + lh;
    const elem* qp = (const elem*)p.q + at.seq * p.q_seq + h * p.q_head + (int64_t)at.t0 * p.q_tok;
    const elem* go = (const elem*)p.dout + at.seq * p.o_seq + (int64_t)at.t0 * p.o_tok + h * p.d;
    load_q(b, qp, p.q_tok, lt * QT, last, p.d, tid);
    load_o(b + kBytes, go, p.o_tok, lt * QT, last, p.d, tid);
    if (wave < 2) {   // 64 rows of lse, of D (QT of them are used)
      const float* st = p.stats + (wave ? p.stat_rows : 0) + ((int64_t)at.seq * p.H + h) * p.N + at.t0;
      __builtin_amdgcn_global_load_lds((const void*)(st + min(lt * QT + lane, last)),
                                       (lds_void_ptr)(b + 2 * kBytes + wave * 256), 4, 0, 0);
    }
    if (++lt == lo + per) lt = lo, ++lh;
  };
  if (from < all) issue(smem);
  op k[DP / 16], v[DP / 16];
  {
    frag x[DP / 16];
    T::template row<VEC>(x, (const elem*)p.k + kv + (int64_t)min(kj, last) * p.k_tok, p.d, half);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) k[s] = factor(x[s]);
    T::template row<VEC>(x, (const elem*)p.v + kv + (int64_t)min(kj, last) * p.k_tok, p.d, half);
#pragma unroll
    for (int s = 0; s < DP / 16; ++s) v[s] = factor(x[s]);
  }

  const float c = p.scale * kLog2e;
  f32x16 ak[DP / 32] = {}, av[DP / 32] = {};
  auto step = [&](const unsigned char* __restrict__ qb, unsigned char* __restrict__ nb, int n, int q0) __attribute__((always_inline)) {
    const unsigned char* ob = qb + kBytes;
    const float* ls = (const float*)(qb + 2 * kBytes);
    if (n + 1 < all) issue(nb);
#pragma unroll
    for (int g = 0; g < QT / 32; ++g) {
      const int g0 = q0 + 32 * g;
      if (w0 > last || g0 > last || g0 + 31 < w0 || (g0 - (w0 + 31) >= window && w0 >= p.prefix)) continue;
      f32x16 x = {}, y = {};
#pragma unroll
      for (int s = 0; s < DP / 16; ++s) {
        mma(x, T::along(qb, 32 * g + (lane & 31), s, half), k[s]);
        mma(y, T::along(ob, 32 * g + (lane & 31), s, half), v[s]);
      }
      if (g0 < w0 + 31 || g0 + 31 > last || g0 + 31 - w0 >= window) {
        mask_tile<false>(x, g0 + 4 * half, kj, window, p.prefix, w0 < p.prefix);
#pragma unroll
        for (int r = 0; r < 16; ++r)
          x[r] = g0 + 4 * half + 8 * (r >> 2) + (r & 3) <= last ? x[r] : -__builtin_inff();
      }
      f32x16 ds;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const f32x4 l4 = *(const f32x4*)(ls + 32 * g + 8 * u + 4 * half), d4 = *(const f32x4*)(ls + 64 + 32 * g + 8 * u + 4 * half);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = 4 * u + e;
          x[r] = __builtin_amdgcn_exp2f(fmaf(x[r], c, -l4[e]));
          ds[r] = x[r] * (y[r] - d4[e]);
        }
      }
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const op w = operand<op>(x, s), z = operand<op>(ds, s);
#pragma unroll
        for (int e = 0; e < DP / 32; ++e) {
          mma(av[e], T::across(ob, 32 * g, s, 32 * e, lane), w);
          mma(ak[e], T::across(qb, 32 * g, s, 32 * e, lane), z);
        }
      }
    }
    };
  int qt = lt0;
  auto turn = [&](int n, int buf) __attribute__((always_inline)) {
    const int q0 = qt * QT;
    if (++qt == lo + per) qt = lo;
    landed();
    step(smem + buf * kStage, smem + (buf ^ 1) * kStage, n, q0);
  };
  for (int n = from; n < all; n += 2) {
    turn(n, 0);
    if (n + 1 < all) turn(n + 1, 1);
  }
  if (kj > last) return;
#pragma unroll
  for (int e = 0; e < DP / 32; ++e)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int ch = 32 * e + 8 * g + 4 * half;
      const f32x4 x = f32x4{ak[e][4 * g], ak[e][4 * g + 1], ak[e][4 * g + 2], ak[e][4 * g + 3]} * p.scale;
      const f32x4 y = {av[e][4 * g], av[e][4 * g + 1], av[e][4 * g + 2], av[e][4 * g + 3]};
      const int64_t row = (int64_t)kj * p.k_tok;
      if (p.parts == 1) {
        T::template store4<VEC>(dk + row, ch, p.d, x);
        T::template store4<VEC>(dv + row, ch, p.d, y);
      } else {
        Tile<false, DP>::template store4<VEC>(pk + kv + row, ch, p.d, x);
        Tile<false, DP>::template store4<VEC>(pv + kv + row, ch, p.d, y);
      }
    }
}

// dk and dv from their parts, in the parts' order
template <bool BF16>
__global__ void __launch_bounds__(256) attention_join_kernel(Params p) {
  typedef typename Types<BF16>::elem elem;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= p.part_size) return;
  const float* from = blockIdx.y ? p.parts_v : p.parts_k;
  float sum = from[i];
#pragma unroll 4
  for (int n = 1; n < p.parts; ++n) sum += from[n * p.part_size + i];
  ((elem*)(blockIdx.y ? p.dv : p.dk))[i] = (elem)sum;
}

// Workgroups that share a tile of keys' queries: so many that the device is
// full where tiles are few, with 4 tiles of queries each where there are.
// 3001 packed tokens, 2 key heads, d 80, fp32: 257 us, one workgroup a tile
// 1078; 2048 tokens, 4 key heads, d 64, bf16: 99, 281.  With twice as many both
// take as long, and 4096 tokens, 16 heads, d 128 2% longer.  Tiles are counted
// for the call, empty ones of short sequences too: 16 sequences, 4 key heads, d 64,
// one of 8192 tokens and the others of 256 have one workgroup a tile, 897 us for dk
// and dv, where that sequence alone has several, 419.
int parts_of(const AttentionShape& s) {
  const int64_t blocks = attention_blocks(s, kRows, 1), tiles = ((int64_t)s.N + 31) / 32 * (s.H / s.Hk);
  int64_t parts = 768 / (blocks > 0 ? blocks : 1);
  if (parts > tiles / 4) parts = tiles / 4;
  return parts < 1 ? 1 : parts > 8 ? 8 : (int)parts;
}

int64_t key_elements(const AttentionShape& s) { return (s.packed ? 1 : (int64_t)s.B) * s.N * s.Hk * s.d; }
int64_t stat_bytes(const AttentionShape& s) { return ((s.packed ? 1 : (int64_t)s.B) * s.H * s.N * 8 + 15) / 16 * 16; }

}  // namespace

int64_t attention_backward_ws_bytes(const AttentionShape& s) {
  const int parts = parts_of(s);
  return stat_bytes(s) + (parts > 1 ? key_elements(s) * parts * 8 : 0);
}

hipError_t launch_attention_backward(const AttentionShape& s, const void* q, const void* k, const void* v,
                                     const int32_t* offsets, const int32_t* lengths, const void* out, const float* lse,
                                     const void* dout, void* dq, void* dk, void* dv, float* ws, hipStream_t stream) {
  if (s.N == 0) return hipSuccess;
  Params p = attention_params(s);
  p.q = q, p.k = k, p.v = v, p.out = (void*)out, p.lse = (float*)lse, p.dout = dout, p.offsets = offsets, p.lengths = lengths;
  p.dq = dq, p.dk = dk, p.dv = dv, p.stats = ws, p.stat_rows = (s.packed ? 1 : (int64_t)s.B) * s.H * s.N;
  p.streams = s.packed ? s.Hk : s.B * s.Hk, p.units = (int)attention_units(s, kRows);
  p.parts = parts_of(s), p.part_size = key_elements(s);
  p.parts_k = ws + stat_bytes(s) / 4, p.parts_v = p.parts_k + p.parts * p.part_size;
  hipError_t err = by_type(s.io, s.d, [&](auto bf16, auto dp, auto vec) {
    constexpr bool BF16 = decltype(bf16)::value;
    constexpr int DP = decltype(dp)::value, VEC = decltype(vec)::value;
    constexpr int lds = 4 * tile_of<BF16, DP>() * Tile<BF16, DP>::RB, stats = 4 * 64 * 4;
    attention_dq_kernel<BF16, DP, VEC>
        <<<(unsigned)attention_blocks(s, kRows, s.H / s.Hk), kThreads, lds, stream>>>(p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    auto kernel = attention_dkv_kernel<BF16, DP, VEC>;
    e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds + stats);
    if (e != hipSuccess) return e;
    // the keys of the prefix are seen by all queries, those behind it only in the window
    if (s.window && !s.packed) p.ahead = (int)(((int64_t)s.prefix + kRows - 1) / kRows);
    kernel<<<dim3((unsigned)attention_blocks(s, kRows, 1), p.parts), kThreads, lds + stats, stream>>>(p);
    return hipGetLastError();
  });
  if (err != hipSuccess || p.parts == 1) return err;
  const dim3 grid((unsigned)((p.part_size + 255) / 256), 2);
  if (s.io == TM_IO_BF16)
    attention_join_kernel<true><<<grid, 256, 0, stream>>>(p);
  else
    attention_join_kernel<false><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace titans
