// Attention of a few new tokens a sequence over a cache of keys and values,
// the form of tm_attention.hip that a model answers with: the new tokens are
// the last n of lengths[b], token i of them at position lengths[b] - n + i,
// and see what that kernel's mask lets them see.
//
// The call is bound by reading the cache once.  All query heads of a key head
// and all new tokens are rows of one product (up to 32 of them for one pass
// over the keys), and the keys are split over workgroups and over the waves in
// them; every wave runs through its own tiles of 32 keys in its own piece of
// LDS, the next tile under way, and meets the others only at the end, where
// the waves' maxima, sums and outputs are joined.  Parts of a row in several
// workgroups are joined by a second kernel, in the parts' order.
//
// Measured: 192 sequences of up to 2048 keys, 16 query heads, 4 key heads, d 128, bf16:
// 82 us, 4.9 TB/s, what a copy reaches.  One sequence of 16384, 16 heads, d 64: 14 us,
// 4.7 TB/s, and 4 us for the second kernel.  fp32 at d 96 and more has two waves a
// workgroup and one workgroup a CU (a wave's stages are 64 KB): 24 x 16 x 4096 x 128
// 541 us, 3.0 TB/s, bound by the splitting into planes; at d 64 168 us, 4.8 TB/s.
//
// bf16 weights meet the values as two bf16 numbers, what they are rounded to and
// what that left: out is then off by its own rounding alone, and beside the
// reading of the cache it costs 1 to 2% (192 sequences 80.7 us by one number, 81.5;
// 128 queries a key head, 8 sequences of 4096, d 128, 66.6 both).
//
// New keys and values come in with the call and are stored to the cache by the
// wave whose tile they belong to; nobody reads those rows of the cache.
#include "tm_attention.h"

namespace titans {
namespace {

using namespace att;

constexpr int kKeys = 32;        // of a tile
constexpr int kMostParts = 64;   // of a row: a lane each when they are joined

struct StepParams {
  const void *q, *k_new, *v_new;
  void *k, *v, *out;
  const int32_t* lengths;
  float *po, *pml;   // parts: outputs [row][part][d], (m, l) [row][part][2], each from 16 bytes on
  int B, H, Hk, n, C, d, window, prefix, row_tiles, parts;
  float scale;
};

template <bool BF16, int DP>
constexpr int waves_of() { return Tile<BF16, DP>::RB > 256 ? 2 : 4; }

// LDS of a wave: two stages of keys and values, in the end its rows' outputs
template <bool BF16, int DP>
constexpr int wave_lds() { return 4 * kKeys * Tile<BF16, DP>::RB; }

// Keys j0 .. j0 + 31 of the cache, those from `fresh` on from the new ones.
template <bool BF16, int DP, int VEC, typename T = Tile<BF16, DP>>
__device__ __forceinline__ void load_keys(const typename T::template Loads<kKeys, 64, VEC>& load, unsigned char* t,
                                          const typename T::elem* cache, const typename T::elem* added, int fresh, int j0,
                                          int last, int d, int lane) {
  typedef typename T::elem elem;
  if (j0 + kKeys <= fresh) {
    load(t, cache, d, j0, last, d, lane);
    return;
  }
#pragma unroll 4
  for (int i = 0; i < load.kCount; ++i) {
    const int at = i * 64 + lane, r = at / T::NC, c = (at % T::NC) ^ T::swz(r), j = min(j0 + r, last);
    const elem* row = j >= fresh ? added + (int64_t)(j - fresh) * d : cache + (int64_t)j * d;
    if constexpr (VEC != kOdd) {
      if (VEC == kFull && DP == T::LS ? true : c * T::PC < d)
        __builtin_amdgcn_global_load_lds((const void*)(row + c * T::PC), (lds_void_ptr)(t + i * 1024), 16, 0, 0);
    } else {
      *(typename T::piece*)(t + at * 16) = T::odd(row, c * T::PC, d);
    }
  }
}

template <bool BF16, int DP, int VEC>
__global__ void __launch_bounds__((64 * waves_of<BF16, DP>())) attention_step_kernel(StepParams p) {
  typedef Tile<BF16, DP> T;
  typedef typename T::elem elem;
  typedef typename T::op op;
  constexpr int W = waves_of<BF16, DP>(), kBytes = kKeys * T::RB;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  __shared__ float ml[W][2][32];
  const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = blockIdx.x % p.parts, rt = blockIdx.x / p.parts % p.row_tiles, stream = blockIdx.x / p.parts / p.row_tiles;
  const int b = stream / p.Hk, hk = stream % p.Hk, G = p.H / p.Hk, rows = G * p.n;
  const int len = __builtin_amdgcn_readfirstlane(min(max(p.lengths[b], 0), p.C)), last = len - 1;
  const int r = 32 * rt + (lane & 31), pos = r < rows ? len - p.n + r % p.n : -1;
  const int fresh = p.k_new ? max(len - p.n, 0) : INT_MAX;
  const int skip = max(p.n - len, 0);   // new tokens that have no place
  const elem* kn = (const elem*)p.k_new + ((int64_t)stream * p.n + skip) * p.d;
  const elem* vn = (const elem*)p.v_new + ((int64_t)stream * p.n + skip) * p.d;
  elem* kc = (elem*)p.k + (int64_t)stream * p.C * p.d;
  elem* vc = (elem*)p.v + (int64_t)stream * p.C * p.d;
  const int window = p.window ? p.window : INT_MAX;

  // tiles: those of the prefix, then those in reach of the first new token
  const int first = max(len - p.n, 0);
  const int lo = p.window ? max(0, first - p.window + 1) / kKeys : 0;
  const int pre = min((p.prefix + kKeys - 1) / kKeys, lo);
  const int total = len ? pre + last / kKeys - lo + 1 : 0, per = (total + p.parts - 1) / p.parts;
  const int end = min(total, (part + 1) * per);
  unsigned char* mine = smem + wave * wave_lds<BF16, DP>();
  int x = part * per + wave;
  if (VEC == kPieces && p.d < DP) clear(mine, 4 * kBytes, lane, 64);
  auto tile = [&](int i) __attribute__((always_inline)) { return i < pre ? i : lo + i - pre; };
  const typename T::template Loads<kKeys, 64, VEC> load(p.d, lane);
  auto issue = [&](unsigned char* t, int i) __attribute__((always_inline)) {
    // (of the prefix's tiles only the persistent tokens are read: a NaN behind them is not met by a weight of 0)
    const int to = i < pre ? min(last, p.prefix - 1) : last;
    load_keys<BF16, DP, VEC>(load, t, kc, kn, fresh, tile(i) * kKeys, to, p.d, lane);
    load_keys<BF16, DP, VEC>(load, t + kBytes, vc, vn, fresh, tile(i) * kKeys, to, p.d, lane);
  };
  // (what was cleared is there before a load may write beside it)
  landed_in_wave();
  if (x < end) issue(mine, x);
  op q[DP / 16];
  {
    typename T::frag f[DP / 16];
    T::template row<VEC>(f, (const elem*)p.q + ((int64_t)stream * rows + min(r, rows - 1)) * p.d, p.d, half);
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) q[i] = factor(f[i]);
  }

  const float c = p.scale * kLog2e;
  float m = kLowest, l = 0.f;
  f32x16 o[DP / 32] = {};
  auto step = [&](const unsigned char* __restrict__ kb, unsigned char* __restrict__ nb) __attribute__((always_inline)) {
    const unsigned char* vb = kb + kBytes;
    const int k0 = tile(x) * kKeys;
    if (x + W < end) issue(nb, x + W);
    f32x16 s = {};
#pragma unroll
    for (int i = 0; i < DP / 16; ++i) mma(s, T::along(kb, lane & 31, i, half), q[i]);
    if (k0 + kKeys > first || last - k0 >= window) mask_tile<true>(s, k0 + 4 * half, pos, window, p.prefix, k0 < p.prefix);
    float mx = s[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
    mx = fmaxf(mx, other_half(mx)) * c;
    const float to = fmaxf(m, mx), f = __builtin_amdgcn_exp2f(m - to);
    m = to;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      s[i] = __builtin_amdgcn_exp2f(fmaf(s[i], c, -m));
      sum += s[i];
    }
    l = fmaf(l, f, sum);
#pragma unroll
    for (int e = 0; e < DP / 32; ++e)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[e][i] *= f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const op w = operand<op>(s, i);
      bf16x8 rest;
      if constexpr (BF16) rest = remainder(s, i, w);
#pragma unroll
      for (int e = 0; e < DP / 32; ++e) {
        const op y = T::across(vb, 0, i, 32 * e, lane);
        if constexpr (BF16) mma(o[e], y, rest);
        mma(o[e], y, w);
      }
    }
    // the tile's new rows go to the cache
    if (rt == 0 && k0 + kKeys > fresh)
      for (int j = max(fresh, k0); j < min(len, k0 + kKeys); ++j)
        for (int e = lane; e < p.d; e += 64) {
          kc[(int64_t)j * p.d + e] = kn[(int64_t)(j - fresh) * p.d + e];
          vc[(int64_t)j * p.d + e] = vn[(int64_t)(j - fresh) * p.d + e];
        }
  };
  for (; x < end; x += W) {
    landed_in_wave();   // its tile is there
    step(mine, mine + 2 * kBytes);
    x += W;
    if (x >= end) break;
    landed_in_wave();
    step(mine + 2 * kBytes, mine);
  }

  // join the waves: each leaves its rows' outputs in LDS, [row][DP + 4]
  constexpr int LD = DP + 4;
  static_assert(32 * LD * 4 <= wave_lds<BF16, DP>(), "");
  l += other_half(l);
  landed_in_wave();
#pragma unroll
  for (int e = 0; e < DP / 32; ++e)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      *(f32x4*)(mine + ((lane & 31) * LD + 32 * e + 8 * g + 4 * half) * 4) =
          f32x4{o[e][4 * g], o[e][4 * g + 1], o[e][4 * g + 2], o[e][4 * g + 3]};
  if (half == 0) ml[wave][0][lane] = m, ml[wave][1][lane] = l;
  __syncthreads();
  constexpr int kLanes = DP / 4;   // of a row
  for (int i = tid / kLanes; i < 32 && 32 * rt + i < rows; i += 64 * W / kLanes) {
    const int ch = tid % kLanes * 4;
    float top = ml[0][0][i], sum = 0.f;
#pragma unroll
    for (int w = 1; w < W; ++w) top = fmaxf(top, ml[w][0][i]);
    f32x4 acc = {};
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = __builtin_amdgcn_exp2f(ml[w][0][i] - top);
      sum = fmaf(ml[w][1][i], f, sum);
      acc += *(const f32x4*)(smem + w * wave_lds<BF16, DP>() + (i * LD + ch) * 4) * f;
    }
    const int row = 32 * rt + i;
    if (p.parts == 1) {
      const float inv = sum != 0.f ? 1.f / sum : 0.f;   // a row that sees nothing: zeros
      elem* to = (elem*)p.out + (((int64_t)b * p.n + row % p.n) * p.H + hk * G + row / p.n) * p.d;
      T::template store4<VEC>(to, ch, p.d, acc * inv);
    } else {
      const int64_t at = ((int64_t)stream * rows + row) * p.parts + part;
      Tile<false, DP>::template store4<VEC>(p.po + at * p.d, ch, p.d, acc);
      if (ch == 0) p.pml[2 * at] = top, p.pml[2 * at + 1] = sum;
    }
  }
}

// Parts of a row, a workgroup each row: its waves share the parts, then a
// column's sums are joined in their order.
template <bool BF16>
__global__ void __launch_bounds__(256) step_join_kernel(StepParams p) {
  typedef typename Types<BF16>::elem elem;
  __shared__ float acc[4][128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, G = p.H / p.Hk, rows = G * p.n;
  const int64_t at = blockIdx.x;
  const float* o = p.po + at * p.parts * p.d;
  float m = kLowest, l = 0.f;
  if (lane < p.parts) {
    const f32x2 x = *(const f32x2*)(p.pml + 2 * (at * p.parts + lane));
    m = x[0], l = x[1];
  }
  // columns lane and 64 + lane of parts wave, wave + 4 ..: loads before the weights are known
  constexpr int kEach = kMostParts / 4;
  float x[kEach][2];
#pragma unroll
  for (int i = 0; i < kEach; ++i)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int s = wave + 4 * i, c = lane + 64 * e;
      x[i][e] = s < p.parts && c < p.d ? o[(int64_t)s * p.d + c] : 0.f;
    }
  float top = m;
#pragma unroll
  for (int i = 1; i < 64; i *= 2) top = fmaxf(top, __shfl_xor(top, i));
  const float f = __builtin_amdgcn_exp2f(m - top);
  float sum = l * f;
#pragma unroll
  for (int i = 1; i < 64; i *= 2) sum += __shfl_xor(sum, i);
  float a[2] = {};
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const float w = __shfl(f, wave + 4 * i);
    a[0] = fmaf(x[i][0], w, a[0]);
    a[1] = fmaf(x[i][1], w, a[1]);
  }
  acc[wave][lane] = a[0], acc[wave][64 + lane] = a[1];
  __syncthreads();
  if (tid >= p.d) return;
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const int row = (int)(at % rows);
  const int64_t stream = at / rows, b = stream / p.Hk, hk = stream % p.Hk;
  elem* out = (elem*)p.out + ((b * p.n + row % p.n) * p.H + hk * G + row / p.n) * p.d;
  out[tid] = (elem)((acc[0][tid] + acc[1][tid] + acc[2][tid] + acc[3][tid]) * inv);
}

int64_t row_tiles_of(const AttentionStepShape& s) { return ((int64_t)s.H / s.Hk * s.n + 31) / 32; }

// Workgroups of a row: so many that every CU has one, with 8 tiles each at
// least.  Each has four waves that load ahead on their own, so more of them
// only add to what is joined.  In us, by one, two and four a CU (bf16, one query a
// key head unless said): 192 sequences of 2048 keys, 4 queries, d 128: 81, 82,
// 93; 64 of them 44, 50, 52; one of 16384, d 64: 18.5, 18.5, 20; 8 of 1024, fp32,
// d 64: 16.8, 16.8, 18.  Lengths, which the host does not know, have no say: among
// 256 rows of one workgroup each a long context is read by its own alone (64
// sequences, 4 key heads, d 128, room for 65536: one full and the others of 512
// tokens 590 us, all of 1528 41).
int parts_of(const AttentionStepShape& s) {
  const int64_t rows = (int64_t)s.B * s.Hk * row_tiles_of(s);
  if (rows == 0) return 1;
  int64_t keys = s.C;
  if (s.window && (int64_t)s.window + s.n + s.prefix < keys) keys = (int64_t)s.window + s.n + s.prefix;
  int64_t parts = (256 + rows - 1) / rows, most = keys / kKeys / 8;
  if (parts > most) parts = most;
  if (parts > kMostParts) parts = kMostParts;
  return parts < 1 ? 1 : (int)parts;
}

// Bytes of the parts' outputs, up to where their maxima and sums (read in pairs) may lie.
int64_t outputs_bytes(const AttentionStepShape& s, int parts) {
  return ((int64_t)s.B * s.H * s.n * parts * s.d * 4 + 15) / 16 * 16;
}

}  // namespace

bool attention_step_supported(const AttentionStepShape& s) {
  // (the queries first: parts_of() multiplies what they bound)
  return (double)s.B * s.H * s.n < (double)kMostBlocks &&
         (double)s.B * s.Hk * row_tiles_of(s) * parts_of(s) < (double)kMostBlocks;
}

int64_t attention_step_ws_bytes(const AttentionStepShape& s) {
  const int parts = parts_of(s);
  return parts == 1 ? 0 : outputs_bytes(s, parts) + (int64_t)s.B * s.H * s.n * parts * 8;
}

hipError_t launch_attention_step(const AttentionStepShape& s, const void* q, void* k, void* v, const void* k_new,
                                 const void* v_new, const int32_t* lengths, void* out, float* ws, hipStream_t stream) {
  if (s.n == 0) return hipSuccess;
  StepParams p = {};
  p.q = q, p.k = k, p.v = v, p.k_new = k_new, p.v_new = v_new, p.lengths = lengths, p.out = out;
  p.B = s.B, p.H = s.H, p.Hk = s.Hk, p.n = s.n, p.C = s.C, p.d = s.d, p.window = s.window, p.prefix = s.prefix;
  p.scale = s.scale, p.row_tiles = (int)row_tiles_of(s), p.parts = parts_of(s);
  const int64_t rows = (int64_t)s.B * s.H * s.n;
  p.po = ws, p.pml = ws + outputs_bytes(s, p.parts) / 4;
  const unsigned grid = (unsigned)(s.B * s.Hk * p.row_tiles * p.parts);
  hipError_t err = by_type(s.io, s.d, [&](auto bf16, auto dp, auto vec) {
    constexpr bool BF16 = decltype(bf16)::value;
    constexpr int DP = decltype(dp)::value, W = waves_of<BF16, DP>(), lds = W * wave_lds<BF16, DP>();
    auto kernel = attention_step_kernel<BF16, DP, decltype(vec)::value>;
    hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    kernel<<<grid, 64 * W, lds, stream>>>(p);
    return hipGetLastError();
  });
  if (err != hipSuccess || p.parts == 1) return err;
  if (s.io == TM_IO_BF16)
    step_join_kernel<true><<<(unsigned)rows, 256, 0, stream>>>(p);
  else
    step_join_kernel<false><<<(unsigned)rows, 256, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace titans
