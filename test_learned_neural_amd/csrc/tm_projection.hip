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
// has a tile of out, whose operands go through LDS in slices of kT steps of t,
// loaded straight to it kStages - 1 slices ahead.  Accumulators have c in
// registers and r in lanes; they go through LDS once more, so that bias,
// residual and out are met in whole rows.
//
// fp32 factors go through the bf16 matrix cores as three planes each
// (tm_attention.h).
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
constexpr int kNarrowRows = 64;  // rows up to which the narrow kernel runs

// what a slice's end past t is made of
__device__ const float4 kZeros[1] = {};

struct Gemm {
  const void *P, *Q;
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
// One operand's slice in LDS, and its fragments: EXTENT values of c (or r) by
// kT of t; ALONG: rows are values, else rows are steps of t.
template <bool BF16, bool ALONG, int EXTENT, int THREADS>
struct Slice {
  typedef typename att::Types<BF16>::elem elem;
  typedef typename att::Types<BF16>::frag frag;
  static constexpr int kSize = BF16 ? 2 : 4;
  static constexpr int PC = 16 / kSize;
  static constexpr int ROWS = ALONG ? EXTENT : kT, COLS = ALONG ? kT : EXTENT;
  static constexpr int RB = COLS * kSize, NC = RB / 16;
  static constexpr int kBytes = ROWS * RB;
  static constexpr int kLoads = kBytes / 16 / THREADS;   // of a thread
  static_assert(kBytes % (16 * THREADS) == 0, "");

  static __device__ __forceinline__ int swz(int r) {
    if (NC == 4) return (r >> 1) & 3;
    if (NC == 8) return ALONG ? r & 7 : (r & 1) << 2 | ((r >> 1) & 3);
    return (r & 3) << 2 | ((r >> 2) & 3);
  }

  // values v0.. and steps t0..; `values` and `end` bound both.  Values past the
  // end are some other value (their results are not stored), steps are zero.
  template <bool VEC>
  static __device__ __forceinline__ void load(unsigned char* s, const elem* src, int64_t row, int64_t v0, int64_t values,
                                              int64_t t0, int64_t end, int tid) {
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int base = i * THREADS + wave * 64, at = base + (tid & 63);
      const int r = at / NC, c = ((at % NC) ^ swz(r)) * PC;
      const int64_t t = t0 + (ALONG ? c : r);
      if constexpr (VEC) {
        int64_t v = v0 + (ALONG ? r : c);
        if (v >= values) v = ALONG ? values - 1 : values - PC;
        const elem* p = src + (ALONG ? v * row + t : t * row + v);
        if (t >= end) p = (const elem*)kZeros;
        __builtin_amdgcn_global_load_lds((const void*)p, (lds_void_ptr)(s + base * 16), 16, 0, 0);
      } else {
        elem x[PC];
#pragma unroll
        for (int e = 0; e < PC; ++e) {
          int64_t v = v0 + (ALONG ? r : c + e);
          v = v < values ? v : values - 1;
          const int64_t te = t + (ALONG ? e : 0);
          x[e] = te < end ? src[ALONG ? v * row + te : te * row + v] : (elem)0.f;
        }
#pragma unroll
        for (int e = 0; e < PC; ++e) ((elem*)(s + at * 16))[e] = x[e];
      }
    }
  }

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

// ---------------------------------------------------------------- the tile kernel
// TR x TC of out by WR x WC waves.
template <bool BF16_, int TR_, int TC_, int WR_, int WC_, int STAGES_>
struct Shape2 {
  static constexpr bool BF16 = BF16_;
  static constexpr int TR = TR_, TC = TC_, WR = WR_, WC = WC_, STAGES = STAGES_;
  static constexpr int kThreads = 64 * WR * WC;
};

template <typename S, bool P_ALONG, bool Q_ALONG, bool VEC, bool F32_OUT>
__global__ void __launch_bounds__(S::kThreads, 2) gemm_kernel(Gemm g) {
  constexpr bool BF16 = S::BF16;
  constexpr int NR = S::TR / S::WR / 32, NCOL = S::TC / S::WC / 32, CW = 32 * NCOL;
  typedef Slice<BF16, P_ALONG, S::TC, S::kThreads> SP;
  typedef Slice<BF16, Q_ALONG, S::TR, S::kThreads> SQ;
  typedef typename SP::elem elem;
  typedef typename att::Types<BF16>::op Op;
  constexpr int kStage = SP::kBytes + SQ::kBytes, kLoads = SP::kLoads + SQ::kLoads;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wr = wave / S::WC, wc = wave % S::WC;

  // Blocks go round the 8 XCDs; each takes a run of tiles that walks the
  // columns of 8 row tiles at a time, so that both factors stay in its L2
  const unsigned tiles = (unsigned)g.row_tiles * g.col_tiles, all = tiles * g.parts;
  const unsigned share = (all + 7) / 8;
  unsigned id = (blockIdx.x & 7) * share + (blockIdx.x >> 3);
  if (id >= all || (blockIdx.x >> 3) >= share) return;
  const int part = id / tiles;
  id -= part * tiles;
  const int group = id / (8 * g.col_tiles), rows_here = min(8, g.row_tiles - 8 * group);
  id -= group * 8 * g.col_tiles;
  const int64_t r0 = (int64_t)(8 * group + id % rows_here) * S::TR;
  const int c0 = id / rows_here * S::TC;

  const int64_t t0 = part * g.per, t1 = t0 + g.per < g.T ? t0 + g.per : g.T;
  const int slices = t1 > t0 ? (int)((t1 - t0 + kT - 1) / kT) : 0;
  auto issue = [&](unsigned char* s, int i) {
    SP::template load<VEC>(s, (const elem*)g.P, g.p_row, c0, g.C, t0 + (int64_t)i * kT, t1, tid);
    SQ::template load<VEC>(s + SP::kBytes, (const elem*)g.Q, g.q_row, r0, g.R, t0 + (int64_t)i * kT, t1, tid);
  };
  f32x16 acc[NR][NCOL] = {};
  auto step = [&](const unsigned char* __restrict__ cur, unsigned char* __restrict__ next, int i) {
    if (i < slices) issue(next, i);
#pragma unroll
    for (int k = 0; k < kT / 16; ++k) {
      Op q[NR];
#pragma unroll
      for (int a = 0; a < NR; ++a) q[a] = factor(SQ::get(cur + SP::kBytes, 32 * (NR * wr + a), k, lane));
#pragma unroll
      for (int b = 0; b < NCOL; ++b) {
        const Op p = factor(SP::get(cur, 32 * (NCOL * wc + b), k, lane));
#pragma unroll
        for (int a = 0; a < NR; ++a) att::mma(acc[a][b], p, q[a]);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < S::STAGES - 1; ++i)
    if (i < slices) issue(smem + i * kStage, i);
  int cur = 0, next = S::STAGES - 1;
  for (int i = 0; i < slices; ++i) {
    // this slice has landed; those issued after it may still be under way
    if (!VEC || S::STAGES == 2 || i + S::STAGES - 2 >= slices)
      att::landed();
    else
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((S::STAGES - 2) * kLoads) : "memory");
    step(smem + cur * kStage, smem + next * kStage, i + S::STAGES - 1);
    cur = cur + 1 == S::STAGES ? 0 : cur + 1;
    next = next + 1 == S::STAGES ? 0 : next + 1;
  }

  // through LDS, 32 rows of the wave's columns at a time
  constexpr int LD = CW + 4, kLanes = CW / 8;
  static_assert(32 * LD * 4 * S::WR * S::WC <= S::STAGES * kStage, "");
  __syncthreads();
  float* mine = (float*)(smem + wave * 32 * LD * 4);
  const int ch = lane % kLanes * 8, c = c0 + wc * CW + ch;
  const bool whole = F32_OUT ? g.C % 4 == 0 : g.C % 8 == 0;   // rows of 16-byte pieces
  float bias[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) bias[e] = g.bias && c + e < g.C ? g.bias[c + e] : 0.f;
#pragma unroll
  for (int a = 0; a < NR; ++a) {
    att::landed_in_wave();   // (the rows before have been read)
#pragma unroll
    for (int b = 0; b < NCOL; ++b)
#pragma unroll
      for (int u = 0; u < 4; ++u)
        *(f32x4*)(mine + (lane & 31) * LD + 32 * b + 8 * u + 4 * (lane >> 5)) =
            f32x4{acc[a][b][4 * u], acc[a][b][4 * u + 1], acc[a][b][4 * u + 2], acc[a][b][4 * u + 3]};
    att::landed_in_wave();
#pragma unroll
    for (int i = 0; i < 32 * kLanes / 64; ++i) {
      const int row = i * (64 / kLanes) + lane / kLanes;
      const int64_t r = r0 + 32 * (NR * wr + a) + row;
      if (r >= g.R || c >= g.C) continue;
      const f32x4 x0 = *(const f32x4*)(mine + row * LD + ch), x1 = *(const f32x4*)(mine + row * LD + ch + 4);
      f32x8 x = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
      const int64_t o = r * g.C + c;
      if constexpr (F32_OUT) {
        float* out = (float*)g.out + (int64_t)part * g.R * g.C + o;
        if (whole) {
          *(f32x4*)out = x0;
          if (c + 4 < g.C) *(f32x4*)(out + 4) = x1;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < g.C) out[e] = x[e];
        }
      } else {
        typedef __attribute__((ext_vector_type(8))) elem elem8;
        elem* out = (elem*)g.out + o;
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += bias[e];
        if (g.pre) {
          elem* pre = (elem*)g.pre + o;
          if (whole)
            *(elem8*)pre = __builtin_convertvector(x, elem8);
          else
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (c + e < g.C) pre[e] = (elem)x[e];
        }
        if (g.silu)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= sigmoid(x[e]);
        if (g.residual) {
          const elem* res = (const elem*)g.residual + o;
          if (whole)
            x += __builtin_convertvector(*(const elem8*)res, f32x8);
          else
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (c + e < g.C) x[e] += (float)res[e];
        }
        if (whole)
          *(elem8*)out = __builtin_convertvector(x, elem8);
        else
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c + e < g.C) out[e] = (elem)x[e];
      }
    }
  }
}

// ---------------------------------------------------------------- few rows
// A workgroup has 16 columns and all rows (in blocks of 16) of out; its waves
// share t, every wave taking 32 of each 256 steps, from memory straight to the
// operands, and meet in LDS.  Bound by reading W once.
template <bool BF16, int BLOCKS, bool VEC>
__global__ void __launch_bounds__(512) narrow_kernel(Gemm g) {
  typedef typename att::Types<BF16>::elem elem;
  typedef typename att::Types<BF16>::frag frag;
  typedef typename att::Types<BF16>::op Op;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c0 = blockIdx.x * 16, v = lane & 15;
  const elem* p = (const elem*)g.P + (int64_t)min(c0 + v, g.C - 1) * g.p_row;
  f32x4 acc[BLOCKS] = {};
  auto get = [&](const elem* row, int t) {
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
// dz = dout act'(pre), rounded to the io type that the two products read, and
// its column sums: a workgroup has 64 lanes x PC columns and `per` rows, which
// its 4 waves share.
template <bool BF16, bool VEC>
__global__ void __launch_bounds__(256) slope_kernel(const void* dout_, const void* pre_, void* dz_, float* sums, int64_t R,
                                                    int C, int64_t per) {
  typedef typename att::Types<BF16>::elem elem;
  constexpr int PC = VEC ? (BF16 ? 8 : 4) : 1;
  typedef __attribute__((ext_vector_type(PC))) elem piece;
  const elem *dout = (const elem*)dout_, *pre = (const elem*)pre_;
  elem* dz = (elem*)dz_;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = ((int)blockIdx.x * 64 + lane) * PC;
  const int64_t r0 = blockIdx.y * per, r1 = r0 + per < R ? r0 + per : R;
  float sum[PC] = {};
  if (c < C)
#pragma unroll 4
    for (int64_t r = r0 + wave; r < r1; r += 4) {
      const int64_t o = r * C + c;
      piece x = *(const piece*)(dout + o);
      if (pre) {
        const piece z = *(const piece*)(pre + o);
#pragma unroll
        for (int e = 0; e < PC; ++e) {
          const float a = (float)z[e], sg = sigmoid(a);
          x[e] = (elem)((float)x[e] * sg * fmaf(a, 1.f - sg, 1.f));
        }
        *(piece*)(dz + o) = x;
      }
#pragma unroll
      for (int e = 0; e < PC; ++e) sum[e] += (float)x[e];
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
template <typename S, bool P_ALONG, bool Q_ALONG, bool VEC, bool F32_OUT>
hipError_t launch_tiles(Gemm g, hipStream_t stream) {
  constexpr int lds = S::STAGES * (Slice<S::BF16, P_ALONG, S::TC, S::kThreads>::kBytes +
                                   Slice<S::BF16, Q_ALONG, S::TR, S::kThreads>::kBytes);
  g.row_tiles = (int)((g.R + S::TR - 1) / S::TR), g.col_tiles = (g.C + S::TC - 1) / S::TC;
  const int64_t all = (int64_t)g.row_tiles * g.col_tiles * g.parts;
  auto kernel = gemm_kernel<S, P_ALONG, Q_ALONG, VEC, F32_OUT>;
  hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (e != hipSuccess) return e;
  kernel<<<(unsigned)((all + 7) / 8 * 8), S::kThreads, lds, stream>>>(g);
  return hipGetLastError();
}

template <bool BF16>
using Large = Shape2<BF16, BF16 ? 256 : 128, 128, BF16 ? 4 : 2, BF16 ? 1 : 2, BF16 ? 3 : 2>;
template <bool BF16>
using Small = Shape2<BF16, 64, 64, 2, 2, BF16 ? 3 : 2>;

// Large tiles from one for every CU on, small ones below.
bool large(int64_t R, int64_t C, int io) {
  const int64_t tr = io == TM_IO_BF16 ? 256 : 128;
  return (R + tr - 1) / tr * ((C + 127) / 128) >= 192;
}

template <bool P_ALONG, bool Q_ALONG, bool F32_OUT, bool BF16, bool VEC>
hipError_t launch_sized(const Gemm& g, bool big, hipStream_t stream) {
  return big ? launch_tiles<Large<BF16>, P_ALONG, Q_ALONG, VEC, F32_OUT>(g, stream)
             : launch_tiles<Small<BF16>, P_ALONG, Q_ALONG, VEC, F32_OUT>(g, stream);
}

template <bool P_ALONG, bool Q_ALONG, bool F32_OUT>
hipError_t launch_gemm(const Gemm& g, int io, bool big, hipStream_t stream) {
  const int pc = io == TM_IO_BF16 ? 8 : 4;
  const bool vec = g.p_row % pc == 0 && g.q_row % pc == 0;
  if (io == TM_IO_BF16)
    return vec ? launch_sized<P_ALONG, Q_ALONG, F32_OUT, true, true>(g, big, stream)
               : launch_sized<P_ALONG, Q_ALONG, F32_OUT, true, false>(g, big, stream);
  return vec ? launch_sized<P_ALONG, Q_ALONG, F32_OUT, false, true>(g, big, stream)
             : launch_sized<P_ALONG, Q_ALONG, F32_OUT, false, false>(g, big, stream);
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

// the weight's gradient: parts of the rows that together fill the device
int weight_parts(const ProjectionShape& s, bool* big) {
  *big = large(s.O, s.K, s.io) || (s.O >= 128 && s.K >= 128);
  const int64_t tr = *big ? (s.io == TM_IO_BF16 ? 256 : 128) : 64, tc = *big ? 128 : 64;
  const int64_t tiles = (s.O + tr - 1) / tr * ((s.K + tc - 1) / tc);
  int64_t parts = (512 + tiles - 1) / tiles, most = s.M / 256;   // a part has 256 rows at least
  if (parts > most) parts = most;
  return parts < 1 ? 1 : parts > 64 ? 64 : (int)parts;
}

int slope_parts(const ProjectionShape& s) {
  const int64_t pc = s.io == TM_IO_BF16 ? (s.O % 8 ? 1 : 8) : s.O % 4 ? 1 : 4;
  const int64_t cols = (s.O + 64 * pc - 1) / (64 * pc);
  int64_t parts = (1024 + cols - 1) / cols, most = (s.M + 15) / 16;
  if (parts > most) parts = most;
  return parts < 1 ? 1 : parts > 1024 ? 1024 : (int)parts;
}

int64_t round16(int64_t x) { return (x + 15) / 16 * 16; }
int64_t round_t(int64_t x) { return (x + kT - 1) / kT * kT; }

}  // namespace

bool projection_supported(const ProjectionShape& s) {
  const double m = (double)(s.M / 64 + 1), k = (double)(s.K / 64 + 1), o = (double)(s.O / 64 + 1);
  return m * o < (double)kMostBlocks && m * k < (double)kMostBlocks && o * k * 64 < (double)kMostBlocks;
}

hipError_t launch_projection(const ProjectionShape& s, const void* x, const void* weight, const float* bias,
                             const void* residual, void* out, void* pre, hipStream_t stream) {
  if (s.M == 0) return hipSuccess;
  Gemm g = {};
  g.P = weight, g.Q = x, g.p_row = g.q_row = s.K, g.R = s.M, g.C = s.O, g.T = s.K;
  g.per = round_t(s.K), g.parts = 1, g.bias = bias, g.residual = residual, g.out = out, g.pre = pre, g.silu = s.silu;
  if (s.M <= kNarrowRows) {
    const bool vec = s.K % (s.io == TM_IO_BF16 ? 8 : 4) == 0;
    if (s.io == TM_IO_BF16) return vec ? launch_narrow<true, true>(g, stream) : launch_narrow<true, false>(g, stream);
    return vec ? launch_narrow<false, true>(g, stream) : launch_narrow<false, false>(g, stream);
  }
  return launch_gemm<true, true, false>(g, s.io, large(s.M, s.O, s.io), stream);
}

// dz (where there is an activation), the weight's parts, the bias's sums
int64_t projection_backward_ws_bytes(const ProjectionShape& s) {
  bool big;
  const int parts = weight_parts(s, &big);
  return (s.silu ? round16(s.M * s.O * (s.io == TM_IO_BF16 ? 2 : 4)) : 0) +
         (parts > 1 ? round16((int64_t)parts * s.O * s.K * 4) : 0) + round16((int64_t)slope_parts(s) * s.O * 4);
}

hipError_t launch_projection_backward(const ProjectionShape& s, const void* x, const void* weight, const void* pre,
                                      const void* dout, void* dx, float* dweight, float* dbias, void* ws,
                                      hipStream_t stream) {
  const int64_t esz = s.io == TM_IO_BF16 ? 2 : 4;
  bool big;
  const int parts = weight_parts(s, &big), sparts = slope_parts(s);
  char* at = (char*)ws;
  void* dz = s.silu ? at : nullptr;
  if (s.silu) at += round16(s.M * s.O * esz);
  float* wparts = parts > 1 ? (float*)at : nullptr;
  if (wparts) at += round16((int64_t)parts * s.O * s.K * 4);
  float* bparts = (float*)at;
  const bool whole = s.O % (16 / esz) == 0;
  const int pc = whole ? (int)(16 / esz) : 1;
  const dim3 grid((s.O + 64 * pc - 1) / (64 * pc), sparts);
  const int64_t per = (s.M + sparts - 1) / sparts;
  auto slope = s.io == TM_IO_BF16 ? (whole ? slope_kernel<true, true> : slope_kernel<true, false>)
                                  : (whole ? slope_kernel<false, true> : slope_kernel<false, false>);
  slope<<<grid, 256, 0, stream>>>(dout, s.silu ? pre : nullptr, dz, sparts > 1 ? bparts : dbias, s.M, s.O, per);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const void* z = s.silu ? dz : dout;
  Gemm g = {};
  if (s.M > 0) {
    g.P = weight, g.Q = z, g.p_row = s.K, g.q_row = s.O, g.R = s.M, g.C = s.K, g.T = s.O, g.per = round_t(s.O);
    g.parts = 1, g.out = dx;
    err = launch_gemm<false, true, false>(g, s.io, large(s.M, s.K, s.io), stream);
    if (err != hipSuccess) return err;
  }
  g = Gemm();
  g.P = x, g.Q = z, g.p_row = s.K, g.q_row = s.O, g.R = s.O, g.C = s.K, g.T = s.M;
  g.parts = parts, g.per = round_t((s.M + parts - 1) / parts), g.out = parts > 1 ? wparts : dweight;
  err = launch_gemm<false, false, true>(g, s.io, big, stream);
  if (err != hipSuccess || (parts == 1 && sparts == 1)) return err;
  const int64_t n = (int64_t)s.O * s.K;
  const unsigned blocks = parts > 1 ? (unsigned)((n + 1023) / 1024) : 0;
  parts_kernel<<<blocks + (sparts > 1 ? (unsigned)((s.O + 15) / 16) : 0), 256, 0, stream>>>(
      wparts, parts, n, dweight, bparts, sparts, s.O, dbias, blocks);
  return hipGetLastError();
}

}  // namespace titans
