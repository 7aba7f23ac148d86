// Gradients through the gated delta memory (tm_delta_chunk.h has the forward
// chunk form: F the residuals, T = (I + B)^-1, P, G, E, D).
//
// With dW the adjoint of the state after a chunk and dY that of its outputs,
// and dE that of E = V - diag(G) K W^T (so dV = dE):
//
//   dF  = P^T dY + diag(E theta) K dW^T,   dE = T^T dF
//   dW' = G_C dW + dY^T diag(G) Q - dE^T diag(G) K      (before the chunk)
//   X[t,j] = D[t,j] dY_t.F_j (j <= t),   M[t,j] = -D[t,j] dE_t.F_j (j < t)
//   dQ  = diag(G) dY W + (X theta) K
//   dK  = (X theta)^T Q + ((M theta) + (M theta)^T) K - diag(G) dE W + diag(E theta) F dW
//   Z[t,j] = X (q_t.k_j) + M (k_t.k_j),   e_j = E_j k_j.(F_j dW)
//   dtheta_j = sum_t Z[t,j] + e_j
//   dalpha_t = -(1/a_t) (what passes token t's decay): the sum over rows
//     i >= t (a token, or the chunk's end) and columns before t (its start,
//     or a token j < t) of Z theta, with q_i.dq_i + k_i.dk_i of the terms
//     through W in the start's column, e theta in the end's row and
//     G_C <W, dW> in their corner.
//
// The last sum is taken over the rectangle itself, by suffix sums down the
// columns: as a difference of row and column sums it would cancel.  In it (and
// nowhere else) a = 0 (alpha = 1) is held as 2^-64, which leaves the quotient
// its limit; what passes two such tokens vanishes beside it.
//
// What is serial is W forwards and dW backwards, and neither needs the other:
// one launch sweeps both ways, each on chain and builder waves as the forward
// kernel has them, and leaves W and dW at every chunk's edges, F and dE.  A
// second launch takes every chunk of a key head by itself, with the value
// heads that share the key head in turn, so dQ and dK are sums in registers
// in a fixed order.
//
// 128 streams x 1024 tokens, d 64, bf16: 75 us for the sweeps (2.3 us a chunk,
// the chain's and builders' latencies: a third of the cycles issue vector
// instructions; 86 MB read and 203 MB written) and 110 us for the pieces (two
// workgroups a CU, again a third; 253 MB read and 52 MB written, half of a
// copy's rate).  The 594 MB alone would take 115 us at a copy's rate, the
// inputs and outputs 24: W and its adjoint at every chunk's edges are most of
// it.
#include "tm_delta_chunk.h"

namespace titans {
namespace {

constexpr float kForgetGrad = -64.f;

// Per (stream, chunk) in the workspace: W and dW [ld x ld] fp32, row-major,
// and F and dE as the chains' tiles, [ld / 16][64 lanes][8] fp32.
struct GradParams {
  const void *k, *v, *q, *dy;
  const float *alpha, *theta, *W_in, *dW_out;
  const int32_t* lengths;
  void *dk, *dv, *dq;
  float *dalpha, *dtheta, *dW_in;
  float *ws_W, *ws_dW, *ws_F, *ws_dE;
  int B, H, Hk, N, d, ld, chunks, parts;
};

template <int DP, bool F32, int CW>
using GradLds = ChunkLds<DP, F32 ? 3 : 1, CW * 16>;

// ---- the two sweeps: blocks of the first half forwards, of the second backwards ----
template <int DP, bool F32, int CW, int PB, int NB, int VB>
__global__ void __launch_bounds__((CW + PB * (F32 ? 2 : 1)) * 64) delta_sweep_kernel(GradParams p) {
  constexpr int NP = F32 ? 3 : 1;
  constexpr int NT = DP / 16, NK = DP / 32, kE = F32 ? 4 : 2;
  using Lds = GradLds<DP, F32, CW>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const Ring<Lds, CW, PB, NB, F32> ring{smem};
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int half = gridDim.x / 2;   // a multiple of 8
  const bool back = (int)blockIdx.x >= half;
  const int bid = back ? blockIdx.x - half : blockIdx.x, idx = bid >> 3;
  const int s = (idx / p.parts) * 8 + (bid & 7), part = idx % p.parts;
  if (s >= p.B * p.H) return;
  const int b = s / p.H, h = s % p.H, d = p.d;
  const int n = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
  const int chunks = chunks_of(n);
  ring.init(wave, lane);

  if (wave >= CW) {
    const int col0 = part * CW * 16;
    const int64_t krow = ((int64_t)b * p.Hk + h / (p.H / p.Hk)) * p.N * d, vrow = (int64_t)s * p.N * d + col0;
    const Rows in = {(const char*)p.k + krow * kE,   (const char*)p.q + krow * kE,  (const char*)(back ? p.dy : p.v) + vrow * kE,
                     p.alpha + (int64_t)s * p.N, p.theta + (int64_t)s * p.N, chunks, n, d, d - col0};
    if (back)
      run_builder<DP, F32, VB, CW * 16, true, true>(ring, wave, lane, in);
    else
      run_builder<DP, F32, VB, CW * 16, false, false>(ring, wave, lane, in);
    return;
  }

  const int cg = part * CW + wave, col = cg * 16 + li;
  const bool kept = cg * 16 < p.ld;   // a whole tile of columns, or none
  f32x4 S[NT];
  if (back && !p.dW_out) {
#pragma unroll
    for (int i = 0; i < NT; ++i) S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  } else {
    load_state<NT, VB>(S, back ? p.dW_out : p.W_in, s, col, d, g);
  }
  arrived(S);
  for (int i = 0; i < chunks; ++i) {
    const int c = back ? chunks - 1 - i : i;
    const int64_t at = (int64_t)s * p.chunks + c;
    float* state = (back ? p.ws_dW : p.ws_W) + (at * p.ld + col) * p.ld + 4 * g;
    f32x4* tiles = (f32x4*)((back ? p.ws_dE : p.ws_F) + ((at * (p.ld / 16) + cg) * 64 + lane) * 8);
    if (kept) {
#pragma unroll
      for (int ti = 0; ti < NT; ++ti)
        if (16 * ti < p.ld) *(f32x4*)(state + 16 * ti) = S[ti];
    }
    wait_for(ring.built() + i % PB, i + 1);
    const Lds L = ring.buffer(i);
    // (as in the forward kernel, LDS reads go out a product ahead of their use)
    f32x4 ks[2], V[2], G[2], E[2], X[2];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) ks[rt] = X[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    bf16x8 ka[NK][2][NP], vp[3];
#pragma unroll
    for (int kx = 0; kx < NK; ++kx) read2<NP>(L.k() + li * Lds::RS + 8 * g + 32 * kx, Lds::KP, 16 * Lds::RS, ka[kx]);
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        V[e >> 2][e & 3] = ((const float*)L.v())[(16 * (e >> 2) + 4 * g + (e & 3)) * Lds::VS + 16 * wave + li];
    } else {
      vp[0] = read_transposed<false>((const uint16_t*)L.v(), Lds::VS, 16 * wave, lane);
    }
    const float gc = L.gc()[0], scale = L.gc()[1];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      G[rt] = *(const f32x4*)(L.g() + 16 * rt + 4 * g);
      E[rt] = *(const f32x4*)(L.eth() + 16 * rt + 4 * g);
    }
    if (!F32) in_order();
#pragma unroll
    for (int kx = 0; kx < NK; ++kx) {
      bf16x8 sp[3];
      split8<3>(S[2 * kx], S[2 * kx + 1], sp);
      mul2<false, 3>(ka[kx], sp, ks);
    }
    if constexpr (!F32) {
      const u32x4 x = __builtin_bit_cast(u32x4, vp[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) V[e >> 2][e & 3] = e & 1 ? top(flt(x[e >> 1])) : flt(x[e >> 1] << 16);
    }
    // forwards: R = V - G K W^T, X = F = T R; backwards: R = dF, X = dE = T^T dF
    f32x4 R[2];
    bf16x8 ta[2][3], rp[3];
    if (!back) {
      read2<3>(L.t() + li * kCS + 8 * g, Lds::CP, 16 * kCS, ta);
      if (!F32) in_order();
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) R[rt] = V[rt] - G[rt] * ks[rt];
    } else {
      bf16x8 pt[2][3];
#pragma unroll
      for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) pt[rt][e] = read_transposed<true>(L.p() + e * Lds::CP, kCS, 16 * rt, lane);
#pragma unroll
      for (int e = 0; e < 3; ++e)
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) ta[rt][e] = read_transposed<true>(L.t() + e * Lds::CP, kCS, 16 * rt, lane);
      if (!F32) in_order();
      if constexpr (F32) {
        split8<3>(V[0], V[1], vp);
        mul2<false, 3>(pt, vp, X);
      } else {
        mul2<false, 1>(pt, vp, X);
      }
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        R[rt] = ks[rt] * E[rt] * scale + X[rt];
        X[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
    }
    split8<3>(R[0], R[1], rp);
    if (!F32) in_order();
    bf16x8 kt[NT][NP];
    auto read_rows = [&](const uint16_t* rows) {
#pragma unroll
      for (int ti = 0; ti < NT; ++ti)
#pragma unroll
        for (int e = 0; e < NP; ++e) kt[ti][e] = read_transposed<true>(rows + e * Lds::KP, Lds::RS, 16 * ti, lane);
    };
    // forwards: W' = G_C W + K^T (E theta F); backwards: dW' = G_C dW + Q^T (G dY) - K^T (G dE)
    f32x4 U[2], acc[NT];
    bf16x8 up[3];
    auto fold = [&] {
#pragma unroll
      for (int f = 0; f < products<NP, 3>(); ++f) {
        const Planes x = product<NP, 3>(f);
#pragma unroll
        for (int ti = 0; ti < NT; ++ti) acc[ti] = mfma(kt[ti][x.i], up[x.j], acc[ti]);
      }
    };
    const bool scaled = !back && __builtin_amdgcn_readfirstlane(bits(scale)) != 0x3f800000u;
#pragma unroll
    for (int ti = 0; ti < NT; ++ti) {
      const f32x4 x = S[ti] * gc;
      S[ti] = scaled ? x : f32x4{0.f, 0.f, 0.f, 0.f};
      acc[ti] = scaled ? f32x4{0.f, 0.f, 0.f, 0.f} : x;
    }
    if (back) {   // Q's part does not wait for dE
      read_rows(L.q());
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) U[rt] = V[rt] * G[rt];
      split8<3>(U[0], U[1], up);
      fold();
    }
    read_rows(L.k());
    mul2<false, 3>(ta, rp, X);
    if (kept) tiles[0] = X[0], tiles[1] = X[1];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) U[rt] = back ? X[rt] * -G[rt] : X[rt] * E[rt];
    split8<3>(U[0], U[1], up);
    fold();
    raise_to(ring.used() + wave, i + 1, lane);
#pragma unroll
    for (int ti = 0; ti < NT; ++ti) S[ti] = scaled ? S[ti] + acc[ti] * scale : acc[ti];
  }
  if (back) store_state<NT, VB>(S, p.dW_in, s, col, d, g);
}

// ---- a chunk of a key head ----
template <int DP, bool F32>
struct PieceLds {
  static constexpr int NP = F32 ? 3 : 1, RS = DP + 8, KP = kC * RS, CP = kC * kCS, FP = DP * kCS,
                       NW = DP / 16;
  static constexpr int K = 0, Q = K + NP * KP * 2, DY = Q + NP * KP * 2, F = DY + NP * KP * 2, DE = F + 3 * FP * 2,
                       X = DE + 3 * FP * 2, M = X + 3 * CP * 2, Z = M + 3 * CP * 2, GATES = Z + kC * kBS * 4,
                       DOTS = GATES + 9 * kC * 4, BYTES = DOTS + NW * (2 * kC + 1) * 4;
};

template <bool F32>
__device__ __forceinline__ void put(void* p, int64_t i, float x) {
  if (F32)
    ((float*)p)[i] = x;
  else
    ((__bf16*)p)[i] = (__bf16)x;
}

// four consecutive channels from c on at element `at`; VB 0: rows that may not be aligned, or end within the four
template <bool F32, int VB>
__device__ __forceinline__ void put_four(void* p, int64_t at, const f32x4& x, int c, int d) {
  if constexpr (VB > 0) {
    if (c >= d) return;
    if constexpr (F32)
      *(f32x4*)((float*)p + at + c) = x;
    else
      *(bf16x4*)((__bf16*)p + at + c) = __builtin_convertvector(x, bf16x4);
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (c + r < d) put<F32>(p, at + c + r, x[r]);
  }
}

// the values that NP planes (`plane` apart) of four neighbours stand for
template <int NP>
__device__ __forceinline__ f32x4 whole(const uint16_t* at, int plane) {
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = NP - 1; i >= 0; --i) {
    const uint2 u = *(const uint2*)(at + i * plane);
    sum += f32x4{flt(u.x << 16), top(flt(u.x)), flt(u.y << 16), top(flt(u.y))};
  }
  return sum;
}

// sum over the four lane groups, in every lane
__device__ __forceinline__ float groups_sum(float x) {
  x += __shfl_xor(x, 16, 64);
  return x + __shfl_xor(x, 32, 64);
}

// A wave has 16 channels of its own: of K's for dQ and dK (and, when staging,
// of V's).  Products of tokens by those channels are computed transposed, so
// that a lane has four neighbouring channels of one token.
template <int DP, bool F32, int VB>
__global__ void __launch_bounds__(DP * 4, 2) delta_piece_kernel(GradParams p) {
  using L = PieceLds<DP, F32>;
  constexpr int NP = L::NP, NW = L::NW, NK = DP / 32, RS = L::RS, KP = L::KP, CP = L::CP, FP = L::FP;
  constexpr int kE = F32 ? 4 : 2;
  // K, Q and dY are staged by blocks of kCols columns, kParts waves to a tensor, kRows blocks to a wave (blocks of 32
  // columns keep the wide rows in few registers: 284 us against 361 for 128 streams x 512, d 128, fp32)
  constexpr int kCols = DP == 64 && !F32 ? DP : 32, kParts = DP / kCols, kRows = (3 * kParts + NW - 1) / NW;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  uint16_t *Ks = (uint16_t*)(smem + L::K), *Qs = (uint16_t*)(smem + L::Q), *dYs = (uint16_t*)(smem + L::DY);
  uint16_t *Fs = (uint16_t*)(smem + L::F), *dEs = (uint16_t*)(smem + L::DE);   // [channel][token]
  uint16_t *Xs = (uint16_t*)(smem + L::X), *Ms = (uint16_t*)(smem + L::M);
  float *Z = (float*)(smem + L::Z), *gates = (float*)(smem + L::GATES), *dots = (float*)(smem + L::DOTS);
  // log2 G as float pairs, theta, G and E; the last four with a floored (what Z uses)
  float *gh = gates, *gl = gates + kC, *th = gates + 2 * kC, *Gt = gates + 3 * kC, *Et = gates + 4 * kC;
  float *zh = gates + 5 * kC, *zl = gates + 6 * kC, *Gz = gates + 7 * kC, *Ez = gates + 8 * kC;
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = blockIdx.x % p.chunks, bk = blockIdx.x / p.chunks, b = bk / p.Hk, hk = bk % p.Hk;
  const int share = p.H / p.Hk, d = p.d, t0 = c * kC;
  const int n = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
  const int live = min(max(n - t0, 0), kC), rows = min(kC, p.N - t0);   // tokens of the sequence, and of the tensors
  const int64_t krow = ((int64_t)bk * p.N + t0) * d;
  const int ch = 16 * w + li, ch4 = 16 * w + 4 * g;
  if (live == 0) {   // past the sequence: zeros
    const int64_t s0 = (int64_t)b * p.H + hk * share;
    for (int e = threadIdx.x; e < rows * d; e += NW * 64) {
      put<F32>(p.dk, krow + e, 0.f);
      put<F32>(p.dq, krow + e, 0.f);
      for (int x = 0; x < share; ++x) put<F32>(p.dv, ((s0 + x) * p.N + t0) * d + e, 0.f);
    }
    if ((int)threadIdx.x < rows)
      for (int x = 0; x < share; ++x) p.dalpha[(s0 + x) * p.N + t0 + threadIdx.x] = p.dtheta[(s0 + x) * p.N + t0 + threadIdx.x] = 0.f;
    return;
  }
  const bool tile = 16 * w < p.ld;
  float la_z = 0.f;   // the last wave's lane t: log2 a_t, floored
  f32x4 dq[2], dk[2];
#pragma unroll
  for (int rt = 0; rt < 2; ++rt) dq[rt] = dk[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int x = 0; x < share; ++x) {
    const int s = b * p.H + hk * share + x;
    const int64_t at = (int64_t)s * p.chunks + c;
    // what a wave reads is on its way before any of it is staged: its rows
    // (blocks of K and Q, once, and of dY), its tiles of F and dE, and W and
    // dW as operands over their rows with the wave's channels as columns
    const char* src[3] = {(const char*)p.k + krow * kE, (const char*)p.q + krow * kE,
                          (const char*)p.dy + ((int64_t)s * p.N + t0) * d * kE};
    const int col0 = w % kParts * kCols;
    RowLoad<DP, kCols, F32, VB> row[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int which = w / kParts + i * (NW / kParts);
      if (which < 3 && (which == 2 || x == 0) && col0 < d)
        row[i].load(src[which] + col0 * kE, live, d, d - col0, lane);
    }
    f32x4 f[2], e[2], Wf[NK][2], dWf[NK][2];
    {
      const int64_t o = ((at * (p.ld / 16) + (tile ? w : 0)) * 64 + lane) * 8;
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        f[rt] = ((const f32x4*)(p.ws_F + o))[rt];
        e[rt] = ((const f32x4*)(p.ws_dE + o))[rt];
      }
    }
    // (uniform row addresses and one offset a lane)
    const float *W = p.ws_W + at * p.ld * p.ld, *dW = p.ws_dW + at * p.ld * p.ld;
    const uint32_t lane_off = 4 * g * p.ld + (tile ? ch : li);
#pragma unroll
    for (int kx = 0; kx < NK; ++kx)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 32 * kx + 16 * (i >> 2), at_row = (r < p.ld ? r + (i & 3) : i & 3) * p.ld;
        Wf[kx][i >> 2][i & 3] = (W + at_row)[lane_off];
        dWf[kx][i >> 2][i & 3] = (dW + at_row)[lane_off];
      }
    if (x > 0) __syncthreads();   // the last head's LDS is done with
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      const int which = w / kParts + i * (NW / kParts);
      if (which >= 3 || (which < 2 && x > 0)) continue;
      uint16_t* to = which == 0 ? Ks : which == 1 ? Qs : dYs;
      if (col0 < d) {
        store_planes<DP, F32>(row[i], to, lane, col0);
      } else {   // columns past d: zeros
        for (int e = lane; e < NP * kC * kCols / 4; e += 64)
          *(uint2*)(to + e / (kC * kCols / 4) * KP + e / (kCols / 4) % kC * RS + col0 + e % (kCols / 4) * 4) = make_uint2(0, 0);
      }
    }
    if (w == NW - 1) {
      const int64_t gt = (int64_t)s * p.N + t0 + min(lane, live - 1);
      const bool in = lane < live;
      const float la = in ? log2_keep(p.alpha[gt]) : 0.f, theta = in ? p.theta[gt] : 0.f;
      la_z = la < kForgetGrad ? kForgetGrad : la;
      double all, all_z;
      const double sum = prefix_sums(la, lane, all), sum_z = prefix_sums(la_z, lane, all_z);
      const float hi = (float)sum, hi_z = (float)sum_z;
      if (lane < kC) {
        gh[lane] = hi;
        gl[lane] = (float)(sum - (double)hi);
        th[lane] = theta;
        Gt[lane] = exp2_of(hi);
        Et[lane] = exp2_of((float)(all - sum));
        zh[lane] = hi_z;
        zl[lane] = (float)(sum_z - (double)hi_z);
        Gz[lane] = exp2_of(hi_z);
        Ez[lane] = exp2_of((float)(all_z - sum_z));
      }
      // X's upper right block
#pragma unroll
      for (int i = 0; i < 3; ++i) *(uint2*)(Xs + i * CP + li * kCS + 8 * g + 4) = make_uint2(0, 0);
    }
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) {
      if (!tile) f[rt] = e[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
      put4<3>(Fs + ch * kCS + 8 * g + 4 * rt, FP, f[rt][0], f[rt][1], f[rt][2], f[rt][3]);
      put4<3>(dEs + ch * kCS + 8 * g + 4 * rt, FP, e[rt][0], e[rt][1], e[rt][2], e[rt][3]);
    }
#pragma unroll
    for (int kx = 0; kx < NK; ++kx)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (!tile || 32 * kx + 16 * i >= p.ld) Wf[kx][i] = dWf[kx][i] = f32x4{0.f, 0.f, 0.f, 0.f};
    __syncthreads();
    // X, M and Z by tiles, transposed (rows j, columns t): wave 0 (t 0, j 0), 1 (t 1, j 0), 2 (t 1, j 1)
    if (w < 3) {
      const int tt = w > 0, jt = w > 1, t = 16 * tt + li, j0 = 16 * jt + 4 * g;
      f32x4 xx = {0.f, 0.f, 0.f, 0.f}, mm = xx, kk = xx, qk = xx;
#pragma unroll
      for (int kx = 0; kx < NK; ++kx) {
        asm volatile("" : "+v"(xx), "+v"(mm), "+v"(kk), "+v"(qk) : : "memory");
        bf16x8 fo[3], eo[3], y[NP], kj[NP], kt[NP], qt[NP];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          fo[i] = read_transposed<true>(Fs + i * FP + 32 * kx * kCS, kCS, 16 * jt, lane);
          eo[i] = read_transposed<true>(dEs + i * FP + 32 * kx * kCS, kCS, 16 * tt, lane);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          const int o = i * KP + li * RS + 32 * kx + 8 * g;
          y[i] = *(const bf16x8*)(dYs + o + 16 * tt * RS);
          kj[i] = *(const bf16x8*)(Ks + o + 16 * jt * RS);
          kt[i] = *(const bf16x8*)(Ks + o + 16 * tt * RS);
          qt[i] = *(const bf16x8*)(Qs + o + 16 * tt * RS);
        }
#pragma unroll
        for (int o = 2; o >= 0; --o)
#pragma unroll
          for (int i = o; i >= 0; --i) {
            if (o - i < NP) xx = mfma(fo[i], y[o - i], xx);
            mm = mfma(fo[i], eo[o - i], mm);
            if (i < NP && o - i < NP) {
              kk = mfma(kj[i], kt[o - i], kk);
              qk = mfma(kj[i], qt[o - i], qk);
            }
          }
      }
      const float tg = gh[t], tl = gl[t], tg_z = zh[t], tl_z = zl[t];
      f32x4 z;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = j0 + r;
        // (above the diagonal the powers may be infinite: they are dropped, not multiplied by 0)
        const float D = t < j ? 0.f : exp2_of((tg - gh[j]) + (tl - gl[j])) * th[j];
        const float Dz = t < j ? 0.f : exp2_of((tg_z - zh[j]) + (tl_z - zl[j]));
        if (t == j) mm[r] = 0.f;
        z[r] = Dz * (xx[r] * qk[r] - mm[r] * kk[r]);
        xx[r] *= D;
        mm[r] *= -D;
      }
      *(f32x4*)(Z + t * kBS + j0) = z;
      put4<3>(Xs + t * kCS + 8 * g + 4 * jt, CP, xx[0], xx[1], xx[2], xx[3]);
      // M and its transpose; the zeros of a diagonal tile's upper half are the transpose's places
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int j = j0 + r;
        float v = mm[r];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const uint16_t u = (uint16_t)(bits(v) >> 16);
          v -= top(v);
          if (t >= j) Ms[i * CP + t * kCS + perm32(j)] = u;
          if (t > j) Ms[i * CP + j * kCS + perm32(t)] = u;
        }
      }
    }
    // what goes through W and dW, and its dots with q and k
    {
      f32x4 a[2], m[2], u[2];
      float corner = 0.f;
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) a[rt] = m[rt] = u[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kx = 0; kx < NK; ++kx) {
        // (tied to the sums: the reads of later steps stay behind, and in registers)
        asm volatile("" : "+v"(a[0]), "+v"(m[0]), "+v"(u[0]) : : "memory");
        bf16x8 wp[3], y[2][NP], o[2][3];
        split8<3>(Wf[kx][0], Wf[kx][1], wp);
        read2<NP>(dYs + li * RS + 32 * kx + 8 * g, KP, 16 * RS, y);
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) o[rt][i] = read_transposed<true>(dEs + i * FP + 32 * kx * kCS, kCS, 16 * rt, lane);
        mul2<true, 3>(y, wp, a);
        mul2<true, 3>(o, wp, m);
        split8<3>(dWf[kx][0], dWf[kx][1], wp);
#pragma unroll
        for (int i = 0; i < 3; ++i)
#pragma unroll
          for (int rt = 0; rt < 2; ++rt) o[rt][i] = read_transposed<true>(Fs + i * FP + 32 * kx * kCS, kCS, 16 * rt, lane);
        mul2<true, 3>(o, wp, u);
#pragma unroll
        for (int i = 0; i < 8; ++i) corner = fmaf(Wf[kx][i >> 2][i & 3], dWf[kx][i >> 2][i & 3], corner);
      }
      const int pos = (ch4 & ~31) + perm32(ch4 & 31);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        const int t = 16 * rt + li;
        const f32x4 kv = whole<NP>(Ks + t * RS + pos, KP), qv = whole<NP>(Qs + t * RS + pos, KP);
        float start = 0.f, end = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          start = fmaf(qv[r], a[rt][r], fmaf(-kv[r], m[rt][r], start));
          end = fmaf(kv[r], u[rt][r], end);
        }
        start = groups_sum(start) * Gz[t];
        end = groups_sum(end) * Ez[t];
        if (g == 0) dots[w * 2 * kC + t] = start, dots[(w * 2 + 1) * kC + t] = end;
        dq[rt] += a[rt] * Gt[t];
        dk[rt] += u[rt] * (Et[t] * th[t]) - m[rt] * Gt[t];
        // dV, from dE's planes
        const uint16_t* from = dEs + (ch4 + (li >> 2)) * kCS;
        f32x4 dv = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 2; i >= 0; --i) {
          typedef __attribute__((address_space(3))) bf16x4 lds4;
          const bf16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds4*)(from + i * FP + perm32(16 * rt + 4 * (li & 3))));
          dv += __builtin_convertvector(v, f32x4);
        }
        if (t < rows) put_four<F32, VB>(p.dv, ((int64_t)s * p.N + t0 + t) * d, t < live ? dv : f32x4{0.f, 0.f, 0.f, 0.f}, ch4, d);
      }
#pragma unroll
      for (int i = 1; i < 64; i *= 2) corner += __shfl_xor(corner, i, 64);
      if (lane == 0) dots[NW * 2 * kC + w] = corner;
    }
    __syncthreads();
    // through the chunk's own tokens
    {
      bf16x8 xr[2][3], xt[2][3], mr[2][3], kT[NP], qT[NP];
      read2<3>(Xs + li * kCS + 8 * g, CP, 16 * kCS, xr);
      read2<3>(Ms + li * kCS + 8 * g, CP, 16 * kCS, mr);
#pragma unroll
      for (int i = 0; i < 3; ++i)
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) xt[rt][i] = read_transposed<true>(Xs + i * CP, kCS, 16 * rt, lane);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        kT[i] = read_transposed<true>(Ks + i * KP, RS, 16 * w, lane);
        qT[i] = read_transposed<true>(Qs + i * KP, RS, 16 * w, lane);
      }
      mul2<true, NP>(xr, kT, dq);
      mul2<true, NP>(xt, qT, dk);
      mul2<true, NP>(mr, kT, dk);
    }
    // the gates: lane j < 32 sums column j of Z theta up from the end's row, lane 32 the start's column
    if (w == NW - 1) {
      const float tj = lane < kC ? th[lane] : 1.f;
      float end = 0.f, start = 0.f, corner = 0.f;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        start += dots[i * 2 * kC + (lane & 31)];
        end += dots[(i * 2 + 1) * kC + (lane & 31)];
        corner += dots[NW * 2 * kC + i];
      }
      if (lane < kC) Z[lane * kBS + kC] = start;
      wave_fence();
      const int col = min(lane, kC);
      float z[kC], dtheta = 0.f, sum = lane < kC ? end * tj : corner * Gz[kC - 1];
#pragma unroll
      for (int i = 0; i < kC; ++i) z[i] = Z[i * kBS + col];
      wave_fence();
#pragma unroll
      for (int i = kC - 1; i >= 0; --i) {
        const float v = lane >= kC || i >= lane ? z[i] : 0.f;   // (above the diagonal nothing was written)
        dtheta += v;
        sum = fmaf(v, tj, sum);
        if (lane <= kC) Z[i * kBS + col] = sum;
      }
      wave_fence();
      const int t = lane & 31;
      float through = Z[t * kBS + kC];
#pragma unroll
      for (int j = 0; j < kC; ++j) {
        const float v = Z[t * kBS + j];
        through += j < t ? v : 0.f;
      }
      if (lane < rows) {
        const int64_t gt = (int64_t)s * p.N + t0 + lane;
        p.dtheta[gt] = lane < live ? dtheta + end : 0.f;
        p.dalpha[gt] = lane < live ? -through * exp2_of(-la_z) : 0.f;
      }
    }
  }
#pragma unroll
  for (int rt = 0; rt < 2; ++rt) {
    const int t = 16 * rt + li;
    if (t >= rows) continue;
    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
    put_four<F32, VB>(p.dq, krow + (int64_t)t * d, t < live ? dq[rt] : none, ch4, d);
    put_four<F32, VB>(p.dk, krow + (int64_t)t * d, t < live ? dk[rt] : none, ch4, d);
  }
}

template <int DP, bool F32, int CW, int VB>
hipError_t launch_sweep(GradParams p, hipStream_t stream) {
  // (two workgroups of 2 chain waves share a CU where LDS allows)
  constexpr int NB = F32 ? (DP == 64 ? 3 : 2) : DP == 64 && CW == 2 ? 3 : 4,
                PB = F32 ? (DP == 64 ? 2 : 1) : DP == 64 && CW == 4 ? 3 : 2;
  using R = Ring<GradLds<DP, F32, CW>, CW, PB, NB, F32>;
  static_assert(R::BYTES <= 160 * 1024, "LDS of one workgroup");
  p.parts = ((p.d + 15) / 16 + CW - 1) / CW;
  auto sweep = delta_sweep_kernel<DP, F32, CW, PB, NB, VB>;
  hipError_t err = hipFuncSetAttribute((const void*)sweep, hipFuncAttributeMaxDynamicSharedMemorySize, R::BYTES);
  if (err != hipSuccess) return err;
  const unsigned half = (unsigned)((p.B * p.H + 7) / 8 * 8 * p.parts);
  sweep<<<2 * half, R::WAVES * 64, R::BYTES, stream>>>(p);
  return hipGetLastError();
}

// Four chain waves in a workgroup share the builders' work, two take less time
// a chunk: four where there are more workgroups of two than CUs.  Whole calls
// with two and with four, in us, 512 tokens of the most streams that take two
// and of the next that were tried:
//   bf16  d 64   64: 64 66     96: 81 78      fp32  d 64   64: 100 109   96: 148 134
//         d 80   32: 70 74     64: 120 102          d 80   32: 121 138   64: 217 181
//         d 96   32: 72 76     64: 125 106          d 96   32: 119 136   64: 216 183
//         d 128  32: 94 96     64: 165 147          d 128  32: 151 175   64: 282 241
template <int DP, bool F32, int VB>
hipError_t launch_grad(GradParams p, hipStream_t stream) {
  constexpr int kCus = 256, piece = PieceLds<DP, F32>::BYTES;
  static_assert(piece <= 160 * 1024, "LDS of one workgroup");
  const int groups = (p.d + 15) / 16;
  hipError_t err = 2 * p.B * p.H * ((groups + 1) / 2) > kCus ? launch_sweep<DP, F32, 4, VB>(p, stream)
                                                             : launch_sweep<DP, F32, 2, VB>(p, stream);
  if (err != hipSuccess || p.chunks == 0) return err;
  auto pieces = delta_piece_kernel<DP, F32, VB>;
  err = hipFuncSetAttribute((const void*)pieces, hipFuncAttributeMaxDynamicSharedMemorySize, piece);
  if (err != hipSuccess) return err;
  pieces<<<(unsigned)(p.B * p.Hk * p.chunks), DP * 4, piece, stream>>>(p);
  return hipGetLastError();
}

// (128 streams x 512 x 96: 355 us in fp32 and 201 in bf16, padded to 128 444
// and 253)
template <bool F32, int VB>
hipError_t launch_width(const GradParams& p, hipStream_t stream) {
  if (p.d <= 64) return launch_grad<64, F32, VB>(p, stream);
  return p.d <= 96 ? launch_grad<96, F32, VB>(p, stream) : launch_grad<128, F32, VB>(p, stream);
}

int64_t state_floats(const DeltaShape& s) {
  const int64_t ld = (s.d + 15) / 16 * 16;
  return (int64_t)s.B * s.H * chunks_of(s.N) * ld * ld;
}
int64_t tile_floats(const DeltaShape& s) {
  const int64_t ld = (s.d + 15) / 16 * 16;
  return (int64_t)s.B * s.H * chunks_of(s.N) * kC * ld;
}

}  // namespace

bool delta_backward_supported(const DeltaShape& s) {
  // the pieces' launch: a workgroup a chunk, and fewer than 2^32 threads
  return (int64_t)s.B * s.Hk * chunks_of(s.N) * (s.d <= 64 ? 256 : 512) < (int64_t)1 << 32;
}

int64_t delta_backward_ws_bytes(const DeltaShape& s) { return 8 * (state_floats(s) + tile_floats(s)); }

hipError_t launch_delta_backward(const DeltaShape& s, const void* k, const void* v, const void* q, const float* alpha,
                                 const float* theta, const int32_t* lengths, const float* W_in, const void* dy,
                                 const float* dW_out, void* dk, void* dv, void* dq, float* dalpha, float* dtheta,
                                 float* dW_in, float* ws, hipStream_t stream) {
  GradParams p = {k, v, q, dy, alpha, theta, W_in, dW_out, lengths, dk, dv, dq, dalpha, dtheta, dW_in};
  p.ws_W = ws, p.ws_dW = ws + state_floats(s);
  p.ws_F = ws + 2 * state_floats(s), p.ws_dE = p.ws_F + tile_floats(s);
  p.B = s.B, p.H = s.H, p.Hk = s.Hk, p.N = s.N, p.d = s.d, p.ld = (s.d + 15) / 16 * 16;
  p.chunks = chunks_of(s.N);
  if (s.io == TM_IO_BF16) {
    if (s.d % 8 == 0) return launch_width<false, 16>(p, stream);
    return s.d % 4 == 0 ? launch_width<false, 8>(p, stream) : launch_width<false, 0>(p, stream);
  }
  return s.d % 4 == 0 ? launch_width<true, 16>(p, stream) : launch_width<true, 0>(p, stream);
}

}  // namespace titans
