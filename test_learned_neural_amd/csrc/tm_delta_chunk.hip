// The gated delta memory over sequences, by chunks of 32 tokens on the matrix
// cores (the chunk form and its precision: tm_delta_chunk.h).
//
// What is serial is W alone, and a column of W^T (a value channel) meets no
// other.  So a "chain" wave owns 16 value channels of a stream for the whole
// sequence: W^T's [d x 16] slice stays in its accumulators, and every product
// of a chunk (K W^T, T R, P F, K^T U) has those accumulators' tiles as the
// operand in place, so the chain needs no exchange, no transposition and no
// barrier of its own.  What is not serial (K K^T, Q K^T, the decays, the
// triangular inverse, the bf16 planes) "builder" waves of the same workgroup
// prepare in LDS, PW chunks ahead of the chain, with the loads of the chunks
// after those in flight in their registers; one barrier every PW chunks.
// Nothing but the inputs and outputs touches memory.
#include "tm_delta_chunk.h"

namespace titans {
namespace {

struct ChainParams {
  const void *k, *v, *q;
  const float *alpha, *theta, *W_in;
  const int32_t* lengths;
  void* y;
  float* W_out;
  int streams, H, Hk, N, d, parts;
};

template <int DP, bool F32, int CW, int PW, int VB>
__global__ void __launch_bounds__((CW + PW) * 64) delta_chain_kernel(ChainParams p) {
  constexpr int NP = F32 ? 3 : 1, NPP = F32 ? 3 : 2, NS = F32 ? 3 : 2;   // planes: inputs, P, and W and F for y
  constexpr int NT = DP / 16, NK = DP / 32, kE = F32 ? 4 : 2;
  using Lds = ChunkLds<DP, NP, NPP>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the parts of a stream read the same K and Q: workgroups 8 apart share an XCD's L2
  const int idx = blockIdx.x >> 3;
  const int s = (idx / p.parts) * 8 + (blockIdx.x & 7), part = idx % p.parts;
  if (s >= p.streams) return;
  const int b = s / p.H, h = s % p.H, d = p.d;
  const int n = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
  const int chunks = (n + kC - 1) / kC, steps = (chunks + PW - 1) / PW;

  if (wave >= CW) {
    // ---- builder ----
    const int pw = wave - CW;
    const int64_t krow = ((int64_t)b * p.Hk + h / (p.H / p.Hk)) * p.N;
    const float *alpha = p.alpha + (int64_t)s * p.N, *theta = p.theta + (int64_t)s * p.N;
    for (int i = 0; i < 2; ++i) {   // T's block that stays zero
      Lds L{smem + (i * PW + pw) * Lds::BYTES};
      for (int x = 0; x < 3; ++x) *(uint2*)(L.t() + x * Lds::CP + li * kCS + 8 * g + 4) = make_uint2(0, 0);
    }
    RowLoad<DP, F32, VB> kr, qr;
    float al = 0.f, th = 0.f;
    auto fetch = [&](int c) {
      const int t0 = c * kC, m = min(kC, n - t0);
      if (m <= 0) return;
      kr.load((const char*)p.k + (krow + t0) * d * kE, m, d, lane);
      qr.load((const char*)p.q + (krow + t0) * d * kE, m, d, lane);
      al = lane < m ? alpha[t0 + lane] : 0.f;
      th = lane < m ? theta[t0 + lane] : 0.f;
    };
    fetch(pw);
    for (int i = 0; i <= steps; ++i) {
      const int c = i * PW + pw;
      if (c < chunks) {
        Lds L{smem + ((i & 1) * PW + pw) * Lds::BYTES};
        kr.store(L.k(), lane);
        qr.store(L.q(), lane);
        const float la = log2_keep(al), th0 = th;
        fetch(c + PW);
        wave_fence();
        build_chunk<DP, NP, NPP>(L, la, th0, lane);
      }
      __syncthreads();
    }
    return;
  }

  // ---- chain ----
  const int col = (part * CW + wave) * 16 + li;   // this lane's value channel
  const bool live = col < d;
  const float* W_in = p.W_in + (int64_t)s * d * d + (int64_t)col * d;
  f32x4 S[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int c = 16 * i + 4 * g;
    S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (VB) {
      if (live && c < d) S[i] = *(const f32x4*)(W_in + c);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool in = live && c + r < d;
        const float w = p.W_in[in ? (int64_t)s * d * d + col * d + c + r : 0];
        S[i][r] = in ? w : 0.f;
      }
    }
  }
  // v and y: a uniform address per chunk and this lane's offsets within it
  const char* vsrc = (const char*)p.v + (int64_t)s * p.N * d * kE;
  char* ydst = (char*)p.y + (int64_t)s * p.N * d * kE;
  uint32_t off[8];
#pragma unroll
  for (int r = 0; r < 8; ++r) off[r] = ((16 * (r >> 2) + 4 * g + (r & 3)) * d + min(col, d - 1)) * kE;
  uint32_t vr[PW][8];
  // Rows past the end read the last token's v: their K, theta and so their
  // effect is zero.
  auto fetch_v = [&](int step) {
#pragma unroll
    for (int x = 0; x < PW; ++x) {
      const int t0 = (step * PW + x) * kC;
      if (t0 >= n) return;
      const char* at = vsrc + (int64_t)t0 * d * kE;
      auto take = [&](uint32_t o) { return F32 ? *(const uint32_t*)(at + o) : *(const uint16_t*)(at + o); };
      if (t0 + kC <= n) {
#pragma unroll
        for (int r = 0; r < 8; ++r) vr[x][r] = take(off[r]);
      } else {
#pragma unroll
        for (int r = 0; r < 8; ++r)
          vr[x][r] = take((uint32_t)(min(16 * (r >> 2) + 4 * g + (r & 3), n - 1 - t0) * d + min(col, d - 1)) * kE);
      }
    }
  };
  if (n > 0) fetch_v(0);
  __syncthreads();
  for (int i = 0; i < steps; ++i) {
    float v[PW][8];
#pragma unroll
    for (int x = 0; x < PW; ++x)
#pragma unroll
      for (int r = 0; r < 8; ++r) v[x][r] = flt(F32 ? vr[x][r] : vr[x][r] << 16);
    fetch_v(i + 1);
#pragma unroll
    for (int x = 0; x < PW; ++x) {
      const int t0 = (i * PW + x) * kC;
      if (t0 >= n) break;
      const Lds L{smem + ((i & 1) * PW + x) * Lds::BYTES};
      const uint16_t *ka = L.k() + li * Lds::RS + 8 * g, *qa = L.q() + li * Lds::RS + 8 * g;
      const uint16_t *ta = L.t() + li * kCS + 8 * g, *pa = L.p() + li * kCS + 8 * g;
      f32x4 ks[2], qs[2];
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) ks[rt] = qs[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int kx = 0; kx < NK; ++kx) {
        bf16x8 sp[3];
        split8<3>(S[2 * kx], S[2 * kx + 1], sp);
        mul2<NP, 3>(ka + 32 * kx, Lds::KP, 16 * Lds::RS, sp, ks);
        bf16x8 sq[NS];
#pragma unroll
        for (int e = 0; e < NS; ++e) sq[e] = sp[e];
        mul2<NP, NS>(qa + 32 * kx, Lds::KP, 16 * Lds::RS, sq, qs);
      }
      f32x4 G[2], E[2], R[2], F[2];
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) {
        G[rt] = *(const f32x4*)(L.g() + 16 * rt + 4 * g);
        E[rt] = *(const f32x4*)(L.eth() + 16 * rt + 4 * g);
#pragma unroll
        for (int r = 0; r < 4; ++r) R[rt][r] = fmaf(-G[rt][r], ks[rt][r], v[x][4 * rt + r]);
        F[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      bf16x8 rp[3];
      split8<3>(R[0], R[1], rp);
      mul2<3, 3>(ta, Lds::CP, 16 * kCS, rp, F);
      // W' = G_C W + K^T (E theta F)
      {
        f32x4 U[2];
#pragma unroll
        for (int rt = 0; rt < 2; ++rt) U[rt] = F[rt] * E[rt];
        bf16x8 up[3];
        split8<3>(U[0], U[1], up);
        const float gc = L.gc()[0], scale = L.gc()[1];
        const bool scaled = __builtin_amdgcn_readfirstlane(bits(scale)) != 0x3f800000u;
        f32x4 acc[NT];
#pragma unroll
        for (int ti = 0; ti < NT; ++ti) acc[ti] = S[ti] * gc;
        if (scaled) {   // seldom: theta far from 1 all over the chunk
#pragma unroll
          for (int ti = 0; ti < NT; ++ti) S[ti] = acc[ti], acc[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        bf16x8 kt[NT][NP];
#pragma unroll
        for (int ti = 0; ti < NT; ++ti)
#pragma unroll
          for (int e = 0; e < NP; ++e) kt[ti][e] = read_transposed(L.k() + e * Lds::KP, Lds::RS, 16 * ti, lane);
#pragma unroll
        for (int o = 2; o >= 0; --o)
#pragma unroll
          for (int e = NP - 1; e >= 0; --e)
            if (o - e >= 0) {
#pragma unroll
              for (int ti = 0; ti < NT; ++ti) acc[ti] = mfma(kt[ti][e], up[o - e], acc[ti]);
            }
        if (scaled) {
#pragma unroll
          for (int ti = 0; ti < NT; ++ti) S[ti] += acc[ti] * scale;
        } else {
#pragma unroll
          for (int ti = 0; ti < NT; ++ti) S[ti] = acc[ti];
        }
      }
      // Y = diag(G) Q W^T + P F
      f32x4 out[2];
      bf16x8 fp[NS];
      split8<NS>(F[0], F[1], fp);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) out[rt] = G[rt] * qs[rt];
      mul2<NPP, NS>(pa, Lds::CP, 16 * kCS, fp, out);
      char* at = ydst + (int64_t)t0 * d * kE;
      auto store = [&](int e) {
        if (F32)
          *(float*)(at + off[e]) = out[e >> 2][e & 3];
        else
          *(uint16_t*)(at + off[e]) = __builtin_bit_cast(uint16_t, (__bf16)out[e >> 2][e & 3]);
      };
      if (t0 + kC <= n) {   // a whole chunk: one branch
        if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) store(e);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (live && t0 + 16 * (e >> 2) + 4 * g + (e & 3) < n) store(e);
      }
    }
    __syncthreads();
  }
  if (!live) return;
  float* W_out = p.W_out + (int64_t)s * d * d + (int64_t)col * d;
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    const int c = 16 * i + 4 * g;
    if (VB) {
      if (c < d) *(f32x4*)(W_out + c) = S[i];
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (c + r < d) W_out[c + r] = S[i][r];
    }
  }
}

template <int DP, bool F32, int CW, int PW, int VB>
hipError_t launch_as(ChainParams p, hipStream_t stream) {
  constexpr int lds = 2 * PW * ChunkLds<DP, F32 ? 3 : 1, F32 ? 3 : 2>::BYTES;
  static_assert(lds <= 160 * 1024, "LDS of one workgroup");
  p.parts = ((p.d + 15) / 16 + CW - 1) / CW;
  auto kernel = delta_chain_kernel<DP, F32, CW, PW, VB>;
  hipError_t err = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (err != hipSuccess) return err;
  const unsigned grid = (unsigned)((p.streams + 7) / 8 * 8 * p.parts);
  kernel<<<grid, (CW + PW) * 64, lds, stream>>>(p);
  return hipGetLastError();
}

template <int DP, bool F32, int VB>
hipError_t launch_chain(const ChainParams& p, hipStream_t stream) {
  constexpr int PW = F32 ? 1 : 2;
  if (p.streams >= 256) return launch_as<DP, F32, 4, PW, VB>(p, stream);
  return launch_as<DP, F32, 2, PW, VB>(p, stream);
}

template <bool F32, int VB>
hipError_t launch_width(const ChainParams& p, hipStream_t stream) {
  return p.d <= 64 ? launch_chain<64, F32, VB>(p, stream) : launch_chain<128, F32, VB>(p, stream);
}

}  // namespace

hipError_t launch_delta_chunked(const DeltaShape& s, const void* k, const void* v, const void* q, const float* alpha,
                                const float* theta, const int32_t* lengths, const float* W_in, void* y, float* W_out,
                                hipStream_t stream) {
  const ChainParams p = {k, v, q, alpha, theta, W_in, lengths, y, W_out, s.B * s.H, s.H, s.Hk, s.N, s.d, 0};
  if (s.io == TM_IO_BF16) {
    if (s.d % 8 == 0) return launch_width<false, 16>(p, stream);
    return s.d % 4 == 0 ? launch_width<false, 8>(p, stream) : launch_width<false, 0>(p, stream);
  }
  return s.d % 4 == 0 ? launch_width<true, 16>(p, stream) : launch_width<true, 0>(p, stream);
}

}  // namespace titans
