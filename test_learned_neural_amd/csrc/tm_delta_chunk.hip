// The gated delta memory over sequences, by chunks of 32 tokens on the matrix
// cores (the chunk form and its precision: tm_delta_chunk.h).
//
// What is serial is W alone, and a column of W^T (a value channel) meets no
// other.  So a "chain" wave owns 16 value channels of a stream for the whole
// sequence: W^T's [d x 16] slice stays in its accumulators, and every product
// of a chunk (K W^T, T R, P F, K^T U) has those accumulators' tiles as the
// operand in place, so the chain needs no exchange and no transposition.
// What is not serial (the loads of K, Q and V, K K^T, Q K^T, the decays, the
// triangular inverse, the bf16 planes) "builder" waves of the same workgroup
// prepare in a ring of NB chunk buffers in LDS, PB chunks at once, with the
// loads of the chunks after those in flight in their registers.  The waves
// meet through counters in LDS: a builder's last finished chunk, a chain
// wave's, and for fp32 inputs that of a builder's helper (Q and V).  All waves
// of a workgroup are resident, a builder and its helper wait only for chunks
// built before their own to be consumed and a chain wave only for the next
// chunk, so every wait ends.  Nothing but the inputs and outputs
// touches memory.
//
// Measured at 128 streams x 16384 tokens, d 64, bf16: 721 us, 1.41 us a chunk
// against a serial path of 320 vector and 60 matrix instructions (2250 cycles
// of issue, 0.94 us); the inputs and outputs alone would take 210 us at a
// copy's rate.  y from two planes of W, F and P instead of three took 682 us,
// and was off by 2^-17 of the largest term.
//
// Few streams and many chunks: the sequence is cut into segments.  A segment
// maps the state before it to the one after it by W -> W Phi + W_0; a first
// launch finds every segment's Phi and W_0 at once (the chain run on the unit
// vectors without values, and on the values from a zero state), a second
// passes the state through them in order (delta_join_kernel), a third runs
// the segments side by side from their true starts.  That is about 2.4 times
// the work, for as many times the parallelism as there are segments: 16
// streams x 65536 tokens take 511 us so and 2810 in one piece.  (Rows whose
// maps overflow are run in one piece: delta_join_kernel.)
#include "tm_delta_chunk.h"

namespace titans {
namespace {

struct ChainParams {
  const void *k, *v, *q;
  const float *alpha, *theta, *W_in;
  const int32_t* lengths;
  void* y;
  float* W_out;
  // segments of seg_chunks chunks; ws_phi, ws_loc, ws_start: [stream][segment][ld x ld] (rows: value channels of
  // W_0 and the starts, inputs of Phi)
  float *ws_phi, *ws_loc, *ws_start;
  int32_t* ws_whole;   // [stream][ld / 16]: value channels whose sequence is run in one piece
  int streams, H, Hk, N, d, parts, segments, seg_chunks, ld;
};

// a state of the workspace, as a chain wave holds it
template <int NT>
__device__ __forceinline__ void load_ws(f32x4 (&S)[NT], const float* W, int row, int ld, int g) {
#pragma unroll
  for (int i = 0; i < NT; ++i) {
    S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (row < ld && 16 * i < ld) S[i] = *(const f32x4*)(W + row * ld + 16 * i + 4 * g);
  }
}
template <int NT>
__device__ __forceinline__ void store_ws(const f32x4 (&S)[NT], float* W, int row, int ld, int g) {
#pragma unroll
  for (int i = 0; i < NT; ++i)
    if (row < ld && 16 * i < ld) *(f32x4*)(W + row * ld + 16 * i + 4 * g) = S[i];
}

// TRANS: the segments' maps instead of y: column groups up to d from zero with
// the values, as many again from the unit vectors without.
template <int DP, bool F32, int CW, int PB, int NB, int VB, bool TRANS>
__global__ void __launch_bounds__((CW + PB * (F32 ? 2 : 1)) * 64) delta_chain_kernel(ChainParams p) {
  constexpr int NP = F32 ? 3 : 1;   // planes of an input
  constexpr int NT = DP / 16, NK = DP / 32, kE = F32 ? 4 : 2;
  using Lds = ChunkLds<DP, NP, CW * 16>;
  extern __shared__ __attribute__((aligned(16))) unsigned char smem[];
  const Ring<Lds, CW, PB, NB, F32> ring{smem};
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // the parts of a stream's segment read the same K and Q: workgroups 8 apart share an XCD's L2
  const int segs = TRANS ? p.segments - 1 : p.segments, idx = blockIdx.x >> 3;
  const int unit_id = idx / p.parts * 8 + (blockIdx.x & 7), part = idx % p.parts;
  if (unit_id >= p.streams * segs) return;
  const int s = unit_id / segs, seg = unit_id % segs;
  const int b = s / p.H, h = s % p.H, d = p.d;
  const int all = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
  const int first = (int)min((int64_t)seg * p.seg_chunks * kC, (int64_t)all);   // the segment's tokens: first .. first + n - 1
  int n = seg + 1 < p.segments ? (int)min((int64_t)(all - first), (int64_t)p.seg_chunks * kC) : all - first;
  if (!TRANS && p.segments > 1) {   // the first segment takes the sequence, where its maps are of no use
    const int tiles = p.ld / 16, end = min((part + 1) * CW, tiles);
    int whole = 0;
    for (int i = part * CW; i < end; ++i) whole |= p.ws_whole[s * tiles + i];
    if (whole && seg > 0) return;
    if (whole) n = all;
  }
  // the segment with the sequence's last token leaves the final state (W_in itself, if there is no token)
  if (!TRANS && n == 0 && (seg > 0 || p.W_in == p.W_out)) return;   // (in place another call may be at such a state)
  const bool last = first + n == all;
  const int chunks = chunks_of(n);
  ring.init(wave, lane);

  if (wave >= CW) {
    const int col0 = part * CW * 16, vcols = max(d - col0, 0);
    const int64_t krow = (((int64_t)b * p.Hk + h / (p.H / p.Hk)) * p.N + first) * d;
    const int64_t vrow = ((int64_t)s * p.N + first) * d + (vcols > 0 ? col0 : 0), gate = (int64_t)s * p.N + first;
    const Rows in = {(const char*)p.k + krow * kE, (const char*)p.q + krow * kE, (const char*)p.v + vrow * kE,
                     p.alpha + gate, p.theta + gate, chunks, n, d, vcols};
    run_builder<DP, F32, VB, CW * 16, !TRANS, false>(ring, wave, lane, in);
    return;
  }

  // ---- chain ----
  const int cg = part * CW + wave, groups = (d + 15) / 16;
  const int col = cg * 16 + li;   // this lane's value channel
  const int unit = col - groups * 16;   // TRANS: its unit vector, if not negative
  const int64_t at_ws = ((int64_t)s * p.segments + seg) * p.ld * p.ld;
  f32x4 S[NT];
  if (TRANS) {
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[i][r] = 16 * i + 4 * g + r == unit && unit < d ? 1.f : 0.f;
  } else if (p.segments > 1) {
    load_ws(S, p.ws_start + at_ws, col, p.ld, g);
  } else {
    load_state<NT, VB>(S, p.W_in, s, col, d, g);
  }
  arrived(S);
  // y's tiles are computed transposed: a lane has 4 consecutive channels of
  // a token, stored in one piece at a uniform address per chunk plus this
  const int ych = cg * 16 + 4 * g;
  char* ydst = (char*)p.y + ((int64_t)s * p.N + first) * d * kE;
  const uint32_t yoff = ((uint32_t)li * d + ych) * kE;
  int ready = 0;   // what built[c % PB] was when last read
  for (int c = 0; c < chunks; ++c) {
    if (ready <= c) wait_for(ring.built() + c % PB, c + 1);
    acquire();
    const Lds L = ring.buffer(c);
    const uint16_t *ka = L.k() + li * Lds::RS + 8 * g, *qa = L.q() + li * Lds::RS + 8 * g;
    const uint16_t *ta = L.t() + li * kCS + 8 * g, *pa = L.p() + li * kCS + 8 * g;
    // The order below keeps LDS reads a product ahead of their use, and
    // products off the serial path (Q W^T, P F) in its gaps.
    f32x4 ks[2], qs[2], V[2], G[2], E[2], R[2], F[2];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) ks[rt] = qs[rt] = F[rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    bf16x8 ra[NK][2][NP];
#pragma unroll
    for (int kx = 0; kx < NK; ++kx) read2<NP>(ka + 32 * kx, Lds::KP, 16 * Lds::RS, ra[kx]);
    bf16x8 vr;
    if constexpr (F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        V[e >> 2][e & 3] = ((const float*)L.v())[(16 * (e >> 2) + 4 * g + (e & 3)) * Lds::VS + 16 * wave + li];
    } else {
      vr = read_transposed<false>((const uint16_t*)L.v(), Lds::VS, 16 * wave, lane);
    }
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) G[rt] = *(const f32x4*)(L.g() + 16 * rt + 4 * g);
    if (!F32) in_order();
    bf16x8 sp[NK][3];
#pragma unroll
    for (int kx = 0; kx < NK; ++kx) {
      split8<3>(S[2 * kx], S[2 * kx + 1], sp[kx]);
      mul2<false, 3>(ra[kx], sp[kx], ks);
    }
    bf16x8 rt3[2][3];
    read2<3>(ta, Lds::CP, 16 * kCS, rt3);
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) E[rt] = *(const f32x4*)(L.eth() + 16 * rt + 4 * g);
    if (!F32) in_order();
    bf16x8 rq[NK][2][NP];
    if (!TRANS)
#pragma unroll
    for (int kx = 0; kx < NK; ++kx) read2<NP>(qa + 32 * kx, Lds::KP, 16 * Lds::RS, rq[kx]);
    if constexpr (!F32) {
      const u32x4 x = __builtin_bit_cast(u32x4, vr);
#pragma unroll
      for (int e = 0; e < 8; ++e) V[e >> 2][e & 3] = e & 1 ? top(flt(x[e >> 1])) : flt(x[e >> 1] << 16);
    }
#pragma unroll
    for (int rt = 0; rt < 2; ++rt)
#pragma unroll
      for (int r = 0; r < 4; ++r) R[rt][r] = fmaf(-G[rt][r], ks[rt][r], V[rt][r]);
    bf16x8 rp[3];
    split8<3>(R[0], R[1], rp);
    if (!F32) in_order();
    bf16x8 kt[NT][NP], rp2[2][3];
    if (!F32) {
#pragma unroll
      for (int ti = 0; ti < NT; ++ti) kt[ti][0] = read_transposed<true>(L.k(), Lds::RS, 16 * ti, lane);
      if (!TRANS) read2<3>(pa, Lds::CP, 16 * kCS, rp2);
    }
    const float gc = L.gc()[0], scale = L.gc()[1];
    // F = T R, with Q W^T between the steps of its accumulation chains
    {
      constexpr int kF = products<3, 3>(), kQ = products<NP, 3>();
#pragma unroll
      for (int f = 0; f < kF; ++f) {
        mul2_one<false, 3>(f, rt3, rp, F);
        if (TRANS) continue;
#pragma unroll
        for (int x = f * NK * kQ / kF; x < (f + 1) * NK * kQ / kF; ++x) mul2_one<true, 3>(x % kQ, rq[x / kQ], sp[x / kQ], qs);
        if (!F32) in_order();
      }
    }
    // W' = G_C W + K^T (E theta F)
    f32x4 U[2], acc[NT], out[2];
    bf16x8 up[3], fp[3];
#pragma unroll
    for (int rt = 0; rt < 2; ++rt) U[rt] = F[rt] * E[rt];
    split8<3>(U[0], U[1], up);
    const bool scaled = __builtin_amdgcn_readfirstlane(bits(scale)) != 0x3f800000u;
#pragma unroll
    for (int ti = 0; ti < NT; ++ti) acc[ti] = S[ti] * gc;
    if (scaled) {   // seldom: theta far from 1 all over the chunk
#pragma unroll
      for (int ti = 0; ti < NT; ++ti) S[ti] = acc[ti], acc[ti] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (F32) {
#pragma unroll
      for (int ti = 0; ti < NT; ++ti)
#pragma unroll
        for (int e = 0; e < NP; ++e) kt[ti][e] = read_transposed<true>(L.k() + e * Lds::KP, Lds::RS, 16 * ti, lane);
      if (!TRANS) read2<3>(pa, Lds::CP, 16 * kCS, rp2);
    }
#pragma unroll
    for (int f = 0; f < products<NP, 3>(); ++f) {
      const Planes x = product<NP, 3>(f);
#pragma unroll
      for (int ti = 0; ti < NT; ++ti) acc[ti] = mfma(kt[ti][x.i], up[x.j], acc[ti]);
    }
    // Y^T = W Q^T diag(G) + F^T P^T
    if (!TRANS) {
      split8<3>(F[0], F[1], fp);
#pragma unroll
      for (int rt = 0; rt < 2; ++rt) out[rt] = qs[rt] * L.g()[16 * rt + li];
    }
    ready = seen(ring.built() + (c + 1) % PB);
    if (!TRANS) mul2<true, 3>(rp2, fp, out);
#pragma unroll
    for (int ti = 0; ti < NT; ++ti) S[ti] = scaled ? S[ti] + acc[ti] * scale : acc[ti];
    raise_to(ring.used() + wave, c + 1, lane);
    const int t0 = c * kC;
    char* at = ydst + (int64_t)t0 * d * kE;
    auto store = [&](int rt) {
      char* to = at + (yoff + 16u * rt * d * kE);
      if constexpr (VB > 0) {
        if constexpr (F32)
          *(f32x4*)to = out[rt];
        else
          *(bf16x4*)to = __builtin_convertvector(out[rt], bf16x4);
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (ych + r < d) {
            if constexpr (F32)
              ((float*)to)[r] = out[rt][r];
            else
              ((__bf16*)to)[r] = (__bf16)out[rt][r];
          }
      }
    };
    if (!TRANS && ych < d) {
      if (n - t0 >= kC) {
        store(0);
        store(1);
      } else {
#pragma unroll
        for (int rt = 0; rt < 2; ++rt)
          if (t0 + 16 * rt + li < n) store(rt);
      }
    }
  }
  if (TRANS) {
    if (unit < 0)
      store_ws(S, p.ws_loc + at_ws, col, p.ld, g);
    else
      store_ws(S, p.ws_phi + at_ws, unit, p.ld, g);
  } else if (last) {
    store_state<NT, VB>(S, p.W_out, s, col, d, g);
  }
}

// The state before every segment: a workgroup takes 16 rows (value channels)
// of a stream through W <- W Phi + W_0, in fp32 matrix instructions, the rows
// in LDS between segments.  The next segment's Phi and W_0 are read while one
// is computed: what remains serial is a product's 16 or 32 steps (in two
// accumulation chains) and the rows' way through LDS.
//
// A map may overflow where no state does: with a > 1 a direction that no key
// touches grows over the whole segment, and a state without a part in it meets
// 0 x inf.  Rows that come out of a join not finite are therefore taken
// through the sequence in one piece.
constexpr int kJoinThreads = 256;
template <int DP>
__global__ void __launch_bounds__(kJoinThreads) delta_join_kernel(ChainParams p) {
  constexpr int T = DP / 64, K = DP / 4;   // column tiles of a wave, steps of a product
  __shared__ float rows[16][DP + 4];
  const int ld = p.ld, blocks = ld / 16, s = blockIdx.x / blocks, row0 = blockIdx.x % blocks * 16, d = p.d;
  const int lane = threadIdx.x & 63, g = lane >> 4, li = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t base = (int64_t)s * p.segments * ld * ld;
  for (int e = threadIdx.x; e < 16 * DP; e += kJoinThreads) {
    const int r = e / DP, c = e % DP;
    const bool in = row0 + r < d && c < d;
    const float x = in ? p.W_in[((int64_t)s * d + row0 + r) * d + c] : 0.f;
    rows[r][c] = x;
    if (c < ld) p.ws_start[base + (row0 + r) * ld + c] = x;
  }
  struct Step {
    float phi[T][K];
    f32x4 loc[T];
  };
  // columns past ld read the last tile's (and are not stored), steps past it the last row, for zeros of `rows`
  int lost = 0;   // a value that is not finite
  auto read = [&](int seg, Step& x) {
    const float *phi = p.ws_phi + base + (int64_t)seg * ld * ld, *loc = p.ws_loc + base + (int64_t)seg * ld * ld;
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const int c = min((w + 4 * i) * 16, ld - 16) + li;
#pragma unroll
      for (int k = 0; k < K; ++k) x.phi[i][k] = phi[min(4 * k + g, ld - 1) * ld + c];
#pragma unroll
      for (int r = 0; r < 4; ++r) x.loc[i][r] = loc[(row0 + 4 * g + r) * ld + c];
    }
  };
  auto step = [&](int seg, const Step& x) {
    float* next = p.ws_start + base + (int64_t)(seg + 1) * ld * ld;
    f32x4 acc[T][2];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T; ++i) acc[i][0] = x.loc[i], acc[i][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < T; ++i)
        acc[i][k & 1] = __builtin_amdgcn_mfma_f32_16x16x4f32(rows[li][4 * k + g], x.phi[i][k], acc[i][k & 1], 0, 0, 0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const int c = (w + 4 * i) * 16 + li;
      if ((w + 4 * i) * 16 >= ld) continue;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float v = acc[i][0][r] + acc[i][1][r];
        lost |= (bits(v) & 0x7f800000u) == 0x7f800000u;
        rows[4 * g + r][c] = v;
        next[(row0 + 4 * g + r) * ld + c] = v;
      }
    }
  };
  const int n = p.segments - 1;
  Step a, b;
  read(0, a);
  for (int seg = 0; seg < n; seg += 2) {
    read(min(seg + 1, n - 1), b);
    step(seg, a);
    if (seg + 1 >= n) break;
    read(min(seg + 2, n - 1), a);
    step(seg + 1, b);
  }
  lost = __syncthreads_or(lost);
  if (threadIdx.x == 0) p.ws_whole[blockIdx.x] = lost;
}

template <int DP, bool F32, int CW, int VB, bool TRANS>
hipError_t launch_as(ChainParams p, hipStream_t stream) {
  // as many buffers as LDS holds, and builders as keep the chain fed
  constexpr int NB = F32 ? (DP == 64 ? 3 : 2) : 4, PB = F32 ? (DP == 64 ? 2 : 1) : DP == 64 ? 3 : 2;
  using R = Ring<ChunkLds<DP, F32 ? 3 : 1, CW * 16>, CW, PB, NB, F32>;
  constexpr int lds = R::BYTES;
  static_assert(lds <= 160 * 1024, "LDS of one workgroup");
  p.parts = ((p.d + 15) / 16 * (TRANS ? 2 : 1) + CW - 1) / CW;
  auto kernel = delta_chain_kernel<DP, F32, CW, PB, NB, VB, TRANS>;
  hipError_t err = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
  if (err != hipSuccess) return err;
  const int units = p.streams * (TRANS ? p.segments - 1 : p.segments);
  const unsigned grid = (unsigned)((units + 7) / 8 * 8 * p.parts);
  kernel<<<grid, R::WAVES * 64, lds, stream>>>(p);
  return hipGetLastError();
}

// How a call is cut.  Times of a chunk of 32 tokens in a workgroup that has a
// CU to itself, in tenths of a microsecond: d up to 64 with 2 chain waves 13,
// with 4 18 (128: 17 and 24; fp32: 20 and 30, 46 and 62), two thirds of that
// without y.  They are those of a full device; alone, 16 to 64 streams take 13
// and 14 to 15 (128: 18 and 25; fp32: 18 to 19 and 25, 44 and 58), and d from
// 65 to 96 a fifth less than 128, whichever way it is cut (15 to 18 and 22;
// fp32: 36 and 47), so it is cut as 128 is.
struct Plan {
  int wide;       // 4 chain waves in a workgroup of the (last) launch
  int segments;   // 1: one launch
  int seg_chunks;
};
constexpr int kCus = 256;
int chunk_cost(const DeltaShape& s, int cw) {
  if (s.io == TM_IO_BF16) return s.d <= 64 ? (cw == 2 ? 13 : 18) : cw == 2 ? 17 : 24;
  return s.d <= 64 ? (cw == 2 ? 20 : 30) : cw == 2 ? 46 : 62;
}
Plan plan_of(const DeltaShape& s) {
  const int64_t streams = (int64_t)s.B * s.H, chunks = chunks_of(s.N), groups = (s.d + 15) / 16;
  auto rounds = [&](int64_t segs, int64_t columns, int cw) {
    return (streams * segs * ((columns + cw - 1) / cw) + kCus - 1) / kCus * chunk_cost(s, cw);
  };
  Plan best = {0, 1, (int)chunks};
  int64_t cost = chunks * rounds(1, groups, 2);
  if (chunks * rounds(1, groups, 4) < cost) cost = chunks * rounds(1, groups, 4), best.wide = 1;
  for (int segs : {2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64, 96, 128}) {
    const int64_t per = (chunks + segs - 1) / segs, n = (chunks + per - 1) / per;
    if (n < 2) break;
    for (int wide = 0; wide < 2; ++wide) {
      // the maps' launch and the segments', the joins (0.5 and 0.8 us each), and two more launches
      const int64_t c = per * (rounds(n - 1, 2 * groups, 4) * 2 / 3 + rounds(n, groups, wide ? 4 : 2)) +
                        (s.d <= 64 ? 5 : 8) * n + 120;
      if (c < cost) cost = c, best = {wide, (int)n, (int)per};
    }
  }
  return best;
}

int64_t segment_floats(const DeltaShape& s, const Plan& plan) {
  const int64_t ld = (s.d + 15) / 16 * 16;
  return plan.segments > 1 ? (int64_t)s.B * s.H * plan.segments * ld * ld : 0;
}

template <int DP, bool F32, int VB>
hipError_t launch_chain(const ChainParams& p, bool wide, hipStream_t stream) {
  if (p.segments > 1) {
    hipError_t err = launch_as<DP, F32, 4, VB, true>(p, stream);
    if (err != hipSuccess) return err;
    delta_join_kernel<DP == 64 ? 64 : 128><<<p.streams * (p.ld / 16), kJoinThreads, 0, stream>>>(p);
    if ((err = hipGetLastError()) != hipSuccess) return err;
  }
  return wide ? launch_as<DP, F32, 4, VB, false>(p, stream) : launch_as<DP, F32, 2, VB, false>(p, stream);
}

// Widths from 65 to 96 have kernels of their own: 3 of 4 tiles' work, 30
// streams x 777 x 96, fp32, in 115 us against 136 with rows padded to 128
// (256 x 1024 x 80, bf16: 163 against 189).
template <bool F32, int VB>
hipError_t launch_width(const ChainParams& p, bool wide, hipStream_t stream) {
  if (p.d <= 64) return launch_chain<64, F32, VB>(p, wide, stream);
  return p.d <= 96 ? launch_chain<96, F32, VB>(p, wide, stream) : launch_chain<128, F32, VB>(p, wide, stream);
}

}  // namespace

int64_t delta_chunked_ws_bytes(const DeltaShape& s) {
  const Plan plan = plan_of(s);
  return 12 * segment_floats(s, plan) + (plan.segments > 1 ? (int64_t)s.B * s.H * ((s.d + 15) / 16) * 4 : 0);
}

hipError_t launch_delta_chunked(const DeltaShape& s, const void* k, const void* v, const void* q, const float* alpha,
                                const float* theta, const int32_t* lengths, const float* W_in, void* y, float* W_out,
                                float* ws, hipStream_t stream) {
  const Plan plan = plan_of(s);
  ChainParams p = {k, v, q, alpha, theta, W_in, lengths, y, W_out};
  p.ws_phi = ws, p.ws_loc = ws + segment_floats(s, plan), p.ws_start = ws + 2 * segment_floats(s, plan);
  p.ws_whole = (int32_t*)(ws + 3 * segment_floats(s, plan));
  p.streams = s.B * s.H, p.H = s.H, p.Hk = s.Hk, p.N = s.N, p.d = s.d, p.ld = (s.d + 15) / 16 * 16;
  p.segments = plan.segments, p.seg_chunks = plan.seg_chunks;
  if (s.io == TM_IO_BF16) {
    if (s.d % 8 == 0) return launch_width<false, 16>(p, plan.wide, stream);
    return s.d % 4 == 0 ? launch_width<false, 8>(p, plan.wide, stream) : launch_width<false, 0>(p, plan.wide, stream);
  }
  return s.d % 4 == 0 ? launch_width<true, 16>(p, plan.wide, stream) : launch_width<true, 0>(p, plan.wide, stream);
}

}  // namespace titans
