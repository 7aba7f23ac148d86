// The gated delta memory (linear memory, token-exact, momentum-free), token
// by token.  Per (batch, head) stream and token, with a = 1 - alpha:
//
//   f = v - a W k,   W <- a W + theta f k^T,   y = W q
//
// i.e. the delta rule of the linear memory M(k) = W k ("Titans: Learning to
// Memorize at Test Time", mer.dev notes, section 3.1, "Objective" and
// "Forgetting Mechanism") with the residual taken at the decayed memory of
// the token before.
//
// A row of W meets nothing of another row: row i needs v_i, and k, q and the
// gates that all rows share.  So a row lives in 16 lanes' registers (float4
// pieces), a wave holds 4 rows, a workgroup of 4 waves a slice of
// the state's rows, and the two dot products of a token are sums over 16
// lanes by DPP.  Nothing is exchanged between waves.  The state is read and
// written once; for a few tokens that traffic (8 d^2 bytes a stream) is the
// bound: a step of 192 x 16 heads of 128 x 128 takes 72 us, 5.6 TB/s (a large
// copy reaches 5.2), and 37 in place with every other slot idle.  A small call is
// launch and latency, about 3 us.
#include "tm_internal.h"

namespace titans {
namespace {

constexpr int kRecThreads = 256;

template <bool BF16>
__device__ __forceinline__ float load_io(const void* p, int64_t i) {
  if (BF16) return __builtin_bit_cast(float, (uint32_t)((const uint16_t*)p)[i] << 16);
  return ((const float*)p)[i];
}

// round to nearest even, NaN kept
__device__ __forceinline__ uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

template <bool BF16>
__device__ __forceinline__ void store_io(void* p, int64_t i, float x) {
  if (BF16)
    ((uint16_t*)p)[i] = to_bf16(x);
  else
    ((float*)p)[i] = x;
}

template <int ROR>
__device__ __forceinline__ float dpp_ror(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x120 + ROR, 0xf, 0xf, true));
}

// sum over the 16 lanes of a DPP row, in every lane
__device__ __forceinline__ float row_sum(float x) {
  x += dpp_ror<8>(x);
  x += dpp_ror<4>(x);
  x += dpp_ror<2>(x);
  x += dpp_ror<1>(x);
  return x;
}

struct RecParams {
  const void *k, *v, *q;
  const float *alpha, *theta, *W_in;
  const int32_t* lengths;
  void* y;
  float* W_out;
  int H, Hk, N, d, blocks;   // blocks: row slices per stream
};

// EPL: state elements of a row in one lane (4: d <= 64, 8: d <= 128).
// VEC: d is a multiple of 4, so that a lane's float4 pieces are whole and
// aligned.  Columns past d hold zeros throughout.
template <bool BF16, int EPL, int SETS, bool VEC>
__global__ void __launch_bounds__(kRecThreads) delta_recurrent_kernel(RecParams p) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int s = blockIdx.x / p.blocks, slice = blockIdx.x % p.blocks;
  const int b = s / p.H, h = s % p.H;
  const int d = p.d, c0 = (lane & 15) * 4;
  const int row0 = (slice * 4 + wave) * 4 * SETS + (lane >> 4);
  const int n = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
  const int64_t kbase = ((int64_t)b * p.Hk + h / (p.H / p.Hk)) * p.N * d;
  const int64_t vbase = (int64_t)s * p.N * d, gbase = (int64_t)s * p.N;
  const float* W_in = p.W_in + (int64_t)s * d * d;
  float* W_out = p.W_out + (int64_t)s * d * d;
  if (n == 0 && p.W_in == p.W_out) return;   // (another call may be at this state)

  float w[SETS][EPL];
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const int row = row0 + 4 * i;
#pragma unroll
    for (int e = 0; e < EPL; e += 4) {
      const int c = c0 + 16 * e;
      if (VEC) {
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (row < d && c < d) x = *(const float4*)(W_in + (int64_t)row * d + c);
        w[i][e] = x.x, w[i][e + 1] = x.y, w[i][e + 2] = x.z, w[i][e + 3] = x.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[i][e + j] = row < d && c + j < d ? W_in[(int64_t)row * d + c + j] : 0.f;
      }
    }
  }
  // token t's shared vectors, its gates, and v of this lane's rows
  auto fetch = [&](int t, float (&k)[EPL], float (&q)[EPL], float (&v)[SETS], float& al, float& th) {
    const int64_t at = kbase + (int64_t)t * d;
#pragma unroll
    for (int e = 0; e < EPL; e += 4) {
      const int c = c0 + 16 * e;
#pragma unroll
      for (int j = 0; j < 4; ++j) k[e + j] = q[e + j] = 0.f;
      if (VEC) {
        if (c < d) {
          if (BF16) {
            const uint2 x = *(const uint2*)((const uint16_t*)p.k + at + c), z = *(const uint2*)((const uint16_t*)p.q + at + c);
            k[e] = __builtin_bit_cast(float, x.x << 16), k[e + 1] = __builtin_bit_cast(float, x.x & 0xffff0000u);
            k[e + 2] = __builtin_bit_cast(float, x.y << 16), k[e + 3] = __builtin_bit_cast(float, x.y & 0xffff0000u);
            q[e] = __builtin_bit_cast(float, z.x << 16), q[e + 1] = __builtin_bit_cast(float, z.x & 0xffff0000u);
            q[e + 2] = __builtin_bit_cast(float, z.y << 16), q[e + 3] = __builtin_bit_cast(float, z.y & 0xffff0000u);
          } else {
            const float4 x = *(const float4*)((const float*)p.k + at + c), z = *(const float4*)((const float*)p.q + at + c);
            k[e] = x.x, k[e + 1] = x.y, k[e + 2] = x.z, k[e + 3] = x.w;
            q[e] = z.x, q[e + 1] = z.y, q[e + 2] = z.z, q[e + 3] = z.w;
          }
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < d) k[e + j] = load_io<BF16>(p.k, at + c + j), q[e + j] = load_io<BF16>(p.q, at + c + j);
      }
    }
#pragma unroll
    for (int i = 0; i < SETS; ++i)
      v[i] = row0 + 4 * i < d ? load_io<BF16>(p.v, vbase + (int64_t)t * d + row0 + 4 * i) : 0.f;
    al = p.alpha[gbase + t];
    th = p.theta[gbase + t];
  };

  float k[EPL], q[EPL], v[SETS], al, th;
  if (n > 0) fetch(0, k, q, v, al, th);
  for (int t = 0; t < n; ++t) {
    float kn[EPL], qn[EPL], vn[SETS], aln, thn;
    fetch(min(t + 1, n - 1), kn, qn, vn, aln, thn);
    // 1 - alpha is never formed: x - alpha x in one fma is x (1 - alpha) rounded once
    const float na = al > 1.f ? __builtin_nanf("") : -al;
#pragma unroll
    for (int i = 0; i < SETS; ++i) {
      float kw = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) kw = fmaf(w[i][e], k[e], kw);
      kw = row_sum(kw);
      const float u = th * (v[i] - fmaf(na, kw, kw));
      float y = 0.f;
#pragma unroll
      for (int e = 0; e < EPL; ++e) {
        w[i][e] = fmaf(u, k[e], fmaf(na, w[i][e], w[i][e]));
        y = fmaf(w[i][e], q[e], y);
      }
      y = row_sum(y);
      const int row = row0 + 4 * i;
      if ((lane & 15) == 0 && row < d) store_io<BF16>(p.y, vbase + (int64_t)t * d + row, y);
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) k[e] = kn[e], q[e] = qn[e];
#pragma unroll
    for (int i = 0; i < SETS; ++i) v[i] = vn[i];
    al = aln, th = thn;
  }
#pragma unroll
  for (int i = 0; i < SETS; ++i) {
    const int row = row0 + 4 * i;
    if (row >= d) continue;
#pragma unroll
    for (int e = 0; e < EPL; e += 4) {
      const int c = c0 + 16 * e;
      if (VEC) {
        if (c < d) *(float4*)(W_out + (int64_t)row * d + c) = make_float4(w[i][e], w[i][e + 1], w[i][e + 2], w[i][e + 3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (c + j < d) W_out[(int64_t)row * d + c + j] = w[i][e + j];
      }
    }
  }
}

template <bool BF16, int EPL>
hipError_t launch_recurrent(const DeltaShape& s, const RecParams& p0, hipStream_t stream) {
  constexpr int kSets = 1;
  RecParams p = p0;
  p.blocks = (s.d + 16 * kSets - 1) / (16 * kSets);
  const dim3 grid((unsigned)((int64_t)s.B * s.H * p.blocks));
  if (s.d % 4 == 0)
    delta_recurrent_kernel<BF16, EPL, kSets, true><<<grid, kRecThreads, 0, stream>>>(p);
  else
    delta_recurrent_kernel<BF16, EPL, kSets, false><<<grid, kRecThreads, 0, stream>>>(p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_delta_recurrent(const DeltaShape& s, const void* k, const void* v, const void* q,
                                  const float* alpha, const float* theta, const int32_t* lengths, const float* W_in,
                                  void* y, float* W_out, hipStream_t stream) {
  const RecParams p = {k, v, q, alpha, theta, W_in, lengths, y, W_out, s.H, s.Hk, s.N, s.d, 0};
  const bool bf = s.io == TM_IO_BF16;
  if (s.d <= 64) return bf ? launch_recurrent<true, 4>(s, p, stream) : launch_recurrent<false, 4>(s, p, stream);
  return bf ? launch_recurrent<true, 8>(s, p, stream) : launch_recurrent<false, 8>(s, p, stream);
}

}  // namespace titans
