// Group norm with an activation behind the memory, and its gradient: the
// "normalization and gating" before a block's output projection ("Titans:
// Learning to Memorize at Test Time", mer.dev notes, section 4.4,
// "Architectural Details").  A group is one head's d channels of one token:
//
//   xh = (x - mean) / sqrt(var + eps),  n = xh w + b
//   out = act(gate) n   with a gate,   act(n)   without one
//
// x lies heads-first [B,H,N,d], as the memory writes y, or channels-last
// [B,N,H d]; the rest is channels-last, as a projection reads it.
//
// Gradient, with z the activation's argument, f = act(z), f' its slope:
//   with a gate   dn = dout f,  dgate = dout n f';   without one  dn = dout f'
//   dxh = dn w,  dx = (dxh - mean(dxh) - xh mean(dxh xh)) / sqrt(var + eps)
//   dw = sum over tokens of dn xh,  db = sum over tokens of dn
//
// Every kernel is bound by memory: x, gate and out are passed over once, and
// the gradient computes the statistics again from the x that it reads anyway.
// A group lies in L lanes (a power of two), each with IT pieces of VEC
// consecutive channels in registers, so the sums over a group are log2 L
// shuffles.  A workgroup keeps one head, so w and b are loaded once, and
// takes 1/grid.x of the tokens (slices_of).  The gradient's workgroup sums its tokens'
// shares of dw and db in registers and LDS, in a fixed order, into one row of
// the workspace; a second kernel sums the rows, again in a fixed order (a
// single row, of a few tokens, is the result).
// 8 x 16384 tokens x 1024 channels, bf16, gated: 170 us, 4.7 TB/s (a large copy
// reaches 5.2); the gradient at 8 x 16384: 279 us, 4.8 TB/s.
#include "tm_internal.h"

namespace titans {
namespace {

constexpr int kThreads = 256;

struct NormParams {
  const void *x, *gate, *dout;
  const float *weight, *bias;
  const int32_t* lengths;
  void *out, *dx, *dgate;
  float* partial;            // [slices][2][H d]
  float *dweight, *dbias;    // written here by a single slice
  int H, N, d, silu, first;
  int64_t rows;     // B N
  int64_t per;      // rows per workgroup
  float eps;
};

__device__ __forceinline__ uint16_t to_bf16(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ float low_bf16(uint32_t x) { return __builtin_bit_cast(float, x << 16); }
__device__ __forceinline__ float high_bf16(uint32_t x) { return __builtin_bit_cast(float, x & 0xffff0000u); }

template <bool BF16, int VEC>
__device__ __forceinline__ void load_piece(const void* p, int64_t i, float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    x[0] = BF16 ? low_bf16(((const uint16_t*)p)[i]) : ((const float*)p)[i];
  } else if constexpr (BF16 && VEC == 4) {
    const uint2 v = *(const uint2*)((const uint16_t*)p + i);
    x[0] = low_bf16(v.x), x[1] = high_bf16(v.x), x[2] = low_bf16(v.y), x[3] = high_bf16(v.y);
  } else if constexpr (BF16) {
    const uint4 v = *(const uint4*)((const uint16_t*)p + i);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) x[2 * j] = low_bf16(u[j]), x[2 * j + 1] = high_bf16(u[j]);
  } else {
    const float4 v = *(const float4*)((const float*)p + i);
    x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
  }
}

template <bool BF16, int VEC>
__device__ __forceinline__ void store_piece(void* p, int64_t i, const float (&x)[VEC]) {
  if constexpr (VEC == 1) {
    if (BF16)
      ((uint16_t*)p)[i] = to_bf16(x[0]);
    else
      ((float*)p)[i] = x[0];
  } else if constexpr (BF16) {
    typedef __attribute__((ext_vector_type(VEC))) float fv;
    typedef __attribute__((ext_vector_type(VEC))) __bf16 bv;
    fv v;
#pragma unroll
    for (int j = 0; j < VEC; ++j) v[j] = x[j];
    *(bv*)((uint16_t*)p + i) = __builtin_convertvector(v, bv);
  } else {
    *(float4*)((float*)p + i) = make_float4(x[0], x[1], x[2], x[3]);
  }
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// sum over L neighbouring lanes, in every lane: DPP within a row of 16 (each
// step adds the other half, mirrored), which stays out of LDS
template <int L>
__device__ __forceinline__ float group_sum(float x) {
  if (L >= 2) x = dpp_add<0xB1>(x);    // quad_perm 1 0 3 2
  if (L >= 4) x = dpp_add<0x4E>(x);    // quad_perm 2 3 0 1
  if (L >= 8) x = dpp_add<0x141>(x);   // row_half_mirror
  if (L >= 16) x = dpp_add<0x140>(x);  // row_mirror
  if (L >= 32) x += __shfl_xor(x, 16, 64);
  if (L >= 64) x += __shfl_xor(x, 32, 64);
  return x;
}

// 1 / (1 + exp(-z)): a few units in the last place where exp(-z) is small or
// of order one, and about |z| / 2 of them where it is large (the power's
// exponent, |z| log2 e, is rounded: 40 units at z = -80, where the value is
// 1e-35).  A reciprocal instruction, a division being ten; 0 and 1 at the ends
__device__ __forceinline__ float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

template <bool BF16, int VEC, int L, int IT, bool GRAD>
__global__ void __launch_bounds__(kThreads) group_norm_kernel(NormParams p) {
  constexpr int kGroups = kThreads / L;   // groups a workgroup holds at a time
  const int tid = threadIdx.x, l = tid % L, g = tid / L, h = blockIdx.y, C = p.H * p.d;
  const bool gated = p.gate != nullptr;
  const float inv_d = 1.f / (float)p.d;
  float w[IT][VEC], bias[IT][VEC], dw[IT][VEC], db[IT][VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = (i * L + l) * VEC + j;
      w[i][j] = c < p.d ? (p.weight ? p.weight[h * p.d + c] : 1.f) : 0.f;
      bias[i][j] = c < p.d && p.bias ? p.bias[h * p.d + c] : 0.f;
      dw[i][j] = db[i][j] = 0.f;
    }
  const int64_t r0 = (int64_t)blockIdx.x * p.per, r1 = min(r0 + p.per, p.rows);
  // every lane of a wave runs the same rounds: groups past the end do no loads, but take part in the sums
  const uint32_t N = max(p.N, 1);
  int64_t b = (r0 + g) / N;
  uint32_t t = (uint32_t)((r0 + g) - b * N);
  for (int64_t rb = r0; rb < r1; rb += kGroups) {
    const int64_t r = rb + g;
    bool live = r < r1, past = false;
    if (live && p.lengths && (int64_t)t >= p.lengths[b]) live = false, past = true;
    const int64_t ct = r * C + (int64_t)h * p.d;
    const int64_t xt = p.first ? ((b * p.H + h) * (int64_t)p.N + t) * p.d : ct;
    t += kGroups;
    if (t >= N) {
      const uint32_t more = t / N;
      b += more;
      t -= more * N;
    }
    float x[IT][VEC], z[IT][VEC], go[IT][VEC], sum = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + l) * VEC;
      const bool in = live && c < p.d;
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[i][j] = z[i][j] = go[i][j] = 0.f;
      if (in) load_piece<BF16, VEC>(p.x, xt + c, x[i]);
      if (in && gated) load_piece<BF16, VEC>(p.gate, ct + c, z[i]);
      if (GRAD && in) load_piece<BF16, VEC>(p.dout, ct + c, go[i]);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum += x[i][j];
    }
    const float mean = group_sum<L>(sum) * inv_d;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const bool in = (i * L + l) * VEC < p.d;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        x[i][j] = in ? x[i][j] - mean : 0.f;
        sum = fmaf(x[i][j], x[i][j], sum);
      }
    }
    const float var = group_sum<L>(sum) * inv_d;
    const float rstd = live ? 1.f / sqrtf(var + p.eps) : 0.f;   // 0: a dead group adds nothing, whatever eps
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int i = 0; i < IT; ++i) {
      const int c = (i * L + l) * VEC;
      float o[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float xh = x[i][j] * rstd, n = fmaf(xh, w[i][j], bias[i][j]);
        const float a = gated ? z[i][j] : n;
        const float sg = p.silu ? sigmoid(a) : 1.f;
        const float f = p.silu ? a * sg : a;
        if (!GRAD) {
          o[j] = gated ? f * n : f;
        } else {
          const float slope = p.silu ? sg * fmaf(a, 1.f - sg, 1.f) : 1.f;
          const float dn = live ? go[i][j] * (gated ? f : slope) : 0.f;   // (the slope at an infinite bias is NaN)
          o[j] = live ? go[i][j] * n * slope : 0.f;   // dgate
          dw[i][j] = fmaf(dn, xh, dw[i][j]);
          db[i][j] += dn;
          const float dxh = dn * w[i][j];
          s1 += dxh;
          s2 = fmaf(dxh, xh, s2);
          x[i][j] = xh;
          go[i][j] = dxh;
        }
      }
      if (!GRAD && live && c < p.d) store_piece<BF16, VEC>(p.out, ct + c, o);
      if (GRAD && gated && (live || past) && c < p.d) store_piece<BF16, VEC>(p.dgate, ct + c, o);
    }
    if (GRAD) {
      s1 = group_sum<L>(s1) * inv_d;
      s2 = group_sum<L>(s2) * inv_d;
#pragma unroll
      for (int i = 0; i < IT; ++i) {
        const int c = (i * L + l) * VEC;
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = live ? rstd * (go[i][j] - s1 - x[i][j] * s2) : 0.f;
        if ((live || past) && c < p.d) store_piece<BF16, VEC>(p.dx, xt + c, o);
      }
    }
  }
  if (!GRAD) return;
  // the workgroup's sums of dw and db: its kGroups groups' shares, in order
  __shared__ float red[kThreads * VEC];
#pragma unroll
  for (int i = 0; i < IT; ++i)
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < VEC; ++j) red[(g * L + l) * VEC + j] = which ? db[i][j] : dw[i][j];
      __syncthreads();
      for (int c = tid; c < L * VEC; c += kThreads) {
        float sum = 0.f;
        for (int k = 0; k < kGroups; ++k) sum += red[k * L * VEC + c];
        const int ch = i * L * VEC + c;
        if (ch >= p.d) continue;
        if (gridDim.x == 1)
          (which ? p.dbias : p.dweight)[h * p.d + ch] = sum;
        else
          p.partial[((int64_t)blockIdx.x * 2 + which) * C + h * p.d + ch] = sum;
      }
    }
}

// dweight and dbias: column sums of the slices' rows.  16 threads share a
// column's rows, then one adds their sums in order.
__global__ void __launch_bounds__(kThreads) norm_reduce_kernel(const float* partial, int slices, int C, float* dweight,
                                                               float* dbias) {
  __shared__ float red[16][17];
  const int c = blockIdx.x * 16 + (threadIdx.x & 15), k = threadIdx.x >> 4, which = blockIdx.y;
  float sum = 0.f;
  if (c < C)
    for (int i = k; i < slices; i += 16) sum += partial[((int64_t)i * 2 + which) * C + c];
  red[k][threadIdx.x & 15] = sum;
  __syncthreads();
  if (k || c >= C) return;
  sum = 0.f;
  for (int i = 0; i < 16; ++i) sum += red[i][threadIdx.x & 15];
  (which ? dbias : dweight)[c] = sum;
}

template <bool BF16, int VEC, int L, int IT>
hipError_t launch_as(const NormParams& p, int slices, bool grad, hipStream_t stream) {
  const dim3 grid(slices, p.H);
  if (grad)
    group_norm_kernel<BF16, VEC, L, IT, true><<<grid, kThreads, 0, stream>>>(p);
  else
    group_norm_kernel<BF16, VEC, L, IT, false><<<grid, kThreads, 0, stream>>>(p);
  return hipGetLastError();
}

// The widest pieces that d's rows are aligned for, and the fewest lanes that
// hold a group.
template <bool BF16>
hipError_t launch(const NormParams& p, int slices, bool grad, hipStream_t stream) {
  const int d = p.d;
  if (d % 4) {
    if (d <= 16) return launch_as<BF16, 1, 16, 1>(p, slices, grad, stream);
    if (d <= 32) return launch_as<BF16, 1, 16, 2>(p, slices, grad, stream);
    if (d <= 48) return launch_as<BF16, 1, 16, 3>(p, slices, grad, stream);
    if (d <= 64) return launch_as<BF16, 1, 16, 4>(p, slices, grad, stream);
    if (d <= 128) return launch_as<BF16, 1, 32, 4>(p, slices, grad, stream);
    if (d <= 256) return launch_as<BF16, 1, 64, 4>(p, slices, grad, stream);
    return launch_as<BF16, 1, 64, 16>(p, slices, grad, stream);
  }
  if (!BF16 || d % 8) {
    if (d <= 16) return launch_as<BF16, 4, 4, 1>(p, slices, grad, stream);
    if (d <= 32) return launch_as<BF16, 4, 8, 1>(p, slices, grad, stream);
    if (d <= 64) return launch_as<BF16, 4, 16, 1>(p, slices, grad, stream);
    if (d <= 128) return launch_as<BF16, 4, 32, 1>(p, slices, grad, stream);
    if (d <= 256) return launch_as<BF16, 4, 64, 1>(p, slices, grad, stream);
    return launch_as<BF16, 4, 64, 4>(p, slices, grad, stream);
  }
  if constexpr (BF16) {
    if (d <= 16) return launch_as<BF16, 8, 2, 1>(p, slices, grad, stream);
    if (d <= 32) return launch_as<BF16, 8, 4, 1>(p, slices, grad, stream);
    if (d <= 64) return launch_as<BF16, 8, 8, 1>(p, slices, grad, stream);
    if (d <= 128) return launch_as<BF16, 8, 16, 1>(p, slices, grad, stream);
    if (d <= 256) return launch_as<BF16, 8, 32, 1>(p, slices, grad, stream);
    return launch_as<BF16, 8, 64, 2>(p, slices, grad, stream);
  }
}

// Groups that a workgroup holds at a time, as launch() lays them out.
int groups_of(const NormShape& s) {
  const int vec = s.d % 4 ? 1 : s.io == TM_IO_BF16 && s.d % 8 == 0 ? 8 : 4, held = vec == 1 ? 4 : vec;
  int lanes = 16 / vec;
  while (lanes < 64 && lanes * held < s.d) lanes *= 2;
  return kThreads / lanes;
}

// Workgroups along the tokens, none with less than 2 rounds of its groups (4
// in the gradient, whose slices are summed again: 1 x 32 heads x 2048 x 128,
// bf16, 23.7 us, with 2 26.0).
//
// From 8 heads on 2048 in all (the device holds about as many; 4096 or 8192
// cost the gradient 4% and 9%, 1024 the norm 2% to 25%).  With fewer heads the
// norm takes 1024 (one head x 65536 x 1024, bf16: 86 us, in 256 workgroups
// 176, in 4096 79; 2 heads x 65536 x 512, fp32: 164, in 2048 193), the
// gradient 256 a head (2 heads x 131072 x 64, bf16: 41, in 1024 43 and in 2048
// 52) and 512 for a single one (one head x 65536 x 1024, bf16: 179, in 256 280
// and in 1024 194).
//
// With thousands of heads one slice a head would do, but its thousands of
// tokens would be summed one after the other: the gradient's slices have 2048
// rows at most (4096 heads x 16384 x 16, bf16: 2739 us, in one slice 4358),
// as far as a launch of fewer than 2^32 threads goes.
int slices_of(const NormShape& s, bool grad) {
  const int64_t rows = (int64_t)s.B * s.N, least = (grad ? 4 : 2) * groups_of(s);
  const int all = s.H >= 8 ? 2048 : !grad ? 1024 : s.H == 1 ? 512 : 256 * s.H;
  int64_t n = (rows + least - 1) / least;
  if (n > (all + s.H - 1) / s.H) n = (all + s.H - 1) / s.H;
  if (grad && n < (rows + 2047) / 2048) n = (rows + 2047) / 2048;
  if (n > (1 << 23) / s.H) n = (1 << 23) / s.H;
  return n < 1 ? 1 : (int)n;
}

NormParams params_of(const NormShape& s, int slices) {
  NormParams p = {};
  p.H = s.H, p.N = s.N, p.d = s.d, p.silu = s.silu, p.first = s.first, p.eps = s.eps;
  p.rows = (int64_t)s.B * s.N;
  p.per = (p.rows + slices - 1) / slices;
  return p;
}

}  // namespace

int64_t norm_backward_ws_bytes(const NormShape& s) { return (int64_t)slices_of(s, true) * 2 * s.H * s.d * 4; }

hipError_t launch_group_norm(const NormShape& s, const void* x, const void* gate, const float* weight,
                             const float* bias, const int32_t* lengths, void* out, hipStream_t stream) {
  const int slices = slices_of(s, false);
  NormParams p = params_of(s, slices);
  p.x = x, p.gate = gate, p.weight = weight, p.bias = bias, p.lengths = lengths, p.out = out;
  return s.io == TM_IO_BF16 ? launch<true>(p, slices, false, stream) : launch<false>(p, slices, false, stream);
}

hipError_t launch_group_norm_backward(const NormShape& s, const void* x, const void* gate, const float* weight,
                                      const float* bias, const int32_t* lengths, const void* dout, void* dx,
                                      void* dgate, float* dweight, float* dbias, float* ws, hipStream_t stream) {
  const int slices = slices_of(s, true), C = s.H * s.d;
  NormParams p = params_of(s, slices);
  p.x = x, p.gate = gate, p.weight = weight, p.bias = bias, p.lengths = lengths, p.dout = dout;
  p.dx = dx, p.dgate = dgate, p.partial = ws, p.dweight = dweight, p.dbias = dbias;
  hipError_t err = s.io == TM_IO_BF16 ? launch<true>(p, slices, true, stream) : launch<false>(p, slices, true, stream);
  if (err != hipSuccess || slices == 1) return err;
  norm_reduce_kernel<<<dim3((C + 15) / 16, 2), kThreads, 0, stream>>>(ws, slices, C, dweight, dbias);
  return hipGetLastError();
}

}  // namespace titans
