// Internal declarations shared by the host layer and the kernel files of
// libtitans_mem.so.  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>

#include "titans_mem.h"

namespace titans {

constexpr int kMaxLayers = 8;        // generic path
constexpr int kMaxChunkGeneric = 4096;
constexpr int kMaxWidthGeneric = 8192;
constexpr int kRetrieveTile = 8;     // tokens per block in titans_mem_retrieve
constexpr int kMaxWidthRetrieve = 1024;

struct Shape {
  int streams, N, d, hidden, L, io, read_mode;
  int chunk_gates;   // gates given per chunk (TM_FLAG_CHUNK_GATES)
  unsigned flags;    // the desc's TM_FLAG_* bits
  int widths[kMaxLayers + 1];
  int64_t off[kMaxLayers + 1];
  int64_t P;
  int maxw;
};

// Workspace floats per stream of the generic kernel for chunk b (one region).
int64_t generic_ws_floats_per_stream(const Shape& s, int b);
// Workspace floats per stream of launch_generic (the forward call).
int64_t generic_forward_ws_floats_per_stream(const Shape& s, int chunk);

// The library's second stream on a device and the events that order it
// against the caller's stream: created on first use (default priority) and
// kept until the process ends.  side_stream() returns the current device's
// with `lock` held, which serialises the calls that enqueue on it (each
// call records every event before waiting on it).
struct SideStream {
  hipStream_t st = nullptr;
  hipEvent_t fork = nullptr, join = nullptr, prod[2] = {nullptr, nullptr}, cons[2] = {nullptr, nullptr};
};
hipError_t side_stream(int dev, SideStream** out, std::unique_lock<std::mutex>& lock);
// Makes `stream` wait for everything enqueued so far on the side stream.
// Every launcher calls it on each return path after its first enqueue on the
// side stream (errors included), so that work the caller enqueues on
// `stream` afterwards, such as freeing buffers, never overtakes it; returns
// `err` when that is an error, else the join's own status.
hipError_t join_side(SideStream* x, hipStream_t stream, hipError_t err);

hipError_t launch_generic(const Shape& s, int chunk, const void* k, const void* v, const void* q,
                          const float* alpha, const float* eta, const float* theta,
                          const float* W_in, const float* S_in, void* y, float* W_out,
                          float* S_out, float* ws, hipStream_t stream);

hipError_t launch_retrieve_generic(const Shape& s, const void* q, const float* W, void* y,
                                   hipStream_t stream);

// The linear memory (L = 1, d <= 64 and a multiple of 4, chunk <= 64) on one
// workgroup per stream with the state and the chunk in LDS; part of the
// generic path (fp32 arithmetic, no workspace).
bool linear_supported(const Shape& s, int chunk);
hipError_t launch_linear(const Shape& s, int chunk, const void* k, const void* v, const void* q,
                         const float* alpha, const float* eta, const float* theta, const float* W_in,
                         const float* S_in, void* y, float* W_out, float* S_out, hipStream_t stream);

// Specialised 2-layer d=64 hidden=256 MFMA kernel (chunk <= 64, bf16 io).
bool mlp2_supported(const Shape& s, int chunk);
int64_t mlp2_ws_bytes(const Shape& s, int chunk);
// byte offset of the kernel's status word in its workspace (1 = a pair gave up)
int64_t mlp2_status_offset(const Shape& s);
// The allocation-free variant's scratch: a file-scope device array of
// mlp2_scratch_bytes() bytes in tm_mlp2_group.hip.  mlp2_scratch gives its device
// address on the current device, looked up there on the first call with
// lookup = true (nullptr while it never was).
int64_t mlp2_scratch_bytes();
hipError_t mlp2_scratch(void** out, bool lookup);
hipError_t launch_mlp2(const Shape& s, int chunk, const void* k, const void* v, const void* q,
                       const float* alpha, const float* eta, const float* theta,
                       const float* W_in, const float* S_in, void* y, float* W_out,
                       float* S_out, void* ws, hipStream_t stream);

// Deep memories on the matrix cores: L >= 2, widths multiples of 64, bf16 io,
// chunk <= 256; one launch per step of a chunk over all streams.
bool deep_supported(const Shape& s, int chunk);
int64_t deep_ws_bytes(const Shape& s, int chunk);
hipError_t launch_deep(const Shape& s, int chunk, const void* k, const void* v, const void* q, const float* alpha,
                       const float* eta, const float* theta, const float* W_in, const float* S_in, void* y,
                       float* W_out, float* S_out, void* ws, hipStream_t stream);

// Retrieval at a fixed state on the matrix cores (2-layer, d=64, hidden=256, bf16).
bool retrieve_mlp2_supported(const Shape& s);
hipError_t launch_retrieve_mlp2(const Shape& s, const void* q, const float* W, void* y, hipStream_t stream);

// The generic kernel as a state sweep only (no retrieval), writing (W, S) at
// every chunk start to ckpt; W, S and ckpt are strided per stream.  The last
// chunk is not folded: W, S end at its start state.
hipError_t launch_generic_checkpoints(const Shape& s, int chunk, const void* k, const void* v, const void* q,
                                      const float* alpha, const float* eta, const float* theta, const float* W_in,
                                      const float* S_in, float* W, float* S, int64_t state_stride, float* ckpt,
                                      int64_t ckpt_stride, float* ws, int64_t ws_stride, hipStream_t stream);

// Backward pass through the memory (generic fp32, one workgroup per stream).
constexpr int kMaxWidthBackward = 1024;
bool backward_supported(const Shape& s, int chunk);
int64_t backward_ws_floats_per_stream(const Shape& s, int chunk);
hipError_t launch_backward(const Shape& s, int chunk, const void* k, const void* v, const void* q,
                           const float* alpha, const float* eta, const float* theta, const float* W_in,
                           const float* S_in, const float* dy, const float* dW_out, const float* dS_out, float* dk,
                           float* dv, float* dq, float* dalpha, float* deta, float* dtheta, float* dW_in,
                           float* dS_in, float* ws, hipStream_t stream);

// Input side (x -> k, v, q and the gates): bf16 MFMA GEMM with a fused
// convolution / SiLU / l2-norm / sigmoid epilogue.
bool input_supported(int D, int H, int d, int w);
int64_t input_grid(int64_t R, int D, int H, int d, int w);
hipError_t launch_input(int B, int N, int D, int H, int d, int w, const void* x, const void* w_proj,
                        const float* conv_w, const void* w_gate, const float* b_gate, const float scale[3],
                        void* const kvq[3], float* const gates[3], hipStream_t stream);

// The gated delta memory (token-exact linear memory).  W [B,H,d,d] fp32;
// lengths may be null.  W_out == W_in is allowed.
constexpr int kMaxWidthDelta = 128;
constexpr int64_t kMaxStreamsDelta = 1 << 20;   // every launch stays under 2^32 threads
struct DeltaShape {
  int B, H, Hk, N, d, io;
  unsigned flags;
};
hipError_t launch_delta_recurrent(const DeltaShape& s, const void* k, const void* v, const void* q,
                                  const float* alpha, const float* theta, const int32_t* lengths, const float* W_in,
                                  void* y, float* W_out, hipStream_t stream);
// Chunks of 32 tokens on the matrix cores, for sequences of 12 tokens or more:
// one border for all.  bf16 alone would change over at 8 to 11 tokens, fp32 at
// 12 to 15.  11 and 16 tokens one by one against a chunk of up to 32, in us:
//   bf16  d 64, 512 streams   15  19  15    fp32  d 64, 512 streams   16  21  17
//         d 64, 2048          61  82  52          d 64, 2048          49  67  63
//         d 96, 512           40  53  31          d 96, 512           33  44  40
//         d 128, 128          15  19  11          d 128, 128          13  18  14
//         d 128, 2048        178 245 138          d 128, 2048        167 225 198
constexpr int kMinTokensDeltaChunked = 12;
hipError_t launch_delta_chunked(const DeltaShape& s, const void* k, const void* v, const void* q, const float* alpha,
                                const float* theta, const int32_t* lengths, const float* W_in, void* y, float* W_out,
                                float* ws, hipStream_t stream);
int64_t delta_chunked_ws_bytes(const DeltaShape& s);

// Gradients through the gated delta memory; dy and dk, dv, dq in the io type.
bool delta_backward_supported(const DeltaShape& s);
int64_t delta_backward_ws_bytes(const DeltaShape& s);
hipError_t launch_delta_backward(const DeltaShape& s, const void* k, const void* v, const void* q, const float* alpha,
                                 const float* theta, const int32_t* lengths, const float* W_in, const void* dy,
                                 const float* dW_out, void* dk, void* dv, void* dq, float* dalpha, float* dtheta,
                                 float* dW_in, float* ws, hipStream_t stream);

// Group norm with an activation (one head's d channels of a token a group)
// and its gradient.  gate, weight, bias and lengths may be null; first: x is
// [B,H,N,d], else [B,N,H d].
constexpr int kMaxWidthNorm = 1024;
constexpr int kMaxHeadsNorm = 65535;   // a grid's second dimension
struct NormShape {
  int B, H, N, d, io, silu, first;
  float eps;
};
int64_t norm_backward_ws_bytes(const NormShape& s);
hipError_t launch_group_norm(const NormShape& s, const void* x, const void* gate, const float* weight,
                             const float* bias, const int32_t* lengths, void* out, hipStream_t stream);
hipError_t launch_group_norm_backward(const NormShape& s, const void* x, const void* gate, const float* weight,
                                      const float* bias, const int32_t* lengths, const void* dout, void* dx,
                                      void* dgate, float* dweight, float* dbias, float* ws, hipStream_t stream);

// Causal attention over prompts, its gradient, and single tokens over a cache.
// packed: one row of N tokens, cut by offsets (then B sequences); last: heads
// behind tokens.  window is 0 or less than N, prefix at most N.
constexpr int kMaxWidthAttention = 128;
constexpr int64_t kMostBlocks = 1 << 24;   // of 256 threads: a launch stays under 2^32
struct AttentionShape {
  int B, H, Hk, N, d, io, window, prefix, packed, last;
  float scale;
};
bool attention_supported(const AttentionShape& s);
hipError_t launch_attention(const AttentionShape& s, const void* q, const void* k, const void* v,
                            const int32_t* offsets, const int32_t* lengths, void* out, float* lse,
                            hipStream_t stream);
int64_t attention_backward_ws_bytes(const AttentionShape& s);
hipError_t launch_attention_backward(const AttentionShape& s, const void* q, const void* k, const void* v,
                                     const int32_t* offsets, const int32_t* lengths, const void* out, const float* lse,
                                     const void* dout, void* dq, void* dk, void* dv, float* ws, hipStream_t stream);
// n new tokens a sequence over a cache of C; k_new and v_new are both null or
// both there.  window is 0 or less than C, prefix at most C.
constexpr int kMostRoom = 0x7fffffff - 31;   // the end of the last tile of 32 keys is an int, too
struct AttentionStepShape {
  int B, H, Hk, n, C, d, io, window, prefix;
  float scale;
};
bool attention_step_supported(const AttentionStepShape& s);
int64_t attention_step_ws_bytes(const AttentionStepShape& s);
hipError_t launch_attention_step(const AttentionStepShape& s, const void* q, void* k, void* v, const void* k_new,
                                 const void* v_new, const int32_t* lengths, void* out, float* ws, hipStream_t stream);

// A matrix product with bias, activation and residual, M rows from K to O
// channels, and its gradient.  bias, residual and pre may be null.
struct ProjectionShape {
  int64_t M;
  int K, O, io, silu;
};
bool projection_supported(const ProjectionShape& s, bool backward);
hipError_t launch_projection(const ProjectionShape& s, const void* x, const void* weight, const float* bias,
                             const void* residual, void* out, void* pre, hipStream_t stream);
int64_t projection_backward_ws_bytes(const ProjectionShape& s);
hipError_t launch_projection_backward(const ProjectionShape& s, const void* x, const void* weight, const void* pre,
                                      const void* dout, void* dx, float* dweight, float* dbias, void* ws,
                                      hipStream_t stream);

}  // namespace titans
