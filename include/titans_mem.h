/*
 * titans_mem.h -- C ABI of the MI355X (gfx950) Titans neural long-term memory.
 *
 * One call runs the memory's whole hot path over a batch of independent
 * (batch, head) streams: the chunked test-time update and per-token retrieval
 * of "Titans: Learning to Memorize at Test Time" (mer.dev notes):
 *
 *   loss      l(M; x_t) = ||M(k_t) - v_t||^2          section 3.1, "Objective"
 *   surprise  S_t = eta_t S_{t-1} - theta_t grad l    section 3.1, "Learning
 *                                                      Process and Surprise Metric"
 *   write     M_t = (1 - alpha_t) M_{t-1} + S_t        section 3.1, "Forgetting
 *                                                      Mechanism"
 *   read      y_t = M*(q_t), no weight change          section 3.1, "Retrieving
 *                                                      a Memory"
 *   chunking  gradients of a chunk of b tokens taken at the chunk-start
 *             weights M_{t'}                           section 3.2, "How to
 *                                                      Parallelize ..."
 *
 * The memory M is a matrix W (n_layers == 1, M(k) = W k) or a bias-free MLP
 * (n_layers >= 2) d -> hidden -> ... -> hidden -> d with SiLU after every
 * layer but the last (section 3.1 "Memory Architecture"; block details in
 * section 4.4 use SiLU).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - All tensors are contiguous and row-major.  Streams are indexed
 *   s = b * H + h.  Token rows are [N, d] per stream.
 * - Parameter layout per stream: layers 1..L concatenated, layer l stored
 *   row-major as [n_l x n_{l-1}] (column-vector convention M(k) = W k); S
 *   has the same layout.  P = sum_l n_l n_{l-1} (titans_mem_param_count).
 * - The gradient used is (M(k) - v) dM/dW, i.e. the gradient of
 *   0.5 ||M(k) - v||^2, the scale section 3.2 prints for the linear case.
 *   Pass 2*theta for the gradient of ||.||^2 itself (theta enters linearly).
 * - Tokens are 0-indexed; chunk c covers [c*chunk, min((c+1)*chunk, N)) and
 *   differentiates at the state left by the previous chunk.  N need not be
 *   a multiple of chunk: the last chunk is shorter.
 * - Gates are not range-checked; non-finite values propagate.
 * - Device pointers must be 16-byte aligned.
 * - Calls are asynchronous on `stream` (a hipStream_t; NULL = the default
 *   stream): they return after enqueueing and never synchronise.  Argument
 *   errors (codes -1..-4) are detected on the host before anything is
 *   enqueued, so they can be tested without a GPU.
 * - The library allocates no device memory at run time; the caller owns
 *   every buffer.  (The scratch of titans_mem_forward_noalloc is a device
 *   array of the library's code object, present once per GPU from load.)
 * - Process-wide state: per device, one HIP stream of the library's own
 *   (default priority) and six events, created on the first call that needs
 *   them and kept until the process ends.  The shape-generic forward (when
 *   the state does not fit on chip) and the backward run part of their work
 *   there, forked from and joined back into the caller's `stream` with
 *   events, on every return path; a mutex serialises the enqueueing of such
 *   calls.  Calls are thread-safe.
 */
#ifndef TITANS_MEM_H
#define TITANS_MEM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define TITANS_MEM_ABI_VERSION 1

/* status codes */
#define TM_OK               0
#define TM_ERR_INVALID     -1  /* null pointer, dimension <= 0, chunk <= 0, misaligned pointer, bad enum, wrong abi_version */
#define TM_ERR_UNSUPPORTED -2  /* shape / dtype / flag combination the library has no kernel for */
#define TM_ERR_WORKSPACE   -3  /* workspace smaller than titans_mem_workspace_bytes() */
#define TM_ERR_ALIAS       -4  /* illegal overlap between buffers */
#define TM_ERR_HIP         -5  /* the HIP runtime reported an error when launching */
#define TM_ERR_GAVE_UP     -6  /* titans_mem_workspace_status: the MFMA kernel's paired
                                  workgroups gave up waiting for each other; the call's
                                  y, W_out and S_out hold NaN */

/* dtype of k, v, q and y (the io tensors); state and gates are always fp32 */
#define TM_IO_F32  0
#define TM_IO_BF16 1

#define TM_ACT_SILU 0
#define TM_ACT_NONE 1   /* titans_mem_group_norm only */

/* which state retrieval reads (section 3.1 "Retrieving a Memory" has no
 * time index; the write-then-read memory view of section 2.1 reads M_t) */
#define TM_READ_AFTER_WRITE 0  /* y_t = M_{W_t}(q_t): the state after token t's write */
#define TM_READ_CHUNK_START 1  /* y_t = M_{W_t'}(q_t): the state at the start of t's chunk */

/* flags */
#define TM_FLAG_FORCE_GENERIC 1u  /* run the shape-generic fp32 kernel even where a specialised one exists */
#define TM_FLAG_CHUNK_GATES   2u  /* alpha, eta, theta hold one value per chunk, [B,H,ceil(N/chunk)],
                                     shared by the chunk's tokens ("Titans: Learning to Memorize at
                                     Test Time", mer.dev notes, section 3.2 "Parameters as the
                                     Function of Chunks": inside a chunk the update is then
                                     time-invariant) */
#define TM_FLAG_NO_WAIT       4u  /* test hook for the failure path of the MFMA kernel: its paired
                                     workgroups give up at their first wait for each other, so the
                                     call ends normally with NaN outputs and the give-up status
                                     (ignored by the other kernels) */

/* kernel paths reported by titans_mem_select_path */
#define TM_PATH_GENERIC_F32   0   /* any shape: fp32 (matrix instructions), state in global memory */
#define TM_PATH_MLP2_D64_H256 1   /* 2-layer, d=64, hidden=256, chunk<=64, bf16 io, either read mode:
                                     MFMA, register-resident state */
#define TM_PATH_DEEP_BF16     2   /* MLP (n_layers >= 2) with d and hidden multiples of 64, chunk<=256,
                                     bf16 io, N >= 1, either read mode: bf16 MFMA products with fp32
                                     sums, fp32 state in W_out/S_out; every step of a chunk one launch
                                     over all streams, the reads on the library's second stream */

typedef struct {
    int32_t abi_version;  /* must equal TITANS_MEM_ABI_VERSION */
    int32_t B, H, N;      /* batch, heads, tokens per stream (N >= 0) */
    int32_t d;            /* key = value = query width */
    int32_t hidden;       /* MLP width; ignored when n_layers == 1 */
    int32_t n_layers;     /* 1 = linear memory W (d x d); >= 2 = MLP */
    int32_t activation;   /* TM_ACT_SILU */
    int32_t io_dtype;     /* TM_IO_F32 or TM_IO_BF16 */
    int32_t read_mode;    /* TM_READ_AFTER_WRITE or TM_READ_CHUNK_START */
    uint32_t flags;       /* TM_FLAG_* */
} titans_mem_desc;

/* ABI version this library was built with. */
int32_t titans_mem_abi_version(void);

/* Parameters per stream (P), or a negative status for an invalid shape. */
int64_t titans_mem_param_count(const titans_mem_desc* desc);

/* Kernel path titans_mem_forward would run for (desc, chunk), or a negative
 * status (TM_ERR_INVALID / TM_ERR_UNSUPPORTED). */
int32_t titans_mem_select_path(const titans_mem_desc* desc, int32_t chunk);

/* Device workspace titans_mem_forward needs for (desc, chunk), in bytes
 * (0 when the selected kernel needs none), or a negative status. */
int64_t titans_mem_workspace_bytes(const titans_mem_desc* desc, int32_t chunk);

/*
 * titans_mem_forward -- chunked update plus retrieval over all B*H streams.
 *
 *   k, v, q    [B,H,N,d]  io dtype, device, read-only
 *   alpha, eta, theta  [B,H,N] fp32, device, read-only: forgetting gate,
 *              surprise decay, momentary-surprise weight
 *              ([B,H,ceil(N/chunk)] with TM_FLAG_CHUNK_GATES)
 *   W_in, S_in [B,H,P]  fp32, device, read-only: memory weights and
 *              surprise momentum before token 0
 *   chunk      b >= 1: tokens per chunk (gradients at the chunk-start state)
 *   y_out      [B,H,N,d]  io dtype, device, written: y_t per token
 *              (computed in fp32, rounded once to nearest-even)
 *   W_out, S_out [B,H,P] fp32, device, written: state after token N-1.
 *              W_out == W_in and/or S_out == S_in (exact in-place) is
 *              allowed; any other overlap among all buffers is TM_ERR_ALIAS.
 *   workspace  device scratch of at least titans_mem_workspace_bytes(desc,
 *              chunk) bytes (may be NULL when that is 0); its contents on
 *              entry do not matter and are undefined on return.
 *   stream     hipStream_t to enqueue on (NULL = default stream).  On the
 *              deep-memory path (TM_PATH_DEEP_BF16), and on the
 *              shape-generic kernel when the state does not fit on chip
 *              and chunk >= 16 (and the call is not in place), part of the
 *              work (the retrieval) runs on a second stream of the
 *              library's own (one per device, default priority), ordered
 *              against `stream` with events and joined back into it before
 *              the call's work ends.
 *
 * Returns TM_OK or a negative status.  Resuming: passing (W_out, S_out) of
 * a call as (W_in, S_in) of the next, with a split on a chunk boundary,
 * continues the same sequence.
 *
 * The MFMA path (TM_PATH_MLP2_D64_H256) runs each stream on two workgroups
 * that wait for each other every chunk.  Both must be resident at once; the
 * launch sizes its grid to half the device's CUs, but work that other
 * streams or processes keep on the CUs can hold one back.  A workgroup whose
 * partner does not arrive within a bounded wait (about 2^21 polls) gives up
 * instead of hanging: the call still completes, y, W_out and S_out of the
 * pair's streams hold NaN, and titans_mem_workspace_status reports
 * TM_ERR_GAVE_UP.
 */
int titans_mem_forward(const titans_mem_desc* desc,
                       const void* k, const void* v, const void* q,
                       const float* alpha, const float* eta, const float* theta,
                       const float* W_in, const float* S_in,
                       int32_t chunk,
                       void* y_out, float* W_out, float* S_out,
                       void* workspace, int64_t workspace_bytes,
                       void* stream);

/*
 * titans_mem_forward_noalloc -- titans_mem_forward for callers that cannot
 * allocate device memory or pass a workspace (code under HIP graph capture,
 * tight serving loops, harnesses that forbid allocation).
 *
 * Same arguments, results and asynchrony as titans_mem_forward without the
 * workspace, for the shapes of the MFMA path (TM_PATH_MLP2_D64_H256:
 * 2-layer, d = 64, hidden = 256, bf16 io, chunk <= 64; any B*H, N and read
 * mode); TM_ERR_UNSUPPORTED for every other shape.  Its scratch (the
 * workgroups' tagged exchange and hand-over words and the status word) is a
 * library-owned device array of 42,467,584 bytes (40.5 MiB + 256: enough for
 * the kernel's largest grids, 128 workgroup pairs or, with at most 64
 * streams, 64 groups of four workgroups; TM_ERR_WORKSPACE if a shape ever
 * needed more), one per GPU,
 * allocated with the library's code and held until the process ends.  The
 * call allocates nothing: it enqueues a small fill kernel and the memory
 * kernel on `stream`.  The first call on a device looks up the array's
 * address there.  All calls on one GPU share the array: calls that follow
 * one another on a stream are independent, calls that overlap in time on one
 * GPU (other streams, other threads) race and must not be issued.
 * titans_mem_workspace_status with workspace NULL reports on the last such
 * call on the current device.
 */
int titans_mem_forward_noalloc(const titans_mem_desc* desc,
                               const void* k, const void* v, const void* q,
                               const float* alpha, const float* eta, const float* theta,
                               const float* W_in, const float* S_in,
                               int32_t chunk,
                               void* y_out, float* W_out, float* S_out,
                               void* stream);

/*
 * titans_mem_workspace_status -- outcome of the last titans_mem_forward call
 * that used `workspace` (same desc and chunk).  Waits for `stream` to drain
 * (hipStreamSynchronize) and reads the status word the MFMA kernel keeps in
 * its workspace.
 *
 * Returns TM_OK when the call completed, TM_ERR_GAVE_UP when paired
 * workgroups of the MFMA kernel gave up waiting for each other (its outputs
 * hold NaN), an argument error (-1..-3) like titans_mem_forward's, or
 * TM_ERR_HIP when the copy or the synchronisation fails.  Paths without
 * cross-workgroup waits always report TM_OK.  workspace NULL stands for the
 * scratch of titans_mem_forward_noalloc on the current device.
 */
int titans_mem_workspace_status(const titans_mem_desc* desc, int32_t chunk,
                                const void* workspace, int64_t workspace_bytes,
                                void* stream);

/*
 * titans_mem_retrieve -- pure retrieval y = M*_W(q) at a fixed state
 * (section 3.1 "Retrieving a Memory": a forward pass without weight
 * adjustment), e.g. a lookup after a context has been consumed.
 *
 *   q      [B,H,N,d] io dtype, device
 *   W      [B,H,P]   fp32, device (the state to read)
 *   y_out  [B,H,N,d] io dtype, device, must not overlap q or W
 * Uses desc's shape fields; read_mode is ignored.  The 2-layer d=64
 * hidden=256 bf16 memory runs on the matrix cores (bf16 operands, fp32 sums);
 * every other shape, and any call with TM_FLAG_FORCE_GENERIC, on the
 * shape-generic fp32 kernel (widths up to 1024).
 */
int titans_mem_retrieve(const titans_mem_desc* desc, const void* q, const float* W,
                        void* y_out, void* stream);

/*
 * titans_mem_backward -- gradients through titans_mem_forward, for training
 * what produces the memory's inputs (section 3.1, "Objective": the memory's
 * weights are fitted in an inner loop at test time; the rest of the model
 * learns in an outer loop, through the memory).
 *
 * Returns the vector-Jacobian products of the forward map (same desc,
 * inputs and chunk as the forward call) with the output adjoints:
 *   dy               [B,H,N,d] fp32, device, or NULL (zero): dL/dy
 *   dW_out, dS_out   [B,H,P] fp32, device, or NULL (zero): dL/dW_out, dL/dS_out
 * into
 *   dk, dv, dq       [B,H,N,d] fp32, device, written
 *   dalpha, deta, dtheta  [B,H,N] fp32 ([B,H,ceil(N/chunk)] with
 *                    TM_FLAG_CHUNK_GATES), device, written
 *   dW_in, dS_in     [B,H,P] fp32, device, written
 * The derivative includes the second-order term of the chunk-start
 * gradients (each token's inner gradient depends on W at its chunk start).
 * Both read modes.  Arithmetic is fp32 whatever the io dtype (bf16 inputs
 * are read exactly).  Outputs must not overlap each other or any input.
 * Supported: every layer width a multiple of 4, at most 1024, N >= 1,
 * chunk <= 4096 (TM_ERR_UNSUPPORTED otherwise).
 * The workspace holds (W, S) at every chunk start and two chunks' token
 * vectors: titans_mem_backward_workspace_bytes(desc, chunk) bytes.
 * The work is ordered on `stream`; part of it runs on a second stream of
 * the library's own (one per device, created on the first call, default
 * priority), forked from and joined back into `stream` with events, so
 * work enqueued on `stream` after the call sees every result.
 */
int64_t titans_mem_backward_workspace_bytes(const titans_mem_desc* desc, int32_t chunk);

int titans_mem_backward(const titans_mem_desc* desc,
                        const void* k, const void* v, const void* q,
                        const float* alpha, const float* eta, const float* theta,
                        const float* W_in, const float* S_in, int32_t chunk,
                        const float* dy, const float* dW_out, const float* dS_out,
                        float* dk, float* dv, float* dq,
                        float* dalpha, float* deta, float* dtheta,
                        float* dW_in, float* dS_in,
                        void* workspace, int64_t workspace_bytes, void* stream);

/*
 * titans_mem_input -- the step before the memory: model activations x to
 * the memory's keys, values, queries and gates, for whole sequences.
 *
 * Per sequence b, token t, head h (mer.dev notes):
 *   projections  k = x W_K, v = x W_V      section 3.1, "Objective"
 *                q = x W_Q                 section 3.1, "Retrieving a Memory"
 *   convolution  causal depthwise over time after each projection, width w:
 *                u_t[c] = sum_{j<w} conv_w[c][j] * proj_{t-j}[c], tokens before
 *                the sequence start count as zero   section 4.4, "Convolution"
 *   activation   SiLU on k, v and q; k and q divided by their l2 norm over
 *                the head's d channels (floored at 1e-6)
 *                                          section 4.4, "Architectural Details"
 *   gates        alpha, eta, theta = scale_g * sigmoid(x . w_gate[g][h] +
 *                b_gate[g][h]): per token and head, input dependent
 *                                          section 3.1, "Learning Process and
 *                                          Surprise Metric"
 * There are no projection biases.  Arithmetic: bf16 x bf16 products, fp32
 * sums and epilogue, k, v, q rounded once to bf16 (nearest-even).
 *
 *   x          [B,N,D]     bf16, device, read-only
 *   w_proj     [3,H*d,D]   bf16, device: rows of W_K, then W_V, then W_Q;
 *              channel c of head h is row h*d + c (out = x . row)
 *   conv_w     [3,H*d,w]   fp32, device: tap j weighs the token j steps back
 *   w_gate     [3,H,D]     bf16, device: logit weights of alpha, eta, theta
 *   b_gate     [3,H]       fp32, device: logit biases
 *   *_scale    host scalars multiplying the three sigmoids
 *   k_out, v_out, q_out  [B,H,N,d] bf16, device, written (the layout
 *              titans_mem_forward reads)
 *   alpha_out, eta_out, theta_out  [B,H,N] fp32, device, written
 * Supported: D a positive multiple of 32, d in {16, 32, 64, 128}, H*d a
 * multiple of 128, 1 <= w <= 4 (else TM_ERR_UNSUPPORTED).  Outputs must not
 * overlap each other or any input (TM_ERR_ALIAS).  N == 0 enqueues nothing.
 */
typedef struct {
    int32_t abi_version;  /* must equal TITANS_MEM_ABI_VERSION */
    int32_t B, N;         /* sequences, tokens per sequence (N >= 0) */
    int32_t D;            /* model width */
    int32_t H, d;         /* heads, head width */
    int32_t conv_width;   /* w: causal depthwise taps */
    uint32_t flags;       /* must be 0 */
} titans_input_desc;

int titans_mem_input(const titans_input_desc* desc,
                     const void* x, const void* w_proj, const float* conv_w,
                     const void* w_gate, const float* b_gate,
                     float alpha_scale, float eta_scale, float theta_scale,
                     void* k_out, void* v_out, void* q_out,
                     float* alpha_out, float* eta_out, float* theta_out,
                     void* stream);

/*
 * titans_mem_delta_forward -- the gated delta memory: the linear memory
 * M(k) = W k updated after every token, without momentum, its residual taken
 * at the decayed memory of the token before.  Per stream and token:
 *
 *   f_t = v_t - (1 - alpha_t) W_{t-1} k_t      section 3.1, "Objective"
 *   W_t = (1 - alpha_t) W_{t-1} + theta_t f_t k_t^T   "Forgetting Mechanism"
 *   y_t = W_t q_t                              "Retrieving a Memory"
 *
 * Unlike titans_mem_forward's linear memory (gradients at the chunk's start)
 * this is the token-by-token rule at every length; the chunks of the chunked
 * kernel are an implementation detail that no result depends on.
 *
 *   k, q       [B,Hk,N,d]  io dtype, device, read-only; value head h reads
 *              key head h / (H / Hk)
 *   v          [B,H,N,d]   io dtype, device, read-only
 *   alpha, theta  [B,H,N]  fp32, device, read-only: forgetting gate
 *              (alpha <= 1; 1 forgets everything; NaN comes out of more)
 *              and step size
 *   lengths    [B] int32, device, read-only, or NULL (all N): tokens of each
 *              sequence, clamped to 0..N.  Later tokens are not read, their
 *              rows of y_out are left as they were, and W_out is the state
 *              after the last token of its sequence (W_in for length 0).
 *   W_in, W_out  [B,H,d,d] fp32, device, row-major [n_out x n_in]; W_out ==
 *              W_in (exact in-place) is allowed, any other overlap of a
 *              written buffer is TM_ERR_ALIAS.  In place the states of
 *              sequences of length 0 are not written: calls on several
 *              streams may share one state, if no sequence has tokens in two
 *   y_out      [B,H,N,d]   io dtype, device, written
 *   workspace  titans_mem_delta_workspace_bytes(desc) bytes of device
 *              scratch (may be NULL when that is 0)
 *
 * State, sums and gates are fp32; products of bf16 inputs are exact.  y is
 * rounded once.  d <= 128 and B*H <= 2^20 (TM_ERR_UNSUPPORTED otherwise);
 * N == 0 copies the state.  Where chunks are used, a NaN or infinity of a
 * token may reach the 31 tokens before it (of its stream) too, and the product
 * of 1 - alpha over up to 32 tokens in a row has to be a finite float (a gate
 * never makes it larger than 1; a negative alpha can, and multiplies rounding
 * errors by up to that product).  TM_FLAG_FORCE_GENERIC runs the
 * token-by-token kernel at any N.  titans_mem_delta_select_path reports the
 * kernel that a call runs.
 */
#define TM_PATH_DELTA_RECURRENT 0   /* token by token */
#define TM_PATH_DELTA_CHUNKED   1   /* by chunks, on the matrix cores */

typedef struct {
    int32_t abi_version;  /* must equal TITANS_MEM_ABI_VERSION */
    int32_t B, H, Hk;     /* batch, value heads, key heads (Hk divides H) */
    int32_t N, d;         /* tokens per sequence (N >= 0), width of k, v, q */
    int32_t io_dtype;     /* TM_IO_F32 or TM_IO_BF16 */
    uint32_t flags;       /* 0 or TM_FLAG_FORCE_GENERIC */
} titans_delta_desc;

int32_t titans_mem_delta_select_path(const titans_delta_desc* desc);
int64_t titans_mem_delta_workspace_bytes(const titans_delta_desc* desc);

int titans_mem_delta_forward(const titans_delta_desc* desc,
                             const void* k, const void* v, const void* q,
                             const float* alpha, const float* theta,
                             const int32_t* lengths, const float* W_in,
                             void* y_out, float* W_out,
                             void* workspace, int64_t workspace_bytes,
                             void* stream);

/*
 * titans_mem_delta_backward -- gradients through titans_mem_delta_forward:
 * the vector-Jacobian products with the output adjoints
 *   dy         [B,H,N,d]   io dtype, device, read-only: dL/dy
 *   dW_out     [B,H,d,d]   fp32, device, read-only, or NULL (zero)
 * into
 *   dk, dq     [B,Hk,N,d]  io dtype, device, written: sums over the value
 *              heads of a key head, in their order
 *   dv         [B,H,N,d]   io dtype, device, written
 *   dalpha, dtheta  [B,H,N] fp32, device, written
 *   dW_in      [B,H,d,d]   fp32, device, written
 * Same inputs as the forward call.  Tokens past a sequence's length get zero
 * gradients, whatever dy holds there.  At alpha = 1 dalpha is the derivative
 * there.  Arithmetic is fp32; dk, dv and dq are rounded once.  Any overlap of
 * a written buffer is TM_ERR_ALIAS.  The workspace holds W and its adjoint at
 * every 32nd token: titans_mem_delta_backward_workspace_bytes(desc) bytes.
 * TM_ERR_UNSUPPORTED from B*Hk*ceil(N/32) = 2^24 on (2^23 where d > 64).
 */
int64_t titans_mem_delta_backward_workspace_bytes(const titans_delta_desc* desc);

int titans_mem_delta_backward(const titans_delta_desc* desc,
                              const void* k, const void* v, const void* q,
                              const float* alpha, const float* theta,
                              const int32_t* lengths, const float* W_in,
                              const void* dy, const float* dW_out,
                              void* dk, void* dv, void* dq,
                              float* dalpha, float* dtheta, float* dW_in,
                              void* workspace, int64_t workspace_bytes,
                              void* stream);

/*
 * titans_mem_group_norm -- group norm with an activation, from the memory's
 * y to the channels-last rows that a block's output projection reads
 * (section 4.4, "Architectural Details": normalization and gating before the
 * output projection).  A group is one head's d channels of one token:
 *
 *   n = (x - mean) / sqrt(var + eps) * weight + bias
 *   out = act(gate) * n  with a gate,  act(n)  without one
 *
 * act is SiLU (TM_ACT_SILU) or the identity (TM_ACT_NONE); var is the mean
 * of the squared deviations.
 *
 *   x          [B,H,N,d] io dtype, device, read-only (the layout of y); with
 *              TM_FLAG_CHANNELS_LAST [B,N,H*d]
 *   gate       [B,N,H*d] io dtype, device, read-only, or NULL
 *   weight, bias  [H*d] fp32, device, read-only, or NULL (ones, zeros)
 *   lengths    [B] int32, device, read-only, or NULL (all N): later tokens
 *              are neither read nor written
 *   out        [B,N,H*d] io dtype, device, written
 * Sums and the normalised values are fp32; out is rounded once.
 * Supported: d <= 1024, H <= 65535 (TM_ERR_UNSUPPORTED otherwise), eps >= 0.
 * Any overlap of out with an input is TM_ERR_ALIAS.
 */
#define TM_FLAG_CHANNELS_LAST 8u   /* titans_mem_group_norm: x is [B,N,H*d] */

typedef struct {
    int32_t abi_version;  /* must equal TITANS_MEM_ABI_VERSION */
    int32_t B, H, N, d;   /* batch, groups, tokens (N >= 0), channels per group */
    int32_t io_dtype;     /* TM_IO_F32 or TM_IO_BF16 */
    int32_t activation;   /* TM_ACT_SILU or TM_ACT_NONE */
    float eps;
    uint32_t flags;       /* 0 or TM_FLAG_CHANNELS_LAST */
} titans_norm_desc;

int titans_mem_group_norm(const titans_norm_desc* desc, const void* x,
                          const void* gate, const float* weight,
                          const float* bias, const int32_t* lengths,
                          void* out, void* stream);

/*
 * titans_mem_group_norm_backward -- its vector-Jacobian products with
 *   dout       [B,N,H*d] io dtype, device, read-only: dL/dout
 * into
 *   dx         x's layout, io dtype, device, written
 *   dgate      [B,N,H*d] io dtype, device, written (NULL iff gate is NULL)
 *   dweight, dbias  [H*d] fp32, device, written (also where weight and bias
 *              are NULL)
 * Rows past a sequence's length get zero gradients and add nothing to
 * dweight and dbias, which are summed in a fixed order.  Any overlap of a
 * written buffer is TM_ERR_ALIAS.
 */
int64_t titans_mem_group_norm_backward_workspace_bytes(const titans_norm_desc* desc);

int titans_mem_group_norm_backward(const titans_norm_desc* desc, const void* x,
                                   const void* gate, const float* weight,
                                   const float* bias, const int32_t* lengths,
                                   const void* dout, void* dx, void* dgate,
                                   float* dweight, float* dbias,
                                   void* workspace, int64_t workspace_bytes,
                                   void* stream);

/*
 * titans_mem_attention -- causal softmax attention over whole prompts: the
 * short-term memory that the architectures set beside the neural one (section
 * 2.1 for the formula, 4.2 "Memory as a Gate" and 4.3 for the sliding window
 * over persistent tokens and the sequence).  Token i of a sequence sees token
 * j of it where
 *
 *   j <= i  and  (window == 0  or  i - j < window  or  j < prefix)
 *
 *   lse_i = log sum_j exp(scale q_i . k_j),  out_i = sum_j exp(scale q_i . k_j - lse_i) v_j
 *
 * The first `prefix` tokens of a sequence are the persistent ones.
 *
 *   q          [B,H,N,d]   io dtype, device, read-only
 *   k, v       [B,Hk,N,d]  io dtype, device, read-only; query head h reads
 *              key head h / (H / Hk)
 *              with TM_FLAG_CHANNELS_LAST [B,N,H*d] and [B,N,Hk*d]
 *   offsets    [B+1] int32, device, read-only, or NULL.  With it the tensors
 *              hold one row of N tokens ([H,N,d]; [N,H*d] with the flag), and
 *              sequence s is its tokens offsets[s] .. offsets[s+1] - 1, in
 *              order, clamped to 0..N
 *   lengths    [B] int32, device, read-only, or NULL (all N; NULL with
 *              offsets): tokens of each sequence, clamped to 0..N
 *   out        [B,N,H*d]   ([N,H*d]) io dtype, device, written: channels last
 *              in either layout, as titans_mem_group_norm reads a gate
 *   lse        [B,H,N] ([H,N]) fp32, device, written, or NULL
 *
 * Tokens of no sequence are not read, and their rows of out and lse are left
 * as they were.  Sums and the softmax are fp32; for bf16 tensors the weights
 * are rounded to bf16 before they meet v, and out is rounded once.  A NaN or
 * infinity in v may reach other queries too that come up to 127 tokens
 * before it, or that it is out of the window of by up to 190.  An infinity in
 * an fp32 q or k is a NaN in the scores that it is part of.  Scores may be up to
 * 2^29 either way; behind that NaN may come out.
 * d <= 128, 0 < scale <= 2e38 (TM_ERR_UNSUPPORTED, TM_ERR_INVALID otherwise);
 * H d <= 2^22, and fewer than 2^24 tiles of 32 tokens of a query head: B H
 * ceil(N / 32), or H (N / 32 + B) with offsets (TM_ERR_UNSUPPORTED).
 */
typedef struct {
    int32_t abi_version;  /* must equal TITANS_MEM_ABI_VERSION */
    int32_t B, H, Hk;     /* sequences, query heads, key heads (Hk divides H) */
    int32_t N, d;         /* tokens of a row (N >= 0), width of a head */
    int32_t io_dtype;     /* TM_IO_F32 or TM_IO_BF16 */
    int32_t window;       /* 0: all tokens before */
    int32_t prefix;       /* tokens that every later one sees (>= 0) */
    float scale;          /* of the scores, 1/sqrt(d) as a rule */
    uint32_t flags;       /* 0 or TM_FLAG_CHANNELS_LAST */
} titans_attention_desc;

int titans_mem_attention(const titans_attention_desc* desc, const void* q,
                         const void* k, const void* v, const int32_t* offsets,
                         const int32_t* lengths, void* out, float* lse,
                         void* stream);

/*
 * titans_mem_attention_backward -- gradients through titans_mem_attention:
 * the vector-Jacobian products with
 *   out, lse         what the forward call wrote, device, read-only
 *   dout             out's layout, io dtype, device, read-only: dL/dout
 * into
 *   dq, dk, dv       the layouts of q, k and v, io dtype, device, written; dk
 *                    and dv are sums over the query heads of a key head
 * Same inputs as the forward call.  Tokens of no sequence get zero gradients.
 * Sums are fp32 and in a fixed order; for bf16 tensors the weights and their
 * derivatives are rounded to bf16 before they meet q, k and dout, and results
 * once.  Weights are formed from lse, whose rounding they carry (2^-22 of its
 * size, relative to them).  A NaN or infinity in q, k, v or dout may reach the
 * gradients of the 255 tokens before it and behind it too, and in q or dout,
 * where there is a window, those of the 31 tokens behind the persistent ones.
 * Any overlap of a written buffer is TM_ERR_ALIAS.
 * packed: whether the call has offsets.
 */
int64_t titans_mem_attention_backward_workspace_bytes(const titans_attention_desc* desc, int32_t packed);

int titans_mem_attention_backward(const titans_attention_desc* desc,
                                  const void* q, const void* k, const void* v,
                                  const int32_t* offsets, const int32_t* lengths,
                                  const void* out, const float* lse, const void* dout,
                                  void* dq, void* dk, void* dv,
                                  void* workspace, int64_t workspace_bytes,
                                  void* stream);

/*
 * titans_mem_attention_step -- the attention of N new tokens a sequence (one,
 * as a rule) over a cache of what came before them.  Row b's cache has
 * lengths[b] tokens, the new ones the last N among them: new token i is token
 * lengths[b] - N + i of the sequence, and sees what titans_mem_attention's
 * mask lets it see.
 *
 *   q          [B,H,N,d]   io dtype, device, read-only
 *   k, v       [B,Hk,C,d]  io dtype, device: the cache, room for C tokens
 *   k_new, v_new  [B,Hk,N,d] io dtype, device, read-only, or both NULL.  With
 *              them the call stores the new tokens' keys and values at their
 *              places; without them the cache holds them already
 *   lengths    [B] int32, device, read-only, clamped to 0..C
 *   out        [B,N,H*d]   io dtype, device, written; zeros for a token whose
 *              place would be before the first (an idle row has length 0)
 * Nothing else of the cache is written, and nothing past a length is read.
 * Arithmetic and limits as in titans_mem_attention, but that weights keep 16
 * bits before they meet v for bf16 tensors, and that a NaN or infinity in v may
 * reach all new tokens of its row.  A call reads the cache
 * once for every 32 of the H/Hk * N queries of a key head.  Any overlap of a
 * written buffer is TM_ERR_ALIAS (the cache is one if k_new is there).  C <=
 * 2^31 - 32, fewer than 2^24 queries (B H N) and, for every part of the cache (64
 * at most), 2^24 tiles of 32 of them (TM_ERR_UNSUPPORTED otherwise).
 */
typedef struct {
    int32_t abi_version;  /* must equal TITANS_MEM_ABI_VERSION */
    int32_t B, H, Hk;     /* sequences, query heads, key heads (Hk divides H) */
    int32_t N, C, d;      /* new tokens (N >= 0), the cache's room, width of a head */
    int32_t io_dtype;     /* TM_IO_F32 or TM_IO_BF16 */
    int32_t window, prefix;   /* as in titans_attention_desc */
    float scale;
    uint32_t flags;       /* must be 0 */
} titans_attention_step_desc;

int64_t titans_mem_attention_step_workspace_bytes(const titans_attention_step_desc* desc);

int titans_mem_attention_step(const titans_attention_step_desc* desc,
                              const void* q, void* k, void* v,
                              const void* k_new, const void* v_new,
                              const int32_t* lengths, void* out,
                              void* workspace, int64_t workspace_bytes,
                              void* stream);

/*
 * titans_mem_projection -- the projection that closes a block (section 4.4,
 * "Architectural Details": the output projection behind normalization and
 * gating, and the residual connection), its bias, activation and residual in
 * one pass:
 *
 *   z = x W^T + bias,  out = act(z) + residual
 *
 * act is SiLU (TM_ACT_SILU) or the identity (TM_ACT_NONE).
 *
 *   x          [rows,K]    io dtype, device, read-only
 *   weight     [O,K]       io dtype, device, read-only (out = x . row)
 *   bias       [O] fp32, device, read-only, or NULL
 *   residual   [rows,O]    io dtype, device, read-only, or NULL
 *   out        [rows,O]    io dtype, device, written; out == residual (exact
 *              in-place) is allowed, any other overlap is TM_ERR_ALIAS
 *   pre_out    [rows,O]    io dtype, device, written, or NULL: z, which the
 *              gradient of an activation needs
 * Products of bf16 inputs are exact, sums, bias and activation fp32, out is
 * rounded once.  fp32 products go through three bf16 numbers a factor, by
 * which each is off by 2^-22 of itself at most, of either sign (where a factor is
 * below 2^-110, as if it were off by 2^-133); a row or column of fp32 with an
 * infinity in it comes out as NaN.
 * TM_ERR_UNSUPPORTED for more than 2^22 channels, or where out (in the gradient's
 * call dx, or dweight) is too large for a launch; up to 2^22 - 8 tiles of 64 x 64
 * of it never are.
 */
typedef struct {
    int32_t abi_version;  /* must equal TITANS_MEM_ABI_VERSION */
    int32_t K, O;         /* channels in, channels out */
    int32_t io_dtype;     /* TM_IO_F32 or TM_IO_BF16 */
    int64_t rows;         /* tokens (>= 0) */
    int32_t activation;   /* TM_ACT_SILU or TM_ACT_NONE */
    uint32_t flags;       /* must be 0 */
} titans_projection_desc;

int titans_mem_projection(const titans_projection_desc* desc, const void* x,
                          const void* weight, const float* bias,
                          const void* residual, void* out, void* pre_out,
                          void* stream);

/*
 * titans_mem_projection_backward -- its vector-Jacobian products with
 *   dout       [rows,O]    io dtype, device, read-only: dL/dout
 *   pre        [rows,O]    io dtype, device, read-only: pre_out of the forward
 *              call with TM_ACT_SILU, NULL with TM_ACT_NONE
 * into
 *   dx         [rows,K]    io dtype, device, written
 *   dweight    [O,K]       fp32, device, written
 *   dbias      [O]         fp32, device, written
 * (dL/dresidual is dout.)  dz = dout act'(z) is rounded to the io dtype before
 * the product for dx; dweight takes a bf16 one's remainder along (16 bits), and
 * dbias what it was.  Sums are fp32, in a fixed order.  rows == 0 writes
 * zeros.  Any overlap of a written buffer is TM_ERR_ALIAS.
 */
int64_t titans_mem_projection_backward_workspace_bytes(const titans_projection_desc* desc);

int titans_mem_projection_backward(const titans_projection_desc* desc,
                                   const void* x, const void* weight,
                                   const void* pre, const void* dout,
                                   void* dx, float* dweight, float* dbias,
                                   void* workspace, int64_t workspace_bytes,
                                   void* stream);

/* Static text for a status code. */
const char* titans_mem_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* TITANS_MEM_H */
