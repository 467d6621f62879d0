/*
 * ssd.h -- C ABI of the SSD selective-state scan library (libssd.so, sm_103a).
 *
 * The operation (page "Mamba-2架构与LaCT并行计算技术解析", §1.1, the state
 * equations, and §1.2, independent heads): for every head h and every token t
 *
 *     delta_t = softplus(raw_dt_t + delta_init)
 *     H_t     = exp(-delta_t) * H_{t-1} + delta_t * x_t B_t^T       (H is P x N, fp32)
 *     y_t     = H_t C_t
 *
 * with H = 0 before the first token of every sequence (the zero-initial-state
 * note under the same equations).  The library evaluates it in the chunked,
 * semiseparable way of page "长序列 Mamba 多卡训练算力和显存怎么同时省" §一:
 * diagonal blocks inside each chunk, a small state passed between chunks.
 * Packed variable-length input follows the cu_seqlens convention of the same
 * page, §三: the state restarts at every sequence boundary.
 *
 * General rules for every entry point:
 *  - All tensor arguments are DEVICE pointers on the current CUDA device,
 *    contiguous, row-major, 16-byte aligned (ssd_step_host alone takes host
 *    buffers).  The caller owns every buffer; the library allocates nothing on
 *    the device and keeps no pointer after a call returns.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy
 *    default stream).  No call synchronises except the queries of a status
 *    (ssd_device_status(), ssd_forward_noalloc_status(), ssd_layer_status()).
 *  - Host-side argument checks run before any launch; on failure nothing is
 *    launched and a nonzero ssd_status_t is returned.  Errors that only the
 *    device can see (a malformed cu_seqlens array) are recorded in a status
 *    word inside the workspace and read with ssd_device_status().
 *  - Calls that share a workspace must not overlap on the GPU.
 *
 * Layouts (T = batch * seqlen tokens, H heads, P = headdim, N = dstate,
 * G = ngroups; head h reads B/C group h / (H / G)):
 *     x, y, dy, dx     [T][H][P]   dtype = problem.dtype
 *     raw_dt, d_raw_dt [T][H]      float32
 *     B, C, dB, dC     [T][G][N]   dtype = problem.dtype
 *     final_state      [nseq or batch][H][P][N] float32
 *     cu_seqlens       [nseq + 1]  int32, cu[0] = 0, cu[nseq] = T, non-decreasing
 */
#ifndef SSD_H_
#define SSD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSD_API_VERSION 1

typedef enum {
    SSD_OK = 0,
    SSD_ERR_INVALID_ARG = 1,   /* null pointer, bad size or inconsistent problem */
    SSD_ERR_UNSUPPORTED = 2,   /* valid problem outside the supported shape set */
    SSD_ERR_ALIGNMENT = 3,     /* a pointer is not 16-byte aligned (workspace: 256) */
    SSD_ERR_WORKSPACE = 4,     /* workspace missing or smaller than ssd_workspace_size(); as a
                                  device status: the workspace does not hold the forward that
                                  ssd_backward_after_forward was told to reuse */
    SSD_ERR_CUDA = 5,          /* a CUDA runtime call failed (launch error) */
    SSD_ERR_TIMEOUT = 6,       /* a bounded device-side wait gave up (device status) */
    SSD_ERR_DEVICE = 7         /* device-side check failed, e.g. bad cu_seqlens (device status) */
} ssd_status_t;

typedef enum { SSD_DTYPE_F32 = 0, SSD_DTYPE_BF16 = 1 } ssd_dtype_t;

typedef struct {
    int64_t batch;       /* rows of a dense batch; must be 1 when cu_seqlens is used */
    int64_t seqlen;      /* tokens per row; with cu_seqlens: total packed tokens T */
    int32_t nheads;      /* H */
    int32_t headdim;     /* P */
    int32_t dstate;      /* N */
    int32_t ngroups;     /* G, divides H (B and C are shared by H / G heads) */
    int32_t chunk_size;  /* Q, the diagonal-block length; the result does not depend on it */
    int32_t nseq;        /* 0: dense batch; > 0: number of packed sequences in cu_seqlens */
    float delta_init;    /* added to raw_dt before softplus (e.g. -4.6) */
    int32_t dtype;       /* ssd_dtype_t of x, B, C, y, dy, dx, dB, dC */
} ssd_problem_t;

/* Supported shapes: P in {8,16,32,64,128}; N in {8,16,32,64,128};
 * chunk_size in {16,32,64,128,256}; T <= 2^31 - 1; G divides H.
 * bf16 problems with P = 64, N in {64,128}, chunk_size = 64 and at least chunk_size
 * tokens in all run on the tensor-core path (any number of heads per group); every
 * other supported problem runs on the SIMT path. */

/* Bytes of device workspace that ssd_forward (for_backward = 0) or
 * ssd_backward (for_backward = 1) needs for `prob`.  Host function, no launch; on the
 * tensor-core path with dense rows the segment length, and with it the size, follows
 * the current device's SM count, so query it with the device current that will run
 * the calls.  Returns SSD_ERR_INVALID_ARG / SSD_ERR_UNSUPPORTED for a bad problem. */
ssd_status_t ssd_workspace_size(const ssd_problem_t* prob, int for_backward, size_t* bytes);

/* Forward scan.  Reads x, raw_dt, B, C (and cu_seqlens when prob->nseq > 0,
 * else it must be NULL); writes y and, when final_state is not NULL, the
 * state after the last token of every sequence (row) -- the quantity that
 * crosses from one chunk to the next, page "长序列 Mamba 多卡训练算力和显存
 * 怎么同时省" §一.  workspace: >= ssd_workspace_size(prob, 0) bytes, 256-byte
 * aligned, contents ignored on entry. */
ssd_status_t ssd_forward(const ssd_problem_t* prob, const void* x, const float* raw_dt,
                         const void* B, const void* C, const int32_t* cu_seqlens, void* y,
                         float* final_state, void* workspace, size_t workspace_bytes,
                         void* stream);

/* ssd_forward from a given state per sequence: H = initial_state[seq] before the first
 * token of every sequence (dense row) instead of zero -- the carried-over state of page
 * "Mamba-2架构与LaCT并行计算技术解析" §1.1 (the note on initialising H from the previous
 * frame's final state).  initial_state: [nseq or batch][H][P][N] float32 device memory,
 * 16-byte aligned, or NULL for zero (then this is ssd_forward).  The final state of an
 * empty packed sequence is its initial state. */
ssd_status_t ssd_forward_state(const ssd_problem_t* prob, const void* x, const float* raw_dt,
                               const void* B, const void* C, const int32_t* cu_seqlens,
                               const float* initial_state, void* y, float* final_state,
                               void* workspace, size_t workspace_bytes, void* stream);

/* Backward of ssd_forward for an upstream gradient dy of y (the gradient of
 * final_state is taken as zero).  Writes dx [T][H][P], d_raw_dt [T][H]
 * (float32, includes the softplus derivative), dB and dC [T][G][N] (summed
 * over the heads of each group, fp32 accumulation, one rounding to dtype).
 * Reverse-mode derivative of the recurrence of page "Mamba-2架构与LaCT并行
 * 计算技术解析" §1.1; the forward states are recomputed, per the
 * recompute-from-checkpoints idea of that page's §4.1.  workspace: >=
 * ssd_workspace_size(prob, 1) bytes, 256-byte aligned. */
ssd_status_t ssd_backward(const ssd_problem_t* prob, const void* x, const float* raw_dt,
                          const void* B, const void* C, const int32_t* cu_seqlens,
                          const void* dy, void* dx, float* d_raw_dt, void* dB, void* dC,
                          void* workspace, size_t workspace_bytes, void* stream);

/* ssd_backward for the workspace that the preceding ssd_forward call used, on the same
 * stream, with the same problem and the same x, raw_dt, B, C (and cu_seqlens) buffers,
 * whose contents have not changed since.  On the tensor-core path it takes the
 * forward's segment table, masked C B^T tiles, chunk factors and segment states from the
 * workspace instead of recomputing them (activations saved by the forward, in the
 * sense of page "Mamba-2架构与LaCT并行计算技术解析" §4.1); the results are those of
 * ssd_backward.  The forward records its problem and input pointers (initial_state
 * included) in the workspace;
 * if they differ from this call's, the device status becomes SSD_ERR_WORKSPACE and no
 * gradient is computed (ssd_device_status reports it).  Buffer contents are not
 * compared: changing them between the two calls gives the gradient at the old inputs.
 * The forward's own device status is kept.  On the SIMT path this call is ssd_backward.
 * workspace: >= ssd_workspace_size(prob, 1) bytes, passed to the forward as well. */
ssd_status_t ssd_backward_after_forward(const ssd_problem_t* prob, const void* x,
                                        const float* raw_dt, const void* B, const void* C,
                                        const int32_t* cu_seqlens, const void* dy, void* dx,
                                        float* d_raw_dt, void* dB, void* dC, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* Backward of ssd_forward_state: the gradient of
 *     L = sum_t dy_t . y_t + sum_seq <d_final_state[seq], final_state[seq]>
 * with respect to x, raw_dt, B, C (written as by ssd_backward) and, when d_initial_state is
 * not NULL, to initial_state: d_initial_state[seq] = dL / dH before the sequence's first
 * token ([nseq or batch][H][P][N] float32; an empty sequence's is its d_final_state).
 * initial_state (NULL: zero) must be the one the forward used; d_final_state ([nseq or
 * batch][H][P][N] float32, NULL: zero) is the upstream gradient of final_state.  Reverse
 * mode of the recurrence of page "Mamba-2架构与LaCT并行计算技术解析" §1.1.
 * after_forward != 0: as ssd_backward_after_forward (the preceding ssd_forward_state on the
 * same workspace, inputs and initial_state); 0: as ssd_backward.  workspace: >=
 * ssd_workspace_size(prob, 1) bytes. */
ssd_status_t ssd_backward_state(const ssd_problem_t* prob, const void* x, const float* raw_dt,
                                const void* B, const void* C, const int32_t* cu_seqlens,
                                const float* initial_state, const void* dy,
                                const float* d_final_state, void* dx, float* d_raw_dt, void* dB,
                                void* dC, float* d_initial_state, int after_forward,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Bidirectional mode (page "Mamba-2架构与LaCT并行计算技术解析" §3.1): the scan over each
 * sequence (dense row or packed sequence) and the scan over the same sequence reversed,
 * on the same x, raw_dt, B, C; the reverse direction's output is put back at its tokens'
 * positions and the two are concatenated along the last dimension:
 *     y[t][h] = [ y_forward[t][h] (P values) | y_reverse[t][h] (P values) ],
 * y_reverse[t] depending on tokens t .. the sequence's end.  y: [T][H][2P] (dtype of x).
 * final_state_fwd / final_state_rev ([nseq or batch][H][P][N] float32, NULL: not written):
 * each direction's state after its last token (the state size doubles).  workspace: >=
 * ssd_bidirectional_workspace_size(prob, 0) bytes, 256-byte aligned; it holds the
 * reversed inputs and both directions' outputs besides ssd_forward's workspace. */
ssd_status_t ssd_bidirectional_workspace_size(const ssd_problem_t* prob, int for_backward,
                                              size_t* bytes);
ssd_status_t ssd_bidirectional_forward(const ssd_problem_t* prob, const void* x,
                                       const float* raw_dt, const void* B, const void* C,
                                       const int32_t* cu_seqlens, void* y,
                                       float* final_state_fwd, float* final_state_rev,
                                       void* workspace, size_t workspace_bytes, void* stream);
/* Backward of ssd_bidirectional_forward for an upstream gradient dy [T][H][2P] of y (zero
 * final-state gradients): dx, d_raw_dt, dB, dC as ssd_backward writes them, each the sum of
 * the two directions' contributions.  workspace: >= ssd_bidirectional_workspace_size(prob,
 * 1) bytes. */
ssd_status_t ssd_bidirectional_backward(const ssd_problem_t* prob, const void* x,
                                        const float* raw_dt, const void* B, const void* C,
                                        const int32_t* cu_seqlens, const void* dy, void* dx,
                                        float* d_raw_dt, void* dB, void* dC, void* workspace,
                                        size_t workspace_bytes, void* stream);

/* One token of the recurrence for every sequence of a batch (single-token decode), from
 * a carried state (page "Mamba-2架构与LaCT并行计算技术解析" §1.1):
 *     delta = softplus(raw_dt + delta_init),
 *     state <- exp(-delta) state + delta x B^T,   y = state C.
 * prob: batch = number of sequences, seqlen = 1, nseq = 0; H, P, N, G, dtype, delta_init
 * as for ssd_forward (chunk_size must be a supported value and is otherwise unused).
 * state_in, state_out: [batch][H][P][N] float32 (the same pointer updates in place; other
 * overlaps are SSD_ERR_INVALID_ARG); x, y: [batch][H][P]; raw_dt: [batch][H] float32;
 * B, C: [batch][G][N].  Device memory, 16-byte aligned; no workspace.  Bound by the
 * state's bytes: it is read and written once. */
ssd_status_t ssd_decode_step(const ssd_problem_t* prob, const float* state_in, float* state_out,
                             const void* x, const float* raw_dt, const void* B, const void* C,
                             void* y, void* stream);

/* Device bytes that ssd_step_host needs for `prob`: the backward workspace followed by
 * device copies of the step's inputs and results.  Pure host function. */
ssd_status_t ssd_step_host_size(const ssd_problem_t* prob, size_t* bytes);

/* One forward + backward step on HOST buffers (the layouts above, in host memory):
 * x, raw_dt, B, C, cu_seqlens (a host array; NULL for a dense batch) and dy are read from
 * host memory; y, final_state (NULL: not written), dx, d_raw_dt, dB and dC are written to
 * host memory.  With dy = NULL the step is the forward alone (dx, d_raw_dt, dB and dC
 * are then not used and may be NULL).  The call copies the inputs into `device` (>= ssd_step_host_size bytes of
 * device memory owned by the caller, 256-byte aligned), runs ssd_forward and
 * ssd_backward_after_forward there, and copies the results back.  Asynchronous on
 * `stream` like every other call: the host outputs are complete once the stream has
 * passed the call (e.g. after cudaStreamSynchronize), and every host buffer must stay
 * valid until then.  Page-locked host memory lets the copies run asynchronously
 * (pageable memory is staged synchronously by the CUDA runtime).  Inside a call, dy is
 * copied in while the forward runs and y and final_state out while the backward runs,
 * on copy streams the library creates once per device; each call is ordered after the
 * caller's earlier work on `stream` and the caller's later work after all of it.  Two
 * calls on different streams with different `device` buffers overlap one step's copies
 * with the other's kernels.  The workspace is the first region of `device`, so
 * ssd_device_status(device, ...) reads the step's device status.  Errors: those of
 * ssd_forward and ssd_backward; SSD_ERR_WORKSPACE if `device` is NULL or smaller than
 * ssd_step_host_size(); SSD_ERR_ALIGNMENT if it is not 256-byte aligned; SSD_ERR_CUDA if
 * a copy or an event could not be enqueued.  One host thread at a time enqueues a step
 * (calls from several threads are serialised). */
ssd_status_t ssd_step_host(const ssd_problem_t* prob, const void* x, const float* raw_dt,
                           const void* B, const void* C, const int32_t* cu_seqlens,
                           const void* dy, void* y, float* final_state, void* dx,
                           float* d_raw_dt, void* dB, void* dC, void* device,
                           size_t device_bytes, void* stream);

/* Size of the device scratch array that ssd_forward_noalloc works in. */
#define SSD_NOALLOC_SCRATCH_BYTES (64u << 20)

/* ssd_forward for callers that cannot allocate device memory.  The pages have
 * no counterpart to this call: it exists for host applications whose device
 * memory is owned by someone else -- a plugin or callback inside a framework
 * that hands out no workspace, or code on a latency-critical path where
 * cudaMalloc / cudaFree (which may synchronise the device) are not allowed.
 * Such a caller passes only inputs and outputs; the scratch that ssd_forward
 * takes as `workspace` comes instead from one SSD_NOALLOC_SCRATCH_BYTES array
 * that the library declares in device memory.  Every GPU on which the library
 * is loaded holds that array until the process exits (with CUDA's default lazy
 * module loading, from the first call on that GPU).
 *  - Same arguments, layouts and results as ssd_forward, minus the workspace.
 *  - Problems whose forward workspace (ssd_workspace_size(prob, 0)) exceeds
 *    SSD_NOALLOC_SCRATCH_BYTES are rejected with SSD_ERR_WORKSPACE before any
 *    launch.
 *  - The first call on a device looks up the array's device address for that
 *    device (the current one); make that first call before any stream capture.
 *  - Every call on a device uses the same array, which keeps the previous
 *    call's contents (the call clears what it needs cleared); calls that may
 *    overlap on the GPU, from any stream or thread, race and must be ordered
 *    by the caller.
 *  - Allocates nothing: no cudaMalloc, cudaFree or allocating library call.
 *  - Errors that only the device sees (a malformed cu_seqlens, a wait that timed out)
 *    go to the status word inside the array; ssd_forward_noalloc_status() reads it.
 *  - The array's address is kept per device for the life of the process: calling
 *    cudaDeviceReset() after the first call on a device is not supported. */
ssd_status_t ssd_forward_noalloc(const ssd_problem_t* prob, const void* x, const float* raw_dt,
                                 const void* B, const void* C, const int32_t* cu_seqlens,
                                 void* y, float* final_state, void* stream);

/* The device status word that the last ssd_forward_noalloc call on the current device
 * left (SSD_OK, SSD_ERR_DEVICE, SSD_ERR_TIMEOUT), read like ssd_device_status():
 * synchronises `stream` first.  Returns SSD_ERR_CUDA if that failed. */
ssd_status_t ssd_forward_noalloc_status(void* stream, int32_t* device_status);

/* ---------------------------------------------------------------- around the scan
 *
 * The operators next to the scan in a layer of a language model: the short causal
 * convolution that makes x, B and C from the in-projection, the one-token step that
 * carries the convolution's window beside the scan's state, the norm in front of the layer
 * and the gated norm behind the scan.  Here pointers need the alignment of their element
 * type only (workspaces: 256 bytes; the scan state: 16); tensors whose rows all start
 * on 16 bytes move in bulk copies and vectors of that size, others in vectors of two elements
 * or one.  Strides
 * are counted in elements, from one token or row to the next.  Weights, biases and their
 * gradients are float32 or bf16 (wdtype), whatever the activations are.  An output must not
 * overlap another output or, unless the call's comment says so, an input
 * (SSD_ERR_INVALID_ARG); a tensor counts as everything from its first to its last element, and
 * a workspace as an output. */

/* Synchronises `stream` and returns in *device_status what the calls of this section have
 * recorded on the current device since the last query: SSD_OK, or SSD_ERR_TIMEOUT if a
 * kernel's bounded wait for one of its copies ran out (its outputs are then not valid).
 * Returns SSD_ERR_CUDA if the synchronisation itself failed. */
ssd_status_t ssd_layer_status(void* stream, int32_t* device_status);

/* Causal depthwise convolution over the tokens of a sequence, then SiLU:
 *     pre[i] = bias + sum_{j < width} weight[c][width - 1 - j] u[i - j],
 *     out[i] = pre[i] / (1 + exp(-pre[i])).
 * Tokens before the sequence's first come from its carried state, or are zero.  A
 * sequence's state is `width` rows of channels in the type of u, row p mod width holding the
 * token at position p; a call reads the width - 1 positions before its first token
 * (positions[seq], or 0) and leaves the last `width` positions.  cu_seqlens is read with
 * every entry clamped to 0 .. T (a malformed array gives wrong values, no access out of
 * range); tokens from cu_seqlens[nseq] on belong to no sequence: their outputs and
 * gradients are zero. */
typedef struct {
    int64_t batch;       /* rows of a dense batch; 1 with cu_seqlens */
    int64_t seqlen;      /* tokens per row; with cu_seqlens: all tokens T (<= 2^31 - 1) */
    int64_t u_stride;    /* elements from one token of u to the next (>= channels) */
    int64_t du_stride;   /* the same of du (0 in a forward) */
    int32_t split[3];    /* channels of the up to three contiguous outputs (unused ones 0) */
    int32_t width;       /* taps: 2, 3 or 4 */
    int32_t nseq;        /* 0: dense batch; > 0: number of packed sequences */
    int32_t dtype;       /* ssd_dtype_t of u, the outputs and the states */
    int32_t wdtype;      /* ssd_dtype_t of weight, bias and their gradients */
    int32_t activation;  /* 1: SiLU, 0: none */
} ssd_conv_t;

/* Writes out0 .. out2 ([T][split[i]], contiguous) and, when final_state is not NULL, the
 * states after the last tokens.  weight [channels][width]; bias [channels] or NULL;
 * positions int32 [nseq or batch] or NULL (0); initial_state, final_state
 * [nseq or batch][width][channels] or NULL. */
ssd_status_t ssd_conv_forward(const ssd_conv_t* conv, const void* u, const void* weight,
                              const void* bias, const int32_t* cu_seqlens,
                              const int32_t* positions, const void* initial_state, void* out0,
                              void* out1, void* out2, void* final_state, void* stream);

/* Bytes of workspace ssd_conv_backward needs (it follows the current device's SM count). */
ssd_status_t ssd_conv_workspace_size(const ssd_conv_t* conv, size_t* bytes);

/* Gradients of u, weight, bias (d_bias may be NULL) and, when d_initial_state is not NULL,
 * of the carried states, from those of the outputs and (d_final_state, or NULL: zero) of the
 * final states.  The same inputs give the same bits in every call. */
ssd_status_t ssd_conv_backward(const ssd_conv_t* conv, const void* u, const void* weight,
                               const void* bias, const int32_t* cu_seqlens,
                               const int32_t* positions, const void* initial_state,
                               const void* dout0, const void* dout1, const void* dout2,
                               const void* d_final_state, void* du, void* d_weight, void* d_bias,
                               void* d_initial_state, void* workspace, size_t workspace_bytes,
                               void* stream);

/* One token for each of prob->batch rows (prob->seqlen = 1): the convolution with SiLU over
 * the row of u (channels x [H][P], B [G][N], C [G][N]), then the scan's step.  Row i uses
 * cache slot slots[i] (NULL: i) of state [nslots][H][P][N] float32 and conv_state
 * [nslots][width][channels], both updated in place; a slot outside 0 .. nslots - 1 marks a
 * padding row, whose y is zero and which touches no state.  The live rows' slots must
 * differ.  positions int32 [batch]: the position of the new token.  y [batch][H][P]. */
ssd_status_t ssd_conv_decode_step(const ssd_problem_t* prob, int32_t width, int32_t wdtype,
                                  int32_t nslots, int64_t u_stride, float* state,
                                  void* conv_state, const void* u, const float* raw_dt,
                                  const void* weight, const void* bias, const int32_t* positions,
                                  const int32_t* slots, void* y, void* stream);

/* Norm over the columns of each row, after the residual add:
 *     v = x + residual;  y = (v - mu) rstd weight + bias,
 *     rstd = (mean((v - mu)^2) + eps)^-1/2,  mu = mean(v) (SSD_NORM_RMS: 0).
 * Rows of up to 16384 columns, 8192 where a row does not start on 16 bytes. */
typedef enum { SSD_NORM_LAYER = 0, SSD_NORM_RMS = 1 } ssd_norm_kind_t;
typedef struct {
    int64_t rows;
    int64_t x_stride;    /* x; dx in the backward */
    int64_t r_stride;    /* residual; dh in the backward */
    int64_t h_stride;    /* h */
    int64_t y_stride;    /* y; dy in the backward */
    int32_t dim;
    int32_t kind;        /* ssd_norm_kind_t */
    int32_t dtype;       /* ssd_dtype_t of x, y and their gradients */
    int32_t rdtype;      /* of residual, h and their gradients: dtype, or float32 */
    int32_t wdtype;      /* of weight, bias and their gradients */
    float eps;
} ssd_norm_t;

/* Writes y, h = v (with a residual only; both NULL or neither) and stats [rows][2] float32
 * (mu, rstd; may be NULL).  bias may be NULL.  y may be x and h may be residual. */
ssd_status_t ssd_norm_forward(const ssd_norm_t* norm, const void* x, const void* residual,
                              const void* weight, const void* bias, void* y, void* h,
                              float* stats, void* stream);

ssd_status_t ssd_norm_workspace_size(const ssd_norm_t* norm, size_t* bytes);

/* Gradients from dy and (dh, or NULL) the gradient of h that arrives by the residual stream:
 * dx = the gradient of v in dtype; d_residual [rows][dim] the same in rdtype (may be NULL);
 * d_weight, d_bias (may be NULL).  h is what the norm was taken of: the forward's h, or its
 * x without a residual.  dx may be dy or dh, d_residual may be dh.  The same inputs give the
 * same bits in every call. */
ssd_status_t ssd_norm_backward(const ssd_norm_t* norm, const void* dy, const void* h,
                               const void* dh, const void* weight, const float* stats, void* dx,
                               void* d_residual, void* d_weight, void* d_bias, void* workspace,
                               size_t workspace_bytes, void* stream);

/* The scan's output y under its gate z, normed in each of `groups` equal groups of columns:
 *     v = y z / (1 + exp(-z));  out = v rstd weight,  rstd = (mean over the group of v^2 + eps)^-1/2.
 * Groups of up to 16384 columns, 8192 where a row does not start on 16 bytes. */
typedef struct {
    int64_t rows;
    int64_t y_stride, z_stride, out_stride;  /* out_stride: out; dout in the backward */
    int64_t dy_stride, dz_stride;            /* backward (any value >= dim in a forward) */
    int32_t dim;
    int32_t groups;
    int32_t dtype;       /* ssd_dtype_t of y, z, out and their gradients */
    int32_t wdtype;      /* of weight and its gradient */
    float eps;
} ssd_gated_norm_t;

/* Writes out and rstd [rows][groups] float32 (may be NULL).  out may be y or z. */
ssd_status_t ssd_gated_norm_forward(const ssd_gated_norm_t* norm, const void* y, const void* z,
                                    const void* weight, void* out, float* rstd, void* stream);

ssd_status_t ssd_gated_norm_workspace_size(const ssd_gated_norm_t* norm, size_t* bytes);

/* dy, dz, d_weight from dout and the forward's rstd.  dy and dz may each be one of the
 * inputs.  The same inputs give the same bits in every call. */
ssd_status_t ssd_gated_norm_backward(const ssd_gated_norm_t* norm, const void* dout, const void* y,
                                     const void* z, const void* weight, const float* rstd,
                                     void* dy, void* dz, void* d_weight, void* workspace,
                                     size_t workspace_bytes, void* stream);

/* ------------------------------------------- linear attention and beam search
 *
 * The rules of the section above hold here too (alignment of the element type, strides,
 * overlaps, ssd_layer_status); workspaces are 256-byte aligned.
 *
 * Linear attention with a decay for each head: with a = exp(log_decay[h]), every token t
 *     S_t = a S_{t-1} + v_t k_t^T            (S is P x N, float32)
 *     o_t = scale S_t q_t
 * with S = initial_state (or zero) before the first token of every sequence.  log_decay is
 * float32 device memory, zero or negative (-inf: nothing is remembered), and takes no
 * gradient.  Query heads h read key and value head h / (H / G); each has a state of its own, in
 * the layout of the scan's.  q [T][H][N], k [T][G][N], v [T][G][P], o [T][H][P]: the heads of a
 * token lie next to one another, tokens `stride` elements apart; tensors of the same stride may
 * lie between one another's tokens (slices of one projection's rows).  cu_seqlens is read with
 * every entry clamped to 0 .. T; borders that fall give wrong values, no access out of range.
 * Outputs and gradients of tokens before the first border or from the last one on are zero.
 * bf16 calls with N and P 64 or 128, whose rows all start on 16 bytes, run on the tensor cores in
 * blocks of 128 tokens: there a NaN or an infinity in a token reaches the outputs of all tokens
 * of its sequence in its block.  So do bf16 calls of other N and P, or with rows off 16 bytes, with
 * 16384 rows (of a head and token) or more and N + P at least a quarter of what they come to
 * rounded up to 64 or 128, by copies in the workspace.  Forwards of up to 16 tokens a sequence (a batch row, or all packed
 * ones) are stepped through token by token, and all other calls run the walk on the plain cores, in
 * float32. */
typedef struct {
    int64_t batch;       /* rows of a dense batch; 1 with cu_seqlens */
    int64_t seqlen;      /* tokens per row; with cu_seqlens: all tokens T (<= 2^31 - 1) */
    int64_t q_stride, k_stride, v_stride;
    int64_t o_stride;    /* o; its gradient in the backward */
    int64_t dq_stride, dk_stride, dv_stride; /* backward (0 in a forward) */
    int32_t nheads;      /* H */
    int32_t ngroups;     /* G, divides H */
    int32_t headdim;     /* P, 1 to 128 */
    int32_t dstate;      /* N, 1 to 128 */
    int32_t nseq;        /* 0: dense batch; > 0: number of packed sequences */
    int32_t dtype;       /* ssd_dtype_t of q, k, v, o and their gradients */
    float scale;
} ssd_linattn_t;

/* Bytes of workspace of ssd_linear_attention_forward (for_backward = 0, may be 0) or
 * _backward; they follow the current device's SM count.  They do for any tensors of these
 * strides.  Where the strides are multiples of 8 elements but a tensor does not start on 16
 * bytes, a larger workspace, of the size for a q_stride that is no such multiple, lets the call go
 * by copies too; otherwise it runs on the plain cores. */
ssd_status_t ssd_linear_attention_workspace_size(const ssd_linattn_t* prob, int for_backward,
                                                 size_t* bytes);

/* initial_state, final_state: [nseq or batch][H][P][N] float32, or NULL.  The final state of an
 * empty sequence is its initial one. */
ssd_status_t ssd_linear_attention_forward(const ssd_linattn_t* prob, const void* q, const void* k,
                                          const void* v, const float* log_decay,
                                          const int32_t* cu_seqlens, const float* initial_state,
                                          void* o, float* final_state, void* workspace,
                                          size_t workspace_bytes, void* stream);

/* Gradients of q, k and v (k's and v's summed over the heads that share them) and, when
 * d_initial_state is not NULL, of the initial states, from those of o and (d_final_state, or
 * NULL: zero) of the final states.  The same inputs give the same bits in every call. */
ssd_status_t ssd_linear_attention_backward(const ssd_linattn_t* prob, const void* q, const void* k,
                                           const void* v, const float* log_decay,
                                           const int32_t* cu_seqlens, const float* initial_state,
                                           const void* dout, const float* d_final_state, void* dq,
                                           void* dk, void* dv, float* d_initial_state,
                                           void* workspace, size_t workspace_bytes, void* stream);

/* One token for each of prob->batch rows (prob->seqlen = 1, nseq = 0).  Row i uses cache slot
 * slots[i] (NULL: i) of state [nslots][H][P][N] float32, updated in place; a slot outside
 * 0 .. nslots - 1 marks a padding row, whose o is zero and which touches no state.  The live
 * rows' slots must differ.  Where N is a multiple of 4, state is 16-byte aligned. */
ssd_status_t ssd_linear_attention_step(const ssd_linattn_t* prob, int32_t nslots, float* state,
                                       const void* q, const void* k, const void* v,
                                       const float* log_decay, const int32_t* slots, void* o,
                                       void* stream);

/* Beam search: of the candidates (beam i, token t) of each batch row, with the score
 *     scores[i] + logits[i][t] - log sum_u exp(logits[i][u]),
 * the `keep` best, best first.  Candidates of one beam are ordered by their logits, those of
 * different beams by their scores in float64, before they are rounded (or overflow) to float32; equal
 * ones by beam, then token.  The sums under the logarithms are float32's: beams may be off against one
 * another by some 10^-8, and where few logits make up a sum by a few 10^-7.
 * finished (one byte a beam, not 0: ended; NULL: none has): such a beam has the one candidate
 * pad_token, at its score.  What is left out, tokens with a logit of -inf and every token of a
 * beam whose score is not finite or whose logits hold a NaN or +inf or nothing but -inf, has the
 * score -inf. */
typedef struct {
    int64_t batch;
    int64_t stride;      /* elements from one beam's logits to the next (>= vocab) */
    int32_t beams;       /* 1 to 64 */
    int32_t vocab;       /* <= 2^24 */
    int32_t keep;        /* 1 to 64, <= beams * vocab */
    int32_t pad_token;
    int32_t dtype;       /* ssd_dtype_t of the logits */
} ssd_beam_t;

ssd_status_t ssd_beam_select_workspace_size(const ssd_beam_t* beam, size_t* bytes);

/* logits [batch][beams][vocab], scores [batch][beams] float32; out_scores float32, parents
 * (the beam) and tokens int32, all [batch][keep]. */
ssd_status_t ssd_beam_select(const ssd_beam_t* beam, const void* logits, const float* scores,
                             const uint8_t* finished, float* out_scores, int32_t* parents,
                             int32_t* tokens, void* workspace, size_t workspace_bytes,
                             void* stream);

/* Beam search over cached states: beam j of each batch row goes on from the state of beam
 * parents[j] (parents, slots, new_slots: int32 [batch][beams], beams 1 to 64).  The first beam
 * with a parent takes its parent's slot; each other one takes the next slot, in the order of
 * the beams, of a beam that nobody goes on from, and the parent's state is copied there in each
 * of `ncaches` caches: cache i holds nslots slots of slot_bytes[i] bytes, slot_strides[i] bytes
 * apart (host arrays).  So only the states of beams that are doubled move, in place.  A beam
 * whose parent lies outside 0 .. beams - 1 gets slot -1; a slot outside 0 .. nslots - 1 is
 * passed on and its states are left alone.  The slots of live beams must differ. */
ssd_status_t ssd_beam_reorder(int64_t batch, int32_t beams, const int32_t* slots,
                              const int32_t* parents, int32_t* new_slots, int32_t ncaches,
                              void* const* caches, const int64_t* slot_bytes,
                              const int64_t* slot_strides, int32_t nslots, void* stream);

/* Synchronises `stream` and returns in *device_status the status word that
 * the last call using `workspace` left (SSD_OK, SSD_ERR_DEVICE, SSD_ERR_TIMEOUT).
 * Returns SSD_ERR_CUDA if the synchronisation itself failed. */
ssd_status_t ssd_device_status(const void* workspace, void* stream, int32_t* device_status);

/* Which kernel path a problem takes: "tensor-core", "simt", or NULL for an
 * unsupported problem.  Pure host function. */
const char* ssd_dispatch_path(const ssd_problem_t* prob, int for_backward);

/* Number of kernels the last ssd_forward / ssd_backward call, or the last call of an
 * operator around the scan, on this host thread launched (memsets not counted). */
int ssd_last_launch_count(void);

/* Per-kernel timing.  While enabled, every kernel launch is bracketed by CUDA
 * events recorded on the launch stream; ssd_profiler_entry() synchronises
 * them and reports, per kernel name, the launch count and total device time.
 * Not thread-safe; meant for benchmarks. */
ssd_status_t ssd_profiler_enable(int on);
/* Restricts the timing to launches of the kernel called `name` (as reported by
 * ssd_profiler_entry); NULL times every kernel again.  Each pair of events holds the
 * launch that follows it back until the kernel before it has finished, so timing
 * only the kernel of interest leaves the other kernel boundaries of a pass alone. */
ssd_status_t ssd_profiler_only(const char* name);
void ssd_profiler_reset(void);
int ssd_profiler_count(void);
ssd_status_t ssd_profiler_entry(int index, const char** name, int64_t* launches,
                                double* total_ms);

const char* ssd_status_string(ssd_status_t status);
int ssd_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SSD_H_ */
