/*
 * kda.h -- C ABI of libkda.so: the Kimi Delta Attention (KDA) layer on one
 * GB300 (sm_103a).
 *
 * What the layer computes, per head of width D (page "Kimi K3 / Architecture",
 * panel "Kimi Delta Attention . one head at token t", and page "Animated Kimi
 * K3 architecture diagram", section "LOCAL MEMORY: A FIXED MATRIX THAT
 * PREDICTS, FORGETS, AND CORRECTS"):
 *
 *   short conv  u = sum_{j=0..3} w[j] x[t-3+j] per channel, then SiLU
 *   L2 norm     q <- q / sqrt(|q|^2 + eps_l2), same for k (v is not normalised)
 *   decay       S_bar = Diag(exp(g_t)) S_{t-1}           (g_t: log-decay per key channel)
 *   correct     e_t = v_t - S_bar^T k_t
 *   write       S_t = S_bar + beta_t k_t e_t^T          (beta_t: one scalar per token, head)
 *   read        o_t = scale * S_t^T q_t
 *   epilogue    y_t = o_t / sqrt(mean(o_t^2) + eps_rms) * w_rms * sigmoid(gate_t)
 *
 * The state S is a fixed D x D fp32 matrix per (sequence, head), row = key
 * channel, column = value channel.
 *
 * Conventions for every entry point:
 *  - Ownership: the caller owns every buffer.  The library allocates nothing
 *    on the device.  Its only device memory of its own is the fixed scratch
 *    array of kda_prefill_noalloc (below), and its only state between calls is
 *    a per-device cache of device attributes (SM count, compute capability).
 *  - Asynchrony: calls only enqueue work on `stream` (a cudaStream_t; NULL is
 *    the legacy default stream) and never synchronise.
 *  - Errors: invalid arguments return before anything is launched.  A launch
 *    failure returns KDA_ERR_CUDA.  Conditions found on the device (an
 *    inconsistent cu_seqlens) are written to the optional `d_status` word
 *    (a device int the caller zeroes) and the affected work is skipped; no
 *    kernel traps or asserts.
 *  - Value ranges: g is expected in [-5, 0] (the pages bound the log-decay
 *    below by -5) and beta in [0, 1].  They are not range-checked on the
 *    device.  Outside that range results may overflow to inf/NaN: on every
 *    path for g > 0 (growing state), and on the tensor-core path also for
 *    g < -5, whose split decay factors reach e^{16 |g|} (e^{96} > FLT_MAX at
 *    g = -6).  Both ends of the range, g = -5 and g = 0, are supported.
 *  - Shapes: D in {16, 32, 64, 128}; the tensor-core prefill path needs
 *    D = 128, chunk = 64 and bf16 inputs, everything else takes the fp32 SIMT
 *    path.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t, declared without the CUDA headers. */
typedef struct CUstream_st* kda_stream_t;

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1, /* null pointer, bad size, misalignment, aliasing, bad cu_seqlens */
    KDA_ERR_UNSUPPORTED = 2, /* shape or dtype this library does not implement */
    KDA_ERR_WORKSPACE = 3,   /* workspace missing or smaller than kda_prefill_workspace_size */
    KDA_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
    KDA_ERR_TIMEOUT = 5,     /* a bounded device-side wait gave up (reported via d_status) */
    KDA_ERR_DEVICE_ARG = 6   /* the device copy of cu_seqlens was inconsistent (via d_status) */
} kda_status;

typedef enum { KDA_BF16 = 0, KDA_FP32 = 1 } kda_dtype;

/* Static English text for a status code. */
const char* kda_status_string(int status);

/* Text describing the last error returned on the calling host thread. */
const char* kda_last_error(void);

/* Library version as major*10000 + minor*100 + patch. */
int kda_version(void);

/* ------------------------------------------------------------------------
 * kda_short_conv -- causal depthwise short convolution + SiLU (+ L2 on q, k).
 * Page "Kimi K3 / Architecture", panel "KDA short convolution . one channel
 * c at token t": window of width 4 over x[t-3..t] of one channel, only time
 * is mixed, left padding keeps the length, SiLU after the 4-tap sum; Q and K
 * are then L2-normalised per head, V is not.  Filter banks Wq, Wk, Wv; the
 * rolling state keeps the previous 3 raw values per channel ([B,36864,3] for
 * 96 heads of 128).
 *
 *   x         [T_total][row stride x_row_stride elements], channels q|k|v:
 *             channel = part*H*D + h*D + d (part 0=q, 1=k, 2=v); io dtype.
 *   w         [3*H*D][4] fp32; tap 3 multiplies x[t], tap 0 multiplies x[t-3].
 *   cu_seqlens device int32 [N+1]: cu[0]=0, non-decreasing, cu[N]=T_total.
 *             Sequences never see each other's tokens.
 *   cu_seqlens_host optional host copy; when given it is validated on the
 *             host (no device sync is ever needed).
 *   conv_state_in  [N][3*H*D][3] io dtype, oldest first, or NULL (zeros).
 *   conv_state_out [N][3*H*D][3] io dtype or NULL: the last 3 raw values of
 *             each sequence (taking conv_state_in into account for short
 *             sequences).  Must not overlap conv_state_in.
 *   y         [T_total][y_row_stride elements] io dtype; must not overlap x.
 *   l2norm_qk nonzero: L2-normalise the q and k parts per head with eps_l2.
 * Alignment: x, y 16-byte aligned; row strides multiples of 8 elements (bf16)
 * or 4 elements (fp32); D, H >= 1 with D in {16,32,64,128}.
 * ------------------------------------------------------------------------ */
kda_status kda_short_conv(const void* x, int64_t x_row_stride, const float* w,
                          const int32_t* cu_seqlens, const int32_t* cu_seqlens_host, int N,
                          int64_t T_total, int H, int D, const void* conv_state_in,
                          void* conv_state_out, void* y, int64_t y_row_stride, int l2norm_qk,
                          float eps_l2, kda_dtype io, int* d_status, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_prefill -- the whole layer over packed variable-length sequences.
 * Page "Kimi K3 / Architecture", KDA panel: the chunkwise form (the state
 * recurs from chunk to chunk, the tokens of a chunk are taken together as
 * dense tensor-core tiles); page "Animated Kimi K3 architecture diagram": the
 * state is carried across chunks.  Chunks of `chunk` tokens start at every
 * sequence start; the last chunk of a sequence may be partial.  The result
 * does not depend on `chunk` beyond rounding.
 * ------------------------------------------------------------------------ */
typedef struct {
    int N;                 /* sequences */
    int H;                 /* heads */
    int D;                 /* head width (dk = dv = D) */
    int chunk;             /* 16, 32 or 64 */
    int64_t T_total;       /* packed tokens */
    kda_dtype io;          /* dtype of q, k, v, gate and the conv states */
    kda_dtype out_dtype;   /* dtype of out */
    const int32_t* cu_seqlens;       /* device [N+1] */
    const int32_t* cu_seqlens_host;  /* host [N+1] or NULL (then only device-checked) */
    const void* q;         /* [T_total][qkv_row_stride] raw projections, before the conv */
    const void* k;         /* same layout as q */
    const void* v;         /* same layout as q */
    int64_t qkv_row_stride;/* elements between tokens of q/k/v; 0 means H*D */
    const float* conv_w;   /* [3][H*D][4] fp32 (q, k, v filter banks) */
    const void* conv_state_in;  /* [N][3*H*D][3] or NULL (zero left padding) */
    void* conv_state_out;       /* [N][3*H*D][3] or NULL; must not overlap conv_state_in */
    const float* g;        /* [T_total][H][D] fp32 log-decay, expected in [-5, 0] */
    const float* beta;     /* [T_total][H] fp32, expected in [0, 1] */
    const void* gate;      /* [T_total][H][D] pre-sigmoid output gate, io dtype, or NULL */
    const float* rms_w;    /* [D] fp32 RMSNorm weight, or NULL (ones) */
    float eps_l2;          /* typical 1e-6 */
    float eps_rms;         /* typical 1e-6 */
    float scale;           /* readout scale, typical 1.0 */
    const float* initial_state; /* [N][H][D][D] fp32 or NULL (zeros) */
    float* final_state;    /* [N][H][D][D] fp32 or NULL; may equal initial_state */
    void* out;             /* [T_total][H][D] out_dtype; must not overlap any input */
    void* workspace;       /* device scratch, 256-byte aligned, or NULL if size 0 */
    size_t workspace_bytes;
    int* d_status;         /* optional device int for device-side conditions */
    int flags;             /* KDA_FLAG_* */
    int segments;          /* tensor-core path: segments each sequence is cut into (below);
                              0 = chosen from N*H and the SM count, 1 = none, 2..16 forced */
} kda_prefill_args;

#define KDA_FLAG_FORCE_SIMT 1    /* take the fp32 SIMT path even where tensor cores apply */
#define KDA_FLAG_NO_RECURRENT 2  /* never take the recurrent short-sequence path (below) */
/* Test only: on the tensor-core path, the staging of each CTA's first q/k rows is never
 * issued, so the mbarrier wait for them runs out (after about 2 s of GPU clock); the kernel
 * then writes KDA_ERR_TIMEOUT to *d_status and returns without writing out or final_state.
 * Exercises the device-side timeout path without a fault or a hang; ignored by the other
 * paths. */
#define KDA_FLAG_TEST_DROP_STAGING 4

/* Paths of kda_prefill (reported by kda_prefill_plan):
 *  KDA_PATH_SIMT         fp32 SIMT chunkwise path (any D, chunk, dtype);
 *  KDA_PATH_TENSOR_CORE  tcgen05 chunkwise path (D = 128, chunk = 64, bf16 inputs);
 *  KDA_PATH_RECURRENT    token-by-token path for batches of short sequences:
 *                        D = 128, cu_seqlens_host given and every sequence at most
 *                        KDA_RECURRENT_MAX_LEN tokens (multi-token decode, speculative
 *                        verification); each (sequence, head) state is read and
 *                        written once, no workspace.  `chunk` does not matter there:
 *                        the result equals the chunkwise one up to rounding. */
#define KDA_PATH_SIMT 0
#define KDA_PATH_TENSOR_CORE 1
#define KDA_PATH_RECURRENT 2
#define KDA_RECURRENT_MAX_LEN 8

/* Segment-parallel scan (tensor-core path).  One (sequence, head) is a chain
 * of chunks, each depending on the state the previous one leaves.  When the
 * batch has too few (sequence, head) units to fill the GPU, each sequence's
 * chunks are cut into P contiguous segments of ceil(chunks / P) chunks.  Every
 * step of the recurrence maps the state affinely, S -> (I - beta k k^T)
 * Diag(e^g) S + beta k v^T, so a whole segment s maps its start state as
 * S_{s+1} = M_s S_s + B_s, and each of its outputs as o_t = o_t' + S_s^T f_t.
 * Segment 0 runs from the initial state as usual; every later segment runs
 * twice, in parallel with the others: from a zero state (its outputs o_t'
 * and B_s) and with v = 0 from the identity (f_t and M_s).  A second kernel
 * composes S_1 .. S_{P-1} and the final state in order, and a third adds
 * S_s^T f_t to o_t' and applies RMSNorm and the gate.  The results equal
 * the single-pass ones up to rounding.  Workspace: 3 P N H D^2 + 2 T_total H D
 * floats when P > 1, else none.  `segments` is ignored by the SIMT path. */
#define KDA_MAX_SEGMENTS 16

/* Bytes of workspace kda_prefill needs for these arguments (0 allowed). */
kda_status kda_prefill_workspace_size(const kda_prefill_args* args, size_t* bytes);

kda_status kda_prefill(const kda_prefill_args* args, kda_stream_t stream);

/* The plan kda_prefill takes for these arguments on the current device:
 * *path = one of KDA_PATH_*, and *segments = segments per sequence (1
 * except on the tensor-core path when segmenting applies).  Reads the sizes,
 * dtypes, flags, `segments`, the alignment of the state pointers and, when
 * given, cu_seqlens_host; no device pointer is dereferenced; launches nothing. */
kda_status kda_prefill_plan(const kda_prefill_args* args, int* path, int* segments);

/* ------------------------------------------------------------------------
 * kda_prefill_noalloc -- kda_prefill for callers that cannot allocate device
 * memory when they call it: a plugin inside a host application that owns
 * every device allocation and hands over only input and output buffers, a
 * service that reserved its whole memory budget at start-up, or a
 * latency-critical loop that cannot afford the device-wide synchronisation
 * of cudaMalloc/cudaFree.  The pages have no counterpart to this entry
 * point; it is a packaging convenience of this library.
 *
 * It runs the fp32 SIMT path (the path that stages data in scratch) with its
 * scratch taken from a fixed array of KDA_NOALLOC_SCRATCH_BYTES compiled
 * into the library.  Every GPU that loads the library holds that array
 * until the process exits.  args->workspace and args->workspace_bytes are
 * ignored; everything else means what it means for kda_prefill, and the
 * caller still provides every input and output buffer.  The call allocates
 * nothing: no cudaMalloc, no cudaFree, no allocating library routine.
 *
 * Limit: the SIMT path needs 16*T_total*H*D bytes of scratch (two 256-byte
 * aligned parts); a call needing more than KDA_NOALLOC_SCRATCH_BYTES returns
 * KDA_ERR_WORKSPACE before launching anything (use kda_prefill with a
 * workspace instead).
 *
 * Set-up: every call looks up the array's device address on the current
 * device (a host-side lookup that allocates nothing), so the address is
 * right after cudaDeviceReset or under another context too.  The first
 * lookup in a context also loads the library's device code there: make the
 * first call on each device before any stream capture begins.
 *
 * Sharing: all calls use the same array, which keeps the previous call's
 * contents.  Nothing in it needs to start at zero (every scratch byte a call
 * reads is written earlier in the same call).  Calls whose work overlaps on
 * the GPU (different streams, or host threads without ordering between
 * them) race on the array: order them on one stream.
 * ------------------------------------------------------------------------ */
#define KDA_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20) /* 64 MiB per device */

kda_status kda_prefill_noalloc(const kda_prefill_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_decode_step -- one new token for each of N sequences, states updated
 * in place.  Page "Kimi K3 / Architecture", panel "KDA short convolution":
 * the rolling state keeps the previous 3 raw values of every channel; page
 * "Animated Kimi K3 architecture diagram": the four moves on one token.
 * ------------------------------------------------------------------------ */
typedef struct {
    int N, H, D;
    kda_dtype io;          /* dtype of q, k, v, gate and conv_state */
    kda_dtype out_dtype;   /* dtype of out */
    const void* q;         /* [N][qkv_row_stride] raw new token, before the conv */
    const void* k;
    const void* v;
    int64_t qkv_row_stride;/* 0 means H*D */
    const void* gate;      /* [N][H][D] or NULL */
    const float* g;        /* [N][H][D] */
    const float* beta;     /* [N][H] */
    const float* conv_w;   /* [3][H*D][4] */
    const float* rms_w;    /* [D] or NULL */
    float eps_l2, eps_rms, scale;
    float* state;          /* [N][H][D][D] fp32, read and written in place */
    void* conv_state;      /* [N][3*H*D][3] io dtype, rolled in place */
    void* out;             /* [N][H][D] out_dtype */
    int* d_status;
} kda_decode_args;

kda_status kda_decode_step(const kda_decode_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_gemm -- the projections around the layer on the tensor cores, with the
 * activation of their consumer fused into the epilogue:
 *
 *   C[M][N] = epilogue( A[M][K] . W[N][K]^T )
 *
 * Page "Kimi K3 / Architecture", KDA panel: the normalized input x_t goes through
 * linear projections to q, k, v and to alpha_t / beta_t (channel-wise
 * retention, one write strength per head, log-decay bounded below by -5); the
 * head output y_t leaves through W_o.  The gated-MLA panel of the same page writes
 * the output gate as sigmoid(W_g x_t), full rank, one value per output channel.
 * The pages give no activation for alpha and beta; this library reads "bounded
 * log-decay >= -5" as g = -5 sigmoid(z) and the write strength as beta =
 * sigmoid(z), so that g and beta land in the ranges kda_prefill expects.
 *
 *   KDA_EPI_NONE     C = acc              (e.g. gate pre-activations x W_g^T, or y W_o^T)
 *   KDA_EPI_DECAY    C = -5 sigmoid(acc)  (the log-decay g of kda_prefill, fp32)
 *   KDA_EPI_SIGMOID  C = sigmoid(acc)     (the write strength beta, fp32)
 *
 *   A  [M][lda] bf16 row-major (K contiguous); lda >= K, lda * 2 a multiple of 16 bytes.
 *   W  [N][ldw] bf16 row-major, the [out][in] layout of a linear layer's weight; ldw >= K,
 *      ldw * 2 a multiple of 16 bytes.
 *   C  [M][ldc] c_dtype (bf16 or fp32) row-major; ldc >= N; must not overlap A or W.
 *   K  a positive multiple of 64; M, N >= 0 (any value: ragged tiles are masked).
 * A, W and C 16-byte aligned.  Accumulation is fp32 on the tensor cores (tcgen05);
 * the result is rounded once to c_dtype.  Needs an sm_103 device (KDA_ERR_UNSUPPORTED
 * otherwise).  A wait that times out on the device is reported through d_status
 * (KDA_ERR_TIMEOUT).
 * ------------------------------------------------------------------------ */
typedef enum { KDA_EPI_NONE = 0, KDA_EPI_DECAY = 1, KDA_EPI_SIGMOID = 2 } kda_epilogue;

typedef struct {
    int M, N, K;
    const void* A;         /* [M][lda] bf16 */
    int64_t lda;
    const void* W;         /* [N][ldw] bf16 */
    int64_t ldw;
    void* C;               /* [M][ldc] c_dtype */
    int64_t ldc;
    kda_dtype c_dtype;
    int epilogue;          /* kda_epilogue */
    int* d_status;         /* optional device int for device-side conditions */
} kda_gemm_args;

kda_status kda_gemm(const kda_gemm_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_backward -- the gradients of the layer (training).  Page "Kimi K3 /
 * Architecture": the model is trained, so kda_prefill's layer needs its
 * reverse-mode derivatives; page "Animated Kimi K3 architecture diagram",
 * LOCAL MEMORY section: each token's four moves are an affine map of the
 * state, whose adjoint runs the same moves backwards.
 *
 * Given dy = dL/d out and dS_fin = dL/d final_state of one kda_prefill call,
 * it returns dL/d of every input of that call:
 *
 *   dq, dk, dv      [T_total][H][D] fp32 (raw projections, before the conv)
 *   dconv_w         [3][H*D][4] fp32 (summed over all tokens and sequences)
 *   dg              [T_total][H][D] fp32;  dbeta  [T_total][H] fp32
 *   dgate           [T_total][H][D] fp32, or NULL (not wanted; 0 when gate is NULL)
 *   drms_w          [D] fp32, or NULL (computed as for weights of ones when rms_w is NULL)
 *   dinitial_state  [N][H][D][D] fp32, or NULL
 *   dconv_state_in  [N][3*H*D][3] fp32, or NULL (the gradient of the left padding
 *                   when conv_state_in is NULL)
 *
 * The forward is recomputed, not saved: `fwd` holds the kda_prefill arguments
 * (N, H, T_total, io, cu_seqlens and its host copy, q, k, v, qkv_row_stride,
 * conv_w, conv_state_in, g, beta, gate, rms_w, eps_l2, eps_rms, scale,
 * initial_state); out_dtype there is the dtype of dy.  Its out, final_state,
 * conv_state_out, chunk, flags and segments are ignored; its workspace and
 * workspace_bytes are this call's scratch (kda_backward_workspace_size).
 * Supported: D = 128, io bf16 or fp32; arithmetic is fp32 (the decays e^g
 * and the gate sigmoid through the IEEE functions, the recomputed SiLU and its
 * derivative through the fast exponential and reciprocal, a few ulp; the
 * chunk products on the tensor cores as three TF32 terms of hi/lo splits,
 * close to fp32), so the result does not depend on the forward's path.
 *
 * Method: conv + SiLU + L2 norms recomputed per token; for every 16-token
 * chunk, all at once, the parts that do not involve the state (decayed keys
 * and queries, the chunk's triangular products and (I + A)^-1); the
 * recurrence replayed chunk by chunk, saving o_t, e_t = v_t - S_bar^T k_t and
 * the state at the start of every 64-token segment; the epilogue's derivative
 * per row; the state gradient run backwards chunk by chunk, saving
 * w_t = dS^T k_t and the gradient at the end of every segment; then every
 * segment in parallel, chunk by chunk from its two checkpoints (with e and w
 * known): dq, dk and the log-decay's gradient, which follows from g entering
 * only through the decayed read keys and queries and the un-decayed written
 * keys; last the L2 norm's, SiLU's and the conv's derivatives.  No per-token
 * state is stored.
 *
 * Needs cu_seqlens_host (the checkpoint layout is planned on the host).  The
 * outputs must not overlap each other or any input.  dconv_w and drms_w are
 * zeroed by the call and accumulated with atomics, so their last bits depend
 * on the order blocks finish.  Every pointer 16-byte aligned except beta,
 * dbeta (4-byte).
 * ------------------------------------------------------------------------ */
typedef struct {
    kda_prefill_args fwd;       /* the forward call (see above) + this call's workspace */
    const void* dy;             /* [T_total][H][D] fwd.out_dtype */
    const float* d_final_state; /* [N][H][D][D] fp32, or NULL (zero) */
    float* dq;
    float* dk;
    float* dv;
    float* dconv_w;
    float* dg;
    float* dbeta;
    float* dgate;
    float* drms_w;
    float* dinitial_state;
    float* dconv_state_in;
} kda_backward_args;

/* Bytes of workspace kda_backward needs (reads fwd.N, H, D, T_total and
 * fwd.cu_seqlens_host, which is required), each part rounded up to 256:
 *   36 T_total H D + 8 T_total H + 8 slots D^2 + 8 slots D
 *   + 16 slots (49 D + 784) + 4 N H D + 8 (N + 1),
 * slots = H times the sum over sequences of ceil(len / 64): 6.6 GB for one
 * sequence of 8192 tokens with 96 heads. */
kda_status kda_backward_workspace_size(const kda_backward_args* args, size_t* bytes);

kda_status kda_backward(const kda_backward_args* args, kda_stream_t stream);

/* ========================================================================
 * The operators around the layer in a hybrid block: the layer norm in front
 * of the projections, 8-bit storage of the activations that a backward pass
 * reads, and a second recurrent mixer, the selective state space scan with
 * its short causal convolution.  They keep the conventions at the top of this
 * file.  Unlike the entry points above, they put no rule on the alignment of
 * rows or row strides beyond the element's own size: a layout that allows
 * 16-byte accesses takes them, any other takes scalar ones.
 * ======================================================================== */

/* ------------------------------------------------------------------------
 * kda_layer_norm -- y = (x - mean) / sqrt(var + eps) * weight + bias over the
 * last axis of x, var the mean of the squared deviations (two passes over the
 * registers, so a row whose mean is large loses nothing).  fp32 throughout: a
 * variance beyond its range makes rstd 0 and y the bias.  How a row is summed
 * depends on M (many rows share a block's work), so its last bits may too.
 *
 *   x, y    [M][row stride] io; y must not overlap x.
 *   weight, bias  [C] fp32, or NULL (ones, zeros).
 *   stats   [M][2] fp32 (mean, 1 / sqrt(var + eps)), what kda_layer_norm_backward
 *           reads, or NULL (not wanted); 8-byte aligned.
 * C in [1, 32768]; M >= 0.
 * ------------------------------------------------------------------------ */
typedef struct {
    int64_t M;
    int C;
    kda_dtype io;
    const void* x;
    int64_t x_stride;      /* elements between rows; 0 means C */
    const float* weight;
    const float* bias;
    float eps;
    void* y;
    int64_t y_stride;      /* 0 means C */
    float* stats;
} kda_norm_args;

kda_status kda_layer_norm(const kda_norm_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_layer_norm_backward -- with xh = (x - mean) rstd and p = dy weight:
 *   dx = rstd (p - mean(p) - xh mean(p xh)),  dweight = sum_rows dy xh,  dbias = sum_rows dy.
 * The mean is subtracted from x first, so that a large one costs no digits here either.
 *
 *   x        the forward's input (io), or its 8-bit form (x_scales non-NULL: x is
 *            then [M][C] codes and x_scales [M][ceil(C/32)], both dense, as
 *            kda_pack8 writes them; the pass reads them directly).
 *   stats    what the forward wrote (of the unrounded x).
 *   dx       [M][dx_stride] io, rounded once; must not overlap an input.
 *   dweight, dbias  [C] fp32, or NULL (not wanted).  Summed in a fixed order
 *            (per block over its rows, then over the blocks): two calls give the
 *            same bits.
 *   workspace  kda_layer_norm_backward_workspace_size bytes, 256-byte aligned
 *            (0 when neither dweight nor dbias is wanted); read and written by
 *            this call alone, nothing in it needs a value before.
 * ------------------------------------------------------------------------ */
typedef struct {
    int64_t M;
    int C;
    kda_dtype io;
    const void* dy;
    int64_t dy_stride;     /* 0 means C */
    const void* x;
    int64_t x_stride;      /* 0 means C; ignored for 8-bit x */
    const uint8_t* x_scales;
    const float* stats;
    const float* weight;
    void* dx;
    int64_t dx_stride;     /* 0 means C */
    float* dweight;
    float* dbias;
    void* workspace;
    size_t workspace_bytes;
} kda_norm_backward_args;

kda_status kda_layer_norm_backward_workspace_size(const kda_norm_backward_args* args, size_t* bytes);
kda_status kda_layer_norm_backward(const kda_norm_backward_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_pack8 / kda_unpack8 -- rows stored in 8 bits for a backward pass.
 *
 * Every 32 channels of a row share one power of two 2^e, the smallest with
 * max|x| <= 448 * 2^e (e >= -126; -126 for a block of zeros); codes hold
 * x 2^-e rounded to e4m3 (nearest, ties to even: at most 2^-4 relative, or
 * 2^-10 * 2^e absolute below the smallest normal code), scales hold e + 127.
 * Scaling by powers of two is exact, so the code's rounding is the only one.
 * NaN and infinities are kept as NaN and leave the block's maximum alone.
 *
 *   x       [M][x_stride] dtype (kda_pack8 in, kda_unpack8 out); 0 means C
 *   codes   [M][C] bytes;  scales [M][ceil(C/32)] bytes; both dense; C <= 2^30
 * ------------------------------------------------------------------------ */
#define KDA_PACK8_BLOCK 32

kda_status kda_pack8(const void* x, int64_t x_stride, kda_dtype dtype, int64_t M, int C, uint8_t* codes,
                     uint8_t* scales, kda_stream_t stream);
kda_status kda_unpack8(const uint8_t* codes, const uint8_t* scales, int64_t M, int C, void* x,
                       int64_t x_stride, kda_dtype dtype, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * The selective state space mixer: a second recurrent mixer beside the KDA
 * layer, with a diagonal state of N values per channel and a decay that
 * depends on the token.  Per channel c and state n:
 *
 *   conv   u_t = act(bias + sum_{j=0..3} w[j] x[t-3+j]),  act = SiLU or none
 *   step   delta_t = softplus(dt_t + dt_bias)       (softplus = 0: delta_t = dt_t + dt_bias)
 *   scan   h_t[n] = exp(delta_t A[c][n]) h_{t-1}[n] + delta_t u_t B_t[g][n]
 *   read   y_t = (sum_n C_t[g][n] h_t[n] + D u_t) silu(z_t)
 *
 * Channels 0 .. C-1 form G groups of C/G consecutive ones; a group shares its
 * B and C rows.  Between conv and scan a model projects u to dt, B and C
 * (kda_gemm), which is why they are two entry points.  Sequences are packed
 * (cu_seqlens as for kda_prefill; zero lengths allowed, their final state is
 * their initial state) and never see each other's tokens.  States, decays and
 * every sum are fp32; only what is stored in io is rounded to it.
 *
 * kda_ssm_conv -- the convolution over packed sequences.
 *   x, y      [T_total][row stride] io, C channels; y must not overlap x.
 *   C         up to 2^20
 *   w         [C][4] fp32 (tap 3 multiplies x[t]; shorter filters: leading zeros)
 *   bias      [C] fp32 or NULL (zeros);  silu nonzero: SiLU after the sum
 *   conv_state_in   [N][C][3] io, oldest first, or NULL (zeros)
 *   conv_state_out  [N][C][3] io or NULL: the last three raw values of every
 *             sequence (conv_state_in's where it is shorter); must not overlap
 *             conv_state_in.
 * ------------------------------------------------------------------------ */
typedef struct {
    int N;                 /* sequences */
    int C;                 /* channels */
    int64_t T_total;       /* packed tokens */
    kda_dtype io;
    int silu;
    const int32_t* cu_seqlens;       /* device [N+1] */
    const int32_t* cu_seqlens_host;  /* host [N+1] or NULL (then only device-checked) */
    const void* x;
    int64_t x_stride;      /* elements between tokens; 0 means C */
    const float* w;
    const float* bias;
    const void* conv_state_in;
    void* conv_state_out;
    void* y;
    int64_t y_stride;      /* 0 means C */
    int* d_status;
} kda_ssm_conv_args;

kda_status kda_ssm_conv(const kda_ssm_conv_args* args, kda_stream_t stream);

/* One token for each of N sequences (T_total is ignored, x and y have N rows, cu_seqlens is
 * ignored): conv_state_out is read and rolled in place, conv_state_in must be NULL. */
kda_status kda_ssm_conv_step(const kda_ssm_conv_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_ssm_conv_backward -- with pre_t the convolution's sum before the activation and
 * dpre_t = dy_t act'(pre_t):
 *   dx_t = sum_j w[j] dpre_{t+3-j} (inside the sequence);  dw[j] = sum_t dpre_t x[t-3+j];
 *   dbias = sum_t dpre_t;  dconv_state_in the same sum at the three places before the start.
 * fwd: N, C, T_total, io, silu, cu_seqlens (and host copy), x, x_stride, w, bias and
 * conv_state_in as in the forward call; the rest of it is ignored.  dx is [T_total][dx_stride] io,
 * rounded once; dw [C][4], dbias [C] (NULL: not wanted) and dconv_state_in [N][C][3] (NULL: not
 * wanted) are fp32.  dw and dbias are summed in a fixed order.  workspace:
 * kda_ssm_conv_backward_workspace_size bytes, 256-byte aligned.
 * ------------------------------------------------------------------------ */
typedef struct {
    kda_ssm_conv_args fwd;
    const void* dy;
    int64_t dy_stride;     /* 0 means C */
    void* dx;
    int64_t dx_stride;     /* 0 means C */
    float* dw;
    float* dbias;
    float* dconv_state_in;
    void* workspace;
    size_t workspace_bytes;
} kda_ssm_conv_backward_args;

kda_status kda_ssm_conv_backward_workspace_size(const kda_ssm_conv_backward_args* args, size_t* bytes);
kda_status kda_ssm_conv_backward(const kda_ssm_conv_backward_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_ssm_scan -- the scan over packed sequences.
 *   u, dt, z, y  [T_total][row stride] io, C channels; z NULL: no gate.  y must not overlap an input.
 *   A         [C][Nst] fp32, expected <= 0 (positive values grow the state without bound)
 *   B, Cm     [T_total][row stride] io, each row G groups of Nst
 *   D         [C] fp32 or NULL (zeros);  dt_bias [C] fp32 or NULL (zeros)
 *   initial_state  [N][C][Nst] fp32 or NULL (zeros)
 *   final_state    [N][C][Nst] fp32 or NULL; must not overlap initial_state
 * C up to 2^20; Nst in {8, 16, 32, 64}; G >= 1 divides C.  A, the states and the workspace 16-byte aligned
 * (the workspace 256).
 *
 * A long stream with few channels is cut into equal pieces of the packed token axis (whatever the
 * sequences' borders): a first kernel takes every piece but the last from a zero state, a second
 * joins them (the state at a piece's start is the carried one times exp(A times the sum of delta),
 * plus what the piece before added), and the main kernel runs all pieces at once.  The workspace
 * holds one state and one sum of delta per piece; none when one piece suffices.
 * ------------------------------------------------------------------------ */
typedef struct {
    int N;                 /* sequences */
    int C;                 /* channels */
    int Nst;               /* states per channel */
    int G;                 /* groups of B and Cm */
    int64_t T_total;
    kda_dtype io;
    int softplus;
    const int32_t* cu_seqlens;
    const int32_t* cu_seqlens_host;
    const void* u;
    int64_t u_stride;      /* 0 means C */
    const void* dt;
    int64_t dt_stride;     /* 0 means C */
    const float* A;
    const void* B;
    int64_t B_stride;      /* 0 means G*Nst */
    const void* Cm;
    int64_t C_stride;      /* 0 means G*Nst */
    const float* D;
    const void* z;
    int64_t z_stride;      /* 0 means C */
    const float* dt_bias;
    const float* initial_state;
    float* final_state;
    void* y;
    int64_t y_stride;      /* 0 means C */
    void* workspace;
    size_t workspace_bytes;
    int* d_status;
} kda_ssm_args;

kda_status kda_ssm_scan_workspace_size(const kda_ssm_args* args, size_t* bytes);
kda_status kda_ssm_scan(const kda_ssm_args* args, kda_stream_t stream);

/* One token for each of N sequences: rows of u, dt, B, Cm, z and y are the sequences, and
 * final_state is read and updated in place (initial_state must be NULL; T_total, cu_seqlens and
 * the workspace are ignored).  Row strides are below 4 GB. */
kda_status kda_ssm_step(const kda_ssm_args* args, kda_stream_t stream);

/* ------------------------------------------------------------------------
 * kda_ssm_backward -- the gradients of one kda_ssm_scan call.  With g_t = dy_t silu(z_t) and
 * lambda_t the gradient of h_t:
 *   lambda_t = C_t g_t + a_{t+1} lambda_{t+1}   (d_final_state joins at a sequence's last token)
 *   dC_t = sum_c g_t h_t;  dB_t = sum_c lambda_t delta_t u_t;  dA = sum_t lambda_t a_t h_{t-1} delta_t
 *   du_t = delta_t sum_n lambda_t B_t + D g_t;  dD = sum_t g_t u_t
 *   ddelta_t = u_t sum_n lambda_t B_t + sum_n lambda_t a_t h_{t-1} A;  ddt_t = ddelta_t softplus'
 *   dz_t = dy_t (sum_n C_t h_t + D u_t) silu'(z_t);  dinitial_state = a_1 lambda_1
 * fwd: the forward call's arguments; its y, final_state and workspace are ignored (the states are
 * recomputed).  du, ddt, dz, dB and dC are io, dense ([T_total][C], [T_total][G][Nst]), rounded
 * once; dA [C][Nst], dD [C], ddt_bias [C] and dinitial_state [N][C][Nst] are fp32.  dz, dD,
 * ddt_bias and dinitial_state may be NULL (not wanted); the others must not.  G is at most 65535.  Sums over channels
 * and tokens go through the workspace in a fixed order.  The workspace grows with the tokens: it holds the fp32 states
 * in front of every fourth one, T_total * C * Nst bytes, and the parts of dB and dC (13 GB and more for 65,536 tokens x
 * 12,288 channels x 16 states), for this call alone.
 * ------------------------------------------------------------------------ */
typedef struct {
    kda_ssm_args fwd;
    const void* dy;
    int64_t dy_stride;     /* 0 means C */
    const float* d_final_state;  /* [N][C][Nst] fp32 or NULL (zeros) */
    void* du;
    void* ddt;
    float* dA;
    void* dB;
    void* dC;
    float* dD;
    void* dz;
    float* ddt_bias;
    float* dinitial_state;
    void* workspace;
    size_t workspace_bytes;
} kda_ssm_backward_args;

kda_status kda_ssm_backward_workspace_size(const kda_ssm_backward_args* args, size_t* bytes);
kda_status kda_ssm_backward(const kda_ssm_backward_args* args, kda_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
