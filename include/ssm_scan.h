/*
 * ssm_scan.h -- C ABI of libssmscan.so, the selective state-space scan
 * (Mamba's S6 layer core) for AMD Instinct MI355X (gfx950), and beside it the
 * head-decay mixer: decay attention and the group norm that follows it; and what
 * stands around the scan in a layer of packed sequences: the packed scan, the short
 * convolution and the residual norm (their own conventions stand with them below).
 *
 * What is computed.  For every batch row b, channel d and state n the library
 * runs one diagonal single-input single-output state-space model:
 *
 *   Abar_t[n] = exp(Delta[b,t,d] * A[d,n])
 *   Bbar_t[n] = Delta[b,t,d] * B[b,t,n]                       (SSM_DISC_DELTA_B)
 *             = (exp(Delta[b,t,d] A[d,n]) - 1) / A[d,n] * B[b,t,n]   (SSM_DISC_ZOH)
 *   h_t[n]    = Abar_t[n] * h_{t-1}[n] + Bbar_t[n] * u[b,t,d]
 *   y[b,t,d]  = sum_n C[b,t,n] * h_t[n] + Dskip[d] * u[b,t,d]
 *
 * with h_{-1} = h0 (zero when h0 is NULL) and u the scan input: x itself, or
 * the causal depthwise conv1d + SiLU of x when conv_w is given,
 *
 *   u[b,t,d] = silu(conv_b[d] + sum_{k<K} conv_w[d,k] * x[b, t-K+1+k, d]),
 *   x[b, t<0, d] = conv_state_in[b, d, K-1+t] (0 when conv_state_in is NULL),
 *   silu(z) = z / (1 + exp(-z)).
 *
 * Optional fused steps around the scan:
 *   - step size from its pre-activation: Delta = delta + delta_bias[d], and
 *     with delta_softplus Delta = softplus(delta + delta_bias[d]),
 *     softplus(v) = log(1 + exp(v));
 *   - output gate: y[b,t,d] is multiplied by silu(z[b,t,d]);
 *   - conv window across calls: conv_state_out[b, d, j] = x[b, L-K+1+j, d]
 *     (the last K-1 inputs, oldest first, reaching into conv_state_in when
 *     L < K-1), so a sequence scanned in pieces, or a prefill followed by
 *     ssm_step calls, sees the same window as one call.
 *
 * Passages defining each step (web pages on Mamba; section names as printed):
 *   - continuous SSM, ZOH discretization Abar = exp(Delta A),
 *     Bbar = (Delta A)^-1 (exp(Delta A) - I) Delta B, and the discrete
 *     recurrence h_k = Abar h_{k-1} + Bbar x_k, y_k = C h_k + D x_k:
 *     gsyq.cn "Mamba 状态空间模型深度解析", section "连续到离散的转换";
 *   - the simplified Bbar = Delta * B and the scan h = associative_scan(
 *     A_bar, B_bar * x), y = C * h: same page, section "硬件优化并行扫描算法";
 *   - A kept continuous and discretized on the fly; one independent SSM per
 *     channel with A (D, N), B and C (batch, L, N), Delta (batch, L, D); C is
 *     a 1 x N row, so the readout contracts over n: VMamba reading note,
 *     sections "离散化SSM", "S4中三个矩阵的维度表示、维度变化" and
 *     "mamba：从S4到S6的算法变化流程";
 *   - the causal depthwise Conv1d (padding d_conv - 1, groups = d_model) before
 *     the SSM and the skip D * x_conv on the conv output: gsyq.cn section
 *     "选择性的实现细节" (SelectiveSSM);
 *   - the single-token recurrent step with a cached state (constant cost per
 *     generated token): 53ai.com explainer, section "一、Motivation", and the
 *     datacamp tutorial's complexity table;
 *   - Delta = Softplus(Linear(x)), the bias of that projection being
 *     delta_bias: gsyq.cn section "选择性的数学解析"; VMamba note section
 *     "mamba：从S4到S6的算法变化流程" (tau_Delta = softplus);
 *   - the gated block around the SSM (H3 block merged with a gated MLP):
 *     VMamba note section "简化的SSM架构".  The page's figure with the gate
 *     formula is lost; y * silu(z), applied after the skip term, is the
 *     reading taken.
 *
 * Conventions shared by every entry point.
 *   Layout     all arrays are dense, row-major, last dimension fastest:
 *              x, Delta, y (batch, L, D); B, C (batch, L, N); A (D, N);
 *              Dskip, conv_b, delta_bias (D); conv_w (D, K); h0, h_last
 *              (batch, D, N); z like x; conv_state_in / conv_state_out
 *              (batch, D, K-1) fp32, oldest input first.
 *              Base pointers must be aligned to their element size; B and C
 *              rows are read with scalar loads, so B and C base pointers must
 *              be 4-byte aligned and are best 64-byte aligned.
 *   Memory     every pointer is a DEVICE pointer owned by the caller.  The
 *              library allocates nothing, keeps no pointer after the call and
 *              holds no global mutable state apart from the scratch array of
 *              ssm_scan_fwd_noalloc and its per-device address table; every
 *              entry point except that one is reentrant and thread-safe.
 *   Streams    hip_stream is a hipStream_t (NULL = the default stream).  Work
 *              is enqueued asynchronously; the call never synchronizes.  A
 *              call enqueues kernel launches only (plus the optional timing
 *              events), with no memset or copy, so it may be recorded by
 *              stream capture into a HIP graph and replayed; a replay reads
 *              the buffers whose addresses were passed when it was captured.
 *   Errors     all argument checks run on the host before anything is
 *              enqueued; on any error the outputs are untouched and the
 *              status says why (ssm_last_error_message() has the detail).  A
 *              failed launch returns SSM_ERR_HIP; faults inside kernels
 *              surface at the caller's next synchronization.
 *   Dtypes     x, Delta, B, C, z share in_dtype (fp32 or bf16); y has
 *              out_dtype; A, Dskip, delta_bias, conv weights, conv states and
 *              h are fp32; arithmetic and the state are fp32; bf16 outputs are
 *              rounded to nearest even.
 *   Empty      seqlen == 0 or batch * dim == 0 is valid.  With seqlen == 0 and
 *              batch * dim > 0, h_last (if given) receives h0 (zeros if h0 is
 *              NULL), conv_state_out (if given) receives conv_state_in (zeros
 *              if NULL), and nothing else is touched.
 */
#ifndef SSM_SCAN_H_
#define SSM_SCAN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SSM_ABI_VERSION 3

typedef enum {
  SSM_OK = 0,
  SSM_ERR_NULL = 1,        /* a required pointer (or the args struct) is NULL */
  SSM_ERR_SHAPE = 2,       /* negative sizes, or byte counts overflow int64 */
  SSM_ERR_DTYPE = 3,       /* unknown dtype or discretization enum value */
  SSM_ERR_UNSUPPORTED = 4, /* dstate not in {1,2,4,8,16}, conv_k not in 1..4,
                              misaligned pointer, negative chunk_len, reserved != 0,
                              delta_softplus not 0/1, conv state without conv_w,
                              h_saved with a split scan whose chunk_len is not a
                              multiple of 4 */
  SSM_ERR_ALIAS = 5,       /* an output overlaps an input or another output */
  SSM_ERR_WORKSPACE = 6,   /* workspace NULL or smaller than required */
  SSM_ERR_HIP = 7          /* the HIP runtime rejected a launch */
} ssm_status_t;

typedef enum { SSM_F32 = 0, SSM_BF16 = 1 } ssm_dtype_t;

typedef enum { SSM_DISC_DELTA_B = 0, SSM_DISC_ZOH = 1 } ssm_disc_t;

typedef struct {
  int64_t batch, seqlen, dim, dstate; /* Bt, L, D, N */
  int32_t in_dtype;                   /* ssm_dtype_t of x, delta, Bm, Cm */
  int32_t out_dtype;                  /* ssm_dtype_t of y */
  int32_t disc;                       /* ssm_disc_t */
  int32_t conv_k;                     /* taps of the conv prologue (1..4); ignored if conv_w is NULL */
  const void* x;                      /* (Bt, L, D) */
  const void* delta;                  /* (Bt, L, D), the step size, already positive */
  const float* A;                     /* (D, N), continuous-time diagonal */
  const void* Bm;                     /* (Bt, L, N) */
  const void* Cm;                     /* (Bt, L, N) */
  const float* Dskip;                 /* (D) or NULL = no skip term */
  const float* h0;                    /* (Bt, D, N) or NULL = zero initial state */
  float* h_last;                      /* (Bt, D, N) or NULL: state after the last token */
  void* y;                            /* (Bt, L, D) output */
  const float* conv_w;                /* (D, K) or NULL = no conv prologue */
  const float* conv_b;                /* (D) or NULL = zero bias */
  void* workspace;                    /* device scratch of >= ssm_scan_workspace_size() bytes */
  size_t workspace_bytes;
  int32_t chunk_len;                  /* time steps per chunk; 0 = library's choice */
  int32_t reserved;                   /* must be 0 */
  void* ev_main_start;                /* optional hipEvent_t recorded on hip_stream right */
  void* ev_main_stop;                 /* before / after the output-pass kernel; NULL = none */
  /* since ABI 2 */
  const float* delta_bias;            /* (D) or NULL = 0, added to delta */
  int32_t delta_softplus;             /* 1: Delta = softplus(delta + delta_bias); 0: no softplus */
  int32_t reserved2;                  /* must be 0 */
  const void* z;                      /* (Bt, L, D) gate or NULL = no gate: y *= silu(z) */
  const float* conv_state_in;         /* (Bt, D, K-1) inputs before token 0, or NULL = zeros;
                                         requires conv_w */
  float* conv_state_out;              /* (Bt, D, K-1) receives the last K-1 inputs, or NULL;
                                         requires conv_w; must not overlap any other buffer */
  /* since ABI 3 */
  float* h_saved;                     /* (Bt, S, D, N) fp32 or NULL, S = ceil(L / 16) - 1:
                                         receives the state entering steps 16, 32, ..., 16 S
                                         (h_saved[b][k-1] = h before step 16 k), for
                                         ssm_scan_bwd; must not overlap any other buffer.
                                         When the scan is split into chunks, their length
                                         must be a multiple of 4 (the planned length is) */
} ssm_scan_args_t;

typedef struct {
  int64_t batch, dim, dstate;         /* Bt, D, N */
  int32_t in_dtype;                   /* ssm_dtype_t of x, delta, Bm, Cm */
  int32_t out_dtype;                  /* ssm_dtype_t of y */
  int32_t disc;                       /* ssm_disc_t */
  int32_t reserved;                   /* must be 0 */
  const void* x;                      /* (Bt, D) the new token's scan input */
  const void* delta;                  /* (Bt, D) */
  const float* A;                     /* (D, N) */
  const void* Bm;                     /* (Bt, N) */
  const void* Cm;                     /* (Bt, N) */
  const float* Dskip;                 /* (D) or NULL */
  float* h;                           /* (Bt, D, N) cached state, updated in place;
                                         aligned to 4 * min(N, 4) bytes */
  void* y;                            /* (Bt, D) output, read from the updated state */
  /* since ABI 2 */
  const float* delta_bias;            /* (D) or NULL = 0, added to delta */
  int32_t delta_softplus;             /* 1: Delta = softplus(delta + delta_bias) */
  int32_t conv_k;                     /* taps of the conv (1..4); ignored if conv_w is NULL */
  const void* z;                      /* (Bt, D) gate or NULL: y *= silu(z) */
  const float* conv_w;                /* (D, K) or NULL = no conv: u = x */
  const float* conv_b;                /* (D) or NULL = zero bias */
  float* conv_state;                  /* (Bt, D, K-1) conv window, updated in place (shifted to
                                         end with x); required when conv_w is given and K > 1 */
} ssm_step_args_t;

/* Backward selective scan: gradients of
 *   loss = sum(dy * y) + sum(dh_last * h_last)
 * for ssm_scan_fwd without fused steps (no conv prologue, Delta as given, no
 * gate).  The derivative of the recurrence defined above (the pages name
 * training as the purpose of the parallel scan -- explainer, section "3.6
 * Empirical Evaluation"; VMamba note, section "硬件感知的设计" -- and print
 * no gradient formula; the chain rule of the definition is the reading):
 *   g_t = C_t dy_t + Abar_{t+1} g_{t+1} (g_{L-1} also receives dh_last),
 *   dx_t = sum_n g_t f_t B_t + Dskip dy_t, dDelta_t, dA, dB, dC, dD, dh0.
 * All gradients are fp32 and overwritten (not accumulated).  Inputs are as
 * in ssm_scan_args_t; dy has in_dtype.  The adjoint is chunked like the
 * forward scan and the forward states are recomputed between states kept
 * every 16 steps, so nothing of size batch x L x D x N is stored.  The
 * states every 16 steps are either computed here (a forward summary and
 * carry pass) or taken from the forward scan of the same inputs (h_saved of
 * ssm_scan_args_t), which skips that pass. */
typedef struct {
  int64_t batch, seqlen, dim, dstate; /* Bt, L, D, N */
  int32_t in_dtype;                   /* ssm_dtype_t of x, delta, Bm, Cm, dy */
  int32_t disc;                       /* ssm_disc_t */
  int32_t super_chunk;                /* steps per adjoint chunk (multiple of 16); 0 = plan */
  int32_t reserved;                   /* must be 0 */
  const void* x;                      /* (Bt, L, D) */
  const void* delta;                  /* (Bt, L, D) */
  const float* A;                     /* (D, N) */
  const void* Bm;                     /* (Bt, L, N) */
  const void* Cm;                     /* (Bt, L, N) */
  const float* Dskip;                 /* (D) or NULL */
  const float* h0;                    /* (Bt, D, N) or NULL */
  const void* dy;                     /* (Bt, L, D) gradient of y */
  const float* dh_last;               /* (Bt, D, N) gradient of h_last, or NULL */
  float* dx;                          /* (Bt, L, D) */
  float* ddelta;                      /* (Bt, L, D) */
  float* dA;                          /* (D, N) */
  float* dB;                          /* (Bt, L, N) */
  float* dC;                          /* (Bt, L, N) */
  float* dD;                          /* (D) or NULL */
  float* dh0;                         /* (Bt, D, N) or NULL */
  void* workspace;                    /* >= ssm_scan_bwd_workspace_size() bytes */
  size_t workspace_bytes;
  void* ev_main_start;                /* optional hipEvent_t recorded on hip_stream right */
  void* ev_main_stop;                 /* before / after the main backward kernel; NULL = none */
  /* since ABI 3 */
  const float* h_saved;               /* (Bt, ceil(L / 16) - 1, D, N) or NULL: the states
                                         ssm_scan_fwd wrote to its h_saved for the same x,
                                         delta, A, Bm, h0 (and disc); NULL = computed here */
} ssm_scan_bwd_args_t;

/* Bytes of device scratch the allocation-free forward entry point holds per
 * GPU (see ssm_scan_fwd_noalloc). */
#define SSM_NOALLOC_SCRATCH_BYTES (64u << 20)

/* Returns SSM_ABI_VERSION. */
int ssm_abi_version(void);

/* Bytes of device workspace ssm_scan_fwd needs for these arguments (0 when the
 * plan scans each sequence in one piece).  Reads only the sizes, chunk_len and
 * dtypes; pure host function, no HIP call.  Returns 0 for invalid sizes. */
size_t ssm_scan_workspace_size(const ssm_scan_args_t* args);

/* Time steps per chunk the plan uses for these arguments (equal to seqlen
 * when the scan is not split).  Pure host function; 0 for invalid sizes.
 * With chunk_len = 0, sequences of at most 32 steps are not split, and short
 * sequences of few channels (seqlen <= 512 and batch * dim * ceil(seqlen /
 * 64) <= min(4096, 64 * seqlen)) run as one
 * pass with the time steps across a wave's lanes, each block of 64 steps
 * solved by a parallel associative scan over the lanes (53ai.com explainer,
 * section 3.3); that plan reports seqlen and needs no workspace. */
int64_t ssm_scan_plan_chunk_len(const ssm_scan_args_t* args);

/* 1 when the plan for these arguments is that one-pass lane scan (one
 * kernel, k_scan_wave), 0 when it is the chunked passes (chunk summaries,
 * carry combine and output pass; a single chunk runs the output pass alone)
 * or the sizes are invalid.  Pure host function, no HIP call. */
int32_t ssm_scan_plan_lane_scan(const ssm_scan_args_t* args);

/* Selective-scan forward: y and (optionally) h_last from the inputs above.
 * The time axis may be split into chunks scanned in parallel; their carries
 * are combined with the associative operator
 *   (a, b) o (a', b') = (a a', a' b + b')
 * which is exact up to floating-point rounding order. */
ssm_status_t ssm_scan_fwd(const ssm_scan_args_t* args, void* hip_stream);

/* ssm_scan_fwd for callers that cannot allocate device memory: code under
 * HIP graph capture, serving loops, and harnesses that forbid hipMalloc.
 * Same arguments and results as ssm_scan_fwd, except that workspace and
 * workspace_bytes are ignored: the chunk summaries, carries and group
 * carries live in a device array of SSM_NOALLOC_SCRATCH_BYTES that the
 * library keeps on every GPU it runs on, until the process ends.  The call
 * allocates nothing.
 *   - Plan: the library's plan when its summaries fit the array; otherwise
 *     the same plan with chunks lengthened until they do (results then
 *     differ from ssm_scan_fwd's by rounding order only).  A chunk_len the
 *     caller forces is kept, and the call fails with SSM_ERR_WORKSPACE if
 *     its summaries do not fit.  ssm_scan_plan_chunk_len reports the
 *     ordinary plan, not this one.
 *   - The array's device address is looked up (hipGetSymbolAddress) on the
 *     first call on each device that needs it, with that device current;
 *     make that first call outside stream capture.  hip_stream must belong
 *     to the current device (SSM_ERR_UNSUPPORTED otherwise).
 *   - Every call on one GPU shares that GPU's array: calls that overlap in
 *     time on one GPU (concurrent streams, or threads) race and corrupt each
 *     other's results.  Serialize them, e.g. on one stream.  Nothing in the
 *     array needs clearing between calls; it keeps the last call's contents.
 * Errors as for ssm_scan_fwd. */
ssm_status_t ssm_scan_fwd_noalloc(const ssm_scan_args_t* args, void* hip_stream);

/* One recurrent decode step per sequence: u = x (or the conv over the
 * window conv_state followed by x, then SiLU), h <- Abar h + Bbar u, then
 * y = (C . h + Dskip * u) (* silu(z)), with h and conv_state updated in
 * place.  Same arithmetic as ssm_scan_fwd with seqlen = 1, h0 = h_last = h
 * and conv_state_in = conv_state_out = conv_state.  y must not overlap h,
 * conv_state or any input. */
ssm_status_t ssm_step(const ssm_step_args_t* args, void* hip_stream);

/* Bytes of device workspace ssm_scan_bwd needs (never 0 for a non-empty
 * problem; smaller when h_saved is given).  Pure host function; 0 for
 * invalid sizes. */
size_t ssm_scan_bwd_workspace_size(const ssm_scan_bwd_args_t* args);

/* Backward selective scan (see ssm_scan_bwd_args_t).  Asynchronous on
 * hip_stream; outputs must not overlap each other, the inputs or the
 * workspace.  Errors as for ssm_scan_fwd. */
ssm_status_t ssm_scan_bwd(const ssm_scan_bwd_args_t* args, void* hip_stream);

/* ---------------------------------------------------------------------------
 * Decay attention: linear attention with a decay for each head, the state-space
 * model whose A is one scalar per head.  For every batch row b and head h
 *
 *   S_t = exp(log_decay[b,t,h]) S_{t-1} + k_t v_t^T       S (key_dim, value_dim)
 *   o_t = S_t^T q_t
 *
 * with S_{-1} = h0 (zero when NULL), v_t = v[b,t,h,:] and q_t, k_t those of key
 * head h / (heads / key_heads): heads that share a key head are consecutive.
 * The recurrence is the one of "连续到离散的转换" (gsyq.cn, "Mamba 状态空间模型
 * 深度解析") with Abar a scalar of the head, Bbar x = k v^T and C = q.
 *
 * Conventions, where they differ from the scan's:
 *   Layout   q, k (batch, L, key_heads, key_dim); v, o, dout (batch, L, heads,
 *            value_dim); log_decay (batch, L, heads); states (batch, heads,
 *            key_dim, value_dim) fp32.  The last dimension of q, k, v, dout is
 *            contiguous; the others have the strides given (in elements, not
 *            negative, 0 for a broadcast), so slices of one projection's
 *            output need no copy.  Outputs and states are dense.
 *   Lengths  lengths[b] (device, int32, taken as clamped to 0..L; NULL = all L)
 *            is the number of tokens of row b.  Later tokens are not read (they
 *            may hold anything, NaN included): o and every gradient are 0
 *            there, and h_last is the state after the last of the row's tokens
 *            (h0 for a row without any).
 *   Decay    any log_decay is taken, growth (above 0) included: -inf, or a value
 *            whose exp is 0 in fp32, resets the state, and what is zero stays
 *            zero however much it grows.  From a block of 64 tokens on whose
 *            log decays above 0 add up to more than 22, its head is walked token
 *            by token (4 x 8192 x 20 heads of 128 x 128, bf16: 1.8 ms for 0.24).
 *   Dtypes   q, k, v, o, dout, dq, dk, dv share dtype; log_decay and dlog_decay
 *            have decay_dtype; states and their gradients are fp32, and so are
 *            all sums.  With bf16 inputs the products of decayed scores with
 *            values, and of the state as it is read with q, run on operands
 *            rounded once to bf16 (in dq and dk kept to 16 bits): o has 1.4 times
 *            the error of its own rounding, where the single-token form, which
 *            reads the state in full, has once.  Updates of the state keep 24
 *            bits.
 *   Non-finite values of a token reach what the recurrence takes them to: that
 *            token and later ones, in gradients going backward that token and
 *            earlier ones.  A head is walked token by token from such a token's block on, where
 *            v (gradients: k, q or dout) holds them.  Rows past a length reach
 *            none.
 *   Sizes    1 <= key_dim, value_dim <= 256; heads a multiple of key_heads.
 *            Empty problems are valid: with L == 0, h_last = h0, dh0 = dh_last.
 * ------------------------------------------------------------------------- */

typedef struct {
  int64_t batch, seqlen, heads, key_heads, key_dim, value_dim;
  int32_t dtype;                      /* ssm_dtype_t of q, k, v, o */
  int32_t decay_dtype;                /* ssm_dtype_t of log_decay */
  int32_t span;                       /* tokens per span of the time axis, a multiple of 64;
                                         0 = plan */
  int32_t reserved;                   /* must be 0 */
  const void* q;                      /* (batch, L, key_heads, key_dim) */
  const void* k;                      /* (batch, L, key_heads, key_dim) */
  const void* v;                      /* (batch, L, heads, value_dim) */
  const void* log_decay;              /* (batch, L, heads) */
  int64_t q_stride[3];                /* batch, token, head, in elements */
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t decay_stride[3];
  const int32_t* lengths;             /* (batch) or NULL */
  const float* h0;                    /* (batch, heads, key_dim, value_dim) or NULL = 0 */
  float* h_last;                      /* like h0, or NULL */
  void* o;                            /* (batch, L, heads, value_dim) */
  void* workspace;                    /* >= ssm_decay_attn_workspace_size() bytes */
  size_t workspace_bytes;
} ssm_decay_attn_args_t;

typedef struct {
  int64_t batch, heads, key_heads, key_dim, value_dim;
  int32_t dtype;                      /* ssm_dtype_t of q, k, v, o */
  int32_t decay_dtype;                /* ssm_dtype_t of log_decay */
  const void* q;                      /* (batch, key_heads, key_dim) */
  const void* k;                      /* (batch, key_heads, key_dim) */
  const void* v;                      /* (batch, heads, value_dim) */
  const void* log_decay;              /* (batch, heads) */
  int64_t q_stride[2];                /* batch, head, in elements */
  int64_t k_stride[2];
  int64_t v_stride[2];
  int64_t decay_stride[2];
  float* h;                           /* (batch, heads, key_dim, value_dim), updated in place */
  void* o;                            /* (batch, heads, value_dim), read from the updated state */
} ssm_decay_attn_step_args_t;

/* Gradients of  loss = sum(dout * o) + sum(dh_last * h_last).  With G_t the
 * gradient of S_t (chain rule of the recurrence; G_{L-1} also gets dh_last):
 *   G_t = q_t dout_t^T + exp(log_decay_{t+1}) G_{t+1},
 *   dq_t = S_t dout_t, dk_t = G_t v_t, dv_t = G_t^T k_t,
 *   dlog_decay_t = exp(log_decay_t) <S_{t-1}, G_t>, dh0 = exp(log_decay_0) G_0;
 * dlog_decay is formed from the terms that pass token t alone (0 at a reset).
 * The workspace holds the state at every 64 tokens (fp32 rows: 32);
 * dq and dk are summed over the heads that share a key head, in a fixed
 * order.  All gradients are dense and overwritten. */
typedef struct {
  int64_t batch, seqlen, heads, key_heads, key_dim, value_dim;
  int32_t dtype;                      /* ssm_dtype_t of q, k, v, dout, dq, dk, dv */
  int32_t decay_dtype;                /* ssm_dtype_t of log_decay, dlog_decay */
  int32_t span;                       /* as in ssm_decay_attn_args_t */
  int32_t reserved;                   /* must be 0 */
  const void* q;
  const void* k;
  const void* v;
  const void* log_decay;
  const void* dout;                   /* (batch, L, heads, value_dim) gradient of o */
  int64_t q_stride[3];
  int64_t k_stride[3];
  int64_t v_stride[3];
  int64_t decay_stride[3];
  int64_t dout_stride[3];
  const int32_t* lengths;             /* (batch) or NULL */
  const float* h0;                    /* or NULL = 0 */
  const float* dh_last;               /* gradient of h_last, or NULL = 0 */
  void* dq;                           /* (batch, L, key_heads, key_dim) */
  void* dk;                           /* (batch, L, key_heads, key_dim) */
  void* dv;                           /* (batch, L, heads, value_dim) */
  void* dlog_decay;                   /* (batch, L, heads) */
  float* dh0;                         /* (batch, heads, key_dim, value_dim) or NULL */
  void* workspace;                    /* >= ssm_decay_attn_bwd_workspace_size() bytes */
  size_t workspace_bytes;
} ssm_decay_attn_bwd_args_t;

/* Bytes of device workspace the call needs (0: none).  Pure host functions that
 * read the sizes, dtypes and span; 0 for invalid sizes. */
size_t ssm_decay_attn_workspace_size(const ssm_decay_attn_args_t* args);
size_t ssm_decay_attn_bwd_workspace_size(const ssm_decay_attn_bwd_args_t* args);

/* Decay attention over whole sequences. */
ssm_status_t ssm_decay_attn_fwd(const ssm_decay_attn_args_t* args, void* hip_stream);

/* One token per sequence, the state updated in place. */
ssm_status_t ssm_decay_attn_step(const ssm_decay_attn_step_args_t* args, void* hip_stream);

/* Its gradients. */
ssm_status_t ssm_decay_attn_bwd(const ssm_decay_attn_bwd_args_t* args, void* hip_stream);

/* ---------------------------------------------------------------------------
 * Group norm with an activation or a gate, channels last.  Every row (token)
 * of x is normalized on its own, in groups of channels / groups neighbouring
 * channels (a causal model's statistics cannot span tokens):
 *
 *   u = x, or x silu(z) (SSM_NORM_GATE_FIRST)
 *   n = (u - mean) / sqrt(var + eps), or u / sqrt(mean(u^2) + eps) with rms
 *   a = n * weight + bias
 *   y = a (SSM_NORM_PLAIN, SSM_NORM_GATE_FIRST), silu(a) (SSM_NORM_SILU) or
 *       a silu(z) (SSM_NORM_GATE)
 *
 * var is the mean of (u - mean)^2.  x, z, y, dy, dx, dz share dtype; x, z and
 * dy have contiguous channels and the row strides given; outputs are dense;
 * weight, bias (NULL = 1, 0) and their gradients are (channels) fp32;
 * statistics and sums are fp32.  y may not overlap an input.
 * ------------------------------------------------------------------------- */

typedef enum {
  SSM_NORM_PLAIN = 0,
  SSM_NORM_SILU = 1,
  SSM_NORM_GATE = 2,
  SSM_NORM_GATE_FIRST = 3
} ssm_norm_mode_t;

typedef struct {
  int64_t rows, channels, groups;
  int64_t x_stride, z_stride;         /* elements from row to row (z_stride ignored without z) */
  int32_t dtype;                      /* ssm_dtype_t of x, z, y */
  int32_t mode;                       /* ssm_norm_mode_t */
  int32_t rms;                        /* 1: no mean is subtracted; 0: group norm */
  float eps;                          /* >= 0 */
  const void* x;                      /* (rows, channels) */
  const void* z;                      /* (rows, channels), with the two gate modes only */
  const float* weight;                /* (channels) or NULL = 1 */
  const float* bias;                  /* (channels) or NULL = 0 */
  void* y;                            /* (rows, channels) */
} ssm_group_norm_args_t;

typedef struct {
  int64_t rows, channels, groups;
  int64_t x_stride, z_stride, dy_stride;
  int32_t dtype;                      /* ssm_dtype_t of x, z, dy, dx, dz */
  int32_t mode;
  int32_t rms;
  float eps;
  const void* x;
  const void* z;
  const float* weight;
  const float* bias;
  const void* dy;                     /* (rows, channels) gradient of y */
  void* dx;                           /* (rows, channels) */
  void* dz;                           /* (rows, channels), with the two gate modes only */
  float* dweight;                     /* (channels) or NULL */
  float* dbias;                       /* (channels) or NULL */
  void* workspace;                    /* >= ssm_group_norm_bwd_workspace_size() bytes */
  size_t workspace_bytes;
} ssm_group_norm_bwd_args_t;

ssm_status_t ssm_group_norm_fwd(const ssm_group_norm_args_t* args, void* hip_stream);

/* Bytes of device workspace ssm_group_norm_bwd needs (0 without dweight and
 * dbias, or for invalid sizes).  Pure host function. */
size_t ssm_group_norm_bwd_workspace_size(const ssm_group_norm_bwd_args_t* args);

/* Gradients of sum(dy * y); the statistics are formed again from x (and z), and
 * dweight and dbias are summed over the rows in a fixed order. */
ssm_status_t ssm_group_norm_bwd(const ssm_group_norm_bwd_args_t* args, void* hip_stream);

/* ---------------------------------------------------------------------------
 * Around the scan in a layer, for sequences of unequal lengths laid one behind
 * the other: the packed scan, the short convolution by itself (its output is
 * what a layer projects to Delta, B and C, which the convolution fused into
 * ssm_scan_fwd comes too late for), and the residual's addition with the
 * root-mean-square norm.
 *
 * Conventions, where they differ from the scan's:
 *   Packed     rows are tokens; sequence s holds the tokens offsets[s] ..
 *              offsets[s + 1] - 1 (device, int32, seqs + 1 of them, not
 *              falling, within 0 .. tokens; values outside are taken as clamped,
 *              falling ones give unspecified outputs).  Sequences may be empty.
 *              Tokens before offsets[0] and from offsets[seqs] on belong to
 *              none: they are not read for any output (they may hold anything),
 *              and their rows of y are left as they were; gradients are 0 there.
 *   Slots      states and windows lie in a cache of `slots` entries; sequence s
 *              uses entry slot[s] (device, int32), or entry s where slot is
 *              NULL.  A sequence whose slot is not within 0 .. slots - 1 (a padding row's
 *              -1) starts from zero and keeps nothing.  Two sequences of a call
 *              with one slot: it ends up with parts of either's state.
 *   Resume     resume[s] (device, one byte; NULL = all 1) says whether sequence
 *              s takes up its slot's entry (nonzero) or starts from zero.
 *   Strides    inputs have contiguous channels and the row strides given (in
 *              elements, not negative), so slices of a projection need no copy;
 *              outputs, states and weights are dense.
 *   Dtypes     x and the other inputs of a row share dtype (fp32 or bf16), and so
 *              does y; A, weights, biases, states and windows are fp32, sums too.
 * ------------------------------------------------------------------------- */

/* The scan of ssm_scan_args_t over packed sequences:
 *   h_t = Abar_t h_{t-1} + Bbar_t x_t,  y_t = (sum_n C_t h_t + Dskip x_t) silu(z_t)
 * with h before a sequence's first token from h0 (zero when h0 is NULL or the
 * sequence is not resumed), and its last state to h_last.  An empty sequence's
 * last state is its first.  h_last may be h0 itself (a cache updated in place);
 * otherwise the two do not overlap. */
typedef struct {
  int64_t tokens, seqs, slots, dim, dstate;
  int64_t x_stride, delta_stride, z_stride, b_stride, c_stride;
  int32_t dtype;                      /* ssm_dtype_t of x, delta, z, Bm, Cm, y */
  int32_t disc;                       /* ssm_disc_t */
  int32_t delta_softplus;             /* 1: Delta = softplus(delta + delta_bias) */
  int32_t chunk_len;                  /* tokens per chunk, a multiple of 4; 0 = plan */
  const void* x;                      /* (tokens, dim) */
  const void* delta;                  /* (tokens, dim) */
  const float* A;                     /* (dim, dstate) */
  const void* Bm;                     /* (tokens, dstate) */
  const void* Cm;                     /* (tokens, dstate) */
  const float* Dskip;                 /* (dim) or NULL */
  const float* delta_bias;            /* (dim) or NULL, added to delta */
  const void* z;                      /* (tokens, dim) or NULL = no gate */
  const int32_t* offsets;             /* (seqs + 1) */
  const int32_t* slot;                /* (seqs) or NULL (slots = seqs) */
  const uint8_t* resume;              /* (seqs) or NULL */
  const float* h0;                    /* (slots, dim, dstate) or NULL */
  float* h_last;                      /* (slots, dim, dstate) or NULL */
  float* h_saved;                     /* (ceil(tokens / 16) - 1, dim, dstate) or NULL: receives the state
                                         before tokens 16, 32, ..., for ssm_packed_scan_bwd (left as
                                         it was at tokens of no sequence) */
  void* y;                            /* (tokens, dim) */
  void* workspace;                    /* >= ssm_packed_scan_workspace_size() bytes */
  size_t workspace_bytes;
} ssm_packed_scan_args_t;

/* One token for each row of a batch, row b's state in entry slot[b] of h (NULL:
 * entry b; slots = batch), updated in place; a row whose slot is out of range
 * reads a zero state and keeps nothing. */
typedef struct {
  int64_t batch, slots, dim, dstate;
  int64_t x_stride, delta_stride, z_stride, b_stride, c_stride;
  int32_t dtype;
  int32_t disc;
  int32_t delta_softplus;
  int32_t reserved;                   /* must be 0 */
  const void* x;                      /* (batch, dim) */
  const void* delta;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;
  const float* delta_bias;
  const void* z;
  const int32_t* slot;                /* (batch) or NULL */
  float* h;                           /* (slots, dim, dstate) */
  void* y;                            /* (batch, dim) */
} ssm_packed_step_args_t;

/* Gradients of  sum(dy * y) + sum(dh_last * h_last)  of the packed scan without
 * softplus, bias and gate, every sequence's state in entry s of h0 (NULL = all
 * from zero), dh_last (NULL = 0) and dh0 (seqs of them).  h_saved is what the
 * forward call of the same inputs kept.  Gradients are fp32 and overwritten. */
typedef struct {
  int64_t tokens, seqs, dim, dstate;
  int64_t x_stride, delta_stride, b_stride, c_stride, dy_stride;
  int32_t dtype;                      /* ssm_dtype_t of x, delta, Bm, Cm, dy */
  int32_t disc;
  int32_t super_chunk;                /* tokens per adjoint chunk, a multiple of 16; 0 = plan */
  int32_t reserved;                   /* must be 0 */
  const void* x;
  const void* delta;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* Dskip;
  const int32_t* offsets;             /* (seqs + 1) */
  const float* h0;                    /* (seqs, dim, dstate) or NULL */
  const float* h_saved;               /* (ceil(tokens / 16) - 1, dim, dstate) */
  const void* dy;                     /* (tokens, dim) gradient of y */
  const float* dh_last;               /* (seqs, dim, dstate) or NULL */
  float* dx;                          /* (tokens, dim) */
  float* ddelta;                      /* (tokens, dim) */
  float* dA;                          /* (dim, dstate) */
  float* dB;                          /* (tokens, dstate) */
  float* dC;                          /* (tokens, dstate) */
  float* dD;                          /* (dim) or NULL */
  float* dh0;                         /* (seqs, dim, dstate) or NULL */
  void* workspace;                    /* >= ssm_packed_scan_bwd_workspace_size() bytes */
  size_t workspace_bytes;
} ssm_packed_scan_bwd_args_t;

/* Workspace sizes: pure host functions of the sizes and row strides, chunk_len or
 * super_chunk and whether z, h0 and h_last are given, not of where anything lies; 0 for
 * invalid sizes. */
size_t ssm_packed_scan_workspace_size(const ssm_packed_scan_args_t* args);
size_t ssm_packed_scan_bwd_workspace_size(const ssm_packed_scan_bwd_args_t* args);
ssm_status_t ssm_packed_scan_fwd(const ssm_packed_scan_args_t* args, void* hip_stream);
ssm_status_t ssm_packed_step(const ssm_packed_step_args_t* args, void* hip_stream);
ssm_status_t ssm_packed_scan_bwd(const ssm_packed_scan_bwd_args_t* args, void* hip_stream);

/* Short causal convolution, depthwise, over packed sequences:
 *   y[t,c] = act(bias[c] + sum_{k<K} weight[c,k] x[t-K+1+k, c])
 * where inputs before a sequence's first token come from its window, the last
 * K - 1 inputs before it, oldest first (zero when state is NULL or it is not
 * resumed), and the window moves on in place.  Without offsets the sequences
 * have seqlen tokens each (tokens = seqs * seqlen). */
typedef enum { SSM_ACT_NONE = 0, SSM_ACT_SILU = 1 } ssm_act_t;

typedef struct {
  int64_t tokens, seqs, seqlen, slots, channels;
  int64_t x_stride;
  int32_t dtype;                      /* ssm_dtype_t of x, y */
  int32_t taps;                       /* K, 1..4 */
  int32_t act;                        /* ssm_act_t */
  int32_t reserved;                   /* must be 0 */
  const void* x;                      /* (tokens, channels) */
  const float* weight;                /* (channels, K), the newest input's tap last */
  const float* bias;                  /* (channels) or NULL */
  const int32_t* offsets;             /* (seqs + 1) or NULL */
  const int32_t* slot;                /* (seqs) or NULL (slots = seqs) */
  const uint8_t* resume;              /* (seqs) or NULL */
  float* state;                       /* (slots, channels, K - 1) or NULL */
  void* y;                            /* (tokens, channels) */
} ssm_short_conv_args_t;

typedef struct {
  int64_t batch, slots, channels;
  int64_t x_stride;
  int32_t dtype;
  int32_t taps;
  int32_t act;
  int32_t reserved;
  const void* x;                      /* (batch, channels) */
  const float* weight;
  const float* bias;
  const int32_t* slot;                /* (batch) or NULL (slots = batch) */
  float* state;                       /* (slots, channels, K - 1); may be NULL with K = 1 */
  void* y;                            /* (batch, channels) */
} ssm_short_conv_step_args_t;

/* Gradients of sum(dy * y) with every sequence from an empty window:
 *   da = dy act'(a);  dx[t] = sum_k weight[k] da[t+K-1-k] within t's sequence;
 *   dweight[k] = sum_t da[t] x[t-K+1+k];  dbias = sum_t da[t],
 * the sums in a fixed order.  dx has dtype; dweight and dbias are fp32. */
typedef struct {
  int64_t tokens, seqs, seqlen, channels;
  int64_t x_stride, dy_stride;
  int32_t dtype;                      /* ssm_dtype_t of x, dy, dx */
  int32_t taps;
  int32_t act;
  int32_t reserved;
  const void* x;
  const float* weight;
  const float* bias;
  const int32_t* offsets;
  const void* dy;                     /* (tokens, channels) */
  void* dx;                           /* (tokens, channels) */
  float* dweight;                     /* (channels, K) or NULL */
  float* dbias;                       /* (channels) or NULL */
  void* workspace;                    /* >= ssm_short_conv_bwd_workspace_size() bytes */
  size_t workspace_bytes;
} ssm_short_conv_bwd_args_t;

/* (0 without dweight and dbias, or for invalid sizes; a pure host function) */
size_t ssm_short_conv_bwd_workspace_size(const ssm_short_conv_bwd_args_t* args);
ssm_status_t ssm_short_conv_fwd(const ssm_short_conv_args_t* args, void* hip_stream);
ssm_status_t ssm_short_conv_step(const ssm_short_conv_step_args_t* args, void* hip_stream);
ssm_status_t ssm_short_conv_bwd(const ssm_short_conv_bwd_args_t* args, void* hip_stream);

/* The residual's addition and the root-mean-square norm of the sum, row by row:
 *   s = x + residual (x when residual is NULL)
 *   y = s / sqrt(mean(s^2) + eps) * weight
 * s is kept in the residual's type in `sum` (which may be the residual itself,
 * updated in place); y is formed from the unrounded s, in x's type, or in 8 bits:
 * values of e4m3 (the OCP format: largest 448, NaN, no infinities) and a scale
 * for each `block` neighbouring channels of a row (the last block may be short;
 * 0: one for the row), y ~ q scale, scale = max|y| / 448 of its block, NaN left out, at
 * least 2^-126, and 1 where that maximum is 0 or no y is a number.  q is rounded once, to
 * nearest even, and NaN where y is. */
#define SSM_E4M3 2                    /* a y_dtype of ssm_add_norm_args_t only */

typedef struct {
  int64_t rows, channels, block;
  int64_t x_stride, residual_stride;
  int32_t dtype;                      /* ssm_dtype_t of x */
  int32_t residual_dtype;             /* dtype or SSM_F32 */
  int32_t y_dtype;                    /* dtype or SSM_E4M3 */
  float eps;                          /* >= 0 */
  const void* x;                      /* (rows, channels) */
  const void* residual;               /* (rows, channels) or NULL */
  const float* weight;                /* (channels) or NULL = 1 */
  void* sum;                          /* (rows, channels) in residual_dtype; NULL: not kept */
  void* y;                            /* (rows, channels) */
  float* scale;                       /* (rows, ceil(channels / block)), with SSM_E4M3 only */
} ssm_add_norm_args_t;

/* Its gradients:  with n = s r, r = 1 / sqrt(mean(s^2) + eps),
 *   ds = dsum + r (dy weight - n mean(dy weight n)),  dweight = sum_rows dy n.
 * s is what `sum` holds: the kept sum, or x of a call without residual.  A sum kept in
 * fp32 is the forward call's s.  One kept in bf16 is s rounded: from it come the gradients
 * at the rounded sum, of which dweight is off by about 2e-3 of its norm; those of
 * the forward call are ssm_add_norm_bwd_residual's.
 * dx and dresidual are both ds: dx in dtype, dresidual in sum_dtype where that is
 * another type (NULL: not wanted). */
typedef struct {
  int64_t rows, channels;
  int64_t sum_stride, dy_stride, dsum_stride;
  int32_t dtype;                      /* ssm_dtype_t of dy, dx */
  int32_t sum_dtype;                  /* dtype or SSM_F32: of sum, dsum, dresidual */
  int32_t reserved;                   /* must be 0 */
  float eps;
  const void* sum;                    /* (rows, channels) */
  const void* dy;                     /* (rows, channels) gradient of y */
  const void* dsum;                   /* (rows, channels) gradient of the kept sum, or NULL = 0 */
  const float* weight;                /* (channels) or NULL = 1 */
  void* dx;                           /* (rows, channels) */
  void* dresidual;                    /* (rows, channels) or NULL */
  float* dweight;                     /* (channels) or NULL */
  void* workspace;                    /* >= ssm_add_norm_bwd_workspace_size() bytes */
  size_t workspace_bytes;
} ssm_add_norm_bwd_args_t;

/* (0 without dweight, or for invalid sizes; a pure host function) */
size_t ssm_add_norm_bwd_workspace_size(const ssm_add_norm_bwd_args_t* args);
ssm_status_t ssm_add_norm_fwd(const ssm_add_norm_args_t* args, void* hip_stream);
ssm_status_t ssm_add_norm_bwd(const ssm_add_norm_bwd_args_t* args, void* hip_stream);

/* The same from what the forward call was given: `sum` is x (in dtype) and s = x +
 * residual, (rows, channels) in sum_dtype with its row stride, formed again as the forward
 * call forms it.  The residual is required, and still what it was: a sum that took its
 * place has overwritten it. */
ssm_status_t ssm_add_norm_bwd_residual(const ssm_add_norm_bwd_args_t* args, const void* residual,
                                       int64_t residual_stride, void* hip_stream);

/* Static description of a status code. */
const char* ssm_status_string(ssm_status_t status);

/* Detail of the last failure on the calling thread ("" if none). */
const char* ssm_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* SSM_SCAN_H_ */
