/*
 * cba.h -- C ABI of libcba: the backward pass of a darknet/caffe-style
 * convolutional layer (convolution + optional batch norm + activation) on
 * one NVIDIA GB300 (sm_103a).
 *
 * What one call computes (source pages cited by title and section):
 *
 *   delta'   = delta * f'(output)                    gradient_array, leaky
 *              f'(y) = (y > 0) ? 1 : 0.1, linear f' = 1
 *              ("YOLOv3反向传播原理 之 全流程源码分析" §3.1, §7)
 *   db      += sum_{n,p,q} delta'                    backward_bias (§3.1, §4)
 *   with batch norm (training-mode statistics mean, var; §4):
 *   dgamma  += sum_{n,p,q} delta' * x_norm           backward_scale_cpu
 *   dz       = normalize_delta(scale_bias(delta'))   mean_delta_cpu,
 *              variance_delta_cpu, normalize_delta_cpu; x_norm = (z - mean)
 *              / sqrt(var + eps)
 *   without batch norm: dz = delta'
 *   dW      += dz . im2col(x)^T                      gemm(0,1,...,1,...) of §3.1
 *   prev_delta (= or +=) col2im(W^T . dz) + residual gemm(1,0,...) + col2im_cpu
 *              of §3.1 / §3.2; residual = the shortcut-layer delta (§5)
 *
 * The batch-norm steps are evaluated in the algebraically equal form
 *   dz = a_k * delta' + b_k + c_k * (z - mean_k),
 *   a_k = gamma_k / sigma_k, b_k = -a_k * S1_k / m, c_k = -a_k * S2_k / (m sigma_k),
 *   sigma_k = sqrt(var_k + eps), S1 = sum delta', S2 = sum delta' * x_norm,
 * m = N*P*Q, which is also caffe's BatchNormLayer::Backward_cpu times gamma
 * ("BatchNorm 理解", Backward_cpu).
 *
 * Layouts: every tensor is contiguous fp32.  Activations are NCHW
 * (batch-major): x, residual, prev_delta are [N][C][H][W]; output, z, delta,
 * dz_out are [N][K][P][Q] with P = (H + 2 pad - R)/stride + 1 and
 * Q = (W + 2 pad - S)/stride + 1 (floor division, im2col_cpu of §3.2).
 * W and dW are [K][C][R][S]; gamma, mean, var, db, dgamma are [K].
 *
 * Ownership: every pointer is DEVICE memory owned by the caller.  The
 * library allocates nothing and frees nothing; scratch comes from the
 * caller's workspace (size from cba_workspace_bytes).  Calls are
 * stream-ordered and asynchronous: they enqueue kernels on `stream` (a
 * cudaStream_t; NULL = the legacy default stream) and return without
 * synchronising.  Two calls that share a workspace must not overlap in time.
 * cba_conv_bn_act_backward and its traced variant can be captured into a
 * CUDA graph (stream capture) and replayed on the same buffers; make one call
 * on the device before capturing (it sets per-kernel attributes).
 *
 * Errors: a negative return code; on any error nothing has been launched and
 * no output touched, except CBA_ERR_CUDA (a launch failed; the CUDA error is
 * cleared and recorded, see cba_last_cuda_error).  Device-side failures
 * (a bounded wait that ran out) are reported through cba_get_status.
 */
#ifndef CBA_H_
#define CBA_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

#define CBA_OK 0
#define CBA_ERR_ARG (-1)         /* bad dimension, NULL required pointer, P or Q <= 0 */
#define CBA_ERR_UNSUPPORTED (-2) /* shape beyond the library's limits (e.g. > 2^31 elements) */
#define CBA_ERR_ALIGN (-3)       /* a pointer not 16-byte aligned */
#define CBA_ERR_WORKSPACE (-4)   /* workspace NULL or smaller than cba_workspace_bytes() */
#define CBA_ERR_CUDA (-5)        /* a CUDA launch or runtime call failed */
#define CBA_ERR_DEVICE_TIMEOUT (-6) /* reported by cba_get_status: a device wait ran out */
#define CBA_ERR_SCRATCH_LIMIT (-7)  /* cba_bn_act_backward_noalloc: K > CBA_NOALLOC_MAX_K */

/* Activation of the layer; its gradient is evaluated on the output y, as the
 * *_gradient functions of "YOLOv3反向传播原理" §7 are (gradient_array, §3.1):
 *   LINEAR 1              LEAKY   y>0 ? 1 : .1       LOGISTIC (1-y)y
 *   RELU   [y>0]          RELIE   y>0 ? 1 : .01      RAMP     [y>0] + .1
 *   TANH   1 - y^2        PLSE    y<0 or y>1 ? .01 : .125
 *   ELU    [y>=0] + [y<0](y+1)    SELU [y>=0] 1.0507 + [y<0](y + 1.0507*1.6732)
 *   LHTAN  0<y<1 ? 1 : .001       HARDTAN -1<y<1 ? 1 : 0
 *   LOGGY  2(1-t)t, t = (y+1)/2   STAIR floor(y) == y ? 0 : 1
 * LINEAR and LEAKY are applied inside the reduction and GEMM operand passes;
 * the others by one extra elementwise pass that writes delta * f'(y) into the
 * workspace (cba_workspace_bytes counts it). */
typedef enum {
    CBA_ACT_LINEAR = 0, CBA_ACT_LEAKY = 1, CBA_ACT_LOGISTIC = 2, CBA_ACT_RELU = 3,
    CBA_ACT_RELIE = 4, CBA_ACT_RAMP = 5, CBA_ACT_TANH = 6, CBA_ACT_PLSE = 7, CBA_ACT_ELU = 8,
    CBA_ACT_SELU = 9, CBA_ACT_LHTAN = 10, CBA_ACT_HARDTAN = 11, CBA_ACT_LOGGY = 12,
    CBA_ACT_STAIR = 13
} cba_act_t;

/* Arithmetic of the two convolution GEMMs.  TF32: tensor cores (tcgen05,
 * inputs read as TF32, fp32 accumulation).  FFMA: fp32 fused multiply-add on
 * the CUDA cores.  The reductions and the BN transform are fp32 (with fp64
 * cross-block sums) in both modes. */
typedef enum { CBA_MATH_TF32 = 0, CBA_MATH_FFMA = 1 } cba_math_t;

typedef struct {
    int N, C, H, W;     /* layer input x: batch, channels, height, width */
    int K, R, S;        /* filters, kernel height, kernel width */
    int stride, pad;    /* the same in both spatial dimensions */
    int act;            /* cba_act_t */
    int batch_normalize;/* 0: no BN.  1: BN in training mode; mean/var are the batch
                           statistics ("YOLOv3反向传播原理" §4).  2: BN with frozen
                           statistics; mean/var are constants of the forward, so
                           the BN-input gradient is gamma * delta' / sqrt(var + eps)
                           (caffe use_global_stats, "BatchNorm 理解" Backward_cpu);
                           db and dgamma accumulate as in mode 1.  With BN, z,
                           gamma, mean, var and dgamma are used. */
    int accumulate;     /* prev_delta: 0 writes, 1 adds onto its contents */
    float eps;          /* BN epsilon inside the square root (1e-5 in darknet) */
    int math;           /* cba_math_t */
} cba_desc_t;

/* Bytes of scratch one call with this descriptor needs (0 if the descriptor is
 * invalid).  The workspace must be 256-byte aligned device memory. */
size_t cba_workspace_bytes(const cba_desc_t *d);

/* With CBA_WS_RECOMPUTE_Z: the bytes of a z-free call (BN on, z = NULL), which
 * recomputes z = conv(x, W) -- the pre-BN convolution output, stride and pad
 * of the descriptor, no bias; forward_convolutional_layer's W . im2col(x) of
 * "YOLOv3反向传播原理" §3.2 -- into the workspace before the backward.  With
 * flags = 0 the same as cba_workspace_bytes.  0 on an invalid descriptor or an
 * unknown flag. */
#define CBA_WS_RECOMPUTE_Z 1u
size_t cba_workspace_bytes_ex(const cba_desc_t *d, unsigned flags);

/* The backward of one conv(+BN)+activation layer; see the header comment.
 *   x        [N,C,H,W] layer input (darknet net.input); required
 *   output   [N,K,P,Q] post-activation output; required unless act = LINEAR
 *   z        [N,K,P,Q] pre-BN convolution output (darknet l.x); with BN, NULL
 *            recomputes it from x and W (the workspace must then hold
 *            cba_workspace_bytes_ex(d, CBA_WS_RECOMPUTE_Z) bytes); unused
 *            without BN
 *   delta    [N,K,P,Q] gradient at the output; required; NOT modified
 *   W        [K,C,R,S] weights; required
 *   gamma, mean, var [K] BN scale and statistics (batch_normalize 1: the
 *            batch's, biased variance; 2: the frozen ones); required iff BN
 *   residual [N,C,H,W] shortcut delta added into prev_delta; may be NULL
 *   dW       [K,C,R,S] += ; required
 *   db       [K]       += ; required
 *   dgamma   [K]       += ; required iff BN
 *   prev_delta [N,C,H,W] (= or += per accumulate); NULL skips the input
 *            gradient (darknet's `if (net.delta)` at the first layer)
 *   dz_out   [N,K,P,Q] optional debug copy of dz; usually NULL
 *   workspace, workspace_bytes: scratch, see cba_workspace_bytes
 *   stream   cudaStream_t to enqueue on
 * Returns CBA_OK or a negative CBA_ERR_* code. */
int cba_conv_bn_act_backward(const cba_desc_t *d, const float *x, const float *output,
                             const float *z, const float *delta, const float *W,
                             const float *gamma, const float *mean, const float *var,
                             const float *residual, float *dW, float *db, float *dgamma,
                             float *prev_delta, float *dz_out, void *workspace,
                             size_t workspace_bytes, void *stream);

/* Grouped convolution (the l.groups loop of backward_convolutional_layer,
 * "YOLOv3反向传播原理" §3.1): output channels in groups of K/groups, input
 * channels in groups of C/groups, output channel k meeting only the input
 * channels of its group.  W and dW are [K][C/groups][R][S]; every other
 * argument as for cba_conv_bn_act_backward (descriptor C and K are the totals,
 * both multiples of groups).  The call launches the same kernels as an
 * ungrouped one, once for all groups: the per-channel reductions do not
 * depend on the grouping, and the two convolution gradients run as the dense
 * K x C product with zero weights between groups (so their cost is that of
 * the ungrouped layer), dW receiving only the pairs within a group.  It needs
 * cba_workspace_bytes_grouped(d, groups, flags) bytes (flags as for
 * cba_workspace_bytes_ex: CBA_WS_RECOMPUTE_Z for calls without z).
 * groups = 1 is cba_conv_bn_act_backward.  CBA_ERR_ARG also when groups < 1
 * or does not divide C and K. */
int cba_conv_bn_act_backward_grouped(const cba_desc_t *d, int groups, const float *x,
                                     const float *output, const float *z, const float *delta,
                                     const float *W, const float *gamma, const float *mean,
                                     const float *var, const float *residual, float *dW,
                                     float *db, float *dgamma, float *prev_delta, float *dz_out,
                                     void *workspace, size_t workspace_bytes, void *stream);
size_t cba_workspace_bytes_grouped(const cba_desc_t *d, int groups, unsigned flags);
/* The same, for profiling: phase_events and launches as for
 * cba_conv_bn_act_backward_traced (below). */
int cba_conv_bn_act_backward_grouped_traced(const cba_desc_t *d, int groups, const float *x,
                                            const float *output, const float *z,
                                            const float *delta, const float *W,
                                            const float *gamma, const float *mean,
                                            const float *var, const float *residual, float *dW,
                                            float *db, float *dgamma, float *prev_delta,
                                            float *dz_out, void *workspace,
                                            size_t workspace_bytes, void *stream,
                                            void *const *phase_events, int *launches);

/* Same computation as cba_conv_bn_act_backward, for profiling.
 * phase_events: NULL, or an array of CBA_PHASE_EVENTS (5) cudaEvent_t created
 *   by the caller; the call records, all on `stream`:
 *     [0] before the reduction pass (after the workspace's counters are
 *         cleared; a call without z recomputes z after [0]),
 *     [1] after it: the per-channel coefficients are ready,
 *     [2] after the GEMM operand layout pass (dz written in the layouts the
 *         tensor-core GEMMs read, and x re-laid out where the weight gradient
 *         needs it; see cba_plan_info) -- right after [1] on the FFMA path,
 *         whose GEMMs transform delta as they load it,
 *     [3] after the weight gradient,
 *     [4] after the input gradient (right after [3] when prev_delta is NULL).
 *   Recording events between the kernels stops a kernel from starting while
 *   its predecessor drains, so traced calls can take slightly longer.
 * launches: NULL, or receives the number of kernels this call enqueued.
 * Return codes as cba_conv_bn_act_backward. */
int cba_conv_bn_act_backward_traced(const cba_desc_t *d, const float *x, const float *output,
                                    const float *z, const float *delta, const float *W,
                                    const float *gamma, const float *mean, const float *var,
                                    const float *residual, float *dW, float *db, float *dgamma,
                                    float *prev_delta, float *dz_out, void *workspace,
                                    size_t workspace_bytes, void *stream,
                                    void *const *phase_events, int *launches);

#define CBA_PHASE_EVENTS 5

/* Which kernels a call with this descriptor runs, and what its operand layout
 * pass moves: a host-side query that launches nothing (groups as for
 * cba_conv_bn_act_backward_grouped, 1 for an ungrouped layer; with_prev:
 * whether the call will compute prev_delta).  Fills *info and returns CBA_OK,
 * or CBA_ERR_ARG / CBA_ERR_UNSUPPORTED for a descriptor the backward call
 * would refuse.  The path depends on the descriptor and on whether the CUDA
 * driver offers tensor-map encoding (without a driver every call plans the
 * FFMA kernels). */
typedef enum {
    CBA_PATH_FFMA = 0,        /* both GEMMs on the CUDA cores, BN transform on load */
    CBA_PATH_TC_ROWS = 1,     /* tcgen05 TF32; weight gradient reads x rows by TMA
                                 (stride-1 3x3 and 1x1 layers whose input rows are
                                 16-byte strided; a 1x1 layer's plane is one row) */
    CBA_PATH_TC_BATCH_INNER = 2, /* tcgen05 TF32; weight gradient on batch-innermost
                                    copies of x and dz */
    CBA_PATH_TC_GEMM_1X1 = 3     /* tcgen05 TF32; 1x1 stride-1 unpadded layers with
                                    16-byte rows (H*W and C multiples of 4, one
                                    group): both gradients as plain TMA-fed GEMMs */
} cba_path_t;
typedef struct {
    int path;                      /* cba_path_t */
    long long layout_bytes_read;   /* the operand layout pass (phase events [1]..[2]) */
    long long layout_bytes_written;
} cba_plan_info_t;
int cba_plan_info(const cba_desc_t *d, int groups, int with_prev, cba_plan_info_t *info);

/* Reads (and clears) the device status word of a workspace after the work on
 * `stream` has finished: synchronises `stream`, then returns CBA_OK or
 * CBA_ERR_DEVICE_TIMEOUT (a bounded device wait ran out; the kernel stopped
 * early and its outputs are not valid), or CBA_ERR_CUDA. */
int cba_get_status(void *workspace, size_t workspace_bytes, void *stream);

/* Self-test of the bounded device wait: launches one block whose thread waits
 * on a barrier phase that never completes, with a limit of `timeout_us`
 * microseconds (1 .. 2,000,000).  The wait gives up and records
 * CBA_ERR_DEVICE_TIMEOUT in the workspace status (read it back with
 * cba_get_status).  Needs cba_workspace_bytes of any valid descriptor. */
int cba_selftest_bounded_wait(void *workspace, size_t workspace_bytes, unsigned timeout_us,
                              void *stream);

/* Largest K that cba_bn_act_backward_noalloc accepts (its static scratch). */
#define CBA_NOALLOC_MAX_K 16384

/* The activation-gradient and BN-backward pass of cba_conv_bn_act_backward
 * (db, dgamma and, optionally, dz) WITHOUT a workspace and without allocating.
 * No counterpart in the source pages: it exists for callers that cannot call
 * cudaMalloc where they run the backward and have no buffer to lend, e.g. a
 * plugin called from another runtime's enqueue hook (that runtime owns all
 * device memory and forbids allocation after start-up) or a latency-bounded
 * loop (cudaMalloc may synchronise the device).
 *
 * Scratch: one static 1 MiB device array inside the library, placed on every
 * device that loads the library and held until the process exits.  The first
 * call on each device looks up the array's address (cudaGetSymbolAddress) with
 * that device current; make that first call before any stream capture.  The
 * address is kept for the life of the process, so resetting the device
 * (cudaDeviceReset) after the first call is not supported.  All
 * calls on a device share the array and it keeps the last call's contents;
 * each call first clears the reduction's per-channel counters (4 * K bytes,
 * a memset on the stream) and writes every other word before reading it.
 * Calls that overlap on one device (other streams or host threads with no
 * ordering between them) race on it: order them, e.g. on one stream.
 *
 * Arguments as cba_conv_bn_act_backward (only N, K and the output size P, Q of
 * the descriptor matter; math is ignored):
 *   output [N,K,P,Q] required unless act = LINEAR; z, gamma, mean, var and
 *   dgamma required iff BN; delta required; db [K] += and dgamma [K] += ;
 *   dz_out [N,K,P,Q] receives dz when not NULL.  Device pointers, 16-byte
 *   aligned; stream = cudaStream_t on the device that holds delta (the call
 *   runs on that device).
 * Returns CBA_OK, CBA_ERR_ARG / CBA_ERR_ALIGN / CBA_ERR_UNSUPPORTED,
 * CBA_ERR_SCRATCH_LIMIT when K > CBA_NOALLOC_MAX_K (nothing is enqueued), or
 * CBA_ERR_CUDA. */
int cba_bn_act_backward_noalloc(const cba_desc_t *d, const float *output, const float *z,
                                const float *delta, const float *gamma, const float *mean,
                                const float *var, float *db, float *dgamma, float *dz_out,
                                void *stream);

/* ---- Backward of the data-movement layers next to the convolution ----
 * Same conventions as above: device pointers owned by the caller, enqueued on
 * `stream` (cudaStream_t, NULL = legacy default) without synchronising, no
 * allocation; on an error nothing is launched.  Returns CBA_OK or a code. */

/* YOLO layer ("YOLOv3反向传播原理 之 全流程源码分析" §2, backward_yolo_layer):
 * net_delta[i] += l_delta[i] for i < n (the layer's delta passed back with one
 * axpy of factor 1; n = batch * inputs).  l_delta and net_delta: fp32, n
 * elements each, not overlapping.  CBA_ERR_ARG: n < 0, or a NULL pointer with
 * n > 0. */
int cba_yolo_backward(const float *l_delta, float *net_delta, long long n, void *stream);

/* Most inputs a route layer may have in one call. */
#define CBA_ROUTE_MAX_INPUTS 8

/* Route layer (same page, §6, backward_route_layer).  Its output lays its
 * n_inputs inputs side by side per image: outputs = sum of input_sizes, and
 * route_delta is [batch][outputs].  For input i (offset_i = the sum of the
 * earlier sizes) and image j:
 *   input_deltas[i][j * input_sizes[i] + t] += route_delta[j * outputs + offset_i + t]
 * for t < input_sizes[i].  input_sizes and input_deltas are HOST arrays of
 * n_inputs entries; input_deltas[i] are DEVICE pointers ([batch][size_i] fp32),
 * pairwise disjoint and disjoint from route_delta.  CBA_ERR_ARG: batch < 1,
 * n_inputs outside 1..CBA_ROUTE_MAX_INPUTS, a size < 1, or a NULL pointer. */
int cba_route_backward(const float *route_delta, int batch, int n_inputs,
                       const long long *input_sizes, float *const *input_deltas, void *stream);

/* Max pooling ("LeNet反向过程" 第五层 Pooling, caffe PoolingLayer MAX): bottom
 * [N,C,H,W], top [N,C,PH,PW] with caffe's sizes PH = cba_pooled_size(H,
 * kernel_h, stride_h, pad_h) and PW likewise. */
typedef struct {
    int N, C, H, W;
    int kernel_h, kernel_w, stride_h, stride_w, pad_h, pad_w; /* 0 <= pad < kernel */
} cba_pool_desc_t;

/* caffe's pooled size: ceil((in + 2 pad - kernel) / stride) + 1, one less when
 * the last window would start in the bottom padding; -1 on bad arguments. */
int cba_pooled_size(int in, int kernel, int stride, int pad);

/* bottom_diff = 0, then bottom_diff[n][c][mask / W][mask % W] += top_diff for
 * every top element (mask[n][c][ph][pw] = h * W + w of the element the forward
 * took as the window's maximum).  Each bottom element is written once: it sums
 * the top gradients that point at it in ascending (ph, pw), the page's order.
 * A mask value outside its own window is ignored (never dereferenced).
 * top_diff fp32 and mask int32 [N,C,PH,PW], bottom_diff fp32 [N,C,H,W].
 * CBA_ERR_ARG: a non-positive size, kernel or stride, pad outside 0..kernel-1,
 * PH or PW < 1, a NULL pointer; CBA_ERR_UNSUPPORTED: N*C*H*W or N*C*PH*PW past
 * 2^62, H*W past 2^31. */
int cba_maxpool_backward(const cba_pool_desc_t *d, const float *top_diff, const int *mask,
                         float *bottom_diff, void *stream);

/* ---- Operators of transformer layers: layer norm, attention, query and key norms
 * with rotation, dropout, orthogonalised updates ----
 * Conventions as above: device pointers owned by the caller, stream-ordered,
 * asynchronous, no allocation, capturable; scratch from the caller's 256-byte
 * aligned workspace (two calls that share one must not overlap in time); on an
 * error nothing is launched.  Sums, statistics and products accumulate in
 * fp32 whatever the element type, in a fixed order: the same inputs give the
 * same bits. */

/* Element type of a tensor. */
typedef enum { CBA_F32 = 0, CBA_F16 = 1, CBA_BF16 = 2 } cba_dtype_t;

/* Layer norm over the last axis of [rows][cols].  With mu = mean_c x and
 * r = 1 / sqrt(mean_c (x - mu)^2 + eps):
 *   forward   y = (x - mu) r gamma + beta; mean = mu, rstd = r
 *   backward  g = dy gamma, h = (x - mu) r,
 *             dx = r (g - mean_c g - h mean_c(g h)) + residual
 *             dgamma (= or +=) sum_rows dy h,  dbeta (= or +=) sum_rows dy
 * x, y, dy, residual and dx have elements of `type`; gamma and beta [cols] of
 * `param_type` (fp32, or the same as type: CBA_ERR_UNSUPPORTED otherwise);
 * mean, rstd [rows], dgamma and dbeta [cols] are fp32.  ld_*: elements from one
 * row of a tensor to the next (0: cols).  Rows of 16-byte multiples on 16-byte
 * aligned bases and strides move as vectors; any other element-aligned layout
 * is correct and slower. */
typedef struct {
    long long rows;   /* may be 0 */
    int cols;
    int type, param_type; /* cba_dtype_t */
    int accumulate;   /* dgamma, dbeta: 0 writes, 1 adds onto their contents */
    float eps;
    long long ld_x, ld_y, ld_dy, ld_dx, ld_residual;
} cba_layernorm_desc_t;

/* gamma, beta: NULL for 1 and 0.  mean, rstd: NULL when not wanted.  y may be x
 * (of the same ld). */
int cba_layernorm_forward(const cba_layernorm_desc_t *d, const void *x, const void *gamma,
                          const void *beta, void *y, float *mean, float *rstd, void *stream);

/* Bytes of scratch of one backward call (0 on an invalid descriptor). */
size_t cba_layernorm_workspace_bytes(const cba_layernorm_desc_t *d);

/* residual (nullable): the shortcut's delta, added to dx.  gamma NULL: 1.
 * dgamma, dbeta: NULL when not wanted.  dx may be x, dy or residual (of the same
 * ld).  With rows = 0, dgamma and dbeta become 0 (accumulate = 0) or stay. */
int cba_layernorm_backward(const cba_layernorm_desc_t *d, const void *x, const void *dy,
                           const void *gamma, const float *mean, const float *rstd,
                           const void *residual, void *dx, float *dgamma, float *dbeta,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Attention's backward pass.  For each query head h, with the key/value head
 * h / (heads_q / heads_kv):
 *   S = scale q k^T,  P = exp(S - lse) on the allowed pairs (0 elsewhere),
 *   D = rowsum(dout o),  dS = P (dout v^T - D),
 *   dq = scale dS k,  dk = scale sum_h dS^T q,  dv = sum_h P^T dout
 * q, o, dout, dq: heads_q heads; k, v, dk, dv: heads_kv heads; elements f16 or
 * bf16 (CBA_F32: CBA_ERR_UNSUPPORTED); dim a multiple of 8 up to 128.  o and lse
 * are the forward's: lse fp32 = log sum_j exp S_ij, contiguous [batch][heads_q]
 * [len_q] (packed: [heads_q][total_q]).  Row i of a sequence sees the keys
 * j <= i + len_k - len_q when causal, all of them otherwise.  A row that sees
 * none (or whose lse is -infinity) has P = 0 and D = 0, whatever its o holds (a
 * softmax over nothing is NaN): it gets dq = 0 and adds nothing.
 *
 * Dense: `batch` sequences of len_q queries and len_k keys, element (b, t, h, c)
 * of a tensor at b * batch + t * token + h * head + c.  Packed: `batch`
 * sequences one after another, cu_q and cu_k DEVICE int32 [batch + 1] with their
 * first tokens (non-decreasing, within 0 and total_q / total_k; tokens outside
 * all sequences are neither used nor written); len_q and len_k are upper bounds
 * of the sequences' lengths (tokens past them are not computed; total_q and
 * total_k will do) and the batch strides are not used.  A sequence may be
 * empty.  Strides all 0 mean contiguous [batch][token][head][dim].  Strides must
 * be multiples of 8 elements and bases 16-byte aligned (CBA_ERR_ALIGN).  Outputs
 * must not overlap inputs.
 *
 * P and dS are rounded to the elements' type for their products (f16: times
 * powers of two, dS's from the largest finite rows of dout and v of its own
 * sequence and key/value head), the sums are fp32.  In a sequence's own rows,
 * infinities and NaN spread as in the formulas (a masked pair still multiplies
 * its row by 0); another sequence's never do. */
typedef struct { long long batch, token, head; } cba_attn_strides_t;
typedef struct {
    int batch, heads_q, heads_kv, dim;
    int len_q, len_k;
    int packed;                 /* 0 dense, 1 packed (cu_q, cu_k) */
    int type;                   /* cba_dtype_t */
    long long total_q, total_k; /* packed: tokens */
    int causal;
    float scale;
    cba_attn_strides_t q, k, v, o, dout, dq, dk, dv;
} cba_attention_desc_t;

/* Bytes of scratch of one call (0 on an invalid descriptor).  cba_get_status
 * reads the same workspace after the call. */
size_t cba_attention_workspace_bytes(const cba_attention_desc_t *d);
int cba_attention_backward(const cba_attention_desc_t *d, const void *q, const void *k,
                           const void *v, const void *o, const float *lse, const void *dout,
                           const int *cu_q, const int *cu_k, void *dq, void *dk, void *dv,
                           void *workspace, size_t workspace_bytes, void *stream);

/* Attention's forward pass, whose o and lse the backward pass above takes: with S as
 * there, over the allowed pairs,
 *   lse = log sum_j exp S_ij,  o = sum_j exp(S_ij - lse) v_j
 * The descriptor is the backward's (dout, dq, dk and dv and their strides do not count):
 * the same types, layouts, head sharing, masks, packing and limits.  lse: NULL when not
 * wanted.  A row that sees no key gets o = 0 and lse = -infinity.  o must not overlap
 * the inputs; tokens outside all packed sequences, or past the bounds of the lengths,
 * are not written.
 *
 * P is rounded to the elements' type for its product with v, as a share of the row's
 * largest (f16: times a power of two); its sums, the maxima and o's are fp32.  Shares are of
 * a running largest, so up to 2^8 before the division: in bf16, o is finite as long as
 * 2^8 sum |v| over a row's keys is within fp32's range.  Few rows
 * with many keys are cut along the keys and joined in a fixed order.  In a sequence's
 * own rows, infinities and NaN spread as in the formulas (a masked pair may still
 * multiply its row of v by 0); another sequence's never do. */
size_t cba_attention_forward_workspace_bytes(const cba_attention_desc_t *d);
int cba_attention_forward(const cba_attention_desc_t *d, const void *q, const void *k,
                          const void *v, const int *cu_q, const int *cu_k, void *o, float *lse,
                          void *workspace, size_t workspace_bytes, void *stream);

/* Norms of queries and keys for each head, with the rotation by position in the same
 * pass.  For every head's elements x of q [batch][len][heads_q][dim] and of k
 * [batch][len][heads_k][dim]:
 *   forward   r = 1 / sqrt(mean_c x^2 + eps), n = x r, h = n gamma (norm = 0: h = x),
 *             y = h with the pairs j < rot_dim / 2 turned: (a, b) becomes
 *             (a cos - b sin, a sin + b cos), cos and sin = table[position][j];
 *             a and b are the elements j and j + rot_dim / 2 (interleaved = 1: 2j and
 *             2j + 1), those from rot_dim on stay
 *   backward  g = dy turned back, w = g gamma, dx = r (w - n mean_c(w n)) (norm = 0:
 *             dx = g), dgamma (= or +=) sum g n over the tokens and heads
 * q, k and the outputs have elements of `type`; gamma_q and gamma_k [dim] of `param_type`
 * (fp32, or the same as type: CBA_ERR_UNSUPPORTED otherwise); dgamma_q and dgamma_k [dim]
 * are fp32.  table: fp32 [positions][rot_dim / 2][2], cos and sin.  pos: int32
 * [batch][len], contiguous, the tokens' rows of the table; NULL: a token's index in its
 * sequence (len <= positions, or CBA_ERR_ARG).  Values outside 0 .. positions - 1 are
 * taken as the nearest of these.  dim: a multiple of 8 up to 256, rot_dim even, heads up
 * to 2^30.  heads_k may be 0 (then k and what belongs to it are not used).
 *
 * Heads of any finite elements give the formula's values, with eps = 0 too; but dx of a head
 * with r past the largest fp32 number (a root mean square below 2^-128) is infinite or NaN.
 *
 * Strides as of attention, in multiples of 16 bytes, bases (gamma and table too) 16-byte
 * aligned (CBA_ERR_ALIGN); all 0: contiguous.  An output may be the input of the same
 * strides (yq q; dq dyq or q), and must not overlap inputs otherwise. */
typedef struct {
    int batch, len, heads_q, heads_k, dim;
    int type, param_type; /* cba_dtype_t */
    int norm;             /* 1: norm and rotation, 0: rotation alone (gamma, dgamma NULL) */
    int rot_dim, interleaved;
    int positions;        /* rows of the table */
    int accumulate;       /* dgamma: 0 writes, 1 adds onto its contents */
    float eps;
    cba_attn_strides_t q, k, yq, yk, dyq, dyk, dq, dk;
} cba_qk_norm_rope_desc_t;

/* gamma_q, gamma_k: NULL for 1.  table: may be NULL with rot_dim = 0. */
int cba_qk_norm_rope_forward(const cba_qk_norm_rope_desc_t *d, const void *q, const void *k,
                             const void *gamma_q, const void *gamma_k, const float *table,
                             const int *pos, void *yq, void *yk, void *stream);

/* Bytes of scratch of one backward call (0 on an invalid descriptor). */
size_t cba_qk_norm_rope_workspace_bytes(const cba_qk_norm_rope_desc_t *d);

/* q, k: the forward's inputs (norm = 0: not used).  dgamma_q, dgamma_k: NULL when not
 * wanted.  With len = 0, dgamma becomes 0 (accumulate = 0) or stays. */
int cba_qk_norm_rope_backward(const cba_qk_norm_rope_desc_t *d, const void *q, const void *k,
                              const void *gamma_q, const void *gamma_k, const float *table,
                              const int *pos, const void *dyq, const void *dyk, void *dq, void *dk,
                              float *dgamma_q, float *dgamma_k, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Dropout whose mask is never stored, with the shortcut added.  With i = row * cols + col:
 *   y = (word_i >= p 2^32 ? x / (1 - p) : 0) + residual
 * word_i: word i mod 4 of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, 2011) with the
 * key `seed` (low word first) and the counter offset + *step + i / 4 in its low 64 bits,
 * modulo 2^64; p 2^32 is rounded to a whole number, and p = 1 drops all.  Dropped elements count as 0
 * whatever they hold.  The gradient is the same call on dy without the residual.
 * A call uses the counters from offset + *step on, (rows * cols + 3) / 4 of them: the
 * next one starts behind them.
 *
 * step: NULL for 0, or DEVICE memory (8-byte aligned) read when the call runs, so that
 * a captured call that is replayed draws anew once the program has moved it on.
 * residual: NULL for none.  ld_*: elements from one row to the next (0: cols).  y may be x or
 * residual (of the same ld).  Tensors without gaps between rows, or with rows and
 * strides of 16-byte multiples, on 16-byte aligned bases move as vectors; any other
 * element-aligned layout is correct and slower. */
typedef struct {
    long long rows, cols; /* rows may be 0; rows * cols up to 2^40 */
    int type;             /* cba_dtype_t */
    float p;              /* 0 to 1 */
    unsigned long long seed, offset;
    long long ld_x, ld_residual, ld_y;
} cba_dropout_desc_t;

int cba_dropout(const cba_dropout_desc_t *d, const void *x, const void *residual,
                const unsigned long long *step, void *y, void *stream);

/* Orthogonalising a matrix by Newton-Schulz products (the update of a Muon
 * optimiser, e.g. of a momentum of dW [K][C*R*S]).  For each of `batch` matrices
 * G [rows][cols]:
 *   X = G / (|G|_F + eps); `steps` times: X <- a X + (b S + c S^2) X, S = X X^T
 *   O = scale X
 * (with rows > cols the same from the right, S = X^T X).  Every singular value s
 * of G / (|G|_F + eps) becomes p(p(...p(s))), p(s) = a s + b s^3 + c s^5; with
 * (3.4445, -4.7750, 2.0315) and 5 steps they end near 1.
 *
 * The products' operands are f16 scaled by powers of two, their sums fp32,
 * whatever the element types are: with the coefficients above O's error is 1e-3
 * to 4e-3 of its norm (so its type is usually bf16), and to 1e-2 in matrices of
 * a few rows, whose singular values may all meet the polynomial where it is
 * steep.  Singular values far below the leading ones grow by a factor of `a` a
 * step, and with them the rounding errors in their directions: where they span
 * four decades, 5e-2 of the norm of a matrix of 2 rows, 2e-2 of one of 24 rows,
 * 5e-3 of one of 1000.  The scaling has room for singular values up to 2 before
 * every step, whatever the coefficients (those that converge keep them below
 * 1.3).  Elements of G below 1e-19 count as 0 in its norm.
 *
 * Element types f32, f16 or bf16.  ld_*: elements from one row to the next (0:
 * cols); batch_*: from one matrix to the next (0: rows * ld).  O may be G when
 * type and strides agree. */
typedef struct {
    int batch, rows, cols;
    int in_type, out_type;  /* cba_dtype_t */
    int steps;              /* 1 to 100 */
    float a, b, c;
    float eps, scale;
    long long ld_in, ld_out, batch_in, batch_out;
} cba_orthogonalize_desc_t;

/* Bytes of scratch of one call (0 on an invalid descriptor).  cba_get_status
 * reads the same workspace after the call. */
size_t cba_orthogonalize_workspace_bytes(const cba_orthogonalize_desc_t *d);
int cba_orthogonalize(const cba_orthogonalize_desc_t *d, const void *G, void *O, void *workspace,
                      size_t workspace_bytes, void *stream);

/* Human-readable text of a CBA_* code (static storage). */
const char *cba_error_string(int code);

/* The cudaError_t of the last CBA_ERR_CUDA in this process (0 if none). */
int cba_last_cuda_error(void);

/* Library version, major*10000 + minor*100 + patch. */
int cba_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CBA_H_ */
