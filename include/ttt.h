/*
 * ttt.h -- C ABI of libttt: forward pass (prefill / inference) of a
 * Test-Time-Training (TTT) layer on one NVIDIA GB300 (sm_103a).
 *
 * The layer.  For every (batch, head) sequence the hidden state is the weight set W
 * of a small inner model f(x; W).  W starts at W0 and is trained on the sequence
 * itself by gradient descent on the reconstruction loss
 *     l_t(W) = 1/2 || f(k_t; W) - v_t ||^2
 * ("Fast weights 与 TTT layers", opening formula; "TTT：Test-Time Training",
 * section TTT, MSE loss).  Tokens are taken in consecutive mini-batches of b
 * tokens; every token of a mini-batch takes its gradient at the W that the previous
 * mini-batch left ("Learning to (Learn at Test Time)" walkthrough, section 1.2.2,
 * mini-batch gradient descent, formula 6).  The output is z_t = f(q_t; W_t)
 * (same walkthrough, section 1.2, output rule), where
 *   causal = 1:  W_t = W_start - sum_{s in t's mini-batch, s <= t} eta_s grad l_s(W_start)
 *                (the cumulative-sum channel of section 1.2.2: W_t includes token
 *                t's own write);
 *   causal = 0:  every query of a mini-batch reads the W at the end of that
 *                mini-batch (b = T gives one full-batch step, the vision variant of
 *                the ViT3 article, observation 2).
 * b = 1 is the delta rule ("Fast weights 与 TTT layers", section 1).
 *
 * Inner models (walkthrough section 2.2.1; ViT3 article, observations 4 and 6):
 *   ttt_linear_fwd:  f(x; W) = x W,                      W in R^{d x d}
 *   ttt_mlp_fwd:     f(x) = act(x W1 + c1) W2 + c2,       W1 d x m, W2 m x d
 *   ttt_dwconv_fwd:  a depthwise 3 x 3 convolution over a token grid
 *   (optionally x + LN(f(x)) for the first two: the inner norm and residual).
 * ttt_eta_gate computes the per-token rates eta = eta_base * sigma(theta_lr . x)
 * from the layer input (walkthrough section 2.2.3) in the layout the others read.
 * Row convention throughout: a token x is a 1 x d row vector.
 *
 * Conventions shared by every entry point
 *   - All data pointers are DEVICE pointers owned by the caller.  The library
 *     allocates no device memory.  Its device state is one small status word per
 *     device and the fixed 4 MiB scratch array of ttt_linear_fwd_seqpar_noalloc
 *     (a static device array, held on every device that loads the library until
 *     the process exits).
 *   - Work is enqueued on `stream` (a cudaStream_t passed as void*; NULL = the
 *     legacy default stream) and runs asynchronously.  The return value reports
 *     argument validation and launch errors synchronously.  A kernel-side wait that
 *     timed out (never expected; every on-chip wait is bounded to about 2 s) is
 *     reported by ttt_sync_status().
 *   - Layouts are C-contiguous: q, k, v, z are [B, H, T, d] in io_dtype; eta is
 *     [B, H, T] fp32; weights are fp32.
 *   - Alignment: q, k, v, z must be 16-byte aligned (TTT_ERR_ALIGN otherwise);
 *     eta and the fp32 weight arrays 4-byte aligned.
 *   - T may be 0 (then only the final weights are written, equal to the initial
 *     ones) and need not be a multiple of b: the last mini-batch is shorter.
 *   - Final-weight outputs may be NULL (not written).  They may alias the
 *     corresponding initial-weight inputs when those are given per (batch, head)
 *     (in-place continuation of a sequence); they may not overlap shared
 *     ([H, ...]) initial weights (TTT_ERR_ARG).
 */
#ifndef TTT_H_
#define TTT_H_

#include <stddef.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TTT_OK = 0,
    TTT_ERR_ARG = -1,          /* null / negative / inconsistent argument            */
    TTT_ERR_UNSUPPORTED = -2,  /* valid but not implemented (e.g. d not in the set)   */
    TTT_ERR_ALIGN = -3,        /* pointer misaligned for the bulk-copy engine         */
    TTT_ERR_LAUNCH = -4,       /* CUDA reported an error at or before launch          */
    TTT_ERR_TIMEOUT = -5,      /* a kernel wait ran out (reported by ttt_sync_status) */
    TTT_ERR_SCRATCH = -6,      /* ttt_linear_fwd_seqpar_noalloc: more than its fixed scratch */
    TTT_ERR_RANGE = -7         /* ttt_rope: a position outside its table (reported by
                                  ttt_sync_status; the launch itself stays in bounds)  */
} ttt_status;

typedef enum { TTT_F32 = 0, TTT_BF16 = 1 } ttt_dtype;

/* Inner loss of TTT-Linear.
 *   TTT_LOSS_MSE: l_t(W) = 1/2 || k_t W - v_t ||^2 (the reconstruction loss above).
 *   TTT_LOSS_DOT: l_t(W) = -(k_t W) . v_t, the negative dot product ("TTT：Test-Time
 *                 Training", section 如何理解; the inner loss of the ViT3 block).  Its
 *                 gradient -k_t^T v_t does not depend on W, so the layer becomes
 *                 linear attention with state W0 + sum eta_s k_s^T v_s. */
typedef enum { TTT_LOSS_MSE = 0, TTT_LOSS_DOT = 1 } ttt_loss;

/* TTT-Linear problem description. */
typedef struct {
    int B, H, T, d;            /* batch, heads, tokens, head dim (d in {16,32,64,128}) */
    int mini_batch;            /* b >= 1                                               */
    int causal;                /* 1 causal, 0 non-causal (queries read block-end W)    */
    ttt_dtype io_dtype;        /* dtype of q, k, v and z                               */
    long long w0_batch_stride; /* elements between batches of W0; 0 = W0 is [H,d,d]
                                  shared by every batch entry, H*d*d = [B,H,d,d]       */
    int loss;                  /* ttt_loss (0 = TTT_LOSS_MSE)                          */
    int epochs;                /* inner gradient steps on the mini-batch: 0 or 1 = one;
                                  > 1 (the ViT3 article's inner epochs) needs causal = 0
                                  and mini_batch >= T, every query reading the last W;
                                  bf16 supports it for d = 64, T <= 256
                                  (TTT_ERR_UNSUPPORTED otherwise)                       */
    const float *ln_gamma;     /* inner layer norm + residual: f(x) = x + LN(x W) with
                                  LN(y) = ln_gamma * (y - mean) / sqrt(var + ln_eps)
                                  + ln_beta over the d outputs ("Learning to (Learn at
                                  Test Time)" walkthrough, section 2.2.1); [H,d] fp32
                                  device arrays, fixed (not trained by the inner step),
                                  or both NULL for f(x) = x W.  MSE loss and one epoch
                                  only; bf16 needs mini_batch 16 and d <= 64
                                  (TTT_ERR_UNSUPPORTED otherwise)                       */
    const float *ln_beta;
    float ln_eps;              /* > 0 when the norm is used (1e-6 in the paper's code)  */
} ttt_linear_desc;

/*
 * TTT-Linear forward.
 *   q, k, v : [B,H,T,d] io_dtype (queries, keys = training view, values = labels)
 *   eta     : [B,H,T] fp32 per-token learning rate of the writing token, or NULL to
 *             use eta_scalar for every token (walkthrough section 2.2.3)
 *   W0      : fp32 initial weights, W0[i][j] multiplies input i into output j
 *   z       : [B,H,T,d] io_dtype output
 *   W_out   : [B,H,d,d] fp32 final weights, or NULL
 * io_dtype TTT_BF16 runs the tensor-core path: bf16 operands, fp32 accumulation and
 * fp32 weight state.  TTT_F32 runs an fp32 CUDA-core path (no reduced precision).
 */
ttt_status ttt_linear_fwd(const ttt_linear_desc *desc,
                          const void *q, const void *k, const void *v,
                          const float *eta, float eta_scalar,
                          const float *W0, void *z, float *W_out, void *stream);

/*
 * Sequence-parallel TTT-Linear forward: the same results as ttt_linear_fwd (up to the
 * order of floating-point rounding), for problems with fewer (batch, head) chains
 * than the GPU has SMs and long sequences.
 *
 * One mini-batch step is affine in the weights, W' = (I - K^T diag(eta) K) W +
 * K^T diag(eta) V ("Learning to (Learn at Test Time)" walkthrough, section 1.2.2,
 * formula 6, for the linear inner model of section 2.2.1), so each chain is cut
 * into segments of whole 64-token blocks: the affine maps W -> A W + B of the
 * segments are computed in parallel, a scan turns them into every segment's start
 * weights, and the segments' outputs are computed in parallel from those.  The
 * first segment runs from W0 while the maps are formed.
 *
 * Applies to io_dtype TTT_BF16 with mini_batch 16, or 1 (the delta rule, whose
 * 16-token chunks are affine in the weights as well), d in {16, 32, 64} and the MSE
 * loss, when the GPU has at least two SMs per chain; otherwise the call runs
 * ttt_linear_fwd (workspace unused, may be NULL).
 *   workspace       : device scratch owned by the caller, 256-byte aligned, at least
 *                     ttt_linear_seqpar_workspace(desc) bytes; it holds the maps and
 *                     start weights and must not be touched until the work queued
 *                     on `stream` has finished.
 * The work is queued on `stream`; internally it forks to a second stream of the
 * library's own (one per device, created on the first split call) and joins back
 * with events, so later work on `stream` sees the outputs.  W_out must not overlap
 * W0 here (TTT_ERR_ARG): the first segment may still read W0 while the last one
 * writes W_out.  TTT_ERR_ARG also for a missing, misaligned or too small workspace.
 */
size_t ttt_linear_seqpar_workspace(const ttt_linear_desc *desc);

ttt_status ttt_linear_fwd_seqpar(const ttt_linear_desc *desc,
                                 const void *q, const void *k, const void *v,
                                 const float *eta, float eta_scalar,
                                 const float *W0, void *z, float *W_out,
                                 void *workspace, size_t workspace_bytes, void *stream);

/*
 * ttt_linear_fwd_seqpar_noalloc: the sequence-parallel forward without a caller
 * workspace and without any device allocation.  (The pages have no counterpart:
 * this is a deployment variant of ttt_linear_fwd_seqpar.)
 *
 * For callers that cannot allocate device memory while they run: a serving
 * process that has handed the free device memory to its own pool or cache has none
 * left for cudaMalloc, cudaFree may synchronise the device in the middle of its
 * pipeline, and a plugin inside another framework may have no access to that
 * framework's allocator.  The scratch is instead a fixed array of 4 MiB inside the
 * library, held on every device that loads it until the process exits.
 *
 * Same arguments and results as ttt_linear_fwd_seqpar (up to floating-point
 * rounding), all work on `stream` alone: one launch for the first segment's state
 * chain and the later segments' affine maps, the scan, then every segment's
 * outputs in one launch (segments of equal length).  Problems that do not split
 * run ttt_linear_fwd.  A split needs 4 (BH (P-1) + 2 BH (P-2)) d^2 bytes for P
 * segments of BH = B*H chains (e.g. d = 64, two segments: up to 256 chains);
 * larger problems return TTT_ERR_SCRATCH before any work is queued.  W_out must
 * not overlap W0 (TTT_ERR_ARG).
 *
 * The first call on a device looks up the array's device address (once per
 * device, with that device current); make that first call before any stream
 * capture.  Every call uses the same array: calls whose work overlaps on the GPU
 * (other streams, other host threads) race on it and must be ordered by the
 * caller.  Nothing in the array needs clearing between calls.
 */
ttt_status ttt_linear_fwd_seqpar_noalloc(const ttt_linear_desc *desc,
                                         const void *q, const void *k, const void *v,
                                         const float *eta, float eta_scalar,
                                         const float *W0, void *z, float *W_out, void *stream);

/* Inner activation of TTT-MLP.
 *   TTT_ACT_SILU: SiLU(h) = h sigma(h) (the ViT3 article, observation 4).
 *   TTT_ACT_GELU: GELU(h) = h Phi(h), Phi the standard normal CDF, in its exact
 *                 (erf) form (the walkthrough's TTT-MLP, section 2.2.1). */
typedef enum { TTT_ACT_SILU = 0, TTT_ACT_GELU = 1 } ttt_activation;

/* TTT-MLP problem description. */
typedef struct {
    int B, H, T, d, m;         /* d in {16,32,64}; m = hidden width, multiple of 16    */
    int mini_batch;            /* b >= 1                                               */
    int causal;
    ttt_dtype io_dtype;
    int params_per_batch;      /* 0: W1,c1,W2,c2 are [H,...] shared over the batch;
                                  1: they are [B,H,...]                                */
    int activation;            /* ttt_activation (0 = TTT_ACT_SILU)                    */
    const float *ln_gamma;     /* inner layer norm + residual: f(x) = x + LN(act(x W1 +
                                  c1) W2 + c2), LN over the d outputs as in
                                  ttt_linear_desc ("Learning to (Learn at Test Time)"
                                  walkthrough, section 2.2.1); [H,d] fp32 device arrays,
                                  fixed, or both NULL for the plain MLP.  bf16 I/O needs
                                  d = 64, m = 256 and mini_batch <= 16 or one
                                  non-causal full batch (mini_batch >= T); otherwise
                                  TTT_ERR_UNSUPPORTED                                   */
    const float *ln_beta;
    float ln_eps;              /* > 0 when the norm is used                             */
} ttt_mlp_desc;

/*
 * TTT-MLP forward, f(x) = act(x W1 + c1) W2 + c2, act = SiLU or GELU (desc->activation),
 * or x + LN(f(x)) with the inner norm (desc->ln_gamma, ln_beta, ln_eps).
 *   W1 [..,d,m], c1 [..,m], W2 [..,m,d], c2 [..,d] fp32 initial inner weights;
 *   the *_out arrays are [B,H,...] fp32 final weights (each may be NULL).
 * Other arguments as for ttt_linear_fwd.
 */
ttt_status ttt_mlp_fwd(const ttt_mlp_desc *desc,
                       const void *q, const void *k, const void *v,
                       const float *eta, float eta_scalar,
                       const float *W1, const float *c1, const float *W2, const float *c2,
                       void *z, float *W1_out, float *c1_out, float *W2_out, float *c2_out,
                       void *stream);

/* Depthwise-convolution TTT problem description. */
typedef struct {
    int B, H;                  /* batch, heads                                          */
    int height, width;         /* token grid: N = height * width tokens per sequence,
                                  row-major (token y * width + x)                       */
    int d;                     /* channels per head, a multiple of 8                    */
    ttt_dtype io_dtype;        /* dtype of q, k, v and z                                */
    int loss;                  /* ttt_loss                                              */
    int epochs;                /* full-batch inner steps, >= 1                          */
    long long w0_batch_stride; /* 0: W0 is [H,9,d] shared over the batch; H*9*d: [B,H,9,d] */
} ttt_dwconv_desc;

/*
 * TTT with a depthwise 3x3 convolution as the inner model, full-batch inner GD over
 * all N tokens, non-causal (the ViT3 article, observation 6, a small convolution as
 * the inner model of vision TTT, and observation 2, full-batch inner training):
 *     f(X; W)[p][c] = sum_{o = (di+1)*3 + (dj+1), di, dj in {-1,0,1}} X[p + (di,dj)][c] W[o][c]
 * on the token grid with zero padding.  Each epoch takes the gradient of
 * sum_p eta_p l_p at the epoch's start taps and steps by it; z = f(q; W_final).
 *   q, k, v, z : [B,H,N,d] io_dtype; eta: [B,H,N] fp32 or NULL (eta_scalar)
 *   W0         : fp32 taps, see w0_batch_stride; W_out: [B,H,9,d] fp32 or NULL
 * The sequence is held on chip: two padded grids of (height+2) (width+2) d
 * sizeof(io) bytes and V of N d sizeof(io) bytes, each rounded up to 128 bytes, plus
 * 256 + 4 (9 d + N + 9 * 512) bytes must fit in 227 KB (bf16, d = 64: up to 22 x 22
 * tokens), else TTT_ERR_UNSUPPORTED.  Pointers: q, k,
 * v, z 16-byte aligned (TTT_ERR_ALIGN), fp32 arrays 4-byte aligned.
 */
ttt_status ttt_dwconv_fwd(const ttt_dwconv_desc *desc,
                          const void *q, const void *k, const void *v,
                          const float *eta, float eta_scalar,
                          const float *W0, void *z, float *W_out, void *stream);

/* Input-dependent inner learning rate problem description. */
typedef struct {
    int B, T;                  /* batch, tokens per sequence                            */
    int H;                     /* heads, 1 .. 64 (TTT_ERR_UNSUPPORTED above)            */
    int dm;                    /* width of the layer's input tokens, a multiple of 8
                                  (TTT_ERR_UNSUPPORTED otherwise)                       */
} ttt_gate_desc;

/*
 * The inner learning rate as a function of the input token ("Learning to (Learn at
 * Test Time)" walkthrough, section 2.2.3): a learnable vector of the outer loop per
 * head, a sigmoid, and a base rate (1 for TTT-Linear, 0.1 for TTT-MLP):
 *     eta[b,h,t] = eta_base * sigma(theta[h] . x[b,t]),  sigma(a) = 1 / (1 + e^-a)
 *   x     : [B,T,dm] bf16, the layer's input tokens, 16-byte aligned
 *   theta : [H,dm] bf16, one vector per head, 16-byte aligned
 *   eta   : [B,H,T] fp32 (written), 4-byte aligned: the per-token rates that
 *           ttt_linear_fwd, ttt_linear_fwd_seqpar and ttt_mlp_fwd read
 * The dot products accumulate in fp32 from the bf16 operands.  All pointers are
 * device memory owned by the caller; eta must not overlap x or theta (TTT_ERR_ARG).
 * B = 0 or T = 0 queues nothing.  Misaligned pointers: TTT_ERR_ALIGN.
 */
ttt_status ttt_eta_gate(const ttt_gate_desc *desc, const void *x, const void *theta, float eta_base,
                        float *eta, void *stream);

/* Rotary positions problem description.  Strides are in elements, in the order
 * batch, head, token; the features of one head are contiguous.  A batch, head or
 * token stride of an input may be 0 (a broadcast input). */
typedef struct {
    int B, T;                  /* batch, tokens per sequence                            */
    int Hq, Hk;                /* heads of q; heads of k and v                          */
    int d;                     /* head dim, 1 .. 1024 (TTT_ERR_UNSUPPORTED above)       */
    int rot;                   /* leading features that are rotated, even, 0 .. d; the
                                  rest is copied                                        */
    int interleaved;           /* 0: feature i pairs with i + rot/2; 1: 2i with 2i + 1  */
    int inverse;               /* 1: the transposed rotation, which turns the gradients
                                  of the outputs into those of the inputs               */
    ttt_dtype io_dtype;
    int table_rows;            /* positions the table covers: 0 .. table_rows - 1       */
    int period;                /* > 0: positions are taken modulo period (<= table_rows),
                                  e.g. the mini-batch of the TTT layer                  */
    long long pos0;            /* position of token 0 when positions is NULL, >= 0      */
    long long positions_batch_stride; /* T, or 0: positions is [T] for every batch entry */
    long long q_stride[3], k_stride[3], v_stride[3];
    long long q_out_stride[3], k_out_stride[3], v_out_stride[3];
} ttt_rope_desc;

/*
 * Rotary positions on the layer's queries and keys, with the change of layout from
 * the projections (e.g. one [B,T,3,H,d] buffer) to the [B,H,T,d] the layer reads:
 *     out_a = a cos - b sin,  out_b = a sin + b cos
 * for every feature pair (a, b) of the first rot features, (cos, sin) =
 * table[position][pair].  v, when given, is copied into its new layout in the same
 * launch; k and v may be NULL.
 *   table     : [table_rows, rot/2, 2] fp32, cos and sin of every position and pair,
 *               8-byte aligned; scaled for long contexts by whoever makes it
 *   positions : [B,T] (or [T]) 64-bit integers on the device, or NULL for pos0 + t.
 *               A position < 0 or (with period 0) >= table_rows reads nothing: the
 *               token's rotated features become NaN and ttt_sync_status returns
 *               TTT_ERR_RANGE.  pos0 + t is checked before the launch (TTT_ERR_ARG).
 * An output may be its own input (same pointer and strides).  Otherwise it may not share
 * memory with an input, with another output, with the table or the positions, nor hold an
 * element twice: each of its dimensions steps over all of those inside it.  Slices of one
 * buffer with equal strides are told apart exactly, other views by their ends
 * (TTT_ERR_ARG).  Data pointers: aligned to their element (TTT_ERR_ALIGN); 16-byte
 * aligned pointers and strides with rot/2 a multiple of 8 (bf16) or 4 (fp32) move 16
 * bytes at a time.  The rotation is computed in fp32 and rounded once.
 */
ttt_status ttt_rope(const ttt_rope_desc *desc, const void *q, const void *k, const void *v, const float *table,
                    const long long *positions, void *q_out, void *k_out, void *v_out, void *stream);

/* Most axes of ttt_rope_axes. */
#define TTT_ROPE_MAX_AXES 4

/* Rotary positions with several axes.  rope.period is 0. */
typedef struct {
    ttt_rope_desc rope;
    int axes;                       /* 1 .. TTT_ROPE_MAX_AXES                             */
    int grid[TTT_ROPE_MAX_AXES];    /* extents of the token grid, when positions is NULL  */
    long long positions_axis_stride; /* elements from one axis' positions to the next's   */
} ttt_rope_axes_desc;

/*
 * ttt_rope for the tokens of images and video: pair i of a head turns by the token's
 * position on axis pair_axis[i] (time, height, width, ..), (cos, sin) =
 * table[position on that axis][i].
 *   pair_axis : [rot/2] bytes on the host, each < axes; read during the call
 *   positions : [axes,B,T] or [axes,T] 64-bit integers on the device (the strides in the
 *               description), or NULL: token t is element pos0 + t of a row-major grid
 *               (the last axis moves fastest), pos0 + T <= the product of its extents
 *               < 2^31, no extent above table_rows (TTT_ERR_ARG)
 * Everything else is ttt_rope's: layouts, tables, outputs, positions out of range (the
 * pairs of that axis become NaN).  Neighbouring pairs of one axis, 8 (bf16) or 4 (fp32)
 * at a time, read the table 16 bytes at a time.
 */
ttt_status ttt_rope_axes(const ttt_rope_axes_desc *desc, const unsigned char *pair_axis, const void *q, const void *k,
                         const void *v, const float *table, const long long *positions, void *q_out, void *k_out,
                         void *v_out, void *stream);

/* Norms of ttt_block_norm_fwd / _bwd, over the D features of a token.
 *   TTT_NORM_RMS:   w v / sqrt(mean(v^2) + eps)
 *   TTT_NORM_LAYER: w (v - mean) / sqrt(var + eps) + b */
typedef enum { TTT_NORM_NONE = 0, TTT_NORM_RMS = 1, TTT_NORM_LAYER = 2 } ttt_norm;

/* The gate's activation (TTT_GATE_NONE: no gate tensor). */
typedef enum { TTT_GATE_NONE = 0, TTT_GATE_SIGMOID = 1, TTT_GATE_SILU = 2, TTT_GATE_GELU = 3 } ttt_gate_act;

/* Block norm problem description.  Strides are in elements; features are contiguous
 * (y: inside each head). */
typedef struct {
    int B, T, D;               /* batch, tokens, features 1 .. 8192 (TTT_ERR_UNSUPPORTED above) */
    int heads;                 /* y is [B,heads,T,D/heads] (the TTT layer's z); 1: [B,T,D]      */
    ttt_dtype io_dtype;        /* dtype of every token tensor                                   */
    int post, pre;             /* ttt_norm of y and of h                                        */
    int act;                   /* ttt_gate_act                                                  */
    float post_eps, pre_eps;   /* >= 0; 0 only where no row is constant zero                    */
    float alpha;               /* factor of the residual x                                      */
    long long y_stride[3];     /* batch, head, token                                            */
    long long x_stride[2], gate_stride[2], dh_stride[2], du_stride[2]; /* batch, token          */
} ttt_block_norm_desc;

/* Parameter vectors, fp32 [D] on the device, each may be NULL (weights and scale 1,
 * biases 0); biases go with TTT_NORM_LAYER only. */
typedef struct {
    const float *post_weight, *post_bias, *scale, *pre_weight, *pre_bias;
} ttt_block_norm_params;

/* Their gradients (overwritten, not added to), each may be NULL. */
typedef struct {
    float *post_weight, *post_bias, *scale, *pre_weight, *pre_bias;
} ttt_block_norm_grads;

/*
 * The norms before and after a block, its gate and its residual in one pass:
 *     p = N_post(y),  h = alpha x + scale * act(gate) * p,  u = N_pre(h)
 * y is the inner layer's output, gate [B,T,D] its gate's argument, x [B,T,D] the
 * residual stream (NULL: h = scale * act(gate) * p, the input of an output projection),
 * h the new residual stream and u the next layer's input (written when pre is not
 * TTT_NORM_NONE).  ("Learning to (Learn at Test Time)" walkthrough, section 2.2.1: the
 * layer norm behind the layer; the backbone's gate and residual around it.)
 *   h, u  : [B,T,D] contiguous io_dtype; u NULL exactly when pre is TTT_NORM_NONE
 *   stats : [B,T,4] fp32, 16-byte aligned, or NULL: mean and 1/spread of both norms,
 *           which the backward pass reads
 * u is the norm of h before its rounding to io_dtype.  Outputs may not overlap inputs,
 * except h being x (same pointer, contiguous).  Data pointers: aligned to their
 * element; 16-byte aligned pointers, strides of whole 16 bytes and D and D / heads
 * multiples of 8 move 16 bytes at a time.
 */
ttt_status ttt_block_norm_fwd(const ttt_block_norm_desc *desc, const ttt_block_norm_params *params, const void *y,
                              const void *x, const void *gate, void *h, void *u, float *stats, void *stream);

/* Bytes of workspace the backward pass needs (0 for a description it refuses). */
size_t ttt_block_norm_bwd_workspace(const ttt_block_norm_desc *desc);

/*
 * Gradients of ttt_block_norm_fwd: from dh and du (of h and u; dh NULL: zero; du NULL
 * exactly when pre is TTT_NORM_NONE), the forward's inputs and its stats.
 *   dy    : contiguous in y's layout ([B,heads,T,D/heads] or [B,T,D])
 *   dx    : [B,T,D] or NULL;  dgate: [B,T,D], NULL exactly when act is TTT_GATE_NONE
 *   grads : gradients of the parameter vectors, summed over all tokens, or NULL.  The order
 *           of the sums is fixed by the sizes, dtype, norms and gate, the alignment and
 *           strides of the tensors, the gradients asked for and the device: the same call
 *           gives the same bits on every run
 *   workspace : device scratch, 16-byte aligned, at least
 *           ttt_block_norm_bwd_workspace(desc) bytes (NULL allowed when no parameter
 *           gradient is asked for), free again once the work on `stream` is done
 * Outputs may not overlap inputs.
 */
ttt_status ttt_block_norm_bwd(const ttt_block_norm_desc *desc, const ttt_block_norm_params *params, const void *dh,
                              const void *du, const void *y, const void *x, const void *gate, const float *stats,
                              void *dy, void *dx, void *dgate, const ttt_block_norm_grads *grads, void *workspace,
                              size_t workspace_bytes, void *stream);

/* Gate of the recurrence below.
 *   TTT_RECUR_DECAY:   a = f, c = 1         (f is the decay itself)
 *   TTT_RECUR_SIGMOID: a = sigma(f), c = 1
 *   TTT_RECUR_MIX:     a = sigma(f), c = 1 - a */
typedef enum { TTT_RECUR_DECAY = 0, TTT_RECUR_SIGMOID = 1, TTT_RECUR_MIX = 2 } ttt_recurrence_mode;

/* Tokens from one stored state to the next (ttt_recurrence_fwd's states). */
#define TTT_RECURRENCE_CHUNK 128

/* Gated linear recurrence problem description.  Strides in elements (batch, token);
 * channels are contiguous. */
typedef struct {
    int B, T, C;               /* batch (<= 65535), tokens, channels                    */
    ttt_dtype io_dtype;        /* dtype of x, f, h, dh, dx, df                          */
    int mode;                  /* ttt_recurrence_mode                                   */
    long long x_stride[2], f_stride[2], dh_stride[2];
} ttt_recurrence_desc;

/*
 * Gated linear recurrence, every channel by itself:
 *     h_t = a_t h_{t-1} + c_t x_t
 * TTT_RECUR_MIX is the TTT layer whose inner model is a constant, f(k; w) = w, trained
 * on 1/2 ||w - x_t||^2 by one gradient step a token with the rate 1 - a_t of every
 * channel (w_t = w_{t-1} - (1 - a_t)(w_{t-1} - x_t)), mini-batches of one token.
 *   x, f   : [B,T,C] io_dtype
 *   reset  : [B,T] bytes or NULL; where not zero, h_{t-1} is taken as zero (a packed
 *            sequence begins), whatever it held
 *   h0     : [B,C] fp32 start states or NULL (zeros)
 *   h      : [B,T,C] io_dtype, contiguous
 *   h_last : [B,C] fp32 or NULL: the last state (h0 when T = 0); may be h0 itself, so
 *            that a decoder steps its states in place
 *   states : [B, ceil(T / TTT_RECURRENCE_CHUNK), C] fp32 or NULL: the state before every
 *            chunk of tokens, which the backward pass reads
 * States are fp32 throughout; sums run in an order that is fixed by the sizes, dtype, mode,
 * alignment and strides of the tensors and the device (the same call gives the same bits on
 * every run).  TTT_RECUR_DECAY is meant for |f| <= 1: with larger factors h is right as long as
 * the product of any 2048 neighbouring ones stays inside fp32's range, past which it can be
 * infinite or NaN where the state itself would not be.  Data
 * pointers: aligned to their element; 16-byte alignment, strides of whole 16 bytes and C a
 * multiple of 8 move wide vectors.  Outputs may not overlap inputs (h_last as above).
 */
ttt_status ttt_recurrence_fwd(const ttt_recurrence_desc *desc, const void *x, const void *f,
                              const unsigned char *reset, const float *h0, void *h, float *h_last, float *states,
                              void *stream);

/*
 * Gradients of ttt_recurrence_fwd from dh [B,T,C] (of h; NULL: zero) and dh_last [B,C]
 * fp32 (of h_last; NULL: zero), the forward's x, f, reset and the states it stored.
 *   dx, df : [B,T,C] io_dtype, contiguous (df: of f, the logit or the decay itself)
 *   dh0    : [B,C] fp32 or NULL
 */
ttt_status ttt_recurrence_bwd(const ttt_recurrence_desc *desc, const void *dh, const void *x, const void *f,
                              const unsigned char *reset, const float *states, const float *dh_last, void *dx,
                              void *df, float *dh0, void *stream);

/* Activation of the short convolution. */
typedef enum { TTT_CONV_NONE = 0, TTT_CONV_SILU = 1 } ttt_conv_act;

/* Short causal convolution problem description.  Strides in elements (batch, token);
 * channels are contiguous. */
typedef struct {
    int B, T, C;               /* batch, tokens, channels (B T < 2^31, T and C <= 2^30)  */
    int width;                 /* K, taps of a channel: 1 .. 4 (TTT_ERR_UNSUPPORTED above) */
    ttt_dtype io_dtype;        /* dtype of x, y, the states, dy, dx                     */
    int act;                   /* ttt_conv_act                                          */
    long long x_stride[2], dy_stride[2]; /* dy's: the backward pass alone reads them      */
} ttt_short_conv_desc;

/*
 * Short causal convolution along the tokens, every channel by itself (the temporal
 * convolution of the Mamba backbone, "Learning to (Learn at Test Time)" walkthrough,
 * section 2.2.4):
 *     y_t = act(bias + sum_{j=0}^{K-1} weight[j] x_{t-K+1+j})
 *   x         : [B,T,C] io_dtype
 *   weight    : [C,K] fp32, bias: [C] fp32 or NULL
 *   reset     : [B,T] bytes or NULL; where not zero, a packed sequence begins: its tokens
 *               see zeros for every row before it, whatever they hold
 *   state     : [B,K-1,C] io_dtype, the K-1 inputs before the first token, oldest first,
 *               or NULL (zeros)
 *   y         : [B,T,C] io_dtype, contiguous
 *   state_out : [B,K-1,C] io_dtype or NULL: the last K-1 inputs of the running sequence
 *               (zeros before its start); may be state itself
 * Sums in fp32, rounded once.  Data pointers: aligned to their element; where pointers,
 * strides and C are multiples of four elements, four move at a time.  Outputs may not
 * overlap inputs or each other (state_out as above).
 */
ttt_status ttt_short_conv_fwd(const ttt_short_conv_desc *desc, const void *x, const float *weight, const float *bias,
                              const unsigned char *reset, const void *state, void *y, void *state_out, void *stream);

/* Bytes of workspace the backward pass needs (0 for a description it refuses). */
size_t ttt_short_conv_bwd_workspace(const ttt_short_conv_desc *desc);

/*
 * Gradients of ttt_short_conv_fwd from dy [B,T,C] (of y) and dstate_out [B,K-1,C] fp32 (of
 * state_out; NULL: zero), with the forward's inputs.
 *   dx       : [B,T,C] io_dtype, contiguous
 *   dweight  : [C,K] fp32, dbias: [C] fp32, dstate: [B,K-1,C] fp32, each may be NULL
 *              (overwritten, not added to)
 *   workspace: device scratch, 16-byte aligned, at least ttt_short_conv_bwd_workspace(desc)
 *              bytes (NULL allowed when neither dweight nor dbias is asked for), free again
 *              once the work on `stream` is done
 * Sums over the tokens run in an order that is fixed by the sizes, dtype, alignment and
 * strides: the same call gives the same bits.
 */
ttt_status ttt_short_conv_bwd(const ttt_short_conv_desc *desc, const void *dy, const void *x, const float *weight,
                              const float *bias, const unsigned char *reset, const void *state,
                              const float *dstate_out, void *dx, float *dweight, float *dbias, float *dstate,
                              void *workspace, size_t workspace_bytes, void *stream);

/* Tokens from one stored state to the next (ttt_selective_scan_fwd's states). */
#define TTT_SCAN_CHUNK 32

/* Selective scan problem description.  Strides in elements; channels (B and C: states)
 * are contiguous. */
typedef struct {
    int B, T, C;               /* batch (<= 65535), tokens (<= 2^30), channels            */
    int N;                     /* states of a channel, 1 .. 64; B T G and C N at most
                                  0x7fff0000 (TTT_ERR_UNSUPPORTED above, as for B and T)  */
    int G;                     /* groups of C / G neighbouring channels with one B and C  */
    ttt_dtype io_dtype;        /* dtype of every token tensor                           */
    int softplus;              /* 1: the rate is softplus(delta + bias); 0: delta + bias  */
    long long x_stride[2], delta_stride[2], z_stride[2], dy_stride[2]; /* batch, token; dy's:
                                  the backward pass alone reads them                    */
    long long b_stride[3], c_stride[3];                                /* batch, token, group */
} ttt_scan_desc;

/* Parameters, fp32 on the device; D and delta_bias may be NULL (zeros). */
typedef struct {
    const float *A;            /* [C,N]                                                 */
    const float *D, *delta_bias; /* [C]                                                 */
} ttt_scan_params;

/* Their gradients (overwritten, not added to), each may be NULL. */
typedef struct {
    float *A, *D, *delta_bias;
} ttt_scan_grads;

/* Bytes of workspace of the forward pass (0 where it needs none). */
size_t ttt_selective_scan_fwd_workspace(const ttt_scan_desc *desc);

/*
 * Selective state space scan (the Mamba backbone's layer behind the short convolution),
 * every channel c with N states:
 *     d_t = softplus(delta_t + bias),  h_t[n] = exp(d_t A[n]) h_{t-1}[n] + d_t x_t B_t[n],
 *     y_t = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
 *   x, delta : [B,T,C] io_dtype;  z: [B,T,C] or NULL (no gate)
 *   Bm, Cm   : [B,T,G,N] io_dtype
 *   reset    : [B,T] bytes or NULL; where not zero, h_{t-1} is taken as zero (a packed
 *              sequence begins), whatever it held
 *   h0       : [B,C,N] fp32 start states or NULL (zeros)
 *   y        : [B,T,C] io_dtype, contiguous
 *   h_last   : [B,C,N] fp32 or NULL: the last state (h0 when T = 0); may be h0 itself, so
 *              that a decoder steps its states in place
 *   states   : [B, ceil(T / TTT_SCAN_CHUNK), C, N] fp32 or NULL: the state before every chunk
 *              of tokens, which the backward pass reads
 *   workspace: device scratch, 16-byte aligned, at least ttt_selective_scan_fwd_workspace(desc)
 *              bytes, free again once the work on `stream` is done
 * A is finite and meant for d A <= 0 (decays).  States are fp32 throughout; sums run in an
 * order that is fixed by the sizes, dtype, alignment and strides (the same call gives the
 * same bits).  Data pointers: aligned to their element; where all have 16-byte alignment, strides
 * of whole 16 bytes, C / G and N multiples of 8 (bf16) or 4 (fp32), 16 bytes move at a time.
 * Outputs may not overlap inputs or each other (h_last as above).
 */
ttt_status ttt_selective_scan_fwd(const ttt_scan_desc *desc, const ttt_scan_params *params, const void *x,
                                  const void *delta, const void *Bm, const void *Cm, const void *z,
                                  const unsigned char *reset, const float *h0, void *y, float *h_last, float *states,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Bytes of workspace the backward pass needs (0 for a description it refuses). */
size_t ttt_selective_scan_bwd_workspace(const ttt_scan_desc *desc);

/*
 * Gradients of ttt_selective_scan_fwd from dy [B,T,C] (of y) and dh_last [B,C,N] fp32 (of
 * h_last; NULL: zero), the forward's inputs and the states it stored.
 *   dx, ddelta : [B,T,C] io_dtype, contiguous (ddelta: of delta itself, through the softplus)
 *   dz         : [B,T,C], NULL exactly when z is NULL
 *   dB, dC     : [B,T,G,N] io_dtype, contiguous, summed over a group's channels
 *   dh0        : [B,C,N] fp32 or NULL
 *   workspace  : device scratch, 16-byte aligned, ttt_selective_scan_bwd_workspace(desc) bytes
 * Sums over channels and tokens run in fixed orders, as the forward pass's.
 */
ttt_status ttt_selective_scan_bwd(const ttt_scan_desc *desc, const ttt_scan_params *params, const void *dy,
                                  const void *x, const void *delta, const void *Bm, const void *Cm, const void *z,
                                  const unsigned char *reset, const float *states, const float *dh_last, void *dx,
                                  void *ddelta, void *dB, void *dC, void *dz, const ttt_scan_grads *grads, float *dh0,
                                  void *workspace, size_t workspace_bytes, void *stream);

/* Waits for `stream`, then reports (and clears) a kernel wait timeout
 * (TTT_ERR_TIMEOUT) or a position out of range (TTT_ERR_RANGE) recorded on the current
 * device, or a CUDA error seen while waiting.  Of both, the timeout is reported first and
 * the position by the next call. */
ttt_status ttt_sync_status(void *stream);

/* Static description of a status code. */
const char *ttt_status_str(ttt_status s);

/* Number of kernel launches this library has enqueued on the calling process
 * (all devices); used to count this library's launches inside a timed region. */
unsigned long long ttt_launch_count(void);

/*
 * Test hook of the timeout path (never needed in normal use; the pages have no
 * counterpart).  With ns > 0, every later TTT-Linear launch of the b = 16 kernel
 * (causal or not, mini_batch 16, d <= 64) and of the full-batch kernel (bf16, d = 64,
 * mini_batch >= T <= 256, one epoch) makes its first consumer-side wait on a barrier
 * that nothing arrives at, bounded by ns nanoseconds: the wait runs out, the kernel
 * records TTT_ERR_TIMEOUT in the device status word, skips its products (outputs
 * undefined), still waits for its own copies in flight and frees its tensor memory,
 * and ttt_sync_status() reports the timeout.  So do the recurrence's tile kernels (more than
 * 16 tokens): each cluster's last block gives up first, then its other blocks, which
 * wait for it.  ns = 0 restores normal operation.  The
 * setting is process-wide (read at each launch); other kernels ignore it.
 */
void ttt_debug_wait_limit(unsigned long long ns);

#ifdef __cplusplus
}
#endif

#endif /* TTT_H_ */
