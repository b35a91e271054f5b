// ttt_internal.h -- host-side launch interface between the C ABI (ttt_api.cu)
// and the kernels.  Not installed; not part of the public ABI.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

namespace ttt {

struct LinearArgs {
    int B, H, T, d, b, causal;
    int loss = 0, epochs = 1;  // loss: 0 MSE, 1 negative dot product; inner GD steps per mini-batch
    const float *ln_gamma = nullptr, *ln_beta = nullptr;  // inner norm [H][d] (null: f(x) = x W)
    float ln_eps = 1e-6f;
    const void *q, *k, *v;
    const float *eta;
    float eta_scalar;
    const float *W0;
    long long w0_bstride;
    void *z;
    float *W_out;
    int *status;         // device status word (timeouts)
    cudaStream_t stream;
    // test hook (ttt_debug_wait_limit): > 0 makes the first consumer wait of the b = 16
    // and full-batch kernels wait this long on a barrier nothing arrives at
    unsigned long long test_stall_ns = 0;
};

struct MlpArgs {
    int B, H, T, d, m, b, causal, per_batch;
    int act = 0;  // inner activation: 0 SiLU, 1 GELU
    const float *ln_gamma = nullptr, *ln_beta = nullptr;  // inner norm [H][d] (null: plain MLP)
    float ln_eps = 1e-6f;
    const void *q, *k, *v;
    const float *eta;
    float eta_scalar;
    const float *W1, *c1, *W2, *c2;
    void *z;
    float *W1o, *c1o, *W2o, *c2o;
    int *status;
    cudaStream_t stream;
    unsigned long long test_stall_ns = 0;  // > 0: the timeout test (full-batch kernel)
};

struct DwconvArgs {
    int B, H, hh, ww, d, loss, epochs, bf16;
    const void *q, *k, *v;
    const float *eta;
    float eta_scalar;
    const float *W0;
    long long w0_bstride;
    void *z;
    float *W_out;
    int *status;  // device status word (timeouts)
    cudaStream_t stream;
};

struct GateArgs {
    int B, T, H, dm;
    const void *x, *theta;  // bf16 [B][T][dm], [H][dm]
    float eta_base;
    float *eta;             // fp32 [B][H][T]
    int *status;            // device status word (timeouts)
    cudaStream_t stream;
};

struct RopeArgs {
    int B, T, Hq, Hk, d, rot, interleaved, inverse, bf16, table_rows, period;
    long long pos0, pos_bstride;
    const void *q, *k, *v;  // k, v may be null
    void *q_out, *k_out, *v_out;
    long long in_stride[3][3], out_stride[3][3];  // [q, k, v][batch, head, token], elements
    const float *table;          // [table_rows][rot/2][2] cos, sin
    const long long *positions;  // or null: pos0 + t
    int *range_status;           // device status word of positions out of range
    int axes = 0;                // > 0: several axes, positions [axes][..] or coordinates on the grid
    long long axis_stride = 0;
    int grid[4] = {};
    const unsigned char *pair_axis = nullptr;  // host, [rot/2]
    cudaStream_t stream;
};

struct BlockNormArgs {
    int B, T, D, dh, bf16, post, pre, act;  // dh = D / heads
    float eps1, eps2, alpha;
    const void *y, *x, *gate;
    long long ys[3], xs[2], gs[2], dhs[2], dus[2];
    const float *w1, *b1, *scale, *w2, *b2;
    void *h, *u;   // forward
    float *stats;  // written by the forward, read by the backward
    const void *dh_in, *du;
    void *dy, *dx, *dgate;
    float *dvec[5];  // gradients of w1, b1, scale, w2, b2 (null: not asked for)
    void *ws;
    cudaStream_t stream;
};

constexpr int kRecurDecay = 0, kRecurSigmoid = 1, kRecurMix = 2;
constexpr int kRecurChunk = 128;  // tokens from one stored state to the next

struct RecurArgs {
    int B, T, C, bf16, mode;
    const void *x, *f, *dh;
    long long xs[2], fs[2], ds[2];
    const unsigned char *reset;
    const float *h0, *dh_last;
    void *h, *dx, *df;
    float *h_last, *states, *dh0;  // states: written by the forward, read by the backward
    int *status;                   // device status word (timeouts)
    unsigned long long test_stall_ns = 0;
    cudaStream_t stream;
};

constexpr int kConvMaxWidth = 4;

struct ConvArgs {
    int B, T, C, K, bf16, silu;
    const void *x, *dy;
    long long xs[2], dys[2];
    const float *weight, *bias;
    const unsigned char *reset;
    const void *state;         // [B][K-1][C] io dtype or null
    void *y, *state_out;       // forward
    const float *dstate_out;   // backward, [B][K-1][C] fp32 or null
    void *dx;
    float *dweight, *dbias, *dstate;
    void *ws;
    cudaStream_t stream;
};

constexpr int kScanChunk = 32;      // tokens from one stored state to the next
constexpr int kScanMaxN = 64;
constexpr int kScanStepTokens = 8;  // up to here token after token straight from memory

struct ScanArgs {
    int B, T, C, N, G, bf16, softplus;
    const void *x, *delta, *z, *Bm, *Cm, *dy;
    long long xs[2], ds[2], zs[2], dys[2], bs[3], cs[3];
    const float *A, *D, *bias;
    const unsigned char *reset;
    const float *h0;
    void *y;
    float *h_last, *states;  // states: written by the forward, read by the backward
    const float *dh_last;
    void *dx, *ddelta, *dz, *dB, *dC;
    float *dA, *dD, *dbias, *dh0;
    void *ws;
    cudaStream_t stream;
};

// TMA descriptor of a bf16 token tensor viewed as [BH][T][d]: boxes of `rows`
// tokens x `cols` features (0: min(d, 64)), swizzled to the box row length, rows
// past T zero-filled on loads and dropped on stores.  Returns false if the driver
// entry point is unavailable or rejects it.
bool encode_token_map(CUtensorMap *m, const void *ptr, int BH, int T, int d, int rows, int cols = 0);

// Descriptor of a token tensor [BH][hh][ww][d] (bf16 or fp32) whose box is one
// sequence's zero-bordered grid: d x (ww+2) x (hh+2) at coordinates (0, -1, -1, bh),
// the border read as zeros (out of range).  False if d > 256, hh + 2 or ww + 2 > 256,
// or the encoding fails.
bool encode_grid_map(CUtensorMap *m, const void *ptr, bool bf16, int BH, int hh, int ww, int d);

// Descriptor of rows [batch][rows][width] (bf16 or fp32) with element strides, boxes of
// `height` rows x `cols` elements, out-of-range elements read as zeros.  False if a stride
// is zero or not a multiple of 16 bytes, the pointer is not 16-byte aligned, or the
// encoding fails.
bool encode_rows_map(CUtensorMap *m, const void *ptr, bool bf16, int width, int rows, int batch, long long row_stride,
                     long long batch_stride, int cols, int height);

// q, k, v descriptors (zeroed, unused when T == 0); false on an encoding failure.
inline bool encode_qkv(CUtensorMap *maps, const void *q, const void *k, const void *v, int BH, int T,
                       int d, int rows)
{
    for (int i = 0; i < 3; ++i)
        for (size_t j = 0; j < sizeof(CUtensorMap); ++j) reinterpret_cast<char *>(&maps[i])[j] = 0;
    if (T == 0) return true;
    return encode_token_map(&maps[0], q, BH, T, d, rows) && encode_token_map(&maps[1], k, BH, T, d, rows) &&
           encode_token_map(&maps[2], v, BH, T, d, rows);
}

// Each returns 0 or a negative ttt_status code.
int launch_linear_bf16(const LinearArgs &a);
int launch_linear_b16(const LinearArgs &a);  // b = 16 specialisation (d <= 64)
int launch_linear_b1(const LinearArgs &a);   // b = 1 (delta rule), column-parallel
int launch_linear_fb_tc(const LinearArgs &a);  // full batch, one epoch, on tcgen05
// b = 16, d <= 64 kernel over segments of each chain (segment 0 = tokens [0, len0),
// segment s >= 1 = [len0 + (s-1) seg_len, len0 + s seg_len)).  prep = false: output
// units for segments seg0 .. seg0+nseg-1 of every chain, from start weights W0
// (segment 0) or Wst (segment s: Wst[bh][s-1]).  prep = true: the state chain of
// segment 0 (its end weights to Wst[bh][0]) and the affine maps of segments
// 1 .. nsplit-2 (to mapbuf).  maps: the q, k, v descriptors (64-token boxes).
int launch_linear_b16_segments(const LinearArgs &a, int nsplit, int len0, int seg_len, int seg0, int nseg,
                               bool prep, float *Wst, float *mapbuf, const CUtensorMap *maps);
int launch_linear_fb(const LinearArgs &a);   // one full-batch mini-batch (b = T <= 256, non-causal, d = 64); -2 otherwise
int launch_linear_f32(const LinearArgs &a);
int launch_mlp_f32(const MlpArgs &a);
int launch_mlp_bf16(const MlpArgs &a);
// one full-batch mini-batch (b >= T, non-causal), d = 64, m = 256, on tcgen05; -2 otherwise
int launch_mlp_fb_tc(const MlpArgs &a);
// Sequence-parallel TTT-Linear (ttt_linear_seqpar.cu): the segment plan for a
// problem (false: the problem is not split, run the one-unit-per-chain path).
struct SeqparPlan {
    int nsplit = 0, len0 = 0, seg_len = 0;   // segments per chain, segment lengths
    size_t map_bytes = 0, wst_bytes = 0;     // scratch: affine maps, start weights
};
bool seqpar_plan(const LinearArgs &a, SeqparPlan &pl);
size_t seqpar_workspace_bytes(const SeqparPlan &pl);
// Enqueues the split forward on a.stream (forks a side stream and joins it back);
// ws: at least seqpar_workspace_bytes(pl) bytes of device memory, 256-byte aligned.
int launch_linear_seqpar(const LinearArgs &a, const SeqparPlan &pl, void *ws);
// The same split enqueued on a.stream alone: the preparing launch, the scan, then
// every segment's outputs in one launch (equal segments; seqpar_plan_serial).
bool seqpar_plan_serial(const LinearArgs &a, SeqparPlan &pl);
int launch_linear_seqpar_serial(const LinearArgs &a, const SeqparPlan &pl, void *ws);

// Depthwise 3x3 convolution inner model (ttt_dwconv.cu): shared memory bytes of
// one CTA and the launch.
size_t dwconv_smem(int hh, int ww, int d, int es);
int launch_dwconv(const DwconvArgs &a);
int launch_eta_gate(const GateArgs &a);  // H <= 64; -2 otherwise
// May this kernel be launched with that much dynamic shared memory on the current device?
// Its limit is raised once, to the most the device has, and never lowered: host threads
// that launch the same kernel with other sizes do not disturb each other.
bool allow_shared(const void *kernel, int bytes);
template <typename... KArgs> bool allow_shared(void (*kernel)(KArgs...), int bytes)
{
    return allow_shared(reinterpret_cast<const void *>(kernel), bytes);
}

int launch_rope(const RopeArgs &a);
int launch_recurrence(const RecurArgs &a, bool backward);
// how the scan's two directions cut a sequence: pieces, tokens of one
struct ScanPieces {
    int segs, len;
};
size_t conv_bwd_workspace(int B, int T, int C, int K);
int launch_conv_fwd(const ConvArgs &a);
int launch_conv_bwd(const ConvArgs &a);  // 2 kernels
size_t scan_fwd_workspace(int B, int T, int C, int N, int G);
size_t scan_bwd_workspace(int B, int T, int C, int N, int G);
// each returns the number of its launches or a negative status
int launch_scan_fwd(const ScanArgs &a);
int launch_scan_bwd(const ScanArgs &a);
int launch_block_norm_fwd(const BlockNormArgs &a);
int launch_block_norm_bwd(const BlockNormArgs &a);
int block_norm_bwd_blocks(int D, long long rows);  // partial sums per parameter gradient

// Largest d*m the fp32 MLP path holds on chip.
bool mlp_f32_fits(int d, int m);

}  // namespace ttt
