// ttt_block_norm.cu -- launches of the block norm (ttt_block_norm.cuh), and the kernel that
// adds the backward pass's partial parameter gradients.
#include <mutex>

#include "ttt_block_norm.cuh"

namespace ttt {
namespace {

constexpr int kMaxD = 8192;

// What an absent parameter vector stands for.
#define TTT_4(x) x, x, x, x
#define TTT_64(x) TTT_4(TTT_4(TTT_4(x)))
#define TTT_1024(x) TTT_4(TTT_4(TTT_64(x)))
__device__ __align__(16) float g_ones[kMaxD] = {TTT_4(TTT_1024(1.f)), TTT_4(TTT_1024(1.f))};
__device__ __align__(16) float g_zeros[kMaxD];

bool defaults(const float *&ones, const float *&zeros)
{
    static std::mutex mu;
    static float *addr[64][2] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev][1]) {
        void *a = nullptr, *b = nullptr;
        if (cudaGetSymbolAddress(&a, g_ones) != cudaSuccess || cudaGetSymbolAddress(&b, g_zeros) != cudaSuccess) return false;
        addr[dev][0] = static_cast<float *>(a);
        addr[dev][1] = static_cast<float *>(b);
    }
    ones = addr[dev][0];
    zeros = addr[dev][1];
    return true;
}

bool vectors(const BlockNormArgs &a, NormVectors &v)
{
    const float *ones, *zeros;
    if (!defaults(ones, zeros)) return false;
    v = {a.w1 ? a.w1 : ones, a.b1 ? a.b1 : zeros, a.scale ? a.scale : ones, a.w2 ? a.w2 : ones, a.b2 ? a.b2 : zeros};
    return true;
}

// Adds the blocks' partial parameter gradients in a fixed order: 32 columns a block, 32
// threads a column, eight loads of each in flight.  Starts while the backward kernel ends
// and waits for it on the device.
struct ReduceParams {
    const float *part;
    float *out[5];  // by slot
    int nblocks, nvec, D;
};

__global__ void __launch_bounds__(1024) ttt_block_norm_reduce_kernel(const __grid_constant__ ReduceParams p)
{
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, c = blockIdx.x * 32 + lane, slot = blockIdx.y;
    const size_t row = (size_t)p.nvec * p.D;
    const float *src = p.part + (size_t)slot * p.D + c;
    cudaGridDependencySynchronize();
    float v = 0.f;
    if (c < p.D)
        for (int i = y; i < p.nblocks; i += 32 * 8) {
            float w[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) w[u] = i + 32 * u < p.nblocks ? src[(i + 32 * u) * row] : 0.f;
#pragma unroll
            for (int u = 0; u < 8; ++u) v += w[u];
        }
    s[y][lane] = v;
    __syncthreads();
    v = s[lane][y];  // column y, partial sums across the warp
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    const int col = blockIdx.x * 32 + y;
    if (lane == 0 && col < p.D) p.out[slot][col] = v;
}

// Threads of a row and chunks of a thread: part of a warp up to 256 features, then one
// block a row with one chunk a thread, two past `two_from` features.  (A warp with three
// chunks a lane for 768 features, no barrier: 35.5 us against 30.6 for a block of three
// warps at 8 x 2048 x 768, sandwich forward; the chunks cost registers, so warps.)
NormShape row_shape(int D, int two_from)
{
    NormShape s;
    s.block = D > 32 * kNormChunk;
    s.K = s.block && D > two_from ? 2 : 1;
    if (s.block) {
        const int need = (D + kNormChunk * s.K - 1) / (kNormChunk * s.K);
        s.lanes = s.threads = (need + 31) / 32 * 32;
    } else {
        s.lanes = 1;
        while (s.lanes * kNormChunk < D) s.lanes *= 2;
        s.threads = 128;
    }
    return s;
}

// Two chunks from 1024 features on halve what a row costs every thread: 2 x 32768 x 2048
// forward 287 us against 327 before the parameter vectors were held in registers, backward
// (whose sums then take all 255 registers) 512 against 579; backward only with 16-byte rows.
NormShape fwd_shape(int D) { return row_shape(D, 1024); }
NormShape bwd_shape(int D, bool whole) { return row_shape(D, whole ? 1024 : 512 * kNormChunk); }

// Features that stand together in every tensor: eight (16-byte pointers and strides, D and
// the heads multiples of eight), two (pairs aligned), or one.
int features_together(int es, int D, int dh, const void *const *ptr, int np, const void *const *vec, const long long *st, int ns)
{
    long long elems = D | dh, bytes = 0;
    for (int i = 0; i < np; ++i) bytes |= (long long)reinterpret_cast<uintptr_t>(ptr[i]);
    for (int i = 0; i < ns; ++i) bytes |= st[i] * es;
    long long vb = 0;
    for (int i = 0; i < 5; ++i) vb |= (long long)reinterpret_cast<uintptr_t>(vec[i]);
    if (elems % kNormChunk == 0 && bytes % 16 == 0 && vb % 16 == 0) return kNormChunk;
    return elems % 2 == 0 && bytes % (2 * es) == 0 && vb % 8 == 0 ? 2 : 1;
}

// Is a token-major tensor contiguous, or absent?
bool even(const BlockNormArgs &a, const void *p, long long sb, long long st)
{
    return !p || ((a.T == 1 || st == a.D) && (a.B == 1 || sb == (long long)a.T * a.D));
}

}  // namespace

// The most blocks of the backward pass, by size alone (the workspace holds their sums): 512
// threads an SM, no fewer than the kernels' registers allow.
int block_norm_bwd_blocks(int D, long long rows)
{
    const NormShape s = bwd_shape(D, false);
    const long long per = s.block ? 1 : s.threads / s.lanes, groups = (rows + per - 1) / per;
    const long long fit = 152LL * (512 / s.threads);
    return (int)(groups < fit ? groups : fit);
}

int launch_block_norm_fwd(const BlockNormArgs &a)
{
    NormFwdParams p;
    if (!vectors(a, p.v)) return -4;
    p.y = a.y;
    p.x = a.x;
    p.g = a.gate;
    p.h = a.h;
    p.u = a.u;
    p.stats = a.stats;
    for (int i = 0; i < 3; ++i) p.ys[i] = a.ys[i];
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i];
        p.gs[i] = a.gs[i];
    }
    const NormShape s = fwd_shape(a.D);
    p.rows = (uint32_t)((long long)a.B * a.T);
    p.byT = make_div(a.T);
    p.T = a.T;
    p.D = a.D;
    p.dh = a.dh;
    p.lanes = s.lanes;
    p.post = a.post;
    p.pre = a.pre;
    p.act = a.act;
    p.even = a.dh == a.D && even(a, a.y, a.ys[0], a.ys[2]) && even(a, a.x, a.xs[0], a.xs[1]) &&
             even(a, a.gate, a.gs[0], a.gs[1]);
    p.eps1 = a.eps1;
    p.eps2 = a.eps2;
    p.alpha = a.alpha;
    const void *ptr[] = {a.y, a.x, a.gate, a.h, a.u}, *vec[] = {a.w1, a.b1, a.scale, a.w2, a.b2};
    const long long st[] = {a.ys[0], a.ys[1], a.ys[2], a.xs[0], a.xs[1], a.gs[0], a.gs[1]};
    const int group = features_together(a.bf16 ? 2 : 4, a.D, a.dh, ptr, 5, vec, st, 7);
    return a.bf16 ? norm_fwd_bf16(p, s, group, a.stream) : norm_fwd_f32(p, s, group, a.stream);
}

int launch_block_norm_bwd(const BlockNormArgs &a)
{
    NormBwdParams p;
    if (!vectors(a, p.v)) return -4;
    p.y = a.y;
    p.x = a.x;
    p.g = a.gate;
    p.dh_in = a.dh_in;
    p.du = a.du;
    p.dy = a.dy;
    p.dx = a.dx;
    p.dg = a.dgate;
    p.stats = a.stats;
    p.part = static_cast<float *>(a.ws);
    for (int i = 0; i < 3; ++i) p.ys[i] = a.ys[i];
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i];
        p.gs[i] = a.gs[i];
        p.dhs[i] = a.dhs[i];
        p.dus[i] = a.dus[i];
    }
    const void *ptr[] = {a.y, a.x, a.gate, a.dh_in, a.du, a.dy, a.dx, a.dgate}, *vec[] = {a.w1, a.b1, a.scale, a.w2, a.b2};
    const long long st[] = {a.ys[0],  a.ys[1],  a.ys[2],  a.xs[0],  a.xs[1], a.gs[0],
                            a.gs[1], a.dhs[0], a.dhs[1], a.dus[0], a.dus[1]};
    const int group = features_together(a.bf16 ? 2 : 4, a.D, a.dh, ptr, 8, vec, st, 11);
    const NormShape s = bwd_shape(a.D, group == kNormChunk);
    p.rows = (uint32_t)((long long)a.B * a.T);
    p.byT = make_div(a.T > 0 ? a.T : 1);
    p.T = a.T;
    p.D = a.D;
    p.dh = a.dh;
    p.lanes = s.lanes;
    p.post = a.post;
    p.pre = a.pre;
    p.act = a.act;
    p.even = a.dh == a.D && even(a, a.y, a.ys[0], a.ys[2]) && even(a, a.x, a.xs[0], a.xs[1]) &&
             even(a, a.gate, a.gs[0], a.gs[1]) && even(a, a.dh_in, a.dhs[0], a.dhs[1]) && even(a, a.du, a.dus[0], a.dus[1]);
    p.alpha = a.alpha;
    ReduceParams q = {};
    p.nvec = 0;
    for (int i = 0; i < 5; ++i) {
        p.slot[i] = a.dvec[i] ? p.nvec : -1;
        if (a.dvec[i]) q.out[p.nvec++] = a.dvec[i];
    }
    int blocks = 0;
    if (p.rows > 0) {  // no tokens: only the sums, all zero
        const int limit = block_norm_bwd_blocks(a.D, p.rows);
        const int rc = a.bf16 ? norm_bwd_bf16(p, s, group, limit, a.stream, &blocks) : norm_bwd_f32(p, s, group, limit, a.stream, &blocks);
        if (rc) return rc;
    }
    if (p.nvec) {
        q.part = p.part;
        q.nblocks = blocks;
        q.nvec = p.nvec;
        q.D = a.D;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((a.D + 31) / 32, p.nvec);
        cfg.blockDim = dim3(1024);
        cfg.stream = a.stream;
        cudaLaunchAttribute at;
        at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &at;
        cfg.numAttrs = 1;
        if (cudaLaunchKernelEx(&cfg, ttt_block_norm_reduce_kernel, q) != cudaSuccess) return -4;
    }
    return 0;
}

}  // namespace ttt
