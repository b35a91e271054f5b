// ttt_block_norm.cu -- what stands around a block's inner layer, in one pass over the
// rows (tokens), forward and backward:
//     p = N1(y),  m = scale * act(gate) * p,  h = alpha x + m,  u = N2(h)
// N1, N2: none, RMS (v / sqrt(mean v^2 + eps) * w) or layer norm ((v - mean) /
// sqrt(var + eps) * w + b) over the D features; y token-major or the TTT layer's
// head-major output.  Backward with dn the gradient of a normalised row n = (v - mean) r:
//     dv = r (dn - [layer] mean(dn) - n mean(dn n)).
//
// Bound by HBM: every tensor is read or written once.  A row belongs to a group of
// `lanes` threads (part of a warp for D <= 256, else the whole block), a thread holding K
// chunks of eight features in fp32 registers, so a row's statistics and its outputs come
// from one read.  The variance is taken about the mean (each warp's own, joined by the
// parallel-variance formula), never as a difference of squares.
#include "ttt_device.cuh"
#include "ttt_internal.h"
#include "ttt_vec.cuh"

namespace ttt {
namespace {

constexpr int kSMs = 152;
constexpr int kC = 8;  // features of a chunk

// row / T for rows below 2^31: multiply by ceil(2^(32 + shift) / T), keep the high part
// (Granlund and Montgomery, Division by invariant integers using multiplication).
struct Div {
    uint32_t d, mul, shift;
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const
    {
        return d == 1 ? n : __umulhi(n, mul) >> shift;
    }
};

Div make_div(int d)
{
    Div r = {(uint32_t)d, 0, 0};
    if (d > 1) {
        while ((1u << r.shift) < (uint32_t)d) ++r.shift;  // 2^shift >= d, shift >= 1
        --r.shift;
        r.mul = (uint32_t)(((1ull << (32 + r.shift)) + d - 1) / d);
    }
    return r;
}

struct Vectors {  // fp32 [D], null: 1 (weights, scale) or 0 (biases)
    const float *w1, *b1, *sc, *w2, *b2;
};

struct FwdParams {
    const void *y, *x, *g;
    void *h, *u;
    float *stats;
    Vectors v;
    long long ys[3], xs[2], gs[2];
    uint32_t rows;
    Div byT;
    int T, D, dh, lanes, post, pre, act;
    float eps1, eps2, alpha;
};

struct BwdParams {
    const void *y, *x, *g, *dh_in, *du;
    void *dy, *dx, *dg;
    const float *stats;
    float *part;  // [blocks][nvec][D] partial parameter gradients
    Vectors v;
    long long ys[3], xs[2], gs[2], dhs[2], dus[2];
    uint32_t rows;
    Div byT;
    int T, D, dh, lanes, post, pre, act;
    int slot[5];  // slot of each parameter gradient among the nvec, -1: absent
    int nvec;
    float alpha;
};

// ------------------------------------------------------------------- activations

// act(g) and its derivative: 1 sigmoid, 2 SiLU, 3 GELU (g Phi(g)).  The logistic from
// exp(-g): past the range of exp it is 0 or 1.  Phi: for bf16 tensors by Abramowitz &
// Stegun 7.1.26 (|error| <= 1.5e-7, far below the rounding of the output, one exponential
// shared with the density), for fp32 CUDA's normcdff.
__device__ __forceinline__ float logistic(float g) { return __fdividef(1.f, 1.f + __expf(-g)); }

template <typename T> __device__ __forceinline__ float gelu_cdf(float g, float &density)
{
    float e, c;
    if constexpr (sizeof(T) == 2) {
        c = norm_cdf(g, e);
    } else {
        c = normcdff(g);
        e = __expf(-0.5f * g * g);
    }
    density = e * 0.3989422804014327f;
    return c;
}

// v *= act(g)
template <typename T> __device__ __forceinline__ void apply_act(int act, const float (&g)[8], float (&v)[8])
{
    if (act == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= g[j] * logistic(g[j]);
    } else if (act == 3) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float d;
            v[j] *= g[j] * gelu_cdf<T>(g[j], d);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= logistic(g[j]);
    }
}

template <typename T> __device__ __forceinline__ void act_and_slope(int act, const float (&g)[8], float (&a)[8], float (&da)[8])
{
    if (act == 2) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float s = logistic(g[j]);
            a[j] = g[j] * s;
            da[j] = fmaf(a[j], 1.f - s, s);
        }
    } else if (act == 3) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float d;
            const float c = gelu_cdf<T>(g[j], d);
            a[j] = g[j] * c;
            da[j] = fmaf(g[j], d, c);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            a[j] = logistic(g[j]);
            da[j] = a[j] * (1.f - a[j]);
        }
    }
}

// ------------------------------------------------------------------ chunk access

// Eight features as they lie in memory.
template <typename T, bool VEC> struct Raw {
    static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, N = kC / V;
    Pack<T, V> q[N];
    __device__ __forceinline__ void get(float (&v)[kC]) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float w[V];
            unpack(q[i], w);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i * V + j] = w[j];
        }
    }
    __device__ __forceinline__ void put(const float (&v)[kC])
    {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float w[V];
#pragma unroll
            for (int j = 0; j < V; ++j) w[j] = v[i * V + j];
            pack(q[i], w);
        }
    }
};

// Which eight features of a row a thread holds: consecutive ones (VEC) or `lanes` apart;
// features past D are absent and read as zeros.
template <typename T, bool VEC> struct Chunk {
    using R = Raw<T, VEC>;
    int c0, step, D;
    __device__ __forceinline__ Chunk(int r, int k, int lanes, int D_)
        : c0(VEC ? (k * lanes + r) * kC : r + k * kC * lanes), step(VEC ? 1 : lanes), D(D_)
    {
    }
    __device__ __forceinline__ bool has(int j) const { return VEC ? c0 < D : c0 + j * step < D; }
    // plain loads: h may be written over x
    __device__ __forceinline__ void load(const T *row, R &r) const
    {
#pragma unroll
        for (int i = 0; i < R::N; ++i) {
            r.q[i].raw = {};
            if (has(i)) r.q[i].load_rw(row + c0 + i * (VEC ? R::V : step));
        }
    }
    __device__ __forceinline__ void store(T *row, const float (&v)[kC]) const
    {
        R r;
        r.put(v);
#pragma unroll
        for (int i = 0; i < R::N; ++i)
            if (has(i)) r.q[i].store(row + c0 + i * (VEC ? R::V : step));
    }
    // through a tensor whose features lie in heads of dh, sh elements apart; with VEC the
    // chunk lies inside one head (dh is a multiple of eight) and hoff() is its offset
    __device__ __forceinline__ long long hoff(int dh, long long sh) const { return (long long)(c0 / dh) * (sh - dh); }
    __device__ __forceinline__ void load_heads(const T *tok, int dh, long long sh, long long off, R &r) const
    {
        if constexpr (VEC) {
            load(tok + off, r);
        } else {
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                const int c = c0 + j * step;
                r.q[j].raw = {};
                if (c < D) r.q[j].load_rw(tok + (long long)(c / dh) * (sh - dh) + c);
            }
        }
    }
    __device__ __forceinline__ void store_heads(T *tok, int dh, long long sh, long long off, const float (&v)[kC]) const
    {
        if constexpr (VEC) {
            store(tok + off, v);
        } else {
            R r;
            r.put(v);
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                const int c = c0 + j * step;
                if (c < D) r.q[j].store(tok + (long long)(c / dh) * (sh - dh) + c);
            }
        }
    }
    // a parameter vector (or its default)
    __device__ __forceinline__ void vec(const float *p, float none, float (&v)[kC]) const
    {
#pragma unroll
        for (int j = 0; j < kC; ++j) v[j] = none;
        if (!p) return;
        if constexpr (VEC) {
            if (c0 < D)
#pragma unroll
                for (int j = 0; j < kC; j += 4) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(p + c0 + j));
                    v[j] = w.x;
                    v[j + 1] = w.y;
                    v[j + 2] = w.z;
                    v[j + 3] = w.w;
                }
        } else {
#pragma unroll
            for (int j = 0; j < kC; ++j)
                if (has(j)) v[j] = __ldg(p + c0 + j * step);
        }
    }
};

// -------------------------------------------------------------------- reductions

// Sums over a row's group of threads.  BLOCK: over the block, through two shared slots
// used in turn (a slot is written again only after the next reduction's barrier).
template <bool BLOCK> struct Group {
    int lanes, nw, turn;
    float2 (*red)[32];
    float n;          // features held by this warp's (or group's) threads
    const float *nb;  // BLOCK: that count for every warp

    __device__ __forceinline__ float warp_sum(float v) const
    {
        for (int o = (BLOCK ? 32 : lanes) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    __device__ __forceinline__ float2 *post(float a, float b)
    {
        float2 *q = red[turn];
        if ((threadIdx.x & 31) == 0) q[threadIdx.x >> 5] = make_float2(a, b);
        __syncthreads();
        turn ^= 1;
        return q;
    }
    __device__ __forceinline__ float2 sum2(float a, float b)
    {
        a = warp_sum(a);
        b = warp_sum(b);
        if constexpr (BLOCK) {
            const float2 *q = post(a, b);
            a = b = 0.f;
            for (int i = 0; i < nw; ++i) {
                a += q[i].x;
                b += q[i].y;
            }
        }
        return make_float2(a, b);
    }
    // mean of the row and mean square about it; s: this thread's sum, dev(m): its sum of
    // squares about m
    template <typename F> __device__ __forceinline__ float2 moments(float s, int D, F dev)
    {
        float mean = warp_sum(s) / n;
        float m2 = warp_sum(dev(mean));
        if constexpr (BLOCK) {
            const float2 *q = post(mean, m2);
            mean = m2 = 0.f;
            for (int i = 0; i < nw; ++i) mean = fmaf(nb[i], q[i].x, mean);
            mean /= (float)D;
            for (int i = 0; i < nw; ++i) {
                const float d = q[i].x - mean;
                m2 += fmaf(nb[i] * d, d, q[i].y);
            }
        }
        return make_float2(mean, m2 / (float)D);
    }
};

struct GroupShared {
    float2 red[2][32];
    float nb[32];
};

template <typename T, bool VEC, int K, bool BLOCK>
__device__ __forceinline__ Group<BLOCK> make_group(GroupShared &sh, int r, int lanes, int D)
{
    int n = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const Chunk<T, VEC> c(r, k, lanes, D);
#pragma unroll
        for (int j = 0; j < kC; ++j) n += c.has(j);
    }
    Group<BLOCK> g;
    g.lanes = lanes;
    g.nw = (blockDim.x + 31) >> 5;
    g.turn = 0;
    g.red = sh.red;
    g.nb = sh.nb;
    for (int o = (BLOCK ? 32 : lanes) >> 1; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    g.n = (float)max(n, 1);  // a warp without features: mean 0 with weight 0
    if constexpr (BLOCK) {
        if ((threadIdx.x & 31) == 0) sh.nb[threadIdx.x >> 5] = (float)n;
        __syncthreads();
    }
    return g;
}

// mean and 1 / sqrt(.. + eps) of a row held as v[K][8] (absent features are zeros)
template <typename T, bool VEC, int K, bool BLOCK>
__device__ __forceinline__ float2 row_stats(Group<BLOCK> &g, int kind, float eps, const float (&v)[K][kC], int r, int D)
{
    if (kind == 1) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < kC; ++j) s = fmaf(v[k][j], v[k][j], s);
        return make_float2(0.f, rsqrtf(g.sum2(s, 0.f).x / (float)D + eps));
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < kC; ++j) s += v[k][j];
    const float2 m = g.moments(s, D, [&](float mean) {
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, g.lanes, D);
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                const float d = v[k][j] - mean;
                if (c.has(j)) q = fmaf(d, d, q);
            }
        }
        return q;
    });
    return make_float2(m.x, rsqrtf(m.y + eps));
}

// ----------------------------------------------------------------------- forward

// A row's tensors are loaded one row ahead: each register set is refilled for the next
// row as soon as this row's values are unpacked.
template <typename T, bool VEC, int K, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : 128) ttt_block_norm_fwd_kernel(const __grid_constant__ FwdParams p)
{
    __shared__ GroupShared sh;
    const int lanes = p.lanes, r = BLOCK ? threadIdx.x : threadIdx.x % lanes;
    const uint32_t per = BLOCK ? 1 : blockDim.x / lanes, mine = BLOCK ? 0 : threadIdx.x / lanes;
    Group<BLOCK> g = make_group<T, VEC, K, BLOCK>(sh, r, lanes, p.D);
    // a warp's groups leave the loop together: rows past the end are computed, not written
    const uint32_t warp_first = BLOCK ? 0 : (threadIdx.x & ~31u) / lanes;
    const T *yb = static_cast<const T *>(p.y), *xb = static_cast<const T *>(p.x), *gb = static_cast<const T *>(p.g);
    long long hoff[K];
#pragma unroll
    for (int k = 0; k < K; ++k) hoff[k] = Chunk<T, VEC>(r, k, lanes, p.D).hoff(p.dh, p.ys[1]);
    Raw<T, VEC> yr[K], xr[K], gr[K];
    uint32_t base = blockIdx.x * per;
    if (base + warp_first >= p.rows) return;
    uint32_t row = min(base + mine, p.rows - 1), b = p.byT(row), t = row - b * p.T;
    {
        const T *y = yb + b * p.ys[0] + t * p.ys[2], *gt = gb + b * p.gs[0] + t * p.gs[1], *x = xb + b * p.xs[0] + t * p.xs[1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            c.load_heads(y, p.dh, p.ys[1], hoff[k], yr[k]);
            if (p.act) c.load(gt, gr[k]);
            if (xb) c.load(x, xr[k]);
        }
    }
    while (true) {
        const bool live = base + mine < p.rows;
        const uint32_t next = base + gridDim.x * per, row0 = row;
        const bool more = next + warp_first < p.rows;
        row = min(next + mine, p.rows - 1);
        b = p.byT(row);
        t = row - b * p.T;
        float v[K][kC], w[kC], q[kC];
        const T *y = yb + b * p.ys[0] + t * p.ys[2], *gt = gb + b * p.gs[0] + t * p.gs[1], *x = xb + b * p.xs[0] + t * p.xs[1];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            yr[k].get(v[k]);
            if (more) Chunk<T, VEC>(r, k, lanes, p.D).load_heads(y, p.dh, p.ys[1], hoff[k], yr[k]);
        }
        float2 s1 = make_float2(0.f, 1.f), s2 = make_float2(0.f, 1.f);
        if (p.post) s1 = row_stats<T, VEC, K, BLOCK>(g, p.post, p.eps1, v, r, p.D);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            if (p.post) {
                c.vec(p.v.w1, 1.f, w);
                c.vec(p.v.b1, 0.f, q);
#pragma unroll
                for (int j = 0; j < kC; ++j) v[k][j] = fmaf((v[k][j] - s1.x) * s1.y, w[j], q[j]);
            }
            if (p.act) {
                gr[k].get(w);
                if (more) c.load(gt, gr[k]);
                apply_act<T>(p.act, w, v[k]);
            }
            if (p.v.sc) {
                c.vec(p.v.sc, 1.f, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) v[k][j] *= w[j];
            }
            if (xb) {
                xr[k].get(w);
                if (more) c.load(x, xr[k]);
#pragma unroll
                for (int j = 0; j < kC; ++j) v[k][j] = fmaf(p.alpha, w[j], v[k][j]);
            }
#pragma unroll
            for (int j = 0; j < kC; ++j)
                if (!c.has(j)) v[k][j] = 0.f;
            if (live) c.store(static_cast<T *>(p.h) + (size_t)row0 * p.D, v[k]);
        }
        if (p.pre) {
            // of h in fp32, before the rounding that stores it
            s2 = row_stats<T, VEC, K, BLOCK>(g, p.pre, p.eps2, v, r, p.D);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const Chunk<T, VEC> c(r, k, lanes, p.D);
                c.vec(p.v.w2, 1.f, w);
                c.vec(p.v.b2, 0.f, q);
#pragma unroll
                for (int j = 0; j < kC; ++j) v[k][j] = fmaf((v[k][j] - s2.x) * s2.y, w[j], q[j]);
                if (live) c.store(static_cast<T *>(p.u) + (size_t)row0 * p.D, v[k]);
            }
        }
        if (p.stats && live && r == 0)
            *reinterpret_cast<float4 *>(p.stats + 4 * (size_t)row0) = make_float4(s1.x, s1.y, s2.x, s2.y);
        if (!more) break;
        base = next;
    }
}

// ---------------------------------------------------------------------- backward

// Parameter gradients: every thread sums its own features over the block's rows (K = 1:
// in registers; K > 1: in shared memory), blocks write partial sums, a second kernel adds
// those in order.  The result depends on the sizes and the SM count only.
template <typename T, bool VEC, int K, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT) ttt_block_norm_bwd_kernel(const __grid_constant__ BwdParams p)
{
    __shared__ GroupShared sh;
    extern __shared__ float accs[];  // K > 1: [nvec][K][8][threads]; K = 1, not BLOCK: [threads][8]
    const int lanes = p.lanes, r = BLOCK ? threadIdx.x : threadIdx.x % lanes;
    const uint32_t per = BLOCK ? 1 : blockDim.x / lanes, mine = BLOCK ? 0 : threadIdx.x / lanes;
    Group<BLOCK> g = make_group<T, VEC, K, BLOCK>(sh, r, lanes, p.D);
    const uint32_t warp_first = BLOCK ? 0 : (threadIdx.x & ~31u) / lanes;
    float acc[K == 1 ? 5 : 1][kC];
#pragma unroll
    for (int i = 0; i < (K == 1 ? 5 : 1); ++i)
#pragma unroll
        for (int j = 0; j < kC; ++j) acc[i][j] = 0.f;
    if constexpr (K > 1)
        for (int i = threadIdx.x; i < p.nvec * K * kC * (int)blockDim.x; i += blockDim.x) accs[i] = 0.f;
    __syncthreads();
    auto add = [&](int which, int k, const float (&v)[kC]) {
        if constexpr (K == 1) {
#pragma unroll
            for (int j = 0; j < kC; ++j) acc[which][j] += v[j];
        } else if (p.slot[which] >= 0) {
#pragma unroll
            for (int j = 0; j < kC; ++j) accs[((p.slot[which] * K + k) * kC + j) * blockDim.x + threadIdx.x] += v[j];
        }
    };
    const float inv = 1.f / (float)p.D;
    const T *yb = static_cast<const T *>(p.y), *xb = static_cast<const T *>(p.x), *gb = static_cast<const T *>(p.g);
    const T *dhb = static_cast<const T *>(p.dh_in), *dub = static_cast<const T *>(p.du);
    long long hoff[K], dyoff[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        hoff[k] = Chunk<T, VEC>(r, k, lanes, p.D).hoff(p.dh, p.ys[1]);
        dyoff[k] = Chunk<T, VEC>(r, k, lanes, p.D).hoff(p.dh, (long long)p.T * p.dh);
    }
    Raw<T, VEC> yr[K], xr[K], gr[K], hr[K], ur[K];
    float4 sn;
    uint32_t base = blockIdx.x * per, row = 0, b = 0, t = 0;
    if (base + warp_first < p.rows) {
        row = min(base + mine, p.rows - 1);
        b = p.byT(row);
        t = row - b * p.T;
        sn = *reinterpret_cast<const float4 *>(p.stats + 4 * (size_t)row);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            c.load_heads(yb + b * p.ys[0] + t * p.ys[2], p.dh, p.ys[1], hoff[k], yr[k]);
            if (p.act) c.load(gb + b * p.gs[0] + t * p.gs[1], gr[k]);
            if (p.pre) {
                if (xb) c.load(xb + b * p.xs[0] + t * p.xs[1], xr[k]);
                c.load(dub + b * p.dus[0] + t * p.dus[1], ur[k]);
            }
            if (dhb) c.load(dhb + b * p.dhs[0] + t * p.dhs[1], hr[k]);
        }
    }
    for (; base + warp_first < p.rows; base += gridDim.x * per) {
        const bool live = base + mine < p.rows;
        const uint32_t row0 = row, b0 = b, t0 = t, next = base + gridDim.x * per;
        const bool more = next + warp_first < p.rows;
        const float4 st = sn;
        if (more) {
            row = min(next + mine, p.rows - 1);
            b = p.byT(row);
            t = row - b * p.T;
            sn = *reinterpret_cast<const float4 *>(p.stats + 4 * (size_t)row);
        }
        float yn[K][kC], A[K][kC], dA[K][kC], hn[K][kC], G[K][kC], pv[kC], w[kC], q[kC];
        float a = 0.f, c2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            yr[k].get(yn[k]);
            if (more) c.load_heads(yb + b * p.ys[0] + t * p.ys[2], p.dh, p.ys[1], hoff[k], yr[k]);
#pragma unroll
            for (int j = 0; j < kC; ++j) yn[k][j] = (yn[k][j] - st.x) * st.y;  // y itself without a post norm
            if (p.act) {
                gr[k].get(w);
                if (more) c.load(gb + b * p.gs[0] + t * p.gs[1], gr[k]);
                act_and_slope<T>(p.act, w, A[k], dA[k]);
            } else {
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    A[k][j] = 1.f;
                    dA[k][j] = 0.f;
                }
            }
            if (p.pre) {
                // h again from the inputs, its normalised form, and the norm's backward sums
                c.vec(p.v.w1, 1.f, w);
                c.vec(p.v.b1, 0.f, q);
#pragma unroll
                for (int j = 0; j < kC; ++j) hn[k][j] = fmaf(yn[k][j], w[j], q[j]) * A[k][j];
                if (p.v.sc) {
                    c.vec(p.v.sc, 1.f, w);
#pragma unroll
                    for (int j = 0; j < kC; ++j) hn[k][j] *= w[j];
                }
                if (xb) {
                    xr[k].get(w);
                    if (more) c.load(xb + b * p.xs[0] + t * p.xs[1], xr[k]);
#pragma unroll
                    for (int j = 0; j < kC; ++j) hn[k][j] = fmaf(p.alpha, w[j], hn[k][j]);
                }
                ur[k].get(G[k]);
                if (more) c.load(dub + b * p.dus[0] + t * p.dus[1], ur[k]);
                c.vec(p.v.w2, 1.f, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    hn[k][j] = c.has(j) ? (hn[k][j] - st.z) * st.w : 0.f;
                    q[j] = G[k][j] * hn[k][j];
                }
                if (live) {
                    add(3, k, q);
                    add(4, k, G[k]);
                }
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    G[k][j] *= w[j];
                    a += G[k][j];
                    c2 = fmaf(G[k][j], hn[k][j], c2);
                }
            }
        }
        float ma = 0.f, mc = 0.f;
        if (p.pre) {
            const float2 m = g.sum2(a, c2);
            if (p.pre == 2) ma = m.x * inv;
            mc = m.y * inv;
        }
        a = c2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
#pragma unroll
            for (int j = 0; j < kC; ++j) G[k][j] = p.pre ? st.w * (G[k][j] - ma - hn[k][j] * mc) : 0.f;
            if (dhb) {
                hr[k].get(w);
                if (more) c.load(dhb + b * p.dhs[0] + t * p.dhs[1], hr[k]);
#pragma unroll
                for (int j = 0; j < kC; ++j) G[k][j] += w[j];
            }
            if (p.dx && live) {
#pragma unroll
                for (int j = 0; j < kC; ++j) w[j] = p.alpha * G[k][j];
                c.store(static_cast<T *>(p.dx) + (size_t)row0 * p.D, w);
            }
            c.vec(p.v.w1, 1.f, w);
            c.vec(p.v.b1, 0.f, q);
#pragma unroll
            for (int j = 0; j < kC; ++j) pv[j] = fmaf(yn[k][j], w[j], q[j]);
            if (p.v.sc) {
                c.vec(p.v.sc, 1.f, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    q[j] = G[k][j] * A[k][j] * pv[j];
                    G[k][j] *= w[j];
                }
                if (live) add(2, k, q);
            }
            if (p.act) {
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    q[j] = G[k][j] * pv[j] * dA[k][j];
                    G[k][j] *= A[k][j];
                }
                if (live) c.store(static_cast<T *>(p.dg) + (size_t)row0 * p.D, q);
            }
            // G is now dp
            if (p.post) {
#pragma unroll
                for (int j = 0; j < kC; ++j) q[j] = c.has(j) ? G[k][j] * yn[k][j] : 0.f;
                if (live) {
                    add(0, k, q);
                    add(1, k, G[k]);
                }
                c.vec(p.v.w1, 1.f, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    G[k][j] = c.has(j) ? G[k][j] * w[j] : 0.f;
                    a += G[k][j];
                    c2 = fmaf(G[k][j], yn[k][j], c2);
                }
            }
        }
        ma = mc = 0.f;
        if (p.post) {
            const float2 m = g.sum2(a, c2);
            if (p.post == 2) ma = m.x * inv;
            mc = m.y * inv;
        }
        // dy is contiguous in y's own layout
        T *dy = static_cast<T *>(p.dy) + (size_t)b0 * p.T * p.D + (size_t)t0 * p.dh;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            if (p.post)
#pragma unroll
                for (int j = 0; j < kC; ++j) G[k][j] = st.y * (G[k][j] - ma - yn[k][j] * mc);
            if (live) c.store_heads(dy, p.dh, (long long)p.T * p.dh, dyoff[k], G[k]);
        }
    }
    if (p.nvec == 0) return;
    float *part = p.part + (size_t)blockIdx.x * p.nvec * p.D;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        if (p.slot[i] < 0) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            float s[kC];
            if constexpr (K > 1) {
#pragma unroll
                for (int j = 0; j < kC; ++j) s[j] = accs[((p.slot[i] * K + k) * kC + j) * blockDim.x + threadIdx.x];
            } else if constexpr (BLOCK) {
#pragma unroll
                for (int j = 0; j < kC; ++j) s[j] = acc[i][j];
            } else {
                // the block's row groups, added in order
#pragma unroll
                for (int j = 0; j < kC; ++j) accs[j * blockDim.x + threadIdx.x] = acc[i][j];
                __syncthreads();
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    s[j] = 0.f;
                    if (mine == 0)
                        for (int m = 0; m < per; ++m) s[j] += accs[j * blockDim.x + m * lanes + r];
                }
                __syncthreads();
            }
            if (mine == 0)
#pragma unroll
                for (int j = 0; j < kC; ++j)
                    if (c.has(j)) part[(size_t)p.slot[i] * p.D + c.c0 + j * c.step] = s[j];
        }
    }
}

// Adds the blocks' partial parameter gradients in a fixed order.
struct ReduceParams {
    const float *part;
    float *out[5];  // by slot
    int nblocks, nvec, D;
};

__global__ void __launch_bounds__(512) ttt_block_norm_reduce_kernel(const __grid_constant__ ReduceParams p)
{
    __shared__ float s[16][33];
    const int lane = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane, slot = blockIdx.y;
    float v = 0.f;
    if (c < p.D)
        for (int i = y; i < p.nblocks; i += 16) v += p.part[((size_t)i * p.nvec + slot) * p.D + c];
    s[y][lane] = v;
    __syncthreads();
    if (y == 0 && c < p.D) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += s[i][lane];
        p.out[slot][c] = t;
    }
}

// ------------------------------------------------------------------------ launch

// Threads of a row and chunks of a thread.  Forward: part of a warp up to 256 features, a
// warp with up to four chunks a lane up to 1024 (no barrier), then one block a row.
// Backward: its sums want few features a thread, so blocks from 256 features on.  Blocks
// hold one chunk a thread, two past 4096 features.
struct Shape {
    int lanes, threads, K;
    bool block;
};

Shape row_shape(int D, bool wide_warps)
{
    Shape s;
    s.block = D > 32 * kC * (wide_warps ? 4 : 1);
    if (s.block) {
        s.K = D > 512 * kC ? 2 : 1;
        const int need = (D + kC * s.K - 1) / (kC * s.K);
        s.lanes = s.threads = (need + 31) / 32 * 32;
    } else {
        s.K = (D + 32 * kC - 1) / (32 * kC);
        s.lanes = s.K > 1 ? 32 : 1;
        while (s.lanes * kC * s.K < D) s.lanes *= 2;
        s.threads = 128;
    }
    return s;
}

int grid_blocks(const Shape &s, long long rows, int threads_per_sm)
{
    const long long groups = s.block ? rows : (rows + s.threads / s.lanes - 1) / (s.threads / s.lanes);
    const long long fit = (long long)kSMs * (threads_per_sm / s.threads > 0 ? threads_per_sm / s.threads : 1);
    return (int)(groups < fit ? groups : fit);
}

constexpr int kBwdThreadsPerSM = 512, kFwdThreadsPerSM = 1024;

// 16-byte accesses: rows, strides and pointers in whole vectors, eight features a chunk.
bool vector_ok(int es, int D, int dh, const void *const *ptr, int np, const long long *st, int ns)
{
    const int v = 16 / es;
    if (D % kC || dh % kC) return false;
    for (int i = 0; i < np; ++i)
        if (ptr[i] && reinterpret_cast<uintptr_t>(ptr[i]) % 16) return false;
    for (int i = 0; i < ns; ++i)
        if (st[i] % v) return false;
    return true;
}

template <typename T, bool VEC>
void run_fwd(const FwdParams &p, const Shape &s, int blocks, cudaStream_t st)
{
    if (s.block) {
        if (s.K == 1) ttt_block_norm_fwd_kernel<T, VEC, 1, true><<<blocks, s.threads, 0, st>>>(p);
        else ttt_block_norm_fwd_kernel<T, VEC, 2, true><<<blocks, s.threads, 0, st>>>(p);
        return;
    }
    switch (s.K) {
    case 1: ttt_block_norm_fwd_kernel<T, VEC, 1, false><<<blocks, s.threads, 0, st>>>(p); break;
    case 2: ttt_block_norm_fwd_kernel<T, VEC, 2, false><<<blocks, s.threads, 0, st>>>(p); break;
    case 3: ttt_block_norm_fwd_kernel<T, VEC, 3, false><<<blocks, s.threads, 0, st>>>(p); break;
    default: ttt_block_norm_fwd_kernel<T, VEC, 4, false><<<blocks, s.threads, 0, st>>>(p); break;
    }
}

template <typename T, bool VEC>
int run_bwd(const BwdParams &p, const Shape &s, int blocks, cudaStream_t st)
{
    if (!s.block) {
        ttt_block_norm_bwd_kernel<T, VEC, 1, false, 128><<<blocks, s.threads, s.threads * kC * 4, st>>>(p);
    } else if (s.K == 1) {
        if (s.threads <= 256) ttt_block_norm_bwd_kernel<T, VEC, 1, true, 256><<<blocks, s.threads, 0, st>>>(p);
        else ttt_block_norm_bwd_kernel<T, VEC, 1, true, 512><<<blocks, s.threads, 0, st>>>(p);
    } else {
        const int smem = p.nvec * 2 * kC * s.threads * 4;
        if (cudaFuncSetAttribute(ttt_block_norm_bwd_kernel<T, VEC, 2, true, 512>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, 5 * 2 * kC * 512 * 4) != cudaSuccess)
            return -4;
        ttt_block_norm_bwd_kernel<T, VEC, 2, true, 512><<<blocks, s.threads, smem, st>>>(p);
    }
    return 0;
}

}  // namespace

int block_norm_bwd_blocks(int D, long long rows) { return grid_blocks(row_shape(D, false), rows, kBwdThreadsPerSM); }

int launch_block_norm_fwd(const BlockNormArgs &a)
{
    const Shape s = row_shape(a.D, true);
    FwdParams p;
    p.y = a.y;
    p.x = a.x;
    p.g = a.gate;
    p.h = a.h;
    p.u = a.u;
    p.stats = a.stats;
    p.v = {a.w1, a.b1, a.scale, a.w2, a.b2};
    for (int i = 0; i < 3; ++i) p.ys[i] = a.ys[i];
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i];
        p.gs[i] = a.gs[i];
    }
    p.rows = (uint32_t)((long long)a.B * a.T);
    p.byT = make_div(a.T > 0 ? a.T : 1);
    p.T = a.T;
    p.D = a.D;
    p.dh = a.dh;
    p.lanes = s.lanes;
    p.post = a.post;
    p.pre = a.pre;
    p.act = a.act;
    p.eps1 = a.eps1;
    p.eps2 = a.eps2;
    p.alpha = a.alpha;
    const void *ptr[] = {a.y, a.x, a.gate, a.h, a.u, a.w1, a.b1, a.scale, a.w2, a.b2};
    const long long st[] = {a.ys[0], a.ys[1], a.ys[2], a.xs[0], a.xs[1], a.gs[0], a.gs[1]};
    const int blocks = grid_blocks(s, p.rows, kFwdThreadsPerSM);
    const bool vec = vector_ok(a.bf16 ? 2 : 4, a.D, a.dh, ptr, 10, st, 7);
    if (a.bf16)
        if (vec) run_fwd<__nv_bfloat16, true>(p, s, blocks, a.stream);
        else run_fwd<__nv_bfloat16, false>(p, s, blocks, a.stream);
    else if (vec) run_fwd<float, true>(p, s, blocks, a.stream);
    else run_fwd<float, false>(p, s, blocks, a.stream);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

int launch_block_norm_bwd(const BlockNormArgs &a)
{
    const Shape s = row_shape(a.D, false);
    BwdParams p;
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
    p.v = {a.w1, a.b1, a.scale, a.w2, a.b2};
    for (int i = 0; i < 3; ++i) p.ys[i] = a.ys[i];
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i];
        p.gs[i] = a.gs[i];
        p.dhs[i] = a.dhs[i];
        p.dus[i] = a.dus[i];
    }
    p.rows = (uint32_t)((long long)a.B * a.T);
    p.byT = make_div(a.T > 0 ? a.T : 1);
    p.T = a.T;
    p.D = a.D;
    p.dh = a.dh;
    p.lanes = s.lanes;
    p.post = a.post;
    p.pre = a.pre;
    p.act = a.act;
    p.alpha = a.alpha;
    ReduceParams q = {};
    p.nvec = 0;
    for (int i = 0; i < 5; ++i) {
        p.slot[i] = a.dvec[i] ? p.nvec : -1;
        if (a.dvec[i]) q.out[p.nvec++] = a.dvec[i];
    }
    const void *ptr[] = {a.y, a.x, a.gate, a.dh_in, a.du, a.dy, a.dx, a.dgate, a.w1, a.b1, a.scale, a.w2, a.b2};
    const long long st[] = {a.ys[0],  a.ys[1],  a.ys[2],  a.xs[0],  a.xs[1], a.gs[0],
                            a.gs[1], a.dhs[0], a.dhs[1], a.dus[0], a.dus[1]};
    const int blocks = grid_blocks(s, p.rows, kBwdThreadsPerSM);
    const bool vec = vector_ok(a.bf16 ? 2 : 4, a.D, a.dh, ptr, 13, st, 11);
    int rc = 0;
    if (blocks == 0)
        ;  // no tokens: only the sums, all zero
    else if (a.bf16)
        rc = vec ? run_bwd<__nv_bfloat16, true>(p, s, blocks, a.stream) : run_bwd<__nv_bfloat16, false>(p, s, blocks, a.stream);
    else
        rc = vec ? run_bwd<float, true>(p, s, blocks, a.stream) : run_bwd<float, false>(p, s, blocks, a.stream);
    if (rc || cudaGetLastError() != cudaSuccess) return -4;
    if (p.nvec) {
        q.part = p.part;
        q.nblocks = blocks;  // 0 rows: the sums are zeros
        q.nvec = p.nvec;
        q.D = a.D;
        ttt_block_norm_reduce_kernel<<<dim3((a.D + 31) / 32, p.nvec), 512, 0, a.stream>>>(q);
        if (cudaGetLastError() != cudaSuccess) return -4;
    }
    return 0;
}

}  // namespace ttt
