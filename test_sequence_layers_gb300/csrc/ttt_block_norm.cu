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
#include "ttt_internal.h"
#include "ttt_vec.cuh"

namespace ttt {
namespace {

constexpr int kSMs = 152;
constexpr int kC = 8;  // features of a chunk

struct Vectors {  // fp32 [D], null: 1 (weights, scale) or 0 (biases)
    const float *w1, *b1, *sc, *w2, *b2;
};

struct FwdParams {
    const void *y, *x, *g;
    void *h, *u;
    float *stats;
    Vectors v;
    long long ys[3], xs[2], gs[2];
    long long rows;
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
    long long rows;
    int T, D, dh, lanes, post, pre, act;
    int slot[5];  // slot of each parameter gradient among the nvec, -1: absent
    int nvec;
    float alpha;
};

// ------------------------------------------------------------------- activations

// act(g) and its derivative: 0 none, 1 sigmoid, 2 SiLU, 3 GELU (g Phi(g)).
__device__ __forceinline__ float act_value(int act, float g)
{
    if (act == 0) return 1.f;
    if (act == 3) return g * normcdff(g);
    const float s = 1.f / (1.f + __expf(-g));
    return act == 1 ? s : g * s;
}

__device__ __forceinline__ float act_value(int act, float g, float &deriv)
{
    if (act == 0) {
        deriv = 0.f;
        return 1.f;
    }
    if (act == 3) {
        const float c = normcdff(g);
        deriv = fmaf(g * 0.3989422804014327f, __expf(-0.5f * g * g), c);
        return g * c;
    }
    const float s = 1.f / (1.f + __expf(-g));
    if (act == 1) {
        deriv = s * (1.f - s);
        return s;
    }
    deriv = s * fmaf(g, 1.f - s, 1.f);
    return g * s;
}

// ------------------------------------------------------------------ chunk access

// Eight features of a row: consecutive (VEC) or `lanes` apart, features past D absent.
template <typename T, bool VEC> struct Chunk {
    int c0, step, D;
    __device__ __forceinline__ Chunk(int r, int k, int lanes, int D_)
        : c0(VEC ? (k * lanes + r) * kC : r + k * kC * lanes), step(VEC ? 1 : lanes), D(D_)
    {
    }
    __device__ __forceinline__ bool has(int j) const { return VEC ? c0 < D : c0 + j * step < D; }
    // RW: the tensor may also be an output (h written over x)
    template <bool RW = false> __device__ __forceinline__ void load(const T *row, float (&v)[kC]) const
    {
        if constexpr (VEC) {
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int i = 0; i < kC; i += V) {
                float w[V] = {};
                if (c0 < D) {
                    Pack<T, V> q;
                    if (RW) q.load_rw(row + c0 + i);
                    else q.load(row + c0 + i);
                    unpack(q, w);
                }
#pragma unroll
                for (int j = 0; j < V; ++j) v[i + j] = w[j];
            }
        } else {
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                float w[1] = {};
                if (has(j)) {
                    Pack<T, 1> q;
                    if (RW) q.load_rw(row + c0 + j * step);
                    else q.load(row + c0 + j * step);
                    unpack(q, w);
                }
                v[j] = w[0];
            }
        }
    }
    __device__ __forceinline__ void store(T *row, const float (&v)[kC]) const
    {
        if constexpr (VEC) {
            constexpr int V = 16 / sizeof(T);
            if (c0 < D)
#pragma unroll
                for (int i = 0; i < kC; i += V) {
                    float w[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) w[j] = v[i + j];
                    Pack<T, V> q;
                    pack(q, w);
                    q.store(row + c0 + i);
                }
        } else {
#pragma unroll
            for (int j = 0; j < kC; ++j)
                if (has(j)) {
                    const float w[1] = {v[j]};
                    Pack<T, 1> q;
                    pack(q, w);
                    q.store(row + c0 + j * step);
                }
        }
    }
    // the same through a tensor whose features lie in heads of dh, sh elements apart
    __device__ __forceinline__ void load_heads(const T *tok, int dh, long long sh, float (&v)[kC]) const
    {
        if constexpr (VEC) {
            // the chunk lies inside one head (dh is a multiple of eight)
            load(tok + (long long)(c0 / dh) * (sh - dh), v);
        } else {
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                const int c = c0 + j * step;
                float w[1] = {};
                if (c < D) {
                    Pack<T, 1> q;
                    q.load(tok + (long long)(c / dh) * (sh - dh) + c);
                    unpack(q, w);
                }
                v[j] = w[0];
            }
        }
    }
    __device__ __forceinline__ void store_heads(T *tok, int dh, long long sh, const float (&v)[kC]) const
    {
        if constexpr (VEC) {
            store(tok + (long long)(c0 / dh) * (sh - dh), v);
        } else {
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                const int c = c0 + j * step;
                if (c < D) {
                    const float w[1] = {v[j]};
                    Pack<T, 1> q;
                    pack(q, w);
                    q.store(tok + (long long)(c / dh) * (sh - dh) + c);
                }
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

template <typename T, bool VEC, int K, bool BLOCK>
__global__ void __launch_bounds__(512) ttt_block_norm_fwd_kernel(const __grid_constant__ FwdParams p)
{
    __shared__ GroupShared sh;
    const int lanes = p.lanes, r = BLOCK ? threadIdx.x : threadIdx.x % lanes;
    const int per = BLOCK ? 1 : blockDim.x / lanes, mine = BLOCK ? 0 : threadIdx.x / lanes;
    Group<BLOCK> g = make_group<T, VEC, K, BLOCK>(sh, r, lanes, p.D);
    // a warp's groups leave the loop together: rows past the end are computed, not written
    const int warp_first = BLOCK ? 0 : (threadIdx.x & ~31) / lanes;
    for (long long base = (long long)blockIdx.x * per; base + warp_first < p.rows; base += (long long)gridDim.x * per) {
        const bool live = base + mine < p.rows;
        const long long row = live ? base + mine : p.rows - 1;
        const long long b = row / p.T, t = row % p.T;
        const T *y = static_cast<const T *>(p.y) + b * p.ys[0] + t * p.ys[2];
        const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + t * p.xs[1];
        const T *gt = static_cast<const T *>(p.g) + b * p.gs[0] + t * p.gs[1];
        float v[K][kC], w[kC], q[kC];
#pragma unroll
        for (int k = 0; k < K; ++k) Chunk<T, VEC>(r, k, lanes, p.D).load_heads(y, p.dh, p.ys[1], v[k]);
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
                c.load(gt, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) v[k][j] *= act_value(p.act, w[j]);
            }
            if (p.v.sc) {
                c.vec(p.v.sc, 1.f, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) v[k][j] *= w[j];
            }
            if (p.x) {
                c.template load<true>(x, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) v[k][j] = fmaf(p.alpha, w[j], v[k][j]);
            }
#pragma unroll
            for (int j = 0; j < kC; ++j)
                if (!c.has(j)) v[k][j] = 0.f;
            if (live) c.store(static_cast<T *>(p.h) + row * p.D, v[k]);
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
                if (live) c.store(static_cast<T *>(p.u) + row * p.D, v[k]);
            }
        }
        if (p.stats && live && r == 0)
            *reinterpret_cast<float4 *>(p.stats + 4 * row) = make_float4(s1.x, s1.y, s2.x, s2.y);
    }
}

// ---------------------------------------------------------------------- backward

// Parameter gradients: every thread sums its own features over the block's rows (K = 1:
// in registers; K > 1: in shared memory), blocks write partial sums, a second kernel adds
// those in order.  The result depends on the sizes and the SM count only.
template <typename T, bool VEC, int K, bool BLOCK>
__global__ void __launch_bounds__(512) ttt_block_norm_bwd_kernel(const __grid_constant__ BwdParams p)
{
    __shared__ GroupShared sh;
    extern __shared__ float accs[];  // K > 1: [nvec][K][8][threads]; K = 1, not BLOCK: [threads][8]
    const int lanes = p.lanes, r = BLOCK ? threadIdx.x : threadIdx.x % lanes;
    const int per = BLOCK ? 1 : blockDim.x / lanes, mine = BLOCK ? 0 : threadIdx.x / lanes;
    Group<BLOCK> g = make_group<T, VEC, K, BLOCK>(sh, r, lanes, p.D);
    const int warp_first = BLOCK ? 0 : (threadIdx.x & ~31) / lanes;
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
    for (long long base = (long long)blockIdx.x * per; base + warp_first < p.rows; base += (long long)gridDim.x * per) {
        const bool live = base + mine < p.rows;
        const long long row = live ? base + mine : p.rows - 1;
        const long long b = row / p.T, t = row % p.T;
        const T *y = static_cast<const T *>(p.y) + b * p.ys[0] + t * p.ys[2];
        const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + t * p.xs[1];
        const T *gt = static_cast<const T *>(p.g) + b * p.gs[0] + t * p.gs[1];
        const T *dhp = static_cast<const T *>(p.dh_in) + b * p.dhs[0] + t * p.dhs[1];
        const T *dup = static_cast<const T *>(p.du) + b * p.dus[0] + t * p.dus[1];
        const float4 st = *reinterpret_cast<const float4 *>(p.stats + 4 * row);
        float yn[K][kC], G[K][kC], w[kC], q[kC];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            Chunk<T, VEC>(r, k, lanes, p.D).load_heads(y, p.dh, p.ys[1], yn[k]);
#pragma unroll
            for (int j = 0; j < kC; ++j) yn[k][j] = (yn[k][j] - st.x) * st.y;  // y itself without a post norm
        }
        if (p.pre) {
            // h again from the inputs, its normalised form, and the norm's backward sums
            float hn[K][kC], a = 0.f, c2 = 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const Chunk<T, VEC> c(r, k, lanes, p.D);
                if (p.post) {
                    c.vec(p.v.w1, 1.f, w);
                    c.vec(p.v.b1, 0.f, q);
#pragma unroll
                    for (int j = 0; j < kC; ++j) hn[k][j] = fmaf(yn[k][j], w[j], q[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < kC; ++j) hn[k][j] = yn[k][j];
                }
                if (p.act) {
                    c.load(gt, w);
#pragma unroll
                    for (int j = 0; j < kC; ++j) hn[k][j] *= act_value(p.act, w[j]);
                }
                if (p.v.sc) {
                    c.vec(p.v.sc, 1.f, w);
#pragma unroll
                    for (int j = 0; j < kC; ++j) hn[k][j] *= w[j];
                }
                if (p.x) {
                    c.load(x, w);
#pragma unroll
                    for (int j = 0; j < kC; ++j) hn[k][j] = fmaf(p.alpha, w[j], hn[k][j]);
                }
                c.load(dup, G[k]);
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
            const float2 m = g.sum2(a, c2);
            const float ma = p.pre == 2 ? m.x * inv : 0.f, mc = m.y * inv;
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < kC; ++j) G[k][j] = st.w * (G[k][j] - ma - hn[k][j] * mc);
        } else {
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int j = 0; j < kC; ++j) G[k][j] = 0.f;
        }
        float a = 0.f, c2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            if (p.dh_in) {
                c.load(dhp, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) G[k][j] += w[j];
            }
            if (p.dx && live) {
#pragma unroll
                for (int j = 0; j < kC; ++j) w[j] = p.alpha * G[k][j];
                c.store(static_cast<T *>(p.dx) + row * p.D, w);
            }
            float pv[kC];
            if (p.post) {
                c.vec(p.v.w1, 1.f, w);
                c.vec(p.v.b1, 0.f, q);
#pragma unroll
                for (int j = 0; j < kC; ++j) pv[j] = fmaf(yn[k][j], w[j], q[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kC; ++j) pv[j] = yn[k][j];
            }
            if (p.act) {
                float A[kC], dA[kC];
                c.load(gt, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) A[j] = act_value(p.act, w[j], dA[j]);
                if (p.v.sc) {
                    c.vec(p.v.sc, 1.f, w);
#pragma unroll
                    for (int j = 0; j < kC; ++j) {
                        q[j] = G[k][j] * A[j] * pv[j];
                        G[k][j] *= w[j];
                    }
                    if (live) add(2, k, q);
                }
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    q[j] = G[k][j] * pv[j] * dA[j];
                    G[k][j] *= A[j];
                }
                if (live) c.store(static_cast<T *>(p.dg) + row * p.D, q);
            } else if (p.v.sc) {
                c.vec(p.v.sc, 1.f, w);
#pragma unroll
                for (int j = 0; j < kC; ++j) {
                    q[j] = G[k][j] * pv[j];
                    G[k][j] *= w[j];
                }
                if (live) add(2, k, q);
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
        float ma = 0.f, mc = 0.f;
        if (p.post) {
            const float2 m = g.sum2(a, c2);
            if (p.post == 2) ma = m.x * inv;
            mc = m.y * inv;
        }
        const long long drow = b * (long long)p.T * p.D;  // dy is contiguous in y's own layout
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, lanes, p.D);
            if (p.post)
#pragma unroll
                for (int j = 0; j < kC; ++j) G[k][j] = st.y * (G[k][j] - ma - yn[k][j] * mc);
            if (live) c.store_heads(static_cast<T *>(p.dy) + drow + t * p.dh, p.dh, (long long)p.T * p.dh, G[k]);
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

// Threads of a row and chunks of a thread: part of a warp up to 256 features, then one
// block a row, eight features a thread, sixteen past 4096.
struct Shape {
    int lanes, threads, K;
    bool block;
};

Shape row_shape(int D)
{
    Shape s;
    s.block = D > 32 * kC;
    s.K = D > 512 * kC ? 2 : 1;
    if (s.block) {
        const int need = (D + kC * s.K - 1) / (kC * s.K);
        s.lanes = s.threads = (need + 31) / 32 * 32;
    } else {
        s.lanes = 1;
        while (s.lanes * kC < D) s.lanes *= 2;
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
    if (!s.block) ttt_block_norm_fwd_kernel<T, VEC, 1, false><<<blocks, s.threads, 0, st>>>(p);
    else if (s.K == 1) ttt_block_norm_fwd_kernel<T, VEC, 1, true><<<blocks, s.threads, 0, st>>>(p);
    else ttt_block_norm_fwd_kernel<T, VEC, 2, true><<<blocks, s.threads, 0, st>>>(p);
}

template <typename T, bool VEC>
int run_bwd(const BwdParams &p, const Shape &s, int blocks, cudaStream_t st)
{
    if (!s.block) {
        ttt_block_norm_bwd_kernel<T, VEC, 1, false><<<blocks, s.threads, s.threads * kC * 4, st>>>(p);
    } else if (s.K == 1) {
        ttt_block_norm_bwd_kernel<T, VEC, 1, true><<<blocks, s.threads, 0, st>>>(p);
    } else {
        const int smem = p.nvec * 2 * kC * s.threads * 4;
        if (cudaFuncSetAttribute(ttt_block_norm_bwd_kernel<T, VEC, 2, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 5 * 2 * kC * 512 * 4) != cudaSuccess)
            return -4;
        ttt_block_norm_bwd_kernel<T, VEC, 2, true><<<blocks, s.threads, smem, st>>>(p);
    }
    return 0;
}

}  // namespace

int block_norm_bwd_blocks(int D, long long rows) { return grid_blocks(row_shape(D), rows, kBwdThreadsPerSM); }

int launch_block_norm_fwd(const BlockNormArgs &a)
{
    const Shape s = row_shape(a.D);
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
    p.rows = (long long)a.B * a.T;
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
    const Shape s = row_shape(a.D);
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
    p.rows = (long long)a.B * a.T;
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
