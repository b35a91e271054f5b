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

// Eight features as four pairs: the arithmetic is on paired fp32 instructions, which
// halves what these kernels are short of, issue slots.
constexpr int kP = kC / 2;
struct V8 {
    float2 p[kP];
};
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ V8 splat(float v)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kP; ++i) r.p[i] = both(v);
    return r;
}
__device__ __forceinline__ V8 mul(const V8 &a, const V8 &b)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kP; ++i) r.p[i] = __fmul2_rn(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ V8 mul(const V8 &a, float b)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kP; ++i) r.p[i] = __fmul2_rn(a.p[i], both(b));
    return r;
}
__device__ __forceinline__ V8 add(const V8 &a, const V8 &b)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kP; ++i) r.p[i] = __fadd2_rn(a.p[i], b.p[i]);
    return r;
}
__device__ __forceinline__ V8 fma(const V8 &a, const V8 &b, const V8 &c)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kP; ++i) r.p[i] = __ffma2_rn(a.p[i], b.p[i], c.p[i]);
    return r;
}
__device__ __forceinline__ V8 fma(const V8 &a, float b, const V8 &c)
{
    V8 r;
#pragma unroll
    for (int i = 0; i < kP; ++i) r.p[i] = __ffma2_rn(a.p[i], both(b), c.p[i]);
    return r;
}
// (a - m) r: the difference first, so that what it cancels does not come back scaled
__device__ __forceinline__ V8 centre(const V8 &a, float m, float r)
{
    V8 v;
#pragma unroll
    for (int i = 0; i < kP; ++i) v.p[i] = __fmul2_rn(__fadd2_rn(a.p[i], both(-m)), both(r));
    return v;
}
__device__ __forceinline__ float total(const V8 &a)
{
    const float2 s = __fadd2_rn(__fadd2_rn(a.p[0], a.p[1]), __fadd2_rn(a.p[2], a.p[3]));
    return s.x + s.y;
}
__device__ __forceinline__ float dot(const V8 &a, const V8 &b)
{
    float2 s = __fmul2_rn(a.p[0], b.p[0]);
#pragma unroll
    for (int i = 1; i < kP; ++i) s = __ffma2_rn(a.p[i], b.p[i], s);
    return s.x + s.y;
}

// ------------------------------------------------------------------- activations

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 1 / (1 + exp(-g)); 0 and 1 where exp(-g) leaves the range
__device__ __forceinline__ float2 logistic(float2 g)
{
    const float2 t = __fmul2_rn(g, both(-1.4426950408889634f));
    const float2 d = __fadd2_rn(make_float2(exp2_approx(t.x), exp2_approx(t.y)), both(1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}

// Phi(g) and the normal density.  For bf16 tensors Phi is 1 - w or w with w =
// poly(1 / (1 + 0.3275911 |g| / sqrt 2)) exp(-g^2 / 2) / 2 (Abramowitz & Stegun 7.1.26, error
// below 1e-7, far below the output's rounding; the exponential is the density's too); for
// fp32 tensors CUDA's normcdff.
template <typename T> __device__ __forceinline__ float2 gelu_cdf(float2 g, float2 &density)
{
    if constexpr (sizeof(T) == 2) {
        const float2 m = make_float2(fabsf(g.x), fabsf(g.y));
        const float2 d = __ffma2_rn(m, both(0.3275911f * 0.70710678118654752f), both(1.f));
        const float2 t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        const float2 q = __fmul2_rn(__fmul2_rn(g, g), both(-0.5f * 1.4426950408889634f));
        const float2 e = make_float2(exp2_approx(q.x), exp2_approx(q.y));
        float2 w = __ffma2_rn(t, both(0.5f * 1.061405429f), both(-0.5f * 1.453152027f));
        w = __ffma2_rn(t, w, both(0.5f * 1.421413741f));
        w = __ffma2_rn(t, w, both(-0.5f * 0.284496736f));
        w = __ffma2_rn(t, w, both(0.5f * 0.254829592f));
        w = __fmul2_rn(__fmul2_rn(t, w), e);
        density = __fmul2_rn(e, both(0.3989422804014327f));
        const float2 h = __ffma2_rn(w, both(-1.f), both(0.5f));
        return __fadd2_rn(make_float2(copysignf(h.x, g.x), copysignf(h.y, g.y)), both(0.5f));
    } else {
        density = make_float2(expf(-0.5f * g.x * g.x) * 0.3989422804014327f, expf(-0.5f * g.y * g.y) * 0.3989422804014327f);
        return make_float2(normcdff(g.x), normcdff(g.y));
    }
}

// act(g): 1 sigmoid, 2 SiLU, 3 GELU (g Phi(g))
template <typename T> __device__ __forceinline__ V8 act_value(int act, const V8 &g)
{
    V8 r;
    if (act == 2) {
#pragma unroll
        for (int i = 0; i < kP; ++i) r.p[i] = __fmul2_rn(g.p[i], logistic(g.p[i]));
    } else if (act == 3) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            float2 d;
            r.p[i] = __fmul2_rn(g.p[i], gelu_cdf<T>(g.p[i], d));
        }
    } else {
#pragma unroll
        for (int i = 0; i < kP; ++i) r.p[i] = logistic(g.p[i]);
    }
    return r;
}

// act(g) and its derivative
template <typename T> __device__ __forceinline__ void act_and_slope(int act, const V8 &g, V8 &a, V8 &da)
{
    if (act == 2) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const float2 s = logistic(g.p[i]);
            a.p[i] = __fmul2_rn(g.p[i], s);
            da.p[i] = __ffma2_rn(a.p[i], __ffma2_rn(s, both(-1.f), both(1.f)), s);
        }
    } else if (act == 3) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            float2 d;
            const float2 c = gelu_cdf<T>(g.p[i], d);
            a.p[i] = __fmul2_rn(g.p[i], c);
            da.p[i] = __ffma2_rn(g.p[i], d, c);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            a.p[i] = logistic(g.p[i]);
            da.p[i] = __fmul2_rn(a.p[i], __ffma2_rn(a.p[i], both(-1.f), both(1.f)));
        }
    }
}

// ------------------------------------------------------------------ chunk access

// Eight features in the I/O type, for storing.
template <typename T, bool VEC> struct Raw {
    static constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, N = kC / V;
    Pack<T, V> q[N];
    __device__ __forceinline__ void put(const V8 &r)
    {
        const float *v = &r.p[0].x;
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
//
// A row comes through shared memory: fetch() starts copies of the thread's own eight
// features, get() reads them back once they have landed.  Only the thread itself reads
// what it copied, so there is no barrier, and no load waits in a register.  slot: the
// thread's place in a stage, 16-byte units `pitch` apart.  Where the copies do not go
// (DIRECT: bf16 rows that are not 16-byte aligned, as copies are 4 bytes at least, and
// widths whose sums leave no room for stages) the slot holds the row's address and get()
// loads.
template <typename T, bool VEC, bool DIRECT = (!VEC && sizeof(T) == 2)> struct Chunk {
    using R = Raw<T, VEC>;
    static constexpr int kUnits = DIRECT ? 1 : kC * (int)sizeof(T) / 16;  // 16-byte units of a chunk
    // rows in flight or landed: enough to cover the latency, few enough to leave room for
    // the blocks of an SM
    static constexpr int kAhead = DIRECT ? 1 : sizeof(T) == 2 ? 3 : 2;
    int c0, step, D;
    __device__ __forceinline__ Chunk(int r, int k, int lanes, int D_)
        : c0(VEC ? (k * lanes + r) * kC : r + k * kC * lanes), step(VEC ? 1 : lanes), D(D_)
    {
    }
    __device__ __forceinline__ bool has(int j) const { return VEC ? c0 < D : c0 + j * step < D; }
    // zeros in the absent features
    __device__ __forceinline__ void mask(V8 &v) const
    {
        float *f = &v.p[0].x;
#pragma unroll
        for (int j = 0; j < kC; ++j) f[j] = has(j) ? f[j] : 0.f;
    }
    // row: the token's first feature; dh, sh: features of a head and elements from one head
    // to the next (dh = D: no heads).  With VEC a chunk lies inside one head and off =
    // hoff() is what its head adds.
    __device__ __forceinline__ long long hoff(int dh, long long sh) const { return (long long)(c0 / dh) * (sh - dh); }
    __device__ __forceinline__ void fetch(const T *row, int dh, long long sh, long long off, uint4 *slot, int pitch) const
    {
        if constexpr (DIRECT) {
            *reinterpret_cast<const T **>(slot) = row;
        } else if constexpr (VEC) {
            if (c0 < D)
#pragma unroll
                for (int i = 0; i < kUnits; ++i) copy_async16(slot + i * pitch, row + off + c0 + i * (16 / (int)sizeof(T)));
        } else {
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                const int c = c0 + j * step;
                if (c < D)
                    copy_async4(reinterpret_cast<float *>(slot + j / 4 * pitch) + j % 4,
                                row + (dh < D ? (long long)(c / dh) * (sh - dh) : 0) + c);
            }
        }
    }
    __device__ __forceinline__ V8 get(const uint4 *slot, int pitch, int dh, long long sh, long long off) const
    {
        constexpr int V = 16 / (int)sizeof(T);
        V8 r = {};
        float *v = &r.p[0].x;
        if constexpr (!DIRECT || VEC) {
            const T *row = DIRECT ? *reinterpret_cast<const T *const *>(slot) + off + c0 : nullptr;
#pragma unroll
            for (int i = 0; i < kC / V; ++i) {
                Pack<T, V> q;
                if constexpr (DIRECT) {
                    q.raw = {};
                    if (c0 < D) q.load_rw(row + i * V);
                } else {
                    q.raw = slot[i * pitch];
                }
                float w[V];
                unpack(q, w);
#pragma unroll
                for (int j = 0; j < V; ++j) v[i * V + j] = w[j];
            }
            if (!DIRECT && (!VEC || c0 >= D)) mask(r);  // nothing was copied there
        } else {
            const T *row = *reinterpret_cast<const T *const *>(slot);
#pragma unroll
            for (int j = 0; j < kC; ++j) {
                const int c = c0 + j * step;
                if (c < D) {
                    Pack<T, 1> q;
                    float w[1];
                    q.load_rw(row + (dh < D ? (long long)(c / dh) * (sh - dh) : 0) + c);
                    unpack(q, w);
                    v[j] = w[0];
                }
            }
        }
        return r;
    }
    __device__ __forceinline__ void store(T *row, const V8 &v) const
    {
        R r;
        r.put(v);
#pragma unroll
        for (int i = 0; i < R::N; ++i)
            if (has(i)) r.q[i].store(row + c0 + i * (VEC ? R::V : step));
    }
    __device__ __forceinline__ void store_heads(T *tok, int dh, long long sh, long long off, const V8 &v) const
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
    // a parameter vector
    __device__ __forceinline__ V8 vec(const float *p) const
    {
        V8 r = {};
        if constexpr (VEC) {
            if (c0 < D)
#pragma unroll
                for (int j = 0; j < kP; j += 2) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(p + c0 + 2 * j));
                    r.p[j] = make_float2(w.x, w.y);
                    r.p[j + 1] = make_float2(w.z, w.w);
                }
        } else {
            float *v = &r.p[0].x;
#pragma unroll
            for (int j = 0; j < kC; ++j)
                if (has(j)) v[j] = __ldg(p + c0 + j * step);
        }
        return r;
    }
    // v w + b with parameter vectors that may be absent
    __device__ __forceinline__ V8 scale_shift(const V8 &v, const float *w, const float *b) const
    {
        if (w && b) return fma(v, vec(w), vec(b));
        if (w) return mul(v, vec(w));
        return b ? add(v, vec(b)) : v;
    }
};

// -------------------------------------------------------------------- reductions

// Sums over a row's group of threads.  BLOCK: over the block, through two shared slots
// used in turn (a slot is written again only after the next reduction's barrier).
template <bool BLOCK> struct Group {
    int lanes, half_nw, turn;
    float4 (*red)[16];  // pairs of two warps

    __device__ __forceinline__ float warp_sum(float v) const
    {
        for (int o = (BLOCK ? 32 : lanes) >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    __device__ __forceinline__ float2 sum2(float a, float b)
    {
        a = warp_sum(a);
        b = warp_sum(b);
        float2 s = make_float2(a, b);
        if constexpr (BLOCK) {
            float4 *q = red[turn];
            if ((threadIdx.x & 31) == 0) reinterpret_cast<float2 *>(q)[threadIdx.x >> 5] = s;
            __syncthreads();
            turn ^= 1;
            s = make_float2(0.f, 0.f);
#pragma unroll 4
            for (int i = 0; i < half_nw; ++i) {
                const float4 w = q[i];
                s = __fadd2_rn(s, __fadd2_rn(make_float2(w.x, w.y), make_float2(w.z, w.w)));
            }
        }
        return s;
    }
    __device__ __forceinline__ float sum1(float a)
    {
        a = warp_sum(a);
        if constexpr (BLOCK) {
            float2 *q = reinterpret_cast<float2 *>(red[turn]);  // one number a warp
            if ((threadIdx.x & 31) == 0) reinterpret_cast<float *>(q)[threadIdx.x >> 5] = a;
            __syncthreads();
            turn ^= 1;
            a = 0.f;
#pragma unroll 4
            for (int i = 0; i < half_nw; ++i) a += q[i].x + q[i].y;
        }
        return a;
    }
};

struct GroupShared {
    float4 red[2][16];
};

template <bool BLOCK> __device__ __forceinline__ Group<BLOCK> make_group(GroupShared &sh, int lanes)
{
    Group<BLOCK> g;
    g.lanes = lanes;
    g.turn = 0;
    g.red = sh.red;
    g.half_nw = ((int)((blockDim.x + 31) >> 5) + 1) >> 1;
    if constexpr (BLOCK) {  // an odd number of warps: the missing one's slot stays zero
        for (int i = threadIdx.x; i < 32; i += blockDim.x) (&sh.red[0][0])[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        __syncthreads();
    }
    return g;
}

// mean and 1 / sqrt(.. + eps) of a row held as v[K] (absent features are zeros)
template <typename T, bool VEC, int K, bool BLOCK>
__device__ __forceinline__ float2 row_stats(Group<BLOCK> &g, int kind, float eps, float inv, const V8 (&v)[K], int r, int D)
{
    float mean = 0.f, s = 0.f;
    if (kind == 2) {
#pragma unroll
        for (int k = 0; k < K; ++k) s += total(v[k]);
        mean = g.sum1(s) * inv;
        s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, VEC> c(r, k, g.lanes, D);
            V8 d = add(v[k], splat(-mean));
            if constexpr (!VEC) c.mask(d);
            const float q = dot(d, d);
            s += !VEC || c.has(0) ? q : 0.f;
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) s += dot(v[k], v[k]);
    }
    return make_float2(mean, rsqrtf(g.sum1(s) * inv + eps));
}

// ----------------------------------------------------------------------- forward

// The rows' tensors are copied kAhead rows ahead into the thread's ring of stages.
template <typename T, bool VEC, int K, bool BLOCK>
__global__ void __launch_bounds__(BLOCK ? 512 : 128) ttt_block_norm_fwd_kernel(const __grid_constant__ FwdParams p)
{
    using C = Chunk<T, VEC>;
    constexpr int kAhead = C::kAhead;
    __shared__ GroupShared sh;
    extern __shared__ uint4 stages[];  // [kAhead][3][K][units][threads]
    const int lanes = p.lanes, r = BLOCK ? threadIdx.x : threadIdx.x % lanes, pitch = blockDim.x;
    const uint32_t per = BLOCK ? 1 : blockDim.x / lanes, mine = BLOCK ? 0 : threadIdx.x / lanes;
    Group<BLOCK> g = make_group<BLOCK>(sh, lanes);
    // a warp's groups leave the loop together: rows past the end are computed, not written
    const uint32_t warp_first = BLOCK ? 0 : (threadIdx.x & ~31u) / lanes;
    const T *yb = static_cast<const T *>(p.y), *xb = static_cast<const T *>(p.x), *gb = static_cast<const T *>(p.g);
    const float inv = 1.f / (float)p.D;
    const uint32_t stride = gridDim.x * per;
    long long hoff[K];
#pragma unroll
    for (int k = 0; k < K; ++k) hoff[k] = C(r, k, lanes, p.D).hoff(p.dh, p.ys[1]);
    auto slot = [&](int stage, int tensor, int k) {
        return stages + ((stage * 3 + tensor) * K + k) * C::kUnits * pitch + threadIdx.x;
    };
    auto fetch = [&](uint32_t base, int stage) {
        if (base + warp_first < p.rows) {
            const uint32_t row = min(base + mine, p.rows - 1), b = p.byT(row), t = row - b * p.T;
            const T *y = yb + b * p.ys[0] + t * p.ys[2];
            const T *gt = gb + b * p.gs[0] + t * p.gs[1], *x = xb + b * p.xs[0] + t * p.xs[1];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const C c(r, k, lanes, p.D);
                c.fetch(y, p.dh, p.ys[1], hoff[k], slot(stage, 0, k), pitch);
                if (p.act) c.fetch(gt, p.D, 0, 0, slot(stage, 1, k), pitch);
                if (xb) c.fetch(x, p.D, 0, 0, slot(stage, 2, k), pitch);
            }
        }
        copy_commit();
    };
    uint32_t base = blockIdx.x * per;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(base + i * stride, i);
    for (int stage = 0; base + warp_first < p.rows; base += stride, stage = stage + 1 == kAhead ? 0 : stage + 1) {
        const bool live = base + mine < p.rows;
        const uint32_t row = min(base + mine, p.rows - 1);
        copy_wait<kAhead - 1>();
        V8 v[K];
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = C(r, k, lanes, p.D).get(slot(stage, 0, k), pitch, p.dh, p.ys[1], hoff[k]);
        float2 s1 = make_float2(0.f, 1.f), s2 = make_float2(0.f, 1.f);
        if (p.post) s1 = row_stats<T, VEC, K, BLOCK>(g, p.post, p.eps1, inv, v, r, p.D);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D);
            if (p.post) v[k] = c.scale_shift(centre(v[k], s1.x, s1.y), p.v.w1, p.v.b1);
            if (p.act) v[k] = mul(v[k], act_value<T>(p.act, c.get(slot(stage, 1, k), pitch, p.D, 0, 0)));
            if (p.v.sc) v[k] = mul(v[k], c.vec(p.v.sc));
            if (xb) v[k] = fma(c.get(slot(stage, 2, k), pitch, p.D, 0, 0), p.alpha, v[k]);
            if (live) c.store(static_cast<T *>(p.h) + (size_t)row * p.D, v[k]);
            if (!VEC || !c.has(0)) c.mask(v[k]);
        }
        fetch(base + kAhead * stride, stage);
        if (p.pre) {
            // of h in fp32, before the rounding that stores it
            s2 = row_stats<T, VEC, K, BLOCK>(g, p.pre, p.eps2, inv, v, r, p.D);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const C c(r, k, lanes, p.D);
                v[k] = c.scale_shift(centre(v[k], s2.x, s2.y), p.v.w2, p.v.b2);
                if (live) c.store(static_cast<T *>(p.u) + (size_t)row * p.D, v[k]);
            }
        }
        if (p.stats && live && r == 0)
            *reinterpret_cast<float4 *>(p.stats + 4 * (size_t)row) = make_float4(s1.x, s1.y, s2.x, s2.y);
    }
}

// ---------------------------------------------------------------------- backward

// Parameter gradients: every thread sums its own features over the block's rows (K = 1:
// in registers; K > 1: in shared memory), blocks write partial sums, a second kernel adds
// those in order.  The result depends on the sizes and the SM count only.
template <typename T, bool VEC, int K, bool BLOCK, int MAXT>
__global__ void __launch_bounds__(MAXT, 512 / MAXT) ttt_block_norm_bwd_kernel(const __grid_constant__ BwdParams p)
{
    __shared__ GroupShared sh;
    constexpr bool DIRECT = K > 1 || (!VEC && sizeof(T) == 2);
    using C = Chunk<T, VEC, DIRECT>;
    constexpr int kAhead = C::kAhead;
    extern __shared__ uint4 stages[];  // [kAhead][5 units + 1][threads], then the sums:
    // K > 1: [nvec][K][4][threads]; K = 1, not BLOCK: [4][threads]
    constexpr int kStage = 5 * C::kUnits + 1;
    float2 *accs = reinterpret_cast<float2 *>(stages + kAhead * kStage * blockDim.x);
    const int lanes = p.lanes, r = BLOCK ? threadIdx.x : threadIdx.x % lanes, pitch = blockDim.x;
    const uint32_t per = BLOCK ? 1 : blockDim.x / lanes, mine = BLOCK ? 0 : threadIdx.x / lanes;
    Group<BLOCK> g = make_group<BLOCK>(sh, lanes);
    const uint32_t warp_first = BLOCK ? 0 : (threadIdx.x & ~31u) / lanes;
    V8 acc[K == 1 ? 5 : 1];
#pragma unroll
    for (int i = 0; i < (K == 1 ? 5 : 1); ++i) acc[i] = splat(0.f);
    if constexpr (K > 1) {
        for (int i = threadIdx.x; i < p.nvec * K * kP * (int)blockDim.x; i += blockDim.x) accs[i] = make_float2(0.f, 0.f);
        __syncthreads();
    }
    // += a b
    auto add_to = [&](int which, int k, const V8 &x, const V8 &y) {
        if constexpr (K == 1) {
            acc[which] = fma(x, y, acc[which]);
        } else if (p.slot[which] >= 0) {
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                float2 &s = accs[((p.slot[which] * K + k) * kP + i) * blockDim.x + threadIdx.x];
                s = __ffma2_rn(x.p[i], y.p[i], s);
            }
        }
    };
    const V8 one = splat(1.f);
    const float inv = 1.f / (float)p.D;
    const T *yb = static_cast<const T *>(p.y), *xb = static_cast<const T *>(p.x), *gb = static_cast<const T *>(p.g);
    const T *dhb = static_cast<const T *>(p.dh_in), *dub = static_cast<const T *>(p.du);
    long long hoff[K], dyoff[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        hoff[k] = C(r, k, lanes, p.D).hoff(p.dh, p.ys[1]);
        dyoff[k] = C(r, k, lanes, p.D).hoff(p.dh, (long long)p.T * p.dh);
    }
    const uint32_t stride = gridDim.x * per;
    // K > 1 keeps addresses, which the chunks of a row share
    auto slot = [&](int stage, int tensor, int) {
        return stages + (stage * kStage + tensor * C::kUnits) * pitch + threadIdx.x;
    };
    auto fetch = [&](uint32_t base, int stage) {
        if (base + warp_first < p.rows) {
            const uint32_t row = min(base + mine, p.rows - 1), b = p.byT(row), t = row - b * p.T;
            copy_async16(slot(stage, 5, 0), p.stats + 4 * (size_t)row);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const C c(r, k, lanes, p.D);
                c.fetch(yb + b * p.ys[0] + t * p.ys[2], p.dh, p.ys[1], hoff[k], slot(stage, 0, k), pitch);
                if (p.act) c.fetch(gb + b * p.gs[0] + t * p.gs[1], p.D, 0, 0, slot(stage, 1, k), pitch);
                if (p.pre) {
                    if (xb) c.fetch(xb + b * p.xs[0] + t * p.xs[1], p.D, 0, 0, slot(stage, 2, k), pitch);
                    c.fetch(dub + b * p.dus[0] + t * p.dus[1], p.D, 0, 0, slot(stage, 3, k), pitch);
                }
                if (dhb) c.fetch(dhb + b * p.dhs[0] + t * p.dhs[1], p.D, 0, 0, slot(stage, 4, k), pitch);
            }
        }
        copy_commit();
    };
    uint32_t base = blockIdx.x * per;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(base + i * stride, i);
    for (int stage = 0; base + warp_first < p.rows; base += stride, stage = stage + 1 == kAhead ? 0 : stage + 1) {
        const bool live = base + mine < p.rows;
        const uint32_t row = min(base + mine, p.rows - 1);
        copy_wait<kAhead - 1>();
        const float4 st = *reinterpret_cast<const float4 *>(slot(stage, 5, 0));
        V8 yn[K], A[K], dA[K], hn[K], G[K];
        float a = 0.f, c2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D);
            yn[k] = centre(c.get(slot(stage, 0, k), pitch, p.dh, p.ys[1], hoff[k]), st.x, st.y);  // y itself without a post norm
            if (!VEC || !c.has(0)) c.mask(yn[k]);
            if (p.act) {
                act_and_slope<T>(p.act, c.get(slot(stage, 1, k), pitch, p.D, 0, 0), A[k], dA[k]);
            }
            if (p.pre) {
                // h again from the inputs, its normalised form, and the norm's backward sums
                V8 h = c.scale_shift(yn[k], p.v.w1, p.v.b1);
                if (p.act) h = mul(h, A[k]);
                if (p.v.sc) h = mul(h, c.vec(p.v.sc));
                if (xb) h = fma(c.get(slot(stage, 2, k), pitch, p.D, 0, 0), p.alpha, h);
                hn[k] = centre(h, st.z, st.w);
                if (!VEC || !c.has(0)) c.mask(hn[k]);
                G[k] = c.get(slot(stage, 3, k), pitch, p.D, 0, 0);
                if (live) {
                    add_to(3, k, G[k], hn[k]);
                    add_to(4, k, G[k], one);
                }
                if (p.v.w2) G[k] = mul(G[k], c.vec(p.v.w2));
                a += total(G[k]);
                c2 += dot(G[k], hn[k]);
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
            const C c(r, k, lanes, p.D);
            // G = dh + r (dn - mean(dn) - n mean(dn n))
            if (p.pre) {
                G[k] = centre(fma(hn[k], -mc, G[k]), ma, st.w);
            } else {
                G[k] = splat(0.f);
            }
            if (dhb) G[k] = add(G[k], c.get(slot(stage, 4, k), pitch, p.D, 0, 0));
            if (p.dx && live) c.store(static_cast<T *>(p.dx) + (size_t)row * p.D, mul(G[k], p.alpha));
            V8 pv = c.scale_shift(yn[k], p.v.w1, p.v.b1);
            if (p.v.sc) {
                if (live) add_to(2, k, p.act ? mul(G[k], A[k]) : G[k], pv);
                G[k] = mul(G[k], c.vec(p.v.sc));
            }
            if (p.act) {
                if (live) c.store(static_cast<T *>(p.dg) + (size_t)row * p.D, mul(mul(G[k], pv), dA[k]));
                G[k] = mul(G[k], A[k]);
            }
            // G is now dp
            if (p.post) {
                if (live) {
                    add_to(0, k, G[k], yn[k]);
                    add_to(1, k, G[k], one);
                }
                if (p.v.w1) G[k] = mul(G[k], c.vec(p.v.w1));
                if (!VEC || !c.has(0)) c.mask(G[k]);
                a += total(G[k]);
                c2 += dot(G[k], yn[k]);
            }
        }
        fetch(base + kAhead * stride, stage);
        ma = mc = 0.f;
        if (p.post) {
            const float2 m = g.sum2(a, c2);
            if (p.post == 2) ma = m.x * inv;
            mc = m.y * inv;
        }
        // dy is contiguous in y's own layout
        const uint32_t b0 = p.byT(row), t0 = row - b0 * p.T;
        T *dy = static_cast<T *>(p.dy) + (size_t)b0 * p.T * p.D + (size_t)t0 * p.dh;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D);
            if (p.post) G[k] = centre(fma(yn[k], -mc, G[k]), ma, st.y);
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
            const C c(r, k, lanes, p.D);
            V8 s;
            if constexpr (K > 1) {
#pragma unroll
                for (int j = 0; j < kP; ++j) s.p[j] = accs[((p.slot[i] * K + k) * kP + j) * blockDim.x + threadIdx.x];
            } else if constexpr (BLOCK) {
                s = acc[i];
            } else {
                // the block's row groups, added in order
#pragma unroll
                for (int j = 0; j < kP; ++j) accs[j * blockDim.x + threadIdx.x] = acc[i].p[j];
                __syncthreads();
                s = splat(0.f);
                if (mine == 0)
#pragma unroll
                    for (int j = 0; j < kP; ++j)
                        for (uint32_t m = 0; m < per; ++m)
                            s.p[j] = __fadd2_rn(s.p[j], accs[j * blockDim.x + m * lanes + r]);
                __syncthreads();
            }
            const float *f = &s.p[0].x;
            if (mine == 0)
#pragma unroll
                for (int j = 0; j < kC; ++j)
                    if (c.has(j)) part[(size_t)p.slot[i] * p.D + c.c0 + j * c.step] = f[j];
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
// block a row with one chunk a thread, two past 4096 features.  (A warp with three chunks
// a lane for 768 features, no barrier: 42 us against 33 for a block of three warps at 8 x
// 2048 x 768, sandwich forward; the chunks cost the registers that hide its latency.)
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

template <typename P> int launch(void (*kernel)(P), const P &p, int blocks, int threads, int smem, cudaStream_t st)
{
    if (smem > 40 * 1024 &&  // with the static part, past the 48 KB that need no asking
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
        return -4;
    kernel<<<blocks, threads, smem, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <typename T, bool VEC>
int run_fwd(const FwdParams &p, const Shape &s, int blocks, cudaStream_t st)
{
    using C = Chunk<T, VEC>;
    const int smem = C::kAhead * 3 * s.K * C::kUnits * s.threads * 16;
    if (!s.block) return launch(ttt_block_norm_fwd_kernel<T, VEC, 1, false>, p, blocks, s.threads, smem, st);
    return s.K == 1 ? launch(ttt_block_norm_fwd_kernel<T, VEC, 1, true>, p, blocks, s.threads, smem, st)
                    : launch(ttt_block_norm_fwd_kernel<T, VEC, 2, true>, p, blocks, s.threads, smem, st);
}

template <typename T, bool VEC>
int run_bwd(const BwdParams &p, const Shape &s, int blocks, cudaStream_t st)
{
    const int sums = s.K > 1 ? p.nvec * s.K * kC * 4 : s.block ? 0 : kC * 4;
    using C1 = Chunk<T, VEC>;
    using C2 = Chunk<T, VEC, true>;
    const int stage = s.K > 1 ? C2::kAhead * (5 * C2::kUnits + 1) * 16 : C1::kAhead * (5 * C1::kUnits + 1) * 16;
    const int smem = (stage + sums) * s.threads;
    if (!s.block) return launch(ttt_block_norm_bwd_kernel<T, VEC, 1, false, 128>, p, blocks, s.threads, smem, st);
    if (s.K == 2) return launch(ttt_block_norm_bwd_kernel<T, VEC, 2, true, 512>, p, blocks, s.threads, smem, st);
    return s.threads <= 256 ? launch(ttt_block_norm_bwd_kernel<T, VEC, 1, true, 256>, p, blocks, s.threads, smem, st)
                            : launch(ttt_block_norm_bwd_kernel<T, VEC, 1, true, 512>, p, blocks, s.threads, smem, st);
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
        return vec ? run_fwd<__nv_bfloat16, true>(p, s, blocks, a.stream)
                   : run_fwd<__nv_bfloat16, false>(p, s, blocks, a.stream);
    return vec ? run_fwd<float, true>(p, s, blocks, a.stream) : run_fwd<float, false>(p, s, blocks, a.stream);
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
    if (rc) return rc;
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
