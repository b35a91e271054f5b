// ttt_block_norm.cuh -- what stands around a block's inner layer, in one pass over the
// rows (tokens), forward and backward:
//     p = N1(y),  m = scale * act(gate) * p,  h = alpha x + m,  u = N2(h)
// N1, N2: none, RMS (v / sqrt(mean v^2 + eps) * w) or layer norm ((v - mean) /
// sqrt(var + eps) * w + b) over the D features; y token-major or the TTT layer's
// head-major output.  Backward with dn the gradient of a normalised row n = (v - mean) r:
//     dv = r (dn - [layer] mean(dn) - n mean(dn n)).
//
// Every tensor is read or written once.  A row belongs to a group of `lanes` threads (part
// of a warp up to 256 features, else the whole block), a thread holding K chunks of eight
// features in fp32 registers, so a row's statistics and its outputs come from one read.
// The variance is taken about the mean, never as a difference of squares.
//
// What bounds these kernels is issue slots as much as HBM (some 40 instructions a feature
// forward and 60 backward, against 10 and 16 bytes): arithmetic on paired fp32 instructions, the parts that
// a call has or lacks (POST, PRE, ACT) known at compile time, parameter vectors that are
// absent replaced by ones and zeros instead of branches, rows copied ahead with cp.async.
// Measured (bf16, gate, residual and both norms; of the copy bandwidth): 8 x 2048 x 768
// forward 24 us (0.77) and backward 48 us (0.62), 2 x 32768 x 2048 with layer norm and GELU 227 us
// (0.87) and 515 us (0.61: registers leave eight warps an SM); y and gate alone, layer norm and
// GELU, 8 x 2048 x 768 22 us (0.50: as many instructions, and as many reductions to wait for, for
// three fifths of the bytes).
#pragma once

#include <cstdint>
#include <mutex>

#include <cuda_runtime.h>

#include "ttt_internal.h"
#include "ttt_vec.cuh"

namespace ttt {

constexpr int kNormChunk = 8;  // features of a chunk

// row / T for rows below 2^31: multiply by ceil(2^(32 + shift) / T), keep the high part
// (Granlund and Montgomery, Division by invariant integers using multiplication).
struct Div {
    uint32_t d, mul, shift;
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const
    {
        return d == 1 ? n : __umulhi(n, mul) >> shift;
    }
};

inline Div make_div(int d)
{
    Div r = {(uint32_t)d, 0, 0};
    if (d > 1) {
        while ((1u << r.shift) < (uint32_t)d) ++r.shift;  // 2^shift >= d, shift >= 1
        --r.shift;
        r.mul = (uint32_t)(((1ull << (32 + r.shift)) + d - 1) / d);
    }
    return r;
}

struct NormVectors {  // fp32 [D], never null (absent: ones or zeros)
    const float *w1, *b1, *sc, *w2, *b2;
};

struct NormFwdParams {
    const void *y, *x, *g;
    void *h, *u;
    float *stats;
    NormVectors v;
    long long ys[3], xs[2], gs[2];
    uint32_t rows;
    Div byT;
    int T, D, dh, lanes, post, pre, act;
    int even;  // every tensor token-major and contiguous: one offset for all
    float eps1, eps2, alpha;
};

struct NormBwdParams {
    const void *y, *x, *g, *dh_in, *du;
    void *dy, *dx, *dg;
    const float *stats;
    float *part;  // [blocks][nvec][D] partial parameter gradients
    NormVectors v;
    long long ys[3], xs[2], gs[2], dhs[2], dus[2];
    uint32_t rows;
    Div byT;
    int T, D, dh, lanes, post, pre, act;
    int even;
    int slot[5];  // slot of each parameter gradient among the nvec, -1: absent
    int nvec;
    float alpha;
};

// Threads of a row and chunks of a thread.
struct NormShape {
    int lanes, threads, K;
    bool block;
};

// One direction and type each (a translation unit each); group: features that stand
// together (8, 2, 1); limit: the most blocks.
int norm_fwd_bf16(const NormFwdParams &p, const NormShape &s, int group, cudaStream_t st);
int norm_fwd_f32(const NormFwdParams &p, const NormShape &s, int group, cudaStream_t st);
int norm_bwd_bf16(const NormBwdParams &p, const NormShape &s, int group, int limit, cudaStream_t st, int *blocks);
int norm_bwd_f32(const NormBwdParams &p, const NormShape &s, int group, int limit, cudaStream_t st, int *blocks);

namespace {

constexpr int kSMs = 152, kC = kNormChunk;

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

// 1 / (1 + exp(-g)); 0 and 1 where exp(-g) leaves the range.  bf16 tensors: one ex2 of a rounded
// product, off by |g| 2^-24 of itself, far below the output's rounding.  fp32 tensors: CUDA's
// expf.  e: exp(-g).
template <typename T> __device__ __forceinline__ float2 logistic(float2 g, float2 &e)
{
    if constexpr (sizeof(T) == 2) {
        const float2 t = __fmul2_rn(g, both(-1.4426950408889634f));
        e = make_float2(exp2_approx(t.x), exp2_approx(t.y));
    } else {
        e = make_float2(expf(-g.x), expf(-g.y));
    }
    const float2 d = __fadd2_rn(e, both(1.f));
    return make_float2(rcp_approx(d.x), rcp_approx(d.y));
}
template <typename T> __device__ __forceinline__ float2 logistic(float2 g)
{
    float2 e;
    return logistic<T>(g, e);
}

// GELU of bf16 tensors, from w = Phi(-|g|) = t P(t) exp(-g^2 / 2) with t = 1 / (3.46 + |g|) (the form of
// Hastings, Approximations for Digital Computers; the exponential is the density's too): g Phi(g)
// = max(g, 0) - |g| w, and Phi is w or 1 - w, so the tail is never a difference.  P, of degree 5
// with w(0) = 1/2, minimises over |g| <= 14 the larger of w's absolute error (5e-8; parameter
// gradients, fp32 sums over many tokens, see it) and 1/2400 of its relative one (1.3e-4, 2^-4 of the
// output's rounding where GELU is all tail), by linear programming; in fp32 2e-7 and 1.3e-4 over
// every bf16 g there.
struct GeluTail {
    float2 m, density, neg;  // |g| (finite), phi(g), -w

    __device__ __forceinline__ explicit GeluTail(float2 g)
    {
        m = make_float2(fminf(fabsf(g.x), 1e30f), fminf(fabsf(g.y), 1e30f));
        const float2 d = __fadd2_rn(m, both(3.4602077f)), t = make_float2(rcp_approx(d.x), rcp_approx(d.y));
        const float2 q = __fmul2_rn(__fmul2_rn(g, g), both(-0.5f * 1.4426950408889634f));
        const float2 e = make_float2(exp2_approx(q.x), exp2_approx(q.y));
        density = __fmul2_rn(e, both(0.3989422804014327f));
        neg = __ffma2_rn(t, both(155.2399f), both(-145.96509f));
        neg = __ffma2_rn(t, neg, both(15.05492f));
        neg = __ffma2_rn(t, neg, both(-7.710322f));
        neg = __ffma2_rn(t, neg, both(-1.1785265f));
        neg = __ffma2_rn(t, neg, both(-0.40367082f));
        neg = __fmul2_rn(__fmul2_rn(t, neg), e);
    }
};

template <typename T> __device__ __forceinline__ float2 gelu(float2 g)
{
    if constexpr (sizeof(T) == 2) {
        const GeluTail w(g);
        return __ffma2_rn(w.m, w.neg, make_float2(fmaxf(g.x, 0.f), fmaxf(g.y, 0.f)));
    } else {
        return make_float2(g.x * normcdff(g.x), g.y * normcdff(g.y));
    }
}

// Phi(g) and the normal density (fp32 tensors: CUDA's normcdff)
template <typename T> __device__ __forceinline__ float2 gelu_cdf(float2 g, float2 &density)
{
    if constexpr (sizeof(T) == 2) {
        const GeluTail w(g);
        density = w.density;
        const float2 h = __fadd2_rn(w.neg, both(1.f));
        return make_float2(g.x < 0.f ? -w.neg.x : h.x, g.y < 0.f ? -w.neg.y : h.y);
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
        for (int i = 0; i < kP; ++i) r.p[i] = __fmul2_rn(g.p[i], logistic<T>(g.p[i]));
    } else if (act == 3) {
#pragma unroll
        for (int i = 0; i < kP; ++i) r.p[i] = gelu<T>(g.p[i]);
    } else {
#pragma unroll
        for (int i = 0; i < kP; ++i) r.p[i] = logistic<T>(g.p[i]);
    }
    return r;
}

// act(g) and its derivative
template <typename T> __device__ __forceinline__ void act_and_slope(int act, const V8 &g, V8 &a, V8 &da)
{
    if (act == 2) {
#pragma unroll
        for (int i = 0; i < kP; ++i) {
            const float2 s = logistic<T>(g.p[i]);
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
            float2 e;
            const float2 s = logistic<T>(g.p[i], e), c = __ffma2_rn(s, both(-1.f), both(1.f)), es = __fmul2_rn(e, s);
            a.p[i] = s;
            // 1 - s, which cancels for large g and is exp(-g) s there
            da.p[i] = __fmul2_rn(s, make_float2(g.p[i].x > 0.f ? es.x : c.x, g.p[i].y > 0.f ? es.y : c.y));
        }
    }
}

// ------------------------------------------------------------------ chunk access

// Eight features in the I/O type, G together in memory.
template <typename T, int G> struct Raw {
    static constexpr int V = G == kC ? 16 / (int)sizeof(T) : G, N = kC / V;  // features of a load, loads
    Pack<T, V> q[N];
    __device__ __forceinline__ V8 get() const
    {
        V8 r;
        float *v = &r.p[0].x;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float w[V];
            unpack(q[i], w);
#pragma unroll
            for (int j = 0; j < V; ++j) v[i * V + j] = w[j];
        }
        return r;
    }
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

// Which eight features of a row a thread holds: consecutive ones (G = 8: rows of whole 16
// bytes), or pieces of G `lanes` pieces apart (G = 2: pairs never straddle a row's end or an
// alignment; G = 1).  G = 8: a thread past the row's end works on the row's last chunk
// (`at`) and neither counts nor stores.  Else features past D read as zeros.
//
// How a row's features arrive (FEED):
//   kStaged (16-byte rows): through shared memory.  fetch() starts copies of the thread's
//     own features, get() reads them back once they have landed.  Only the thread itself
//     reads what it copied, so there is no barrier, and no load waits in a register.  slot:
//     the thread's place in a stage, 16-byte units `pitch` apart.
//   kRegisters (other rows): loaded a row ahead into registers, element by element.
//   kDirect (widths whose sums leave room for neither): when they are used.
// Loads do not go through the read-only path, as h may be written over x.
enum Feed { kStaged, kRegisters, kDirect };

template <typename T, int G> struct Chunk {
    using R = Raw<T, G>;
    static constexpr bool VEC = G == kC;
    static constexpr int kUnits = kC * (int)sizeof(T) / 16;  // 16-byte units of a chunk
    // rows in flight or landed (kStaged).  Three were slower than two (8 x 2048 x 768 sandwich
    // forward 35 us against 31, 2 x 32768 x 2048 306 against 287): the stages take the L1
    // that holds the parameter vectors.
    static constexpr int kAhead = 2;
    // fp32: a chunk is two loads, and two threads' chunks make four; where D and the heads are
    // multiples of 16 a thread takes every other one of them (SPLIT), so that the two threads
    // fill a 32-byte sector with each (2 x 8192 x 768 forward 50 us against 64, backward 91
    // against 114).
    static constexpr bool SPLIT = VEC && sizeof(T) == 4;
    int c0, at, step, D;
    __device__ __forceinline__ Chunk(int r, int k, int lanes, int D_, int dh = 1)
        : c0(VEC ? (k * lanes + r) * kC : r * G + k * kC * lanes), step(VEC ? R::V : lanes * G), D(D_)
    {
        at = VEC ? min(c0, D - kC) : c0;
        if (SPLIT && ((D | dh) & 15) == 0) {
            at -= (at & 8) >> 1;
            step = 2 * R::V;
        }
    }
    // first feature of load i, and whether it is there
    __device__ __forceinline__ int col(int i) const { return (VEC ? at : c0) + i * step; }
    __device__ __forceinline__ bool has(int i) const { return VEC ? c0 < D : c0 + i * step < D; }
    // zeros in the absent features (VEC: the whole chunk counts or not, see counted())
    __device__ __forceinline__ void mask(V8 &v) const
    {
        if constexpr (!VEC) {
            float *f = &v.p[0].x;
#pragma unroll
            for (int j = 0; j < kC; ++j) f[j] = has(j / G) ? f[j] : 0.f;
        }
    }
    __device__ __forceinline__ float counted(float sum) const { return !VEC || c0 < D ? sum : 0.f; }
    // Elements that feature c's head adds to its offset in a row whose features lie in heads
    // of dh, sh elements apart (dh = D: none).  A load lies inside one head.
    __device__ __forceinline__ long long head(int c, int dh, long long sh) const
    {
        return dh < D ? (long long)(c / dh) * (sh - dh) : 0;
    }
    // row: the token's first feature; off (VEC): head(at, ..)
    __device__ __forceinline__ void fetch(const T *row, long long off, uint4 *slot, int pitch) const
    {
#pragma unroll
        for (int i = 0; i < kUnits; ++i) copy_async16(slot + i * pitch, row + off + col(i));
    }
    __device__ __forceinline__ V8 get(const uint4 *slot, int pitch) const
    {
        Raw<T, kC> q;
#pragma unroll
        for (int i = 0; i < Raw<T, kC>::N; ++i) q.q[i].raw = slot[i * pitch];
        return q.get();
    }
    __device__ __forceinline__ void load(const T *row, int dh, long long sh, long long off, R &r) const
    {
#pragma unroll
        for (int i = 0; i < R::N; ++i) {
            r.q[i].raw = {};
            if (VEC || has(i)) r.q[i].load_rw(row + (VEC ? off : head(col(i), dh, sh)) + col(i));
        }
    }
    // VEC: row with the head's offset already in it
    __device__ __forceinline__ void store(T *row, const V8 &v) const
    {
        R r;
        r.put(v);
#pragma unroll
        for (int i = 0; i < R::N; ++i)
            if (has(i)) r.q[i].store(row + col(i));
    }
    __device__ __forceinline__ void store_heads(T *row, int dh, long long sh, long long off, const V8 &v) const
    {
        R r;
        r.put(v);
#pragma unroll
        for (int i = 0; i < R::N; ++i)
            if (has(i)) r.q[i].store(row + (VEC ? off : head(col(i), dh, sh)) + col(i));
    }
    // a parameter vector (G = 8: 16-byte, G = 2: 8-byte aligned)
    __device__ __forceinline__ V8 vec(const float *p) const
    {
        V8 r = {};
        if constexpr (VEC) {
#pragma unroll
            for (int j = 0; j < kP; j += 2) {
                const float4 w = __ldg(reinterpret_cast<const float4 *>(p + (SPLIT ? col(j / 2) : at + 2 * j)));
                r.p[j] = make_float2(w.x, w.y);
                r.p[j + 1] = make_float2(w.z, w.w);
            }
        } else if constexpr (G == 2) {
#pragma unroll
            for (int j = 0; j < kP; ++j)
                if (has(j)) r.p[j] = __ldg(reinterpret_cast<const float2 *>(p + col(j)));
        } else {
            float *v = &r.p[0].x;
#pragma unroll
            for (int j = 0; j < kC; ++j)
                if (has(j)) v[j] = __ldg(p + col(j));
        }
        return r;
    }
    // feature j of a chunk, for the partial sums
    __device__ __forceinline__ int feature(int j) const { return SPLIT ? col(j / 4) + j % 4 : VEC ? c0 + j : c0 + j / G * step + j % G; }
};

// -------------------------------------------------------------------- reductions

// Sums over a row's group of threads.  BLOCK: over the block, through two shared slots
// used in turn (a slot is written again only after the next reduction's barrier); the
// slots of warps that are not there stay zero, and four warps' numbers are read at once.
template <bool BLOCK> struct Group {
    int lanes, warps;
    float *red, *mine;  // the slot in use: all warps', this warp's (or half warp's) own

    __device__ __forceinline__ float warp_sum(float v) const
    {
        if constexpr (BLOCK) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        } else {
            for (int o = lanes >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        }
        return v;
    }
    __device__ __forceinline__ void turn()
    {
        const int d = (reinterpret_cast<uintptr_t>(red) & 128) ? -32 : 32;
        red += d;
        mine += d;
    }
    // sums of a and of b
    __device__ __forceinline__ float2 sum2(float a, float b)
    {
        if constexpr (BLOCK) {
            // they share the shuffles: after the first exchange each half of the warp carries
            // one of them
            const bool up = threadIdx.x & 16;
            float v = (up ? b : a) + __shfl_xor_sync(0xffffffffu, up ? a : b, 16);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if ((threadIdx.x & 15) == 0) *mine = v;
            __syncthreads();
            const float4 *q = reinterpret_cast<const float4 *>(red);
            float2 s[2] = {both(0.f), both(0.f)};  // [0]: a of warps 0-3, ..
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * i < warps) {
                    const float4 x = q[i], y = q[4 + i];
                    s[0] = __fadd2_rn(s[0], __fadd2_rn(make_float2(x.x, x.y), make_float2(x.z, x.w)));
                    s[1] = __fadd2_rn(s[1], __fadd2_rn(make_float2(y.x, y.y), make_float2(y.z, y.w)));
                }
            turn();
            return make_float2(s[0].x + s[0].y, s[1].x + s[1].y);
        } else {
            return make_float2(warp_sum(a), warp_sum(b));
        }
    }
    __device__ __forceinline__ float sum1(float a)
    {
        a = warp_sum(a);
        if constexpr (BLOCK) {
            if ((threadIdx.x & 31) == 0) *mine = a;
            __syncthreads();
            const float4 *q = reinterpret_cast<const float4 *>(red);
            float2 s = both(0.f);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (4 * i < warps) {
                    const float4 x = q[i];
                    s = __fadd2_rn(s, __fadd2_rn(make_float2(x.x, x.y), make_float2(x.z, x.w)));
                }
            turn();
            a = s.x + s.y;
        }
        return a;
    }
};

// red: two slots of 16 warps' numbers for each of two sums
template <bool BLOCK> __device__ __forceinline__ Group<BLOCK> make_group(float *red, int lanes)
{
    Group<BLOCK> g;
    g.lanes = lanes;
    g.warps = blockDim.x >> 5;
    g.red = red;
    // the upper half warp carries the second of two sums
    g.mine = red + (threadIdx.x >> 5) + (threadIdx.x & 16);
    if constexpr (BLOCK) {
        for (int i = threadIdx.x; i < 64; i += blockDim.x) red[i] = 0.f;
        __syncthreads();
    }
    return g;
}

// mean and 1 / sqrt(.. + eps) of a row held as v[K] (absent features are zeros or do not
// count)
template <typename T, int G, int K, bool BLOCK>
__device__ __forceinline__ float2 row_stats(Group<BLOCK> &g, int kind, float eps, float inv, const V8 (&v)[K], int r, int D)
{
    float mean = 0.f, s = 0.f;
    if (kind == 2) {
#pragma unroll
        for (int k = 0; k < K; ++k) s += Chunk<T, G>(r, k, g.lanes, D).counted(total(v[k]));
        mean = g.sum1(s) * inv;
        s = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const Chunk<T, G> c(r, k, g.lanes, D);
            V8 d = add(v[k], splat(-mean));
            c.mask(d);
            s += c.counted(dot(d, d));
        }
    } else {
#pragma unroll
        for (int k = 0; k < K; ++k) s += Chunk<T, G>(r, k, g.lanes, D).counted(dot(v[k], v[k]));
    }
    return make_float2(mean, rsqrtf(g.sum1(s) * inv + eps));
}

// ----------------------------------------------------------------------- forward

// POST, PRE: the norm's kind (0 none, 1 RMS, 2 layer), ACT: whether there is a gate; -1: by
// the parameters.  With 16-byte rows the parameter vectors stay in registers: loading
// three to five of them for every row kept L1 85% busy (2 x 32768 x 2048 257 us against
// 225, 8 x 2048 x 768 sandwich 25.3 against 23.2).
//
// Six blocks of 128 threads an SM, 80 registers, for one chunk a thread (8 x 2048 x 768 with
// layer norm, GELU and RMS norm 27.6 us against 33.3 with 84 registers left to the
// compiler; GELU and layer norm alone 21.9 against 23.5), but not with two layer norms, whose five
// vectors would spill (fp32 2 x 8192 x 768: 52.5 against 47.5).
constexpr int fwd_blocks(int K, int post, int pre) { return K == 1 && post >= 0 && post + pre < 4 ? 6 : 1; }
constexpr int fwd_threads(bool block, int K, int post, int pre) { return block && fwd_blocks(K, post, pre) == 1 ? 512 : 128; }

template <typename T, int G, int K, bool BLOCK, int POST, int PRE, int ACT>
__global__ void __launch_bounds__(fwd_threads(BLOCK, K, POST, PRE), fwd_blocks(K, POST, PRE)) ttt_block_norm_fwd_kernel(const __grid_constant__ NormFwdParams p)
{
    using C = Chunk<T, G>;
    constexpr bool VEC = C::VEC;
    constexpr Feed FEED = VEC ? kStaged : kRegisters;
    constexpr int kAhead = FEED == kStaged ? C::kAhead : 1;
    __shared__ __align__(256) float red[64];
    extern __shared__ uint4 stages[];  // kStaged: [kAhead][3][K][units][threads]
    const int lanes = p.lanes, tid = threadIdx.x, r = BLOCK ? tid : tid & (lanes - 1), pitch = blockDim.x;
    const uint32_t per = BLOCK ? 1 : blockDim.x / lanes, mine = BLOCK ? 0 : tid / lanes;
    Group<BLOCK> grp = make_group<BLOCK>(red, lanes);
    const int post = POST < 0 ? p.post : POST, pre = PRE < 0 ? p.pre : PRE;
    const bool act = ACT < 0 ? p.act != 0 : ACT != 0, has_x = p.x != nullptr;
    // a warp's groups leave the loop together: rows past the end are computed, not written
    const uint32_t warp_first = BLOCK ? 0 : (tid & ~31) / lanes;
    const T *yb = static_cast<const T *>(p.y), *xb = static_cast<const T *>(p.x), *gb = static_cast<const T *>(p.g);
    const float inv = 1.f / (float)p.D;
    const uint32_t stride = gridDim.x * per;
    long long hoff[K];
#pragma unroll
    for (int k = 0; k < K; ++k) hoff[k] = VEC ? C(r, k, lanes, p.D, p.dh).head(C(r, k, lanes, p.D, p.dh).at, p.dh, p.ys[1]) : 0;
    // the parameter vectors, held or loaded for every row
    constexpr bool HOLD = VEC;
    V8 par[5][HOLD ? K : 1];
    if constexpr (HOLD)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D, p.dh);
            par[0][k] = c.vec(p.v.w1);
            par[1][k] = c.vec(p.v.b1);
            par[2][k] = c.vec(p.v.sc);
            par[3][k] = c.vec(p.v.w2);
            par[4][k] = c.vec(p.v.b2);
        }
    auto normed = [&](int kind, const V8 &a, float2 s, const V8 &w, const V8 &b, const C &c, const float *wp, const float *bp) {
        if (kind == 2) return fma(centre(a, s.x, s.y), HOLD ? w : c.vec(wp), HOLD ? b : c.vec(bp));
        return mul(mul(a, s.y), HOLD ? w : c.vec(wp));
    };
    Raw<T, G> regs[3][K];
    auto slot = [&](int stage, int tensor, int k) { return stages + ((stage * 3 + tensor) * K + k) * C::kUnits * pitch + tid; };
    auto fetch = [&](uint32_t base, int stage) {
        if (base + warp_first < p.rows) {
            const uint32_t row = BLOCK ? base : min(base + mine, p.rows - 1);
            const T *y, *gt, *x;
            if (p.even) {
                const size_t o = (size_t)row * p.D;
                y = yb + o;
                gt = gb + o;
                x = xb + o;
            } else {
                const uint32_t b = p.byT(row), t = row - b * p.T;
                y = yb + b * p.ys[0] + t * p.ys[2];
                gt = gb + b * p.gs[0] + t * p.gs[1];
                x = xb + b * p.xs[0] + t * p.xs[1];
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const C c(r, k, lanes, p.D, p.dh);
                if constexpr (FEED == kStaged) {
                    c.fetch(y, hoff[k], slot(stage, 0, k), pitch);
                    if (act) c.fetch(gt, 0, slot(stage, 1, k), pitch);
                    if (has_x) c.fetch(x, 0, slot(stage, 2, k), pitch);
                } else {
                    c.load(y, p.dh, p.ys[1], 0, regs[0][k]);
                    if (act) c.load(gt, p.D, 0, 0, regs[1][k]);
                    if (has_x) c.load(x, p.D, 0, 0, regs[2][k]);
                }
            }
        }
        if constexpr (FEED == kStaged) copy_commit();
    };
    uint32_t base = blockIdx.x * per;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(base + i * stride, i);
    for (int stage = 0; base + warp_first < p.rows; base += stride, stage = stage + 1 == kAhead ? 0 : stage + 1) {
        const bool live = BLOCK || base + mine < p.rows;
        const size_t off = (size_t)(base + mine) * p.D;
        if constexpr (FEED == kStaged) copy_wait<kAhead - 1>();
        auto take = [&](int tensor, int k, const C &c) {
            if constexpr (FEED == kStaged) return c.get(slot(stage, tensor, k), pitch);
            else return regs[tensor][k].get();
        };
        V8 v[K];
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] = take(0, k, C(r, k, lanes, p.D, p.dh));
        float2 s1 = make_float2(0.f, 1.f), s2 = make_float2(0.f, 1.f);
        if (post) s1 = row_stats<T, G, K, BLOCK>(grp, post, p.eps1, inv, v, r, p.D);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D, p.dh);
            if (post) v[k] = normed(post, v[k], s1, par[0][HOLD ? k : 0], par[1][HOLD ? k : 0], c, p.v.w1, p.v.b1);
            if (act) v[k] = mul(v[k], act_value<T>(p.act, take(1, k, c)));
            v[k] = mul(v[k], HOLD ? par[2][HOLD ? k : 0] : c.vec(p.v.sc));
            if (has_x) v[k] = fma(take(2, k, c), p.alpha, v[k]);
            if (live) c.store(static_cast<T *>(p.h) + off, v[k]);
            c.mask(v[k]);
        }
        fetch(base + kAhead * stride, stage);
        if (pre) {
            // of h in fp32, before the rounding that stores it
            s2 = row_stats<T, G, K, BLOCK>(grp, pre, p.eps2, inv, v, r, p.D);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const C c(r, k, lanes, p.D, p.dh);
                v[k] = normed(pre, v[k], s2, par[3][HOLD ? k : 0], par[4][HOLD ? k : 0], c, p.v.w2, p.v.b2);
                if (live) c.store(static_cast<T *>(p.u) + off, v[k]);
            }
        }
        if (p.stats && live && r == 0)
            *reinterpret_cast<float4 *>(p.stats + 4 * (size_t)(base + mine)) = make_float4(s1.x, s1.y, s2.x, s2.y);
    }
}

// ---------------------------------------------------------------------- backward

// Parameter gradients: every thread sums its own features over the block's rows (in
// registers; WIDE: in shared memory, which leaves none for stages), blocks write
// partial sums, a second kernel adds those in order.  The order is fixed by the sizes, the
// type, the tensors' alignment, the parts that a call has and asks for, and how many
// blocks the device holds.
template <typename T, int G, int K, bool BLOCK, int MAXT, int POST, int PRE, int ACT>
__global__ void __launch_bounds__(MAXT, MAXT >= 256 ? 1 : 256 / MAXT) ttt_block_norm_bwd_kernel(const __grid_constant__ NormBwdParams p)
{
    constexpr bool WIDE = K > 1 && MAXT > 256;  // sums in shared memory
    using C = Chunk<T, G>;
    constexpr bool VEC = C::VEC;
    constexpr Feed FEED = WIDE ? kDirect : VEC ? kStaged : kRegisters;
    constexpr int kAhead = FEED == kStaged ? C::kAhead : 1, kStage = 5 * K * C::kUnits + 1;
    __shared__ __align__(256) float red[64];
    extern __shared__ uint4 stages[];  // kStaged: [kAhead][5 K units + 1][threads]; the sums:
    // WIDE: [nvec][K][4][threads] pairs; not BLOCK: [4][threads]
    const int lanes = p.lanes, tid = threadIdx.x, threads = blockDim.x, r = BLOCK ? tid : tid & (lanes - 1);
    float2 *accs = reinterpret_cast<float2 *>(stages + (FEED == kStaged ? kAhead * kStage * threads : 0));
    const uint32_t per = BLOCK ? 1 : threads / lanes, mine = BLOCK ? 0 : tid / lanes;
    Group<BLOCK> grp = make_group<BLOCK>(red, lanes);
    const int post = POST < 0 ? p.post : POST, pre = PRE < 0 ? p.pre : PRE;
    const bool act = ACT < 0 ? p.act != 0 : ACT != 0;
    const bool has_x = pre && p.x, has_dh = p.dh_in != nullptr;
    const uint32_t warp_first = BLOCK ? 0 : (tid & ~31) / lanes;
    V8 acc[WIDE ? 1 : 5][K];
#pragma unroll
    for (int i = 0; i < (WIDE ? 1 : 5); ++i)
#pragma unroll
        for (int k = 0; k < K; ++k) acc[i][k] = splat(0.f);
    if constexpr (WIDE)
        for (int i = 0; i < p.nvec * K * kP; ++i) accs[i * threads + tid] = make_float2(0.f, 0.f);
    // += a b
    auto add_to = [&](int which, int k, const V8 &x, const V8 &y) {
        if constexpr (!WIDE) {
            acc[which][k] = fma(x, y, acc[which][k]);
        } else if (p.slot[which] >= 0) {
#pragma unroll
            for (int i = 0; i < kP; ++i) {
                float2 &s = accs[((p.slot[which] * K + k) * kP + i) * threads + tid];
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
        const C c(r, k, lanes, p.D, p.dh);
        hoff[k] = VEC ? c.head(c.at, p.dh, p.ys[1]) : 0;
        dyoff[k] = VEC ? c.head(c.at, p.dh, (long long)p.T * p.dh) : 0;
    }
    const uint32_t stride = gridDim.x * per;
    // the parameter vectors: held (8 x 2048 x 768 47 us against 51), or loaded when they are
    // used where two chunks' sums leave no registers
    constexpr bool HOLD = VEC && K == 1;
    V8 par[4] = {};
    if constexpr (HOLD) {
        const C c(r, 0, lanes, p.D, p.dh);
        par[0] = c.vec(p.v.w1);
        par[1] = c.vec(p.v.b1);
        par[2] = c.vec(p.v.sc);
        par[3] = c.vec(p.v.w2);
    }
    auto w1 = [&](int, const C &c) { return HOLD ? par[0] : c.vec(p.v.w1); };
    auto sc = [&](int, const C &c) { return HOLD ? par[2] : c.vec(p.v.sc); };
    auto w2 = [&](int, const C &c) { return HOLD ? par[3] : c.vec(p.v.w2); };
    Raw<T, G> regs[5][FEED == kRegisters ? K : 1];
    float4 next_st = make_float4(0.f, 1.f, 0.f, 1.f);
    const T *rows[5];  // kDirect: the row's addresses
    auto slot = [&](int stage, int tensor, int k) { return stages + (stage * kStage + (tensor * K + k) * C::kUnits) * threads + tid; };
    auto fetch = [&](uint32_t base, int stage) {
        if (base + warp_first < p.rows) {
            const uint32_t row = BLOCK ? base : min(base + mine, p.rows - 1);
            const T *y, *gt, *x, *du, *dh;
            if (p.even) {
                const size_t o = (size_t)row * p.D;
                y = yb + o;
                gt = gb + o;
                x = xb + o;
                du = dub + o;
                dh = dhb + o;
            } else {
                const uint32_t b = p.byT(row), t = row - b * p.T;
                y = yb + b * p.ys[0] + t * p.ys[2];
                gt = gb + b * p.gs[0] + t * p.gs[1];
                x = xb + b * p.xs[0] + t * p.xs[1];
                du = dub + b * p.dus[0] + t * p.dus[1];
                dh = dhb + b * p.dhs[0] + t * p.dhs[1];
            }
            if constexpr (FEED == kStaged) {
                copy_async16(slot(stage, 5, 0), p.stats + 4 * (size_t)row);
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const C c(r, k, lanes, p.D, p.dh);
                    c.fetch(y, hoff[k], slot(stage, 0, k), threads);
                    if (act) c.fetch(gt, 0, slot(stage, 1, k), threads);
                    if (has_x) c.fetch(x, 0, slot(stage, 2, k), threads);
                    if (pre) c.fetch(du, 0, slot(stage, 3, k), threads);
                    if (has_dh) c.fetch(dh, 0, slot(stage, 4, k), threads);
                }
            } else {
                next_st = *reinterpret_cast<const float4 *>(p.stats + 4 * (size_t)row);
                if constexpr (FEED == kRegisters) {
#pragma unroll
                    for (int k = 0; k < K; ++k) {
                        const C c(r, k, lanes, p.D, p.dh);
                        c.load(y, p.dh, p.ys[1], hoff[k], regs[0][k]);
                        if (act) c.load(gt, p.D, 0, 0, regs[1][k]);
                        if (has_x) c.load(x, p.D, 0, 0, regs[2][k]);
                        if (pre) c.load(du, p.D, 0, 0, regs[3][k]);
                        if (has_dh) c.load(dh, p.D, 0, 0, regs[4][k]);
                    }
                } else {
                    rows[0] = y;
                    rows[1] = gt;
                    rows[2] = x;
                    rows[3] = du;
                    rows[4] = dh;
                }
            }
        }
        if constexpr (FEED == kStaged) copy_commit();
    };
    uint32_t base = blockIdx.x * per;
#pragma unroll
    for (int i = 0; i < kAhead; ++i) fetch(base + i * stride, i);
    for (int stage = 0; base + warp_first < p.rows; base += stride, stage = stage + 1 == kAhead ? 0 : stage + 1) {
        const bool live = BLOCK || base + mine < p.rows;
        const size_t off = (size_t)(base + mine) * p.D;
        float4 st = next_st;
        if constexpr (FEED == kStaged) {
            copy_wait<kAhead - 1>();
            st = *reinterpret_cast<const float4 *>(slot(stage, 5, 0));
        }
        auto take = [&](int tensor, int k, const C &c) {
            if constexpr (FEED == kStaged) {
                return c.get(slot(stage, tensor, k), threads);
            } else if constexpr (FEED == kRegisters) {
                return regs[tensor][k].get();
            } else {
                Raw<T, G> q;
                if (tensor == 0) c.load(rows[0], p.dh, p.ys[1], hoff[k], q);
                else c.load(rows[tensor], p.D, 0, 0, q);
                return q.get();
            }
        };
        V8 yn[K], A[K], dA[K], hn[K], gr[K];
        auto weighted = [&](int k, const C &c) {
            return post == 2 ? fma(yn[k], w1(k, c), HOLD ? par[1] : c.vec(p.v.b1)) : mul(yn[k], w1(k, c));
        };
        float a = 0.f, c2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D, p.dh);
            yn[k] = take(0, k, c);
            if (post) yn[k] = post == 2 ? centre(yn[k], st.x, st.y) : mul(yn[k], st.y);
            c.mask(yn[k]);
            if (act) act_and_slope<T>(p.act, take(1, k, c), A[k], dA[k]);
            if (pre) {
                // h again from the inputs, its normalised form, and the norm's backward sums
                V8 h = post ? weighted(k, c) : yn[k];
                if (act) h = mul(h, A[k]);
                h = mul(h, sc(k, c));
                if (has_x) h = fma(take(2, k, c), p.alpha, h);
                hn[k] = pre == 2 ? centre(h, st.z, st.w) : mul(h, st.w);
                c.mask(hn[k]);
                gr[k] = take(3, k, c);
                if (live) {
                    add_to(3, k, gr[k], hn[k]);
                    if (pre == 2) add_to(4, k, gr[k], one);
                }
                gr[k] = mul(gr[k], w2(k, c));
                if (pre == 2) a += c.counted(total(gr[k]));
                c2 += c.counted(dot(gr[k], hn[k]));
            }
        }
        float ma = 0.f, mc = 0.f;
        if (pre) {
            const float2 m = pre == 2 ? grp.sum2(a, c2) : make_float2(0.f, grp.sum1(c2));
            ma = m.x * inv;
            mc = m.y * inv;
        }
        a = c2 = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D, p.dh);
            // gr = dh + r (dn - mean(dn) - n mean(dn n)), the gradient of h
            gr[k] = pre == 2 ? centre(fma(hn[k], -mc, gr[k]), ma, st.w) : pre ? mul(fma(hn[k], -mc, gr[k]), st.w) : splat(0.f);
            if (has_dh) gr[k] = add(gr[k], take(4, k, c));
            if (p.dx && live) c.store(static_cast<T *>(p.dx) + off, mul(gr[k], p.alpha));
            const V8 pv = post ? weighted(k, c) : yn[k];
            if (live) add_to(2, k, act ? mul(gr[k], A[k]) : gr[k], pv);
            gr[k] = mul(gr[k], sc(k, c));
            if (act) {
                if (live) c.store(static_cast<T *>(p.dg) + off, mul(mul(gr[k], pv), dA[k]));
                gr[k] = mul(gr[k], A[k]);
            }
            // gr is now dp
            if (post) {
                if (live) {
                    add_to(0, k, gr[k], yn[k]);
                    if (post == 2) add_to(1, k, gr[k], one);
                }
                gr[k] = mul(gr[k], w1(k, c));
                c.mask(gr[k]);
                if (post == 2) a += c.counted(total(gr[k]));
                c2 += c.counted(dot(gr[k], yn[k]));
            }
        }
        fetch(base + kAhead * stride, stage);
        if (post) {
            const float2 m = post == 2 ? grp.sum2(a, c2) : make_float2(0.f, grp.sum1(c2));
            ma = m.x * inv;
            mc = m.y * inv;
        }
        // dy is contiguous in y's own layout
        T *dy = static_cast<T *>(p.dy) + off;
        if (p.dh < p.D) {
            const uint32_t row = BLOCK ? base : min(base + mine, p.rows - 1), b = p.byT(row), t = row - b * p.T;
            dy = static_cast<T *>(p.dy) + (size_t)b * p.T * p.D + (size_t)t * p.dh;
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D, p.dh);
            if (post) gr[k] = post == 2 ? centre(fma(yn[k], -mc, gr[k]), ma, st.y) : mul(fma(yn[k], -mc, gr[k]), st.y);
            if (live) c.store_heads(dy, p.dh, (long long)p.T * p.dh, dyoff[k], gr[k]);
        }
    }
    if (p.nvec == 0) return;
    float *part = p.part + (size_t)blockIdx.x * p.nvec * p.D;
    if constexpr (!BLOCK) __syncthreads();
#pragma unroll
    for (int i = 0; i < 5; ++i) {
        if (p.slot[i] < 0) continue;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const C c(r, k, lanes, p.D, p.dh);
            V8 s;
            if constexpr (WIDE) {
#pragma unroll
                for (int j = 0; j < kP; ++j) s.p[j] = accs[((p.slot[i] * K + k) * kP + j) * threads + tid];
            } else if constexpr (BLOCK) {
                s = acc[i][k];
            } else {
                // the block's row groups, added in order
#pragma unroll
                for (int j = 0; j < kP; ++j) accs[j * threads + tid] = acc[i][k].p[j];
                __syncthreads();
                s = splat(0.f);
                if (tid < lanes)
#pragma unroll
                    for (int j = 0; j < kP; ++j)
                        for (int m = r; m < threads; m += lanes) s.p[j] = __fadd2_rn(s.p[j], accs[j * threads + m]);
                __syncthreads();
            }
            const float *f = &s.p[0].x;
            if (BLOCK || tid < lanes)
#pragma unroll
                for (int j = 0; j < kC; ++j)
                    if (VEC ? c.has(0) : c.has(j / G)) part[(size_t)p.slot[i] * p.D + c.feature(j)] = f[j];
        }
    }
}

// ------------------------------------------------------------------------ launch

// Blocks of an SM for this kernel and shared memory (asked once for each).
template <typename P> int resident(void (*kernel)(P), int threads, int smem)
{
    static std::mutex mu;
    static struct {
        void (*k)(P);
        int dev, threads, smem, n;
    } memo[128];
    static int used = 0;
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (memo[i].k == kernel && memo[i].dev == dev && memo[i].threads == threads && memo[i].smem == smem) return memo[i].n;
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess || n < 1) n = 1;
    if (used < 128) memo[used++] = {kernel, dev, threads, smem, n};
    return n;
}

// Launches with as many blocks as the GPU holds at once (no more than limit, if any).
template <typename P>
int launch(void (*kernel)(P), const P &p, const NormShape &s, int limit, int smem, cudaStream_t st, int *blocks)
{
    // with the static part, past the 48 KB that need no asking
    if (smem > 40 * 1024 && !allow_shared(kernel, smem)) return -4;
    const long long per = s.block ? 1 : s.threads / s.lanes, groups = (p.rows + per - 1) / per;
    long long n = (long long)kSMs * resident(kernel, s.threads, smem);
    if (limit > 0 && n > limit) n = limit;
    if (n > groups) n = groups;
    *blocks = (int)n;
    kernel<<<(int)n, s.threads, smem, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <typename T, int G, int POST, int PRE, int ACT>
int run_fwd(const NormFwdParams &p, const NormShape &s, cudaStream_t st)
{
    using C = Chunk<T, G>;
    const int smem = C::VEC ? C::kAhead * 3 * s.K * C::kUnits * s.threads * 16 : 0;
    int n;
    if (!s.block) return launch(ttt_block_norm_fwd_kernel<T, G, 1, false, POST, PRE, ACT>, p, s, 0, smem, st, &n);
    return s.K == 1 ? launch(ttt_block_norm_fwd_kernel<T, G, 1, true, POST, PRE, ACT>, p, s, 0, smem, st, &n)
                    : launch(ttt_block_norm_fwd_kernel<T, G, 2, true, POST, PRE, ACT>, p, s, 0, smem, st, &n);
}

template <typename T, int G, int POST, int PRE, int ACT>
int run_bwd(const NormBwdParams &p, const NormShape &s, int limit, cudaStream_t st, int *blocks)
{
    using C = Chunk<T, G>;
    const int sums = s.block ? 0 : kC * 4, smem = ((C::VEC ? C::kAhead * (5 * s.K * C::kUnits + 1) * 16 : 0) + sums) * s.threads;
    if constexpr (C::VEC)
        if (s.K == 2)
            return launch(ttt_block_norm_bwd_kernel<T, G, 2, true, 256, POST, PRE, ACT>, p, s, limit, smem, st, blocks);
    if (!s.block) return launch(ttt_block_norm_bwd_kernel<T, G, 1, false, 128, POST, PRE, ACT>, p, s, limit, smem, st, blocks);
    return s.threads <= 384
               ? launch(ttt_block_norm_bwd_kernel<T, G, 1, true, 384, POST, PRE, ACT>, p, s, limit, smem, st, blocks)
               : launch(ttt_block_norm_bwd_kernel<T, G, 1, true, 512, POST, PRE, ACT>, p, s, limit, smem, st, blocks);
}

// Past 4096 features: sums in shared memory, the parts by the parameters.
template <typename T, int G>
int run_bwd_wide(const NormBwdParams &p, const NormShape &s, int limit, cudaStream_t st, int *blocks)
{
    const int smem = p.nvec * 2 * kC * 4 * s.threads;
    return launch(ttt_block_norm_bwd_kernel<T, G, 2, true, 512, -1, -1, -1>, p, s, limit, smem, st, blocks);
}

template <typename T> int norm_fwd(const NormFwdParams &p, const NormShape &s, int group, cudaStream_t st)
{
    if (group < kC) return group == 2 ? run_fwd<T, 2, -1, -1, -1>(p, s, st) : run_fwd<T, 1, -1, -1, -1>(p, s, st);
    switch (p.post * 6 + p.pre * 2 + (p.act ? 1 : 0)) {
    case 0: return run_fwd<T, kC, 0, 0, 0>(p, s, st);
    case 1: return run_fwd<T, kC, 0, 0, 1>(p, s, st);
    case 2: return run_fwd<T, kC, 0, 1, 0>(p, s, st);
    case 3: return run_fwd<T, kC, 0, 1, 1>(p, s, st);
    case 4: return run_fwd<T, kC, 0, 2, 0>(p, s, st);
    case 5: return run_fwd<T, kC, 0, 2, 1>(p, s, st);
    case 6: return run_fwd<T, kC, 1, 0, 0>(p, s, st);
    case 7: return run_fwd<T, kC, 1, 0, 1>(p, s, st);
    case 8: return run_fwd<T, kC, 1, 1, 0>(p, s, st);
    case 9: return run_fwd<T, kC, 1, 1, 1>(p, s, st);
    case 10: return run_fwd<T, kC, 1, 2, 0>(p, s, st);
    case 11: return run_fwd<T, kC, 1, 2, 1>(p, s, st);
    case 12: return run_fwd<T, kC, 2, 0, 0>(p, s, st);
    case 13: return run_fwd<T, kC, 2, 0, 1>(p, s, st);
    case 14: return run_fwd<T, kC, 2, 1, 0>(p, s, st);
    case 15: return run_fwd<T, kC, 2, 1, 1>(p, s, st);
    case 16: return run_fwd<T, kC, 2, 2, 0>(p, s, st);
    default: return run_fwd<T, kC, 2, 2, 1>(p, s, st);
    }
}

template <typename T>
int norm_bwd(const NormBwdParams &p, const NormShape &s, int group, int limit, cudaStream_t st, int *blocks)
{
    if (s.threads > 256 && s.K > 1)
        return group == kC  ? run_bwd_wide<T, kC>(p, s, limit, st, blocks)
               : group == 2 ? run_bwd_wide<T, 2>(p, s, limit, st, blocks)
                            : run_bwd_wide<T, 1>(p, s, limit, st, blocks);
    if (group < kC)
        return group == 2 ? run_bwd<T, 2, -1, -1, -1>(p, s, limit, st, blocks) : run_bwd<T, 1, -1, -1, -1>(p, s, limit, st, blocks);
    switch (p.post * 6 + p.pre * 2 + (p.act ? 1 : 0)) {
    case 0: return run_bwd<T, kC, 0, 0, 0>(p, s, limit, st, blocks);
    case 1: return run_bwd<T, kC, 0, 0, 1>(p, s, limit, st, blocks);
    case 2: return run_bwd<T, kC, 0, 1, 0>(p, s, limit, st, blocks);
    case 3: return run_bwd<T, kC, 0, 1, 1>(p, s, limit, st, blocks);
    case 4: return run_bwd<T, kC, 0, 2, 0>(p, s, limit, st, blocks);
    case 5: return run_bwd<T, kC, 0, 2, 1>(p, s, limit, st, blocks);
    case 6: return run_bwd<T, kC, 1, 0, 0>(p, s, limit, st, blocks);
    case 7: return run_bwd<T, kC, 1, 0, 1>(p, s, limit, st, blocks);
    case 8: return run_bwd<T, kC, 1, 1, 0>(p, s, limit, st, blocks);
    case 9: return run_bwd<T, kC, 1, 1, 1>(p, s, limit, st, blocks);
    case 10: return run_bwd<T, kC, 1, 2, 0>(p, s, limit, st, blocks);
    case 11: return run_bwd<T, kC, 1, 2, 1>(p, s, limit, st, blocks);
    case 12: return run_bwd<T, kC, 2, 0, 0>(p, s, limit, st, blocks);
    case 13: return run_bwd<T, kC, 2, 0, 1>(p, s, limit, st, blocks);
    case 14: return run_bwd<T, kC, 2, 1, 0>(p, s, limit, st, blocks);
    case 15: return run_bwd<T, kC, 2, 1, 1>(p, s, limit, st, blocks);
    case 16: return run_bwd<T, kC, 2, 2, 0>(p, s, limit, st, blocks);
    default: return run_bwd<T, kC, 2, 2, 1>(p, s, limit, st, blocks);
    }
}

}  // namespace
}  // namespace ttt
