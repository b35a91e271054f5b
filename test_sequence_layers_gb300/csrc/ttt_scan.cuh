// ttt_scan.cuh -- what the selective scan's kernels share: its launch parameters, the
// rate and gate functions, and sums across lanes.
#pragma once

#include "ttt_internal.h"
#include "ttt_vec.cuh"

namespace ttt {
namespace scan {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// a truth value known at compile time
template <bool V> struct Is {
    static constexpr bool value = V;
};

struct Params {
    const void *x, *delta, *z, *Bm, *Cm, *dy;
    const unsigned char *reset;
    const float *A, *D, *bias;
    long long xs[2], ds[2], zs[2], dys[2], bs[3], cs[3];
    int B, T, C, N, G, softplus;
    int cpg;      // channels of a group
    int blocks;   // channel blocks of a group
    int segs, seg_len;       // pieces of the sequence, tokens of one (a multiple of the chunk)
    int chunks;
    const float *start;      // state before (backward: gradient behind) each piece [B,segs,C,N], or null
    float *y_state;          // h_last or null
    float *states;           // forward: written; backward: read
    void *y;
    float *H, *rate_sum;     // a piece's map h -> exp(A rate_sum) h + H: [B,segs,C,N], [B,segs,C]
    int *cut;                // [B,segs]: a reset inside
    // backward
    void *dx, *ddelta, *dz;
    float *dh0, *bc_part, *a_part, *v_part;
};

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// exp(-v) of a gate or a rate's argument.  bf16 tensors: one ex2 of a rounded product, off by
// |v| 2^-24 of itself, far below the outputs' rounding.  fp32 tensors: CUDA's expf.
template <typename T> __device__ __forceinline__ float exp_neg(float v)
{
    return sizeof(T) == 2 ? ex2(-kLog2e * v) : expf(-v);
}
template <typename T> __device__ __forceinline__ float sigmoid(float v) { return rcp(1.f + exp_neg<T>(v)); }

// log(1 + e) for 0 <= e <= 1 as e P(e), P the Chebyshev interpolation of log(1 + e) / e in
// e on [0, 1]: relative error below 2^-22, also where e is small.
__host__ __device__ constexpr float log1p_term(int i)
{
    constexpr float c[] = {1.f, -4.999989271e-01f, 3.332971036e-01f, -2.495161593e-01f, 1.966327429e-01f,
                           -1.526966691e-01f, 1.054362357e-01f, -5.637361109e-02f, 1.954252645e-02f, -3.176057013e-03f};
    return c[i];
}
__device__ __forceinline__ float log1p_unit(float e)
{
    float p = log1p_term(9);
#pragma unroll
    for (int i = 8; i >= 0; --i) p = fmaf(p, e, log1p_term(i));
    return e * p;
}
__device__ __forceinline__ float2 log1p_unit(float2 e)
{
    float2 p = make_float2(log1p_term(9), log1p_term(9));
#pragma unroll
    for (int i = 8; i >= 0; --i) p = __ffma2_rn(p, e, make_float2(log1p_term(i), log1p_term(i)));
    return __fmul2_rn(e, p);
}

// max(v, 0) + log(1 + exp(-|v|)).  Nothing overflows.
template <typename T> __device__ __forceinline__ float softplus(float v)
{
    const float l = log1p_unit(exp_neg<T>(fabsf(v)));
    return v > 0.f ? v + l : v <= 0.f ? l : v;  // NaN stays
}

// One value, or V neighbouring ones, of a token tensor in fp32.
template <typename T> __device__ __forceinline__ float get(const T *p)
{
    Pack<T, 1> q;
    float v[1];
    q.load(p);
    unpack(q, v);
    return v[0];
}
template <typename T> __device__ __forceinline__ void put(T *p, float x)
{
    Pack<T, 1> q;
    const float v[1] = {x};
    pack(q, v);
    q.store(p);
}

// Rates of V values, two at a time (the polynomial is most of the work).
template <typename T, int V> __device__ __forceinline__ void softplus_all(float (&v)[V])
{
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 e = make_float2(exp_neg<T>(fabsf(v[j])), exp_neg<T>(fabsf(v[j + 1])));
            const float2 l = log1p_unit(e);
            v[j] = v[j] > 0.f ? v[j] + l.x : v[j] <= 0.f ? l.x : v[j];  // NaN stays
            v[j + 1] = v[j + 1] > 0.f ? v[j + 1] + l.y : v[j + 1] <= 0.f ? l.y : v[j + 1];
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = softplus<T>(v[j]);
    }
}

// V floats to or from shared memory, four at a time where there are four.
template <int V> __device__ __forceinline__ void put_floats(float *p, const float (&v)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 4) *reinterpret_cast<float4 *>(p + j) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) p[j] = v[j];
    }
}
template <int V> __device__ __forceinline__ void get_floats(const float *p, float (&v)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(p + j);
            v[j] = q.x;
            v[j + 1] = q.y;
            v[j + 2] = q.z;
            v[j + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = p[j];
    }
}

// Where entry i of a row in shared memory lies: where bit 1 of t is set, its groups of four are
// exchanged two and two, so that threads which store eight entries each, four at a time, meet
// different banks (t: the token for rows of 16, i / 16 for rows of 64).
__device__ __forceinline__ int turned(int i, int t) { return i ^ ((t & 2) << 1); }
template <int V> __device__ __forceinline__ void put_turned(float *row, int i, int t, const float (&v)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 4) *reinterpret_cast<float4 *>(row + turned(i + j, t)) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) row[turned(i + j, t)] = v[j];
    }
}
template <int V> __device__ __forceinline__ void get_turned(const float *row, int i, int t, float (&v)[V])
{
    if constexpr (V % 4 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            const float4 q = *reinterpret_cast<const float4 *>(row + turned(i + j, t));
            v[j] = q.x;
            v[j + 1] = q.y;
            v[j + 2] = q.z;
            v[j + 3] = q.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = row[turned(i + j, t)];
    }
}

// Sums of M values over the L lanes that differ in the bits S, 2 S, .. (L/2) S of the lane
// number, spread over them: while more than one value is left every step halves the values a
// lane keeps (the lane with the bit clear the first half), after that all lanes add up.
// Value i ends in v[i % K] (K = max(M / L, 1)) of the lanes whose bits, the highest step
// first, spell i / K (K > 1 or M == L), or of every lane they do not tell apart.
template <int M, int L, int S> __device__ __forceinline__ void spread_sum(float (&v)[M])
{
    const int lane = threadIdx.x & 31;
    int m = M;
#pragma unroll
    for (int s = L / 2 * S; s >= S; s >>= 1) {
        if (m > 1) {
            m >>= 1;
            const bool up = lane & s;
#pragma unroll
            for (int i = 0; i < M / 2; ++i)
                if (i < m) {
                    const float give = up ? v[i] : v[i + m], keep = up ? v[i + m] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, s);
                }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], s);
        }
    }
}

// A channel's four states of each lane, two and two.
struct Quad {
    float2 a, b;
};
__device__ __forceinline__ Quad quad(float4 v) { return {{v.x, v.y}, {v.z, v.w}}; }
__device__ __forceinline__ float4 four(const Quad &q) { return make_float4(q.a.x, q.a.y, q.b.x, q.b.y); }

// states n0 .. n0 + 3 of a row of N, zeros past its end
__device__ __forceinline__ float4 load_states(const float *row, int n0, int N)
{
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (N % 4 == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
        if (n0 < N) v = *reinterpret_cast<const float4 *>(row + n0);
        return v;
    }
    float *f = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n0 + i < N) f[i] = row[n0 + i];
    return v;
}
__device__ __forceinline__ void store_states(float *row, int n0, int N, float4 v)
{
    if (N % 4 == 0 && (reinterpret_cast<uintptr_t>(row) & 15) == 0) {
        if (n0 < N) *reinterpret_cast<float4 *>(row + n0) = v;
        return;
    }
    const float *f = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (n0 + i < N) row[n0 + i] = f[i];
}

// 2^(d A), A in units of log2 e.  ex2 of arguments between -1 and 0 comes out 5e-9 to 2.2e-8
// too low on average (measured), always the same way, which a slow state sums up over the
// thousand tokens that it remembers; the addend, which costs nothing in the product, leaves
// 9e-9 of either sign.  Where d A is 0 the decay is 1 exactly (measured up to addends of 1.1e-7).
constexpr float kCenter = 2e-8f;
__device__ __forceinline__ float2 decay2(float2 d, float2 A)
{
    const float2 p = __ffma2_rn(d, A, make_float2(kCenter, kCenter));
    return make_float2(ex2(p.x), ex2(p.y));
}
__device__ __forceinline__ Quad decays(float d, const Quad &A)
{
    const float2 dd = make_float2(d, d);
    return {decay2(dd, A.a), decay2(dd, A.b)};
}
__device__ __forceinline__ void step(Quad &h, float d, float u, const Quad &A, float4 Bt)
{
    const Quad a = decays(d, A);
    const float2 uu = make_float2(u, u);
    h.a = __ffma2_rn(a.a, h.a, __fmul2_rn(uu, make_float2(Bt.x, Bt.y)));
    h.b = __ffma2_rn(a.b, h.b, __fmul2_rn(uu, make_float2(Bt.z, Bt.w)));
}
// s += C . h, two and two (first: s = C . h)
__device__ __forceinline__ void dot(float2 &s, const Quad &h, float4 Ct, bool first)
{
    const float2 lo = make_float2(Ct.x, Ct.y);
    s = first ? __fmul2_rn(h.a, lo) : __ffma2_rn(h.a, lo, s);
    s = __ffma2_rn(h.b, make_float2(Ct.z, Ct.w), s);
}


// lanes of a channel, four states each
inline int lanes(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }

// A sequence of `chunks` cut into pieces so that warps x pieces comes to `want`, pieces of at
// least `least` chunks.  Fewer than three are not asked for: their halves' own maps cost what they gain.
// (Three of four chunks, in the backward pass, come to two by rounding.)
inline ScanPieces cut(int chunks, long long warps, long long want, int least)
{
    long long segs = warps > 0 ? want / warps : 1;
    if (segs > chunks / least) segs = chunks / least;
    if (segs > 65535) segs = 65535;
    if (segs < 3) segs = 1;
    const int per = (int)((chunks + segs - 1) / segs);
    return {per > 0 ? (chunks + per - 1) / per : 1, per * kScanChunk};
}

inline void params(const ScanArgs &a, Params &p)
{
    p.x = a.x;
    p.delta = a.delta;
    p.z = a.z;
    p.Bm = a.Bm;
    p.Cm = a.Cm;
    p.dy = a.dy;
    p.reset = a.reset;
    p.A = a.A;
    p.D = a.D;
    p.bias = a.bias;
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i];
        p.ds[i] = a.ds[i];
        p.zs[i] = a.zs[i];
        p.dys[i] = a.dys[i];
    }
    for (int i = 0; i < 3; ++i) {
        p.bs[i] = a.bs[i];
        p.cs[i] = a.cs[i];
    }
    p.B = a.B;
    p.T = a.T;
    p.C = a.C;
    p.N = a.N;
    p.G = a.G;
    p.softplus = a.softplus;
    p.cpg = a.C / a.G;
    p.chunks = (a.T + kScanChunk - 1) / kScanChunk;
    p.states = a.states;
}

// May every tensor be moved 16 bytes at a time: pointers, strides, a group's channels and
// a row of states multiples of them.  One answer for all: where B and C alone are not aligned, or a
// row of states is not whole, the token tensors move one element at a time too.
inline bool wide(const ScanArgs &a)
{
    const int es = a.bf16 ? 2 : 4, V = 16 / es;
    long long mask = (a.C / a.G) | a.N;
    for (const void *q : {a.x, a.delta, a.z, a.Bm, a.Cm, a.dy, (const void *)a.y, (const void *)a.dx, (const void *)a.ddelta, (const void *)a.dz}) {
        if (reinterpret_cast<uintptr_t>(q) % 16) return false;
    }
    for (int i = 0; i < 2; ++i) mask |= a.xs[i] | a.ds[i] | a.zs[i] | a.dys[i];
    for (int i = 0; i < 3; ++i) mask |= a.bs[i] | a.cs[i];
    return mask % V == 0;
}

}  // namespace scan
}  // namespace ttt
