// ttt_recurrence.cu -- the gated linear recurrence of every channel,
//     h_t = a_t h_{t-1} + c_t x_t,
// a = f, c = 1 (decay), a = sigma(f), c = 1 (sigmoid) or a = sigma(f), c = 1 - a (mix: the
// TTT layer with a constant as its inner model, w <- w - eta (w - x), eta = 1 - a, one
// rate a channel).  A reset before token t makes h_{t-1} zero there.  Backward:
//     s_t = dh_t + r_{t+1},  r_t = a_t s_t,  r_T = dh_last,  dh0 = r_0,
//     dx = c s,  dL/da = s (h_{t-1} [- x_t for mix]),  df = dL/da a (1 - a) unless a = f,
// with h_{t-1} computed again from the states that the forward pass leaves every
// kRecurChunk tokens: no rounded h is read, and no more bytes than reading it would take.
#include "ttt_internal.h"
#include "ttt_vec.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 64;

struct RecurParams {
    const void *x, *f, *dh;
    const unsigned char *reset;
    const float *h0, *dh_last, *states_in;
    void *h, *dx, *df;
    float *h_last, *states, *dh0;
    long long xs[2], fs[2], ds[2];
    int B, T, C, chunks;
    int cluster, cblocks;  // tile kernels: blocks of a cluster, channel blocks of a batch entry
};

// a and 1 - a, each accurate on its own: with e = exp(-|f|) <= 1 the smaller of the two is
// e / (1 + e) and the larger 1 / (1 + e), so neither is a difference and nothing overflows.
template <typename T, int MODE> __device__ __forceinline__ void gate(float f, float &a, float &eta)
{
    if (MODE == kRecurDecay) {
        a = f;
        eta = 1.f;
        return;
    }
    // bf16 tensors: exp good to 2^-20; fp32: the accurate one
    const float e = sizeof(T) == 2 ? __expf(-fabsf(f)) : expf(-fabsf(f));
    const float big = __fdividef(1.f, 1.f + e), small = e * big;
    a = f > 0.f ? big : small;
    eta = f > 0.f ? small : big;
}

template <typename T> __device__ __forceinline__ float ld1(const T *p)
{
    Pack<T, 1> q;
    float v[1];
    q.load(p);
    unpack(q, v);
    return v[0];
}
template <typename T> __device__ __forceinline__ void st1(T *p, float x)
{
    Pack<T, 1> q;
    const float v[1] = {x};
    pack(q, v);
    q.store(p);
}

// One thread a channel, token after token: decoding steps and lengths up to kS.
template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) ttt_recurrence_fwd_kernel(const __grid_constant__ RecurParams p)
{
    const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (c >= p.C) return;
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *f = static_cast<const T *>(p.f) + b * p.fs[0] + c;
    float h = p.h0 ? p.h0[(size_t)b * p.C + c] : 0.f;
    for (int t = 0; t < p.T; ++t) {
        if (p.states && t % kRecurChunk == 0) p.states[((size_t)b * p.chunks + t / kRecurChunk) * p.C + c] = h;
        if (p.reset && p.reset[(size_t)b * p.T + t]) h = 0.f;
        const float xv = ld1(x + t * p.xs[1]);
        float a, eta;
        gate<T, MODE>(ld1(f + t * p.fs[1]), a, eta);
        h = fmaf(a, h, MODE == kRecurMix ? eta * xv : xv);
        st1(static_cast<T *>(p.h) + ((size_t)b * p.T + t) * p.C + c, h);
    }
    if (p.h_last) p.h_last[(size_t)b * p.C + c] = h;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kThreads) ttt_recurrence_bwd_kernel(const __grid_constant__ RecurParams p)
{
    __shared__ float before[kRecurChunk][kThreads];  // h_{t-1} of the chunk's tokens
    const int c = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
    if (c >= p.C) return;
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *f = static_cast<const T *>(p.f) + b * p.fs[0] + c;
    const T *dh = static_cast<const T *>(p.dh) + b * p.ds[0] + c;
    const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;
    float r = p.dh_last ? p.dh_last[(size_t)b * p.C + c] : 0.f;
    for (int ch = p.chunks - 1; ch >= 0; --ch) {
        const int t0 = ch * kRecurChunk, t1 = min(p.T, t0 + kRecurChunk);
        float h = p.states_in[((size_t)b * p.chunks + ch) * p.C + c];
        for (int t = t0; t < t1; ++t) {
            if (reset && reset[t]) h = 0.f;
            before[t - t0][threadIdx.x] = h;
            const float xv = ld1(x + t * p.xs[1]);
            float a, eta;
            gate<T, MODE>(ld1(f + t * p.fs[1]), a, eta);
            h = fmaf(a, h, MODE == kRecurMix ? eta * xv : xv);
        }
        for (int t = t1 - 1; t >= t0; --t) {
            const float s = (p.dh ? ld1(dh + t * p.ds[1]) : 0.f) + r, hp = before[t - t0][threadIdx.x];
            float a, eta;
            gate<T, MODE>(ld1(f + t * p.fs[1]), a, eta);
            float da = s * hp;
            if (MODE == kRecurMix) da = s * (hp - ld1(x + t * p.xs[1]));
            if (MODE != kRecurDecay) da *= a * eta;
            const size_t o = ((size_t)b * p.T + t) * p.C + c;
            st1(static_cast<T *>(p.dx) + o, MODE == kRecurMix ? eta * s : s);
            st1(static_cast<T *>(p.df) + o, da);
            r = reset && reset[t] ? 0.f : a * s;
        }
    }
    if (p.dh0) p.dh0[(size_t)b * p.C + c] = r;
}

// ------------------------------------------------------------- tiles along time
//
// A warp takes kS tokens of 32 CPL channels, a block of kW warps a tile of kRecurChunk
// tokens, a cluster of P blocks P neighbouring tiles, and the cluster walks along the
// sequence in rounds of P tiles, the next round's loads in flight.  Every tensor is read
// once: the round's data stay in registers while the warps' maps h -> A h + H (the
// product of the decays, and the tokens' own contribution) are joined, in shared memory
// inside the block and through the cluster's distributed shared memory between blocks.
// The join order is fixed by position, so results do not depend on timing.  NaN and
// infinities do not pass a reset: a map with a reset in it (cut) ignores its input.

constexpr int kS = 16, kW = 8;
static_assert(kS * kW == kRecurChunk, "a tile is one stored-state chunk");

// this block's rank in its cluster, cluster barrier, stores to another block's shared memory
__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void st_remote(const void *local, uint32_t rank, float v)
{
    uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(local)), r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(r), "f"(v) : "memory");
}

// The maps of a round, double-buffered over rounds: per warp (w) and per block of the
// cluster (t).  One barrier a round is enough: a buffer is written again two rounds later,
// behind the next round's barrier.
template <int CPL, int NV> struct TileShared {
    float w[2][NV][kW][32 * CPL];
    float t[2][NV][8][32 * CPL];
    int wcut[2][kW];
    float tcut[2][8];
};

template <int CPL> __device__ __forceinline__ void lds(const float *p, float (&v)[CPL])
{
    if constexpr (CPL == 2) {
        const float2 q = *reinterpret_cast<const float2 *>(p);
        v[0] = q.x;
        v[1] = q.y;
    } else {
        v[0] = *p;
    }
}

// The reset bits of a warp's tokens t0 .. t0 + n - 1.
__device__ __forceinline__ unsigned reset_bits(const unsigned char *reset, int t0, int n, int lane)
{
    return __ballot_sync(0xffffffffu, lane < n && reset[t0 + lane] != 0);
}

template <typename T, int MODE, int CPL, bool RESET>
__global__ void __launch_bounds__(32 * kW, 2) ttt_recurrence_fwd_tile_kernel(const __grid_constant__ RecurParams p)
{
    constexpr int CH = 32 * CPL;
    __shared__ TileShared<CPL, 2> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = p.cluster, rank = P > 1 ? (int)cluster_rank() : 0;
    const int chain = blockIdx.x / P, b = chain / p.cblocks, c = (chain % p.cblocks) * CH + lane * CPL;
    const bool on = c < p.C;  // CPL divides C
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *f = static_cast<const T *>(p.f) + b * p.fs[0] + c;
    const unsigned char *reset = RESET ? p.reset + (size_t)b * p.T : nullptr;
    const size_t bc = (size_t)b * p.C + c;
    float carry[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) carry[j] = on && p.h0 ? p.h0[bc + j] : 0.f;

    Pack<T, CPL> fr[kS], xr[kS];
    auto fetch = [&](int t0) {
        const T *fp = f + t0 * p.fs[1], *xp = x + t0 * p.xs[1];
#pragma unroll
        for (int s = 0; s < kS; ++s)
            if (on && t0 + s < p.T) {
                fr[s].load(fp + s * p.fs[1]);
                xr[s].load(xp + s * p.xs[1]);
            }
    };
    const int rounds = (p.chunks + P - 1) / P;
    int t0 = rank * kRecurChunk + warp * kS, buf = 0;
    fetch(t0);
    if (P > 1) cluster_barrier();  // every block runs before its shared memory is written
    for (int round = 0; round < rounds; ++round, t0 += P * kRecurChunk, buf ^= 1) {
        const int n = min(max(p.T - t0, 0), kS);  // this warp's tokens
        const unsigned cuts = RESET ? reset_bits(reset, t0, n, lane) : 0u;
        float a[kS][CPL], u[kS][CPL];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            float fv[CPL], xv[CPL];
            unpack(fr[s], fv);
            unpack(xr[s], xv);
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                float eta;
                gate<T, MODE>(fv[j], a[s][j], eta);
                u[s][j] = MODE == kRecurMix ? eta * xv[j] : xv[j];
            }
        }
        if (round + 1 < rounds) fetch(t0 + P * kRecurChunk);
        if (n < kS) {  // tokens past the end: the identity
#pragma unroll
            for (int s = 0; s < kS; ++s)
                if (s >= n)
#pragma unroll
                    for (int j = 0; j < CPL; ++j) {
                        a[s][j] = 1.f;
                        u[s][j] = 0.f;
                    }
        }
        // the warp's map
        float A[CPL], H[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            A[j] = 1.f;
            H[j] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (RESET && (cuts >> s & 1u))
#pragma unroll
                for (int j = 0; j < CPL; ++j) H[j] = 0.f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                H[j] = fmaf(a[s][j], H[j], u[s][j]);
                A[j] *= a[s][j];
            }
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            sh.w[buf][0][warp][lane * CPL + j] = A[j];
            sh.w[buf][1][warp][lane * CPL + j] = H[j];
        }
        if (RESET && lane == 0) sh.wcut[buf][warp] = cuts != 0;
        __syncthreads();
        // the state before this block's tile, and the next round's
        float st[CPL];
        if (P > 1) {
            float TA[CPL], TH[CPL];
            bool cut = false;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                TA[j] = 1.f;
                TH[j] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < kW; ++i) {
                float wa[CPL], wh[CPL];
                lds<CPL>(&sh.w[buf][0][i][lane * CPL], wa);
                lds<CPL>(&sh.w[buf][1][i][lane * CPL], wh);
                const bool ci = RESET && sh.wcut[buf][i];
                cut |= ci;
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    TH[j] = ci ? wh[j] : fmaf(wa[j], TH[j], wh[j]);
                    TA[j] *= wa[j];
                }
            }
            if (warp < P) {  // warp i tells block i
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    st_remote(&sh.t[buf][0][rank][lane * CPL + j], warp, TA[j]);
                    st_remote(&sh.t[buf][1][rank][lane * CPL + j], warp, TH[j]);
                }
                if (RESET && lane == 0) st_remote(&sh.tcut[buf][rank], warp, cut ? 1.f : 0.f);
            }
            cluster_barrier();
#pragma unroll
            for (int j = 0; j < CPL; ++j) st[j] = carry[j];
            for (int i = 0; i < P; ++i) {
                float wa[CPL], wh[CPL];
                lds<CPL>(&sh.t[buf][0][i][lane * CPL], wa);
                lds<CPL>(&sh.t[buf][1][i][lane * CPL], wh);
                const bool ci = RESET && sh.tcut[buf][i] != 0.f;
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    carry[j] = ci ? wh[j] : fmaf(wa[j], carry[j], wh[j]);
                    if (i < rank) st[j] = carry[j];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < CPL; ++j) st[j] = carry[j];
        }
        if (warp == 0 && p.states && on && n > 0)
#pragma unroll
            for (int j = 0; j < CPL; ++j)
                p.states[((size_t)b * p.chunks + t0 / kRecurChunk) * p.C + c + j] = st[j];
        // the state before this warp's tokens
        float h[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) h[j] = st[j];
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            float wa[CPL], wh[CPL];
            lds<CPL>(&sh.w[buf][0][i][lane * CPL], wa);
            lds<CPL>(&sh.w[buf][1][i][lane * CPL], wh);
            const bool ci = RESET && sh.wcut[buf][i];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                st[j] = ci ? wh[j] : fmaf(wa[j], st[j], wh[j]);
                if (i < warp) h[j] = st[j];
            }
        }
        if (P == 1)
#pragma unroll
            for (int j = 0; j < CPL; ++j) carry[j] = st[j];
        T *hp = static_cast<T *>(p.h) + ((size_t)b * p.T + t0) * p.C + c;
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (RESET && (cuts >> s & 1u))
#pragma unroll
                for (int j = 0; j < CPL; ++j) h[j] = 0.f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) h[j] = fmaf(a[s][j], h[j], u[s][j]);
            if (on && s < n) {
                Pack<T, CPL> q;
                pack(q, h);
                q.store(hp + (size_t)s * p.C);
            }
        }
    }
    if (p.h_last && on && rank == 0 && warp == 0)
#pragma unroll
        for (int j = 0; j < CPL; ++j) p.h_last[bc + j] = carry[j];
}

// Backward: the same tiles from the end of the sequence to its start.  The warps' maps
// carry three numbers a channel: the product A of the decays (shared by both
// directions), the forward contribution H, which brings h_{t-1} to every warp from the
// tile's stored state, and the backward one R of r -> A r + R.
template <typename T, int MODE, int CPL, bool RESET>
__global__ void __launch_bounds__(32 * kW) ttt_recurrence_bwd_tile_kernel(const __grid_constant__ RecurParams p)
{
    constexpr int CH = 32 * CPL;
    __shared__ TileShared<CPL, 3> sh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = p.cluster, rank = P > 1 ? (int)cluster_rank() : 0;
    const int chain = blockIdx.x / P, b = chain / p.cblocks, c = (chain % p.cblocks) * CH + lane * CPL;
    const bool on = c < p.C;
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *f = static_cast<const T *>(p.f) + b * p.fs[0] + c;
    const T *dh = static_cast<const T *>(p.dh) + b * p.ds[0] + c;
    const unsigned char *reset = RESET ? p.reset + (size_t)b * p.T : nullptr;
    const size_t bc = (size_t)b * p.C + c;
    float carry[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) carry[j] = on && p.dh_last ? p.dh_last[bc + j] : 0.f;

    Pack<T, CPL> fr[kS], xr[kS], dr[kS];
    float sr[CPL] = {};  // the tile's stored state
    auto fetch = [&](int tile) {
        const int t0 = tile * kRecurChunk + warp * kS;
        if (tile < 0 || tile >= p.chunks || !on) return;
#pragma unroll
        for (int j = 0; j < CPL; ++j) sr[j] = p.states_in[((size_t)b * p.chunks + tile) * p.C + c + j];
#pragma unroll
        for (int s = 0; s < kS; ++s)
            if (t0 + s < p.T) {
                fr[s].load(f + (t0 + s) * p.fs[1]);
                xr[s].load(x + (t0 + s) * p.xs[1]);
                if (p.dh) dr[s].load(dh + (t0 + s) * p.ds[1]);
            }
    };
    const int rounds = (p.chunks + P - 1) / P;
    // rank 0 holds the last tile of a round; tiles past the end are empty
    int tile = rounds * P - 1 - rank, buf = 0;
    fetch(tile);
    if (P > 1) cluster_barrier();
    for (int round = 0; round < rounds; ++round, tile -= P, buf ^= 1) {
        const int t0 = tile * kRecurChunk + warp * kS;
        const int n = min(max(p.T - t0, 0), kS);
        const unsigned cuts = RESET ? reset_bits(reset, t0, n, lane) : 0u;
        float a[kS][CPL], eta[kS][CPL], xv[kS][CPL], dv[kS][CPL], start[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) start[j] = sr[j];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            float fv[CPL];
            unpack(fr[s], fv);
            unpack(xr[s], xv[s]);
            unpack(dr[s], dv[s]);
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                gate<T, MODE>(fv[j], a[s][j], eta[s][j]);
                if (!p.dh) dv[s][j] = 0.f;
                if (s >= n) {
                    a[s][j] = 1.f;
                    eta[s][j] = xv[s][j] = dv[s][j] = 0.f;
                }
            }
        }
        if (round + 1 < rounds) fetch(tile - P);
        float A[CPL], H[CPL], R[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            A[j] = 1.f;
            H[j] = R[j] = 0.f;
        }
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (RESET && (cuts >> s & 1u))
#pragma unroll
                for (int j = 0; j < CPL; ++j) H[j] = 0.f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                H[j] = fmaf(a[s][j], H[j], MODE == kRecurMix ? eta[s][j] * xv[s][j] : xv[s][j]);
                A[j] *= a[s][j];
            }
        }
#pragma unroll
        for (int s = kS - 1; s >= 0; --s) {
#pragma unroll
            for (int j = 0; j < CPL; ++j) R[j] = a[s][j] * (dv[s][j] + R[j]);
            if (RESET && (cuts >> s & 1u))
#pragma unroll
                for (int j = 0; j < CPL; ++j) R[j] = 0.f;
        }
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            sh.w[buf][0][warp][lane * CPL + j] = A[j];
            sh.w[buf][1][warp][lane * CPL + j] = H[j];
            sh.w[buf][2][warp][lane * CPL + j] = R[j];
        }
        if (RESET && lane == 0) sh.wcut[buf][warp] = cuts != 0;
        __syncthreads();
        float st[CPL];  // r behind this block's tile
        if (P > 1) {
            float TA[CPL], TR[CPL];
            bool cut = false;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                TA[j] = 1.f;
                TR[j] = 0.f;
            }
#pragma unroll
            for (int i = kW - 1; i >= 0; --i) {
                float wa[CPL], wr[CPL];
                lds<CPL>(&sh.w[buf][0][i][lane * CPL], wa);
                lds<CPL>(&sh.w[buf][2][i][lane * CPL], wr);
                const bool ci = RESET && sh.wcut[buf][i];
                cut |= ci;
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    TR[j] = ci ? wr[j] : fmaf(wa[j], TR[j], wr[j]);
                    TA[j] *= wa[j];
                }
            }
            if (warp < P) {
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    st_remote(&sh.t[buf][0][rank][lane * CPL + j], warp, TA[j]);
                    st_remote(&sh.t[buf][2][rank][lane * CPL + j], warp, TR[j]);
                }
                if (RESET && lane == 0) st_remote(&sh.tcut[buf][rank], warp, cut ? 1.f : 0.f);
            }
            cluster_barrier();
#pragma unroll
            for (int j = 0; j < CPL; ++j) st[j] = carry[j];
            for (int i = 0; i < P; ++i) {
                float wa[CPL], wr[CPL];
                lds<CPL>(&sh.t[buf][0][i][lane * CPL], wa);
                lds<CPL>(&sh.t[buf][2][i][lane * CPL], wr);
                const bool ci = RESET && sh.tcut[buf][i] != 0.f;
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    carry[j] = ci ? wr[j] : fmaf(wa[j], carry[j], wr[j]);
                    if (i < rank) st[j] = carry[j];
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < CPL; ++j) st[j] = carry[j];
        }
        float h[CPL], r[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            h[j] = start[j];
            r[j] = st[j];
        }
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            float wa[CPL], wh[CPL];
            if (i < warp) {
                lds<CPL>(&sh.w[buf][0][i][lane * CPL], wa);
                lds<CPL>(&sh.w[buf][1][i][lane * CPL], wh);
                const bool ci = RESET && sh.wcut[buf][i];
#pragma unroll
                for (int j = 0; j < CPL; ++j) h[j] = ci ? wh[j] : fmaf(wa[j], h[j], wh[j]);
            }
        }
#pragma unroll
        for (int i = kW - 1; i >= 0; --i) {
            float wa[CPL], wr[CPL];
            lds<CPL>(&sh.w[buf][0][i][lane * CPL], wa);
            lds<CPL>(&sh.w[buf][2][i][lane * CPL], wr);
            const bool ci = RESET && sh.wcut[buf][i];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                st[j] = ci ? wr[j] : fmaf(wa[j], st[j], wr[j]);
                if (i > warp) r[j] = st[j];
            }
        }
        if (P == 1)
#pragma unroll
            for (int j = 0; j < CPL; ++j) carry[j] = st[j];
        // h_{t-1} forward, kept in place of x for what df needs of both
        float hb[kS][CPL];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (RESET && (cuts >> s & 1u))
#pragma unroll
                for (int j = 0; j < CPL; ++j) h[j] = 0.f;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                hb[s][j] = MODE == kRecurMix ? h[j] - xv[s][j] : h[j];
                h[j] = fmaf(a[s][j], h[j], MODE == kRecurMix ? eta[s][j] * xv[s][j] : xv[s][j]);
            }
        }
        const size_t o = ((size_t)b * p.T + t0) * p.C + c;
#pragma unroll
        for (int s = kS - 1; s >= 0; --s) {
            float gx[CPL], gf[CPL];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const float sv = dv[s][j] + r[j];
                r[j] = a[s][j] * sv;
                gx[j] = MODE == kRecurMix ? eta[s][j] * sv : sv;
                gf[j] = MODE == kRecurDecay ? sv * hb[s][j] : r[j] * hb[s][j] * eta[s][j];
            }
            if (RESET && (cuts >> s & 1u))
#pragma unroll
                for (int j = 0; j < CPL; ++j) r[j] = 0.f;
            if (on && s < n) {
                Pack<T, CPL> q;
                pack(q, gx);
                q.store(static_cast<T *>(p.dx) + o + (size_t)s * p.C);
                pack(q, gf);
                q.store(static_cast<T *>(p.df) + o + (size_t)s * p.C);
            }
        }
    }
    if (p.dh0 && on && rank == 0 && warp == 0)
#pragma unroll
        for (int j = 0; j < CPL; ++j) p.dh0[bc + j] = carry[j];
}

RecurParams params_of(const RecurArgs &a)
{
    RecurParams p = {};
    p.x = a.x;
    p.f = a.f;
    p.dh = a.dh;
    p.reset = a.reset;
    p.h0 = a.h0;
    p.dh_last = a.dh_last;
    p.states_in = a.states;
    p.h = a.h;
    p.dx = a.dx;
    p.df = a.df;
    p.h_last = a.h_last;
    p.states = a.states;
    p.dh0 = a.dh0;
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i];
        p.fs[i] = a.fs[i];
        p.ds[i] = a.ds[i];
    }
    p.B = a.B;
    p.T = a.T;
    p.C = a.C;
    p.chunks = (a.T + kRecurChunk - 1) / kRecurChunk;
    return p;
}

constexpr int kSMs = 152;

template <typename K> int launch_clusters(K kernel, const RecurParams &p, int blocks, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * kW);
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = p.cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p) == cudaSuccess ? 0 : -4;
}

template <typename T, int MODE, int CPL> int run_tiles(RecurParams p, bool bwd, cudaStream_t st)
{
    p.cblocks = (p.C + 32 * CPL - 1) / (32 * CPL);
    const long long chains = (long long)p.B * p.cblocks;
    p.cluster = 1;
    while (p.cluster < 8 && chains * p.cluster < 2 * kSMs && p.cluster < p.chunks) p.cluster *= 2;
    const int blocks = (int)(chains * p.cluster);
    if (bwd)
        return p.reset ? launch_clusters(ttt_recurrence_bwd_tile_kernel<T, MODE, CPL, true>, p, blocks, st)
                       : launch_clusters(ttt_recurrence_bwd_tile_kernel<T, MODE, CPL, false>, p, blocks, st);
    return p.reset ? launch_clusters(ttt_recurrence_fwd_tile_kernel<T, MODE, CPL, true>, p, blocks, st)
                   : launch_clusters(ttt_recurrence_fwd_tile_kernel<T, MODE, CPL, false>, p, blocks, st);
}

// Two bf16 channels a lane need even strides and pointers aligned to the pair.
bool pairs_ok(const RecurArgs &a)
{
    long long m = a.C;
    for (int i = 0; i < 2; ++i) m |= a.xs[i] | a.fs[i] | a.ds[i];
    uintptr_t q = 0;
    for (const void *v : {a.x, a.f, a.dh, (const void *)a.h, (const void *)a.dx, (const void *)a.df})
        q |= reinterpret_cast<uintptr_t>(v);
    return m % 2 == 0 && q % 4 == 0;
}

template <typename T, int MODE> int run(const RecurArgs &a, bool bwd)
{
    const RecurParams p = params_of(a);
    if (a.T > kS) {
        // a lane holds 4 bytes of a token: one fp32 channel, two of bf16
        if constexpr (sizeof(T) == 2)
            if (pairs_ok(a)) return run_tiles<T, MODE, 2>(p, bwd, a.stream);
        return run_tiles<T, MODE, 1>(p, bwd, a.stream);
    }
    const dim3 grid((a.C + kThreads - 1) / kThreads, a.B);
    if (bwd) ttt_recurrence_bwd_kernel<T, MODE><<<grid, kThreads, 0, a.stream>>>(p);
    else ttt_recurrence_fwd_kernel<T, MODE><<<grid, kThreads, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <typename T> int run_mode(const RecurArgs &a, bool bwd)
{
    switch (a.mode) {
    case kRecurDecay: return run<T, kRecurDecay>(a, bwd);
    case kRecurSigmoid: return run<T, kRecurSigmoid>(a, bwd);
    default: return run<T, kRecurMix>(a, bwd);
    }
}

}  // namespace

int launch_recurrence(const RecurArgs &a, bool backward)
{
    return a.bf16 ? run_mode<__nv_bfloat16>(a, backward) : run_mode<float>(a, backward);
}

}  // namespace ttt
