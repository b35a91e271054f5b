// ttt_recurrence.cu -- the gated linear recurrence of every channel,
//     h_t = a_t h_{t-1} + c_t x_t,
// a = f, c = 1 (decay), a = sigma(f), c = 1 (sigmoid) or a = sigma(f), c = 1 - a (mix: the
// TTT layer with a constant as its inner model, w <- w - eta (w - x), eta = 1 - a, one
// rate a channel).  A reset before token t makes h_{t-1} zero there.  Backward:
//     s_t = dh_t + r_{t+1},  r_t = a_t s_t,  r_T = dh_last,  dh0 = r_0,
//     dx = c s,  dL/da = s (h_{t-1} [- x_t for mix]),  df = dL/da a (1 - a) unless a = f,
// with h_{t-1} computed again from the states that the forward pass leaves every
// kRecurChunk tokens: no rounded h is read, and no more bytes than reading it would take.
#include <mutex>

#include <cuda.h>

#include "ttt_device.cuh"
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
    int *status;           // device status word (timeouts)
    unsigned long long test_stall_ns;  // > 0: the timeout test (see stalled())
};

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

// exp(-|f|): for bf16 tensors by one ex2 (good to 2^-20 over the range that matters), for
// fp32 the accurate one
template <typename T> __device__ __forceinline__ float exp_neg_abs(float f)
{
    return sizeof(T) == 2 ? exp2_approx(fabsf(f) * -1.4426950408889634f) : expf(-fabsf(f));
}

// a and 1 - a, each accurate on its own: with e = exp(-|f|) <= 1 the smaller of the two is
// e / (1 + e) and the larger 1 / (1 + e), so neither is a difference and nothing overflows.
template <typename T, int MODE> __device__ __forceinline__ void gate(float f, float &a, float &eta)
{
    if (MODE == kRecurDecay) {
        a = f;
        eta = 1.f;
        return;
    }
    const float e = exp_neg_abs<T>(f), big = rcp_approx(1.f + e), small = e * big;
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

// One thread a channel, token after token: decoding steps and lengths up to kS, a warp's share
// of a tile (64 x 1 x 768: 2 us, one launch and one trip to memory).
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
// A warp takes kS tokens of 128 bytes of channels, a block of kW warps a tile of kRecurChunk
// tokens, a cluster of P blocks P neighbouring tiles, and the cluster walks along the
// sequence in rounds of P tiles.  Every tensor is read once, by TMA into a ring of stages;
// where rows or pointers are not 16-byte aligned, into the same places with cp.async.  A
// warp folds its tokens into one map h -> A h + H (the product of the decays, the tokens'
// own contribution); the warps' maps are joined in shared memory, the blocks' totals
// through the cluster's distributed shared memory (stores that complete on the reader's
// mbarrier: a cluster barrier would wait for the round's global stores as well).  The join
// order is fixed by position, so results do not depend on timing.  NaN and infinities do
// not pass a reset: a map with a reset in it (cut) ignores its input.
//
// Measured (bf16, mix; of the copy bandwidth by bytes read and written once): 2 x 32768 x
// 2048 forward 150 us (0.79) and backward 257 us (0.77), with two blocks an SM and issue
// slots half busy; 8 x 2048 x 768 21 us (0.52) and 33 us (0.56): 96 chains of six dependent
// rounds.  A thread a channel, token by token, took 1339 us there.

constexpr int kS = 16, kW = 8;
static_assert(kS * kW == kRecurChunk, "a tile is one stored-state chunk");
constexpr int kRowBytes = 128;                       // a tile's row of one tensor, by TMA
constexpr int kPlane = kRecurChunk * kRowBytes;      // one tensor of a stage
constexpr int kMaxCluster = 16;
constexpr int kFwdStages = 2, kBwdStages = 2;

// N channels of a lane, with paired instructions for two.
template <int N> struct F;
template <> struct F<1> {
    float x;
};
template <> struct alignas(8) F<2> {
    float x, y;
};
__device__ __forceinline__ float2 f2(const F<2> &a) { return make_float2(a.x, a.y); }
__device__ __forceinline__ F<2> f2(float2 a) { return {a.x, a.y}; }
__device__ __forceinline__ F<1> fma(F<1> a, F<1> b, F<1> c) { return {fmaf(a.x, b.x, c.x)}; }
__device__ __forceinline__ F<2> fma(F<2> a, F<2> b, F<2> c) { return f2(__ffma2_rn(f2(a), f2(b), f2(c))); }
__device__ __forceinline__ F<1> mul(F<1> a, F<1> b) { return {a.x * b.x}; }
__device__ __forceinline__ F<2> mul(F<2> a, F<2> b) { return f2(__fmul2_rn(f2(a), f2(b))); }
__device__ __forceinline__ F<1> add(F<1> a, F<1> b) { return {a.x + b.x}; }
__device__ __forceinline__ F<2> add(F<2> a, F<2> b) { return f2(__fadd2_rn(f2(a), f2(b))); }
__device__ __forceinline__ F<1> sub(F<1> a, F<1> b) { return {a.x - b.x}; }
__device__ __forceinline__ F<2> sub(F<2> a, F<2> b) { return f2(__ffma2_rn(f2(b), make_float2(-1.f, -1.f), f2(a))); }
template <int N> __device__ __forceinline__ F<N> splat(float v);
template <> __device__ __forceinline__ F<1> splat<1>(float v) { return {v}; }
template <> __device__ __forceinline__ F<2> splat<2>(float v) { return {v, v}; }

template <typename T, int MODE> __device__ __forceinline__ void gates(F<1> f, F<1> &a, F<1> &eta)
{
    gate<T, MODE>(f.x, a.x, eta.x);
}
template <typename T, int MODE> __device__ __forceinline__ void gates(F<2> f, F<2> &a, F<2> &eta)
{
    if (MODE == kRecurDecay) {
        a = f;
        eta = {1.f, 1.f};
        return;
    }
    const F<2> e = {exp_neg_abs<T>(f.x), exp_neg_abs<T>(f.y)}, d = add(e, F<2>{1.f, 1.f});
    const F<2> big = {rcp_approx(d.x), rcp_approx(d.y)}, small = mul(e, big);
    a = {f.x > 0.f ? big.x : small.x, f.y > 0.f ? big.y : small.y};
    eta = {f.x > 0.f ? small.x : big.x, f.y > 0.f ? small.y : big.y};
}
template <typename T> __device__ __forceinline__ F<1> widen(const Pack<T, 1> &p)
{
    float v[1];
    unpack(p, v);
    return {v[0]};
}
template <typename T> __device__ __forceinline__ F<2> widen(const Pack<T, 2> &p)
{
    float v[2];
    unpack(p, v);
    return {v[0], v[1]};
}
template <typename T> __device__ __forceinline__ void put(T *p, F<1> a)
{
    const float v[1] = {a.x};
    Pack<T, 1> q;
    pack(q, v);
    q.store(p);
}
template <typename T> __device__ __forceinline__ void put(T *p, F<2> a)
{
    const float v[2] = {a.x, a.y};
    Pack<T, 2> q;
    pack(q, v);
    q.store(p);
}

// A lane's channels of a [B,C] fp32 array (WIDE: C a multiple of N, aligned to N).
template <int N, bool WIDE> __device__ __forceinline__ F<N> get_state(const float *p, int c, int C)
{
    if constexpr (WIDE) return widen(*reinterpret_cast<const Pack<float, N> *>(p + c));
    F<N> v = splat<N>(0.f);
    float *f = &v.x;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (c + j < C) f[j] = p[c + j];
    return v;
}
template <int N, bool WIDE, typename T> __device__ __forceinline__ void put_part(T *p, int c, int C, F<N> v)
{
    if constexpr (WIDE) {
        put(p + c, v);
    } else {
        const float *f = &v.x;
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (c + j < C) st1(p + c + j, f[j]);
    }
}

// How a tile's rows arrive and leave, by alignment (every tensor's):
//   kTma     16-byte rows: boxes into a ring of stages, outputs as boxes out of them.
//   kWords   4-byte rows (fp32; bf16 of even width): every lane copies its own words into
//            the same places a round ahead, and stores its outputs.
//   kHalves  bf16 rows of odd width: a warp copies the 16-byte blocks around its rows, so
//            that a row begins some bytes into its place, and moves every row to the start
//            of its place once it has landed; outputs leave the same way.  These loops over
//            rows are short on purpose: unrolled into the arithmetic they outgrew the
//            instruction cache (2 x 8192 x 1001 backward, clusters of four, 231 us against
//            151, and loads of single channels 238; 95 with the eight that are chosen).
enum RowFeed { kTma, kWords, kHalves };
constexpr int kRaggedPitch = kRowBytes + 16;
__host__ __device__ constexpr int row_pitch(int feed) { return feed == kHalves ? kRaggedPitch : kRowBytes; }

// A warp's tokens t0 .. of channels c0 on, by words, into its rows dst; zeros past the end.
template <typename T>
__device__ __forceinline__ void copy_words(const void *x, const long long (&st)[2], int b, long long t0, int c0, int T_, int C,
                                           unsigned char *dst)
{
    constexpr int N = 4 / (int)sizeof(T);
    const int n = (int)min(max(T_ - t0, 0LL), (long long)kS), c = c0 + (threadIdx.x & 31) * N;
    const T *q = static_cast<const T *>(x) + b * st[0] + t0 * st[1] + c;
    dst += (threadIdx.x & 31) * 4;
    if (n == kS && c < C) {
#pragma unroll
        for (int s = 0; s < kS; ++s, q += st[1], dst += kRowBytes) copy_async4(dst, q, 4);
    } else {
#pragma unroll 4
        for (int s = 0; s < kS; ++s, q += st[1], dst += kRowBytes) copy_async4(dst, q, s < n && c < C ? 4 : 0);
    }
}

// kHalves.
struct Ragged {
    static constexpr int kPitch = kRaggedPitch, kBlocks = kPitch / 16;
    using T = __nv_bfloat16;

    // base: the tensor, rows: channel c0 of token 0 of the warp's n, stride: elements to the
    // next, bytes: left of a row from there on.  Nothing behind a row's end is read, and
    // before its start only what shares 16 bytes with it inside the tensor.  27 lanes take
    // three rows at a time.
    static __device__ __forceinline__ void copy(const T *base, const T *rows, long long stride, int n, int bytes, unsigned char *dst)
    {
        const int lane = threadIdx.x & 31, r = lane / kBlocks, k = lane - r * kBlocks;
        if (r > 2) return;
        const char *q = reinterpret_cast<const char *>(rows + r * stride) + 16 * k;
        const int have = min(bytes, kRowBytes) - 16 * k;
        // a tensor that does not begin on 16: its first bytes one by one
        const bool head = reinterpret_cast<const char *>(rows) - reinterpret_cast<const char *>(base) < 16;
        dst += r * kPitch + 16 * k;
#pragma unroll
        for (int s = 0; s < kS; s += 3, q += 3 * stride * (int)sizeof(T), dst += 3 * kPitch) {
            if (s + 3 > kS && s + r >= kS) break;
            const int off = (int)(reinterpret_cast<uintptr_t>(q) & 15), size = s + r < n ? min(max(have + off, 0), 16) : 0;
            const char *from = q - off;
            if (head && from < reinterpret_cast<const char *>(base)) {
                // (and zeros behind them: tokens past the end come here too where the rows of a
                // broadcast tensor all begin at its first byte)
                for (int e = 0; e < 16; e += (int)sizeof(T)) {
                    const T *v = reinterpret_cast<const T *>(from + e);
                    *reinterpret_cast<T *>(dst + e) = v >= base && e < size ? *v : T(0.f);
                }
            } else {
                copy_async16_part(dst, from, size);
            }
        }
    }
    // at, step: low bits of the address of a row and of the distance to the next
    static __device__ __forceinline__ void align(uint32_t at, uint32_t step, unsigned char *dst)
    {
        constexpr int kRows = 8;  // at a time
        uint32_t *w = reinterpret_cast<uint32_t *>(dst) + (threadIdx.x & 31);
#pragma unroll 1
        for (int s = 0; s < kS; s += kRows, w += kRows * (kPitch / 4)) {
            uint32_t v[kRows];
#pragma unroll
            for (int j = 0; j < kRows; ++j, at += step) {
                const uint32_t *q = w + j * (kPitch / 4) + (at >> 2 & 3);
                v[j] = __funnelshift_r(q[0], q[1], (at & 2) * 8);
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < kRows; ++j) w[j * (kPitch / 4)] = v[j];
        }
    }
    // n rows of outputs to channels c on of row (its channel 0) and the rows behind it.  bf16
    // rows that begin on an odd half word (odd: the first one's bit, of all lanes) leave as
    // words of neighbouring lanes' halves.
    static __device__ __forceinline__ void store(const unsigned char *src, T *row, int c, int C, int n, uint32_t odd)
    {
        const int lane = threadIdx.x & 31;
        const uint32_t *w = reinterpret_cast<const uint32_t *>(src) + lane;
        T *q = row + c;
        const bool in = c < C, pair = c + 1 < C, left_in = lane > 0 && c <= C;
#pragma unroll 4
        for (int s = 0; s < n; ++s, q += C, w += kPitch / 4) {
            const uint32_t v = *w;
            unsigned short *e = reinterpret_cast<unsigned short *>(q);
            if (((odd + (uint32_t)s * (uint32_t)C) & 1) == 0) {
                if (pair) *reinterpret_cast<uint32_t *>(e) = v;
                else if (in) *e = (unsigned short)v;
            } else {
                const uint32_t left = __shfl_up_sync(0xffffffffu, v, 1);
                if (in && left_in) *reinterpret_cast<uint32_t *>(e - 1) = __byte_perm(left, v, 0x5432);
                else if (left_in) e[-1] = (unsigned short)(left >> 16);
                else if (in) *e = (unsigned short)v;
                if (lane == 31 && pair) e[1] = (unsigned short)(v >> 16);
            }
        }
    }
};

// A map of one direction: v -> a v + c.
template <int N> struct alignas(8 * N) Map {
    F<N> a, c;
};
template <int N> __device__ __forceinline__ F<N> apply(const Map<N> &m, F<N> v, bool cut)
{
    return cut ? m.c : fma(m.a, v, m.c);
}

// The warps' maps of a round, double-buffered over rounds.  One barrier a round is enough:
// a buffer is written again two rounds later, behind the next round's barrier.  The
// blocks' totals lie behind the stages, [2][P][32].  BWD: beside the forward maps the
// constant terms of the backward ones, whose factors are the same.
template <int N, bool BWD> struct TileShared {
    Map<N> w[2][kW][32];
    F<N> r[BWD ? 2 : 1][BWD ? kW : 1][32];
    int wcut[2][kW];
    int tcut[2][kMaxCluster];
    unsigned long long full[2], joined[2];  // mbarriers: a stage's copies, the cluster's totals
    unsigned long long dead;                // one that nothing arrives at (timeout test)
};

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier()
{
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t remote(uint32_t local, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
    return r;
}
// stores to a block of the cluster that count on its mbarrier as they land
__device__ __forceinline__ void send(uint32_t dst, uint32_t bar, const Map<2> &m)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2,%3,%4,%5}, [%1];" ::"r"(dst),
                 "r"(bar), "f"(m.a.x), "f"(m.a.y), "f"(m.c.x), "f"(m.c.y)
                 : "memory");
}
__device__ __forceinline__ void send(uint32_t dst, uint32_t bar, const Map<1> &m)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%2,%3}, [%1];" ::"r"(dst),
                 "r"(bar), "f"(m.a.x), "f"(m.c.x)
                 : "memory");
}
__device__ __forceinline__ void send(uint32_t dst, uint32_t bar, int v)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %2, [%1];" ::"r"(dst), "r"(bar),
                 "r"(v)
                 : "memory");
}

// Tells every block of the cluster this block's total and waits for theirs; then carry
// goes through all of them, and the value before this block's tile is returned.
template <int N, bool RESET, bool BWD>
__device__ __forceinline__ F<N> join_blocks(TileShared<N, BWD> &sh, Map<N> *totals, const Map<N> &total, bool cut, F<N> &carry,
                                            int P, int rank, int buf, int phase, const RecurParams &p, bool &ok)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t bar = smem_u32(&sh.joined[buf]);
    totals += buf * P * 32 + lane;
    if (threadIdx.x == 0) mbar_arrive_expect_tx(bar, P * (32 * (int)sizeof(Map<N>) + (RESET ? 4 : 0)));
    for (int i = warp; i < P; i += kW) {  // warp i tells block i (and i + kW)
        const uint32_t rbar = remote(bar, i);
        send(remote(smem_u32(totals + rank * 32), i), rbar, total);
        if (RESET && lane == 0) send(remote(smem_u32(&sh.tcut[buf][rank]), i), rbar, (int)cut);
    }
    ok &= mbar_wait(bar, phase, p.status, kSiteStage, p.test_stall_ns ? p.test_stall_ns : kWaitLimitNs);
    F<N> before = carry;
    for (int i = 0; i < P; ++i) {
        carry = apply(totals[i * 32], carry, RESET && sh.tcut[buf][i]);
        if (i < rank) before = carry;
    }
    return before;
}

// A box of shared memory to a tensor; elements out of range are dropped.
__device__ __forceinline__ void tma_store_3d(const void *tmap, uint32_t src, int x, int y, int z)
{
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// this thread's stores have read their shared memory
__device__ __forceinline__ void tma_store_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

// The reset bits of a warp's tokens t0 .. t0 + n - 1.
__device__ __forceinline__ unsigned reset_bits(const unsigned char *reset, int t0, int n, int lane)
{
    return __ballot_sync(0xffffffffu, lane < n && reset[t0 + lane] != 0);
}

// The timeout test: a cluster's last block gives up first, on a barrier that nothing arrives
// at, and the others as it does not send its totals.
template <typename S> __device__ __forceinline__ bool stalled(const S &sh, const RecurParams &p, int rank)
{
    return p.test_stall_ns && rank == p.cluster - 1 && !mbar_wait(smem_u32(&sh.dead), 0, p.status, kSiteStage, p.test_stall_ns);
}

// The way out of a block that gave up waiting (never expected): its own copies land (drain),
// its cluster's blocks meet, having sent all that they will, and what they sent to it has a
// hundred microseconds to land, as nothing counts it any more.
__device__ __forceinline__ void settle()
{
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 100000) __nanosleep(1000);
}
__device__ __forceinline__ void drain(unsigned long long *full, int rounds_issued, int stages, int *status)
{
    for (int r = max(0, rounds_issued - stages); r < rounds_issued; ++r)
        if (!mbar_wait(smem_u32(&full[r % stages]), (r / stages) & 1, status, kSiteDrain)) break;
}

// A tensor's tile of channels from c0 on, of a warp's tokens from t0 on, into its rows dst.
template <typename T, int FEED>
__device__ __forceinline__ void copy_rows(const void *x, const long long (&st)[2], int b, long long t0, int c0, int T_, int C,
                                          unsigned char *dst)
{
    if constexpr (FEED == kWords) {
        copy_words<T>(x, st, b, t0, c0, T_, C, dst);
    } else {
        const Ragged::T *base = static_cast<const Ragged::T *>(x);
        Ragged::copy(base, base + b * st[0] + t0 * st[1] + c0, st[1], (int)min(max(T_ - t0, 0LL), (long long)kS),
                     min(C - c0, kRowBytes) * 2, dst);
    }
}
// kHalves: warps' tokens lie whole multiples of 16 bytes apart, so the offsets are token 0's.
__device__ __forceinline__ void align_rows(const void *x, const long long (&st)[2], int b, int c0, unsigned char *dst)
{
    Ragged::align((uint32_t)reinterpret_cast<uintptr_t>(static_cast<const Ragged::T *>(x) + b * st[0] + c0), (uint32_t)st[1] * 2u, dst);
}
__device__ __forceinline__ void store_rows(const unsigned char *src, void *y, int b, int t0, int c, int T_, int C, int n)
{
    Ragged::T *first = static_cast<Ragged::T *>(y) + (size_t)b * T_ * C;
    Ragged::store(src, first + (size_t)t0 * C, c, C, n, (uint32_t)(reinterpret_cast<uintptr_t>(first) >> 1));
}
// Bytes of the stages.  kTma: [stages][f, x(, dh)], forward h; else forward f, x and h, backward
// f, x [2], dh [2]: f (forward: both) is refilled as soon as it is read.
__host__ __device__ constexpr int fwd_bytes(int feed) { return (feed == kTma ? kFwdStages * 2 + 1 : 3) * kRecurChunk * row_pitch(feed); }
__host__ __device__ constexpr int bwd_bytes(int feed) { return (feed == kTma ? kBwdStages * 3 : 5) * kRecurChunk * row_pitch(feed); }

template <typename T, int MODE, bool RESET, int FEED>
__global__ void __launch_bounds__(32 * kW, 2)
    ttt_recurrence_fwd_tile_kernel(const __grid_constant__ RecurParams p, const __grid_constant__ CUtensorMap tf,
                                   const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap th)
{
    constexpr int N = 4 / (int)sizeof(T), CH = 32 * N, kPitch = row_pitch(FEED), kStep = kRecurChunk * kPitch;
    constexpr bool TMA = FEED == kTma;
    using P_ = Pack<T, N>;
    __shared__ TileShared<N, false> sh;
    extern __shared__ unsigned char dynamic[];
    unsigned char *stages = dynamic + (-smem_u32(dynamic) & 127u);
    Map<N> *totals = reinterpret_cast<Map<N> *>(stages + fwd_bytes(FEED));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = p.cluster, rank = P > 1 ? (int)cluster_rank() : 0;
    const int chain = blockIdx.x / P, b = chain / p.cblocks, c0 = (chain % p.cblocks) * CH, c = c0 + lane * N;
    const bool on = c < p.C;
    const unsigned char *reset = RESET ? p.reset + (size_t)b * p.T : nullptr;
    const size_t bC = (size_t)b * p.C;
    const int rounds = (p.chunks + P - 1) / P;
    auto issue = [&](int round) {
        const int st = round % kFwdStages;
        const uint32_t dst = smem_u32(stages) + st * 2 * kPlane, bar = smem_u32(&sh.full[st]);
        mbar_arrive_expect_tx(bar, 2 * kPlane);
        tma_load_3d(dst, &tf, bar, c0, (round * P + rank) * kRecurChunk, b);
        tma_load_3d(dst + kPlane, &tx, bar, c0, (round * P + rank) * kRecurChunk, b);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.joined[i]), 1);
        }
        mbar_init(smem_u32(&sh.dead), 1);
        fence_barrier_init();
        if (TMA)
            for (int i = 0; i < kFwdStages && i < rounds; ++i) issue(i);
    }
    F<N> carry = splat<N>(0.f);
    if (on && p.h0) carry = get_state<N, TMA>(p.h0 + bC, c, p.C);
    unsigned char *own = stages + warp * kS * kPitch;  // this warp's rows of f (not kTma)
    auto copy = [&](int round) {
        const long long t0 = (long long)(round * P + rank) * kRecurChunk + warp * kS;
        copy_rows<T, FEED>(p.f, p.fs, b, t0, c0, p.T, p.C, own);
        copy_rows<T, FEED>(p.x, p.xs, b, t0, c0, p.T, p.C, own + kStep);
        copy_commit();
    };
    int t0 = rank * kRecurChunk + warp * kS;
    if (!TMA) copy(0);
    __syncthreads();
    if (P > 1) cluster_barrier();  // every block runs, its barriers set, before it is written to
    bool ok = !stalled(sh, p, rank);
    int round = 0;
    for (; round < rounds; ++round, t0 += P * kRecurChunk) {
        const int buf = round & 1;
        const int n = min(max(p.T - t0, 0), kS);  // this warp's tokens
        const unsigned cuts = RESET ? reset_bits(reset, t0, n, lane) : 0u;
        const unsigned char *fm = (TMA ? stages + (round % kFwdStages) * 2 * kPlane + warp * kS * kRowBytes : own) + lane * 4;
        const unsigned char *xm = fm + kStep;
        if (TMA) {
            ok &= mbar_wait(smem_u32(&sh.full[round % kFwdStages]), (round / kFwdStages) & 1, p.status, kSiteConsumerFull);
        } else {
            copy_wait<0>();
            __syncwarp();
            if (FEED == kHalves) {
                align_rows(p.f, p.fs, b, c0, own);
                align_rows(p.x, p.xs, b, c0, own + kStep);
            }
        }
        F<N> a[kS], u[kS];
        Map<N> m = {splat<N>(1.f), splat<N>(0.f)};
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            const F<N> x = widen(*reinterpret_cast<const P_ *>(xm + s * kPitch));
            F<N> eta;
            gates<T, MODE>(widen(*reinterpret_cast<const P_ *>(fm + s * kPitch)), a[s], eta);
            u[s] = MODE == kRecurMix ? mul(eta, x) : x;
        }
        if (!TMA && round + 1 < rounds) {
            __syncwarp();
            copy(round + 1);
        }
        if (n < kS) {  // tokens past the end: the identity
#pragma unroll
            for (int s = 0; s < kS; ++s)
                if (s >= n) {
                    a[s] = splat<N>(1.f);
                    u[s] = splat<N>(0.f);
                }
        }
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (RESET && (cuts >> s & 1u)) m.c = splat<N>(0.f);
            m.c = fma(a[s], m.c, u[s]);
            m.a = mul(m.a, a[s]);
        }
        sh.w[buf][warp][lane] = m;
        if (RESET && lane == 0) sh.wcut[buf][warp] = cuts != 0;
        ok = __syncthreads_and(ok);
        if (!ok) break;
        if (TMA && threadIdx.x == 0 && round + kFwdStages < rounds) issue(round + kFwdStages);
        // the state before this block's tile, and the next round's
        F<N> st = carry;
        if (P > 1) {
            Map<N> total = sh.w[buf][0][lane];
            bool cut = RESET && sh.wcut[buf][0];
#pragma unroll
            for (int i = 1; i < kW; ++i) {
                const Map<N> w = sh.w[buf][i][lane];
                const bool ci = RESET && sh.wcut[buf][i];
                total.c = apply(w, total.c, ci);
                total.a = mul(w.a, total.a);
                cut |= ci;
            }
            st = join_blocks<N, RESET>(sh, totals, total, cut, carry, P, rank, buf, (round >> 1) & 1, p, ok);
        }
        if (warp == 0 && p.states && on && n > 0)
            put_part<N, TMA>(p.states + ((size_t)b * p.chunks + t0 / kRecurChunk) * p.C, c, p.C, st);
        // the state before this warp's tokens
        F<N> h = st;
#pragma unroll
        for (int i = 0; i < kW; ++i) {
            st = apply(sh.w[buf][i][lane], st, RESET && sh.wcut[buf][i]);
            if (i + 1 == warp) h = st;
        }
        if (P == 1) carry = st;
        if constexpr (TMA) {
            // the warp's rows through shared memory: no addresses, and the copy drops what is
            // out of range
            unsigned char *out = stages + kFwdStages * 2 * kPlane + warp * kS * kRowBytes;
            if (lane == 0) tma_store_read();
            __syncwarp();
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                if (RESET && (cuts >> s & 1u)) h = splat<N>(0.f);
                h = fma(a[s], h, u[s]);
                put(reinterpret_cast<T *>(out + s * kRowBytes + lane * 4), h);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && n > 0) tma_store_3d(&th, smem_u32(out), c0, t0, b);
        } else {
            T *row = static_cast<T *>(p.h) + ((size_t)b * p.T + t0) * p.C + c;
            unsigned char *out = own + 2 * kStep + lane * 4;
#pragma unroll
            for (int s = 0; s < kS; ++s) {
                if (RESET && (cuts >> s & 1u)) h = splat<N>(0.f);
                h = fma(a[s], h, u[s]);
                if (FEED == kHalves) put(reinterpret_cast<T *>(out + s * kPitch), h);
                else if (s < n && on) put(row + (size_t)s * p.C, h);
            }
            if (FEED == kHalves) store_rows(out - lane * 4, p.h, b, t0, c, p.T, p.C, n);
        }
    }
    if (TMA && lane == 0) tma_store_read();
    if (!TMA) copy_wait<0>();  // a block that gave up has some in flight
    if (!ok && TMA && threadIdx.x == 0) drain(sh.full, min(rounds, round + kFwdStages), kFwdStages, p.status);
    if (P > 1) {
        cluster_barrier();  // no block leaves while another may write to it
        if (!ok) settle();
    }
    if (ok && p.h_last && on && rank == 0 && warp == 0) put_part<N, TMA>(p.h_last + bC, c, p.C, carry);
}

// Backward: the same tiles from the end of the sequence to its start.  Each warp has two
// maps with the same product of decays: forward from the tile's stored state, which brings
// it h_{t-1}, and backward r -> A r + R with R = sum_s (a_0 .. a_s) dh_s, gathered in token
// order beside the forward one.  x and dh are read again from the stage for the outputs,
// so a stage is refilled one round after its own.
template <typename T, int MODE, bool RESET, int FEED>
__global__ void __launch_bounds__(32 * kW, 2)
    ttt_recurrence_bwd_tile_kernel(const __grid_constant__ RecurParams p, const __grid_constant__ CUtensorMap tf,
                                   const __grid_constant__ CUtensorMap tx, const __grid_constant__ CUtensorMap td,
                                   const __grid_constant__ CUtensorMap tdx, const __grid_constant__ CUtensorMap tdf)
{
    constexpr int N = 4 / (int)sizeof(T), CH = 32 * N, kPitch = row_pitch(FEED), kStep = kRecurChunk * kPitch;
    constexpr bool TMA = FEED == kTma;
    using P_ = Pack<T, N>;
    __shared__ TileShared<N, true> sh;
    extern __shared__ unsigned char dynamic[];
    unsigned char *stages = dynamic + (-smem_u32(dynamic) & 127u);
    Map<N> *totals = reinterpret_cast<Map<N> *>(stages + bwd_bytes(FEED));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int P = p.cluster, rank = P > 1 ? (int)cluster_rank() : 0;
    const int chain = blockIdx.x / P, b = chain / p.cblocks, c0 = (chain % p.cblocks) * CH, c = c0 + lane * N;
    const bool on = c < p.C;
    const unsigned char *reset = RESET ? p.reset + (size_t)b * p.T : nullptr;
    const size_t bC = (size_t)b * p.C;
    const int rounds = (p.chunks + P - 1) / P;
    // rank 0 holds the last tile of a round; tiles past the end of the sequence are empty
    const int last = rounds * P - 1 - rank;
    const int planes = p.dh ? 3 : 2;
    auto issue = [&](int round) {
        const int st = round % kBwdStages, t0 = (last - round * P) * kRecurChunk;
        const uint32_t dst = smem_u32(stages) + st * 3 * kPlane, bar = smem_u32(&sh.full[st]);
        mbar_arrive_expect_tx(bar, planes * kPlane);
        tma_load_3d(dst, &tf, bar, c0, t0, b);
        tma_load_3d(dst + kPlane, &tx, bar, c0, t0, b);
        if (p.dh) tma_load_3d(dst + 2 * kPlane, &td, bar, c0, t0, b);
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&sh.full[i]), 1);
            mbar_init(smem_u32(&sh.joined[i]), 1);
        }
        mbar_init(smem_u32(&sh.dead), 1);
        fence_barrier_init();
        if (TMA)
            for (int i = 0; i < kBwdStages && i < rounds; ++i) issue(i);
    }
    F<N> carry = splat<N>(0.f), next_start = splat<N>(0.f);
    if (on && p.dh_last) carry = get_state<N, TMA>(p.dh_last + bC, c, p.C);
    // the tile's stored state, a round ahead
    auto fetch = [&](int tile) {
        if (tile < p.chunks && on) next_start = get_state<N, TMA>(p.states_in + ((size_t)b * p.chunks + tile) * p.C, c, p.C);
    };
    unsigned char *own = stages + warp * kS * kPitch;  // this warp's rows of f (not kTma)
    auto copy = [&](int round) {
        const long long t0 = (long long)(last - round * P) * kRecurChunk + warp * kS;
        copy_rows<T, FEED>(p.f, p.fs, b, t0, c0, p.T, p.C, own);
        copy_rows<T, FEED>(p.x, p.xs, b, t0, c0, p.T, p.C, own + (1 + (round & 1)) * kStep);
        if (p.dh) copy_rows<T, FEED>(p.dh, p.ds, b, t0, c0, p.T, p.C, own + (3 + (round & 1)) * kStep);
        copy_commit();
    };
    if (!TMA) copy(0);
    fetch(last);
    __syncthreads();
    if (P > 1) cluster_barrier();
    bool ok = !stalled(sh, p, rank);
    int round = 0;
    for (; round < rounds; ++round) {
        const int tile = last - round * P, t0 = tile * kRecurChunk + warp * kS, buf = round & 1;
        const int n = min(max(p.T - t0, 0), kS);
        const unsigned cuts = RESET ? reset_bits(reset, t0, n, lane) : 0u;
        unsigned char *rows = TMA ? stages + (round % kBwdStages) * 3 * kPlane + warp * kS * kRowBytes : own;
        unsigned char *fm = rows + lane * 4, *xm = fm + (TMA ? 1 : 1 + (round & 1)) * kStep, *dm = xm + (TMA ? 1 : 2) * kStep;
        if (TMA) {
            ok &= mbar_wait(smem_u32(&sh.full[round % kBwdStages]), (round / kBwdStages) & 1, p.status, kSiteConsumerFull);
        } else {
            copy_wait<0>();
            __syncwarp();
            if (FEED == kHalves) {
                align_rows(p.f, p.fs, b, c0, rows);
                align_rows(p.x, p.xs, b, c0, xm - lane * 4);
                if (p.dh) align_rows(p.dh, p.ds, b, c0, dm - lane * 4);
            }
        }
        auto load_x = [&](int s) { return widen(*reinterpret_cast<const P_ *>(xm + s * kPitch)); };
        auto load_d = [&](int s) { return p.dh ? widen(*reinterpret_cast<const P_ *>(dm + s * kPitch)) : splat<N>(0.f); };
        F<N> a[kS], eta[kS], h = next_start, r;
#pragma unroll
        for (int s = 0; s < kS; ++s)
            gates<T, MODE>(widen(*reinterpret_cast<const P_ *>(fm + s * kPitch)), a[s], eta[s]);
        if (n < kS) {  // tokens past the end, whose x and dh read as zeros: the identity
#pragma unroll
            for (int s = 0; s < kS; ++s)
                if (s >= n) {
                    a[s] = splat<N>(1.f);
                    eta[s] = splat<N>(0.f);
                }
        }
        if (round + 1 < rounds) {
            if (!TMA) {
                __syncwarp();  // every lane is done with f, and with the round before
                copy(round + 1);
            }
            fetch(tile - P);
        }
        Map<N> mf = {splat<N>(1.f), splat<N>(0.f)};
        F<N> back = splat<N>(0.f);
        F<N> live = splat<N>(1.f);  // a_0 .. a_s, and zero from a reset on
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (RESET && (cuts >> s & 1u)) {
                mf.c = splat<N>(0.f);
                live = splat<N>(0.f);
            }
            mf.c = fma(a[s], mf.c, MODE == kRecurMix ? mul(eta[s], load_x(s)) : load_x(s));
            mf.a = mul(mf.a, a[s]);
            // dh behind a reset does not count, whatever it is
            live = RESET ? mul(live, a[s]) : mf.a;
            if (!RESET || !(cuts & ((2u << s) - 1u))) back = fma(live, load_d(s), back);
        }
        sh.w[buf][warp][lane] = mf;
        sh.r[buf][warp][lane] = back;
        if (RESET && lane == 0) sh.wcut[buf][warp] = cuts != 0;
        if (TMA && lane == 0) tma_store_read();  // the round before has left its stage
        ok = __syncthreads_and(ok);
        if (!ok) break;
        // every warp is done with the round before
        if (TMA && threadIdx.x == 0 && round > 0 && round + 1 < rounds && round + 1 >= kBwdStages) issue(round + 1);
        F<N> st = carry;  // r behind this block's tile
        if (P > 1) {
            Map<N> total = {sh.w[buf][kW - 1][lane].a, sh.r[buf][kW - 1][lane]};
            bool cut = RESET && sh.wcut[buf][kW - 1];
#pragma unroll
            for (int i = kW - 2; i >= 0; --i) {
                const Map<N> w = {sh.w[buf][i][lane].a, sh.r[buf][i][lane]};
                const bool ci = RESET && sh.wcut[buf][i];
                total.c = apply(w, total.c, ci);
                total.a = mul(w.a, total.a);
                cut |= ci;
            }
            st = join_blocks<N, RESET>(sh, totals, total, cut, carry, P, rank, buf, (round >> 1) & 1, p, ok);
        }
#pragma unroll
        for (int i = 0; i < kW - 1; ++i)
            if (i < warp) h = apply(sh.w[buf][i][lane], h, RESET && sh.wcut[buf][i]);
        r = st;
#pragma unroll
        for (int i = kW - 1; i >= 0; --i) {
            const Map<N> w = {sh.w[buf][i][lane].a, sh.r[buf][i][lane]};
            st = apply(w, st, RESET && sh.wcut[buf][i]);
            if (i == warp + 1) r = st;
        }
        if (P == 1) carry = st;
        // h_{t-1} [- x_t] in token order, then the outputs from the last token back
        F<N> g[kS];
#pragma unroll
        for (int s = 0; s < kS; ++s) {
            if (RESET && (cuts >> s & 1u)) h = splat<N>(0.f);
            const F<N> x = load_x(s);
            g[s] = MODE == kRecurMix ? sub(h, x) : h;
            h = fma(a[s], h, MODE == kRecurMix ? mul(eta[s], x) : x);
        }
        const size_t o = ((size_t)b * p.T + t0) * p.C + c;
        T *dx = static_cast<T *>(p.dx) + o, *df = static_cast<T *>(p.df) + o;
#pragma unroll
        for (int s = kS - 1; s >= 0; --s) {
            const F<N> sv = add(load_d(s), r);
            r = mul(a[s], sv);
            const F<N> dxv = MODE == kRecurMix ? mul(eta[s], sv) : sv;
            const F<N> dfv = MODE == kRecurDecay ? mul(sv, g[s]) : mul(mul(r, g[s]), eta[s]);
            if (FEED != kWords) {  // over x and dh, which this lane has read
                put(reinterpret_cast<T *>(xm + s * kPitch), dxv);
                put(reinterpret_cast<T *>(dm + s * kPitch), dfv);
            } else if (s < n && on) {
                put(dx + (size_t)s * p.C, dxv);
                put(df + (size_t)s * p.C, dfv);
            }
            if (RESET && (cuts >> s & 1u)) r = splat<N>(0.f);
        }
        if constexpr (TMA) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0 && n > 0) {
                tma_store_3d(&tdx, smem_u32(rows + kPlane), c0, t0, b);
                tma_store_3d(&tdf, smem_u32(rows + 2 * kPlane), c0, t0, b);
            }
        } else if (FEED == kHalves) {
            store_rows(xm - lane * 4, p.dx, b, t0, c, p.T, p.C, n);
            store_rows(dm - lane * 4, p.df, b, t0, c, p.T, p.C, n);
        }
    }
    if (TMA && lane == 0) tma_store_read();
    if (!TMA) copy_wait<0>();  // a block that gave up has some in flight
    if (!ok && TMA && threadIdx.x == 0) drain(sh.full, min(rounds, max(round + 1, kBwdStages)), kBwdStages, p.status);
    if (P > 1) {
        cluster_barrier();
        if (!ok) settle();
    }
    if (ok && p.dh0 && on && rank == 0 && warp == 0) put_part<N, TMA>(p.dh0 + bC, c, p.C, carry);
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
    p.status = a.status;
    p.test_stall_ns = a.test_stall_ns;
    p.B = a.B;
    p.T = a.T;
    p.C = a.C;
    p.chunks = (a.T + kRecurChunk - 1) / kRecurChunk;
    return p;
}

template <typename... KArgs>
bool cluster_config(void (*kernel)(KArgs...), int cluster, int blocks, int smem, cudaStream_t st, cudaLaunchConfig_t &cfg,
                    cudaLaunchAttribute &at)
{
    if (cluster > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
        return false;
    if (smem > 40 * 1024 && !allow_shared(kernel, smem)) return false;
    cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(32 * kW);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = cluster;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return true;
}

// How many clusters of P blocks the GPU holds at once: as many blocks to an SM as fit
// (any), and one to an SM (alone).
struct Capacity {
    int any[kMaxCluster + 1], alone[kMaxCluster + 1];
};

template <typename... KArgs> Capacity query_capacity(void (*kernel)(KArgs...), int smem, int per_block)
{
    Capacity c = {};
    for (int P = 1; P <= kMaxCluster; ++P)
        for (int one = 0; one < 2; ++one) {
            cudaLaunchConfig_t cfg;
            cudaLaunchAttribute at;
            int n = 0;
            // more than half of an SM's shared memory: no second block beside it
            const int need = smem + per_block * P, bytes = one && need < 128 * 1024 ? 128 * 1024 : need;
            if (!cluster_config(kernel, P, P, bytes, nullptr, cfg, at) ||
                cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
                cudaGetLastError();
                n = 0;
            }
            (one ? c.alone : c.any)[P] = n;
        }
    return c;
}

// The same, asked once for each kernel and device.
template <typename... KArgs> Capacity capacity(void (*kernel)(KArgs...), int smem, int per_block)
{
    static std::mutex mu;
    static struct {
        void (*kernel)(KArgs...);
        int dev;
        Capacity c;
    } memo[256];
    static int used = 0;
    int dev = 0;
    cudaGetDevice(&dev);
    std::lock_guard<std::mutex> lock(mu);
    for (int i = 0; i < used; ++i)
        if (memo[i].kernel == kernel && memo[i].dev == dev) return memo[i].c;
    const Capacity c = query_capacity(kernel, smem, per_block);
    if (used < 256) memo[used++] = {kernel, dev, c};
    return c;
}

// Blocks of a cluster.  A round of a block alone on its SM is the unit of time, 1.2 us
// forward and 2.1 us backward (bf16, mix); 1.33 with the exchange between blocks; two
// blocks on an SM take `two` each, 1.95 in bf16, 1.5 in fp32, which has half the channels
// to compute for the same bytes; a start costs about 3, that of a later wave of clusters
// 6.  Fitted to 12 shapes of 1 .. 768 chains and 2 .. 256 chunks of 16-byte rows, timed with
// every P of 1 .. 16, where it picked the fastest P or one within 6% of it: 64 chains of 256
// chunks forward 150 us at P = 4 against 305, 203, 166 at 1, 2, 8; 12 chains 50 us at 16
// against 303 and 59 at 1 and 8; 192 chains of 8 chunks 20 us at 1 against 26 and 29 at 2 and
// 4.  Not fitted to the other rows, whose kernels hold other numbers of clusters: 2 x 8192 x
// 1002 in bf16 backward takes 78 us with its choice and took 71 with an earlier one.
int plan_cluster(long long chains, int chunks, double two, const Capacity &cap)
{
    int best = 1;
    double least = 0.0;
    for (int P = 1; P <= kMaxCluster && P <= chunks; ++P) {
        if (cap.any[P] < 1) continue;
        const int rounds = (chunks + P - 1) / P;
        const long long full = chains / cap.any[P], rest = chains % cap.any[P];
        const double later = P > 1 ? 6.0 : 3.0;
        double t = full * (rounds * two + later) + 3.0 - (full ? later : 0.0);
        if (rest) t += rounds * (rest > cap.alone[P] ? two : P > 1 ? 1.33 : 1.0) + (full ? later : 0.0);
        if (P == 1 || t < least) {
            least = t;
            best = P;
        }
    }
    return best;
}

template <typename... KArgs, typename... Args>
int launch_tiles(void (*kernel)(KArgs...), RecurParams p, int ch, int smem, cudaStream_t st, Args... maps)
{
    p.cblocks = (p.C + ch - 1) / ch;
    const long long chains = (long long)p.B * p.cblocks;
    const int per_block = 2 * ch * 8;  // each block's totals, twice
    smem += 128;                       // alignment
    p.cluster = plan_cluster(chains, p.chunks, ch < 64 ? 1.5 : 1.95, capacity(kernel, smem, per_block));
    cudaLaunchConfig_t cfg;
    cudaLaunchAttribute at;
    if (chains * p.cluster > 0x7fffffffLL ||
        !cluster_config(kernel, p.cluster, (int)(chains * p.cluster), smem + per_block * p.cluster, st, cfg, at))
        return -4;
    return cudaLaunchKernelEx(&cfg, kernel, p, maps...) == cudaSuccess ? 0 : -4;
}

template <typename T, int MODE, bool RESET, int FEED>
int run_tiles(const RecurParams &p, const CUtensorMap *maps, bool bwd, cudaStream_t st)
{
    constexpr int CH = 128 / (int)sizeof(T);
    if (bwd)
        return launch_tiles(ttt_recurrence_bwd_tile_kernel<T, MODE, RESET, FEED>, p, CH, bwd_bytes(FEED), st,
                            maps[0], maps[1], maps[2], maps[3], maps[4]);
    return launch_tiles(ttt_recurrence_fwd_tile_kernel<T, MODE, RESET, FEED>, p, CH, fwd_bytes(FEED), st,
                        maps[0], maps[1], maps[3]);
}

// Descriptors of f, x and dh in boxes of kRecurChunk tokens x 128 bytes of channels (rows
// past T and channels past C read as zeros) and of the outputs, in a warp's kS tokens.
// False: plain loads and stores instead (TMA wants 16-byte pointers and strides).
bool make_maps(const RecurArgs &a, bool bwd, CUtensorMap *maps)
{
    const int es = a.bf16 ? 2 : 4, cols = 128 / es;
    for (const void *v : {(const void *)a.h0, (const void *)a.dh_last, (const void *)a.h_last, (const void *)a.states,
                          (const void *)a.dh0})
        if (reinterpret_cast<uintptr_t>(v) % 8) return false;
    const void *in[3] = {a.f, a.x, a.dh};
    const long long *st[3] = {a.fs, a.xs, a.ds};
    for (int i = 0; i < 3; ++i) {
        if (!in[i]) continue;
        const long long sb = a.B > 1 ? st[i][0] : (long long)a.T * st[i][1];
        if (!encode_rows_map(&maps[i], in[i], a.bf16, a.C, a.T, a.B, st[i][1], sb, cols, kRecurChunk)) return false;
    }
    void *out[2] = {bwd ? a.dx : a.h, bwd ? a.df : nullptr};
    for (int i = 0; i < 2; ++i)
        if (out[i] && !encode_rows_map(&maps[3 + i], out[i], a.bf16, a.C, a.T, a.B, a.C, (long long)a.T * a.C, cols, kS))
            return false;
    return true;
}

// Do two channels of bf16 stand in a word everywhere?
bool pairs_aligned(const RecurArgs &a)
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
    RecurParams p = params_of(a);
    if (a.T > kS) {
        CUtensorMap maps[5] = {};
        if (make_maps(a, bwd, maps))
            return a.reset ? run_tiles<T, MODE, true, kTma>(p, maps, bwd, a.stream)
                           : run_tiles<T, MODE, false, kTma>(p, maps, bwd, a.stream);
        if constexpr (sizeof(T) == 2)
            if (!pairs_aligned(a))
                return a.reset ? run_tiles<T, MODE, true, kHalves>(p, maps, bwd, a.stream)
                               : run_tiles<T, MODE, false, kHalves>(p, maps, bwd, a.stream);
        return a.reset ? run_tiles<T, MODE, true, kWords>(p, maps, bwd, a.stream)
                       : run_tiles<T, MODE, false, kWords>(p, maps, bwd, a.stream);
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
