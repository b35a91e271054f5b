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
};

// a and 1 - a, each accurate on its own (no 1 - a of a rounded a near one)
template <int MODE> __device__ __forceinline__ void gate(float f, float &a, float &eta)
{
    if (MODE == kRecurDecay) {
        a = f;
        eta = 1.f;
        return;
    }
    a = 1.f / (1.f + __expf(-f));
    eta = 1.f / (1.f + __expf(f));
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

// One thread a channel, token after token.
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
        gate<MODE>(ld1(f + t * p.fs[1]), a, eta);
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
            gate<MODE>(ld1(f + t * p.fs[1]), a, eta);
            h = fmaf(a, h, MODE == kRecurMix ? eta * xv : xv);
        }
        for (int t = t1 - 1; t >= t0; --t) {
            const float s = (p.dh ? ld1(dh + t * p.ds[1]) : 0.f) + r, hp = before[t - t0][threadIdx.x];
            float a, eta;
            gate<MODE>(ld1(f + t * p.fs[1]), a, eta);
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

template <typename T, int MODE> int run(const RecurArgs &a, bool bwd)
{
    const RecurParams p = params_of(a);
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
