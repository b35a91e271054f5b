// ttt_short_conv.cu -- the short causal convolution of every channel along the tokens,
//     p_t = b + sum_{j < K} w_j x_{t-K+1+j},   y_t = p_t or p_t sigma(p_t),
// rows before the first token from the state (the last K - 1 inputs so far) or zero; a reset
// at token t (a packed sequence begins) hides every row before t from t on.  Backward:
//     g_t = dy_t act'(p_t),  dx_s = sum_{d < K} w_{K-1-d} g_{s+d},  dw_j = sum_t g_t x_{t-K+1+j},
//     db = sum_t g_t,
// with p computed again from x.
//
// Bound by reading and writing every tensor once: a thread walks along the tokens of one
// piece with the last K - 1 rows of its V neighbouring channels in registers.  Measured, K = 4,
// SiLU, bf16 (of the copy bandwidth by bytes read and written once): 2 x 32768 x 2048 forward
// 94 us (0.84; 92 under ncu), backward 191 us (0.62: 163 registers leave 12 warps an SM, issue slots
// 60% busy; the sums of the taps' gradients alone are 20 of them); 8 x 2048 x 768 forward 14.8 us
// (0.50: ramp-up and tail), backward 24; fp32 2 x 16384 x 2048 86 (0.92) and 165 us (0.72).
// Fewer than 32 vectors of channels leave lanes of the backward pass without work: 64 x 4096
// tokens of 8, 16, 64, 128 channels 95, 71, 58, 67 us, and 46, 25, 8, 5 us for the sums of its blocks.
#include "ttt_internal.h"
#include "ttt_vec.cuh"

namespace ttt {
namespace {

constexpr int kThreads = 128, kSMs = 152;

struct ConvParams {
    const void *x, *dy, *state;
    long long xs[2], dys[2];
    const float *weight, *bias, *dstate_out;
    const unsigned char *reset;
    void *y, *state_out, *dx;
    float *dstate, *part;
    int B, T, C, nv, pieces, len, silu;
    int few;  // forward: fewer than 2^31 threads
};

// bf16 tensors: one ex2 of a rounded product, off by |v| 2^-24 of itself, far below the output's
// rounding.  fp32 tensors: CUDA's expf.
template <typename T> __device__ __forceinline__ float sigmoid(float v)
{
    float e, r;
    if constexpr (sizeof(T) == 2) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v * -1.4426950408889634f));
    else e = expf(-v);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return r;
}

// acc += a b, two and two where V is even.
template <int V> __device__ __forceinline__ void fma_all(float (&acc)[V], const float (&a)[V], const float (&b)[V])
{
    if constexpr (V % 2 == 0) {
#pragma unroll
        for (int j = 0; j < V; j += 2) {
            const float2 r = __ffma2_rn(make_float2(a[j], a[j + 1]), make_float2(b[j], b[j + 1]), make_float2(acc[j], acc[j + 1]));
            acc[j] = r.x;
            acc[j + 1] = r.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] = fmaf(a[j], b[j], acc[j]);
    }
}
template <int V> __device__ __forceinline__ void clear(float (&v)[V])
{
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 0.f;
}

template <typename T, int V> __device__ __forceinline__ void load_row(const T *p, float (&v)[V])
{
    Pack<T, V> q;
    q.load(p);
    unpack(q, v);
}

// The taps of V neighbouring channels ([C,K] fp32), 16 bytes at a time where they lie so.
template <int V, int K> __device__ __forceinline__ void load_taps(const float *w, float (&v)[K][V])
{
    float f[V * K];
    if constexpr (V * K % 4 == 0) {
        if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
#pragma unroll
            for (int i = 0; i < V * K; i += 4) {
                const float4 q = __ldg(reinterpret_cast<const float4 *>(w + i));
                f[i] = q.x;
                f[i + 1] = q.y;
                f[i + 2] = q.z;
                f[i + 3] = q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V * K; ++i) f[i] = __ldg(w + i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < V * K; ++i) f[i] = __ldg(w + i);
    }
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k][j] = f[j * K + k];
}

// Rows t - (K-1) .. t - 1 before a piece (win[i] is row t - K + 1 + i) as the token t sees
// them, but for a reset at t itself.
template <typename T, int V, int K>
__device__ __forceinline__ void rows_before(const ConvParams &p, const T *x, const T *state, const unsigned char *reset, int t,
                                            float (&win)[K][V])
{
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        const int r = t - (K - 1) + i;
#pragma unroll
        for (int j = 0; j < V; ++j) win[i][j] = 0.f;
        if (r >= 0) load_row<T, V>(x + r * p.xs[1], win[i]);
        else if (state) {
            Pack<T, V> q;
            q.load_rw(state + (size_t)(r + K - 1) * p.C);
            unpack(q, win[i]);
        }
    }
    if (reset) {
        // a reset at row r hides the rows before it
#pragma unroll
        for (int i = 1; i < K - 1; ++i) {
            const int r = t - (K - 1) + i;
            if (r >= 0 && reset[r])
#pragma unroll
                for (int k = 0; k < i; ++k)
#pragma unroll
                    for (int j = 0; j < V; ++j) win[k][j] = 0.f;
        }
    }
}

template <typename T, int V, int K> __global__ void __launch_bounds__(kThreads) ttt_short_conv_fwd_kernel(const __grid_constant__ ConvParams p)
{
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    int cv, piece, b;
    if (p.few) {  // 32-bit divisions do
        const unsigned j = (unsigned)i, k = j / (unsigned)p.nv;
        cv = (int)(j - k * (unsigned)p.nv);
        b = (int)(k / (unsigned)p.pieces);
        piece = (int)k - b * p.pieces;
    } else {
        cv = (int)(i % p.nv);
        piece = (int)(i / p.nv % p.pieces);
        b = (int)(i / p.nv / p.pieces);
    }
    if (b >= p.B) return;
    const int c = cv * V, t0 = piece * p.len, t1 = min(p.T, t0 + p.len);
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c;
    const T *state = p.state ? static_cast<const T *>(p.state) + (size_t)b * (K - 1) * p.C + c : nullptr;
    const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;
    T *y = static_cast<T *>(p.y) + (size_t)b * p.T * p.C + c;

    float w[K][V], bias[V], win[K][V];
    load_taps<V, K>(p.weight + (size_t)c * K, w);
#pragma unroll
    for (int j = 0; j < V; ++j) bias[j] = p.bias ? p.bias[c + j] : 0.f;
    rows_before<T, V, K>(p, x, state, reset, t0, win);
    // The state behind the last token, by the thread that has read the one before the first
    // (they may be one array).
    if (K > 1 && piece == 0 && p.state_out) {
        T *out = static_cast<T *>(p.state_out) + (size_t)b * (K - 1) * p.C + c;
        Pack<T, V> last[K];
        bool hidden = false;
#pragma unroll
        for (int k = K - 2; k >= 0; --k) {
            const int r = p.T - (K - 1) + k;
            last[k].raw = {};
            if (r >= 0) {
                if (!hidden) last[k].load(x + r * p.xs[1]);
                hidden = hidden || (reset && reset[r]);
            } else if (!hidden && state) {
                last[k].load_rw(state + (size_t)(r + K - 1) * p.C);
            }
        }
#pragma unroll
        for (int k = 0; k < K - 1; ++k) last[k].store(out + (size_t)k * p.C);
    }
    // kAhead rows are on their way while the ones before them are worked on; the window turns
    // in place over K of them: row t + a goes to place (a + K - 1) % K, row t + a - K + 1 is at
    // a % K
    constexpr int kAhead = K == 3 ? 3 : 4;
    Pack<T, V> q[kAhead], r[kAhead];
    const T *xt = x + t0 * p.xs[1];
    T *yt = y + (size_t)t0 * p.C;
    auto load = [&](int t) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a)
            if (t + a < t1) r[a].load(xt + a * p.xs[1]);
        xt += kAhead * p.xs[1];
    };
    auto token = [&](int a, int t) {
        if (reset && reset[t])
#pragma unroll
            for (int k = 0; k < K; ++k) clear(win[k]);
        unpack(q[a], win[(a + K - 1) % K]);
        float o[V];
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = bias[j];
#pragma unroll
        for (int k = 0; k < K; ++k) fma_all(o, w[k], win[(a + k) % K]);
        if (p.silu)
#pragma unroll
            for (int j = 0; j < V; ++j) o[j] *= sigmoid<T>(o[j]);
        Pack<T, V> out;
        pack(out, o);
        out.store(yt + (size_t)a * p.C);
    };
    load(t0);
    for (int t = t0; t < t1; t += kAhead) {
#pragma unroll
        for (int a = 0; a < kAhead; ++a) q[a] = r[a];
        load(t + kAhead);
        if (t + kAhead <= t1) {
#pragma unroll
            for (int a = 0; a < kAhead; ++a) token(a, t + a);
        } else {
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (t + a < t1) token(a, t + a);
        }
        yt += (size_t)kAhead * p.C;
    }
}

// A piece's rows of dx, and its part of the sums.  Row s is complete when token s + K - 1 has
// been taken (or hidden from it), so the walk runs K - 1 tokens past the piece.  A block is
// 32 channel vectors wide and kRows pieces high, whose sums it adds up.
constexpr int kRows = kThreads / 32;
template <typename T, int V, int K> __global__ void __launch_bounds__(kThreads, 3) ttt_short_conv_bwd_kernel(const __grid_constant__ ConvParams p)
{
    __shared__ float sums[kRows][32][V * (K + 1) + 1];
    const int lane = threadIdx.x & 31, row = threadIdx.x >> 5;
    const int wide = (p.nv + 31) / 32;
    const int cv = (int)(blockIdx.x % wide) * 32 + lane;
    const long long pc = (long long)(blockIdx.x / wide) * kRows + row;
    const int piece = (int)(pc % p.pieces), b = (int)(pc / p.pieces);
    const bool on = cv < p.nv && b < p.B;
    float dw[K][V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        db[j] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][j] = 0.f;
    }
    if (on) {
        const int c = cv * V, t0 = piece * p.len, t1 = min(p.T, t0 + p.len), tend = min(p.T, t1 + K - 1);
        const int lo = piece == 0 ? -(K - 1) : t0;  // the first row this thread writes
        const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *dy = static_cast<const T *>(p.dy) + b * p.dys[0] + c;
        const T *state = p.state ? static_cast<const T *>(p.state) + (size_t)b * (K - 1) * p.C + c : nullptr;
        const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;
        T *dx = static_cast<T *>(p.dx) + (size_t)b * p.T * p.C + c;
        float w[K][V], bias[V], win[K][V], pend[K][V];
        load_taps<V, K>(p.weight + (size_t)c * K, w);
#pragma unroll
        for (int j = 0; j < V; ++j) {
#pragma unroll
            for (int k = 0; k < K; ++k) pend[k][j] = 0.f;
            bias[j] = p.bias ? p.bias[c + j] : 0.f;
        }
        rows_before<T, V, K>(p, x, state, reset, t0, win);
        int age = K - 1;  // rows before the token that it sees, counted up to K - 1
        if (reset)
            for (int r = max(t0 - (K - 1) + 1, 0); r < t0; ++r)
                if (reset[r]) age = min(age, t0 - r);
        int live = p.T;  // rows >= live reach the last state
        if (p.dstate_out) {
            live = p.T - (K - 1);
            if (reset)
                for (int r = max(live + 1, 0); r < p.T; ++r)
                    if (reset[r]) live = r;
        }
        // at token t + a row t + a - d waits at place (a + K - d) % K
        Pack<T, V> qx[K], qg[K], rx[K], rg[K];
        const T *xt = x + t0 * p.xs[1], *gt = dy + t0 * p.dys[1];
        T *dxt = dx + ((long long)t0 - (K - 1)) * p.C;
        auto load = [&](int t) {
#pragma unroll
            for (int a = 0; a < K; ++a)
                if (t + a < tend) {
                    rx[a].load(xt + a * p.xs[1]);
                    rg[a].load(gt + a * p.dys[1]);
                }
            xt += K * p.xs[1];
            gt += K * p.dys[1];
        };
        auto token = [&](int a, int t, bool own) {
            if (reset && reset[t]) {
                age = 0;
#pragma unroll
                for (int k = 0; k < K; ++k) clear(win[k]);
            }
            float g[V];
            unpack(qx[a], win[(a + K - 1) % K]);
            unpack(qg[a], g);
            if (p.silu) {
                float s[V];
#pragma unroll
                for (int j = 0; j < V; ++j) s[j] = bias[j];
#pragma unroll
                for (int k = 0; k < K; ++k) fma_all(s, w[k], win[(a + k) % K]);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float sg = sigmoid<T>(s[j]);
                    g[j] *= sg * fmaf(s[j], 1.f - sg, 1.f);
                }
            }
            if (own) {
#pragma unroll
                for (int j = 0; j < V; ++j) db[j] += g[j];
#pragma unroll
                for (int k = 0; k < K; ++k) fma_all(dw[k], g, win[(a + k) % K]);
            }
#pragma unroll
            for (int d = 0; d < K; ++d)
                if (!reset || d <= age) fma_all(pend[(a + K - d) % K], w[K - 1 - d], g);
            age = min(age + 1, K - 1);
        };
        auto finish = [&](int a, int s) {
            float (&o)[V] = pend[(a + 1) % K];
            if (p.dstate_out && s >= live) {
                const float *ds = p.dstate_out + ((size_t)b * (K - 1) + s - (p.T - (K - 1))) * p.C + c;
#pragma unroll
                for (int j = 0; j < V; ++j) o[j] += ds[j];
            }
            if (s >= 0) {
                Pack<T, V> q;
                pack(q, o);
                q.store(dxt + (long long)a * p.C);
            } else if (p.dstate) {
                float *ds = p.dstate + ((size_t)b * (K - 1) + s + K - 1) * p.C + c;
#pragma unroll
                for (int j = 0; j < V; ++j) ds[j] = o[j];
            }
        };
        load(t0);
        for (int t = t0; t < t1 + K - 1; t += K) {
#pragma unroll
            for (int a = 0; a < K; ++a) {
                qx[a] = rx[a];
                qg[a] = rg[a];
            }
            load(t + K);
            if (t >= t0 + K - 1 && t + K <= t1) {
#pragma unroll
                for (int a = 0; a < K; ++a) {
                    clear(pend[a]);
                    token(a, t + a, true);
                    finish(a, t + a - (K - 1));
                }
            } else {
#pragma unroll
                for (int a = 0; a < K; ++a) {
                    clear(pend[a]);
                    if (t + a < tend) token(a, t + a, t + a < t1);
                    const int s = t + a - (K - 1);
                    if (s >= lo && s < t1) finish(a, s);
                }
            }
            dxt += (long long)K * p.C;
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < V; ++j) {
#pragma unroll
        for (int k = 0; k < K; ++k) sums[row][lane][j * K + k] = dw[k][j];
        sums[row][lane][V * K + j] = db[j];
    }
    __syncthreads();
    // part: [blocks along the pieces][C (K + 1)], the weights' sums, then the biases'
    float *out = p.part + (size_t)(blockIdx.x / wide) * p.C * (K + 1);
    const int first = (int)(blockIdx.x % wide) * 32 * V;
    for (int i = threadIdx.x; i < 32 * V * (K + 1); i += kThreads) {
        const bool isw = i < 32 * V * K;
        const int ch = isw ? i / K : i - 32 * V * K;  // channel of the block
        if (first + ch >= p.C) continue;
        const int at = isw ? ch % V * K + i % K : V * K + ch % V;
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) s += sums[r][ch / V][at];
        out[isw ? (size_t)first * K + i : (size_t)p.C * K + first + ch] = s;
    }
}

// dweight and dbias from the blocks' sums, in an order fixed by their number.
__global__ void __launch_bounds__(256) ttt_short_conv_sum_kernel(const float *part, int rows, long long n, long long nw, float *dw, float *db)
{
    __shared__ float sh[8][32];
    const long long i = (long long)blockIdx.x * 32 + threadIdx.x % 32;
    float s = 0.f;
    if (i < n)
        for (int r = threadIdx.x / 32; r < rows; r += 8) s += part[r * n + i];
    sh[threadIdx.x / 32][threadIdx.x % 32] = s;
    __syncthreads();
    if (threadIdx.x < 32 && i < n) {
        for (int r = 1; r < 8; ++r) s += sh[r][threadIdx.x];
        if (i < nw) {
            if (dw) dw[i] = s;
        } else if (db) {
            db[i - nw] = s;
        }
    }
}

int widest(const ConvArgs &a, int most)
{
    const int es = a.bf16 ? 2 : 4;
    long long mask = a.C;
    for (const void *q : {a.x, a.dy, a.state, (const void *)a.y, (const void *)a.state_out, (const void *)a.dx})
        mask |= (long long)(reinterpret_cast<uintptr_t>(q) / es);
    for (int i = 0; i < 2; ++i) mask |= a.xs[i] | a.dys[i];
    int V = most;
    while (mask & (V - 1)) V >>= 1;
    return V;
}

void conv_params(const ConvArgs &a, ConvParams &p, int V)
{
    p = {};
    p.x = a.x;
    p.dy = a.dy;
    p.state = a.state;
    for (int i = 0; i < 2; ++i) {
        p.xs[i] = a.xs[i];
        p.dys[i] = a.dys[i];
    }
    p.weight = a.weight;
    p.bias = a.bias;
    p.dstate_out = a.dstate_out;
    p.reset = a.reset;
    p.y = a.y;
    p.state_out = a.state_out;
    p.dx = a.dx;
    p.dstate = a.dstate;
    p.B = a.B;
    p.T = a.T;
    p.C = a.C;
    p.nv = a.C / V;
    p.silu = a.silu;
}

template <typename T, int V> int fwd_width(const ConvArgs &a)
{
    ConvParams p;
    conv_params(a, p, V);
    // tokens a thread walks: 4 .. 64, as many as leave 512 threads an SM, 1024 where they move
    // less at a time (K - 1 rows and the taps are read once a piece).  Measured on this build, the
    // rule's own first: 8 x 2048 x 768 bf16: 40 tokens 14.8 us; 4 25.3, 8 17.9, 12 15.6, 16 16.0, 20
    // 16.5, 24 13.5, 32 14.2, 64 17.4.  2 x 32768 x 2048: 64 tokens 94 us; 4 227, 8 151, 16 113, 32 99.
    // 3 x 701 x 1001 fp32, K = 3: 13 tokens 7.8 us; 4 9.4, 8 8.3, 10 7.1, 16 8.5, 27 10.5
    const long long fill = (long long)a.B * a.T * p.nv / ((V == 4 ? 512LL : 1024LL) * kSMs);
    p.len = (int)(fill < 4 ? 4 : fill > 64 ? 64 : fill);
    p.pieces = (a.T + p.len - 1) / p.len;
    const long long n = (long long)a.B * p.pieces * p.nv;
    const long long blocks = (n + kThreads - 1) / kThreads;
    if (blocks > 0x7fffffffLL) return -2;
    p.few = blocks * kThreads <= 0x7fffffffLL;
    switch (a.K) {
    case 1: ttt_short_conv_fwd_kernel<T, V, 1><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    case 2: ttt_short_conv_fwd_kernel<T, V, 2><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    case 3: ttt_short_conv_fwd_kernel<T, V, 3><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    default: ttt_short_conv_fwd_kernel<T, V, 4><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    }
    return cudaGetLastError() == cudaSuccess ? 1 : -4;
}

// The backward pass' pieces: 128 tokens, fewer where that leaves an SM fewer than 300 threads
// (8 x 2048 x 768 bf16: 64 tokens 23.9 us, 32 27.9, 16 34.2; 3 x 701 x 1001 fp32: 32 tokens
// 11.7 us, 64 17.7).  By sizes alone, as the workspace is.
int bwd_len(int B, int T, int C)
{
    const long long vecs = (long long)B * (C % 4 ? C : C / 4);
    int len = 128;
    while (len > 8 && vecs * ((T + len - 1) / len) < 300LL * kSMs) len /= 2;
    return len;
}
long long bwd_part_rows(int B, int T, int C)
{
    const int len = bwd_len(B, T, C);
    return ((long long)B * ((T + len - 1) / len) + kRows - 1) / kRows;
}

template <typename T, int V> int bwd_width(const ConvArgs &a)
{
    ConvParams p;
    conv_params(a, p, V);
    p.len = bwd_len(a.B, a.T, a.C);
    p.pieces = (a.T + p.len - 1) / p.len;
    const bool sums = a.dweight || a.dbias;
    p.part = sums ? static_cast<float *>(a.ws) : nullptr;
    const long long rows = bwd_part_rows(a.B, a.T, a.C), blocks = rows * ((p.nv + 31) / 32);
    if (blocks > 0x7fffffffLL) return -2;
    switch (a.K) {
    case 1: ttt_short_conv_bwd_kernel<T, V, 1><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    case 2: ttt_short_conv_bwd_kernel<T, V, 2><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    case 3: ttt_short_conv_bwd_kernel<T, V, 3><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    default: ttt_short_conv_bwd_kernel<T, V, 4><<<(unsigned)blocks, kThreads, 0, a.stream>>>(p); break;
    }
    if (sums) {
        const long long n = (long long)a.C * (a.K + 1);
        ttt_short_conv_sum_kernel<<<(unsigned)((n + 31) / 32), 256, 0, a.stream>>>(p.part, (int)rows, n, (long long)a.C * a.K, a.dweight, a.dbias);
    }
    return cudaGetLastError() == cudaSuccess ? (sums ? 2 : 1) : -4;
}

}  // namespace

// Four channels a thread at most, 8 bytes of bf16: with eight the window, the taps and their
// sums take so many registers that too few threads are left to wait for memory (2 x 32768 x
// 2048 forward: 107 us in the build that took 95 with four).
int launch_conv_fwd(const ConvArgs &a)
{
    switch (widest(a, 4)) {
    case 4: return a.bf16 ? fwd_width<__nv_bfloat16, 4>(a) : fwd_width<float, 4>(a);
    case 2: return a.bf16 ? fwd_width<__nv_bfloat16, 2>(a) : fwd_width<float, 2>(a);
    default: return a.bf16 ? fwd_width<__nv_bfloat16, 1>(a) : fwd_width<float, 1>(a);
    }
}

size_t conv_bwd_workspace(int B, int T, int C, int K) { return 4 * (size_t)bwd_part_rows(B, T, C) * C * (K + 1); }

int launch_conv_bwd(const ConvArgs &a)
{
    switch (widest(a, 4)) {
    case 4: return a.bf16 ? bwd_width<__nv_bfloat16, 4>(a) : bwd_width<float, 4>(a);
    case 2: return a.bf16 ? bwd_width<__nv_bfloat16, 2>(a) : bwd_width<float, 2>(a);
    default: return a.bf16 ? bwd_width<__nv_bfloat16, 1>(a) : bwd_width<float, 1>(a);
    }
}

}  // namespace ttt
