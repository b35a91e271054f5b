// ttt_scan_fwd.cu -- the selective state space scan, forward:
//     d_t = softplus(delta_t + bias) (or delta_t), h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,
//     y_t = (C_t . h_t + D x_t) silu(z_t),
// for every channel with N states; B_t and C_t are shared by the channels of a group, A is
// [C,N].  A reset before token t makes h_{t-1} zero there.
//
// Bound by the exponentials and the products: one ex2 and four FMA-pipe operations a state
// and token, 32 states a clock and SM by either pipe; the tensors read and written once take
// two thirds of that time at N = 16 in bf16.
#include "ttt_scan.cuh"

namespace ttt {
namespace {

using namespace scan;

constexpr int kTile = kScanChunk;  // tokens staged at a time: a chunk between stored states
constexpr int kCB = 16;            // channels of a block: 32 bytes of a bf16 row, one sector

// ------------------------------------------------------------------ a few tokens
//
// LN neighbouring lanes a channel, four states each, token after token straight from memory:
// decoding steps, whose cost is the states' read and write and one trip to memory.
template <typename T, int LN> __global__ void __launch_bounds__(128) ttt_scan_step_kernel(const __grid_constant__ Params p)
{
    const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) / LN;
    const int n0 = 4 * (threadIdx.x % LN), b = blockIdx.y;
    const bool on = i < p.C;
    const int c = on ? (int)i : p.C - 1, g = c / p.cpg;
    const size_t row = ((size_t)b * p.C + c) * p.N;
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *dl = static_cast<const T *>(p.delta) + b * p.ds[0] + c;
    const T *z = p.z ? static_cast<const T *>(p.z) + b * p.zs[0] + c : nullptr;
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.bs[0] + g * p.bs[2], *Cm = static_cast<const T *>(p.Cm) + b * p.cs[0] + g * p.cs[2];
    Quad h = quad(p.start ? load_states(p.start + row, n0, p.N, 0.f) : make_float4(0.f, 0.f, 0.f, 0.f));
    Quad A = quad(load_states(p.A + (size_t)c * p.N, n0, p.N, 0.f));
    A.a = __fmul2_rn(A.a, make_float2(kLog2e, kLog2e));
    A.b = __fmul2_rn(A.b, make_float2(kLog2e, kLog2e));
    const float D = p.D ? p.D[c] : 0.f, bias = p.bias ? p.bias[c] : 0.f;
    for (int t = 0; t < p.T; ++t) {
        if (p.states && t % kScanChunk == 0 && on)
            store_states(p.states + (((size_t)b * p.chunks + t / kScanChunk) * p.C + c) * p.N, n0, p.N, four(h));
        if (p.reset && p.reset[(size_t)b * p.T + t]) h = quad(make_float4(0.f, 0.f, 0.f, 0.f));
        float4 Bt = make_float4(0.f, 0.f, 0.f, 0.f), Ct = Bt;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + j < p.N) {
                (&Bt.x)[j] = get(Bm + t * p.bs[1] + n0 + j);
                (&Ct.x)[j] = get(Cm + t * p.cs[1] + n0 + j);
            }
        const float xv = get(x + t * p.xs[1]), zv = z ? get(z + t * p.zs[1]) : 0.f;
        float d = get(dl + t * p.ds[1]) + bias, e;
        if (p.softplus) d = softplus(d, e);
        step(h, d, d * xv, A, Bt);
        float y = dot(h, Ct);
#pragma unroll
        for (int s = LN / 2; s > 0; s >>= 1) y += __shfl_xor_sync(0xffffffffu, y, s);
        y = fmaf(D, xv, y);
        if (z) y *= zv * sigmoid(zv);
        if (on && n0 == 0) put(static_cast<T *>(p.y) + ((size_t)b * p.T + t) * p.C + c, y);
    }
    if (p.y_state && on) store_states(p.y_state + row, n0, p.N, four(h));
}

// ------------------------------------------------------------------------- tiles
//
// A block takes kCB channels of a group and one piece of the sequence, a tile of tokens at a
// time: rates, inputs, B and C go to shared memory in fp32 once, then every warp scans its
// 32 / LN channels with LN lanes a channel (the upper lane bits, so that lanes next to each
// other read the same B and C), then the outputs get D x and the gate.  The next tile's
// tensors are on their way in registers during the scan.
// SUM: only the piece's map, from a zero state (its sum of rates, its own contribution).
template <typename T, int LN, bool VEC, bool SUM>
__global__ void __launch_bounds__(kCB *LN) ttt_scan_fwd_kernel(const __grid_constant__ Params p)
{
    constexpr int kThreads = kCB * LN, CL = 32 / LN, NP = 4 * LN;
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;      // elements of one access
    constexpr int kRowVecs = kCB / V, kVecs = kTile * kRowVecs, kIt = (kVecs + kThreads - 1) / kThreads;
    constexpr int kBV = V < NP ? V : NP, kBVecs = kTile * NP / kBV, kBIt = (kBVecs + kThreads - 1) / kThreads;
    constexpr int kYPitch = 24;                           // rows of outputs on different banks
    __shared__ float2 du[kTile][kCB];
    __shared__ __align__(16) float bs[kTile][NP];
    __shared__ __align__(16) float cs[SUM ? 1 : kTile][NP];
    __shared__ __align__(16) float ys[SUM ? 1 : kTile][kYPitch];

    const int g = blockIdx.x / p.blocks, c0 = g * p.cpg + (blockIdx.x % p.blocks) * kCB;
    const int cend = (g + 1) * p.cpg, seg = blockIdx.y, b = blockIdx.z;
    const int tb = seg * p.seg_len, te = min(p.T, tb + p.seg_len);
    const int tid = threadIdx.x, lane = tid & 31;
    const int cl = tid / 32 * CL + lane % CL, n0 = 4 * (lane / CL), c = c0 + cl;
    const bool on = c < cend;

    const T *x = static_cast<const T *>(p.x) + b * p.xs[0], *dl = static_cast<const T *>(p.delta) + b * p.ds[0];
    const T *z = static_cast<const T *>(p.z) + b * p.zs[0];
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.bs[0] + g * p.bs[2], *Cm = static_cast<const T *>(p.Cm) + b * p.cs[0] + g * p.cs[2];
    const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;

    Quad A = quad(make_float4(0.f, 0.f, 0.f, 0.f)), h = A;
    if (on) {
        A = quad(load_states(p.A + (size_t)c * p.N, n0, p.N, 0.f));
        A.a = __fmul2_rn(A.a, make_float2(kLog2e, kLog2e));
        A.b = __fmul2_rn(A.b, make_float2(kLog2e, kLog2e));
        if (!SUM && p.start) h = quad(load_states(p.start + (((size_t)b * p.segs + seg) * p.C + c) * p.N, n0, p.N, 0.f));
    }

    // the tile's raw tensors
    Pack<T, V> px[kIt], pd[kIt], pz[SUM ? 1 : kIt];
    Pack<T, kBV> pb[kBIt], pc[SUM ? 1 : kBIt];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * kThreads, t = t0 + v / kRowVecs, ch = c0 + v % kRowVecs * V;
            px[i].raw = pd[i].raw = {};
            if constexpr (!SUM) pz[i].raw = {};
            if ((kVecs % kThreads == 0 || v < kVecs) && t < te && ch < cend) {
                px[i].load(x + t * p.xs[1] + ch);
                pd[i].load(dl + t * p.ds[1] + ch);
                if constexpr (!SUM)
                    if (p.z) pz[i].load(z + t * p.zs[1] + ch);
            }
        }
#pragma unroll
        for (int i = 0; i < kBIt; ++i) {
            const int v = tid + i * kThreads, t = t0 + v / (NP / kBV), n = v % (NP / kBV) * kBV;
            pb[i].raw = {};
            if constexpr (!SUM) pc[i].raw = {};
            if ((kBVecs % kThreads == 0 || v < kBVecs) && t < te && n < p.N) {
                pb[i].load(Bm + t * p.bs[1] + n);
                if constexpr (!SUM) pc[i].load(Cm + t * p.cs[1] + n);
            }
        }
    };
    float bias[V], Dv[V];
    // (a thread's channels are the same in every pass: kThreads is a multiple of a row's vectors)
    static_assert(kThreads % kRowVecs == 0, "");
    {
        const int ch = c0 + tid % kRowVecs * V;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            bias[j] = p.bias && ch + j < cend ? p.bias[ch + j] : 0.f;
            Dv[j] = p.D && ch + j < cend ? p.D[ch + j] : 0.f;
        }
    }
    float rate_sum = 0.f;  // SUM: of this thread's tokens and channel pieces
    unsigned any_cut = 0;

    fetch(tb);
    for (int t0 = tb; t0 < te; t0 += kTile) {
        const int nt = min(kTile, te - t0);
        if (!SUM && p.states && on)
            store_states(p.states + (((size_t)b * p.chunks + t0 / kScanChunk) * p.C + c) * p.N, n0, p.N, four(h));
        unsigned cut = 0;  // tokens of the tile with a reset
        if (reset) cut = __ballot_sync(0xffffffffu, lane < nt && reset[t0 + lane]);
        any_cut |= cut;
        float xf[kIt][V];
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * kThreads, t = v / kRowVecs, ch = v % kRowVecs * V;
            if (kVecs % kThreads && v >= kVecs) break;
            float d[V];
            unpack(px[i], xf[i]);
            unpack(pd[i], d);
            const bool live = t < nt && c0 + ch < cend;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float e;
                d[j] += bias[j];
                if (p.softplus) d[j] = softplus(d[j], e);
                if (!live) d[j] = 0.f;  // past the end: the state stays
                du[t][ch + j] = make_float2(d[j], d[j] * xf[i][j]);
            }
        }
#pragma unroll
        for (int i = 0; i < kBIt; ++i) {
            const int v = tid + i * kThreads, t = v / (NP / kBV), n = v % (NP / kBV) * kBV;
            if (kBVecs % kThreads && v >= kBVecs) break;
            float f[kBV];
            unpack(pb[i], f);
#pragma unroll
            for (int j = 0; j < kBV; ++j) bs[t][n + j] = f[j];
            if constexpr (!SUM) {
                unpack(pc[i], f);
#pragma unroll
                for (int j = 0; j < kBV; ++j) cs[t][n + j] = f[j];
            }
        }
        float zf[SUM ? 1 : kIt][V];
        if constexpr (!SUM)
#pragma unroll
            for (int i = 0; i < kIt; ++i) unpack(pz[i], zf[i]);
        if (t0 + kTile < te) fetch(t0 + kTile);
        __syncthreads();
        if constexpr (SUM) {
#pragma unroll 4
            for (int t = 0; t < kTile; ++t) {
                const float2 w = du[t][cl];
                if (cut >> t & 1) {
                    h = quad(make_float4(0.f, 0.f, 0.f, 0.f));
                    rate_sum = 0.f;
                }
                step(h, w.x, w.y, A, *reinterpret_cast<const float4 *>(&bs[t][n0]));
                rate_sum += w.x;
            }
            __syncthreads();
        } else {
#pragma unroll 1
            for (int t = 0; t < kTile; t += 4) {
                float yv[4];
                if (cut >> t & 15) {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 w = du[t + k][cl];
                        if (cut >> (t + k) & 1) h = quad(make_float4(0.f, 0.f, 0.f, 0.f));
                        step(h, w.x, w.y, A, *reinterpret_cast<const float4 *>(&bs[t + k][n0]));
                        yv[k] = dot(h, *reinterpret_cast<const float4 *>(&cs[t + k][n0]));
                    }
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 w = du[t + k][cl];
                        step(h, w.x, w.y, A, *reinterpret_cast<const float4 *>(&bs[t + k][n0]));
                        yv[k] = dot(h, *reinterpret_cast<const float4 *>(&cs[t + k][n0]));
                    }
                }
                spread_sum<4, LN, CL>(yv);
                // LN lanes hold the four tokens' sums: 4 / LN each, or LN / 4 lanes the same one
                constexpr int K = LN < 4 ? 4 / LN : 1, dup = LN > 4 ? LN / 4 : 1;
                const int at = lane / CL / dup * K;
                if (lane / CL % dup == 0)
#pragma unroll
                    for (int k = 0; k < K; ++k) ys[t + at + k][cl] = yv[k];
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kIt; ++i) {
                const int v = tid + i * kThreads, t = v / kRowVecs, ch = v % kRowVecs * V;
                if (kVecs % kThreads && v >= kVecs) break;
                if (t >= nt || c0 + ch >= cend) continue;
                float o[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    o[j] = fmaf(Dv[j], xf[i][j], ys[t][ch + j]);
                    if (p.z) o[j] *= zf[i][j] * sigmoid(zf[i][j]);
                }
                Pack<T, V> q;
                pack(q, o);
                q.store(static_cast<T *>(p.y) + ((size_t)b * p.T + t0 + t) * p.C + c0 + ch);
            }
        }
    }
    if constexpr (SUM) {
        const size_t at = ((size_t)b * p.segs + seg) * p.C + c;
        if (on) {
            store_states(p.H + at * p.N, n0, p.N, four(h));
            if (n0 == 0) p.rate_sum[at] = rate_sum;
        }
        if (blockIdx.x == 0 && tid == 0) p.cut[b * p.segs + seg] = any_cut != 0;
    } else if (p.y_state && on && seg == p.segs - 1) {
        store_states(p.y_state + ((size_t)b * p.C + c) * p.N, n0, p.N, four(h));
    }
}

// The state before every piece from the pieces' maps: start [B,segs,C,N] over H (in place),
// one thread a channel and state.  The last piece's map is not made.
__global__ void __launch_bounds__(256) ttt_scan_join_kernel(const __grid_constant__ Params p, const float *h0)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, per = (long long)p.C * p.N;
    const int b = blockIdx.y;
    if (i >= per) return;
    const int c = (int)(i / p.N);
    const float A = p.A[i] * kLog2e;
    float h = h0 ? h0[b * per + i] : 0.f;
    for (int s = 0; s < p.segs; ++s) {
        const size_t at = (size_t)b * p.segs + s;
        float *w = p.H + at * per + i;
        const float own = s + 1 < p.segs ? *w : 0.f;
        *w = h;
        if (s + 1 < p.segs) h = p.cut[at] ? own : fmaf(ex2(A * p.rate_sum[at * p.C + c]), h, own);
    }
}

template <typename T, int LN, bool VEC> int launch_tiles(Params &p, const ScanArgs &a)
{
    p.blocks = (p.cpg + kCB - 1) / kCB;
    const dim3 grid(p.G * p.blocks, p.segs, p.B);
    if (p.segs > 1) {
        const dim3 part(grid.x, p.segs - 1, p.B);
        ttt_scan_fwd_kernel<T, LN, VEC, true><<<part, kCB * LN, 0, a.stream>>>(p);
        const dim3 jg((unsigned)(((long long)p.C * p.N + 255) / 256), p.B);
        ttt_scan_join_kernel<<<jg, 256, 0, a.stream>>>(p, a.h0);
        p.start = p.H;
    }
    ttt_scan_fwd_kernel<T, LN, VEC, false><<<grid, kCB * LN, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? (p.segs > 1 ? 3 : 1) : -4;
}

template <typename T, int LN> int launch_lanes(Params &p, const ScanArgs &a, bool vec)
{
    if (p.T <= kScanStepTokens) {
        const dim3 grid((unsigned)(((long long)p.C * LN + 127) / 128), p.B);
        ttt_scan_step_kernel<T, LN><<<grid, 128, 0, a.stream>>>(p);
        return cudaGetLastError() == cudaSuccess ? 1 : -4;
    }
    return vec ? launch_tiles<T, LN, true>(p, a) : launch_tiles<T, LN, false>(p, a);
}

template <typename T> int launch_type(Params &p, const ScanArgs &a, bool vec)
{
    switch (lanes(p.N)) {
    case 2: return launch_lanes<T, 2>(p, a, vec);
    case 4: return launch_lanes<T, 4>(p, a, vec);
    case 8: return launch_lanes<T, 8>(p, a, vec);
    default: return launch_lanes<T, 16>(p, a, vec);
    }
}

}  // namespace

namespace {

// Pieces of the sequence: as many as give every scheduler two warps, of 256 tokens and more.
ScanPieces pieces(int B, int T, int C, int N, int G)
{
    const int LN = scan::lanes(N), chunks = (T + kScanChunk - 1) / kScanChunk;
    const long long warps = (long long)B * G * ((C / G + kCB - 1) / kCB) * kCB * LN / 32;
    return scan::cut(chunks, warps, 8LL * 152, 8);
}

}  // namespace

size_t scan_fwd_workspace(int B, int T, int C, int N, int G)
{
    const ScanPieces s = pieces(B, T, C, N, G);
    if (T <= kScanStepTokens || s.segs <= 1) return 0;
    return 4 * (size_t)B * s.segs * ((size_t)C * (N + 1) + 1);
}

int launch_scan_fwd(const ScanArgs &a)
{
    Params p = {};
    params(a, p);
    p.start = a.h0;
    p.y = a.y;
    p.y_state = a.h_last;
    const ScanPieces s = pieces(a.B, a.T, a.C, a.N, a.G);
    p.segs = a.T <= kScanStepTokens ? 1 : s.segs;
    p.seg_len = s.len;
    if (p.segs > 1) {
        p.H = static_cast<float *>(a.ws);
        p.rate_sum = p.H + (size_t)a.B * s.segs * a.C * a.N;
        p.cut = reinterpret_cast<int *>(p.rate_sum + (size_t)a.B * s.segs * a.C);
    }
    const bool vec = wide(a);
    return a.bf16 ? launch_type<__nv_bfloat16>(p, a, vec) : launch_type<float>(p, a, vec);
}

}  // namespace ttt
