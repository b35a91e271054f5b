// ttt_scan_fwd.cu -- the selective state space scan, forward:
//     d_t = softplus(delta_t + bias) (or delta_t), h_t = exp(d_t A) h_{t-1} + d_t x_t B_t,
//     y_t = (C_t . h_t + D x_t) silu(z_t),
// for every channel with N states; B_t and C_t are shared by the channels of a group, A is
// [C,N].  A reset before token t makes h_{t-1} zero there.
//
// Bound by the exponentials and the products: one ex2 and four FMA-pipe operations a state
// and token, 32 states a clock and SM by either pipe (measured: 9.5e12 a second), 43 us at
// 8 x 2048 tokens of 1536 channels with 16 states, where the tensors read and written once take
// 30 us.  Three kernels (bf16, 16 states):
//   a few tokens       64 x 1 x 1536           7.6 us from cold caches (states 2 x 6.3 MB)
//   whole sequences    8 x 2048 x 1536         182 us
//   pieces in parallel 1 x 32768 x 2048        214 us the pieces' maps, 9 us joining them,
//                                              300 us the outputs (115 us by either pipe each)
#include "ttt_scan.cuh"

namespace ttt {
namespace {

using namespace scan;

constexpr int kTile = kScanChunk;  // tokens staged at a time: a chunk between stored states

// entries n0 .. n0 + 3 of a row of N of B or C, zeros past its end
template <bool FOURS, typename T> __device__ __forceinline__ float4 load_four(const T *row, int n0, int N)
{
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    if constexpr (FOURS) {
        if (n0 < N) {
            Pack<T, 4> q;
            q.load(row + n0);
            unpack(q, v);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + j < N) v[j] = get(row + n0 + j);
    }
    return make_float4(v[0], v[1], v[2], v[3]);
}

// ------------------------------------------------------------------ a few tokens
//
// LN neighbouring lanes a channel, four states each, token after token straight from memory:
// decoding steps, whose cost is the states' read and write and one trip to memory.
// FOURS: N a multiple of four, all states, B and C aligned to four of theirs: no branch stands
// between the loads, which wait for memory together.
template <typename T, int LN, bool FOURS>
__global__ void __launch_bounds__(128) ttt_scan_step_kernel(const __grid_constant__ Params p)
{
    auto load_states = [](const float *row, int n0, int N) {
        if constexpr (!FOURS) return scan::load_states(row, n0, N);
        else return n0 < N ? *reinterpret_cast<const float4 *>(row + n0) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    auto store_states = [](float *row, int n0, int N, float4 v) {
        if constexpr (!FOURS) scan::store_states(row, n0, N, v);
        else if (n0 < N) *reinterpret_cast<float4 *>(row + n0) = v;
    };
    const long long i = ((long long)blockIdx.x * 128 + threadIdx.x) / LN;
    const int n0 = 4 * (threadIdx.x % LN), b = blockIdx.y;
    const bool on = i < p.C;
    const int c = on ? (int)i : p.C - 1, g = p.G == 1 ? 0 : c / p.cpg;
    const size_t row = ((size_t)b * p.C + c) * p.N;
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *dl = static_cast<const T *>(p.delta) + b * p.ds[0] + c;
    const T *z = p.z ? static_cast<const T *>(p.z) + b * p.zs[0] + c : nullptr;
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.bs[0] + g * p.bs[2], *Cm = static_cast<const T *>(p.Cm) + b * p.cs[0] + g * p.cs[2];
    Quad h = quad(p.start ? load_states(p.start + row, n0, p.N) : make_float4(0.f, 0.f, 0.f, 0.f));
    Quad A = quad(load_states(p.A + (size_t)c * p.N, n0, p.N));
    A.a = __fmul2_rn(A.a, make_float2(kLog2e, kLog2e));
    A.b = __fmul2_rn(A.b, make_float2(kLog2e, kLog2e));
    const float D = p.D ? p.D[c] : 0.f, bias = p.bias ? p.bias[c] : 0.f;
    for (int t = 0; t < p.T; ++t) {
        if (p.states && t % kScanChunk == 0 && on)
            store_states(p.states + (((size_t)b * p.chunks + t / kScanChunk) * p.C + c) * p.N, n0, p.N, four(h));
        if (p.reset && p.reset[(size_t)b * p.T + t]) h = quad(make_float4(0.f, 0.f, 0.f, 0.f));
        const float4 Bt = load_four<FOURS>(Bm + t * p.bs[1], n0, p.N), Ct = load_four<FOURS>(Cm + t * p.cs[1], n0, p.N);
        const float xv = get(x + t * p.xs[1]), zv = z ? get(z + t * p.zs[1]) : 0.f;
        float d = get(dl + t * p.ds[1]) + bias;
        if (p.softplus) d = softplus<T>(d);
        step(h, d, d * xv, A, Bt);
        float2 s2;
        dot(s2, h, Ct, true);
        float y = s2.x + s2.y;
#pragma unroll
        for (int s = LN / 2; s > 0; s >>= 1) y += __shfl_xor_sync(0xffffffffu, y, s);
        y = fmaf(D, xv, y);
        if (z) y *= zv * sigmoid<T>(zv);
        if (on && n0 == 0) put(static_cast<T *>(p.y) + ((size_t)b * p.T + t) * p.C + c, y);
    }
    if (p.y_state && on) store_states(p.y_state + row, n0, p.N, four(h));
}

// ------------------------------------------------------------------------- tiles
//
// A lane keeps 4 Q states of a channel in registers, LN lanes a channel (the upper lane bits,
// so that lanes next to each other read the same B and C), a warp 32 / LN neighbouring
// channels, a block four warps of a group's channels and one piece of the sequence.  B and C
// go to shared memory in fp32, a tile of tokens at a time and one tile ahead; x, delta and z
// come straight from memory, kAt tokens ahead.
// SUM: only the piece's map, from a zero state (its sum of rates, its own contribution).
//
// 16 states a lane: B and C are read once for 512 states, and no output is summed over lanes (4
// states a lane wait for shared memory, 418 us at 1 x 32768 x 2048 for the outputs alone; 16
// with the token tensors staged there as well 337 us; straight from memory 300).  111
// instructions a warp and token, issue slots 62% busy, FMA pipe 52%, ex2 43% (maps 54%).  Four
// blocks an SM by 128 registers; five or six spill (313 and 334 us).
constexpr int kWarps = 4;

template <typename T, int LN, int Q, bool VEC, bool SUM>
__global__ void __launch_bounds__(32 * kWarps, 4) ttt_scan_fwd_kernel(const __grid_constant__ Params p)
{
    constexpr int NT = 32 * kWarps, CL = 32 / LN, CB = kWarps * CL, NP = 4 * LN * Q, kAt = 4;
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;  // elements of one access of B and C
    constexpr int kVecs = kTile * NP / V, kIt = (kVecs + NT - 1) / NT;
    __shared__ __align__(16) float bs[2][kTile][NP];
    __shared__ __align__(16) float cs[SUM ? 1 : 2][SUM ? 1 : kTile][NP];

    const int g = blockIdx.x / p.blocks, cend = (g + 1) * p.cpg, seg = blockIdx.y, b = blockIdx.z;
    const int tb = seg * p.seg_len, te = min(p.T, tb + p.seg_len);
    const int tid = threadIdx.x, lane = tid & 31;
    const int n0 = 4 * (lane / CL);  // this lane's states: n0 + 4 LN q .. + 3
    int c = g * p.cpg + (blockIdx.x % p.blocks) * CB + tid / 32 * CL + lane % CL;
    const bool on = c < cend;
    if (!on) c = cend - 1;  // (reads what it may, writes nothing)

    const T *x = static_cast<const T *>(p.x) + b * p.xs[0] + c, *dl = static_cast<const T *>(p.delta) + b * p.ds[0] + c;
    const T *z = static_cast<const T *>(p.z) + b * p.zs[0] + c;
    const bool gated = p.z;
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.bs[0] + g * p.bs[2], *Cm = static_cast<const T *>(p.Cm) + b * p.cs[0] + g * p.cs[2];
    const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;
    T *y = static_cast<T *>(p.y) + (size_t)b * p.T * p.C + c;
    const float bias = p.bias ? p.bias[c] : 0.f, D = p.D ? p.D[c] : 0.f;

    const Quad zero = quad(make_float4(0.f, 0.f, 0.f, 0.f));
    Quad A[Q], h[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        A[q] = quad(load_states(p.A + (size_t)c * p.N, n0 + 4 * LN * q, p.N));
        A[q].a = __fmul2_rn(A[q].a, make_float2(kLog2e, kLog2e));
        A[q].b = __fmul2_rn(A[q].b, make_float2(kLog2e, kLog2e));
        h[q] = zero;
        if (!SUM && p.start) h[q] = quad(load_states(p.start + (((size_t)b * p.segs + seg) * p.C + c) * p.N, n0 + 4 * LN * q, p.N));
    }

    Pack<T, V> pb[kIt], pc[SUM ? 1 : kIt];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * NT, t = t0 + v / (NP / V), n = v % (NP / V) * V;
            pb[i].raw = {};
            if constexpr (!SUM) pc[i].raw = {};
            if ((kVecs % NT == 0 || v < kVecs) && t < te && n < p.N) {
                pb[i].load(Bm + t * p.bs[1] + n);
                if constexpr (!SUM) pc[i].load(Cm + t * p.cs[1] + n);
            }
        }
    };
    auto stage = [&](int buf) {
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * NT, t = v / (NP / V), n = v % (NP / V) * V;
            if (kVecs % NT && v >= kVecs) break;
            float f[V];
            unpack(pb[i], f);
            put_floats(&bs[buf][t][n], f);
            if constexpr (!SUM) {
                unpack(pc[i], f);
                put_floats(&cs[buf][t][n], f);
            }
        }
    };
    // kAt tokens of the lane's channel from x, dl, z on, zeros past the end
    Pack<T, 1> px[kAt], pd[kAt], pz[SUM ? 1 : kAt];
    const long long xs = p.xs[1], dls = p.ds[1], zs = p.zs[1];
    x += tb * xs;
    dl += tb * dls;
    z += tb * zs;
    y += (size_t)tb * p.C;
    auto load = [&](int t0) {
        if (t0 + kAt <= te) {
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
                px[k].load(x + k * xs);
                pd[k].load(dl + k * dls);
                if constexpr (!SUM)
                    if (gated) pz[k].load(z + k * zs);
            }
        } else {
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
                px[k].raw = pd[k].raw = {};
                if constexpr (!SUM) pz[k].raw = {};
                if (t0 + k < te) {
                    px[k].load(x + k * xs);
                    pd[k].load(dl + k * dls);
                    if constexpr (!SUM)
                        if (gated) pz[k].load(z + k * zs);
                }
            }
        }
        x += kAt * xs;
        dl += kAt * dls;
        if constexpr (!SUM) z += kAt * zs;
    };
    float rate_sum = 0.f, rate_tile = 0.f;  // SUM: of the tiles before, of this one
    unsigned any_cut = 0;

    fetch(tb);
    load(tb);
    stage(0);
    __syncthreads();
    int buf = 0;
    for (int t0 = tb; t0 < te; t0 += kTile, buf ^= 1) {
        const int nt = min(kTile, te - t0);
        const bool more = t0 + kTile < te;
        if (more) fetch(t0 + kTile);
        if (!SUM && p.states && on)
#pragma unroll
            for (int q = 0; q < Q; ++q)
                store_states(p.states + (((size_t)b * p.chunks + t0 / kScanChunk) * p.C + c) * p.N, n0 + 4 * LN * q, p.N, four(h[q]));
        unsigned cut = 0;  // tokens of the tile with a reset
        if (reset) cut = __ballot_sync(0xffffffffu, lane < nt && reset[t0 + lane]);
        any_cut |= cut;
#pragma unroll 1
        for (int t = 0; t < nt; t += kAt) {
            float d[kAt], u[kAt], xf[kAt], zf[kAt];
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
                float v[1];
                unpack(px[k], v);
                xf[k] = v[0];
                unpack(pd[k], v);
                d[k] = v[0] + bias;
                if constexpr (!SUM) {
                    unpack(pz[k], v);
                    zf[k] = v[0];
                }
            }
            load(t0 + t + kAt);
            if (p.softplus) softplus_all<T>(d);
            if (t + kAt > nt)
#pragma unroll
                for (int k = 0; k < kAt; ++k)
                    if (t + k >= nt) d[k] = 0.f;  // past the end: the state stays
#pragma unroll
            for (int k = 0; k < kAt; ++k) u[k] = d[k] * xf[k];
            float o[kAt];
            auto tokens = [&](auto resets) {
#pragma unroll
                for (int k = 0; k < kAt; ++k) {
                    if (decltype(resets)::value && (cut >> (t + k) & 1)) {
#pragma unroll
                        for (int q = 0; q < Q; ++q) h[q] = zero;
                        rate_sum = rate_tile = 0.f;
                    }
                    float2 s = make_float2(0.f, 0.f);
#pragma unroll
                    for (int q = 0; q < Q; ++q) {
                        step(h[q], d[k], u[k], A[q], *reinterpret_cast<const float4 *>(&bs[buf][t + k][n0 + 4 * LN * q]));
                        if constexpr (!SUM) dot(s, h[q], *reinterpret_cast<const float4 *>(&cs[buf][t + k][n0 + 4 * LN * q]), q == 0);
                    }
                    if constexpr (SUM) {
                        rate_tile += d[k];
                    } else {
                        o[k] = s.x + s.y;
#pragma unroll
                        for (int i = CL; i < 32; i *= 2) o[k] += __shfl_xor_sync(0xffffffffu, o[k], i);
                        const float w = gated ? zf[k] * sigmoid<T>(zf[k]) : 1.f;
                        o[k] = fmaf(D, xf[k], o[k]) * w;
                    }
                }
            };
            if (cut >> t & 15) tokens(Is<true>());
            else tokens(Is<false>());
            if constexpr (!SUM) {
                if (on && (LN == 1 || n0 == 0)) {
                    if (t + kAt <= nt) {
#pragma unroll
                        for (int k = 0; k < kAt; ++k) put(y + (size_t)k * p.C, o[k]);
                    } else {
#pragma unroll
                        for (int k = 0; k < kAt; ++k)
                            if (t + k < nt) put(y + (size_t)k * p.C, o[k]);
                    }
                }
                y += (size_t)kAt * p.C;
            }
        }
        if constexpr (SUM) {
            rate_sum += rate_tile;
            rate_tile = 0.f;
        }
        if (more) stage(buf ^ 1);
        __syncthreads();
    }
    if (!on) return;
    if constexpr (SUM) {
        const size_t at = ((size_t)b * p.segs + seg) * p.C + c;
#pragma unroll
        for (int q = 0; q < Q; ++q) store_states(p.H + at * p.N, n0 + 4 * LN * q, p.N, four(h[q]));
        if (n0 == 0) p.rate_sum[at] = rate_sum;
        if (blockIdx.x == 0 && tid == 0) p.cut[b * p.segs + seg] = any_cut != 0;
    } else if (p.y_state && seg == p.segs - 1) {
#pragma unroll
        for (int q = 0; q < Q; ++q) store_states(p.y_state + ((size_t)b * p.C + c) * p.N, n0 + 4 * LN * q, p.N, four(h[q]));
    }
}

// ----------------------------------------------------------- a whole sequence a block
//
// Where batch and channels alone give every scheduler two warps of four states a lane, a
// sequence need not be cut, and its decays are taken once instead of twice.  A block has
// kLaneCB channels with LN lanes each (the upper lane bits); rates, inputs, B and C go to shared
// memory in fp32 once a tile, the next tile's tensors are on their way in registers.  Bound by
// shared memory's data path (64% busy: B and C are read again for every 128 states) and by the
// latency that two and a half warps a scheduler leave: with the loop's tokens one after the other
// 214 us at 8 x 2048 x 1536, three under way at once 187, stores without bank conflicts 182.  768
// blocks on 152 SMs: six on some, five on others.
constexpr int kLaneCB = 16;  // 32 bytes of a bf16 row, one sector

template <typename T, int LN, bool VEC>
__global__ void __launch_bounds__(kLaneCB *LN) ttt_scan_fwd_lanes_kernel(const __grid_constant__ Params p)
{
    constexpr int CB = kLaneCB, NT = CB * LN, CL = 32 / LN, NP = 4 * LN;
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1;
    constexpr int kRowVecs = CB / V, kVecs = kTile * kRowVecs, kIt = (kVecs + NT - 1) / NT;
    constexpr int kBVecs = kTile * NP / V, kBIt = (kBVecs + NT - 1) / NT;
    constexpr int kAt = 4;  // tokens whose outputs are summed over the lanes together
    static_assert(V <= NP && LN <= kAt && NT % kRowVecs == 0, "");
    __shared__ __align__(16) float ds[kTile][CB], us[kTile][CB], ys[kTile][CB];  // rate, rate x, output
    __shared__ __align__(16) float bs[kTile][NP], cs[kTile][NP];

    const int g = blockIdx.x / p.blocks, c0 = g * p.cpg + (blockIdx.x % p.blocks) * CB, cend = (g + 1) * p.cpg, b = blockIdx.y;
    const int tid = threadIdx.x, lane = tid & 31, cl = tid / 32 * CL + lane % CL, n0 = 4 * (lane / CL), c = c0 + cl;
    const bool on = c < cend;
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0], *dl = static_cast<const T *>(p.delta) + b * p.ds[0];
    const T *z = static_cast<const T *>(p.z) + b * p.zs[0];
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.bs[0] + g * p.bs[2], *Cm = static_cast<const T *>(p.Cm) + b * p.cs[0] + g * p.cs[2];
    const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;

    const Quad zero = quad(make_float4(0.f, 0.f, 0.f, 0.f));
    Quad A = zero, h = zero;
    if (on) {
        A = quad(load_states(p.A + (size_t)c * p.N, n0, p.N));
        A.a = __fmul2_rn(A.a, make_float2(kLog2e, kLog2e));
        A.b = __fmul2_rn(A.b, make_float2(kLog2e, kLog2e));
        if (p.start) h = quad(load_states(p.start + ((size_t)b * p.C + c) * p.N, n0, p.N));
    }
    Pack<T, V> px[kIt], pd[kIt], pz[kIt], pb[kBIt], pc[kBIt];
    const int vch = c0 + tid % kRowVecs * V;  // this thread's channels in every pass
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * NT, t = t0 + v / kRowVecs;
            px[i].raw = pd[i].raw = pz[i].raw = {};
            if ((kVecs % NT == 0 || v < kVecs) && t < p.T && vch < cend) {
                px[i].load(x + t * p.xs[1] + vch);
                pd[i].load(dl + t * p.ds[1] + vch);
                if (p.z) pz[i].load(z + t * p.zs[1] + vch);
            }
        }
#pragma unroll
        for (int i = 0; i < kBIt; ++i) {
            const int v = tid + i * NT, t = t0 + v / (NP / V), n = v % (NP / V) * V;
            pb[i].raw = pc[i].raw = {};
            if ((kBVecs % NT == 0 || v < kBVecs) && t < p.T && n < p.N) {
                pb[i].load(Bm + t * p.bs[1] + n);
                pc[i].load(Cm + t * p.cs[1] + n);
            }
        }
    };
    float bias[V], Dv[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        bias[j] = p.bias && vch + j < cend ? p.bias[vch + j] : 0.f;
        Dv[j] = p.D && vch + j < cend ? p.D[vch + j] : 0.f;
    }
    fetch(0);
    for (int t0 = 0; t0 < p.T; t0 += kTile) {
        const int nt = min(kTile, p.T - t0);
        if (p.states && on) store_states(p.states + (((size_t)b * p.chunks + t0 / kScanChunk) * p.C + c) * p.N, n0, p.N, four(h));
        unsigned cut = 0;  // tokens of the tile with a reset
        if (reset) cut = __ballot_sync(0xffffffffu, lane < nt && reset[t0 + lane]);
        Pack<T, V> qx[kIt], qz[kIt];  // kept for the outputs
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * NT, t = v / kRowVecs;
            if (kVecs % NT && v >= kVecs) break;
            qx[i] = px[i];
            qz[i] = pz[i];
            float d[V], u[V];
            unpack(px[i], u);
            unpack(pd[i], d);
            const bool live = t < nt && vch < cend;
#pragma unroll
            for (int j = 0; j < V; ++j) d[j] += bias[j];
            if (p.softplus) softplus_all<T>(d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!live) d[j] = 0.f;  // past the end: the state stays
                u[j] *= d[j];
            }
            put_turned(ds[t], vch - c0, t, d);
            put_turned(us[t], vch - c0, t, u);
        }
#pragma unroll
        for (int i = 0; i < kBIt; ++i) {
            const int v = tid + i * NT, t = v / (NP / V), n = v % (NP / V) * V;
            if (kBVecs % NT && v >= kBVecs) break;
            float f[V];
            unpack(pb[i], f);
            put_turned(bs[t], n, t, f);
            unpack(pc[i], f);
            put_turned(cs[t], n, t, f);
        }
        if (t0 + kTile < p.T) fetch(t0 + kTile);
        __syncthreads();
        // Three tokens are under way at once: one is read, the one before has its decays taken,
        // the one before that moves the states.
        auto tokens = [&](auto resets) {
            float d, u;
            float4 Bt, Ct;
            Quad a, in;
            float4 Cr;
            auto read = [&](int t, int k) {  // (k has t's low bits, known at compile time)
                d = ds[t][turned(cl, k)];
                u = us[t][turned(cl, k)];
                Bt = *reinterpret_cast<const float4 *>(&bs[t][turned(n0, k)]);
                Ct = *reinterpret_cast<const float4 *>(&cs[t][turned(n0, k)]);
            };
            auto ready = [&]() {
                const float2 uu = make_float2(u, u);
                a = decays(d, A);
                in = {__fmul2_rn(uu, make_float2(Bt.x, Bt.y)), __fmul2_rn(uu, make_float2(Bt.z, Bt.w))};
                Cr = Ct;
            };
            read(0, 0);
            ready();
            read(1, 1);
            constexpr int kUnroll = decltype(resets)::value ? 1 : 2;
#pragma unroll kUnroll
            for (int t = 0; t < kTile; t += kAt) {
                float yv[kAt];
#pragma unroll
                for (int k = 0; k < kAt; ++k) {
                    const Quad a1 = a, in1 = in;
                    const float4 C1 = Cr;
                    ready();
                    read((t + k + 2) % kTile, k + 2);  // (the last two are read for nothing)
                    if (decltype(resets)::value && (cut >> (t + k) & 1)) h = zero;
                    h.a = __ffma2_rn(a1.a, h.a, in1.a);
                    h.b = __ffma2_rn(a1.b, h.b, in1.b);
                    float2 s;
                    dot(s, h, C1, true);
                    yv[k] = s.x + s.y;
                }
                spread_sum<kAt, LN, CL>(yv);
                constexpr int K = kAt / LN;
#pragma unroll
                for (int k = 0; k < K; ++k) ys[t + lane / CL * K + k][turned(cl, lane / CL * K + k)] = yv[k];
            }
        };
        if (cut) tokens(Is<true>());
        else tokens(Is<false>());
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * NT, t = v / kRowVecs;
            if ((kVecs % NT && v >= kVecs) || t >= nt || vch >= cend) continue;
            float o[V], xf[V], zf[V];
            get_turned(ys[t], vch - c0, t, o);
            unpack(qx[i], xf);
            unpack(qz[i], zf);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                o[j] = fmaf(Dv[j], xf[j], o[j]);
                if (p.z) o[j] *= zf[j] * sigmoid<T>(zf[j]);
            }
            Pack<T, V> r;
            pack(r, o);
            r.store(static_cast<T *>(p.y) + ((size_t)b * p.T + t0 + t) * p.C + vch);
        }
    }
    if (p.y_state && on) store_states(p.y_state + ((size_t)b * p.C + c) * p.N, n0, p.N, four(h));
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
    // kAhead pieces' maps are read together: only their order is serial
    constexpr int kAhead = 8;
    for (int s0 = 0; s0 < p.segs; s0 += kAhead) {
        float own[kAhead], sum[kAhead];
        int cut[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s0 + k + 1 < p.segs) {
                const size_t at = (size_t)b * p.segs + s0 + k;
                own[k] = p.H[at * per + i];
                sum[k] = p.rate_sum[at * p.C + c];
                cut[k] = p.cut[at];
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s0 + k < p.segs) {
                p.H[((size_t)b * p.segs + s0 + k) * per + i] = h;
                if (s0 + k + 1 < p.segs) h = cut[k] ? own[k] : fmaf(ex2(A * sum[k]), h, own[k]);
            }
    }
}

// The tile kernel's lanes of a channel: 8 or 16 states a lane.
constexpr int tile_lanes(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : 4; }

template <typename T, int LN, int Q, bool VEC> int launch_tiles(Params &p, const ScanArgs &a)
{
    constexpr int CB = kWarps * 32 / LN;
    p.blocks = (p.cpg + CB - 1) / CB;
    const dim3 grid(p.G * p.blocks, p.segs, p.B);
    if (p.segs > 1) {
        const dim3 part(grid.x, p.segs - 1, p.B);
        ttt_scan_fwd_kernel<T, LN, Q, VEC, true><<<part, 32 * kWarps, 0, a.stream>>>(p);
        const dim3 jg((unsigned)(((long long)p.C * p.N + 255) / 256), p.B);
        ttt_scan_join_kernel<<<jg, 256, 0, a.stream>>>(p, a.h0);
        p.start = p.H;
    }
    ttt_scan_fwd_kernel<T, LN, Q, VEC, false><<<grid, 32 * kWarps, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? (p.segs > 1 ? 3 : 1) : -4;
}

template <typename T, int LN, bool VEC> int launch_whole(Params &p, const ScanArgs &a)
{
    p.blocks = (p.cpg + kLaneCB - 1) / kLaneCB;
    ttt_scan_fwd_lanes_kernel<T, LN, VEC><<<dim3(p.G * p.blocks, p.B), kLaneCB * LN, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 1 : -4;
}

template <typename T, int LN> int launch_step(Params &p, const ScanArgs &a)
{
    const dim3 grid((unsigned)(((long long)p.C * LN + 127) / 128), p.B);
    bool fours = a.N % 4 == 0;
    for (const void *q : {(const void *)a.A, (const void *)a.h0, (const void *)a.h_last, (const void *)a.states})
        fours = fours && reinterpret_cast<uintptr_t>(q) % 16 == 0;
    for (const void *q : {a.Bm, a.Cm}) fours = fours && reinterpret_cast<uintptr_t>(q) % (4 * sizeof(T)) == 0;
    for (int i = 0; i < 3; ++i) fours = fours && (a.bs[i] | a.cs[i]) % 4 == 0;
    if (fours) ttt_scan_step_kernel<T, LN, true><<<grid, 128, 0, a.stream>>>(p);
    else ttt_scan_step_kernel<T, LN, false><<<grid, 128, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 1 : -4;
}

// Is the whole-sequence kernel the one to take?  N up to 16, rows that 16-byte accesses can
// take, seven of its warps an SM at least, and fewer than eight of the tile kernel's, which
// would then have to cut every sequence (us for B x T x 1536 channels, N = 16, bf16, whole
// sequences against pieces: 4 x 2048 140 and 130, 6 x 2048 157 and 169, 8 x 2048 192 and 224,
// 16 x 1024 194 and 206, 32 x 512 169 and 149, where the tile kernel needs no pieces either;
// rows of 1533 channels and 12 states 142 and 132).
bool whole_sequences(int B, int T, int C, int N, int G)
{
    if (N > 16 || N % 8 || C / G % 8 || T <= kScanStepTokens) return false;
    const long long LN = N <= 8 ? 2 : 4;
    const long long warps = (long long)B * G * ((C / G + kLaneCB - 1) / kLaneCB) * kLaneCB * LN / 32;
    const long long others = (long long)B * G * ((C / G + 31) / 32);
    return warps >= 7 * 152 && others < 8 * 152;
}

template <typename T> int launch_type(Params &p, const ScanArgs &a, bool vec)
{
    if (p.T <= kScanStepTokens) {
        switch (lanes(p.N)) {
        case 2: return launch_step<T, 2>(p, a);
        case 4: return launch_step<T, 4>(p, a);
        case 8: return launch_step<T, 8>(p, a);
        default: return launch_step<T, 16>(p, a);
        }
    }
    if (whole_sequences(p.B, p.T, p.C, p.N, p.G)) {
        if (p.N <= 8) return vec ? launch_whole<T, 2, true>(p, a) : launch_whole<T, 2, false>(p, a);
        return vec ? launch_whole<T, 4, true>(p, a) : launch_whole<T, 4, false>(p, a);
    }
    if (p.N <= 8) return vec ? launch_tiles<T, 1, 2, true>(p, a) : launch_tiles<T, 1, 2, false>(p, a);
    switch (tile_lanes(p.N)) {
    case 1: return vec ? launch_tiles<T, 1, 4, true>(p, a) : launch_tiles<T, 1, 4, false>(p, a);
    case 2: return vec ? launch_tiles<T, 2, 4, true>(p, a) : launch_tiles<T, 2, 4, false>(p, a);
    default: return vec ? launch_tiles<T, 4, 4, true>(p, a) : launch_tiles<T, 4, 4, false>(p, a);
    }
}

// Pieces of the sequence: as many as fill the SMs with the 16 warps that each holds, of 64
// tokens and more.
ScanPieces pieces(int B, int T, int C, int N, int G)
{
    if (whole_sequences(B, T, C, N, G)) return {1, T};
    const int CL = 32 / tile_lanes(N), chunks = (T + kScanChunk - 1) / kScanChunk;
    const long long warps = (long long)B * G * ((C / G + CL - 1) / CL);
    return scan::cut(chunks, warps, 16LL * 152, 2);
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
