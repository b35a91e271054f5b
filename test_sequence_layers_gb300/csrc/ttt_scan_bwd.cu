// ttt_scan_bwd.cu -- gradients of the selective state space scan.  With g_t = dy_t silu(z_t),
// d the rate, a_t = exp(d_t A) and s_t the gradient of h_t,
//     s_t = g_t C_t + a_{t+1} s_{t+1},      q_t = a_t s_t h_{t-1},
//     dC_t = sum_c g_t h_t,  dB_t = sum_c s_t d_t x_t,  e_t = sum_n s_t B_t,
//     dx_t = e_t d_t + g_t D,  dd_t = e_t x_t + sum_n q_t A,  dA = sum_t q_t d_t,
//     dD = sum g x,  dz = dy y' silu'(z) (y' the output before the gate), dh0 = a_1 s_1,
// and ddelta = dd times the softplus' slope.  h is computed again from the states that the
// forward pass leaves every kScanChunk tokens: to eight tokens' states in registers, from
// states before every eight tokens in shared memory.
//
// A state and token cost three ex2 (four where sequences are cut) and sixteen FMA-pipe
// operations, 170 us at 8 x 2048 x 1536 with 16 states; the sums over channels (dB, dC: eight
// values over the eight lanes of a state) and over states (three values a channel, over four
// lanes) come on top, and take a quarter of the kernel's time (92 and 60 of 650 us in an earlier
// build).  Measured there, bf16: pieces' maps 79 us, joining them 4, main kernel 540, dB and
// dC of the blocks' sums 12, dA, dD and dbias 4; instructions 204 a warp and token of 256
// states, issue slots 50% busy with the eight warps an SM that 251 registers leave.  Three
// blocks an SM (168 registers, one stage of raw tensors) took 562 us, and 519 in shorter pieces
// whose maps cost the difference; pairs of channels instead of states 583.
#include "ttt_scan.cuh"

namespace ttt {
namespace {

using namespace scan;

constexpr int kTile = kScanChunk, kSub = 8, kSubs = kTile / kSub;

// Channels of a block: LN lanes a channel, two channels a thread.
constexpr int block_channels(int LN) { return LN <= 8 ? 64 : 32; }
constexpr int block_threads(int LN) { return block_channels(LN) * LN / 2; }

// Shared memory of a block, in floats: rates, inputs, gated gradients (then e and y' in the
// places of the latter two) and sum q A; B and C; the states before every kSub tokens; a warp's
// sums for dB and dC, twice; a thread's for dA; the tensors as they come, x, delta, dy, z, B, C (kRaw tiles).
template <typename T, int LN, bool VEC> struct Layout {
    static constexpr int CB = block_channels(LN), NT = block_threads(LN), NP = 4 * LN, W = NT / 32;
    static constexpr int kRaw = !VEC ? 0 : sizeof(T) == 2 ? 2 : 1;  // (two of fp32 would leave one block an SM)
    static constexpr int d = 0, u = d + kTile * CB, g = u + kTile * CB, q = g + kTile * CB;
    static constexpr int Bm = q + kTile * CB, Cm = Bm + kTile * NP;
    static constexpr int ck = Cm + kTile * NP;
    static constexpr int red = ck + kSubs * NT * 8, red_one = W * kSub * 2 * NP;
    static constexpr int dA = red + 2 * red_one;  // every thread's sums for dA over the tiles before
    static constexpr int raw = dA + NT * 8;
    static constexpr int raw_tokens = kTile * CB * (int)sizeof(T), raw_bc = kTile * NP * (int)sizeof(T);  // bytes of one tensor
    static constexpr int raw_bytes = 4 * raw_tokens + 2 * raw_bc;
    static constexpr int bytes = raw * 4 + kRaw * raw_bytes;
};

// The gradient map of a piece, v -> exp(A rate_sum) v + R, from its end to its start.
template <typename T, int LN, bool VEC>
__global__ void __launch_bounds__(16 * LN) ttt_scan_bwd_map_kernel(const __grid_constant__ Params p)
{
    constexpr int kCB = 16, kThreads = kCB * LN, CL = 32 / LN, NP = 4 * LN;
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, kRowVecs = kCB / V, kVecs = kTile * kRowVecs;
    constexpr int kIt = (kVecs + kThreads - 1) / kThreads;
    constexpr int kBV = V < NP ? V : NP, kBVecs = kTile * NP / kBV, kBIt = (kBVecs + kThreads - 1) / kThreads;
    __shared__ __align__(16) float ds[kTile][kCB], gs[kTile][kCB];  // rate, gated gradient
    __shared__ __align__(16) float cs[kTile][NP];

    const int blocks = (p.cpg + kCB - 1) / kCB;
    const int grp = blockIdx.x / blocks, c0 = grp * p.cpg + (blockIdx.x % blocks) * kCB, cend = (grp + 1) * p.cpg;
    const int seg = blockIdx.y + 1, b = blockIdx.z;  // the first piece's map is not asked for
    const int tb = seg * p.seg_len, te = min(p.T, tb + p.seg_len);
    const int tid = threadIdx.x, lane = tid & 31, cl = tid / 32 * CL + lane % CL, n0 = 4 * (lane / CL), c = c0 + cl;
    const bool on = c < cend;
    const T *dy = static_cast<const T *>(p.dy) + b * p.dys[0], *dl = static_cast<const T *>(p.delta) + b * p.ds[0];
    const T *z = static_cast<const T *>(p.z) + b * p.zs[0], *Cm = static_cast<const T *>(p.Cm) + b * p.cs[0] + grp * p.cs[2];
    const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;
    Quad A = quad(make_float4(0.f, 0.f, 0.f, 0.f)), r = A;
    if (on) {
        A = quad(load_states(p.A + (size_t)c * p.N, n0, p.N));
        A.a = __fmul2_rn(A.a, make_float2(kLog2e, kLog2e));
        A.b = __fmul2_rn(A.b, make_float2(kLog2e, kLog2e));
    }
    float rate_sum = 0.f, rate_tile = 0.f;  // of the tiles behind, of this one
    unsigned any_cut = 0;
    static_assert(kThreads % kRowVecs == 0, "");
    float bias[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int ch = c0 + tid % kRowVecs * V + j;
        bias[j] = p.bias && ch < cend ? p.bias[ch] : 0.f;
    }
    // the tile's raw tensors, asked for a tile ahead
    Pack<T, V> pg[kIt], pd[kIt], pz[kIt];
    Pack<T, kBV> pc[kBIt];
    const int vch = c0 + tid % kRowVecs * V;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * kThreads, t = t0 + v / kRowVecs;
            pg[i].raw = pd[i].raw = pz[i].raw = {};
            if ((kVecs % kThreads == 0 || v < kVecs) && t < te && vch < cend) {
                pg[i].load(dy + t * p.dys[1] + vch);
                pd[i].load(dl + t * p.ds[1] + vch);
                if (p.z) pz[i].load(z + t * p.zs[1] + vch);
            }
        }
#pragma unroll
        for (int i = 0; i < kBIt; ++i) {
            const int v = tid + i * kThreads, t = t0 + v / (NP / kBV), n = v % (NP / kBV) * kBV;
            pc[i].raw = {};
            if ((kBVecs % kThreads == 0 || v < kBVecs) && t < te && n < p.N) pc[i].load(Cm + t * p.cs[1] + n);
        }
    };
    int t0 = tb + (te - tb - 1) / kTile * kTile;
    fetch(t0);
    for (; t0 >= tb; t0 -= kTile) {
        const int nt = min(kTile, te - t0);
        unsigned cut = 0;
        if (reset) cut = __ballot_sync(0xffffffffu, lane < nt && reset[t0 + lane]);
        any_cut |= cut;
#pragma unroll
        for (int i = 0; i < kIt; ++i) {
            const int v = tid + i * kThreads, t = v / kRowVecs;
            if (kVecs % kThreads && v >= kVecs) break;
            const bool live = t < nt && vch < cend;
            float gf[V], df[V], zf[V];
            unpack(pg[i], gf);
            unpack(pd[i], df);
            unpack(pz[i], zf);
#pragma unroll
            for (int j = 0; j < V; ++j) df[j] += bias[j];
            if (p.softplus) softplus_all<T>(df);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!live) df[j] = 0.f;  // past the end: nothing moves (the gradient is zero there)
                if (p.z) gf[j] *= zf[j] * sigmoid<T>(zf[j]);
            }
            put_floats(&ds[t][vch - c0], df);
            put_floats(&gs[t][vch - c0], gf);
        }
#pragma unroll
        for (int i = 0; i < kBIt; ++i) {
            const int v = tid + i * kThreads, t = v / (NP / kBV), n = v % (NP / kBV) * kBV;
            if (kBVecs % kThreads && v >= kBVecs) break;
            float f[kBV];
            unpack(pc[i], f);
            put_floats(&cs[t][n], f);
        }
        if (t0 > tb) fetch(t0 - kTile);
        __syncthreads();
        auto tokens = [&](auto resets) {
#pragma unroll 8
            for (int t = kTile - 1; t >= 0; --t) {
                const float d = ds[t][cl], w = gs[t][cl];
                const float2 gg = make_float2(w, w);
                const float4 Ct = *reinterpret_cast<const float4 *>(&cs[t][n0]);
                const Quad a = decays(d, A);
                r.a = __fmul2_rn(a.a, __ffma2_rn(gg, make_float2(Ct.x, Ct.y), r.a));
                r.b = __fmul2_rn(a.b, __ffma2_rn(gg, make_float2(Ct.z, Ct.w), r.b));
                rate_tile += d;
                if (decltype(resets)::value && (cut >> t & 1)) {
                    r = quad(make_float4(0.f, 0.f, 0.f, 0.f));
                    rate_sum = rate_tile = 0.f;
                }
            }
        };
        if (cut) tokens(Is<true>());
        else tokens(Is<false>());
        rate_sum += rate_tile;
        rate_tile = 0.f;
        __syncthreads();
    }
    const size_t at = ((size_t)b * p.segs + seg) * p.C + c;
    if (on) {
        store_states(p.H + at * p.N, n0, p.N, four(r));
        if (n0 == 0) p.rate_sum[at] = rate_sum;
    }
    if (blockIdx.x == 0 && tid == 0) p.cut[b * p.segs + seg] = any_cut != 0;
}

// The gradient behind every piece from the maps (in place over H).
__global__ void __launch_bounds__(256) ttt_scan_bwd_join_kernel(const __grid_constant__ Params p, const float *dh_last)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, per = (long long)p.C * p.N;
    const int b = blockIdx.y;
    if (i >= per) return;
    const int c = (int)(i / p.N);
    const float A = p.A[i] * kLog2e;
    float r = dh_last ? dh_last[b * per + i] : 0.f;
    constexpr int kAhead = 8;  // pieces whose maps are read together
    for (int s0 = p.segs - 1; s0 >= 0; s0 -= kAhead) {
        float own[kAhead], sum[kAhead];
        int cut[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s0 - k > 0) {
                const size_t at = (size_t)b * p.segs + s0 - k;
                own[k] = p.H[at * per + i];
                sum[k] = p.rate_sum[at * p.C + c];
                cut[k] = p.cut[at];
            }
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (s0 - k >= 0) {
                p.H[((size_t)b * p.segs + s0 - k) * per + i] = r;
                if (s0 - k > 0) r = cut[k] ? own[k] : fmaf(ex2(A * sum[k]), r, own[k]);
            }
    }
}

template <typename T, int LN, bool VEC>
__global__ void __launch_bounds__(block_threads(LN)) ttt_scan_bwd_kernel(const __grid_constant__ Params p)
{
    using L = Layout<T, LN, VEC>;
    constexpr int CB = L::CB, NT = L::NT, NP = L::NP, CL = 32 / LN;
    constexpr int V = VEC ? 16 / (int)sizeof(T) : 1, kRowVecs = CB / V, kVecs = kTile * kRowVecs;
    constexpr int kBV = V < NP ? V : NP, kBVecs = kTile * NP / kBV;
    static_assert(NT % kRowVecs == 0, "a thread's channels are the same in every pass");
    extern __shared__ __align__(16) float sm[];

    const int grp = blockIdx.x / p.blocks, blk = blockIdx.x % p.blocks;
    const int c0 = grp * p.cpg + blk * CB, cend = (grp + 1) * p.cpg, seg = blockIdx.y, b = blockIdx.z;
    const int tb = seg * p.seg_len, te = min(p.T, tb + p.seg_len);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cl = warp * 2 * CL + lane % CL * 2, ng = lane / CL, n0 = 4 * ng;
    const int ct = turned(cl, cl >> 4);  // where channel cl lies in a row
    const T *x = static_cast<const T *>(p.x) + b * p.xs[0], *dl = static_cast<const T *>(p.delta) + b * p.ds[0];
    const T *z = static_cast<const T *>(p.z) + b * p.zs[0], *dy = static_cast<const T *>(p.dy) + b * p.dys[0];
    const T *Bm = static_cast<const T *>(p.Bm) + b * p.bs[0] + grp * p.bs[2], *Cm = static_cast<const T *>(p.Cm) + b * p.cs[0] + grp * p.cs[2];
    const unsigned char *reset = p.reset ? p.reset + (size_t)b * p.T : nullptr;
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    const float2 zero2 = make_float2(0.f, 0.f);

    // [channel][pair of states]
    float2 A[2][2], r[2][2], dA[2][2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = c0 + cl + k;
        Quad q = quad(zero4);
        if (c < cend) q = quad(load_states(p.A + (size_t)c * p.N, n0, p.N));
        A[k][0] = __fmul2_rn(q.a, make_float2(kLog2e, kLog2e));
        A[k][1] = __fmul2_rn(q.b, make_float2(kLog2e, kLog2e));
        q = quad(zero4);
        if (c < cend && p.start) q = quad(load_states(p.start + (((size_t)b * p.segs + seg) * p.C + c) * p.N, n0, p.N));
        r[k][0] = q.a;
        r[k][1] = q.b;
        dA[k][0] = dA[k][1] = zero2;
        reinterpret_cast<float4 *>(sm + L::dA)[k * NT + tid] = zero4;
    }
    // this thread's channels before and after the scan, and their sums for dD and dbias
    const int vch = tid % kRowVecs * V;
    float bias[V], Dv[V], sD[V], sb[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        const int ch = c0 + vch + j;
        bias[j] = p.bias && ch < cend ? p.bias[ch] : 0.f;
        Dv[j] = p.D && ch < cend ? p.D[ch] : 0.f;
        sD[j] = sb[j] = 0.f;
    }

    // The tile's tensors: asynchronous copies of 16 bytes, each read by the thread that asked
    // for it (token t, channels vch ..), or plain loads where they are not aligned.
    unsigned char *const raw = reinterpret_cast<unsigned char *>(sm + L::raw);
    constexpr int kVecIt = (kVecs + NT - 1) / NT;
    auto copy = [&](int t0, int stage) {
        unsigned char *to = raw + stage * L::raw_bytes;
        const bool in = c0 + vch < cend;
#pragma unroll
        for (int i = 0; i < kVecIt; ++i) {
            const int v = tid + i * NT, t = t0 + v / kRowVecs, n = in && t < te ? 16 : 0;
            if (kVecs % NT && v >= kVecs) break;
            const int r = n ? t : tb, ch = n ? c0 + vch : c0;  // (nothing is read where n is 0)
            copy_async16_part(to + v * 16, x + r * p.xs[1] + ch, n);
            copy_async16_part(to + L::raw_tokens + v * 16, dl + r * p.ds[1] + ch, n);
            copy_async16_part(to + 2 * L::raw_tokens + v * 16, dy + r * p.dys[1] + ch, n);
            if (p.z) copy_async16_part(to + 3 * L::raw_tokens + v * 16, z + r * p.zs[1] + ch, n);
        }
        for (int v = tid; v < kBVecs; v += NT) {
            const int t = t0 + v / (NP / kBV), k = v % (NP / kBV) * kBV, n = t < te && k < p.N ? 16 : 0;
            const int r = n ? t : tb, m = n ? k : 0;
            copy_async16_part(to + 4 * L::raw_tokens + v * 16, Bm + r * p.bs[1] + m, n);
            copy_async16_part(to + 4 * L::raw_tokens + L::raw_bc + v * 16, Cm + r * p.cs[1] + m, n);
        }
        copy_commit();
    };
    // the four tensors' vector v of the tile at t0
    auto tensors = [&](int t0, int nt, int stage, int v, float (&xf)[V], float (&df)[V], float (&gf)[V], float (&zf)[V]) {
        const int t = v / kRowVecs;
        Pack<T, V> px, pd, pg, pz;
        px.raw = pd.raw = pg.raw = pz.raw = {};
        if constexpr (L::kRaw > 0) {
            const unsigned char *from = raw + stage * L::raw_bytes + v * 16;
            px.load_rw(reinterpret_cast<const T *>(from));
            pd.load_rw(reinterpret_cast<const T *>(from + L::raw_tokens));
            pg.load_rw(reinterpret_cast<const T *>(from + 2 * L::raw_tokens));
            if (p.z) pz.load_rw(reinterpret_cast<const T *>(from + 3 * L::raw_tokens));
        } else if (t < nt && c0 + vch < cend) {
            px.load(x + (t0 + t) * p.xs[1] + c0 + vch);
            pd.load(dl + (t0 + t) * p.ds[1] + c0 + vch);
            pg.load(dy + (t0 + t) * p.dys[1] + c0 + vch);
            if (p.z) pz.load(z + (t0 + t) * p.zs[1] + c0 + vch);
        }
        unpack(px, xf);
        unpack(pd, df);
        unpack(pg, gf);
        unpack(pz, zf);
    };

    int t0 = tb + (te - tb - 1) / kTile * kTile, stage = 0;
    if constexpr (L::kRaw > 0) copy(t0, 0);
    for (; t0 >= tb; t0 -= kTile) {
        const int nt = min(kTile, te - t0);
        unsigned cut = 0;
        if (reset) cut = __ballot_sync(0xffffffffu, lane < nt && reset[t0 + lane]);
        float2 h[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int c = c0 + cl + k;
            Quad q = quad(zero4);
            if (c < cend) q = quad(load_states(p.states + (((size_t)b * p.chunks + t0 / kScanChunk) * p.C + c) * p.N, n0, p.N));
            h[k][0] = q.a;
            h[k][1] = q.b;
        }
        if constexpr (L::kRaw > 0) copy_wait<0>();
        if constexpr (L::kRaw == 2)
            if (t0 > tb) copy(t0 - kTile, stage ^ 1);
        // rates, inputs and gated gradients in fp32
#pragma unroll
        for (int i = 0; i < kVecIt; ++i) {
            const int v = tid + i * NT, t = v / kRowVecs;
            if (kVecs % NT && v >= kVecs) break;
            const bool live = t < nt && c0 + vch < cend;
            float xf[V], df[V], gf[V], zf[V];
            tensors(t0, nt, stage, v, xf, df, gf, zf);
#pragma unroll
            for (int j = 0; j < V; ++j) df[j] += bias[j];
            if (p.softplus) softplus_all<T>(df);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (!live) df[j] = 0.f;  // past the end: nothing moves
                xf[j] *= df[j];
            }
            if (p.z)
#pragma unroll
                for (int j = 0; j < V; ++j) gf[j] *= zf[j] * sigmoid<T>(zf[j]);
            const int at = t * CB;
            put_turned(sm + L::d + at, vch, vch >> 4, df);
            put_turned(sm + L::u + at, vch, vch >> 4, xf);
            put_turned(sm + L::g + at, vch, vch >> 4, gf);
        }
        for (int v = tid; v < kBVecs; v += NT) {
            const int t = v / (NP / kBV), n = v % (NP / kBV) * kBV;
            Pack<T, kBV> pb, pc;
            pb.raw = pc.raw = {};
            if constexpr (L::kRaw > 0) {
                const unsigned char *from = raw + stage * L::raw_bytes + 4 * L::raw_tokens + v * 16;
                pb.load_rw(reinterpret_cast<const T *>(from));
                pc.load_rw(reinterpret_cast<const T *>(from + L::raw_bc));
            } else if (t < nt && n < p.N) {
                pb.load(Bm + (t0 + t) * p.bs[1] + n);
                pc.load(Cm + (t0 + t) * p.cs[1] + n);
            }
            float f[kBV];
            unpack(pb, f);
            put_floats(sm + L::Bm + t * NP + n, f);
            unpack(pc, f);
            put_floats(sm + L::Cm + t * NP + n, f);
        }
        __syncthreads();

        auto scan_tile = [&](auto resets) {
            constexpr bool kResets = decltype(resets)::value;
            auto forward = [&](int t, float2 (&hh)[2][2]) {
                const bool zero = kResets && (cut >> t & 1);
                const float2 d = *reinterpret_cast<const float2 *>(&sm[L::d + t * CB + ct]);
                const float2 u = *reinterpret_cast<const float2 *>(&sm[L::u + t * CB + ct]);
                const float4 Bt = *reinterpret_cast<const float4 *>(&sm[L::Bm + t * NP + n0]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 dd = k ? make_float2(d.y, d.y) : make_float2(d.x, d.x), uu = k ? make_float2(u.y, u.y) : make_float2(u.x, u.x);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        const float2 a = decay2(dd, A[k][m]), in = __fmul2_rn(uu, m ? make_float2(Bt.z, Bt.w) : make_float2(Bt.x, Bt.y));
                        const float2 prev = kResets && zero ? zero2 : hh[k][m];
                        hh[k][m] = __ffma2_rn(a, prev, in);
                    }
                }
            };
            // states before every kSub tokens of the tile
            float4 *ck = reinterpret_cast<float4 *>(sm + L::ck) + tid;
#pragma unroll 1
            for (int s = 0; s < kSubs; ++s) {
                ck[(2 * s) * NT] = make_float4(h[0][0].x, h[0][0].y, h[0][1].x, h[0][1].y);
                ck[(2 * s + 1) * NT] = make_float4(h[1][0].x, h[1][0].y, h[1][1].x, h[1][1].y);
                if (s + 1 < kSubs)
#pragma unroll
                    for (int t = 0; t < kSub; ++t) forward(s * kSub + t, h);
            }
#pragma unroll 1
            for (int s = kSubs - 1; s >= 0; --s) {
                const int ts = s * kSub;
                float *const red = sm + L::red + (s & 1) * L::red_one;
                float2 hs[kSub + 1][2][2];
                {
                    const float4 k0 = ck[(2 * s) * NT], k1 = ck[(2 * s + 1) * NT];
                    hs[0][0][0] = make_float2(k0.x, k0.y);
                    hs[0][0][1] = make_float2(k0.z, k0.w);
                    hs[0][1][0] = make_float2(k1.x, k1.y);
                    hs[0][1][1] = make_float2(k1.z, k1.w);
                }
#pragma unroll
                for (int t = 0; t < kSub; ++t) {
#pragma unroll
                    for (int k = 0; k < 2; ++k)
#pragma unroll
                        for (int m = 0; m < 2; ++m) hs[t + 1][k][m] = hs[t][k][m];
                    forward(ts + t, hs[t + 1]);
                }
#pragma unroll
                for (int half = kSub / 4 - 1; half >= 0; --half) {
                    float ve[8], vq[8], vy[8];  // [token of four][channel]: e, sum q A, y'
#pragma unroll
                    for (int i = 3; i >= 0; --i) {
                        const int j = half * 4 + i, t = ts + j;
                        const bool zero = kResets && (cut >> t & 1);
                        const float2 d = *reinterpret_cast<const float2 *>(&sm[L::d + t * CB + ct]);
                        const float2 u = *reinterpret_cast<const float2 *>(&sm[L::u + t * CB + ct]);
                        const float2 g = *reinterpret_cast<const float2 *>(&sm[L::g + t * CB + ct]);
                        const float4 B4 = *reinterpret_cast<const float4 *>(&sm[L::Bm + t * NP + n0]);
                        const float4 C4 = *reinterpret_cast<const float4 *>(&sm[L::Cm + t * NP + n0]);
                        float2 dB[2], dC[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float2 dd = k ? make_float2(d.y, d.y) : make_float2(d.x, d.x);
                            const float2 uu = k ? make_float2(u.y, u.y) : make_float2(u.x, u.x);
                            const float2 gg = k ? make_float2(g.y, g.y) : make_float2(g.x, g.x);
                            float2 e2, q2, y2;
#pragma unroll
                            for (int m = 0; m < 2; ++m) {
                                const float2 Bt = m ? make_float2(B4.z, B4.w) : make_float2(B4.x, B4.y);
                                const float2 Ct = m ? make_float2(C4.z, C4.w) : make_float2(C4.x, C4.y);
                                const float2 s2 = __ffma2_rn(gg, Ct, r[k][m]);
                                dC[m] = k ? __ffma2_rn(gg, hs[j + 1][k][m], dC[m]) : __fmul2_rn(gg, hs[j + 1][k][m]);
                                dB[m] = k ? __ffma2_rn(uu, s2, dB[m]) : __fmul2_rn(uu, s2);
                                y2 = m ? __ffma2_rn(Ct, hs[j + 1][k][m], y2) : __fmul2_rn(Ct, hs[j + 1][k][m]);
                                e2 = m ? __ffma2_rn(Bt, s2, e2) : __fmul2_rn(Bt, s2);
                                const float2 as = __fmul2_rn(decay2(dd, A[k][m]), s2);
                                const float2 q = kResets && zero ? zero2 : __fmul2_rn(as, hs[j][k][m]);
                                q2 = m ? __ffma2_rn(q, A[k][m], q2) : __fmul2_rn(q, A[k][m]);
                                dA[k][m] = __ffma2_rn(q, dd, dA[k][m]);
                                r[k][m] = kResets && zero ? zero2 : as;
                            }
                            ve[2 * i + k] = e2.x + e2.y;
                            vq[2 * i + k] = q2.x + q2.y;
                            vy[2 * i + k] = y2.x + y2.y;
                        }
                        float bc[8] = {dB[0].x, dB[0].y, dB[1].x, dB[1].y, dC[0].x, dC[0].y, dC[1].x, dC[1].y};
                        spread_sum<8, CL, 1>(bc);
                        constexpr int K = CL < 8 ? 8 / CL : 1, dup = CL > 8 ? CL / 8 : 1;
                        float *to = red + (warp * kSub + j) * 2 * NP + n0;
                        if (lane % CL % dup == 0)
#pragma unroll
                            for (int m = 0; m < K; ++m) {
                                const int v = lane % CL / dup * K + m;
                                to[(v / 4) * NP + v % 4] = bc[m];
                            }
                    }
                    spread_sum<8, LN, CL>(ve);
                    spread_sum<8, LN, CL>(vq);
                    spread_sum<8, LN, CL>(vy);
                    __syncwarp();  // these tokens' inputs and gradients have been read: the sums take their places
                    constexpr int K = LN < 8 ? 8 / LN : 1, dup = LN > 8 ? LN / 8 : 1;
                    if (ng % dup == 0)
#pragma unroll
                        for (int m = 0; m < K; ++m) {
                            const int v = ng / dup * K + m, at = (ts + half * 4 + v / 2) * CB + ct + v % 2;
                            sm[L::u + at] = ve[m];
                            sm[L::q + at] = vq[m];
                            sm[L::g + at] = vy[m];
                        }
                }
                __syncthreads();
                // the block's sums over its channels for these kSub tokens (the next ones' go to
                // the other half of red, and come back to this one two barriers later)
                for (int v = tid; v < kSub * 2 * NP; v += NT) {
                    const int j = v / (2 * NP), w = v / NP % 2, n = v % NP;
                    if (ts + j < nt && n < p.N) {
                        float s2 = 0.f;
#pragma unroll
                        for (int i = 0; i < L::W; ++i) s2 += red[(i * kSub + j) * 2 * NP + w * NP + n];
                        p.bc_part[((((size_t)blk * p.B + b) * p.T + t0 + ts + j) * p.G + grp) * 2 * p.N + w * p.N + n] = s2;
                    }
                }
            }
        };
        if (cut) scan_tile(Is<true>());
        else scan_tile(Is<false>());
        // the token tensors' gradients
#pragma unroll
        for (int i = 0; i < kVecIt; ++i) {
            const int v = tid + i * NT, t = v / kRowVecs;
            if ((kVecs % NT && v >= kVecs) || t >= nt || c0 + vch >= cend) continue;
            float xf[V], df[V], gf[V], zf[V], dx[V], dd[V], dz[V], es[V], qs[V], ys[V], ds[V];
            tensors(t0, nt, stage, v, xf, df, gf, zf);
            get_turned(sm + L::u + t * CB, vch, vch >> 4, es);
            get_turned(sm + L::q + t * CB, vch, vch >> 4, qs);
            get_turned(sm + L::g + t * CB, vch, vch >> 4, ys);
            get_turned(sm + L::d + t * CB, vch, vch >> 4, ds);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float slope = 1.f, g = gf[j];
                if (p.softplus) {
                    const float w = df[j] + bias[j], e = exp_neg<T>(fabsf(w));
                    slope = rcp(1.f + e);
                    if (w < 0.f) slope *= e;
                }
                if (p.z) {
                    const float sg = sigmoid<T>(zf[j]), y = fmaf(Dv[j], xf[j], ys[j]);
                    dz[j] = g * y * sg * fmaf(zf[j], 1.f - sg, 1.f);
                    g *= zf[j] * sg;
                }
                dx[j] = fmaf(es[j], ds[j], g * Dv[j]);
                dd[j] = fmaf(es[j], xf[j], kLn2 * qs[j]) * slope;
                sD[j] = fmaf(g, xf[j], sD[j]);
                sb[j] += dd[j];
            }
            const size_t at = ((size_t)b * p.T + t0 + t) * p.C + c0 + vch;
            Pack<T, V> o;
            pack(o, dx);
            o.store(static_cast<T *>(p.dx) + at);
            pack(o, dd);
            o.store(static_cast<T *>(p.ddelta) + at);
            if (p.z) {
                pack(o, dz);
                o.store(static_cast<T *>(p.dz) + at);
            }
        }
        // A tile's part of dA goes to its total by itself: two short sums round less than one
        // over a whole piece.
        float4 *total = reinterpret_cast<float4 *>(sm + L::dA) + tid;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float4 w = total[k * NT];
            w = make_float4(w.x + dA[k][0].x, w.y + dA[k][0].y, w.z + dA[k][1].x, w.w + dA[k][1].y);
            total[k * NT] = w;
            dA[k][0] = dA[k][1] = zero2;
        }
        // (what the next tile writes of d, u, g and q, and asks for in place of its raw tensors,
        // this thread alone has read)
        if constexpr (L::kRaw == 2) stage ^= 1;
        if constexpr (L::kRaw == 1)
            if (t0 > tb) copy(t0 - kTile, 0);
    }
    __syncthreads();

    const size_t part = (size_t)b * p.segs + seg;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int c = c0 + cl + k;
        if (c >= cend) break;
        store_states(p.a_part + (part * p.C + c) * p.N, n0, p.N, reinterpret_cast<const float4 *>(sm + L::dA)[k * NT + tid]);
        if (p.dh0 && seg == 0)
            store_states(p.dh0 + ((size_t)b * p.C + c) * p.N, n0, p.N, make_float4(r[k][0].x, r[k][0].y, r[k][1].x, r[k][1].y));
    }
    // dD and dbias: the threads of one channel, in order
#pragma unroll
    for (int j = 0; j < V; ++j) {
        sm[(tid / kRowVecs) * 2 * CB + vch + j] = sD[j];
        sm[(tid / kRowVecs) * 2 * CB + CB + vch + j] = sb[j];
    }
    __syncthreads();
    for (int v = tid; v < 2 * CB; v += NT) {
        float s = 0.f;
        for (int i = 0; i < NT / kRowVecs; ++i) s += sm[i * 2 * CB + v];
        const int c = c0 + v % CB;
        if (c < cend) p.v_part[(part * 2 + v / CB) * p.C + c] = s;
    }
}

// dB and dC: the channel blocks' sums, in order, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) ttt_scan_bc_kernel(const float *part, int blocks, long long rows, int N, T *dB, T *dC)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x, n = rows * 2 * N;
    if (i >= n) return;
    float s = 0.f;
    for (int k = 0; k < blocks; ++k) s += part[k * n + i];
    const long long row = i / (2 * N);
    const int v = (int)(i - row * 2 * N);
    put((v < N ? dB : dC) + row * N + v % N, s);
}

// out[i] = sum of `rows` partial rows of n, in an order fixed by their number.
struct SumJob {
    const float *part;
    float *out;
    long long n, pitch;
};
struct SumJobs {
    SumJob job[3];
    int rows;
};
__global__ void __launch_bounds__(256) ttt_scan_sum_kernel(const __grid_constant__ SumJobs jobs)
{
    __shared__ float sh[8][32];
    const SumJob &j = jobs.job[blockIdx.y];
    const long long i = (long long)blockIdx.x * 32 + threadIdx.x % 32;
    if ((long long)blockIdx.x * 32 >= j.n || !j.out) return;
    float s = 0.f;
    if (i < j.n)
        for (int r = threadIdx.x / 32; r < jobs.rows; r += 8) s += j.part[r * j.pitch + i];
    sh[threadIdx.x / 32][threadIdx.x % 32] = s;
    __syncthreads();
    if (threadIdx.x < 32 && i < j.n) {
        for (int r = 1; r < 8; ++r) s += sh[r][threadIdx.x];
        j.out[i] = s;
    }
}

ScanPieces pieces(int B, int T, int C, int N, int G)
{
    const int LN = lanes(N), CB = block_channels(LN);
    const long long warps = (long long)B * G * ((C / G + CB - 1) / CB) * block_threads(LN) / 32;
    return scan::cut((T + kScanChunk - 1) / kScanChunk, warps, 16LL * 152, 1);
}

struct Space {
    size_t bc, a, v, H, rate, cut, bytes;  // floats; bytes of all
};
Space space(int B, int T, int C, int N, int G)
{
    const ScanPieces s = pieces(B, T, C, N, G);
    const int CB = block_channels(lanes(N));
    Space w;
    const size_t parts = (size_t)B * s.segs;
    auto up = [](size_t n) { return (n + 3) / 4 * 4; };
    w.bc = 0;
    w.a = up((size_t)((C / G + CB - 1) / CB) * B * T * G * 2 * N);
    w.v = w.a + up(parts * C * N);
    w.H = w.v + up(parts * 2 * C);
    w.rate = w.H + (s.segs > 1 ? up(parts * C * N) : 0);
    w.cut = w.rate + (s.segs > 1 ? up(parts * C) : 0);
    w.bytes = 4 * (w.cut + (s.segs > 1 ? parts : 0));
    return w;
}

template <typename T, int LN, bool VEC> int launch_all(Params &p, const ScanArgs &a)
{
    using L = Layout<T, LN, VEC>;
    int n = 0;
    if (p.segs > 1) {
        const dim3 mg(p.G * ((p.cpg + 15) / 16), p.segs - 1, p.B);
        ttt_scan_bwd_map_kernel<T, LN, VEC><<<mg, 16 * LN, 0, a.stream>>>(p);
        const dim3 jg((unsigned)(((long long)p.C * p.N + 255) / 256), p.B);
        ttt_scan_bwd_join_kernel<<<jg, 256, 0, a.stream>>>(p, a.dh_last);
        p.start = p.H;
        n += 2;
    }
    if (!allow_shared(ttt_scan_bwd_kernel<T, LN, VEC>, L::bytes)) return -4;
    const dim3 grid(p.G * p.blocks, p.segs, p.B);
    ttt_scan_bwd_kernel<T, LN, VEC><<<grid, L::NT, L::bytes, a.stream>>>(p);
    const long long rows = (long long)p.B * p.T * p.G;
    ttt_scan_bc_kernel<T><<<(unsigned)((rows * 2 * p.N + 255) / 256), 256, 0, a.stream>>>(p.bc_part, p.blocks, rows, p.N,
                                                                                         static_cast<T *>(a.dB), static_cast<T *>(a.dC));
    SumJobs j = {};
    j.rows = p.B * p.segs;
    j.job[0] = {p.a_part, a.dA, (long long)p.C * p.N, (long long)p.C * p.N};
    j.job[1] = {p.v_part, a.dD, p.C, 2LL * p.C};
    j.job[2] = {p.v_part + p.C, a.dbias, p.C, 2LL * p.C};
    ttt_scan_sum_kernel<<<dim3((unsigned)(((long long)p.C * p.N + 31) / 32), 3), 256, 0, a.stream>>>(j);
    return cudaGetLastError() == cudaSuccess ? n + 3 : -4;
}

template <typename T> int launch_type(Params &p, const ScanArgs &a, bool vec)
{
    switch (lanes(p.N)) {
    case 2: return vec ? launch_all<T, 2, true>(p, a) : launch_all<T, 2, false>(p, a);
    case 4: return vec ? launch_all<T, 4, true>(p, a) : launch_all<T, 4, false>(p, a);
    case 8: return vec ? launch_all<T, 8, true>(p, a) : launch_all<T, 8, false>(p, a);
    default: return vec ? launch_all<T, 16, true>(p, a) : launch_all<T, 16, false>(p, a);
    }
}

}  // namespace

size_t scan_bwd_workspace(int B, int T, int C, int N, int G) { return space(B, T, C, N, G).bytes; }

int launch_scan_bwd(const ScanArgs &a)
{
    Params p = {};
    params(a, p);
    const ScanPieces s = pieces(a.B, a.T, a.C, a.N, a.G);
    p.segs = s.segs;
    p.seg_len = s.len;
    p.blocks = (p.cpg + block_channels(lanes(a.N)) - 1) / block_channels(lanes(a.N));
    p.start = a.dh_last;
    p.dx = a.dx;
    p.ddelta = a.ddelta;
    p.dz = a.dz;
    p.dh0 = a.dh0;
    const Space w = space(a.B, a.T, a.C, a.N, a.G);
    float *ws = static_cast<float *>(a.ws);
    p.bc_part = ws + w.bc;
    p.a_part = ws + w.a;
    p.v_part = ws + w.v;
    p.H = ws + w.H;
    p.rate_sum = ws + w.rate;
    p.cut = reinterpret_cast<int *>(ws + w.cut);
    const bool vec = wide(a);
    return a.bf16 ? launch_type<__nv_bfloat16>(p, a, vec) : launch_type<float>(p, a, vec);
}

}  // namespace ttt
