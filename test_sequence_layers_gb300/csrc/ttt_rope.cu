// ttt_rope.cu -- rotary positions on q and k with the change of head layout (v is only
// moved):  out_a = a cos - b sin, out_b = a sin + b cos for every pair (a, b) of a head's
// first rot features, (cos, sin) read from a table by position.
//
// Bound by reading and writing every tensor once.  A thread owns V pairs of one token
// and walks over heads of q, then k, then v: the table entries and the position are
// fetched once per thread, and HB heads' loads are in flight together.  In the half
// layout a thread's two vectors are the features [uV, uV + V) and [rot/2 + uV, ...);
// interleaved, two neighbouring vectors.  Features past rot are units of two vectors
// that are copied.  Measured (cold L2, of the copy bandwidth): 2 x 32768 tokens of 3 x 32
// heads of 64 in bf16 251 us (0.95), 8 x 2048 of 3 x 12 heads 28 us (0.79: ramp-up and tail),
// heads of 20 (4- and 8-byte accesses) 0.55.
#include "ttt_internal.h"
#include "ttt_vec.cuh"

namespace ttt {
namespace {

constexpr int kRopeThreads = 256;
constexpr int kSMs = 152;

struct RopeTensor {
    const void *in;
    void *out;
    long long is[3], os[3];  // element strides: batch, head, token
    int heads;
};

struct RopeParams {
    RopeTensor t[3];  // q, k, v (heads 0: absent)
    int T, d, rot, units, tok_per_block, heads_per_thread, rows, period;
    long long ntok, pos0, pos_bstride;
    const long long *positions;
    const float *table;
    int *range_status;
};

// One token's unit of features (at e0 and, if two, e1), turned by cs and sn where rotate, in
// this block's share of the heads.
template <typename T, int V, bool INTER, bool INV>
__device__ __forceinline__ void turn_heads(const RopeParams &p, int b, int t, int e0, int e1, bool two, bool rotate,
                                           const float (&cs)[V], const float (&sn)[V])
{
    constexpr int HB = 4;  // heads whose loads are issued together
    // heads of q, k and v in one row: this block's share [first, last)
    int first = blockIdx.y * p.heads_per_thread, last = first + p.heads_per_thread;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        const RopeTensor &x = p.t[i];
        const int lo = max(first, 0), hi = min(last, x.heads);
        const T *in = static_cast<const T *>(x.in) + b * x.is[0] + t * x.is[2];
        T *out = static_cast<T *>(x.out) + b * x.os[0] + t * x.os[2];
        for (int h = lo; h < hi; h += HB) {
            Pack<T, V> p0[HB], p1[HB];
#pragma unroll
            for (int j = 0; j < HB; ++j)
                if (h + j < hi) {
                    const T *src = in + (h + j) * x.is[1];
                    p0[j].load_rw(src + e0);
                    if (two) p1[j].load_rw(src + e1);
                }
#pragma unroll
            for (int j = 0; j < HB; ++j)
                if (h + j < hi) {
                    if (i < 2 && rotate) {
                        float a[V], c[V], ya[V], yc[V];
                        unpack(p0[j], a);
                        unpack(p1[j], c);
#pragma unroll
                        for (int m = 0; m < V; ++m) {
                            // pair m of the unit: (a[m], c[m]), or neighbours in memory
                            const int i0 = 2 * m, i1 = 2 * m + 1;
                            const float u = INTER ? (i0 < V ? a[i0 % V] : c[i0 % V]) : a[m];
                            const float w = INTER ? (i1 < V ? a[i1 % V] : c[i1 % V]) : c[m];
                            const float s = INV ? -sn[m] : sn[m];
                            const float yu = u * cs[m] - w * s, yw = u * s + w * cs[m];
                            if (INTER) {
                                if (i0 < V) ya[i0 % V] = yu; else yc[i0 % V] = yu;
                                if (i1 < V) ya[i1 % V] = yw; else yc[i1 % V] = yw;
                            } else {
                                ya[m] = yu;
                                yc[m] = yw;
                            }
                        }
                        pack(p0[j], ya);
                        pack(p1[j], yc);
                    }
                    T *dst = out + (h + j) * x.os[1];
                    p0[j].store(dst + e0);
                    if (two) p1[j].store(dst + e1);
                }
        }
        first -= x.heads;
        last -= x.heads;
    }
}

template <typename T, int V, bool INTER, bool INV>
__global__ void __launch_bounds__(1024) ttt_rope_kernel(const __grid_constant__ RopeParams p)
{
    const int unit = threadIdx.x % p.units, slot = threadIdx.x / p.units;
    const long long tok = (long long)blockIdx.x * p.tok_per_block + slot;
    if (tok >= p.ntok) return;
    const int b = (int)(tok / p.T), t = (int)(tok % p.T);
    const int half = p.rot >> 1, rot_units = half / V;
    const bool rotate = unit < rot_units;
    int e0, e1;
    if (rotate) {
        e0 = INTER ? 2 * unit * V : unit * V;
        e1 = INTER ? e0 + V : half + unit * V;
    } else {
        e0 = p.rot + 2 * (unit - rot_units) * V;
        e1 = e0 + V;
    }
    const bool two = e1 < p.d;
    float cs[V], sn[V];
    if (rotate) {
        long long pos = p.positions ? p.positions[b * p.pos_bstride + t] : p.pos0 + t;
        const bool neg = pos < 0;
        if (p.period > 0 && !neg)
            pos = pos <= 0x7fffffffLL ? (long long)((unsigned)pos % (unsigned)p.period) : pos % p.period;
        if (neg || pos >= p.rows) {
            *p.range_status = 1;
#pragma unroll
            for (int j = 0; j < V; ++j) cs[j] = sn[j] = __int_as_float(0x7fffffff);
        } else {
            const float2 *row = reinterpret_cast<const float2 *>(p.table) + pos * half + unit * V;
            if constexpr (V % 2 == 0) {
#pragma unroll
                for (int j = 0; j < V; j += 2) {
                    const float4 w = __ldg(reinterpret_cast<const float4 *>(row + j));
                    cs[j] = w.x;
                    sn[j] = w.y;
                    cs[j + 1] = w.z;
                    sn[j + 1] = w.w;
                }
            } else {
                const float2 w = __ldg(row);
                cs[0] = w.x;
                sn[0] = w.y;
            }
        }
    }
    turn_heads<T, V, INTER, INV>(p, b, t, e0, e1, two, rotate, cs, sn);
}

// Several axes: pair i turns by the position of axis[i], whose column of the table has the
// pair's own frequency.  Positions are given per axis or are the token's coordinates on a
// row-major grid.  Measured (of the copy bandwidth): 256 pictures of 14 x 14 tokens, 3 x 6 heads
// of 64 in bf16 36.9 us (0.92); 4 videos of 16 x 28 x 28, 3 x 12 heads, axes in turn, inverse
// 77 us (0.88): as one axis.
constexpr int kRopeMaxAxes = 4;
struct RopeAxesParams {
    RopeParams r;
    int axes, uniform;  // uniform: a unit's V pairs are of one axis
    long long axis_stride;
    int grid[kRopeMaxAxes];
    unsigned char axis[512];
};

template <typename T, int V, bool INTER, bool INV>
__global__ void __launch_bounds__(1024) ttt_rope_axes_kernel(const __grid_constant__ RopeAxesParams q)
{
    const RopeParams &p = q.r;
    const int unit = threadIdx.x % p.units, slot = threadIdx.x / p.units;
    const long long tok = (long long)blockIdx.x * p.tok_per_block + slot;
    if (tok >= p.ntok) return;
    const int b = (int)(tok / p.T), t = (int)(tok % p.T);
    const int half = p.rot >> 1, rot_units = half / V;
    const bool rotate = unit < rot_units;
    int e0, e1;
    if (rotate) {
        e0 = INTER ? 2 * unit * V : unit * V;
        e1 = INTER ? e0 + V : half + unit * V;
    } else {
        e0 = p.rot + 2 * (unit - rot_units) * V;
        e1 = e0 + V;
    }
    float cs[V], sn[V];
    if (rotate) {
        long long pos[kRopeMaxAxes] = {};
        if (p.positions) {
#pragma unroll
            for (int a = 0; a < kRopeMaxAxes; ++a)
                if (a < q.axes) pos[a] = p.positions[a * q.axis_stride + b * p.pos_bstride + t];
        } else {
            // pos0 + t < 2^31: the grid was checked
            unsigned i = (unsigned)(p.pos0 + t);
#pragma unroll
            for (int a = kRopeMaxAxes - 1; a > 0; --a)
                if (a < q.axes) {
                    const unsigned n = q.grid[a];
                    pos[a] = i % n;
                    i /= n;
                }
            pos[0] = i;
        }
        auto of = [&](int a) { return a == 0 ? pos[0] : a == 1 ? pos[1] : a == 2 ? pos[2] : pos[3]; };
        const float2 *col = reinterpret_cast<const float2 *>(p.table) + unit * V;
        const float nan = __int_as_float(0x7fffffff);
        if (V % 2 == 0 && q.uniform) {
            const long long at = of(q.axis[unit * V]);
            const bool out = at < 0 || at >= p.rows;
            if (out) *p.range_status = 1;
#pragma unroll
            for (int j = 0; j + 1 < V; j += 2) {
                float4 w = make_float4(nan, nan, nan, nan);
                if (!out) w = __ldg(reinterpret_cast<const float4 *>(col + at * half + j));
                cs[j] = w.x;
                sn[j] = w.y;
                cs[j + 1] = w.z;
                sn[j + 1] = w.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const long long at = of(q.axis[unit * V + j]);
                float2 w = make_float2(nan, nan);
                if (at < 0 || at >= p.rows) *p.range_status = 1;
                else w = __ldg(col + at * half + j);
                cs[j] = w.x;
                sn[j] = w.y;
            }
        }
    }
    turn_heads<T, V, INTER, INV>(p, b, t, e0, e1, e1 < p.d, rotate, cs, sn);
}

template <typename T, int V>
int launch_rope_v(const RopeParams &p, const RopeArgs &a)
{
    const int heads = p.t[0].heads + p.t[1].heads + p.t[2].heads;
    const int blocks = (int)((p.ntok + p.tok_per_block - 1) / p.tok_per_block);
    const dim3 grid(blocks, (heads + p.heads_per_thread - 1) / p.heads_per_thread);
    const int threads = p.units * p.tok_per_block;
    if (a.axes) {
        RopeAxesParams q = {};
        q.r = p;
        q.axes = a.axes;
        q.axis_stride = a.axis_stride;
        q.uniform = 1;
        for (int i = 0; i < a.axes; ++i) q.grid[i] = a.grid[i];
        for (int i = 0; i < a.rot / 2; ++i) {
            q.axis[i] = a.pair_axis[i];
            if (q.axis[i] != a.pair_axis[i / V * V]) q.uniform = 0;
        }
        if (a.interleaved)
            if (a.inverse) ttt_rope_axes_kernel<T, V, true, true><<<grid, threads, 0, a.stream>>>(q);
            else ttt_rope_axes_kernel<T, V, true, false><<<grid, threads, 0, a.stream>>>(q);
        else if (a.inverse) ttt_rope_axes_kernel<T, V, false, true><<<grid, threads, 0, a.stream>>>(q);
        else ttt_rope_axes_kernel<T, V, false, false><<<grid, threads, 0, a.stream>>>(q);
        return cudaGetLastError() == cudaSuccess ? 0 : -4;
    }
    if (a.interleaved)
        if (a.inverse) ttt_rope_kernel<T, V, true, true><<<grid, threads, 0, a.stream>>>(p);
        else ttt_rope_kernel<T, V, true, false><<<grid, threads, 0, a.stream>>>(p);
    else if (a.inverse) ttt_rope_kernel<T, V, false, true><<<grid, threads, 0, a.stream>>>(p);
    else ttt_rope_kernel<T, V, false, false><<<grid, threads, 0, a.stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace

int launch_rope(const RopeArgs &a)
{
    const int es = a.bf16 ? 2 : 4;
    RopeParams p = {};
    const void *in[3] = {a.q, a.k, a.v};
    void *out[3] = {a.q_out, a.k_out, a.v_out};
    // the widest vector that divides every offset a unit starts at, every stride and
    // every pointer
    long long mask = (a.rot / 2) | (a.interleaved ? 0 : a.rot) | a.d;
    for (int i = 0; i < 3; ++i) {
        p.t[i].heads = in[i] ? (i == 0 ? a.Hq : a.Hk) : 0;
        if (!p.t[i].heads) continue;
        p.t[i].in = in[i];
        p.t[i].out = out[i];
        mask |= (long long)(reinterpret_cast<uintptr_t>(in[i]) / es) | (long long)(reinterpret_cast<uintptr_t>(out[i]) / es);
        for (int j = 0; j < 3; ++j) {
            p.t[i].is[j] = a.in_stride[i][j];
            p.t[i].os[j] = a.out_stride[i][j];
            mask |= a.in_stride[i][j] | a.out_stride[i][j];
        }
    }
    // the table is read two pairs (16 bytes) at a time when V > 1
    if (reinterpret_cast<uintptr_t>(a.table) % 16) mask |= 1;
    int V = 16 / es;
    while (mask & (V - 1)) V >>= 1;
    p.T = a.T;
    p.d = a.d;
    p.rot = a.rot;
    p.rows = a.table_rows;
    p.period = a.period;
    p.ntok = (long long)a.B * a.T;
    p.pos0 = a.pos0;
    p.pos_bstride = a.pos_bstride;
    p.positions = a.positions;
    p.table = a.table;
    p.range_status = a.range_status;
    p.units = a.rot / 2 / V + (a.d - a.rot + 2 * V - 1) / (2 * V);
    p.tok_per_block = p.units >= kRopeThreads ? 1 : kRopeThreads / p.units;
    if ((long long)p.tok_per_block > p.ntok) p.tok_per_block = (int)p.ntok;
    // heads per thread: all of them once the tokens alone fill the GPU (2048 threads an
    // SM); otherwise the heads are spread over more threads
    const int heads = p.t[0].heads + p.t[1].heads + p.t[2].heads;
    if (heads == 0) return 0;
    const long long fill = p.ntok * p.units * heads / (2048LL * kSMs);
    p.heads_per_thread = (int)(fill < 1 ? 1 : fill > heads ? heads : fill);
    // a grid has 65535 rows of blocks at most
    const int least = (heads + 65534) / 65535;
    if (p.heads_per_thread < least) p.heads_per_thread = least;
    if (a.bf16) {
        switch (V) {
        case 8: return launch_rope_v<__nv_bfloat16, 8>(p, a);
        case 4: return launch_rope_v<__nv_bfloat16, 4>(p, a);
        case 2: return launch_rope_v<__nv_bfloat16, 2>(p, a);
        default: return launch_rope_v<__nv_bfloat16, 1>(p, a);
        }
    }
    switch (V) {
    case 4: return launch_rope_v<float, 4>(p, a);
    case 2: return launch_rope_v<float, 2>(p, a);
    default: return launch_rope_v<float, 1>(p, a);
    }
}

}  // namespace ttt
