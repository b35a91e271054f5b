// ttt_api.cu -- the C ABI declared in include/ttt.h: argument validation, TMA
// descriptor encoding, kernel dispatch and the per-device status word.
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/ttt.h"
#include "ttt_internal.h"
#include "ttt_vec.cuh"

// Status words (one pair per device: every device that loads the library has its own
// copy): [0] written by kernels whose bounded on-chip wait ran out, [1] by ttt_rope for
// a position outside its table.  Neither hides the other.
__device__ int g_ttt_status[2];

// Fixed scratch of ttt_linear_fwd_seqpar_noalloc (affine maps and segment start
// weights of a split run).  Every device that loads the library holds it until the
// process exits.  Every byte a call reads from it is written earlier by the same
// call, so it never needs clearing.
constexpr size_t kNoAllocScratchBytes = 4u << 20;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

namespace {

std::atomic<unsigned long long> g_launches{0};
std::atomic<unsigned long long> g_test_stall_ns{0};  // ttt_debug_wait_limit

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn()
{
    static std::once_flag once;
    static EncodeTiledFn fn = nullptr;
    std::call_once(once, [] {
        void *ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(ptr);
    });
    // The driver call wants this thread to have a context: a host thread whose first CUDA
    // work is a call of this library gets its device's here.
    static thread_local int ready = -1;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
    if (dev != ready) {
        if (cudaSetDevice(dev) != cudaSuccess) return nullptr;
        ready = dev;
    }
    return fn;
}

// Address of this device's status words (looked up once per device).
int *status_word()
{
    static std::mutex mu;
    static int *addr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_ttt_status) != cudaSuccess) return nullptr;
        addr[dev] = static_cast<int *>(p);
    }
    return addr[dev];
}

// Device address of this device's fixed scratch array.  The array's name in host
// code only stands for the symbol: the address comes from cudaGetSymbolAddress,
// looked up once per device with that device current (nullptr on failure).
void *noalloc_scratch()
{
    static std::mutex mu;
    static void *addr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void *p = nullptr;
        if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess) return nullptr;
        addr[dev] = p;
    }
    return addr[dev];
}

}  // namespace

bool ttt::allow_shared(const void *kernel, int bytes)
{
    // what is known of each kernel and device, by open addressing; past its size the
    // limit is set anew each time, to the same value
    static std::mutex mu;
    static struct {
        const void *kernel;
        int dev, most;
    } memo[1024];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return false;
    std::lock_guard<std::mutex> lock(mu);
    unsigned at = (unsigned)((reinterpret_cast<uintptr_t>(kernel) >> 4) * 31 + dev) % 1024;
    int probes = 0;
    for (; probes < 1024 && memo[at].kernel; ++probes, at = (at + 1) % 1024)
        if (memo[at].kernel == kernel && memo[at].dev == dev) return bytes <= memo[at].most;
    int most = 0;
    cudaFuncAttributes attr;
    if (cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev) != cudaSuccess ||
        cudaFuncGetAttributes(&attr, kernel) != cudaSuccess)
        return false;
    most -= (int)attr.sharedSizeBytes;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess) return false;
    if (probes < 1024) memo[at] = {kernel, dev, most};
    return bytes <= most;
}

// q/k/v viewed as a 3-D tensor [B*H][T][d] of bf16; box = `rows` tokens x min(d,64)
// features, swizzled to the box row length so that ldmatrix is conflict-free.
bool ttt::encode_token_map(CUtensorMap *m, const void *ptr, int BH, int T, int d, int rows, int cols)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    if (cols <= 0) cols = d < 64 ? d : 64;
    const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)T, (cuuint64_t)BH};
    const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)T * d * 2};
    const cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)rows, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    // swizzle span = the box row length (128, 64 or 32 bytes)
    const CUtensorMapSwizzle sw = cols >= 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : cols == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                               : CU_TENSOR_MAP_SWIZZLE_32B;
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(ptr), dims, strides, box,
              estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ttt::encode_rows_map(CUtensorMap *m, const void *ptr, bool bf16, int width, int rows, int batch, long long row_stride,
                          long long batch_stride, int cols, int height)
{
    EncodeTiledFn fn = encode_fn();
    const long long es = bf16 ? 2 : 4, rs = row_stride * es, bs = batch_stride * es;
    if (!fn || rs <= 0 || bs <= 0 || rs % 16 || bs % 16 || rs >= (1LL << 40) || bs >= (1LL << 40)) return false;
    if (reinterpret_cast<uintptr_t>(ptr) % 16) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)rows, (cuuint64_t)batch};
    const cuuint64_t strides[2] = {(cuuint64_t)rs, (cuuint64_t)bs};
    const cuuint32_t box[3] = {(cuuint32_t)cols, (cuuint32_t)height, 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, const_cast<void *>(ptr),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool ttt::encode_grid_map(CUtensorMap *m, const void *ptr, bool bf16, int BH, int hh, int ww, int d)
{
    EncodeTiledFn fn = encode_fn();
    if (!fn || d > 256 || ww + 2 > 256 || hh + 2 > 256) return false;
    const cuuint64_t es = bf16 ? 2 : 4;
    const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)ww, (cuuint64_t)hh, (cuuint64_t)BH};
    const cuuint64_t strides[3] = {(cuuint64_t)d * es, (cuuint64_t)ww * d * es, (cuuint64_t)hh * ww * d * es};
    const cuuint32_t box[4] = {(cuuint32_t)d, (cuuint32_t)ww + 2, (cuuint32_t)hh + 2, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void *>(ptr),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool overlaps(const void *a, size_t na, const void *b, size_t nb)
{
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

ttt_status code(int rc) { return static_cast<ttt_status>(rc); }

}  // namespace

namespace {

// Validates a TTT-Linear call and fills the launch arguments (status TTT_OK or the
// error to return).
ttt_status linear_args(const ttt_linear_desc *desc, const void *q, const void *k, const void *v,
                       const float *eta, float eta_scalar, const float *W0, void *z, float *W_out,
                       void *stream, ttt::LinearArgs &a)
{
    if (!desc) return TTT_ERR_ARG;
    const ttt_linear_desc D = *desc;
    if (D.B < 1 || D.H < 1 || D.T < 0 || D.mini_batch < 1 || !W0) return TTT_ERR_ARG;
    if (D.causal != 0 && D.causal != 1) return TTT_ERR_ARG;
    if (D.io_dtype != TTT_F32 && D.io_dtype != TTT_BF16) return TTT_ERR_ARG;
    if (D.T > 0 && (!q || !k || !v || !z)) return TTT_ERR_ARG;
    if (D.d != 16 && D.d != 32 && D.d != 64 && D.d != 128) return TTT_ERR_UNSUPPORTED;
    if (D.loss != TTT_LOSS_MSE && D.loss != TTT_LOSS_DOT) return TTT_ERR_ARG;
    if (D.epochs < 0) return TTT_ERR_ARG;
    if (D.epochs > 1 && (D.causal || D.mini_batch < D.T)) return TTT_ERR_UNSUPPORTED;
    const bool ln = D.ln_gamma || D.ln_beta;
    if (ln && (!D.ln_gamma || !D.ln_beta || !(D.ln_eps > 0.f) || D.loss != TTT_LOSS_MSE)) return TTT_ERR_ARG;
    if (ln && (!aligned(D.ln_gamma, 4) || !aligned(D.ln_beta, 4))) return TTT_ERR_ALIGN;
    if (ln && D.epochs > 1) return TTT_ERR_UNSUPPORTED;
    const long long dd = (long long)D.d * D.d;
    if (D.w0_batch_stride != 0 && D.w0_batch_stride != (long long)D.H * dd) return TTT_ERR_ARG;
    if ((long long)D.B * D.H > 0x7fffffffLL) return TTT_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(z, 16)) return TTT_ERR_ALIGN;
    if (!aligned(W0, 4) || !aligned(eta, 4) || !aligned(W_out, 4)) return TTT_ERR_ALIGN;
    if (W_out && D.w0_batch_stride == 0 &&
        overlaps(W_out, sizeof(float) * dd * D.B * D.H, W0, sizeof(float) * dd * D.H))
        return TTT_ERR_ARG;

    a.B = D.B;
    a.H = D.H;
    a.T = D.T;
    a.d = D.d;
    a.b = D.T > 0 && D.mini_batch > D.T ? D.T : D.mini_batch;  // b >= T is one block
    a.causal = D.causal;
    a.loss = D.loss;
    a.epochs = D.epochs > 1 ? D.epochs : 1;
    a.ln_gamma = ln ? D.ln_gamma : nullptr;
    a.ln_beta = ln ? D.ln_beta : nullptr;
    a.ln_eps = D.ln_eps;
    a.q = q;
    a.k = k;
    a.v = v;
    a.eta = eta;
    a.eta_scalar = eta_scalar;
    a.W0 = W0;
    a.w0_bstride = D.w0_batch_stride;
    a.z = z;
    a.W_out = W_out;
    a.status = status_word();
    a.stream = static_cast<cudaStream_t>(stream);
    a.test_stall_ns = g_test_stall_ns.load(std::memory_order_relaxed);
    if (!a.status) return TTT_ERR_LAUNCH;
    return TTT_OK;
}

int launch_linear(const ttt::LinearArgs &a, ttt_dtype io)
{
    int rc;
    if (io == TTT_BF16 && a.ln_gamma) {  // inner norm: the b = 16 kernel only (one mini-batch of
                                         // T <= 16 tokens is one of its chunks)
        const bool b16 = a.b == 16 || (a.b == a.T && a.T < 16);
        rc = (b16 && a.d <= 64) ? ttt::launch_linear_b16(a) : TTT_ERR_UNSUPPORTED;
    } else if (io == TTT_BF16) {
        rc = ttt::launch_linear_fb_tc(a);  // full-batch mini-batch: no serial chain
        if (rc == TTT_ERR_UNSUPPORTED) rc = ttt::launch_linear_fb(a);  // several epochs
        if (rc == TTT_ERR_UNSUPPORTED && a.epochs == 1)  // repeated epochs: the full-batch kernel only
            rc = (a.b == 1 && a.d <= 64 && !a.loss) ? ttt::launch_linear_b16(a)  // delta rule in 16-token chunks
                 : a.b == 1                          ? ttt::launch_linear_b1(a)   // column-parallel
                 : (a.b == 16 && a.d <= 64)          ? ttt::launch_linear_b16(a)
                                                     : ttt::launch_linear_bf16(a);
    } else
        rc = ttt::launch_linear_f32(a);
    return rc;
}

// The split plan of a validated bf16 call (nsplit 0: not split).
ttt::SeqparPlan seqpar_plan_for(const ttt_linear_desc *desc, const ttt::LinearArgs &a)
{
    ttt::SeqparPlan pl;
    if (desc->io_dtype != TTT_BF16 || !ttt::seqpar_plan(a, pl)) pl = ttt::SeqparPlan{};
    return pl;
}

}  // namespace

extern "C" {

ttt_status ttt_linear_fwd(const ttt_linear_desc *desc, const void *q, const void *k, const void *v,
                          const float *eta, float eta_scalar, const float *W0, void *z,
                          float *W_out, void *stream)
{
    ttt::LinearArgs a;
    const ttt_status st = linear_args(desc, q, k, v, eta, eta_scalar, W0, z, W_out, stream, a);
    if (st != TTT_OK) return st;
    const int rc = launch_linear(a, desc->io_dtype);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

size_t ttt_linear_seqpar_workspace(const ttt_linear_desc *desc)
{
    if (!desc || desc->B < 1 || desc->H < 1 || desc->T < 1 || desc->mini_batch < 1) return 0;
    ttt::LinearArgs a{};
    a.B = desc->B;
    a.H = desc->H;
    a.T = desc->T;
    a.d = desc->d;
    a.b = desc->mini_batch > desc->T ? desc->T : desc->mini_batch;
    a.loss = desc->loss;
    a.epochs = desc->epochs > 1 ? desc->epochs : 1;
    a.ln_gamma = desc->ln_gamma;
    return ttt::seqpar_workspace_bytes(seqpar_plan_for(desc, a));
}

ttt_status ttt_linear_fwd_seqpar(const ttt_linear_desc *desc, const void *q, const void *k, const void *v,
                                 const float *eta, float eta_scalar, const float *W0, void *z,
                                 float *W_out, void *workspace, size_t workspace_bytes, void *stream)
{
    ttt::LinearArgs a;
    const ttt_status st = linear_args(desc, q, k, v, eta, eta_scalar, W0, z, W_out, stream, a);
    if (st != TTT_OK) return st;
    const ttt::SeqparPlan pl = seqpar_plan_for(desc, a);
    int rc, n = 1;
    if (pl.nsplit < 2) {
        rc = launch_linear(a, desc->io_dtype);
    } else {
        const size_t need = ttt::seqpar_workspace_bytes(pl);
        if (!workspace || workspace_bytes < need || !aligned(workspace, 256)) return TTT_ERR_ARG;
        // the first segment reads W0 while the last one writes W_out on another stream
        const size_t dd = sizeof(float) * desc->d * desc->d;
        const size_t nW0 = desc->w0_batch_stride ? dd * desc->B * desc->H : dd * desc->H;
        if (W_out && overlaps(W_out, dd * desc->B * desc->H, W0, nW0)) return TTT_ERR_ARG;
        if (overlaps(workspace, need, z, (size_t)desc->B * desc->H * desc->T * desc->d * 2)) return TTT_ERR_ARG;
        rc = ttt::launch_linear_seqpar(a, pl, workspace);
        n = pl.nsplit > 2 ? 4 : 3;  // segment 0, chain (+ maps), scan, later segments
    }
    if (rc == 0) g_launches.fetch_add(n, std::memory_order_relaxed);
    return code(rc);
}

ttt_status ttt_mlp_fwd(const ttt_mlp_desc *desc, const void *q, const void *k, const void *v,
                       const float *eta, float eta_scalar, const float *W1, const float *c1,
                       const float *W2, const float *c2, void *z, float *W1_out, float *c1_out,
                       float *W2_out, float *c2_out, void *stream)
{
    if (!desc) return TTT_ERR_ARG;
    const ttt_mlp_desc D = *desc;
    if (D.B < 1 || D.H < 1 || D.T < 0 || D.mini_batch < 1 || D.m < 1) return TTT_ERR_ARG;
    if (!W1 || !c1 || !W2 || !c2) return TTT_ERR_ARG;
    if (D.causal != 0 && D.causal != 1) return TTT_ERR_ARG;
    if (D.params_per_batch != 0 && D.params_per_batch != 1) return TTT_ERR_ARG;
    if (D.activation != TTT_ACT_SILU && D.activation != TTT_ACT_GELU) return TTT_ERR_ARG;
    if (D.io_dtype != TTT_F32 && D.io_dtype != TTT_BF16) return TTT_ERR_ARG;
    if (D.T > 0 && (!q || !k || !v || !z)) return TTT_ERR_ARG;
    const bool ln = D.ln_gamma || D.ln_beta;
    if (ln && (!D.ln_gamma || !D.ln_beta || !(D.ln_eps > 0.f))) return TTT_ERR_ARG;
    if (D.d != 16 && D.d != 32 && D.d != 64) return TTT_ERR_UNSUPPORTED;
    if (D.m % 16 != 0) return TTT_ERR_UNSUPPORTED;
    if (ln && D.io_dtype == TTT_BF16 &&  // the bf16 inner norm: d = 64, m = 256, mini-batches of at
        (D.d != 64 || D.m != 256 ||      // most 16 tokens or one non-causal full batch
         ((D.T > 0 && D.mini_batch > D.T ? D.T : D.mini_batch) > 16 && (D.causal || D.mini_batch < D.T))))
        return TTT_ERR_UNSUPPORTED;
    if (ln && (!aligned(D.ln_gamma, 4) || !aligned(D.ln_beta, 4))) return TTT_ERR_ALIGN;
    if ((long long)D.B * D.H > 0x7fffffffLL) return TTT_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(z, 16)) return TTT_ERR_ALIGN;
    const void *f32p[] = {eta, W1, c1, W2, c2, W1_out, c1_out, W2_out, c2_out};
    for (const void *p : f32p)
        if (!aligned(p, 4)) return TTT_ERR_ALIGN;
    if (!D.params_per_batch) {
        const size_t nH = (size_t)D.H, nBH = (size_t)D.B * D.H, dm = (size_t)D.d * D.m;
        const struct { const void *o; size_t no; const void *i; size_t ni; } pairs[] = {
            {W1_out, nBH * dm, W1, nH * dm}, {c1_out, nBH * D.m, c1, nH * D.m},
            {W2_out, nBH * dm, W2, nH * dm}, {c2_out, nBH * D.d, c2, nH * D.d}};
        for (const auto &pr : pairs)
            if (pr.o && overlaps(pr.o, 4 * pr.no, pr.i, 4 * pr.ni)) return TTT_ERR_ARG;
    }

    ttt::MlpArgs a;
    a.test_stall_ns = g_test_stall_ns.load(std::memory_order_relaxed);
    a.B = D.B;
    a.H = D.H;
    a.T = D.T;
    a.d = D.d;
    a.m = D.m;
    a.b = D.T > 0 && D.mini_batch > D.T ? D.T : D.mini_batch;
    a.causal = D.causal;
    a.per_batch = D.params_per_batch;
    a.act = D.activation;
    a.ln_gamma = ln ? D.ln_gamma : nullptr;
    a.ln_beta = ln ? D.ln_beta : nullptr;
    a.ln_eps = D.ln_eps;
    a.q = q;
    a.k = k;
    a.v = v;
    a.eta = eta;
    a.eta_scalar = eta_scalar;
    a.W1 = W1;
    a.c1 = c1;
    a.W2 = W2;
    a.c2 = c2;
    a.z = z;
    a.W1o = W1_out;
    a.c1o = c1_out;
    a.W2o = W2_out;
    a.c2o = c2_out;
    a.status = status_word();
    a.stream = static_cast<cudaStream_t>(stream);
    if (!a.status) return TTT_ERR_LAUNCH;

    int rc;
    if (D.io_dtype == TTT_BF16)
        rc = ttt::launch_mlp_bf16(a);
    else
        rc = ttt::launch_mlp_f32(a);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

ttt_status ttt_linear_fwd_seqpar_noalloc(const ttt_linear_desc *desc, const void *q, const void *k,
                                         const void *v, const float *eta, float eta_scalar, const float *W0,
                                         void *z, float *W_out, void *stream)
{
    ttt::LinearArgs a;
    const ttt_status st = linear_args(desc, q, k, v, eta, eta_scalar, W0, z, W_out, stream, a);
    if (st != TTT_OK) return st;
    ttt::SeqparPlan pl;
    if (desc->io_dtype != TTT_BF16 || !ttt::seqpar_plan_serial(a, pl)) {
        const int rc = launch_linear(a, desc->io_dtype);  // not split: needs no scratch
        if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
        return code(rc);
    }
    if (ttt::seqpar_workspace_bytes(pl) > kNoAllocScratchBytes) return TTT_ERR_SCRATCH;
    const size_t dd = sizeof(float) * desc->d * desc->d;
    const size_t nW0 = desc->w0_batch_stride ? dd * desc->B * desc->H : dd * desc->H;
    if (W_out && overlaps(W_out, dd * desc->B * desc->H, W0, nW0)) return TTT_ERR_ARG;
    void *ws = noalloc_scratch();
    if (!ws) return TTT_ERR_LAUNCH;
    const int rc = ttt::launch_linear_seqpar_serial(a, pl, ws);
    if (rc == 0) g_launches.fetch_add(pl.nsplit > 2 ? 3 : 2, std::memory_order_relaxed);
    return code(rc);
}

ttt_status ttt_dwconv_fwd(const ttt_dwconv_desc *desc, const void *q, const void *k, const void *v,
                          const float *eta, float eta_scalar, const float *W0, void *z, float *W_out,
                          void *stream)
{
    if (!desc) return TTT_ERR_ARG;
    const ttt_dwconv_desc D = *desc;
    if (D.B < 1 || D.H < 1 || D.height < 0 || D.width < 0 || D.d < 1 || D.epochs < 1 || !W0)
        return TTT_ERR_ARG;
    if (D.io_dtype != TTT_F32 && D.io_dtype != TTT_BF16) return TTT_ERR_ARG;
    if (D.loss != TTT_LOSS_MSE && D.loss != TTT_LOSS_DOT) return TTT_ERR_ARG;
    const long long N = (long long)D.height * D.width;
    if (N > 0 && (!q || !k || !v || !z)) return TTT_ERR_ARG;
    if (D.w0_batch_stride != 0 && D.w0_batch_stride != (long long)D.H * 9 * D.d) return TTT_ERR_ARG;
    if (D.d % 8 != 0 || D.d > 512 || (long long)D.B * D.H > 0x7fffffffLL || N > (1 << 20))
        return TTT_ERR_UNSUPPORTED;
    if (ttt::dwconv_smem(D.height, D.width, D.d, D.io_dtype == TTT_BF16 ? 2 : 4) > 227 * 1024)
        return TTT_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(z, 16)) return TTT_ERR_ALIGN;
    if (!aligned(W0, 4) || !aligned(eta, 4) || !aligned(W_out, 4)) return TTT_ERR_ALIGN;
    ttt::DwconvArgs a;
    a.B = D.B;
    a.H = D.H;
    a.hh = D.height;
    a.ww = D.width;
    a.d = D.d;
    a.loss = D.loss;
    a.epochs = D.epochs;
    a.bf16 = D.io_dtype == TTT_BF16;
    a.q = q;
    a.k = k;
    a.v = v;
    a.eta = eta;
    a.eta_scalar = eta_scalar;
    a.W0 = W0;
    a.w0_bstride = D.w0_batch_stride;
    a.z = z;
    a.W_out = W_out;
    a.status = status_word();
    a.stream = static_cast<cudaStream_t>(stream);
    if (!a.status) return TTT_ERR_LAUNCH;
    const int rc = ttt::launch_dwconv(a);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

ttt_status ttt_eta_gate(const ttt_gate_desc *desc, const void *x, const void *theta, float eta_base,
                        float *eta, void *stream)
{
    if (!desc) return TTT_ERR_ARG;
    const ttt_gate_desc D = *desc;
    if (D.B < 0 || D.T < 0 || D.H < 1 || D.dm < 1) return TTT_ERR_ARG;
    if (D.B == 0 || D.T == 0) return TTT_OK;
    if (!x || !theta || !eta) return TTT_ERR_ARG;
    if (D.H > 64 || D.dm % 8 != 0 || D.B > 65535) return TTT_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(theta, 16) || !aligned(eta, 4)) return TTT_ERR_ALIGN;
    const size_t nx = (size_t)D.B * D.T * D.dm * 2, nth = (size_t)D.H * D.dm * 2, ne = (size_t)D.B * D.H * D.T * 4;
    if (overlaps(eta, ne, x, nx) || overlaps(eta, ne, theta, nth)) return TTT_ERR_ARG;
    ttt::GateArgs a;
    a.B = D.B;
    a.T = D.T;
    a.H = D.H;
    a.dm = D.dm;
    a.x = x;
    a.theta = theta;
    a.eta_base = eta_base;
    a.eta = eta;
    a.status = status_word();
    a.stream = static_cast<cudaStream_t>(stream);
    if (!a.status) return TTT_ERR_LAUNCH;
    const int rc = ttt::launch_eta_gate(a);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

namespace {

// Elements from the first to one past the last of a [B,H,T,d] view with these strides.
long long span(const long long st[3], int B, int H, int T, int d)
{
    return st[0] * (B - 1) + st[1] * (H - 1) + st[2] * (T - 1) + d;
}

// A [n0,n1,n2,d] view by rising stride, without its dimensions of one entry.
struct Nest {
    int dims;
    long long stride[3], extent[3];  // extent[i]: elements from first to one past the last, dimensions 0 .. i
    int n[3];
    long long inner(int i) const { return i > 0 ? extent[i - 1] : d; }
    long long d;
    bool nested;  // every dimension steps over all of those inside it: no element twice
};

Nest nest(const long long st[3], const int n[3], int d)
{
    Nest v = {};
    v.d = d;
    v.nested = true;
    for (int i = 0; i < 3; ++i) {
        if (n[i] <= 1) continue;
        int j = v.dims++;
        for (; j > 0 && v.stride[j - 1] > st[i]; --j) {
            v.stride[j] = v.stride[j - 1];
            v.n[j] = v.n[j - 1];
        }
        v.stride[j] = st[i];
        v.n[j] = n[i];
    }
    for (int i = 0; i < v.dims; ++i) {
        v.nested = v.nested && v.stride[i] >= v.inner(i);
        v.extent[i] = v.stride[i] * (v.n[i] - 1) + v.inner(i);
    }
    return v;
}

// Do two nested views with equal strides, the second `off` elements behind the first, share
// an element?  With off = q s + r along the outermost stride s, block k of the first meets
// at most blocks k - q (r further on) and k - q - 1 (s - r before) of the second.
bool share(const Nest &a, const Nest &b, int dims, long long off)
{
    if (dims == 0) return off > -a.d && off < a.d;
    const int i = dims - 1;
    const long long s = a.stride[i], q = off >= 0 ? off / s : -((-off + s - 1) / s), r = off - q * s;
    for (int up = 0; up < 2; ++up) {
        const long long m = -(q + up);  // block 0 of the first meets block m of the second
        if (m < b.n[i] && m > -(long long)a.n[i] && share(a, b, i, r - up * s)) return true;
    }
    return false;
}

// A [B,H,T,d] view: its first element and strides.
struct HeadView {
    const void *p;
    long long st[3];
    int n[3];
};

// Do two views share memory, or may they?  Told apart exactly where their strides agree
// and their dimensions nest (slices of one buffer); else by their ends.
bool shares_memory(const HeadView &a, const HeadView &b, int d, int es)
{
    if (!overlaps(a.p, es * span(a.st, a.n[0], a.n[1], a.n[2], d), b.p, es * span(b.st, b.n[0], b.n[1], b.n[2], d))) return false;
    const long long bytes = (long long)(reinterpret_cast<uintptr_t>(b.p) - reinterpret_cast<uintptr_t>(a.p));
    if (bytes % es) return true;
    long long sa[3], sb[3];
    int na[3], nb[3], n[3];
    for (int i = 0; i < 3; ++i) {
        // a dimension of one entry takes the other's stride
        sa[i] = a.n[i] > 1 ? a.st[i] : b.st[i];
        sb[i] = b.n[i] > 1 ? b.st[i] : a.st[i];
        if (sa[i] != sb[i]) return true;
        n[i] = a.n[i] > b.n[i] ? a.n[i] : b.n[i];
        na[i] = a.n[i];
        nb[i] = b.n[i];
    }
    Nest x = nest(sa, n, d), y = x;  // one order of dimensions for both
    if (!x.nested) return true;
    // x and y have the larger count of each dimension; put their own back
    for (int j = 0; j < x.dims; ++j)
        for (int i = 0; i < 3; ++i)
            if (n[i] > 1 && sa[i] == x.stride[j]) {
                x.n[j] = na[i];
                y.n[j] = nb[i];
            }
    return share(x, y, x.dims, bytes / es);
}

// The same elements in the same order.
bool same_view(const HeadView &a, const HeadView &b)
{
    for (int i = 0; i < 3; ++i)
        if (a.n[i] != b.n[i] || (a.n[i] > 1 && a.st[i] != b.st[i])) return false;
    return a.p == b.p;
}

}  // namespace

namespace {

// ttt_rope, or with `axes` ttt_rope_axes.
ttt_status rope(const ttt_rope_desc &D, const ttt_rope_axes_desc *axes, const unsigned char *pair_axis, const void *q,
                const void *k, const void *v, const float *table, const long long *positions, void *q_out, void *k_out,
                void *v_out, void *stream)
{
    if (D.B < 0 || D.T < 0 || D.Hq < 1 || D.Hk < 0 || D.d < 1 || D.rot < 0 || D.rot > D.d || D.rot % 2) return TTT_ERR_ARG;
    if (D.interleaved < 0 || D.interleaved > 1 || D.inverse < 0 || D.inverse > 1) return TTT_ERR_ARG;
    if (D.io_dtype != TTT_F32 && D.io_dtype != TTT_BF16) return TTT_ERR_ARG;
    if (D.table_rows < 0 || D.period < 0 || D.period > D.table_rows || D.pos0 < 0 || D.pos0 > (1LL << 62) || D.positions_batch_stride < 0)
        return TTT_ERR_ARG;
    if (D.d > 1024 || (long long)D.B * D.T > 0x7fffffffLL || D.Hq + 2LL * D.Hk > 0x7fff0000LL) return TTT_ERR_UNSUPPORTED;
    if (D.B == 0 || D.T == 0) return TTT_OK;
    if (!q || !q_out || (k && !k_out) || (v && !v_out) || ((k || v) && D.Hk < 1)) return TTT_ERR_ARG;
    if (D.rot > 0 && !table) return TTT_ERR_ARG;
    if (D.rot > 0 && !positions && !axes && D.period == 0 && D.pos0 > (long long)D.table_rows - D.T) return TTT_ERR_ARG;
    if (axes && D.rot > 0) {
        if (D.period != 0 || !pair_axis) return TTT_ERR_ARG;
        for (int i = 0; i < D.rot / 2; ++i)
            if (pair_axis[i] >= axes->axes) return TTT_ERR_ARG;
        if (positions) {
            if (axes->positions_axis_stride < 0) return TTT_ERR_ARG;
        } else {
            long long tokens = 1;
            for (int i = 0; i < axes->axes; ++i) {
                if (axes->grid[i] < 1 || axes->grid[i] > D.table_rows) return TTT_ERR_ARG;
                tokens *= axes->grid[i];
                if (tokens > 0x7fffffffLL) return TTT_ERR_ARG;
            }
            if (D.pos0 > tokens - D.T) return TTT_ERR_ARG;
        }
    }
    const int es = D.io_dtype == TTT_BF16 ? 2 : 4;
    ttt::RopeArgs a = {};
    const void *in[3] = {q, k, v};
    void *out[3] = {q_out, k_out, v_out};
    const long long *is[3] = {D.q_stride, D.k_stride, D.v_stride};
    const long long *os[3] = {D.q_out_stride, D.k_out_stride, D.v_out_stride};
    const int H[3] = {D.Hq, D.Hk, D.Hk}, dim[3] = {D.B, 0, D.T};
    for (int i = 0; i < 3; ++i) {
        if (!in[i]) continue;
        if (!aligned(in[i], es) || !aligned(out[i], es)) return TTT_ERR_ALIGN;
        for (int j = 0; j < 3; ++j) {
            const int n = j == 1 ? H[i] : dim[j];
            if (is[i][j] < 0 || os[i][j] < 0 || (n > 1 && os[i][j] == 0)) return TTT_ERR_ARG;
            // a dimension of one entry is never stepped over: its stride says nothing
            a.in_stride[i][j] = n > 1 ? is[i][j] : 0;
            a.out_stride[i][j] = n > 1 ? os[i][j] : 0;
        }
    }
    if (D.rot > 0 && (!aligned(table, 8) || (positions && !aligned(positions, 8)))) return TTT_ERR_ALIGN;
    const size_t table_bytes = (size_t)D.table_rows * D.rot * 4,
                 pos_bytes = positions ? 8 * (size_t)((axes ? axes->positions_axis_stride * (axes->axes - 1) : 0) + D.positions_batch_stride * (D.B - 1) + D.T) : 0;
    HeadView vi[3], vo[3];
    for (int i = 0; i < 3; ++i) {
        if (!in[i]) continue;
        vi[i] = {in[i], {a.in_stride[i][0], a.in_stride[i][1], a.in_stride[i][2]}, {D.B, H[i], D.T}};
        vo[i] = {out[i], {a.out_stride[i][0], a.out_stride[i][1], a.out_stride[i][2]}, {D.B, H[i], D.T}};
        if (!nest(vo[i].st, vo[i].n, D.d).nested) return TTT_ERR_ARG;
        const size_t bytes = es * span(vo[i].st, D.B, H[i], D.T, D.d);
        if (D.rot > 0 && (overlaps(out[i], bytes, table, table_bytes) || (positions && overlaps(out[i], bytes, positions, pos_bytes))))
            return TTT_ERR_ARG;
    }
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j) {
            if (!in[i] || !in[j]) continue;
            if (!(i == j && same_view(vi[i], vo[i])) && shares_memory(vi[i], vo[j], D.d, es)) return TTT_ERR_ARG;
            if (i < j && shares_memory(vo[i], vo[j], D.d, es)) return TTT_ERR_ARG;
        }
    a.B = D.B;
    a.T = D.T;
    a.Hq = D.Hq;
    a.Hk = D.Hk;
    a.d = D.d;
    a.rot = D.rot;
    a.interleaved = D.interleaved;
    a.inverse = D.inverse;
    a.bf16 = D.io_dtype == TTT_BF16;
    a.table_rows = D.table_rows;
    a.period = D.period;
    a.pos0 = D.pos0;
    a.pos_bstride = D.positions_batch_stride;
    a.q = q;
    a.k = k;
    a.v = v;
    a.q_out = q_out;
    a.k_out = k_out;
    a.v_out = v_out;
    a.table = table;
    a.positions = positions;
    int *const status = status_word();
    if (!status) return TTT_ERR_LAUNCH;
    a.range_status = status + 1;
    a.stream = static_cast<cudaStream_t>(stream);
    if (axes) {
        a.axes = axes->axes;
        a.axis_stride = axes->axes > 1 ? axes->positions_axis_stride : 0;
        for (int i = 0; i < axes->axes; ++i) a.grid[i] = axes->grid[i];
        a.pair_axis = pair_axis;
    }
    const int rc = ttt::launch_rope(a);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

}  // namespace

ttt_status ttt_rope(const ttt_rope_desc *desc, const void *q, const void *k, const void *v, const float *table,
                    const long long *positions, void *q_out, void *k_out, void *v_out, void *stream)
{
    if (!desc) return TTT_ERR_ARG;
    return rope(*desc, nullptr, nullptr, q, k, v, table, positions, q_out, k_out, v_out, stream);
}

ttt_status ttt_rope_axes(const ttt_rope_axes_desc *desc, const unsigned char *pair_axis, const void *q, const void *k,
                         const void *v, const float *table, const long long *positions, void *q_out, void *k_out,
                         void *v_out, void *stream)
{
    if (!desc || desc->axes < 1 || desc->axes > TTT_ROPE_MAX_AXES) return TTT_ERR_ARG;
    return rope(desc->rope, desc, pair_axis, q, k, v, table, positions, q_out, k_out, v_out, stream);
}

namespace {

bool norm_desc_ok(const ttt_block_norm_desc &D)
{
    if (D.B < 0 || D.T < 0 || D.D < 1 || D.heads < 1 || D.D % D.heads) return false;
    if (D.io_dtype != TTT_F32 && D.io_dtype != TTT_BF16) return false;
    if (D.post < 0 || D.post > 2 || D.pre < 0 || D.pre > 2 || D.act < 0 || D.act > 3) return false;
    return (!D.post || D.post_eps >= 0.f) && (!D.pre || D.pre_eps >= 0.f);
}

constexpr int kNormMaxD = 8192;

// Checks the part both directions share and fills the launch arguments; TTT_OK with
// *empty set when there are no tokens.
ttt_status norm_args(const ttt_block_norm_desc *desc, const ttt_block_norm_params *params, const void *y, const void *x,
                     const void *gate, void *stream, ttt::BlockNormArgs &a, bool *empty)
{
    if (!desc || !params) return TTT_ERR_ARG;
    const ttt_block_norm_desc &D = *desc;
    const ttt_block_norm_params &P = *params;
    if (!norm_desc_ok(D)) return TTT_ERR_ARG;
    if ((P.post_bias && D.post != TTT_NORM_LAYER) || (P.post_weight && !D.post) ||
        (P.pre_bias && D.pre != TTT_NORM_LAYER) || (P.pre_weight && !D.pre))
        return TTT_ERR_ARG;
    if (D.D > kNormMaxD || (long long)D.B * D.T > 0x7fffffffLL) return TTT_ERR_UNSUPPORTED;
    for (const float *v : {P.post_weight, P.post_bias, P.scale, P.pre_weight, P.pre_bias})
        if (v && !aligned(v, 4)) return TTT_ERR_ALIGN;
    *empty = D.B == 0 || D.T == 0;
    const int es = D.io_dtype == TTT_BF16 ? 2 : 4;
    if (!*empty) {
        if (!y || (D.act != TTT_GATE_NONE) != (gate != nullptr)) return TTT_ERR_ARG;
        if (!aligned(y, es) || (x && !aligned(x, es)) || (gate && !aligned(gate, es))) return TTT_ERR_ALIGN;
    }
    for (int i = 0; i < 3; ++i)
        if (D.y_stride[i] < 0) return TTT_ERR_ARG;
    for (int i = 0; i < 2; ++i)
        if (D.x_stride[i] < 0 || D.gate_stride[i] < 0 || D.dh_stride[i] < 0 || D.du_stride[i] < 0) return TTT_ERR_ARG;
    a = {};
    a.B = D.B;
    a.T = D.T;
    a.D = D.D;
    a.dh = D.D / D.heads;
    a.bf16 = D.io_dtype == TTT_BF16;
    a.post = D.post;
    a.pre = D.pre;
    a.act = D.act;
    a.eps1 = D.post_eps;
    a.eps2 = D.pre_eps;
    a.alpha = D.alpha;
    a.y = y;
    a.x = x;
    a.gate = gate;
    // strides of dimensions with one entry, or of absent tensors, say nothing
    const int n[2] = {D.B, D.T};
    for (int i = 0; i < 3; ++i) a.ys[i] = (i == 1 ? D.heads : n[i / 2]) > 1 ? D.y_stride[i] : 0;
    if (D.heads == 1) a.ys[1] = 0;
    for (int i = 0; i < 2; ++i) {
        a.xs[i] = x && n[i] > 1 ? D.x_stride[i] : 0;
        a.gs[i] = gate && n[i] > 1 ? D.gate_stride[i] : 0;
        a.dhs[i] = n[i] > 1 ? D.dh_stride[i] : 0;
        a.dus[i] = n[i] > 1 ? D.du_stride[i] : 0;
    }
    a.w1 = P.post_weight;
    a.b1 = P.post_bias;
    a.scale = P.scale;
    a.w2 = P.pre_weight;
    a.b2 = P.pre_bias;
    a.stream = static_cast<cudaStream_t>(stream);
    return TTT_OK;
}

size_t rows_span(const long long st[2], int B, int T, int D, int es)
{
    return es * (st[0] * (B - 1) + st[1] * (T - 1) + D);
}

struct Range {
    const void *p;
    size_t n;
};

// Does any output overlap any input?
bool clash(const Range *out, int no, const Range *in, int ni)
{
    for (int i = 0; i < no; ++i)
        for (int j = 0; j < ni; ++j)
            if (out[i].p && in[j].p && overlaps(out[i].p, out[i].n, in[j].p, in[j].n)) return true;
    return false;
}

}  // namespace

ttt_status ttt_block_norm_fwd(const ttt_block_norm_desc *desc, const ttt_block_norm_params *params, const void *y,
                              const void *x, const void *gate, void *h, void *u, float *stats, void *stream)
{
    ttt::BlockNormArgs a;
    bool empty;
    const ttt_status st = norm_args(desc, params, y, x, gate, stream, a, &empty);
    if (st != TTT_OK || empty) return st;
    if (!h || (a.pre != 0) != (u != nullptr)) return TTT_ERR_ARG;
    const int es = a.bf16 ? 2 : 4;
    if (!aligned(h, es) || (u && !aligned(u, es)) || (stats && !aligned(stats, 16))) return TTT_ERR_ALIGN;
    const size_t nt = (size_t)a.B * a.T, n = nt * a.D * es, nd = (size_t)a.D * 4;
    // h may be x itself: a thread reads its features of a row before it writes them
    const bool in_place = x == h && (a.T == 1 || a.xs[1] == a.D) && (a.B == 1 || a.xs[0] == (long long)a.T * a.D);
    const long long ys[3] = {a.ys[0], a.ys[1], a.ys[2]};
    const Range in[] = {{y, es * (size_t)span(ys, a.B, desc->heads, a.T, a.dh)},
                        {gate, rows_span(a.gs, a.B, a.T, a.D, es)},
                        {a.w1, nd}, {a.b1, nd}, {a.scale, nd}, {a.w2, nd}, {a.b2, nd},
                        {in_place ? nullptr : x, rows_span(a.xs, a.B, a.T, a.D, es)}};
    const Range out[] = {{h, n}, {u, n}, {stats, nt * 16}}, xr = {x, rows_span(a.xs, a.B, a.T, a.D, es)};
    if (clash(out, 3, in, 8) || clash(out + 1, 2, &xr, 1) || clash(out, 1, out + 1, 2) || clash(out + 1, 1, out + 2, 1))
        return TTT_ERR_ARG;
    a.h = h;
    a.u = u;
    a.stats = stats;
    const int rc = ttt::launch_block_norm_fwd(a);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

size_t ttt_block_norm_bwd_workspace(const ttt_block_norm_desc *desc)
{
    if (!desc || !norm_desc_ok(*desc) || desc->D > kNormMaxD) return 0;
    const long long rows = (long long)desc->B * desc->T;
    return (size_t)ttt::block_norm_bwd_blocks(desc->D, rows) * 5 * desc->D * 4;
}

ttt_status ttt_block_norm_bwd(const ttt_block_norm_desc *desc, const ttt_block_norm_params *params, const void *dh,
                              const void *du, const void *y, const void *x, const void *gate, const float *stats,
                              void *dy, void *dx, void *dgate, const ttt_block_norm_grads *grads, void *workspace,
                              size_t workspace_bytes, void *stream)
{
    ttt::BlockNormArgs a;
    bool empty;
    const ttt_status st = norm_args(desc, params, y, x, gate, stream, a, &empty);
    if (st != TTT_OK) return st;
    const int es = a.bf16 ? 2 : 4;
    const size_t nt = (size_t)a.B * a.T, n = nt * a.D * es, nd = (size_t)a.D * 4;
    int nvec = 0;
    if (grads) {
        float *const g[5] = {grads->post_weight, grads->post_bias, grads->scale, grads->pre_weight, grads->pre_bias};
        // gradients exist for what takes part: a norm's weight and (layer norm) bias, the scale
        const bool there[5] = {a.post != 0, a.post == 2, true, a.pre != 0, a.pre == 2};
        for (int i = 0; i < 5; ++i) {
            if (g[i] && !there[i]) return TTT_ERR_ARG;
            if (g[i] && !aligned(g[i], 4)) return TTT_ERR_ALIGN;
            a.dvec[i] = g[i];
            nvec += g[i] != nullptr;
        }
        if (g[2] && !a.scale) return TTT_ERR_ARG;
    }
    if (!empty) {
        if (!dy || !stats || (a.pre != 0) != (du != nullptr) || (!dh && !du)) return TTT_ERR_ARG;
        if ((gate != nullptr) != (dgate != nullptr) || (dx && !x)) return TTT_ERR_ARG;
        if (!aligned(stats, 16)) return TTT_ERR_ALIGN;
        for (const void *q : {dh, du, (const void *)dy, (const void *)dx, (const void *)dgate})
            if (q && !aligned(q, es)) return TTT_ERR_ALIGN;
        const size_t need = nvec ? ttt_block_norm_bwd_workspace(desc) : 0;
        if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_ARG;
        if (need && !aligned(workspace, 16)) return TTT_ERR_ALIGN;
        if (!dh) a.dhs[0] = a.dhs[1] = 0;
        if (!du) a.dus[0] = a.dus[1] = 0;
        const long long ys[3] = {a.ys[0], a.ys[1], a.ys[2]};
        const Range in[] = {{y, es * (size_t)span(ys, a.B, desc->heads, a.T, a.dh)},
                            {gate, rows_span(a.gs, a.B, a.T, a.D, es)},
                            {x, rows_span(a.xs, a.B, a.T, a.D, es)},
                            {dh, rows_span(a.dhs, a.B, a.T, a.D, es)},
                            {du, rows_span(a.dus, a.B, a.T, a.D, es)},
                            {stats, nt * 16}, {a.w1, nd}, {a.b1, nd}, {a.scale, nd}, {a.w2, nd}, {a.b2, nd}};
        const Range out[] = {{dy, n}, {dx, n}, {dgate, n}, {need ? workspace : nullptr, need},
                             {a.dvec[0], nd}, {a.dvec[1], nd}, {a.dvec[2], nd}, {a.dvec[3], nd}, {a.dvec[4], nd}};
        if (clash(out, 9, in, 11)) return TTT_ERR_ARG;
        for (int i = 0; i < 9; ++i)
            if (clash(out + i, 1, out + i + 1, 8 - i)) return TTT_ERR_ARG;
    }
    a.dh_in = dh;
    a.du = du;
    a.stats = const_cast<float *>(stats);
    a.dy = dy;
    a.dx = dx;
    a.dgate = dgate;
    a.ws = workspace;
    if (empty && !nvec) return TTT_OK;
    const int rc = ttt::launch_block_norm_bwd(a);
    if (rc == 0) g_launches.fetch_add((empty ? 0 : 1) + (nvec ? 1 : 0), std::memory_order_relaxed);
    return code(rc);
}

namespace {

static_assert(ttt::kRecurChunk == TTT_RECURRENCE_CHUNK && ttt::kRecurMix == TTT_RECUR_MIX, "");

ttt_status recurrence_args(const ttt_recurrence_desc *desc, const void *x, const void *f, const unsigned char *reset,
                           void *stream, ttt::RecurArgs &a)
{
    if (!desc) return TTT_ERR_ARG;
    const ttt_recurrence_desc &D = *desc;
    if (D.B < 0 || D.T < 0 || D.C < 1 || D.mode < 0 || D.mode > 2) return TTT_ERR_ARG;
    if (D.io_dtype != TTT_F32 && D.io_dtype != TTT_BF16) return TTT_ERR_ARG;
    for (int i = 0; i < 2; ++i)
        if (D.x_stride[i] < 0 || D.f_stride[i] < 0 || D.dh_stride[i] < 0) return TTT_ERR_ARG;
    if (D.B > 65535 || D.T > 0x7fff0000) return TTT_ERR_UNSUPPORTED;
    const int es = D.io_dtype == TTT_BF16 ? 2 : 4;
    if (D.B > 0 && D.T > 0) {
        if (!x || !f) return TTT_ERR_ARG;
        if (!aligned(x, es) || !aligned(f, es)) return TTT_ERR_ALIGN;
    }
    a = {};
    a.B = D.B;
    a.T = D.T;
    a.C = D.C;
    a.bf16 = D.io_dtype == TTT_BF16;
    a.mode = D.mode;
    a.x = x;
    a.f = f;
    a.reset = reset;
    const int n[2] = {D.B, D.T};
    for (int i = 0; i < 2; ++i) {
        a.xs[i] = n[i] > 1 ? D.x_stride[i] : 0;
        a.fs[i] = n[i] > 1 ? D.f_stride[i] : 0;
        a.ds[i] = n[i] > 1 ? D.dh_stride[i] : 0;
    }
    a.stream = static_cast<cudaStream_t>(stream);
    return TTT_OK;
}

// The first or last state of a call without tokens: dst = src or zeros.
ttt_status copy_states(float *dst, const float *src, size_t n, cudaStream_t st)
{
    if (!dst || dst == src || n == 0) return TTT_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, n * 4, cudaMemcpyDeviceToDevice, st)
                              : cudaMemsetAsync(dst, 0, n * 4, st);
    return e == cudaSuccess ? TTT_OK : TTT_ERR_LAUNCH;
}

}  // namespace

ttt_status ttt_recurrence_fwd(const ttt_recurrence_desc *desc, const void *x, const void *f,
                              const unsigned char *reset, const float *h0, void *h, float *h_last, float *states,
                              void *stream)
{
    ttt::RecurArgs a;
    const ttt_status st = recurrence_args(desc, x, f, reset, stream, a);
    if (st != TTT_OK) return st;
    if ((h0 && !aligned(h0, 4)) || (h_last && !aligned(h_last, 4)) || (states && !aligned(states, 4))) return TTT_ERR_ALIGN;
    const size_t nbc = (size_t)a.B * a.C;
    if (h0 != h_last && h0 && h_last && overlaps(h0, nbc * 4, h_last, nbc * 4)) return TTT_ERR_ARG;
    if (a.B == 0 || a.T == 0) return copy_states(h_last, h0, nbc, a.stream);
    const int es = a.bf16 ? 2 : 4;
    if (!h) return TTT_ERR_ARG;
    if (!aligned(h, es)) return TTT_ERR_ALIGN;
    const size_t n = nbc * a.T * es, ns = nbc * ((a.T + ttt::kRecurChunk - 1) / ttt::kRecurChunk) * 4;
    const Range in[] = {{x, rows_span(a.xs, a.B, a.T, a.C, es)}, {f, rows_span(a.fs, a.B, a.T, a.C, es)},
                        {reset, (size_t)a.B * a.T}, {h0 == h_last ? nullptr : h0, nbc * 4}};
    const Range out[] = {{h, n}, {h_last, nbc * 4}, {states, ns}}, start = {h0, nbc * 4};
    if (clash(out, 3, in, 4) || clash(out, 1, out + 1, 2) || clash(out + 1, 1, out + 2, 1) || clash(out, 1, &start, 1) ||
        clash(out + 2, 1, &start, 1))
        return TTT_ERR_ARG;
    a.h0 = h0;
    a.h = h;
    a.h_last = h_last;
    a.states = states;
    a.status = status_word();
    if (!a.status) return TTT_ERR_LAUNCH;
    a.test_stall_ns = g_test_stall_ns.load(std::memory_order_relaxed);
    const int rc = ttt::launch_recurrence(a, false);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

ttt_status ttt_recurrence_bwd(const ttt_recurrence_desc *desc, const void *dh, const void *x, const void *f,
                              const unsigned char *reset, const float *states, const float *dh_last, void *dx,
                              void *df, float *dh0, void *stream)
{
    ttt::RecurArgs a;
    const ttt_status st = recurrence_args(desc, x, f, reset, stream, a);
    if (st != TTT_OK) return st;
    if ((dh_last && !aligned(dh_last, 4)) || (dh0 && !aligned(dh0, 4)) || (states && !aligned(states, 4)))
        return TTT_ERR_ALIGN;
    const size_t nbc = (size_t)a.B * a.C;
    if (dh0 && dh_last && overlaps(dh0, nbc * 4, dh_last, nbc * 4)) return TTT_ERR_ARG;
    if (a.B == 0 || a.T == 0) return copy_states(dh0, dh_last, nbc, a.stream);
    const int es = a.bf16 ? 2 : 4;
    if (!dx || !df || !states) return TTT_ERR_ARG;
    if (!aligned(dx, es) || !aligned(df, es) || (dh && !aligned(dh, es))) return TTT_ERR_ALIGN;
    if (!dh) a.ds[0] = a.ds[1] = 0;
    const size_t n = nbc * a.T * es, ns = nbc * ((a.T + ttt::kRecurChunk - 1) / ttt::kRecurChunk) * 4;
    const Range in[] = {{x, rows_span(a.xs, a.B, a.T, a.C, es)}, {f, rows_span(a.fs, a.B, a.T, a.C, es)},
                        {dh, rows_span(a.ds, a.B, a.T, a.C, es)}, {reset, (size_t)a.B * a.T},
                        {states, ns}, {dh_last, nbc * 4}};
    const Range out[] = {{dx, n}, {df, n}, {dh0, nbc * 4}};
    if (clash(out, 3, in, 6) || clash(out, 1, out + 1, 2) || clash(out + 1, 1, out + 2, 1)) return TTT_ERR_ARG;
    a.dh = dh;
    a.dh_last = dh_last;
    a.states = const_cast<float *>(states);
    a.dx = dx;
    a.df = df;
    a.dh0 = dh0;
    a.status = status_word();
    if (!a.status) return TTT_ERR_LAUNCH;
    a.test_stall_ns = g_test_stall_ns.load(std::memory_order_relaxed);
    const int rc = ttt::launch_recurrence(a, true);
    if (rc == 0) g_launches.fetch_add(1, std::memory_order_relaxed);
    return code(rc);
}

namespace {

bool conv_desc_ok(const ttt_short_conv_desc &D)
{
    if (D.B < 0 || D.T < 0 || D.C < 1 || D.width < 1 || D.act < 0 || D.act > 1) return false;
    return D.io_dtype == TTT_F32 || D.io_dtype == TTT_BF16;
}
bool conv_desc_fits(const ttt_short_conv_desc &D)
{
    return D.width <= ttt::kConvMaxWidth && (long long)D.B * D.T <= 0x7fffffffLL && D.T <= 1 << 30 && D.C <= 1 << 30;
}

// Checks the part both directions share and fills the launch arguments.
ttt_status conv_args(const ttt_short_conv_desc *desc, const void *x, const float *weight, const float *bias,
                     const unsigned char *reset, const void *state, void *stream, ttt::ConvArgs &a)
{
    if (!desc || !conv_desc_ok(*desc)) return TTT_ERR_ARG;
    const ttt_short_conv_desc &D = *desc;
    if (D.x_stride[0] < 0 || D.x_stride[1] < 0) return TTT_ERR_ARG;
    if (!conv_desc_fits(D)) return TTT_ERR_UNSUPPORTED;
    const int es = D.io_dtype == TTT_BF16 ? 2 : 4;
    if (!weight) return TTT_ERR_ARG;
    if (!aligned(weight, 4) || (bias && !aligned(bias, 4)) || (state && !aligned(state, es))) return TTT_ERR_ALIGN;
    if (D.B > 0 && D.T > 0) {
        if (!x) return TTT_ERR_ARG;
        if (!aligned(x, es)) return TTT_ERR_ALIGN;
    }
    a = {};
    a.B = D.B;
    a.T = D.T;
    a.C = D.C;
    a.K = D.width;
    a.bf16 = D.io_dtype == TTT_BF16;
    a.silu = D.act == TTT_CONV_SILU;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.reset = reset;
    a.state = D.width > 1 ? state : nullptr;
    const int n[2] = {D.B, D.T};
    for (int i = 0; i < 2; ++i) a.xs[i] = n[i] > 1 ? D.x_stride[i] : 0;
    a.stream = static_cast<cudaStream_t>(stream);
    return TTT_OK;
}

// Does any output overlap an input or another output?
bool any_clash(const Range *out, int no, const Range *in, int ni)
{
    if (clash(out, no, in, ni)) return true;
    for (int i = 0; i + 1 < no; ++i)
        if (clash(out + i, 1, out + i + 1, no - 1 - i)) return true;
    return false;
}

ttt_status copy_bytes(void *dst, const void *src, size_t n, cudaStream_t st)
{
    if (!dst || dst == src || n == 0) return TTT_OK;
    const cudaError_t e = src ? cudaMemcpyAsync(dst, src, n, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(dst, 0, n, st);
    return e == cudaSuccess ? TTT_OK : TTT_ERR_LAUNCH;
}

}  // namespace

ttt_status ttt_short_conv_fwd(const ttt_short_conv_desc *desc, const void *x, const float *weight, const float *bias,
                              const unsigned char *reset, const void *state, void *y, void *state_out, void *stream)
{
    ttt::ConvArgs a;
    const ttt_status st = conv_args(desc, x, weight, bias, reset, state, stream, a);
    if (st != TTT_OK) return st;
    const int es = a.bf16 ? 2 : 4;
    if (a.K == 1) state_out = nullptr;
    if (state_out && !aligned(state_out, es)) return TTT_ERR_ALIGN;
    const size_t ns = (size_t)a.B * (a.K - 1) * a.C * es, n = (size_t)a.B * a.T * a.C * es;
    if (state_out && a.state && state_out != a.state && overlaps(a.state, ns, state_out, ns)) return TTT_ERR_ARG;
    if (a.B == 0 || a.T == 0) return copy_bytes(state_out, a.state, ns, a.stream);
    if (!y) return TTT_ERR_ARG;
    if (!aligned(y, es)) return TTT_ERR_ALIGN;
    const Range in[] = {{x, rows_span(a.xs, a.B, a.T, a.C, es)}, {weight, (size_t)a.C * a.K * 4}, {bias, (size_t)a.C * 4},
                        {reset, (size_t)a.B * a.T}, {state_out == a.state ? nullptr : a.state, ns}};
    const Range out[] = {{y, n}, {state_out, ns}}, start = {a.state, ns};
    if (any_clash(out, 2, in, 5) || clash(out, 1, &start, 1)) return TTT_ERR_ARG;
    a.y = y;
    a.state_out = state_out;
    const int rc = ttt::launch_conv_fwd(a);
    if (rc > 0) g_launches.fetch_add(rc, std::memory_order_relaxed);
    return rc < 0 ? code(rc) : TTT_OK;
}

size_t ttt_short_conv_bwd_workspace(const ttt_short_conv_desc *desc)
{
    if (!desc || !conv_desc_ok(*desc) || !conv_desc_fits(*desc) || desc->B == 0 || desc->T == 0) return 0;
    return ttt::conv_bwd_workspace(desc->B, desc->T, desc->C, desc->width);
}

ttt_status ttt_short_conv_bwd(const ttt_short_conv_desc *desc, const void *dy, const void *x, const float *weight,
                              const float *bias, const unsigned char *reset, const void *state,
                              const float *dstate_out, void *dx, float *dweight, float *dbias, float *dstate,
                              void *workspace, size_t workspace_bytes, void *stream)
{
    ttt::ConvArgs a;
    ttt_status st = conv_args(desc, x, weight, bias, reset, state, stream, a);
    if (st != TTT_OK) return st;
    const int es = a.bf16 ? 2 : 4;
    if (desc->dy_stride[0] < 0 || desc->dy_stride[1] < 0) return TTT_ERR_ARG;
    a.dys[0] = a.B > 1 ? desc->dy_stride[0] : 0;
    a.dys[1] = a.T > 1 ? desc->dy_stride[1] : 0;
    for (const float *q : {dstate_out, (const float *)dweight, (const float *)dbias, (const float *)dstate})
        if (q && !aligned(q, 4)) return TTT_ERR_ALIGN;
    if (a.K == 1) {
        dstate = nullptr;
        dstate_out = nullptr;
    }
    const size_t nr = (size_t)a.B * (a.K - 1) * a.C, n = (size_t)a.B * a.T * a.C * es;
    const size_t need = dweight || dbias ? ttt_short_conv_bwd_workspace(desc) : 0;
    if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_ARG;
    if (need && !aligned(workspace, 16)) return TTT_ERR_ALIGN;
    const bool empty = a.B == 0 || a.T == 0;
    if (!empty) {
        if (!dy || !dx) return TTT_ERR_ARG;
        if (!aligned(dy, es) || !aligned(dx, es)) return TTT_ERR_ALIGN;
    }
    const Range in[] = {{x, empty ? 0 : rows_span(a.xs, a.B, a.T, a.C, es)}, {dy, empty ? 0 : rows_span(a.dys, a.B, a.T, a.C, es)},
                        {weight, (size_t)a.C * a.K * 4}, {bias, (size_t)a.C * 4}, {reset, (size_t)a.B * a.T},
                        {a.state, nr * es}, {dstate_out, nr * 4}};
    const Range out[] = {{empty ? nullptr : dx, n}, {dweight, (size_t)a.C * a.K * 4}, {dbias, (size_t)a.C * 4}, {dstate, nr * 4},
                         {need ? workspace : nullptr, need}};
    if (any_clash(out, 5, in, 7)) return TTT_ERR_ARG;
    if (empty) {
        // no token: the states pass through, the parameters have no gradient
        if ((st = copy_bytes(dstate, dstate_out, nr * 4, a.stream)) != TTT_OK) return st;
        if ((st = copy_bytes(dweight, nullptr, (size_t)a.C * a.K * 4, a.stream)) != TTT_OK) return st;
        return copy_bytes(dbias, nullptr, (size_t)a.C * 4, a.stream);
    }
    a.dy = dy;
    a.dstate_out = dstate_out;
    a.dx = dx;
    a.dweight = dweight;
    a.dbias = dbias;
    a.dstate = dstate;
    a.ws = workspace;
    const int rc = ttt::launch_conv_bwd(a);
    if (rc > 0) g_launches.fetch_add(rc, std::memory_order_relaxed);
    return rc < 0 ? code(rc) : TTT_OK;
}

namespace {

static_assert(ttt::kScanChunk == TTT_SCAN_CHUNK, "");

bool scan_desc_ok(const ttt_scan_desc &D)
{
    if (D.B < 0 || D.T < 0 || D.C < 1 || D.N < 1 || D.G < 1 || D.C % D.G || D.softplus < 0 || D.softplus > 1) return false;
    return D.io_dtype == TTT_F32 || D.io_dtype == TTT_BF16;
}
bool scan_desc_fits(const ttt_scan_desc &D)
{
    return D.N <= ttt::kScanMaxN && D.B <= 65535 && D.T <= 1 << 30 && (long long)D.C * D.N <= 0x7fff0000LL &&
           (long long)D.B * D.T <= 0x7fff0000LL / D.G;
}
size_t scan_bc_span(const long long st[3], int B, int T, int G, int N, int es)
{
    return es * (size_t)(st[0] * (B - 1) + st[1] * (T - 1) + st[2] * (G - 1) + N);
}

// Checks the part both directions share and fills the launch arguments.
ttt_status scan_args(const ttt_scan_desc *desc, const ttt_scan_params *params, const void *x, const void *delta,
                     const void *Bm, const void *Cm, const void *z, const unsigned char *reset, void *stream, ttt::ScanArgs &a)
{
    if (!desc || !params || !scan_desc_ok(*desc)) return TTT_ERR_ARG;
    const ttt_scan_desc &D = *desc;
    for (int i = 0; i < 2; ++i)
        if (D.x_stride[i] < 0 || D.delta_stride[i] < 0 || D.z_stride[i] < 0) return TTT_ERR_ARG;
    for (int i = 0; i < 3; ++i)
        if (D.b_stride[i] < 0 || D.c_stride[i] < 0) return TTT_ERR_ARG;
    if (!scan_desc_fits(D)) return TTT_ERR_UNSUPPORTED;
    if (!params->A) return TTT_ERR_ARG;
    for (const float *q : {params->A, params->D, params->delta_bias})
        if (q && !aligned(q, 4)) return TTT_ERR_ALIGN;
    const int es = D.io_dtype == TTT_BF16 ? 2 : 4;
    if (D.B > 0 && D.T > 0)
        for (const void *q : {x, delta, Bm, Cm}) {
            if (!q) return TTT_ERR_ARG;
            if (!aligned(q, es)) return TTT_ERR_ALIGN;
        }
    if (z && !aligned(z, es)) return TTT_ERR_ALIGN;
    a = {};
    a.B = D.B;
    a.T = D.T;
    a.C = D.C;
    a.N = D.N;
    a.G = D.G;
    a.bf16 = D.io_dtype == TTT_BF16;
    a.softplus = D.softplus;
    a.x = x;
    a.delta = delta;
    a.z = z;
    a.Bm = Bm;
    a.Cm = Cm;
    a.A = params->A;
    a.D = params->D;
    a.bias = params->delta_bias;
    a.reset = reset;
    const int n[3] = {D.B, D.T, D.G};
    for (int i = 0; i < 2; ++i) {
        a.xs[i] = n[i] > 1 ? D.x_stride[i] : 0;
        a.ds[i] = n[i] > 1 ? D.delta_stride[i] : 0;
        a.zs[i] = z && n[i] > 1 ? D.z_stride[i] : 0;
    }
    for (int i = 0; i < 3; ++i) {
        a.bs[i] = n[i] > 1 ? D.b_stride[i] : 0;
        a.cs[i] = n[i] > 1 ? D.c_stride[i] : 0;
    }
    a.stream = static_cast<cudaStream_t>(stream);
    return TTT_OK;
}

// The nine inputs of a call with tokens, as memory ranges.
void scan_inputs(const ttt::ScanArgs &a, Range *in)
{
    const int es = a.bf16 ? 2 : 4;
    const size_t nv = (size_t)a.C * 4;
    in[0] = {a.x, rows_span(a.xs, a.B, a.T, a.C, es)};
    in[1] = {a.delta, rows_span(a.ds, a.B, a.T, a.C, es)};
    in[2] = {a.z, rows_span(a.zs, a.B, a.T, a.C, es)};
    in[3] = {a.Bm, scan_bc_span(a.bs, a.B, a.T, a.G, a.N, es)};
    in[4] = {a.Cm, scan_bc_span(a.cs, a.B, a.T, a.G, a.N, es)};
    in[5] = {a.reset, (size_t)a.B * a.T};
    in[6] = {a.A, nv * a.N};
    in[7] = {a.D, nv};
    in[8] = {a.bias, nv};
}

}  // namespace

size_t ttt_selective_scan_fwd_workspace(const ttt_scan_desc *desc)
{
    if (!desc || !scan_desc_ok(*desc) || !scan_desc_fits(*desc) || desc->B == 0 || desc->T == 0) return 0;
    return ttt::scan_fwd_workspace(desc->B, desc->T, desc->C, desc->N, desc->G);
}

ttt_status ttt_selective_scan_fwd(const ttt_scan_desc *desc, const ttt_scan_params *params, const void *x,
                                  const void *delta, const void *Bm, const void *Cm, const void *z,
                                  const unsigned char *reset, const float *h0, void *y, float *h_last, float *states,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    ttt::ScanArgs a;
    const ttt_status st = scan_args(desc, params, x, delta, Bm, Cm, z, reset, stream, a);
    if (st != TTT_OK) return st;
    for (const float *q : {h0, (const float *)h_last, (const float *)states})
        if (q && !aligned(q, 4)) return TTT_ERR_ALIGN;
    const size_t nh = (size_t)a.B * a.C * a.N * 4;
    if (h0 != h_last && h0 && h_last && overlaps(h0, nh, h_last, nh)) return TTT_ERR_ARG;
    if (a.B == 0 || a.T == 0) return copy_bytes(h_last, h0, nh, a.stream);
    const int es = a.bf16 ? 2 : 4;
    if (!y) return TTT_ERR_ARG;
    if (!aligned(y, es)) return TTT_ERR_ALIGN;
    const size_t need = ttt_selective_scan_fwd_workspace(desc);
    if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_ARG;
    if (need && !aligned(workspace, 16)) return TTT_ERR_ALIGN;
    Range in[10];
    scan_inputs(a, in);
    in[9] = {h0 == h_last ? nullptr : h0, nh};
    const size_t n = (size_t)a.B * a.T * a.C * es, ns = nh * ((a.T + ttt::kScanChunk - 1) / ttt::kScanChunk);
    const Range out[] = {{y, n}, {states, ns}, {need ? workspace : nullptr, need}, {h_last, nh}}, start = {h0, nh};
    if (any_clash(out, 4, in, 10) || clash(out, 3, &start, 1)) return TTT_ERR_ARG;
    a.h0 = h0;
    a.y = y;
    a.h_last = h_last;
    a.states = states;
    a.ws = workspace;
    const int rc = ttt::launch_scan_fwd(a);
    if (rc > 0) g_launches.fetch_add(rc, std::memory_order_relaxed);
    return rc < 0 ? code(rc) : TTT_OK;
}

size_t ttt_selective_scan_bwd_workspace(const ttt_scan_desc *desc)
{
    if (!desc || !scan_desc_ok(*desc) || !scan_desc_fits(*desc) || desc->B == 0 || desc->T == 0) return 0;
    return ttt::scan_bwd_workspace(desc->B, desc->T, desc->C, desc->N, desc->G);
}

ttt_status ttt_selective_scan_bwd(const ttt_scan_desc *desc, const ttt_scan_params *params, const void *dy,
                                  const void *x, const void *delta, const void *Bm, const void *Cm, const void *z,
                                  const unsigned char *reset, const float *states, const float *dh_last, void *dx,
                                  void *ddelta, void *dB, void *dC, void *dz, const ttt_scan_grads *grads, float *dh0,
                                  void *workspace, size_t workspace_bytes, void *stream)
{
    ttt::ScanArgs a;
    ttt_status st = scan_args(desc, params, x, delta, Bm, Cm, z, reset, stream, a);
    if (st != TTT_OK) return st;
    if (desc->dy_stride[0] < 0 || desc->dy_stride[1] < 0) return TTT_ERR_ARG;
    const ttt_scan_grads none = {}, &gr = grads ? *grads : none;
    for (const float *q : {states, dh_last, (const float *)dh0, (const float *)gr.A, (const float *)gr.D, (const float *)gr.delta_bias})
        if (q && !aligned(q, 4)) return TTT_ERR_ALIGN;
    if ((gr.D && !a.D) || (gr.delta_bias && !a.bias)) return TTT_ERR_ARG;
    const size_t nh = (size_t)a.B * a.C * a.N * 4, nv = (size_t)a.C * 4;
    const bool empty = a.B == 0 || a.T == 0;
    const int es = a.bf16 ? 2 : 4;
    const size_t need = ttt_selective_scan_bwd_workspace(desc);
    Range in[12] = {};
    if (!empty) {
        if (!dy || !states || !dx || !ddelta || !dB || !dC || (z != nullptr) != (dz != nullptr)) return TTT_ERR_ARG;
        for (const void *q : {dy, (const void *)dx, (const void *)ddelta, (const void *)dB, (const void *)dC, (const void *)dz})
            if (q && !aligned(q, es)) return TTT_ERR_ALIGN;
        if (!workspace || workspace_bytes < need) return TTT_ERR_ARG;
        if (!aligned(workspace, 16)) return TTT_ERR_ALIGN;
        a.dys[0] = a.B > 1 ? desc->dy_stride[0] : 0;
        a.dys[1] = a.T > 1 ? desc->dy_stride[1] : 0;
        scan_inputs(a, in);
        in[9] = {dy, rows_span(a.dys, a.B, a.T, a.C, es)};
        in[10] = {states, nh * ((a.T + ttt::kScanChunk - 1) / ttt::kScanChunk)};
    }
    in[11] = {dh_last, nh};
    const size_t n = empty ? 0 : (size_t)a.B * a.T * a.C * es, nbc = empty ? 0 : (size_t)a.B * a.T * a.G * a.N * es;
    const Range out[] = {{empty ? nullptr : dx, n}, {empty ? nullptr : ddelta, n}, {empty ? nullptr : dz, n},
                         {empty ? nullptr : dB, nbc}, {empty ? nullptr : dC, nbc}, {gr.A, nv * a.N}, {gr.D, nv},
                         {gr.delta_bias, nv}, {dh0, nh}, {empty ? nullptr : workspace, need}};
    if (any_clash(out, 10, in, 12)) return TTT_ERR_ARG;
    if (empty) {
        // no token: the states pass through, the parameters have no gradient
        if ((st = copy_bytes(dh0, dh_last, nh, a.stream)) != TTT_OK) return st;
        if ((st = copy_bytes(gr.A, nullptr, nv * a.N, a.stream)) != TTT_OK) return st;
        if ((st = copy_bytes(gr.D, nullptr, nv, a.stream)) != TTT_OK) return st;
        return copy_bytes(gr.delta_bias, nullptr, nv, a.stream);
    }
    a.dy = dy;
    a.states = const_cast<float *>(states);
    a.dh_last = dh_last;
    a.dx = dx;
    a.ddelta = ddelta;
    a.dB = dB;
    a.dC = dC;
    a.dz = dz;
    a.dA = gr.A;
    a.dD = gr.D;
    a.dbias = gr.delta_bias;
    a.dh0 = dh0;
    a.ws = workspace;
    const int rc = ttt::launch_scan_bwd(a);
    if (rc > 0) g_launches.fetch_add(rc, std::memory_order_relaxed);
    return rc < 0 ? code(rc) : TTT_OK;
}

ttt_status ttt_sync_status(void *stream)
{
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return TTT_ERR_LAUNCH;
    int v[2] = {0, 0};
    if (cudaMemcpyFromSymbol(v, g_ttt_status, sizeof(v)) != cudaSuccess) return TTT_ERR_LAUNCH;
    for (int i = 0; i < 2; ++i)
        if (v[i] != 0) {
            const int zero = 0;
            cudaMemcpyToSymbol(g_ttt_status, &zero, sizeof(int), i * sizeof(int));
            return i == 0 ? TTT_ERR_TIMEOUT : TTT_ERR_RANGE;
        }
    return TTT_OK;
}

const char *ttt_status_str(ttt_status s)
{
    switch (s) {
    case TTT_OK: return "ok";
    case TTT_ERR_ARG: return "invalid argument";
    case TTT_ERR_UNSUPPORTED: return "unsupported configuration";
    case TTT_ERR_ALIGN: return "pointer misaligned (q, k, v, z need 16 bytes; fp32 arrays 4)";
    case TTT_ERR_LAUNCH: return "CUDA error at launch";
    case TTT_ERR_TIMEOUT: return "kernel wait timed out";
    case TTT_ERR_SCRATCH: return "the split run needs more than the library's fixed 4 MiB scratch";
    case TTT_ERR_RANGE: return "a position lies outside the rotary table";
    }
    return "unknown status";
}

unsigned long long ttt_launch_count(void) { return g_launches.load(std::memory_order_relaxed); }

void ttt_debug_wait_limit(unsigned long long ns) { g_test_stall_ns.store(ns, std::memory_order_relaxed); }

}  // extern "C"
