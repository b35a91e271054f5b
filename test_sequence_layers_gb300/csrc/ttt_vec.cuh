// ttt_vec.cuh -- moving V consecutive elements of a bf16 or fp32 tensor between global
// memory and fp32 registers in one access (V * sizeof(T) <= 16 bytes), for the kernels
// that stream token tensors.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace ttt {

template <int BYTES> struct RawOf;
template <> struct RawOf<2> { using type = unsigned short; };
template <> struct RawOf<4> { using type = unsigned int; };
template <> struct RawOf<8> { using type = uint2; };
template <> struct RawOf<16> { using type = uint4; };

// V elements of T as they lie in memory.
template <typename T, int V> struct Pack {
    using Raw = typename RawOf<V * (int)sizeof(T)>::type;
    Raw raw;
    __device__ __forceinline__ void load(const T *p) { raw = __ldg(reinterpret_cast<const Raw *>(p)); }
    // a plain load: for data the same kernel also writes (in-place operation)
    __device__ __forceinline__ void load_rw(const T *p) { raw = *reinterpret_cast<const Raw *>(p); }
    __device__ __forceinline__ void store(T *p) const { *reinterpret_cast<Raw *>(p) = raw; }
};

__device__ __forceinline__ void unpack(const Pack<float, 1> &p, float (&v)[1]) { v[0] = __uint_as_float(p.raw); }
__device__ __forceinline__ void unpack(const Pack<float, 2> &p, float (&v)[2])
{
    v[0] = __uint_as_float(p.raw.x);
    v[1] = __uint_as_float(p.raw.y);
}
__device__ __forceinline__ void unpack(const Pack<float, 4> &p, float (&v)[4])
{
    v[0] = __uint_as_float(p.raw.x);
    v[1] = __uint_as_float(p.raw.y);
    v[2] = __uint_as_float(p.raw.z);
    v[3] = __uint_as_float(p.raw.w);
}
__device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi)
{
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 1> &p, float (&v)[1])
{
    v[0] = __uint_as_float((uint32_t)p.raw << 16);
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 2> &p, float (&v)[2]) { unpack2(p.raw, v[0], v[1]); }
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 4> &p, float (&v)[4])
{
    unpack2(p.raw.x, v[0], v[1]);
    unpack2(p.raw.y, v[2], v[3]);
}
__device__ __forceinline__ void unpack(const Pack<__nv_bfloat16, 8> &p, float (&v)[8])
{
    unpack2(p.raw.x, v[0], v[1]);
    unpack2(p.raw.y, v[2], v[3]);
    unpack2(p.raw.z, v[4], v[5]);
    unpack2(p.raw.w, v[6], v[7]);
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// The outputs' only rounding: fp32 to the I/O type, to nearest.
__device__ __forceinline__ void pack(Pack<float, 1> &p, const float (&v)[1]) { p.raw = __float_as_uint(v[0]); }
__device__ __forceinline__ void pack(Pack<float, 2> &p, const float (&v)[2])
{
    p.raw = make_uint2(__float_as_uint(v[0]), __float_as_uint(v[1]));
}
__device__ __forceinline__ void pack(Pack<float, 4> &p, const float (&v)[4])
{
    p.raw = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
}
__device__ __forceinline__ void pack(Pack<__nv_bfloat16, 1> &p, const float (&v)[1])
{
    p.raw = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
}
__device__ __forceinline__ void pack(Pack<__nv_bfloat16, 2> &p, const float (&v)[2]) { p.raw = pack2(v[0], v[1]); }
__device__ __forceinline__ void pack(Pack<__nv_bfloat16, 4> &p, const float (&v)[4])
{
    p.raw = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void pack(Pack<__nv_bfloat16, 8> &p, const float (&v)[8])
{
    p.raw = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// Copies 16 or 4 bytes to shared memory behind the thread's back; a thread waits for its
// own groups of copies, oldest first.
__device__ __forceinline__ void copy_async16(void *dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
                 : "memory");
}
// the first `size` of 16 bytes, or four or none, and zeros
__device__ __forceinline__ void copy_async16_part(void *dst, const void *src, int size)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src),
                 "r"(size)
                 : "memory");
}
__device__ __forceinline__ void copy_async4(void *dst, const void *src, int size)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src), "r"(size)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT> __device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

}  // namespace ttt
