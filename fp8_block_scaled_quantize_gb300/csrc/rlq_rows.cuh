// Rows of logits: 16-byte units of bf16 or fp32 elements, loads and stores of units that a
// row's end cuts, and the cluster's exchange of float pairs.  Shared by the translation units
// that stream logits.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "rlq_elem.cuh"

namespace rlq {
namespace {

template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {  // bf16
    static constexpr int N = 8;  // elements per 16 bytes
    static __device__ __forceinline__ float2 get2(const uint4 &v, int j)  // elements 2j, 2j + 1
    {
        const uint32_t w = j == 0 ? v.x : j == 1 ? v.y : j == 2 ? v.z : v.w;
        return make_float2(bf_lo(w), bf_hi(w));
    }
    // maximum of m and the unit's elements; NaN is passed over
    static __device__ __forceinline__ float max_of(float m, const uint4 &v)
    {
        uint32_t a, b;
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(v.x), "r"(v.y));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(v.z), "r"(v.w));
        asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
        return fmaxf(m, fmaxf(bf_lo(a), bf_hi(a)));
    }
    static __device__ __forceinline__ float load(const uint16_t *p) { return __uint_as_float((uint32_t)*p << 16); }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[4])
    {
        return make_uint4(pack_bf16x2(f[0]), pack_bf16x2(f[1]), pack_bf16x2(f[2]), pack_bf16x2(f[3]));
    }
};
template <>
struct Elem<uint32_t> {  // fp32
    static constexpr int N = 4;
    static __device__ __forceinline__ float2 get2(const uint4 &v, int j)
    {
        return j == 0 ? make_float2(__uint_as_float(v.x), __uint_as_float(v.y))
                      : make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    static __device__ __forceinline__ float max_of(float m, const uint4 &v)
    {
        return fmaxf(fmaxf(m, __uint_as_float(v.x)),
                     fmaxf(fmaxf(__uint_as_float(v.y), __uint_as_float(v.z)), __uint_as_float(v.w)));
    }
    static __device__ __forceinline__ float load(const uint32_t *p) { return __uint_as_float(*p); }
    static __device__ __forceinline__ uint4 pack(const float2 (&f)[2])
    {
        return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                          __float_as_uint(f[1].y));
    }
};

// 2^x, results below 2^-126 flushed to zero (one instruction).
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A float pair from shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ float2 ld_cluster2(const float2 *p, uint32_t rank)
{
    uint32_t a;
    float2 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}

// A float from there.
__device__ __forceinline__ float ld_cluster1(const float *p, uint32_t rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"((uint32_t)__cvta_generic_to_shared(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void cluster_arrive()
{
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
// An arrival that orders nothing: it does not wait for the thread's own stores.
__device__ __forceinline__ void cluster_arrive_relaxed()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// 16 bytes of a row, which the same thread may overwrite later in the kernel.
__device__ __forceinline__ uint4 ld_row(const void *p)
{
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

// The unit at elements e0 .. of a row of V, cut by one of the row's ends: the elements
// outside read as -inf and are not written.  (Out of line: a row has at most one such
// unit at each end, unless the gradient's rows lie on another 16-byte phase.)
template <typename T>
__device__ __noinline__ uint4 load_cut(const T *x, int e0, int V)
{
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
#pragma unroll
    for (int j = 0; j < Elem<T>::N; ++j)
        if (e0 + j >= 0 && e0 + j < V) {
            const uint32_t b = (uint32_t)x[e0 + j];
            if (sizeof(T) == 2)
                w[j / 2] = (j & 1) ? (w[j / 2] & 0xFFFFu) | (b << 16) : (w[j / 2] & 0xFFFF0000u) | b;
            else
                w[j & 3] = b;
        }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __noinline__ void store_cut(T *dx, int e0, int V, uint4 v)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < Elem<T>::N; ++j)
        if (e0 + j >= 0 && e0 + j < V)
            dx[e0 + j] = sizeof(T) == 2 ? (T)(w[j / 2] >> (16 * (j & 1))) : (T)w[j & 3];
}

}  // namespace
}  // namespace rlq
