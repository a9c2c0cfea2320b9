// Vector access and the activations the layer kernels share.
#pragma once
#include "common.cuh"

namespace ssd {

// NV consecutive elements in one access; the address has to be aligned for it.
template <typename TI, int NV> struct Pack;
template <> struct Pack<__nv_bfloat16, 8> {
    using T = uint4;
};
template <> struct Pack<__nv_bfloat16, 4> {
    using T = uint2;
};
template <> struct Pack<__nv_bfloat16, 2> {
    using T = uint32_t;
};
template <> struct Pack<float, 4> {
    using T = float4;
};
template <> struct Pack<float, 2> {
    using T = float2;
};
template <typename TI> struct Pack<TI, 1> {
    using T = TI;
};

// An aligned vector.  Volatile, so that a load issued ahead of its use stays
// there: the compiler would otherwise sink it to the use.
template <typename T> __device__ __forceinline__ T load_ahead_as(const void *p)
{
    static_assert(sizeof(T) == 2 || sizeof(T) == 4 || sizeof(T) == 8 || sizeof(T) == 16, "one access");
    T r;
    if constexpr (sizeof(T) == 2)
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(*reinterpret_cast<unsigned short *>(&r)) : "l"(p));
    else if constexpr (sizeof(T) == 4)
        asm volatile("ld.global.u32 %0, [%1];" : "=r"(*reinterpret_cast<unsigned *>(&r)) : "l"(p));
    else if constexpr (sizeof(T) == 8)
        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];"
                     : "=r"(reinterpret_cast<unsigned *>(&r)[0]), "=r"(reinterpret_cast<unsigned *>(&r)[1])
                     : "l"(p));
    else
        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(reinterpret_cast<unsigned *>(&r)[0]), "=r"(reinterpret_cast<unsigned *>(&r)[1]),
                       "=r"(reinterpret_cast<unsigned *>(&r)[2]), "=r"(reinterpret_cast<unsigned *>(&r)[3])
                     : "l"(p));
    return r;
}

template <typename TI, int NV>
__device__ __forceinline__ void unpack(const typename Pack<TI, NV>::T &p, float (&v)[NV])
{
    const TI *e = reinterpret_cast<const TI *>(&p);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        v[i] = to_f32(e[i]);
}

template <typename TI, int NV> __device__ __forceinline__ void load_vec(const TI *p, float (&v)[NV])
{
    using T = typename Pack<TI, NV>::T;
    const T u = *reinterpret_cast<const T *>(p);
    unpack<TI, NV>(u, v);
}

__device__ __forceinline__ void round_pair(float a, float b, __nv_bfloat16 *e)
{
    *reinterpret_cast<__nv_bfloat162 *>(e) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void round_pair(float a, float b, float *e)
{
    e[0] = a;
    e[1] = b;
}
template <typename TI, int NV> __device__ __forceinline__ void store_vec(TI *p, const float (&v)[NV])
{
    using T = typename Pack<TI, NV>::T;
    alignas(16) TI e[NV];
#pragma unroll
    for (int i = 0; i + 1 < NV; i += 2)
        round_pair(v[i], v[i + 1], e + i);
    if (NV % 2)
        e[NV - 1] = from_f32<TI>(v[NV - 1]);
    *reinterpret_cast<T *>(p) = *reinterpret_cast<const T *>(e);
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float rcp(float x)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Asynchronous copies of 4, 8 or 16 bytes into shared memory.
template <int BYTES> __device__ __forceinline__ void copy_async(void *dst, const void *src)
{
    static_assert(BYTES == 4 || BYTES == 8 || BYTES == 16, "one copy");
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"((unsigned)__cvta_generic_to_shared(dst)), "l"(src),
                 "n"(BYTES)
                 : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Waits until at most LEFT of the thread's groups are in flight.
template <int LEFT> __device__ __forceinline__ void copy_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

// 1 / (1 + e^-z) with the hardware's exponential and reciprocal (a few ulp);
// e^-z overflows to inf for z < -88 and the result is then 0.
__device__ __forceinline__ float fast_sigmoid(float z) { return rcp(1.f + ex2(-kLog2e * z)); }

// silu(z) = z sigmoid(z).
__device__ __forceinline__ float fast_silu(float z) { return z * fast_sigmoid(z); }

// Two f32 lanes in one instruction (half the issue slots of two scalar ones).
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pk2(float a, float b)
{
    f32x2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void un2(f32x2 p, float &a, float &b)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c)
{
    f32x2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b)
{
    f32x2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f32x2 ex2_2(f32x2 p)
{
    float a, b;
    un2(p, a, b);
    return pk2(ex2(a), ex2(b));
}
__device__ __forceinline__ float hsum(f32x2 p)
{
    float a, b;
    un2(p, a, b);
    return a + b;
}

__device__ __forceinline__ f32x2 dup2(float a) { return pk2(a, a); }
__device__ __forceinline__ f32x2 sigmoid2(f32x2 z)
{
    float a, b;
    un2(add2(ex2_2(mul2(z, dup2(-kLog2e))), dup2(1.f)), a, b);
    return pk2(rcp(a), rcp(b));
}
// silu'(z) = s (1 + z (1 - s)) = s + s z (1 - s) with s = sigmoid(z)
__device__ __forceinline__ f32x2 silu_grad2(f32x2 z, f32x2 s)
{
    return fma2(mul2(s, z), fma2(s, dup2(-1.f), dup2(1.f)), s);
}

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1].  With
// s = e / (2 + e) <= 1/3, log(1 + e) = 2 artanh(s), which loses no digits to
// 1 + e as e -> 0.  2 artanh(s) / s is a polynomial of degree four in s^2
// (Chebyshev interpolation on [0, 1/9]; relative error 8e-9 with the f32
// coefficients).  In f32 the whole is off by 3.9e-7 of its value for |x| <= 5,
// 9.4e-7 for |x| <= 20 and 3.7e-6 down to -80, where the exponent's rounding
// is what is left.
__device__ __forceinline__ void softplus2(float x0, float x1, float &y0, float &y1)
{
    const f32x2 t = mul2(pk2(-fabsf(x0), -fabsf(x1)), pk2(kLog2e, kLog2e));
    const f32x2 e = ex2_2(t);
    float d0, d1;
    un2(add2(e, pk2(2.f, 2.f)), d0, d1);
    const f32x2 s = mul2(e, pk2(rcp(d0), rcp(d1)));
    const f32x2 q = mul2(s, s);
    f32x2 p = fma2(q, pk2(0.28157780f, 0.28157780f), pk2(0.27965158f, 0.27965158f));
    p = fma2(p, q, pk2(0.40024596f, 0.40024596f));
    p = fma2(p, q, pk2(0.66666323f, 0.66666323f));
    p = fma2(p, q, pk2(2.f, 2.f));
    un2(fma2(s, p, pk2(fmaxf(x0, 0.f), fmaxf(x1, 0.f))), y0, y1);
}
__device__ __forceinline__ float softplus(float x)
{
    float a, b;
    softplus2(x, x, a, b);
    return a;
}

}  // namespace ssd
