// Vector access and the activations the layer kernels share.
#pragma once
#include "common.cuh"

namespace ssd {

// NV consecutive elements as f32: one vector access where `vec` says the
// address is aligned for it, else one element at a time.  Elements at or past
// `n` read as zero and are not written.
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

template <typename TI, int NV> __device__ __forceinline__ void store_vec(TI *p, const float (&v)[NV])
{
    using T = typename Pack<TI, NV>::T;
    T u;
    TI *e = reinterpret_cast<TI *>(&u);
#pragma unroll
    for (int i = 0; i < NV; ++i)
        e[i] = from_f32<TI>(v[i]);
    *reinterpret_cast<T *>(p) = u;
}

// 1 / (1 + e^-z) with the fast exponential and division (a few ulp each);
// e^-z overflows to inf for z < -88 and the quotient is then 0.
__device__ __forceinline__ float fast_sigmoid(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// silu(z) = z sigmoid(z) and its derivative s (1 + z (1 - s)).
__device__ __forceinline__ float fast_silu(float z) { return __fdividef(z, 1.f + __expf(-z)); }
__device__ __forceinline__ float silu_grad(float z, float s) { return s * fmaf(z, 1.f - s, 1.f); }

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| in (0, 1].  With
// s = e / (2 + e) <= 1/3, log(1 + e) = 2 artanh(s) = 2 s (1 + s^2/3 + s^4/5 + ...),
// which keeps full relative precision as e -> 0; the first term left out is
// s^14 / 15 < 2e-8.
__device__ __forceinline__ float softplus(float x)
{
    const float e = __expf(-fabsf(x));
    const float s = __fdividef(e, 2.f + e);
    const float q = s * s;
    float p = fmaf(q, 1.f / 13.f, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    p = fmaf(p, q, 1.f);
    return fmaf(2.f * s, p, fmaxf(x, 0.f));
}

}  // namespace ssd
