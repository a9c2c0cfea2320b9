// Pieces the selective scan's forward, reverse and gradient kernels share.
#pragma once
#include "ssd_internal.h"
#include "vec.cuh"

namespace ssd {

// A thread holds four states, of one channel (the single-token kernel) or of
// each of two adjacent ones; LN = 1, 2, 4, 8 or 16 lanes hold all of a channel's
// (up to 4 LN; the ones past dstate stay zero).
// Tokens of one chunk: a state is kept at each chunk's start for the backward.
constexpr int kScanChunk = 16;

constexpr float kLn2 = 0.6931471805599453f;

// Four consecutive elements as loaded; elements past n are zero.
template <typename TI> using Raw4 = typename Pack<TI, 4>::T;

template <typename TI> __device__ __forceinline__ Raw4<TI> load_raw4(const TI *p, int n, bool vec)
{
    Raw4<TI> r{};
    if (vec && n >= 4)
        return *reinterpret_cast<const Raw4<TI> *>(p);
    TI *e = reinterpret_cast<TI *>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n)
            e[i] = p[i];
    return r;
}
// Four elements at any address.
template <typename TI> __device__ __forceinline__ Raw4<TI> load_four(const TI *p)
{
    Raw4<TI> r;
    TI *e = reinterpret_cast<TI *>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        e[i] = load_ahead_as<TI>(p + i);
    return r;
}
// The first n of W values.
template <typename TI, int W> __device__ __forceinline__ void store_some(TI *p, const float (&v)[W], int n, bool vec)
{
    if (vec && n >= W) {
        store_vec<TI, W>(p, v);
        return;
    }
    if (n >= W) {
#pragma unroll
        for (int i = 0; i < W; ++i)
            p[i] = from_f32<TI>(v[i]);
        return;
    }
#pragma unroll
    for (int i = 0; i < W; ++i)
        if (i < n)
            p[i] = from_f32<TI>(v[i]);
}

// The four states of one lane in an f32 [.., N] array.
__device__ __forceinline__ void load_states(const float *p, int n, float (&v)[4])
{
    if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        load_vec<float, 4>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = i < n ? p[i] : 0.f;
}
__device__ __forceinline__ void store_states(float *p, int n, const float (&v)[4])
{
    if (n >= 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
        store_vec<float, 4>(p, v);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < n)
            p[i] = v[i];
}

// ex2.approx is 2e-8 to 5e-8 low on average for exponents between -1e-2 and
// -1, and a slowly decaying state multiplies hundreds of decays.  This, added
// to the exponents (an fma in place of the product), centres its error there:
// the gradient of A over 4096 tokens is off by 8e-7 of its norm instead of
// 1.7e-6, the final state by 3e-7 instead of 5.9e-7.  2^kDecayNudge itself
// comes out as 1, so a token without a step keeps the state exactly.
constexpr float kDecayNudge = 2.5e-8f;

// A decay rate in log2 units.  -inf becomes the lowest float, so that a token
// without a step (delta = 0, as past a sequence's end) still keeps the state.
__device__ __forceinline__ float decay_rate(float a)
{
    const float r = a * kLog2e;
    return r == -INFINITY ? -3.402823466e38f : r;
}

// e + 2^x v for a whole run's factor 2^x, which may be beyond f32 where the
// states grow: one that is zero stays zero, a small one is scaled in two steps.
constexpr float kLargeExponent = 120.f;
__device__ __forceinline__ float add_scaled(float x, float v, float e)
{
    if (x > kLargeExponent)
        return v == 0.f ? e : fmaf(v * ex2(x - kLargeExponent), ex2(kLargeExponent), e);
    return fmaf(ex2(x), v, e);
}

}  // namespace ssd
