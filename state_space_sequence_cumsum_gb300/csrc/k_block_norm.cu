// The norms between two blocks, fused with the block's gate and the scaled
// residual add.
//
// Row t of `dim` channels, gate row j(t) = t / (ntokens / gate_rows):
//     p = rmsnorm(y) * post_weight   (or y without post_weight)
//     r = residual + scale * gate[j] * p,     out = rmsnorm(r) * weight
// with rmsnorm(v) = v / sqrt(mean(v^2) + eps).  Backward, from y and r:
//     gr = dr + (gn - rh mean(gn rh)) rs_r,   gn = dout weight,  rh = r rs_r
//     dresidual = gr,  dgate[j] = scale sum gr p,  dp = scale gate gr
//     dy = (gp - yh mean(gp yh)) rs_y,  gp = dp post_weight,  yh = y rs_y
//     dweight = sum dout rh,  dpost_weight = sum dp yh
// Both directions should be bound by HBM traffic.  A team of threads holds a
// row in registers from its one read to its one write; the row sums are the
// only communication (shuffles, and shared memory between a team's warps).
// Statistics and sums are f32; r is kept in f32 for `out` and rounded once to
// the residual's type where it is stored.  On a GB300, 16384 rows of 2560 bf16
// channels with an f32 residual, a post norm and a gate:
//     forward   88 us, 5.7 TB/s (85% of the measured copy rate)
//     backward 129 us, 5.9 TB/s (87%); 176 us with the weights read again for
//              every row, row sums of fifteen shuffles and twice the blocks
#include "ssd_internal.h"
#include "vec.cuh"

namespace ssd {
namespace {

// Threads of a row's team at most.  The backward's fewer leave registers for
// two blocks an SM (a row's four inputs, the next row's, and three sums).
constexpr int kFwdTeam = 512, kBwdTeam = 320;
constexpr int kMaxWarps = 16;  // of a team; a power of two

// Adds K values over the team (blockDim.x threads, a multiple of 32); every
// thread of the block must call it.  One barrier: `buf` (one Sum<K> per warp
// of the block) may be used again once another barrier has passed.
template <int K> struct alignas(K > 2 ? 16 : 4 * K) Sum {
    float v[K];
};
template <int K> __device__ __forceinline__ void team_sum(float (&v)[K], Sum<K> *buf)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    const int warps = blockDim.x >> 5;
    if (warps == 1)
        return;
    Sum<K> *s = buf + threadIdx.y * warps;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int k = 0; k < K; ++k)
            s[threadIdx.x >> 5].v[k] = v[k];
    __syncthreads();
    // each lane takes one warp's sums and all add them by shuffles (every
    // thread reading every warp's costs more of the shared memory pipe)
    const int other = threadIdx.x % kMaxWarps;
    Sum<K> t{};
    if (other < warps)
        t = s[other];
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = t.v[k];
#pragma unroll
    for (int o = kMaxWarps / 2; o > 0; o >>= 1)
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

// The same for three values, which share shuffles: at the first two steps a
// lane passes on the values that other lanes go on with (six shuffles instead
// of fifteen), and of the warps' sums a quarter warp adds up one value's.
__device__ __forceinline__ void team_sum3(float (&v)[3], Sum<3> *buf)
{
    const int lane = threadIdx.x & 31;
    const bool hi = lane & 16, odd = lane & 8;
    // lanes 0-15 go on with v[0] and v[1], the others with v[2] and nothing
    float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, hi ? v[0] : v[2], 16);
    const float from = __shfl_xor_sync(0xffffffffu, v[1], 16);
    const float b = hi ? 0.f : v[1] + from;
    // then each quarter with one
    a = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, 8);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1)
        a += __shfl_xor_sync(0xffffffffu, a, o);
    const int warps = blockDim.x >> 5;
    if (warps > 1) {
        float *s = reinterpret_cast<float *>(buf + threadIdx.y * warps);
        if ((lane & 7) == 0)
            s[(threadIdx.x >> 5) * 4 + lane / 8] = a;
        __syncthreads();
        a = 0.f;
#pragma unroll
        for (int w = 0; w < kMaxWarps; w += 8)
            if (w + (lane & 7) < warps)
                a += s[(w + (lane & 7)) * 4 + lane / 8];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1)
            a += __shfl_xor_sync(0xffffffffu, a, o);
    }
    v[0] = __shfl_sync(0xffffffffu, a, 0);
    v[1] = __shfl_sync(0xffffffffu, a, 8);
    v[2] = __shfl_sync(0xffffffffu, a, 16);
}

template <int VEC> __device__ __forceinline__ void scale_by(const float *p, float (&v)[VEC])
{
    float w[VEC];
    load_vec<float, VEC>(p, w);
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        v[i] *= w[i];
}

// One row per team; blockDim = (team, teams).  A thread holds VPT vectors of
// VEC channels, `team` vectors apart.
template <typename TI, typename TR, int VEC, int VPT>
__global__ void __launch_bounds__(kFwdTeam)
block_norm_kernel(const TI *__restrict__ y, const TR *residual, const float *__restrict__ weight,
                  const float *__restrict__ post_weight, const float *__restrict__ gate, TI *__restrict__ out,
                  TR *residual_out, NormGeom g)
{
    __shared__ Sum<1> sum_y[kMaxWarps], sum_r[kMaxWarps];
    const int team = blockDim.x;
    const int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    const bool live = row < g.ntokens;
    const int nv = (int)(g.dim / VEC);
    float yv[VPT][VEC], rv[VPT][VEC];
    float s[1] = {0.f};
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int v = threadIdx.x + q * team;
        if (live && v < nv) {
            load_vec<TI, VEC>(y + row * g.dim + v * VEC, yv[q]);
            if (residual)
                load_vec<TR, VEC>(residual + row * g.dim + v * VEC, rv[q]);
            else
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    rv[q][i] = 0.f;
        } else {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                yv[q][i] = rv[q][i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            s[0] = fmaf(yv[q][i], yv[q][i], s[0]);
    }
    float f = g.scale;
    if (post_weight) {
        team_sum<1>(s, sum_y);
        f *= rsqrtf(s[0] * g.inv_dim + g.eps);
    }
    const float *gr = gate ? gate + (live ? row / g.tokens_per_gate : 0) * g.dim : nullptr;
    s[0] = 0.f;
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int v = threadIdx.x + q * team;
        if (live && v < nv) {
            float a[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                a[i] = f;
            if (post_weight)
                scale_by<VEC>(post_weight + v * VEC, a);
            if (gr)
                scale_by<VEC>(gr + v * VEC, a);
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                rv[q][i] = fmaf(a[i], yv[q][i], rv[q][i]);
                s[0] = fmaf(rv[q][i], rv[q][i], s[0]);
            }
            store_vec<TR, VEC>(residual_out + row * g.dim + v * VEC, rv[q]);
        }
    }
    team_sum<1>(s, sum_r);
    const float rs = rsqrtf(s[0] * g.inv_dim + g.eps);
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int v = threadIdx.x + q * team;
        if (live && v < nv) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                rv[q][i] *= rs;
            scale_by<VEC>(weight + v * VEC, rv[q]);
            store_vec<TI, VEC>(out + row * g.dim + v * VEC, rv[q]);
        }
    }
}

template <typename TI, int VEC>
__device__ __forceinline__ void to_pairs(const typename Pack<TI, VEC>::T &r, f32x2 (&p)[(VEC + 1) / 2])
{
    float v[VEC];
    unpack<TI, VEC>(r, v);
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i)
        p[i] = pk2(v[2 * i], 2 * i + 1 < VEC ? v[(2 * i + 1) % VEC] : 0.f);
}
template <typename TI, int VEC> __device__ __forceinline__ void store_pairs(TI *p, const f32x2 (&o)[(VEC + 1) / 2])
{
    float v[VEC];
#pragma unroll
    for (int i = 0; i < (VEC + 1) / 2; ++i) {
        float x, y;
        un2(o[i], x, y);
        v[2 * i] = x;
        if (2 * i + 1 < VEC)
            v[(2 * i + 1) % VEC] = y;
    }
    store_vec<TI, VEC>(p, v);
}

// A thread's inputs of one vector of a row.  Rows of four-channel vectors, at
// most four a thread, come by asynchronous copies two rows ahead into the
// thread's own slots (no barrier: it reads what it copied itself).
template <typename TI, typename TR, int VEC> struct NormSlot {
    typename Pack<TR, VEC>::T r, d;
    typename Pack<TI, VEC>::T y, n;
};
// The slots' components each in an array of their own (`n` entries): neighbouring
// threads' then lie side by side.
template <typename TI, typename TR, int VEC> struct NormRing {
    typename Pack<TR, VEC>::T *r, *d;
    typename Pack<TI, VEC>::T *y, *n;
    __device__ NormRing(void *smem, int entries)
    {
        r = static_cast<typename Pack<TR, VEC>::T *>(smem);
        d = r + entries;
        y = reinterpret_cast<typename Pack<TI, VEC>::T *>(d + entries);
        n = y + entries;
    }
};
template <int VEC, int VPT> constexpr bool norm_ring = VEC == 4 && VPT <= 4;

// Backward.  A block walks the rows of its items one after another; an item
// is one of `spans` runs of the tokens of one gate row (or of all tokens).
// The parameters' gradients stay in the thread that owns the channels: the
// weights' over all its rows (one partial per block: part[block][0] is
// weight, [1] post_weight), the gate's over an item (written as it is where
// an item is a whole gate row, else one partial per item).  Values are held
// as f32 pairs; the next rows' inputs are in flight while a row is reduced.
//   ONE: rows of one channel.  There a gradient is all radial, so g - x m,
//   its part across the row's direction, is the eps term alone, g eps rs^2,
//   which the difference of the two nearly equal terms would lose.
template <typename TI, typename TR, int VEC, int VPT, bool ONE>
__global__ void __launch_bounds__(kBwdTeam, VEC * VPT <= 8 ? 2 : 1)
block_norm_bwd_kernel(const TI *__restrict__ y, const TR *__restrict__ r, const float *__restrict__ weight,
                      const float *__restrict__ post_weight, const float *__restrict__ gate,
                      const TI *__restrict__ dout, const TR *dr, TI *__restrict__ dy, TR *dresidual,
                      float *__restrict__ part, float *__restrict__ dgate_part, NormGeom g, int64_t groups,
                      int64_t spans)
{
    __shared__ Sum<3> sum_row[2][kMaxWarps];
    __shared__ Sum<1> sum_p[kMaxWarps];
    constexpr int P = (VEC + 1) / 2;
    using VI = typename Pack<TI, VEC>::T;
    using VR = typename Pack<TR, VEC>::T;
    using Slot = NormSlot<TI, TR, VEC>;
    constexpr bool kRing = norm_ring<VEC, VPT>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    int flip = 0;
    const int team = blockDim.x;
    const NormRing<TI, TR, VEC> ring(smem_raw, 2 * VPT * team);  // [row & 1][vector][thread]
    auto slot = [&](int64_t row, int q) { return (((int)row & 1) * VPT + q) * team + (int)threadIdx.x; };
    const int nv = (int)(g.dim / VEC);
    f32x2 dw[VPT][P], dpw[VPT][P], dg[VPT][P];
#pragma unroll
    for (int q = 0; q < VPT; ++q)
#pragma unroll
        for (int i = 0; i < P; ++i)
            dw[q][i] = dpw[q][i] = 0;
    const int64_t tokens = g.ntokens / groups;
    // a vector of a parameter, ones without it
    auto params = [&](const float *p, int v, f32x2 (&o)[P]) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            o[i] = dup2(1.f);
        if (p && v < nv)
            to_pairs<float, VEC>(*reinterpret_cast<const typename Pack<float, VEC>::T *>(p + v * VEC), o);
    };
    // the weights stay in registers where a thread has few
    constexpr bool kKeepW = VEC * VPT <= 8;
    f32x2 w[VPT][P];
    if (kKeepW)
#pragma unroll
        for (int q = 0; q < VPT; ++q)
            params(weight, threadIdx.x + q * team, w[q]);
    auto across = [&](f32x2 v, f32x2 x, float m, float rs) {
        return ONE ? mul2(v, dup2(g.eps * rs * rs)) : fma2(x, dup2(-m), v);
    };
    for (int64_t item = blockIdx.x; item < groups * spans; item += gridDim.x) {
        const int64_t j = item / spans, sp = item - j * spans;
        const int64_t t0 = j * tokens + tokens * sp / spans, t1 = j * tokens + tokens * (sp + 1) / spans;
        // what a row's gradient is scaled by on its way to the block's output:
        // scale gate post_weight, the same for all rows of an item
        f32x2 kp[VPT][P];
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int v = threadIdx.x + q * team;
            f32x2 pw[P], gv[P];
            params(post_weight, v, pw);
            params(gate ? gate + j * g.dim : nullptr, v, gv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                dg[q][i] = 0;
                kp[q][i] = mul2(mul2(gv[i], dup2(g.scale)), pw[i]);
            }
        }
        // the inputs of `row` into its slot of the thread's ring, or nothing
        auto fetch = [&](int64_t row) {
            if (row < t1)
#pragma unroll
                for (int q = 0; q < VPT; ++q)
                    if ((int)threadIdx.x + q * team < nv) {
                        const int64_t k = row * g.dim + (threadIdx.x + q * team) * VEC;
                        const int o = slot(row, q);
                        copy_async<kRing ? (int)sizeof(VI) : 4>(ring.y + o, y + k);
                        copy_async<kRing ? (int)sizeof(VR) : 4>(ring.r + o, r + k);
                        copy_async<kRing ? (int)sizeof(VI) : 4>(ring.n + o, dout + k);
                        if (dr)
                            copy_async<kRing ? (int)sizeof(VR) : 4>(ring.d + o, dr + k);
                    }
            copy_async_commit();
        };
        if constexpr (kRing) {
            fetch(t0);
            fetch(t0 + 1);
        }
        for (int64_t row = t0; row < t1; ++row) {
            f32x2 yv[VPT][P], rv[VPT][P], gn[VPT][P], gr[VPT][P];
            if constexpr (kRing)
                copy_async_wait<1>();
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                Slot o{};
                if ((int)threadIdx.x + q * team < nv) {
                    if constexpr (kRing) {
                        const int i = slot(row, q);
                        o.y = ring.y[i];
                        o.r = ring.r[i];
                        o.n = ring.n[i];
                        if (dr)
                            o.d = ring.d[i];
                    } else {
                        const int64_t k = row * g.dim + (threadIdx.x + q * team) * VEC;
                        o.y = *reinterpret_cast<const VI *>(y + k);
                        o.r = *reinterpret_cast<const VR *>(r + k);
                        o.n = *reinterpret_cast<const VI *>(dout + k);
                        if (dr)
                            o.d = *reinterpret_cast<const VR *>(dr + k);
                    }
                }
                to_pairs<TI, VEC>(o.y, yv[q]);
                to_pairs<TR, VEC>(o.r, rv[q]);
                to_pairs<TI, VEC>(o.n, gn[q]);
                to_pairs<TR, VEC>(o.d, gr[q]);
            }
            if constexpr (kRing)
                fetch(row + 2);
            const int64_t out = row * g.dim;
            f32x2 s0 = 0, s1 = 0, s2 = 0;
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                if (!kKeepW)
                    params(weight, threadIdx.x + q * team, w[q]);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    s0 = fma2(yv[q][i], yv[q][i], s0);
                    s1 = fma2(rv[q][i], rv[q][i], s1);
                    s2 = fma2(mul2(gn[q][i], w[q][i]), rv[q][i], s2);
                }
            }
            float s[3] = {hsum(s0), hsum(s1), hsum(s2)};
            team_sum3(s, sum_row[flip]);
            flip ^= 1;
            const float rs_y = post_weight ? rsqrtf(s[0] * g.inv_dim + g.eps) : 1.f;
            const float rs_r = rsqrtf(s[1] * g.inv_dim + g.eps);
            const float c = s[2] * g.inv_dim * rs_r * rs_r;  // mean(gn rh) rs_r
            f32x2 u2 = 0;
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                const int v = threadIdx.x + q * team;
                if (v < nv) {
                    if (!kKeepW)
                        params(weight, v, w[q]);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        dw[q][i] = fma2(gn[q][i], mul2(rv[q][i], dup2(rs_r)), dw[q][i]);
                        gr[q][i] = fma2(across(mul2(gn[q][i], w[q][i]), rv[q][i], c, rs_r), dup2(rs_r), gr[q][i]);
                    }
                    store_pairs<TR, VEC>(dresidual + out + v * VEC, gr[q]);
#pragma unroll
                    for (int i = 0; i < P; ++i) {
                        const f32x2 yh = mul2(yv[q][i], dup2(rs_y));
                        dg[q][i] = fma2(gr[q][i], yh, dg[q][i]);
                        gr[q][i] = mul2(gr[q][i], kp[q][i]);
                        u2 = fma2(gr[q][i], yh, u2);
                        yv[q][i] = yh;
                    }
                }
            }
            float m = 0.f;
            if (post_weight) {
                float u[1] = {hsum(u2)};
                team_sum<1>(u, sum_p);
                m = u[0] * g.inv_dim;
            }
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                const int v = threadIdx.x + q * team;
                if (v < nv) {
                    if (post_weight)
#pragma unroll
                        for (int i = 0; i < P; ++i)
                            gr[q][i] = mul2(across(gr[q][i], yv[q][i], m, rs_y), dup2(rs_y));
                    store_pairs<TI, VEC>(dy + out + v * VEC, gr[q]);
                }
            }
        }
        // sum gr yh of the item: times scale gate it is post_weight's gradient,
        // times scale post_weight the gate's
#pragma unroll
        for (int q = 0; q < VPT; ++q) {
            const int v = threadIdx.x + q * team;
            f32x2 pw[P], gv[P];
            params(post_weight, v, pw);
            params(gate ? gate + j * g.dim : nullptr, v, gv);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                dg[q][i] = mul2(dg[q][i], dup2(g.scale));
                dpw[q][i] = fma2(dg[q][i], gv[i], dpw[q][i]);
                dg[q][i] = mul2(dg[q][i], pw[i]);
            }
            if (gate && v < nv)
                store_pairs<float, VEC>(dgate_part + item * g.dim + v * VEC, dg[q]);
        }
    }
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int v = threadIdx.x + q * team;
        if (v < nv) {
            store_pairs<float, VEC>(part + ((int64_t)blockIdx.x * 2) * g.dim + v * VEC, dw[q]);
            store_pairs<float, VEC>(part + ((int64_t)blockIdx.x * 2 + 1) * g.dim + v * VEC, dpw[q]);
        }
    }
}

// Rows too wide for the register kernels: a block of kWideThreads per row that
// goes over it in turns, keeping the residual (or its gradient) in shared
// memory.  A thread always has the same channels, so only the sums need
// barriers, and the parameters' gradients are added up in the partials
// themselves.
constexpr int kWideThreads = 512;

template <int VEC> __device__ __forceinline__ void load_or(const float *p, int c, float other, float (&v)[VEC])
{
    if (p)
        load_vec<float, VEC>(p + c, v);
    else
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] = other;
}

template <typename TI, typename TR, int VEC>
__global__ void __launch_bounds__(kWideThreads)
block_norm_wide_kernel(const TI *__restrict__ y, const TR *residual, const float *__restrict__ weight,
                       const float *__restrict__ post_weight, const float *__restrict__ gate,
                       TI *__restrict__ out, TR *residual_out, NormGeom g)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float *r = reinterpret_cast<float *>(smem_raw);
    __shared__ Sum<1> sum_y[kMaxWarps], sum_r[kMaxWarps];
    const int64_t at = (int64_t)blockIdx.x * g.dim;
    const int first = threadIdx.x * VEC, step = kWideThreads * VEC, dim = (int)g.dim;
    float f = g.scale, s[1] = {0.f};
    if (post_weight) {
        for (int c = first; c < dim; c += step) {
            float v[VEC];
            load_vec<TI, VEC>(y + at + c, v);
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                s[0] = fmaf(v[i], v[i], s[0]);
        }
        team_sum<1>(s, sum_y);
        f *= rsqrtf(s[0] * g.inv_dim + g.eps);
    }
    const float *gr = gate ? gate + blockIdx.x / g.tokens_per_gate * g.dim : nullptr;
    s[0] = 0.f;
    for (int c = first; c < dim; c += step) {
        float v[VEC], rv[VEC] = {}, pw[VEC], gv[VEC];
        load_vec<TI, VEC>(y + at + c, v);
        if (residual)
            load_vec<TR, VEC>(residual + at + c, rv);
        load_or<VEC>(post_weight, c, 1.f, pw);
        load_or<VEC>(gr, c, 1.f, gv);
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
            rv[i] = fmaf(f * pw[i] * gv[i], v[i], rv[i]);
            s[0] = fmaf(rv[i], rv[i], s[0]);
        }
        store_vec<float, VEC>(r + c, rv);
        store_vec<TR, VEC>(residual_out + at + c, rv);
    }
    team_sum<1>(s, sum_r);
    const float rs = rsqrtf(s[0] * g.inv_dim + g.eps);
    for (int c = first; c < dim; c += step) {
        float v[VEC], w[VEC];
        load_vec<float, VEC>(r + c, v);
        load_vec<float, VEC>(weight + c, w);
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            v[i] *= rs * w[i];
        store_vec<TI, VEC>(out + at + c, v);
    }
}

template <typename TI, typename TR, int VEC>
__global__ void __launch_bounds__(kWideThreads)
block_norm_bwd_wide_kernel(const TI *__restrict__ y, const TR *__restrict__ r, const float *__restrict__ weight,
                           const float *__restrict__ post_weight, const float *__restrict__ gate,
                           const TI *__restrict__ dout, const TR *dr, TI *__restrict__ dy, TR *dresidual,
                           float *part, float *dgate_part, NormGeom g, int64_t groups, int64_t spans)
{
    extern __shared__ __align__(16) unsigned char smem_raw[];
    float *grad = reinterpret_cast<float *>(smem_raw);
    __shared__ Sum<3> sum_row[2][kMaxWarps];
    __shared__ Sum<1> sum_p[kMaxWarps];
    const int first = threadIdx.x * VEC, step = kWideThreads * VEC, dim = (int)g.dim;
    float *dw = part + (int64_t)blockIdx.x * 2 * g.dim, *dpw = dw + g.dim;
    for (int c = first; c < dim; c += step)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            dw[c + i] = dpw[c + i] = 0.f;
    int flip = 0;
    const int64_t tokens = g.ntokens / groups;
    for (int64_t item = blockIdx.x; item < groups * spans; item += gridDim.x) {
        const int64_t j = item / spans, sp = item - j * spans;
        const int64_t t0 = j * tokens + tokens * sp / spans, t1 = j * tokens + tokens * (sp + 1) / spans;
        const float *gj = gate ? gate + j * g.dim : nullptr;
        float *dg = gate ? dgate_part + item * g.dim : nullptr;
        if (dg)
            for (int c = first; c < dim; c += step)
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    dg[c + i] = 0.f;
        for (int64_t row = t0; row < t1; ++row) {
            const int64_t at = row * g.dim;
            float s[3] = {0.f, 0.f, 0.f};
            for (int c = first; c < dim; c += step) {
                float yv[VEC], rv[VEC], gn[VEC], w[VEC];
                load_vec<TI, VEC>(y + at + c, yv);
                load_vec<TR, VEC>(r + at + c, rv);
                load_vec<TI, VEC>(dout + at + c, gn);
                load_vec<float, VEC>(weight + c, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    s[0] = fmaf(yv[i], yv[i], s[0]);
                    s[1] = fmaf(rv[i], rv[i], s[1]);
                    s[2] = fmaf(gn[i] * w[i], rv[i], s[2]);
                }
            }
            team_sum3(s, sum_row[flip]);
            flip ^= 1;
            const float rs_y = post_weight ? rsqrtf(s[0] * g.inv_dim + g.eps) : 1.f;
            const float rs_r = rsqrtf(s[1] * g.inv_dim + g.eps);
            const float k = s[2] * g.inv_dim * rs_r * rs_r;
            float u[1] = {0.f};
            for (int c = first; c < dim; c += step) {
                float yv[VEC], rv[VEC], gn[VEC], w[VEC], gr[VEC] = {}, pw[VEC], gv[VEC], a[VEC], b[VEC], d[VEC] = {};
                load_vec<TI, VEC>(y + at + c, yv);
                load_vec<TR, VEC>(r + at + c, rv);
                load_vec<TI, VEC>(dout + at + c, gn);
                load_vec<float, VEC>(weight + c, w);
                if (dr)
                    load_vec<TR, VEC>(dr + at + c, gr);
                load_or<VEC>(post_weight, c, 1.f, pw);
                load_or<VEC>(gj, c, 1.f, gv);
                load_vec<float, VEC>(dw + c, a);
                load_vec<float, VEC>(dpw + c, b);
                if (dg)
                    load_vec<float, VEC>(dg + c, d);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    a[i] = fmaf(gn[i], rv[i] * rs_r, a[i]);
                    gr[i] = fmaf(rs_r, fmaf(-rv[i], k, gn[i] * w[i]), gr[i]);
                    const float yh = yv[i] * rs_y, q = g.scale * gr[i] * yh;
                    b[i] = fmaf(q, gv[i], b[i]);
                    d[i] = fmaf(q, pw[i], d[i]);
                    gn[i] = g.scale * gv[i] * pw[i] * gr[i];  // the gradient of yh
                    u[0] = fmaf(gn[i], yh, u[0]);
                }
                store_vec<TR, VEC>(dresidual + at + c, gr);
                store_vec<float, VEC>(grad + c, gn);
                store_vec<float, VEC>(dw + c, a);
                store_vec<float, VEC>(dpw + c, b);
                if (dg)
                    store_vec<float, VEC>(dg + c, d);
            }
            float m = 0.f;
            if (post_weight) {
                team_sum<1>(u, sum_p);
                m = u[0] * g.inv_dim;
            }
            for (int c = first; c < dim; c += step) {
                float yv[VEC], gn[VEC];
                load_vec<float, VEC>(grad + c, gn);
                load_vec<TI, VEC>(y + at + c, yv);
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    gn[i] = post_weight ? rs_y * fmaf(-yv[i] * rs_y, m, gn[i]) : gn[i];
                store_vec<TI, VEC>(dy + at + c, gn);
            }
        }
    }
}

// Adds the partials in a fixed order: blockIdx.y 0 is dweight, 1 dpost_weight
// (may be nullptr), 2 + j row j of dgate.  blockDim = (32, 32).
struct NormSums {
    const float *part, *gate_part;
    float *dweight, *dpost_weight, *dgate;
    int64_t blocks, spans, dim;
};
__global__ void __launch_bounds__(1024) norm_sums_kernel(NormSums a)
{
    __shared__ float red[32][33];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const int which = blockIdx.y;
    const float *src = which < 2 ? a.part + which * a.dim : a.gate_part + (int64_t)(which - 2) * a.spans * a.dim;
    float *out = which == 0 ? a.dweight : which == 1 ? a.dpost_weight : a.dgate + (int64_t)(which - 2) * a.dim;
    if (!out)
        return;
    const int64_t n = which < 2 ? a.blocks : a.spans, stride = which < 2 ? 2 * a.dim : a.dim;
    float s = 0.f;
    if (c < a.dim)
#pragma unroll 16
        for (int64_t p = threadIdx.y; p < n; p += 32)
            s += src[p * stride + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    s = red[threadIdx.x][threadIdx.y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s += __shfl_xor_sync(0xffffffffu, s, o);
    const int64_t cw = (int64_t)blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && cw < a.dim)
        out[cw] = s;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Threads of a row's team, and vectors of each, for a row of nv vectors: few
// vectors a thread while the team stays within `most` threads.  0 vectors:
// the row needs the wide kernel.
void team_shape(int64_t nv, int most, int *team, int *vpt)
{
    for (int v : {1, 2, 4}) {
        *vpt = v;
        *team = (int)((nv + v * 32 - 1) / (v * 32)) * 32;
        if (*team <= most)
            return;
    }
    *vpt = 0;
}

template <typename TI, typename TR, int VEC>
cudaError_t fwd_wide(const void *y, const void *residual, const float *weight, const float *post_weight,
                     const float *gate, void *out, void *residual_out, const NormGeom &g, int, cudaStream_t st)
{
    auto k = block_norm_wide_kernel<TI, TR, VEC>;
    const size_t smem = (size_t)g.dim * sizeof(float);
    static SmemGrant granted;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(k), smem, &granted);
    if (e != cudaSuccess)
        return e;
    k<<<(unsigned)g.ntokens, kWideThreads, smem, st>>>(
        static_cast<const TI *>(y), static_cast<const TR *>(residual), weight, post_weight, gate,
        static_cast<TI *>(out), static_cast<TR *>(residual_out), g);
    note_launch(1);
    return cudaGetLastError();
}

template <typename TI, typename TR, int VEC, int VPT>
cudaError_t fwd_v(const void *y, const void *residual, const float *weight, const float *post_weight,
                  const float *gate, void *out, void *residual_out, const NormGeom &g, int team,
                  cudaStream_t st)
{
    const int teams = team >= 128 ? 1 : 128 / team;
    const int64_t blocks = (g.ntokens + teams - 1) / teams;
    block_norm_kernel<TI, TR, VEC, VPT><<<(unsigned)blocks, dim3(team, teams), 0, st>>>(
        static_cast<const TI *>(y), static_cast<const TR *>(residual), weight, post_weight, gate,
        static_cast<TI *>(out), static_cast<TR *>(residual_out), g);
    note_launch(1);
    return cudaGetLastError();
}

struct BwdPlan {
    int64_t groups, spans, blocks;
};
BwdPlan bwd_plan(const NormGeom &g, bool gate)
{
    BwdPlan p;
    p.groups = gate ? g.ntokens / g.tokens_per_gate : 1;
    // the blocks an SM holds: one wave, and few partials to add up
    int team, vpt;
    team_shape(g.dim % 4 == 0 ? g.dim / 4 : g.dim, kBwdTeam, &team, &vpt);
    const int per_sm = vpt == 0 ? 4 : team <= 48 ? 16 : (team > 256 ? 2 : 768 / team);
    const int64_t want = (int64_t)device_sm_count() * per_sm;
    const int64_t per = g.ntokens / p.groups;
    p.spans = (want + p.groups - 1) / p.groups;
    // one row an item where there are few, up to four where there are many (an
    // item's partials then cost less than its rows)
    const int64_t rows = per < 128 ? 1 : (per < 256 ? 2 : 4);
    if (p.spans > per / rows)
        p.spans = per / rows;
    p.blocks = p.groups * p.spans;
    if (p.blocks > want)
        p.blocks = want;
    return p;
}

template <typename TI, typename TR, int VEC, int VPT>
cudaError_t bwd_v(const void *y, const void *r, const float *weight, const float *post_weight,
                  const float *gate, const void *dout, const void *dr, void *dy, void *dresidual,
                  float *part, float *dgate_part, const NormGeom &g, const BwdPlan &p, int team,
                  cudaStream_t st)
{
    auto k = VEC == 1 && VPT == 1 && g.dim == 1 ? block_norm_bwd_kernel<TI, TR, VEC, VPT, VEC == 1 && VPT == 1>
                                                : block_norm_bwd_kernel<TI, TR, VEC, VPT, false>;
    const size_t smem = norm_ring<VEC, VPT> ? sizeof(NormSlot<TI, TR, VEC>) * 2 * VPT * team : 0;
    static SmemGrant granted;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(k), smem, &granted);
    if (e != cudaSuccess)
        return e;
    k<<<(unsigned)p.blocks, team, smem, st>>>(
        static_cast<const TI *>(y), static_cast<const TR *>(r), weight, post_weight, gate,
        static_cast<const TI *>(dout), static_cast<const TR *>(dr), static_cast<TI *>(dy),
        static_cast<TR *>(dresidual), part, dgate_part, g, p.groups, p.spans);
    note_launch(1);
    return cudaGetLastError();
}

template <typename TI, typename TR, int VEC>
cudaError_t bwd_wide(const void *y, const void *r, const float *weight, const float *post_weight, const float *gate,
                     const void *dout, const void *dr, void *dy, void *dresidual, float *part, float *dgate_part,
                     const NormGeom &g, const BwdPlan &p, int, cudaStream_t st)
{
    auto k = block_norm_bwd_wide_kernel<TI, TR, VEC>;
    const size_t smem = (size_t)g.dim * sizeof(float);
    static SmemGrant granted;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(k), smem, &granted);
    if (e != cudaSuccess)
        return e;
    k<<<(unsigned)p.blocks, kWideThreads, smem, st>>>(
        static_cast<const TI *>(y), static_cast<const TR *>(r), weight, post_weight, gate,
        static_cast<const TI *>(dout), static_cast<const TR *>(dr), static_cast<TI *>(dy),
        static_cast<TR *>(dresidual), part, dgate_part, g, p.groups, p.spans);
    note_launch(1);
    return cudaGetLastError();
}

// F##_v<TI, TR, VEC, VPT> for the team's vectors per thread, or F##_wide.
#define SSD_NORM_VPT(F, TI, TR, VEC, ...)                                                           \
    (vpt == 1   ? F##_v<TI, TR, VEC, 1>(__VA_ARGS__)                                                \
     : vpt == 2 ? F##_v<TI, TR, VEC, 2>(__VA_ARGS__)                                                \
     : vpt == 4 ? F##_v<TI, TR, VEC, 4>(__VA_ARGS__)                                                \
                : F##_wide<TI, TR, VEC>(__VA_ARGS__))
#define SSD_NORM_TYPES(F, VEC, ...)                                                                 \
    (bf16 ? (res_bf16 ? SSD_NORM_VPT(F, __nv_bfloat16, __nv_bfloat16, VEC, __VA_ARGS__)             \
                      : SSD_NORM_VPT(F, __nv_bfloat16, float, VEC, __VA_ARGS__))                    \
          : SSD_NORM_VPT(F, float, float, VEC, __VA_ARGS__))

}  // namespace

cudaError_t launch_block_norm(const void *y, const void *residual, const float *weight,
                              const float *post_weight, const float *gate, void *out, void *residual_out,
                              const NormGeom &g, bool bf16, bool res_bf16, cudaStream_t st)
{
    if (g.ntokens == 0)
        return cudaSuccess;
    int team, vpt;
    const size_t a = bf16 ? 8 : 16, ar = res_bf16 ? 8 : 16;
    if (g.dim % 4 == 0 && aligned(y, a) && aligned(out, a) && aligned(residual, ar) &&
        aligned(residual_out, ar) && aligned(weight, 16) && aligned(post_weight, 16) && aligned(gate, 16)) {
        team_shape(g.dim / 4, kFwdTeam, &team, &vpt);
        return SSD_NORM_TYPES(fwd, 4, y, residual, weight, post_weight, gate, out, residual_out, g, team,
                              st);
    }
    team_shape(g.dim, kFwdTeam, &team, &vpt);
    return SSD_NORM_TYPES(fwd, 1, y, residual, weight, post_weight, gate, out, residual_out, g, team, st);
}

// Partials: two rows per block (weight, post_weight), one per item of the
// gate where items are parts of a gate row.
size_t block_norm_bwd_workspace(const NormGeom &g, bool gate)
{
    const BwdPlan p = bwd_plan(g, gate);
    return (size_t)(2 * p.blocks + (gate && p.spans > 1 ? p.groups * p.spans : 0)) * (size_t)g.dim * sizeof(float);
}

cudaError_t launch_block_norm_bwd(const void *y, const void *r, const float *weight, const float *post_weight,
                                  const float *gate, const void *dout, const void *dr, void *dy,
                                  void *dresidual, float *dweight, float *dpost_weight, float *dgate,
                                  float *workspace, const NormGeom &g, bool bf16, bool res_bf16,
                                  cudaStream_t st)
{
    const BwdPlan p = bwd_plan(g, gate != nullptr);
    float *part = workspace;
    float *gpart = p.spans > 1 ? workspace + 2 * p.blocks * g.dim : dgate;
    int team, vpt;
    const size_t a = bf16 ? 8 : 16, ar = res_bf16 ? 8 : 16;
    bool al = g.dim % 4 == 0;
    for (const float *q : {weight, post_weight, gate, const_cast<const float *>(dgate), const_cast<const float *>(workspace)})
        al = al && aligned(q, 16);
    for (const void *q : {y, dout, static_cast<const void *>(dy)})
        al = al && aligned(q, a);
    for (const void *q : {r, dr, static_cast<const void *>(dresidual)})
        al = al && aligned(q, ar);
    cudaError_t e;
    if (al) {
        team_shape(g.dim / 4, kBwdTeam, &team, &vpt);
        e = SSD_NORM_TYPES(bwd, 4, y, r, weight, post_weight, gate, dout, dr, dy, dresidual, part, gpart,
                           g, p, team, st);
    } else {
        team_shape(g.dim, kBwdTeam, &team, &vpt);
        e = SSD_NORM_TYPES(bwd, 1, y, r, weight, post_weight, gate, dout, dr, dy, dresidual, part, gpart,
                           g, p, team, st);
    }
    if (e != cudaSuccess)
        return e;
    const bool gate_sums = gate && p.spans > 1;
    const NormSums sums{part, gpart, dweight, dpost_weight, dgate, p.blocks, p.spans, g.dim};
    norm_sums_kernel<<<dim3((unsigned)((g.dim + 31) / 32), (unsigned)(2 + (gate_sums ? p.groups : 0))), dim3(32, 32),
                       0, st>>>(sums);
    note_launch(1);
    return cudaGetLastError();
}

}  // namespace ssd
