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
// Both directions are bound by HBM traffic.  A team of threads holds a row in
// registers from its one read to its one write; the row sums are the only
// communication (shuffles, and shared memory between a team's warps).
// Statistics and sums are f32; r is kept in f32 for `out` and rounded once to
// the residual's type where it is stored.
#include "ssd_internal.h"
#include "vec.cuh"

namespace ssd {
namespace {

// Threads of a row's team at most.  The backward's fewer leave registers for
// two blocks an SM (a row's four inputs, the next row's, and three sums).
constexpr int kFwdTeam = 512, kBwdTeam = 320;

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
#pragma unroll
    for (int k = 0; k < K; ++k)
        v[k] = 0.f;
    for (int q = 0; q < warps; ++q) {
        const Sum<K> t = s[q];
#pragma unroll
        for (int k = 0; k < K; ++k)
            v[k] += t.v[k];
    }
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
    __shared__ Sum<1> sum_y[16], sum_r[16];
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

// v - x m, the part of a row's gradient across the row's direction.  In a row
// of one channel the two terms differ by the eps term alone (the gradient is
// all radial), which their difference in f32 would lose: there it is v eps rs^2.
__device__ __forceinline__ float minus_radial(float v, float x, float m, float rs, const NormGeom &g)
{
    return g.dim == 1 ? v * (g.eps * rs * rs) : fmaf(-x, m, v);
}

// Backward.  A block walks the rows of its items one after another; an item
// is one of `spans` runs of the tokens of one gate row (or of all tokens).
// The parameters' gradients stay in the thread that owns the channels: the
// weights' over all its rows (one partial per block: part[block][0] is
// weight, [1] post_weight), the gate's over an item (written as it is where
// an item is a whole gate row, else one partial per item).
template <typename TI, typename TR, int VEC, int VPT>
__global__ void __launch_bounds__(kBwdTeam, VEC * VPT <= 8 ? 2 : 1)
block_norm_bwd_kernel(const TI *__restrict__ y, const TR *__restrict__ r, const float *__restrict__ weight,
                      const float *__restrict__ post_weight, const float *__restrict__ gate,
                      const TI *__restrict__ dout, const TR *dr, TI *__restrict__ dy, TR *dresidual,
                      float *__restrict__ part, float *__restrict__ dgate_part, NormGeom g, int64_t groups,
                      int64_t spans)
{
    __shared__ Sum<3> sum_row[2][16];
    __shared__ Sum<1> sum_p[16];
    int flip = 0;
    const int team = blockDim.x;
    const int nv = (int)(g.dim / VEC);
    float dw[VPT][VEC], dpw[VPT][VEC], dg[VPT][VEC];
#pragma unroll
    for (int q = 0; q < VPT; ++q)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            dw[q][i] = dpw[q][i] = 0.f;
    const int64_t tokens = g.ntokens / groups;
    for (int64_t item = blockIdx.x; item < groups * spans; item += gridDim.x) {
        const int64_t j = item / spans, sp = item - j * spans;
        const int64_t t0 = j * tokens + tokens * sp / spans, t1 = j * tokens + tokens * (sp + 1) / spans;
#pragma unroll
        for (int q = 0; q < VPT; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                dg[q][i] = 0.f;
        using VI = typename Pack<TI, VEC>::T;
        using VR = typename Pack<TR, VEC>::T;
        VI y_raw[VPT], n_raw[VPT];
        VR r_raw[VPT], d_raw[VPT];
        auto fetch = [&](int64_t row) {
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                const int v = threadIdx.x + q * team;
                y_raw[q] = n_raw[q] = VI{};
                r_raw[q] = d_raw[q] = VR{};
                if (v < nv) {
                    const int64_t at = row * g.dim + v * VEC;
                    y_raw[q] = *reinterpret_cast<const VI *>(y + at);
                    r_raw[q] = *reinterpret_cast<const VR *>(r + at);
                    n_raw[q] = *reinterpret_cast<const VI *>(dout + at);
                    if (dr)
                        d_raw[q] = *reinterpret_cast<const VR *>(dr + at);
                }
            }
        };
        if (t0 < t1)
            fetch(t0);
        for (int64_t row = t0; row < t1; ++row) {
            float yv[VPT][VEC], rv[VPT][VEC], gn[VPT][VEC], gr[VPT][VEC];
            float s[3] = {0.f, 0.f, 0.f};
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                unpack<TI, VEC>(y_raw[q], yv[q]);
                unpack<TR, VEC>(r_raw[q], rv[q]);
                unpack<TI, VEC>(n_raw[q], gn[q]);
                unpack<TR, VEC>(d_raw[q], gr[q]);
            }
            if (row + 1 < t1)  // in flight while this row is reduced
                fetch(row + 1);
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                const int v = threadIdx.x + q * team;
                float w[VEC] = {};
                if (v < nv)
                    load_vec<float, VEC>(weight + v * VEC, w);
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    s[0] = fmaf(yv[q][i], yv[q][i], s[0]);
                    s[1] = fmaf(rv[q][i], rv[q][i], s[1]);
                    s[2] = fmaf(gn[q][i] * w[i], rv[q][i], s[2]);
                }
            }
            team_sum<3>(s, sum_row[flip]);
            flip ^= 1;
            const float rs_y = post_weight ? rsqrtf(s[0] * g.inv_dim + g.eps) : 1.f;
            const float rs_r = rsqrtf(s[1] * g.inv_dim + g.eps);
            const float c = s[2] * g.inv_dim * rs_r * rs_r;  // mean(gn rh) rs_r
            float u[1] = {0.f};
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                const int v = threadIdx.x + q * team;
                if (v < nv) {
                    float w[VEC], pw[VEC], k[VEC];
                    load_vec<float, VEC>(weight + v * VEC, w);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        dw[q][i] = fmaf(gn[q][i], rv[q][i] * rs_r, dw[q][i]);
                        gr[q][i] += rs_r * minus_radial(gn[q][i] * w[i], rv[q][i], c, rs_r, g);
                        pw[i] = 1.f;
                        k[i] = g.scale;
                    }
                    store_vec<TR, VEC>(dresidual + row * g.dim + v * VEC, gr[q]);
                    if (post_weight)
                        load_vec<float, VEC>(post_weight + v * VEC, pw);
                    if (gate)
                        scale_by<VEC>(gate + j * g.dim + v * VEC, k);
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        const float yh = yv[q][i] * rs_y;
                        dg[q][i] = fmaf(gr[q][i], yh * pw[i], dg[q][i]);
                        const float dp = k[i] * gr[q][i];
                        dpw[q][i] = fmaf(dp, yh, dpw[q][i]);
                        gr[q][i] = dp * pw[i];
                        yv[q][i] = yh;
                        u[0] = fmaf(gr[q][i], yh, u[0]);
                    }
                }
            }
            float m = 0.f;
            if (post_weight) {
                team_sum<1>(u, sum_p);
                m = u[0] * g.inv_dim;
            }
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                const int v = threadIdx.x + q * team;
                if (v < nv) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        gr[q][i] = post_weight ? rs_y * minus_radial(gr[q][i], yv[q][i], m, rs_y, g) : gr[q][i];
                    store_vec<TI, VEC>(dy + row * g.dim + v * VEC, gr[q]);
                }
            }
        }
        if (gate)
#pragma unroll
            for (int q = 0; q < VPT; ++q) {
                const int v = threadIdx.x + q * team;
                if (v < nv)
#pragma unroll
                    for (int i = 0; i < VEC; ++i)
                        dgate_part[item * g.dim + v * VEC + i] = g.scale * dg[q][i];
            }
    }
#pragma unroll
    for (int q = 0; q < VPT; ++q) {
        const int v = threadIdx.x + q * team;
        if (v < nv) {
            store_vec<float, VEC>(part + ((int64_t)blockIdx.x * 2) * g.dim + v * VEC, dw[q]);
            store_vec<float, VEC>(part + ((int64_t)blockIdx.x * 2 + 1) * g.dim + v * VEC, dpw[q]);
        }
    }
}

// out[row][c] = sum over n of src[(row * n_stride_row + p * stride) + c], in a
// fixed order; blockDim = (32, 8).
__global__ void __launch_bounds__(256) sum_rows_kernel(const float *__restrict__ src, int64_t n, int64_t stride,
                                                       int64_t row_stride, int64_t dim, float *__restrict__ out)
{
    __shared__ float red[8][32];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const float *p0 = src + (int64_t)blockIdx.y * row_stride + c;
    float s = 0.f;
    if (c < dim)
        for (int64_t p = threadIdx.y; p < n; p += 8)
            s += p0[p * stride];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            s += red[q][threadIdx.x];
        out[(int64_t)blockIdx.y * dim + c] = s;
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Threads of a row's team, and vectors of each, for a row of nv vectors: few
// vectors a thread while the team stays within `most` threads.
void team_shape(int64_t nv, int most, int *team, int *vpt)
{
    for (int v : {1, 2, 4, 8, 32, 128}) {
        *vpt = v;
        *team = (int)((nv + v * 32 - 1) / (v * 32)) * 32;
        if (*team <= most)
            return;
    }
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
    const int64_t want = (int64_t)device_sm_count() * 4;
    const int64_t per = g.ntokens / p.groups;
    p.spans = (want + p.groups - 1) / p.groups;
    if (p.spans > per)
        p.spans = per;
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
    block_norm_bwd_kernel<TI, TR, VEC, VPT><<<(unsigned)p.blocks, team, 0, st>>>(
        static_cast<const TI *>(y), static_cast<const TR *>(r), weight, post_weight, gate,
        static_cast<const TI *>(dout), static_cast<const TR *>(dr), static_cast<TI *>(dy),
        static_cast<TR *>(dresidual), part, dgate_part, g, p.groups, p.spans);
    note_launch(1);
    return cudaGetLastError();
}

// F<TI, TR, VEC, VPT> for the team's vectors per thread; MAXV: the most (a
// row of four-channel vectors needs 32, one of single channels 128).
#define SSD_NORM_VPT(F, TI, TR, VEC, MAXV, ...)                                                     \
    (vpt == 1    ? F<TI, TR, VEC, 1>(__VA_ARGS__)                                                   \
     : vpt == 2  ? F<TI, TR, VEC, 2>(__VA_ARGS__)                                                   \
     : vpt == 4  ? F<TI, TR, VEC, 4>(__VA_ARGS__)                                                   \
     : vpt == 8  ? F<TI, TR, VEC, 8>(__VA_ARGS__)                                                   \
     : vpt == 32 ? F<TI, TR, VEC, 32>(__VA_ARGS__)                                                  \
                 : F<TI, TR, VEC, MAXV>(__VA_ARGS__))
#define SSD_NORM_TYPES(F, VEC, MAXV, ...)                                                           \
    (bf16 ? (res_bf16 ? SSD_NORM_VPT(F, __nv_bfloat16, __nv_bfloat16, VEC, MAXV, __VA_ARGS__)       \
                      : SSD_NORM_VPT(F, __nv_bfloat16, float, VEC, MAXV, __VA_ARGS__))              \
          : SSD_NORM_VPT(F, float, float, VEC, MAXV, __VA_ARGS__))

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
        return SSD_NORM_TYPES(fwd_v, 4, 32, y, residual, weight, post_weight, gate, out, residual_out, g, team,
                              st);
    }
    team_shape(g.dim, kFwdTeam, &team, &vpt);
    return SSD_NORM_TYPES(fwd_v, 1, 128, y, residual, weight, post_weight, gate, out, residual_out, g, team, st);
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
        e = SSD_NORM_TYPES(bwd_v, 4, 32, y, r, weight, post_weight, gate, dout, dr, dy, dresidual, part, gpart,
                           g, p, team, st);
    } else {
        team_shape(g.dim, kBwdTeam, &team, &vpt);
        e = SSD_NORM_TYPES(bwd_v, 1, 128, y, r, weight, post_weight, gate, dout, dr, dy, dresidual, part, gpart,
                           g, p, team, st);
    }
    if (e != cudaSuccess)
        return e;
    const unsigned cols = (unsigned)((g.dim + 31) / 32);
    sum_rows_kernel<<<dim3(cols, 1), dim3(32, 8), 0, st>>>(part, p.blocks, 2 * g.dim, 0, g.dim, dweight);
    note_launch(1);
    if (dpost_weight) {
        sum_rows_kernel<<<dim3(cols, 1), dim3(32, 8), 0, st>>>(part + g.dim, p.blocks, 2 * g.dim, 0, g.dim,
                                                               dpost_weight);
        note_launch(1);
    }
    if (gate && p.spans > 1) {
        sum_rows_kernel<<<dim3(cols, (unsigned)p.groups), dim3(32, 8), 0, st>>>(gpart, p.spans, g.dim,
                                                                               p.spans * g.dim, g.dim, dgate);
        note_launch(1);
    }
    return cudaGetLastError();
}

}  // namespace ssd
