// Short causal depthwise convolution with its activation: the step between a
// layer's input projection and its scan.
//
// Per channel c, with x_t = initial state for t < 0 and W = width (2..4):
//     pre[t] = bias + sum_k w[k] x[t - (W-1) + k],   y[t] = silu(pre[t]) or pre[t]
// Backward, with dpre = dy act'(pre) recomputed from x:
//     dx[t] = sum_k w[k] dpre[t + (W-1) - k]  (+ the gradient of the carried rows)
//     dw[k] = sum_t dpre[t] x[t - (W-1) + k],   dbias = sum_t dpre[t]
// Both directions are bound by HBM traffic (one read of x and dy, one write
// of y or dx, about 2 W flops an element): a thread keeps a window of W
// tokens of a few adjacent channels in registers and walks a run of tokens,
// so each element is read once but for the W - 1 tokens before a run.
#include "ssd_internal.h"
#include "vec.cuh"

namespace ssd {
namespace {

constexpr int kConvThreads = 256;
constexpr int kGroup = 4;  // tokens whose loads a thread has in flight

// A thread's VEC x W weights are one run of floats: four at a time where VEC > 1
// (rows then start on 16-byte boundaries).
template <int VEC, int W>
__device__ __forceinline__ void load_weights(const float *__restrict__ w, const float *__restrict__ bias,
                                             int64_t c, float (&wv)[W][VEC], float (&bv)[VEC])
{
    constexpr int NL = VEC > 1 ? 4 : 1;
#pragma unroll
    for (int q = 0; q < VEC * W; q += NL) {
        float v[NL];
        load_vec<float, NL>(w + c * W + q, v);
#pragma unroll
        for (int e = 0; e < NL; ++e)
            wv[(q + e) % W][(q + e) / W] = v[e];
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i)
        bv[i] = bias ? bias[c + i] : 0.f;
}

// One thread: VEC channels of `run` consecutive tokens of one sequence.
template <typename TI, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads)
conv_kernel(const TI *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
            const TI *__restrict__ init, TI *__restrict__ y, TI *__restrict__ fin, ConvGeom g, int run,
            int64_t n_runs)
{
    const int64_t nv = g.dim / VEC;
    const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t r = idx / nv;
    if (r >= g.batch * n_runs)
        return;
    const int64_t c = (idx - r * nv) * VEC;
    const int64_t b = r / n_runs, t0 = (r - b * n_runs) * run;
    float wv[W][VEC], bv[VEC], win[W][VEC];
    load_weights<VEC, W>(w, bias, c, wv, bv);
    const TI *xb = x + b * g.seqlen * g.row + c;
    TI *yb = y + b * g.seqlen * g.dim + c;
    // the W - 1 tokens before the run
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int64_t t = t0 - (W - 1) + k;
        if (t >= 0)
            load_vec<TI, VEC>(xb + t * g.row, win[k]);
        else if (init)
            load_vec<TI, VEC>(init + (b * (W - 1) + (W - 1) + t) * g.dim + c, win[k]);
        else
            for (int i = 0; i < VEC; ++i)
                win[k][i] = 0.f;
    }
    const int64_t t1 = min64(t0 + run, g.seqlen);
    // kGroup tokens' loads are issued before the first is used
    for (int64_t tg = t0; tg < t1; tg += kGroup) {
        typename Pack<TI, VEC>::T raw[kGroup];
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            if (tg + j < t1)
                raw[j] = *reinterpret_cast<const typename Pack<TI, VEC>::T *>(xb + (tg + j) * g.row);
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
            if (tg + j >= t1)
                break;
            unpack<TI, VEC>(raw[j], win[W - 1]);
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float s = bv[i];
#pragma unroll
                for (int k = 0; k < W; ++k)
                    s = fmaf(wv[k][i], win[k][i], s);
                o[i] = g.silu ? fast_silu(s) : s;
#pragma unroll
                for (int k = 0; k < W - 1; ++k)
                    win[k][i] = win[k + 1][i];
            }
            store_vec<TI, VEC>(yb + (tg + j) * g.dim, o);
        }
    }
    if (fin && t1 == g.seqlen)
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            store_vec<TI, VEC>(fin + (b * (W - 1) + k) * g.dim + c, win[k]);
}

// One token of every sequence; state and state_out may be one buffer.
template <typename TI, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads)
conv_step_kernel(const TI *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
                 const TI *state, TI *state_out, TI *__restrict__ y, ConvGeom g)
{
    const int64_t nv = g.dim / VEC;
    const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t b = idx / nv;
    if (b >= g.batch)
        return;
    const int64_t c = (idx - b * nv) * VEC;
    float wv[W][VEC], bv[VEC], win[W][VEC], o[VEC];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        load_vec<TI, VEC>(state + (b * (W - 1) + k) * g.dim + c, win[k]);
    load_vec<TI, VEC>(x + b * g.row + c, win[W - 1]);
    load_weights<VEC, W>(w, bias, c, wv, bv);
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
        float s = bv[i];
#pragma unroll
        for (int k = 0; k < W; ++k)
            s = fmaf(wv[k][i], win[k][i], s);
        o[i] = g.silu ? fast_silu(s) : s;
    }
    store_vec<TI, VEC>(y + b * g.dim + c, o);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        store_vec<TI, VEC>(state_out + (b * (W - 1) + k) * g.dim + c, win[k + 1]);
}

// Backward.  With xf = (initial state | x), L + W - 1 rows, pre[i] reads
// xf[i .. i + W - 1] and xf[e] receives sum_k w[k] dpre[e - k] (dpre = 0
// outside [0, L)).  A thread owns rows [e0, e0 + run) of xf: it walks i from
// e0 - (W - 1), keeping the last W values of xf and of dpre, and sums the
// weight gradient over its own i.  Eight such runs share a block's channels;
// their weight gradients are added in shared memory and written as one
// partial per block: part[p][k][c], k = W for the bias.
constexpr int kBwdCols = 32, kBwdRuns = 8;

template <typename TI, int VEC, int W>
__global__ void __launch_bounds__(kBwdCols *kBwdRuns)
conv_bwd_kernel(const TI *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
                const TI *__restrict__ init, const TI *__restrict__ dy, const TI *__restrict__ dfinal,
                TI *__restrict__ dx, TI *__restrict__ dinit, float *__restrict__ part, ConvGeom g, int run,
                int64_t parts_per_seq)
{
    __shared__ float red[kBwdRuns][kBwdCols][VEC];
    const int64_t c = ((int64_t)blockIdx.x * kBwdCols + threadIdx.x) * VEC;
    const int64_t b = blockIdx.y / parts_per_seq;
    const int64_t e0 = ((blockIdx.y - b * parts_per_seq) * kBwdRuns + threadIdx.y) * run;
    const int64_t L = g.seqlen;
    const bool live = c < g.dim;
    float dw[W + 1][VEC];
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            dw[k][i] = 0.f;
    if (live && e0 < L + W - 1) {
        float wv[W][VEC], bv[VEC], win[W][VEC], dp[W][VEC];
        load_weights<VEC, W>(w, bias, c, wv, bv);
        const TI *xb = x + b * L * g.row + c;
        const TI *dyb = dy + b * L * g.row_dy + c;
        TI *dxb = dx + b * L * g.dim + c;
        auto load_xf = [&](int64_t e, float (&v)[VEC]) {
            const int64_t t = e - (W - 1);
            if (t >= 0 && t < L)
                load_vec<TI, VEC>(xb + t * g.row, v);
            else if (t < 0 && e >= 0 && init)
                load_vec<TI, VEC>(init + (b * (W - 1) + e) * g.dim + c, v);
            else
#pragma unroll
                for (int i = 0; i < VEC; ++i)
                    v[i] = 0.f;
        };
#pragma unroll
        for (int k = 0; k < W; ++k) {
#pragma unroll
            for (int i = 0; i < VEC; ++i)
                dp[k][i] = 0.f;
            if (k < W - 1)
                load_xf(e0 - (W - 1) + k, win[k]);
        }
        const int64_t e1 = min64(e0 + run, L + W - 1);
        for (int64_t eg = e0 - (W - 1); eg < e1; eg += kGroup) {
            using V = typename Pack<TI, VEC>::T;
            V xr[kGroup], yr[kGroup];
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                const int64_t e = eg + j;
                xr[j] = yr[j] = V{};
                if (e < e1) {
                    if (e >= 0 && e < L) {  // xf[e + W - 1] is x[e]
                        xr[j] = *reinterpret_cast<const V *>(xb + e * g.row);
                        yr[j] = *reinterpret_cast<const V *>(dyb + e * g.row_dy);
                    } else if (e < 0 && e + W - 1 >= 0 && init) {
                        xr[j] = *reinterpret_cast<const V *>(init + (b * (W - 1) + e + W - 1) * g.dim + c);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                const int64_t e = eg + j;
                if (e >= e1)
                    break;
                unpack<TI, VEC>(xr[j], win[W - 1]);
                // dp[0] is dpre[e], dp[k] = dpre[e - k]; zero outside [0, L)
                float d[VEC];
                unpack<TI, VEC>(yr[j], d);
                const bool in = e >= 0 && e < L;
                if (g.silu) {
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        float s = bv[i];
#pragma unroll
                        for (int k = 0; k < W; ++k)
                            s = fmaf(wv[k][i], win[k][i], s);
                        d[i] = in ? d[i] * silu_grad(s, fast_sigmoid(s)) : 0.f;
                    }
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
#pragma unroll
                    for (int k = W - 1; k > 0; --k)
                        dp[k][i] = dp[k - 1][i];
                    dp[0][i] = d[i];
                }
                if (e >= e0) {
                    float o[VEC];
#pragma unroll
                    for (int i = 0; i < VEC; ++i) {
                        float s = 0.f;
#pragma unroll
                        for (int k = 0; k < W; ++k) {
                            s = fmaf(wv[k][i], dp[k][i], s);
                            if (in)
                                dw[k][i] = fmaf(d[i], win[k][i], dw[k][i]);
                        }
                        dw[W][i] += d[i];
                        o[i] = s;
                    }
                    const int64_t t = e - (W - 1);
                    if (dfinal && e >= L) {  // the carried rows are the last W - 1 of xf
                        float f[VEC];
                        load_vec<TI, VEC>(dfinal + (b * (W - 1) + e - L) * g.dim + c, f);
#pragma unroll
                        for (int i = 0; i < VEC; ++i)
                            o[i] += f[i];
                    }
                    if (t >= 0)
                        store_vec<TI, VEC>(dxb + t * g.dim, o);
                    else if (dinit)
                        store_vec<TI, VEC>(dinit + (b * (W - 1) + e) * g.dim + c, o);
                }
#pragma unroll
                for (int i = 0; i < VEC; ++i)
#pragma unroll
                    for (int k = 0; k < W - 1; ++k)
                        win[k][i] = win[k + 1][i];
            }
        }
    }
#pragma unroll
    for (int k = 0; k <= W; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < VEC; ++i)
            red[threadIdx.y][threadIdx.x][i] = dw[k][i];
        __syncthreads();
        if (threadIdx.y == 0 && live)
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
                float s = 0.f;
#pragma unroll
                for (int q = 0; q < kBwdRuns; ++q)
                    s += red[q][threadIdx.x][i];
                part[((int64_t)blockIdx.y * (W + 1) + k) * g.dim + c + i] = s;
            }
    }
}

// Sums the partials in a fixed order: dweight[c][k], dbias[c].
__global__ void __launch_bounds__(256) conv_bwd_reduce_kernel(const float *__restrict__ part, int64_t n_parts,
                                                              int64_t dim, int W, float *__restrict__ dw,
                                                              float *__restrict__ dbias)
{
    __shared__ float red[8][32];
    const int64_t c = (int64_t)blockIdx.x * 32 + threadIdx.x;
    const int k = blockIdx.y;
    float s = 0.f;
    if (c < dim)
        for (int64_t p = threadIdx.y; p < n_parts; p += 8)
            s += part[(p * (W + 1) + k) * dim + c];
    red[threadIdx.y][threadIdx.x] = s;
    __syncthreads();
    if (threadIdx.y == 0 && c < dim) {
        s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q)
            s += red[q][threadIdx.x];
        if (k < W)
            dw[c * W + k] = s;
        else if (dbias)
            dbias[c] = s;
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Tokens a forward thread walks: long runs re-read fewer tokens, short ones
// keep the GPU filled when the call is small.
int conv_run(const ConvGeom &g, int vec)
{
    const int64_t threads = g.batch * (g.dim / vec);
    const int64_t want = (int64_t)device_sm_count() * 1024;
    int run = 32;
    while (run > 4 && threads * ((g.seqlen + run - 1) / run) < want)
        run /= 2;
    return run;
}

int64_t conv_bwd_parts_per_seq(const ConvGeom &g, int run)
{
    return (g.seqlen + g.width - 1 + (int64_t)kBwdRuns * run - 1) / ((int64_t)kBwdRuns * run);
}

// Tokens a backward thread walks, eight such runs in a block.
int conv_bwd_run(const ConvGeom &g, int vec)
{
    const int64_t cols = (g.dim / vec + kBwdCols - 1) / kBwdCols;
    const int64_t want = (int64_t)device_sm_count() * 4;
    int run = 32;
    while (run > 4 && cols * g.batch * ((g.seqlen + g.width - 1 + 8 * run - 1) / (8 * run)) < want)
        run /= 2;
    while (conv_bwd_parts_per_seq(g, run) * g.batch > 65535)  // one grid row each
        run *= 2;
    return run;
}

template <typename TI, int VEC, int W>
cudaError_t fwd_w(const void *x, const float *w, const float *bias, const void *init, void *y, void *fin,
                  const ConvGeom &g, cudaStream_t st)
{
    const int run = conv_run(g, VEC);
    const int64_t n_runs = (g.seqlen + run - 1) / run;
    const int64_t threads = g.batch * n_runs * (g.dim / VEC);
    conv_kernel<TI, VEC, W><<<(unsigned)((threads + kConvThreads - 1) / kConvThreads), kConvThreads, 0, st>>>(
        static_cast<const TI *>(x), w, bias, static_cast<const TI *>(init), static_cast<TI *>(y),
        static_cast<TI *>(fin), g, run, n_runs);
    note_launch(1);
    return cudaGetLastError();
}
template <typename TI, int VEC, int W>
cudaError_t step_w(const void *x, const float *w, const float *bias, const void *state, void *state_out,
                   void *y, const ConvGeom &g, cudaStream_t st)
{
    const int64_t threads = g.batch * (g.dim / VEC);
    conv_step_kernel<TI, VEC, W>
        <<<(unsigned)((threads + kConvThreads - 1) / kConvThreads), kConvThreads, 0, st>>>(
            static_cast<const TI *>(x), w, bias, static_cast<const TI *>(state), static_cast<TI *>(state_out),
            static_cast<TI *>(y), g);
    note_launch(1);
    return cudaGetLastError();
}
template <typename TI, int VEC, int W>
cudaError_t bwd_w(const void *x, const float *w, const float *bias, const void *init, const void *dy,
                  const void *dfinal, void *dx, float *dw, float *dbias, void *dinit, float *part,
                  const ConvGeom &g, int run, cudaStream_t st)
{
    const int64_t pps = conv_bwd_parts_per_seq(g, run);
    const dim3 grid((unsigned)((g.dim / VEC + kBwdCols - 1) / kBwdCols), (unsigned)(pps * g.batch));
    conv_bwd_kernel<TI, VEC, W><<<grid, dim3(kBwdCols, kBwdRuns), 0, st>>>(
        static_cast<const TI *>(x), w, bias, static_cast<const TI *>(init), static_cast<const TI *>(dy),
        static_cast<const TI *>(dfinal), static_cast<TI *>(dx), static_cast<TI *>(dinit), part, g, run, pps);
    note_launch(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    conv_bwd_reduce_kernel<<<dim3((unsigned)((g.dim + 31) / 32), W + 1), dim3(32, 8), 0, st>>>(
        part, pps * g.batch, g.dim, W, dw, dbias);
    note_launch(1);
    return cudaGetLastError();
}

// F<TI, VEC, W>: VEC channels by vector accesses where rows allow it.
#define SSD_CONV_WIDTHS(F, TI, VEC, ...)                                                            \
    (g.width == 2 ? F<TI, VEC, 2>(__VA_ARGS__)                                                      \
                  : (g.width == 3 ? F<TI, VEC, 3>(__VA_ARGS__) : F<TI, VEC, 4>(__VA_ARGS__)))

}  // namespace

cudaError_t launch_conv(const void *x, const float *w, const float *bias, const void *init, void *y,
                        void *fin, const ConvGeom &g, bool bf16, cudaStream_t st)
{
    const bool al = aligned(x, 16) && aligned(init, 16) && aligned(y, 16) && aligned(fin, 16) && aligned(w, 16);
    if (bf16) {
        if (al && g.dim % 8 == 0 && g.row % 8 == 0)
            return SSD_CONV_WIDTHS(fwd_w, __nv_bfloat16, 8, x, w, bias, init, y, fin, g, st);
        return SSD_CONV_WIDTHS(fwd_w, __nv_bfloat16, 1, x, w, bias, init, y, fin, g, st);
    }
    if (al && g.dim % 4 == 0 && g.row % 4 == 0)
        return SSD_CONV_WIDTHS(fwd_w, float, 4, x, w, bias, init, y, fin, g, st);
    return SSD_CONV_WIDTHS(fwd_w, float, 1, x, w, bias, init, y, fin, g, st);
}

cudaError_t launch_conv_step(const void *x, const float *w, const float *bias, const void *state,
                             void *state_out, void *y, const ConvGeom &g, bool bf16, cudaStream_t st)
{
    const size_t a = bf16 ? 8 : 16;
    const bool al = aligned(x, a) && aligned(state, a) && aligned(state_out, a) && aligned(y, a) &&
                    aligned(w, 16) && g.dim % 4 == 0 && g.row % 4 == 0;
    if (bf16) {
        if (al)
            return SSD_CONV_WIDTHS(step_w, __nv_bfloat16, 4, x, w, bias, state, state_out, y, g, st);
        return SSD_CONV_WIDTHS(step_w, __nv_bfloat16, 1, x, w, bias, state, state_out, y, g, st);
    }
    if (al)
        return SSD_CONV_WIDTHS(step_w, float, 4, x, w, bias, state, state_out, y, g, st);
    return SSD_CONV_WIDTHS(step_w, float, 1, x, w, bias, state, state_out, y, g, st);
}

// Room for the partials of either vector width (alignment is not known here).
size_t conv_bwd_workspace(const ConvGeom &g)
{
    int64_t parts = 0;
    for (int vec : {4, 1}) {
        const int64_t p = conv_bwd_parts_per_seq(g, conv_bwd_run(g, vec)) * g.batch;
        parts = p > parts ? p : parts;
    }
    return (size_t)(parts * (g.width + 1) * g.dim) * sizeof(float);
}

cudaError_t launch_conv_bwd(const void *x, const float *w, const float *bias, const void *init,
                            const void *dy, const void *dfinal, void *dx, float *dw, float *dbias,
                            void *dinit, float *part, const ConvGeom &g, bool bf16, cudaStream_t st)
{
    const size_t a = bf16 ? 8 : 16;
    bool al = g.dim % 4 == 0 && g.row % 4 == 0 && g.row_dy % 4 == 0 && aligned(w, 16);
    for (const void *p : {x, init, dy, dfinal, static_cast<const void *>(dx), static_cast<const void *>(dinit)})
        al = al && aligned(p, a);
    const int run = conv_bwd_run(g, al ? 4 : 1);
    if (bf16) {
        if (al)
            return SSD_CONV_WIDTHS(bwd_w, __nv_bfloat16, 4, x, w, bias, init, dy, dfinal, dx, dw, dbias,
                                   dinit, part, g, run, st);
        return SSD_CONV_WIDTHS(bwd_w, __nv_bfloat16, 1, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit,
                               part, g, run, st);
    }
    if (al)
        return SSD_CONV_WIDTHS(bwd_w, float, 4, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit, part, g,
                               run, st);
    return SSD_CONV_WIDTHS(bwd_w, float, 1, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit, part, g, run,
                           st);
}

}  // namespace ssd
