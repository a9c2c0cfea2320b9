// Short causal depthwise convolution with its activation: the step between a
// layer's input projection and its scan.
//
// Per channel c, with x_t = initial state for t < 0 and W = width (2..4):
//     pre[t] = bias + sum_k w[k] x[t - (W-1) + k],   y[t] = silu(pre[t]) or pre[t]
// Backward, with dpre = dy act'(pre) recomputed from x:
//     dx[t] = sum_k w[k] dpre[t + (W-1) - k]  (+ the gradient of the carried rows)
//     dw[k] = sum_t dpre[t] x[t - (W-1) + k],   dbias = sum_t dpre[t]
// Both directions should be bound by HBM traffic (one read of x and dy, one
// write of y or dx): a thread keeps a window of W tokens of four adjacent
// channels in registers as f32 pairs and walks a run of tokens, so each element
// is read once but for the W - 1 tokens before a run; its inputs come through
// a ring of asynchronous copies, as loads ahead of time in registers left too
// few threads to cover HBM's latency.  On a GB300, 4 x 4096 tokens of 5376
// bf16 channels, W = 4 (DRAM traffic as computed, nothing read twice):
//     forward   64 us, 5.5 TB/s (82% of the measured copy rate)
//     backward 115 us, 4.6 TB/s (68%); 25 instructions an element by 2.8 warps
//              a scheduler (154 registers), which is too few: half of the issue
//              slots are empty, and of the 5.6 cycles a warp takes for an
//              instruction 1.5 wait for the one before, 0.7 for memory and 0.7
//              for the f32 pipe
#include "ssd_internal.h"
#include "vec.cuh"

namespace ssd {
namespace {

constexpr int kConvThreads = 256, kConvBlocks = 3;  // blocks an SM holds

// A thread's VEC channels (VEC even, or one) as f32 pairs; with one channel
// the second of the pair is unused.
template <int VEC> constexpr int kPairs = (VEC + 1) / 2;
template <typename TI, int VEC> using RawV = typename Pack<TI, VEC>::T;

template <typename TI, int VEC> __device__ __forceinline__ void to_pairs(const RawV<TI, VEC> &r, f32x2 (&p)[kPairs<VEC>])
{
    float v[VEC];
    unpack<TI, VEC>(r, v);
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i)
        p[i] = pk2(v[2 * i], 2 * i + 1 < VEC ? v[(2 * i + 1) % VEC] : 0.f);
}
// A thread's VEC channels are S apart: adjacent (S = 1, one access), or a warp
// apart (S = 32, rows off vector boundaries; accesses of single elements, which
// a warp's threads make side by side).
template <typename TI, int VEC, int S = 1> __device__ __forceinline__ void store_pairs(TI *p, const f32x2 (&o)[kPairs<VEC>])
{
    float v[VEC];
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) {
        float x, y;
        un2(o[i], x, y);
        v[2 * i] = x;
        if (2 * i + 1 < VEC)
            v[(2 * i + 1) % VEC] = y;
    }
    if constexpr (S == 1) {
        store_vec<TI, VEC>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            p[e * S] = from_f32<TI>(v[e]);
    }
}
template <typename TI, int VEC, int S = 1> __device__ __forceinline__ RawV<TI, VEC> load_raw(const TI *p)
{
    RawV<TI, VEC> r;
    if constexpr (S == 1)
        r = *reinterpret_cast<const RawV<TI, VEC> *>(p);
    else
#pragma unroll
        for (int e = 0; e < VEC; ++e)
            reinterpret_cast<TI *>(&r)[e] = p[e * S];
    return r;
}

template <typename TI, int VEC, int S> __device__ __forceinline__ RawV<TI, VEC> load_or_zero(const TI *p)
{
    RawV<TI, VEC> v{};
    if (p) {
        if constexpr (S == 1)
            v = load_ahead_as<RawV<TI, VEC>>(p);
        else
#pragma unroll
            for (int e = 0; e < VEC; ++e)
                reinterpret_cast<TI *>(&v)[e] = load_ahead_as<TI>(p + e * S);
    }
    return v;
}

// Threads that hold a row's channels, and the first channel of thread v.  Where
// channels are a warp apart, the last warp's begin early enough to end with the
// row (dim >= VEC S): the channels it shares with its neighbour are computed
// twice, to the same values.
template <int VEC, int S> __host__ __device__ __forceinline__ int64_t conv_columns(int64_t dim)
{
    return S == 1 ? dim / VEC : (dim + VEC * S - 1) / (VEC * S) * S;
}
template <int VEC, int S> __device__ __forceinline__ int64_t first_channel(int64_t v, int64_t dim)
{
    return S == 1 ? v * VEC : min64(v / S * (VEC * S), dim - VEC * S) + v % S;
}

// A channel's W weights are one run of floats, adjacent channels' too: two at a
// time where VEC channels start on 8-byte boundaries.
template <int VEC, int S, int W>
__device__ __forceinline__ void load_weights(const float *__restrict__ w, const float *__restrict__ bias,
                                             int64_t c, f32x2 (&wv)[W][kPairs<VEC>], f32x2 (&bv)[kPairs<VEC>])
{
    constexpr int NL = VEC > 1 && S == 1 ? 2 : 1;
    float t[kPairs<VEC> * 2 * W] = {};
#pragma unroll
    for (int q = 0; q < VEC * W; q += NL) {
        float v[NL];
        load_vec<float, NL>(w + (c + q / W * (S - 1)) * W + q, v);
#pragma unroll
        for (int e = 0; e < NL; ++e)
            t[q + e] = v[e];
    }
#pragma unroll
    for (int i = 0; i < kPairs<VEC>; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k)
            wv[k][i] = pk2(t[2 * i * W + k], t[(2 * i + 1) * W + k]);
        bv[i] = bias ? pk2(bias[c + 2 * i * S], 2 * i + 1 < VEC ? bias[c + (2 * i + 1) * S] : 0.f) : 0;
    }
}

// A thread's own ring of groups in shared memory: the copies of the groups
// ahead are in flight without holding registers, and as a thread reads only
// what it copied itself, no barrier is needed.  (Two-byte elements, one
// channel a thread, are too small to copy: they are loaded into registers a
// group ahead.)
constexpr int kGroup = 4;   // tokens of a group
constexpr int kStages = 4;  // groups in flight
template <typename TI, int VEC, int S, int TENSORS, int NT> struct Ring {
    static constexpr bool kAsync = S == 1 && sizeof(RawV<TI, VEC>) >= 4;
    static constexpr size_t kBytes = kAsync ? sizeof(RawV<TI, VEC>) * kGroup * kStages * TENSORS * NT : 0;
    const TI *p[TENSORS];   // the next group to copy
    int64_t row[TENSORS];
    int ahead = 0, left;    // groups copied and not yet taken; groups still to copy
    int slot_in = 0, slot_out = 0;
    RawV<TI, VEC> *buf;     // [stage][tensor][token][thread]
    TI next[TENSORS][kAsync ? 1 : kGroup][VEC];

    __device__ __forceinline__ RawV<TI, VEC> *at(int slot, int k, int j)
    {
        return buf + ((slot * TENSORS + k) * kGroup + j) * NT;
    }
    __device__ __forceinline__ void push()
    {
        if (left > 0) {
#pragma unroll
            for (int k = 0; k < TENSORS; ++k) {
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    copy_async<sizeof(RawV<TI, VEC>) < 4 ? 4 : sizeof(RawV<TI, VEC>)>(at(slot_in, k, j),
                                                                                   p[k] + j * row[k]);
                p[k] += kGroup * row[k];
            }
            --left;
        }
        copy_async_commit();  // a group for every push, so that the waits count alike
        slot_in = slot_in + 1 == kStages ? 0 : slot_in + 1;
    }
    __device__ __forceinline__ void start(void *smem, int thread, int groups)
    {
        left = groups;
        buf = static_cast<RawV<TI, VEC> *>(smem) + thread;
        if constexpr (kAsync)
            for (int i = 0; i < kStages - 1; ++i)
                push();
        else
            load_next();
    }
    __device__ __forceinline__ void load_next()
    {
        if (left > 0) {
#pragma unroll
            for (int k = 0; k < TENSORS; ++k) {
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        next[k][j][e] = load_ahead_as<TI>(p[k] + j * row[k] + e * S);
                p[k] += kGroup * row[k];
            }
            --left;
        }
    }
    __device__ __forceinline__ void take(RawV<TI, VEC> (&v)[TENSORS][kGroup])
    {
        if constexpr (kAsync) {
            push();
            copy_async_wait<kStages - 1>();
#pragma unroll
            for (int k = 0; k < TENSORS; ++k)
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
                    v[k][j] = *at(slot_out, k, j);
            slot_out = slot_out + 1 == kStages ? 0 : slot_out + 1;
        } else {
#pragma unroll
            for (int k = 0; k < TENSORS; ++k)
#pragma unroll
                for (int j = 0; j < kGroup; ++j)
#pragma unroll
                    for (int e = 0; e < VEC; ++e)
                        reinterpret_cast<TI *>(&v[k][j])[e] = next[k][j][e];
            load_next();
        }
    }
};

// The convolution of one window.
template <int P, int W>
__device__ __forceinline__ f32x2 window_sum(const f32x2 (&wv)[W][P], const f32x2 (&bv)[P], const f32x2 (&win)[W][P], int i)
{
    f32x2 s = bv[i];
#pragma unroll
    for (int k = 0; k < W; ++k)
        s = fma2(wv[k][i], win[k][i], s);
    return s;
}
template <int P, int W> __device__ __forceinline__ void shift(f32x2 (&win)[W][P])
{
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i)
            win[k][i] = win[k + 1][i];
}

// One thread: VEC channels of `run` consecutive tokens of one sequence, in
// groups of kGroup tokens through the ring.
template <typename TI, int VEC, int S, int W>
__global__ void __launch_bounds__(kConvThreads, kConvBlocks)
conv_kernel(const TI *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
            const TI *__restrict__ init, TI *__restrict__ y, TI *__restrict__ fin, ConvGeom g, int run,
            int64_t n_runs)
{
    constexpr int P = kPairs<VEC>;
    const int64_t nv = conv_columns<VEC, S>(g.dim);
    const int64_t idx = (int64_t)blockIdx.x * kConvThreads + threadIdx.x;
    const int64_t r = idx / nv;
    if (r >= g.batch * n_runs)
        return;
    const int64_t c = first_channel<VEC, S>(idx - r * nv, g.dim);
    const int64_t b = r / n_runs, t0 = (r - b * n_runs) * run;
    f32x2 wv[W][P], bv[P], win[W][P];
    load_weights<VEC, S, W>(w, bias, c, wv, bv);
    const TI *xp = x + (b * g.seqlen + t0) * g.row + c;
    TI *yp = y + (b * g.seqlen + t0) * g.dim + c;
    // the W - 1 tokens before the run
#pragma unroll
    for (int k = 0; k < W - 1; ++k) {
        const int64_t t = t0 - (W - 1) + k;
        RawV<TI, VEC> v{};
        if (t >= 0)
            v = load_raw<TI, VEC, S>(xp + (k - (W - 1)) * g.row);
        else if (init)
            v = load_raw<TI, VEC, S>(init + (b * (W - 1) + (W - 1) + t) * g.dim + c);
        to_pairs<TI, VEC>(v, win[k]);
    }
    const int n = (int)min64(run, g.seqlen - t0);
    auto token = [&](const RawV<TI, VEC> &raw) {
        to_pairs<TI, VEC>(raw, win[W - 1]);
        f32x2 o[P];
#pragma unroll
        for (int i = 0; i < P; ++i) {
            o[i] = window_sum<P, W>(wv, bv, win, i);
            if (g.silu)
                o[i] = mul2(o[i], sigmoid2(o[i]));
        }
        shift<P, W>(win);
        store_pairs<TI, VEC, S>(yp, o);
        yp += g.dim;
    };
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Ring<TI, VEC, S, 1, kConvThreads> ring;
    ring.p[0] = xp;
    ring.row[0] = g.row;
    ring.start(smem_raw, threadIdx.x, n / kGroup);
    int t = 0;
    for (; t + kGroup <= n; t += kGroup) {
        RawV<TI, VEC> raw[1][kGroup];
        ring.take(raw);
#pragma unroll
        for (int j = 0; j < kGroup; ++j)
            token(raw[0][j]);
    }
    xp += t * g.row;
    for (; t < n; ++t) {
        token(load_raw<TI, VEC, S>(xp));
        xp += g.row;
    }
    if (fin && t0 + n == g.seqlen)
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            store_pairs<TI, VEC, S>(fin + (b * (W - 1) + k) * g.dim + c, win[k]);
}

// One token of every sequence (blockIdx.y); state and state_out may be one buffer.
template <typename TI, int VEC, int W>
__global__ void __launch_bounds__(kConvThreads)
conv_step_kernel(const TI *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
                 const TI *state, TI *state_out, TI *__restrict__ y, ConvGeom g)
{
    constexpr int P = kPairs<VEC>;
    const int64_t c = ((int64_t)blockIdx.x * kConvThreads + threadIdx.x) * VEC;
    const int64_t b = blockIdx.y;
    if (c >= g.dim)
        return;
    f32x2 wv[W][P], bv[P], win[W][P], o[P];
    RawV<TI, VEC> raw[W];
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        raw[k] = load_raw<TI, VEC>(state + (b * (W - 1) + k) * g.dim + c);
    raw[W - 1] = load_raw<TI, VEC>(x + b * g.row + c);
    load_weights<VEC, 1, W>(w, bias, c, wv, bv);
#pragma unroll
    for (int k = 0; k < W; ++k)
        to_pairs<TI, VEC>(raw[k], win[k]);
#pragma unroll
    for (int i = 0; i < P; ++i) {
        o[i] = window_sum<P, W>(wv, bv, win, i);
        if (g.silu)
            o[i] = mul2(o[i], sigmoid2(o[i]));
    }
    store_pairs<TI, VEC>(y + b * g.dim + c, o);
#pragma unroll
    for (int k = 0; k < W - 1; ++k)
        *reinterpret_cast<RawV<TI, VEC> *>(state_out + (b * (W - 1) + k) * g.dim + c) = raw[k + 1];
}

// Backward.  With xf = (initial state | x), L + W - 1 rows, pre[i] reads
// xf[i .. i + W - 1] and xf[e] receives sum_k w[k] dpre[e - k] (dpre = 0
// outside [0, L)).  A thread owns rows [e0, e0 + run) of xf (the last one also
// the rows past L): it walks i from e0 - (W - 1), keeping the last W values of
// xf and of dpre, and sums the weight gradient over its own i.  Four such runs
// share a block's channels; their weight gradients are added in shared memory
// and written as one partial per block: part[p][k][c], k = W for the bias.
constexpr int kBwdCols = 32, kBwdRuns = 4;
constexpr int kBwdThreads = kBwdCols * kBwdRuns;
constexpr int kBwdBlocks = 3;  // an SM holds (four, with 128 registers a thread, are no faster)

template <typename TI, int VEC, int S, int W>
__global__ void __launch_bounds__(kBwdThreads, kBwdBlocks)
conv_bwd_kernel(const TI *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
                const TI *__restrict__ init, const TI *__restrict__ dy, const TI *__restrict__ dfinal,
                TI *__restrict__ dx, TI *__restrict__ dinit, float *__restrict__ part, ConvGeom g, int run,
                int64_t parts_per_seq)
{
    constexpr int P = kPairs<VEC>;
    using V = RawV<TI, VEC>;
    __shared__ f32x2 red[W + 1][kBwdRuns][P][kBwdCols];
    extern __shared__ __align__(16) unsigned char smem_raw[];
    static_assert(S == 1 || S == kBwdCols, "a block's channels");
    const int64_t v = (int64_t)blockIdx.x * kBwdCols + threadIdx.x;
    const int64_t c = first_channel<VEC, S>(v, g.dim);
    const int64_t b = blockIdx.y / parts_per_seq;
    const int64_t e0 = ((blockIdx.y - b * parts_per_seq) * kBwdRuns + threadIdx.y) * run;
    const int64_t L = g.seqlen;
    const bool live = v < conv_columns<VEC, S>(g.dim);
    f32x2 dw[W + 1][P];
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i)
            dw[k][i] = 0;
    if (live && (e0 < L || e0 == 0)) {
        f32x2 wv[W][P], bv[P], win[W][P], dp[W][P];
        const TI *xb = x + b * L * g.row + c;
        const TI *dyb = dy + b * L * g.row_dy + c;
        TI *dxb = dx + b * L * g.dim + c;
        auto load_xf = [&](int64_t e) {
            const int64_t t = e - (W - 1);
            return load_or_zero<TI, VEC, S>(t >= 0 && t < L                 ? xb + t * g.row
                                         : t < 0 && e >= 0 && init ? init + (b * (W - 1) + e) * g.dim + c
                                                                         : nullptr);
        };
        auto load_dy = [&](int64_t e) { return load_or_zero<TI, VEC, S>(e >= 0 && e < L ? dyb + e * g.row_dy : nullptr); };
        // All loads of the start are issued before the first is used: the ring's
        // (rows inside the sequence, kGroup tokens at a time, from `own` on), the
        // W - 1 rows of dpre before this thread's own, and what those read.
        const int64_t e1 = e0 + run < L ? e0 + run : L + W - 1, inner = min64(e1, L);
        const int64_t own = e0 < W - 1 ? min64(W - 1, e1) : e0;
        Ring<TI, VEC, S, 2, kBwdThreads> ring;
        ring.p[0] = xb + own * g.row;
        ring.p[1] = dyb + own * g.row_dy;
        ring.row[0] = g.row;
        ring.row[1] = g.row_dy;
        ring.start(smem_raw, threadIdx.y * kBwdCols + threadIdx.x, inner > own ? (int)(inner - own) / kGroup : 0);
        V before[2 * (W - 1)], before_dy[W - 1];
#pragma unroll
        for (int k = 0; k < 2 * (W - 1); ++k)
            before[k] = load_xf(e0 - (W - 1) + k);
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            before_dy[k] = load_dy(e0 - (W - 1) + k);
        load_weights<VEC, S, W>(w, bias, c, wv, bv);
#pragma unroll
        for (int k = 0; k < W; ++k) {
#pragma unroll
            for (int i = 0; i < P; ++i)
                dp[k][i] = 0;
            if (k < W - 1)
                to_pairs<TI, VEC>(before[k], win[k]);
        }
        // dp[0] = dpre[e] from xf[e + W - 1] = x[e] and dy[e]; dp[k] = dpre[e - k]
        auto step_in = [&](const V &xr, const V &yr) {
            to_pairs<TI, VEC>(xr, win[W - 1]);
            f32x2 d[P];
            to_pairs<TI, VEC>(yr, d);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (g.silu) {
                    const f32x2 s = window_sum<P, W>(wv, bv, win, i);
                    d[i] = mul2(d[i], silu_grad2(s, sigmoid2(s)));
                }
#pragma unroll
                for (int k = W - 1; k > 0; --k)
                    dp[k][i] = dp[k - 1][i];
                dp[0][i] = d[i];
            }
        };
        auto sums = [&]() {
#pragma unroll
            for (int i = 0; i < P; ++i) {
#pragma unroll
                for (int k = 0; k < W; ++k)
                    dw[k][i] = fma2(dp[0][i], win[k][i], dw[k][i]);
                dw[W][i] = add2(dw[W][i], dp[0][i]);
            }
        };
        auto grad = [&](f32x2 (&o)[P]) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                o[i] = mul2(wv[0][i], dp[0][i]);
#pragma unroll
                for (int k = 1; k < W; ++k)
                    o[i] = fma2(wv[k][i], dp[k][i], o[i]);
            }
        };
        // any row: before the sequence, past its end, or not yet this thread's own
        auto edge = [&](int64_t e, const V &xr, const V &yr) {
            const bool in = e >= 0 && e < L;
            if (in) {
                step_in(xr, yr);
            } else {
                to_pairs<TI, VEC>(xr, win[W - 1]);
#pragma unroll
                for (int i = 0; i < P; ++i) {
#pragma unroll
                    for (int k = W - 1; k > 0; --k)
                        dp[k][i] = dp[k - 1][i];
                    dp[0][i] = 0;
                }
            }
            if (e >= e0) {
                if (in)
                    sums();
                f32x2 o[P];
                grad(o);
                if (dfinal && e >= L) {  // the carried rows are the last W - 1 of xf
                    f32x2 f[P];
                    to_pairs<TI, VEC>(load_raw<TI, VEC, S>(dfinal + (b * (W - 1) + e - L) * g.dim + c), f);
#pragma unroll
                    for (int i = 0; i < P; ++i)
                        o[i] = add2(o[i], f[i]);
                }
                if (e >= W - 1)
                    store_pairs<TI, VEC, S>(dxb + (e - (W - 1)) * g.dim, o);
                else if (dinit)
                    store_pairs<TI, VEC, S>(dinit + (b * (W - 1) + e) * g.dim + c, o);
            }
            shift<P, W>(win);
        };
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
            edge(e0 - (W - 1) + k, before[W - 1 + k], before_dy[k]);
        int64_t e = e0;
        for (; e < own; ++e)
            edge(e, load_xf(e + W - 1), load_dy(e));
        TI *op = dxb + (e - (W - 1)) * g.dim;
        for (; e + kGroup <= inner; e += kGroup) {
            V raw[2][kGroup];
            ring.take(raw);
#pragma unroll
            for (int j = 0; j < kGroup; ++j) {
                step_in(raw[0][j], raw[1][j]);
                sums();
                f32x2 o[P];
                grad(o);
                store_pairs<TI, VEC, S>(op, o);
                op += g.dim;
                shift<P, W>(win);
            }
        }
        for (; e < e1; ++e)
            edge(e, load_xf(e + W - 1), load_dy(e));
    }
#pragma unroll
    for (int k = 0; k <= W; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i)
            red[k][threadIdx.y][i][threadIdx.x] = dw[k][i];
    __syncthreads();
    if (live)
        for (int k = threadIdx.y; k <= W; k += kBwdRuns) {
            f32x2 s[P];
#pragma unroll
            for (int i = 0; i < P; ++i) {
                s[i] = red[k][0][i][threadIdx.x];
#pragma unroll
                for (int q = 1; q < kBwdRuns; ++q)
                    s[i] = add2(s[i], red[k][q][i][threadIdx.x]);
            }
            store_pairs<float, VEC, S>(part + ((int64_t)blockIdx.y * (W + 1) + k) * g.dim + c, s);
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
#pragma unroll 8
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

// Tokens a thread walks: the run of least waves x (run + start), where `start`
// is what the rows before a run and its first loads cost in tokens.  blocks(run)
// are the call's blocks, `slots` those that the GPU holds at once.
template <typename F> int pick_run(int64_t seqlen, int64_t slots, int start, F blocks)
{
    int best = 4;
    int64_t least = INT64_MAX;
    for (int run = 4; run <= 256; run += 4) {
        const int64_t waves = (blocks(run) + slots - 1) / slots;
        if (waves * (run + start) < least) {
            least = waves * (run + start);
            best = run;
        }
        if (waves == 1 || run >= seqlen)  // longer runs only leave slots idle
            break;
    }
    return best;
}
int conv_run(const ConvGeom &g, int64_t columns)
{
    const int64_t threads = g.batch * columns;
    return pick_run(g.seqlen, (int64_t)device_sm_count() * kConvBlocks, 8, [&](int run) {
        return (threads * ((g.seqlen + run - 1) / run) + kConvThreads - 1) / kConvThreads;
    });
}

int64_t conv_bwd_parts_per_seq(const ConvGeom &g, int run)
{
    return ((g.seqlen > 0 ? g.seqlen : 1) + (int64_t)kBwdRuns * run - 1) / ((int64_t)kBwdRuns * run);
}

// kBwdRuns runs in a block.
int conv_bwd_run(const ConvGeom &g, int64_t columns)
{
    const int64_t cols = (columns + kBwdCols - 1) / kBwdCols;
    int run = pick_run(g.seqlen, (int64_t)device_sm_count() * kBwdBlocks, 12,
                       [&](int r) { return cols * g.batch * conv_bwd_parts_per_seq(g, r); });
    while (conv_bwd_parts_per_seq(g, run) * g.batch > 65535)  // one grid row each
        run *= 2;
    return run;
}

template <typename TI, int VEC, int S, int W>
cudaError_t fwd_w(const void *x, const float *w, const float *bias, const void *init, void *y, void *fin,
                  const ConvGeom &g, cudaStream_t st)
{
    const int64_t columns = conv_columns<VEC, S>(g.dim);
    const int run = conv_run(g, columns);
    const int64_t n_runs = (g.seqlen + run - 1) / run;
    const int64_t threads = g.batch * n_runs * columns;
    constexpr size_t smem = Ring<TI, VEC, S, 1, kConvThreads>::kBytes;
    auto k = conv_kernel<TI, VEC, S, W>;
    static SmemGrant granted;
    const cudaError_t allowed = allow_smem(reinterpret_cast<const void *>(k), smem, &granted);
    if (allowed != cudaSuccess)
        return allowed;
    k<<<(unsigned)((threads + kConvThreads - 1) / kConvThreads), kConvThreads, smem, st>>>(
        static_cast<const TI *>(x), w, bias, static_cast<const TI *>(init), static_cast<TI *>(y),
        static_cast<TI *>(fin), g, run, n_runs);
    note_launch(1);
    return cudaGetLastError();
}
template <typename TI, int VEC, int S, int W>
cudaError_t step_w(const void *x, const float *w, const float *bias, const void *state, void *state_out,
                   void *y, const ConvGeom &g, cudaStream_t st)
{
    const dim3 grid((unsigned)((g.dim / VEC + kConvThreads - 1) / kConvThreads), (unsigned)g.batch);
    conv_step_kernel<TI, VEC, W><<<grid, kConvThreads, 0, st>>>(
            static_cast<const TI *>(x), w, bias, static_cast<const TI *>(state), static_cast<TI *>(state_out),
            static_cast<TI *>(y), g);
    note_launch(1);
    return cudaGetLastError();
}
template <typename TI, int VEC, int S, int W>
cudaError_t bwd_w(const void *x, const float *w, const float *bias, const void *init, const void *dy,
                  const void *dfinal, void *dx, float *dw, float *dbias, void *dinit, float *part,
                  const ConvGeom &g, cudaStream_t st)
{
    const int64_t columns = conv_columns<VEC, S>(g.dim);
    const int run = conv_bwd_run(g, columns);
    const int64_t pps = conv_bwd_parts_per_seq(g, run);
    const dim3 grid((unsigned)((columns + kBwdCols - 1) / kBwdCols), (unsigned)(pps * g.batch));
    constexpr size_t smem = Ring<TI, VEC, S, 2, kBwdThreads>::kBytes;
    auto k = conv_bwd_kernel<TI, VEC, S, W>;
    static SmemGrant granted;
    const cudaError_t allowed = allow_smem(reinterpret_cast<const void *>(k), smem, &granted);
    if (allowed != cudaSuccess)
        return allowed;
    k<<<grid, dim3(kBwdCols, kBwdRuns), smem, st>>>(
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

// F<TI, VEC, S, W> for the call's width and layout: four adjacent channels a
// thread where every row starts on a boundary of four (8 bytes of bf16, 16 of
// f32).  Off them, two channels a warp apart where the type is bf16 (6 x 1769
// tokens of 2707 channels: forward 29 us instead of 42 with one, backward 58
// instead of 86), one where it is f32, whose elements the rings can copy (3 x
// 3331 tokens of 1537 channels: 25 us, 72% of the measured copy rate).
#define SSD_CONV_WIDTHS(F, TI, VEC, S, ...)                                                         \
    (g.width == 2 ? F<TI, VEC, S, 2>(__VA_ARGS__)                                                   \
                  : (g.width == 3 ? F<TI, VEC, S, 3>(__VA_ARGS__) : F<TI, VEC, S, 4>(__VA_ARGS__)))

}  // namespace

cudaError_t launch_conv(const void *x, const float *w, const float *bias, const void *init, void *y,
                        void *fin, const ConvGeom &g, bool bf16, cudaStream_t st)
{
    const size_t a = bf16 ? 8 : 16;
    const bool al = aligned(x, a) && aligned(init, a) && aligned(y, a) && aligned(fin, a) && aligned(w, 8) &&
                    g.dim % 4 == 0 && g.row % 4 == 0;
    if (bf16) {
        if (al)
            return SSD_CONV_WIDTHS(fwd_w, __nv_bfloat16, 4, 1, x, w, bias, init, y, fin, g, st);
        if (g.dim >= 64)
            return SSD_CONV_WIDTHS(fwd_w, __nv_bfloat16, 2, 32, x, w, bias, init, y, fin, g, st);
        return SSD_CONV_WIDTHS(fwd_w, __nv_bfloat16, 1, 1, x, w, bias, init, y, fin, g, st);
    }
    if (al)
        return SSD_CONV_WIDTHS(fwd_w, float, 4, 1, x, w, bias, init, y, fin, g, st);
    return SSD_CONV_WIDTHS(fwd_w, float, 1, 1, x, w, bias, init, y, fin, g, st);
}

// One channel a thread off the boundaries: state_out may be state, so no channel
// is computed twice.
cudaError_t launch_conv_step(const void *x, const float *w, const float *bias, const void *state,
                             void *state_out, void *y, const ConvGeom &g, bool bf16, cudaStream_t st)
{
    const size_t a = bf16 ? 8 : 16;
    const bool al = aligned(x, a) && aligned(state, a) && aligned(state_out, a) && aligned(y, a) &&
                    aligned(w, 8) && g.dim % 4 == 0 && g.row % 4 == 0;
    if (bf16) {
        if (al)
            return SSD_CONV_WIDTHS(step_w, __nv_bfloat16, 4, 1, x, w, bias, state, state_out, y, g, st);
        return SSD_CONV_WIDTHS(step_w, __nv_bfloat16, 1, 1, x, w, bias, state, state_out, y, g, st);
    }
    if (al)
        return SSD_CONV_WIDTHS(step_w, float, 4, 1, x, w, bias, state, state_out, y, g, st);
    return SSD_CONV_WIDTHS(step_w, float, 1, 1, x, w, bias, state, state_out, y, g, st);
}

// Room for the partials of any layout (alignment is not known here).
size_t conv_bwd_workspace(const ConvGeom &g)
{
    int64_t parts = 0;
    for (int64_t columns : {conv_columns<4, 1>(g.dim), conv_columns<2, 32>(g.dim), g.dim}) {
        const int64_t p = conv_bwd_parts_per_seq(g, conv_bwd_run(g, columns)) * g.batch;
        parts = p > parts ? p : parts;
    }
    return (size_t)(parts * (g.width + 1) * g.dim) * sizeof(float);
}

cudaError_t launch_conv_bwd(const void *x, const float *w, const float *bias, const void *init,
                            const void *dy, const void *dfinal, void *dx, float *dw, float *dbias,
                            void *dinit, float *part, const ConvGeom &g, bool bf16, cudaStream_t st)
{
    const size_t a = bf16 ? 8 : 16;
    bool al = g.dim % 4 == 0 && g.row % 4 == 0 && g.row_dy % 4 == 0 && aligned(w, 8);
    for (const void *p : {x, init, dy, dfinal, static_cast<const void *>(dx), static_cast<const void *>(dinit)})
        al = al && aligned(p, a);
    if (bf16) {
        if (al)
            return SSD_CONV_WIDTHS(bwd_w, __nv_bfloat16, 4, 1, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit, part, g, st);
        if (g.dim >= 64)
            return SSD_CONV_WIDTHS(bwd_w, __nv_bfloat16, 2, 32, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit, part, g, st);
        return SSD_CONV_WIDTHS(bwd_w, __nv_bfloat16, 1, 1, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit, part, g, st);
    }
    if (al)
        return SSD_CONV_WIDTHS(bwd_w, float, 4, 1, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit, part, g, st);
    return SSD_CONV_WIDTHS(bwd_w, float, 1, 1, x, w, bias, init, dy, dfinal, dx, dw, dbias, dinit, part, g, st);
}

}  // namespace ssd
