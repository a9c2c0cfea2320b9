// Selective scan, gradients.  With the states entering every chunk of 16
// tokens kept by the forward (h) and by the reverse pass (g, the state
// gradient leaving the chunk on its right), all chunks are independent.  Per
// token, from the chunk's last to its first, with a = exp(delta A),
// dyy = dout silu(z) and e = g + dyy C:
//     dC += dyy h          dB += e delta u        sB = sum_n e B
//     q = e (a h_{t-1})    dA += q delta          sA = sum_n q A
//     g <- a e
//     du = delta sB + D dyy,  ddelta = u sB + sA,  ddt = ddelta softplus'(dt + bias)
//     dz = dout (sum_n C h + D u) silu'(z),        dD += dyy u,  dbias += ddt
// dB and dC are sums over the group's channels: a thread owns four states of
// one channel and goes through four channels for the same eight tokens with
// the sums in registers; a block adds its threads' sums once per eight tokens
// and writes one partial per channel block, and a last kernel adds those in a
// fixed order (no atomics, so results do not depend on scheduling).
// Arithmetic on about 12 issue slots per (token, channel, state) bounds it.
#include "scan.cuh"

namespace ssd {
namespace {

constexpr int kIters = 4;  // channels a thread goes through
constexpr int kSub = 8;    // tokens whose a and a h a thread holds

template <typename TI> struct GradArgs {
    const TI *u, *dt, *bm, *cm, *z, *dy;
    const float *A, *D, *bias, *h0, *g1;
    TI *du, *ddt, *dz;
    float *dB, *dC;        // [channel blocks][B * L][N]
    float *dA;             // [B * chunk groups][dim][N]
    float *dD;             // [B * chunk groups][2][dim]: dD, dbias
    int64_t chunks_per_group;
    bool vec;
};

template <int LN> struct GradSmem {
    static constexpr int CBK = kIters * kScanThreads / LN, NP = 4 * LN;
    float2 dd[kScanChunk][CBK];  // delta, delta u
    float dyy[kScanChunk][CBK];
    float y[kSub][CBK], sB[kSub][CBK], sA[kSub][CBK];
    float4 h[kIters][kScanThreads], e[kIters][kScanThreads], dA[kIters][kScanThreads];
    float m[kScanChunk * NP], c[kScanChunk * NP];
    float red[kSub * 4][kScanThreads];
};

__device__ __forceinline__ void to4(const float4 &f, float (&v)[4])
{
    v[0] = f.x;
    v[1] = f.y;
    v[2] = f.z;
    v[3] = f.w;
}

// Adds each thread's kSub x 4 values over the block's channels and writes the
// [kSub][N] sums of live tokens.
template <int LN>
__device__ __forceinline__ void block_rows_sum(const float (&v)[kSub][4], float (*red)[kScanThreads], float *out,
                                               int nt, int N)
{
    constexpr int CB = kScanThreads / LN;
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kSub; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            red[t * 4 + e][threadIdx.x] = v[t][e];
    __syncthreads();
    for (int o = threadIdx.x; o < kSub * 4 * LN; o += kScanThreads) {
        const int j = o % LN, r = o / LN, t = r / 4, n = 4 * j + r % 4;
        float s = 0.f;
        for (int i = 0; i < CB; ++i)  // starting channels differ to spread the banks
            s += red[r][((i + r) % CB) * LN + j];
        if (t < nt && n < N)
            out[t * N + n] = s;
    }
}

template <typename TI, int LN>
__global__ void __launch_bounds__(kScanThreads) scan_grad_kernel(GradArgs<TI> a, ScanGeom g)
{
    constexpr int CB = kScanThreads / LN, CBK = kIters * CB, T = kScanChunk, NP = 4 * LN;
    constexpr int COLS = CBK / 4, TPR = kScanThreads / COLS;  // elementwise: 4-channel columns x token rows
    extern __shared__ __align__(16) unsigned char smem_raw[];
    GradSmem<LN> &s = *reinterpret_cast<GradSmem<LN> *>(smem_raw);
    const int tid = threadIdx.x;
    const int64_t nblk = (g.kpg + CBK - 1) / CBK;
    const int grp = (int)(blockIdx.x / nblk);
    const int64_t c0 = (blockIdx.x - grp * nblk) * CBK;
    const int nch = (int)min64(CBK, g.kpg - c0);
    const int64_t ch0 = grp * g.kpg + c0;
    const int64_t b = blockIdx.z;
    const int64_t nc = (g.seqlen + T - 1) / T;
    const int64_t cbeg = blockIdx.y * a.chunks_per_group, cend = min64(cbeg + a.chunks_per_group, nc);
    const int cl = tid / LN, n0 = 4 * (tid % LN);
    const int N = (int)g.N, nn = N - n0;
    const int col = 4 * (tid % COLS), trow = tid / COLS;
    float accD[4] = {}, accb[4] = {};
#pragma unroll
    for (int k = 0; k < kIters; ++k)
        s.dA[k][tid] = make_float4(0.f, 0.f, 0.f, 0.f);

    for (int64_t chunk = cbeg; chunk < cend; ++chunk) {
        const int64_t t0 = chunk * T;
        const int nt = (int)min64(T, g.seqlen - t0);
        const int64_t tok0 = b * g.seqlen + t0;
        __syncthreads();  // the chunk before is done with the tiles
        for (int t = trow; t < T; t += TPR) {
            const int n = t < nt ? nch - col : 0;
            const int64_t tok = tok0 + t;
            Raw4<TI> ur{}, dr{}, zr{}, yr{};
            if (n > 0) {
                ur = load_raw4(a.u + tok * g.row_u + ch0 + col, n, a.vec);
                dr = load_raw4(a.dt + tok * g.row_dt + ch0 + col, n, a.vec);
                yr = load_raw4(a.dy + tok * g.row_dy + ch0 + col, n, a.vec);
                if (a.z)
                    zr = load_raw4(a.z + tok * g.row_z + ch0 + col, n, a.vec);
            }
            float uv[4], dv[4], zv[4], yv[4];
            unpack<TI, 4>(ur, uv);
            unpack<TI, 4>(dr, dv);
            unpack<TI, 4>(zr, zv);
            unpack<TI, 4>(yr, yv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float d = 0.f;
                if (e < n) {
                    d = dv[e] + (a.bias ? a.bias[ch0 + col + e] : 0.f);
                    d = g.softplus ? softplus(d) : d;
                }
                s.dd[t][col + e] = make_float2(d, d * uv[e]);
                s.dyy[t][col + e] = a.z ? yv[e] * fast_silu(zv[e]) : yv[e];
            }
        }
        load_rows<TI, LN>(a.bm + tok0 * g.row_b + grp * g.N, g.row_b, nt, N, s.m);
        load_rows<TI, LN>(a.cm + tok0 * g.row_c + grp * g.N, g.row_c, nt, N, s.c);
        __syncthreads();

        const int64_t kept = (b * nc + chunk) * g.dim;
        // the state after the first eight tokens, and the gradient entering the chunk
#pragma unroll 1
        for (int k = 0; k < kIters; ++k) {
            const int c = k * CB + cl;
            float h[4] = {}, A2[4] = {}, e0[4] = {};
            if (c < nch && nn > 0) {
                const int64_t st = (kept + ch0 + c) * g.N + n0;
                load_states(a.h0 + st, nn, h);
                load_states(a.g1 + st, nn, e0);
                load_states(a.A + (ch0 + c) * g.N + n0, nn, A2);
            }
#pragma unroll
            for (int t = 0; t < kSub; ++t) {
                const float2 dd = s.dd[t][c];
                float m[4];
                to4(*reinterpret_cast<const float4 *>(&s.m[t * NP + n0]), m);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    h[e] = fmaf(ex2(dd.x * decay_rate(A2[e])), h[e], dd.y * m[e]);
            }
            s.h[k][tid] = make_float4(h[0], h[1], h[2], h[3]);
            s.e[k][tid] = make_float4(e0[0], e0[1], e0[2], e0[3]);
        }
#pragma unroll 1
        for (int sub = 1; sub >= 0; --sub) {
            const int ts = sub * kSub;
            if (ts >= nt && sub > 0)
                continue;
            float dB[kSub][4] = {}, dC[kSub][4] = {};
#pragma unroll 1
            for (int k = 0; k < kIters; ++k) {
                const int c = k * CB + cl;
                if (k * CB >= nch)
                    break;
                float h[4] = {}, A2[4] = {}, e0[4], acc[4];
                if (c < nch && nn > 0)
                    load_states(a.A + (ch0 + c) * g.N + n0, nn, A2);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    A2[e] = decay_rate(A2[e]);
                if (sub)
                    to4(s.h[k][tid], h);
                else if (c < nch && nn > 0)
                    load_states(a.h0 + (kept + ch0 + c) * g.N + n0, nn, h);
                to4(s.e[k][tid], e0);
                to4(s.dA[k][tid], acc);
                float av[kSub][4], ah[kSub][4];
#pragma unroll
                for (int t = 0; t < kSub; ++t) {
                    const float2 dd = s.dd[ts + t][c];
                    const float dyy = s.dyy[ts + t][c];
                    float m[4], cv[4], y = 0.f;
                    to4(*reinterpret_cast<const float4 *>(&s.m[(ts + t) * NP + n0]), m);
                    to4(*reinterpret_cast<const float4 *>(&s.c[(ts + t) * NP + n0]), cv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        av[t][e] = ex2(dd.x * A2[e]);
                        ah[t][e] = av[t][e] * h[e];
                        h[e] = fmaf(dd.y, m[e], ah[t][e]);
                        dC[t][e] = fmaf(dyy, h[e], dC[t][e]);
                        y = fmaf(cv[e], h[e], y);
                    }
                    y = lane_sum<LN>(y);
                    if (n0 == 0)
                        s.y[t][c] = y;
                }
#pragma unroll
                for (int t = kSub - 1; t >= 0; --t) {
                    const float2 dd = s.dd[ts + t][c];
                    const float dyy = s.dyy[ts + t][c];
                    float m[4], cv[4], sB = 0.f, sA = 0.f;
                    to4(*reinterpret_cast<const float4 *>(&s.m[(ts + t) * NP + n0]), m);
                    to4(*reinterpret_cast<const float4 *>(&s.c[(ts + t) * NP + n0]), cv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        e0[e] = fmaf(dyy, cv[e], e0[e]);
                        dB[t][e] = fmaf(e0[e], dd.y, dB[t][e]);
                        sB = fmaf(e0[e], m[e], sB);
                        const float q = e0[e] * ah[t][e];
                        acc[e] = fmaf(q, dd.x, acc[e]);
                        sA = fmaf(q, A2[e], sA);
                        e0[e] *= av[t][e];
                    }
                    sB = lane_sum<LN>(sB);
                    sA = lane_sum<LN>(sA);
                    if (n0 == 0) {
                        s.sB[t][c] = sB;
                        s.sA[t][c] = sA;
                    }
                }
                s.e[k][tid] = make_float4(e0[0], e0[1], e0[2], e0[3]);
                s.dA[k][tid] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            }
            const int ns = nt - ts;
            float *rows = a.dB + ((int64_t)blockIdx.x * g.batch * g.seqlen + tok0 + ts) * g.N;
            block_rows_sum<LN>(dB, s.red, rows, ns, N);
            rows = a.dC + ((int64_t)blockIdx.x * g.batch * g.seqlen + tok0 + ts) * g.N;
            block_rows_sum<LN>(dC, s.red, rows, ns, N);
            // per (token, channel) results
            for (int t = trow; t < kSub; t += TPR) {
                const int n = t < ns ? nch - col : 0;
                if (n <= 0)
                    continue;
                const int64_t tok = tok0 + ts + t;
                float uv[4], dv[4], zv[4], yv[4], du[4], ddt[4], dz[4];
                unpack<TI, 4>(load_raw4(a.u + tok * g.row_u + ch0 + col, n, a.vec), uv);
                unpack<TI, 4>(load_raw4(a.dt + tok * g.row_dt + ch0 + col, n, a.vec), dv);
                if (a.z) {
                    unpack<TI, 4>(load_raw4(a.z + tok * g.row_z + ch0 + col, n, a.vec), zv);
                    unpack<TI, 4>(load_raw4(a.dy + tok * g.row_dy + ch0 + col, n, a.vec), yv);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (e >= n)
                        continue;
                    const float Dv = a.D ? a.D[ch0 + col + e] : 0.f;
                    const float dyy = s.dyy[ts + t][col + e], delta = s.dd[ts + t][col + e].x;
                    const float sB = s.sB[t][col + e];
                    du[e] = fmaf(delta, sB, Dv * dyy);
                    ddt[e] = fmaf(uv[e], sB, s.sA[t][col + e] * kLn2);
                    if (g.softplus)
                        ddt[e] *= fast_sigmoid(dv[e] + (a.bias ? a.bias[ch0 + col + e] : 0.f));
                    if (a.z) {
                        const float yy = fmaf(Dv, uv[e], s.y[t][col + e]);
                        dz[e] = yv[e] * yy * silu_grad(zv[e], fast_sigmoid(zv[e]));
                    }
                    accD[e] = fmaf(dyy, uv[e], accD[e]);
                    accb[e] += ddt[e];
                }
                store4(a.du + tok * g.dim + ch0 + col, du, n, a.vec);
                store4(a.ddt + tok * g.dim + ch0 + col, ddt, n, a.vec);
                if (a.z)
                    store4(a.dz + tok * g.dim + ch0 + col, dz, n, a.vec);
            }
            __syncthreads();
        }
    }
    // this block's partial sums over its tokens
    const int64_t item = b * gridDim.y + blockIdx.y;
#pragma unroll
    for (int k = 0; k < kIters; ++k) {
        const int c = k * CB + cl;
        if (c < nch && nn > 0) {
            float v[4];
            to4(s.dA[k][tid], v);
            store_states(a.dA + (item * g.dim + ch0 + c) * g.N + n0, nn, v);
        }
    }
    __syncthreads();
    float *red = &s.red[0][0];  // [TPR][2][CBK]
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        red[(trow * 2) * CBK + col + e] = accD[e];
        red[(trow * 2 + 1) * CBK + col + e] = accb[e];
    }
    __syncthreads();
    for (int i = tid; i < 2 * CBK; i += kScanThreads) {
        const int w = i / CBK, c = i % CBK;
        float v = 0.f;
        for (int r = 0; r < TPR; ++r)
            v += red[(r * 2 + w) * CBK + c];
        if (c < nch)
            a.dD[(item * 2 + w) * g.dim + ch0 + c] = v;
    }
}

// out[i][g][n] = sum over the group's channel blocks k of src[g nblk + k][i][n].
template <typename TI>
__global__ void __launch_bounds__(256) sum_blocks_kernel(const float *__restrict__ src, TI *__restrict__ out,
                                                         int64_t tokens, int64_t G, int64_t N, int64_t nblk)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= tokens * G * N)
        return;
    const int64_t n = i % N, r = i / N, grp = r % G, t = r / G;
    const float *p = src + ((grp * nblk) * tokens + t) * N + n;
    float s = 0.f;
    for (int64_t k = 0; k < nblk; ++k)
        s += p[k * tokens * N];
    out[i] = from_f32<TI>(s);
}

// out[i] = sum over p of src[p * stride + i].
__global__ void __launch_bounds__(256) sum_items_kernel(const float *__restrict__ src, float *__restrict__ out,
                                                        int64_t n, int64_t items, int64_t stride)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n)
        return;
    float s = 0.f;
    for (int64_t p = 0; p < items; ++p)
        s += src[p * stride + i];
    out[i] = s;
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct GradPlan {
    int64_t nblk, chunks_per_group, n_groups;
};
GradPlan grad_plan(const ScanGeom &g)
{
    GradPlan p;
    const int64_t cbk = kIters * kScanThreads / scan_lanes(g.N);
    p.nblk = (g.kpg + cbk - 1) / cbk;
    const int64_t nc = (g.seqlen + kScanChunk - 1) / kScanChunk;
    // several blocks per SM, each over a run of chunks so that the sums over
    // tokens leave few partials
    const int64_t want = (int64_t)device_sm_count() * 4;
    const int64_t cols = p.nblk * g.G * g.batch;
    int64_t n = (want + cols - 1) / cols;
    n = n > nc ? nc : n;
    p.chunks_per_group = (nc + n - 1) / n;
    p.n_groups = (nc + p.chunks_per_group - 1) / p.chunks_per_group;
    return p;
}

template <typename TI, int LN>
cudaError_t grad_ln(const GradArgs<TI> &a, const ScanGeom &g, const GradPlan &p, cudaStream_t st)
{
    auto k = scan_grad_kernel<TI, LN>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)sizeof(GradSmem<LN>));
    if (e != cudaSuccess)
        return e;
    k<<<dim3((unsigned)(g.G * p.nblk), (unsigned)p.n_groups, (unsigned)g.batch), kScanThreads,
        sizeof(GradSmem<LN>), st>>>(a, g);
    note_launch(1);
    return cudaGetLastError();
}

struct GradWs {
    float *dB, *dC, *dA, *dD;
    size_t bytes;
};
GradWs grad_layout(const ScanGeom &g, char *base)
{
    const GradPlan p = grad_plan(g);
    GradWs w{};
    size_t off = 0;
    auto take = [&](int64_t n) {
        char *q = base ? base + off : nullptr;
        off += ((size_t)n * sizeof(float) + 255) / 256 * 256;
        return reinterpret_cast<float *>(q);
    };
    w.dB = take(g.G * p.nblk * g.batch * g.seqlen * g.N);
    w.dC = take(g.G * p.nblk * g.batch * g.seqlen * g.N);
    w.dA = take(g.batch * p.n_groups * g.dim * g.N);
    w.dD = take(g.batch * p.n_groups * 2 * g.dim);
    w.bytes = off;
    return w;
}

template <typename TI>
cudaError_t grad_t(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *D,
                   const void *z, const float *bias, const void *dy, const float *h0, const float *g1, void *du,
                   void *ddt, float *dA, void *dB, void *dC, float *dD, void *dz, float *dbias, void *ws,
                   const ScanGeom &g, cudaStream_t st)
{
    const GradPlan p = grad_plan(g);
    const GradWs w = grad_layout(g, static_cast<char *>(ws));
    GradArgs<TI> a{};
    a.u = static_cast<const TI *>(u);
    a.dt = static_cast<const TI *>(dt);
    a.bm = static_cast<const TI *>(Bm);
    a.cm = static_cast<const TI *>(Cm);
    a.z = static_cast<const TI *>(z);
    a.dy = static_cast<const TI *>(dy);
    a.A = A;
    a.D = D;
    a.bias = bias;
    a.h0 = h0;
    a.g1 = g1;
    a.du = static_cast<TI *>(du);
    a.ddt = static_cast<TI *>(ddt);
    a.dz = static_cast<TI *>(dz);
    a.dB = w.dB;
    a.dC = w.dC;
    a.dA = w.dA;
    a.dD = w.dD;
    a.chunks_per_group = p.chunks_per_group;
    const size_t al = 4 * sizeof(TI);
    a.vec = (g.kpg % 4 == 0 || g.G == 1) && g.dim % 4 == 0 && g.row_u % 4 == 0 && g.row_dt % 4 == 0 &&
            g.row_dy % 4 == 0 && (!z || g.row_z % 4 == 0);
    for (const void *q : {u, dt, z, dy, static_cast<const void *>(du), static_cast<const void *>(ddt),
                          static_cast<const void *>(dz)})
        a.vec = a.vec && aligned(q, al);
    cudaError_t e;
    switch (scan_lanes(g.N)) {
    case 1: e = grad_ln<TI, 1>(a, g, p, st); break;
    case 2: e = grad_ln<TI, 2>(a, g, p, st); break;
    case 4: e = grad_ln<TI, 4>(a, g, p, st); break;
    case 8: e = grad_ln<TI, 8>(a, g, p, st); break;
    default: e = grad_ln<TI, 16>(a, g, p, st); break;
    }
    if (e != cudaSuccess)
        return e;
    const int64_t tokens = g.batch * g.seqlen, nbc = tokens * g.G * g.N;
    const unsigned bb = (unsigned)((nbc + 255) / 256);
    sum_blocks_kernel<TI><<<bb, 256, 0, st>>>(w.dB, static_cast<TI *>(dB), tokens, g.G, g.N, p.nblk);
    sum_blocks_kernel<TI><<<bb, 256, 0, st>>>(w.dC, static_cast<TI *>(dC), tokens, g.G, g.N, p.nblk);
    const int64_t items = g.batch * p.n_groups, dn = g.dim * g.N;
    sum_items_kernel<<<(unsigned)((dn + 255) / 256), 256, 0, st>>>(w.dA, dA, dn, items, dn);
    note_launch(3);
    const unsigned db = (unsigned)((g.dim + 255) / 256);
    if (dD) {
        sum_items_kernel<<<db, 256, 0, st>>>(w.dD, dD, g.dim, items, 2 * g.dim);
        note_launch(1);
    }
    if (dbias) {
        sum_items_kernel<<<db, 256, 0, st>>>(w.dD + g.dim, dbias, g.dim, items, 2 * g.dim);
        note_launch(1);
    }
    return cudaGetLastError();
}

}  // namespace

size_t scan_grad_workspace(const ScanGeom &g) { return grad_layout(g, nullptr).bytes; }

cudaError_t launch_scan_grad(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                             const float *D, const void *z, const float *bias, const void *dy, const float *h0,
                             const float *g1, void *du, void *ddt, float *dA, void *dB, void *dC, float *dD,
                             void *dz, float *dbias, void *ws, const ScanGeom &g, bool bf16, cudaStream_t st)
{
    return bf16 ? grad_t<__nv_bfloat16>(u, dt, A, Bm, Cm, D, z, bias, dy, h0, g1, du, ddt, dA, dB, dC, dD, dz,
                                        dbias, ws, g, st)
                : grad_t<float>(u, dt, A, Bm, Cm, D, z, bias, dy, h0, g1, du, ddt, dA, dB, dC, dD, dz, dbias, ws,
                                g, st);
}

}  // namespace ssd
