// Selective scan: the state space recurrence with a decay of its own for
// every channel and state,
//     delta = softplus(dt + dt_bias),
//     h[n] <- exp(delta A[d,n]) h[n] + delta u B[g,n],
//     y = sum_n C[g,n] h[n] + D u,   out = y silu(z)
// for prompts (token tiles with the states in registers), for single tokens,
// and the reverse recurrence the backward starts from,
//     g_t[n] = exp(delta_t A[d,n]) (g_{t+1}[n] + dy_t C_t[n]).
// With no decay shared between states there is no matrix product to form:
// a token costs one exponential and about six f32 operations per (channel,
// state), which at 16 states outweigh the HBM traffic (u, dt, z in, out).
#include "scan.cuh"

namespace ssd {
namespace {

// One pass over a run of chunks of one sequence and one block of channels.
// Forward (REV = false): m = B, x = u, z gates the output.  Reverse: m = C,
// x = dout gated by z, tokens from the last to the first.
template <typename TI> struct PassArgs {
    const TI *x, *dt, *z, *m, *cm;
    const float *A, *D, *bias;
    const float *start;  // [B][segments][dim][N], nullptr: zeros
    TI *y;               // forward output, or nullptr: states only
    float *last;         // final state (forward), initial state's gradient (reverse), or nullptr
    float *kept;         // [B][nc][dim][N] state entering each chunk, or nullptr
    float *seg_end;      // [B][segments][dim][N] end state of each segment, or nullptr
    float *seg_dsum;     // [B][segments][dim] sum of delta of each segment
    int64_t row_x;
    int64_t chunks_per_seg, first_seg, n_seg;
    bool vec;
};

template <typename TI, int LN, bool REV>
__global__ void __launch_bounds__(kScanThreads) scan_pass_kernel(PassArgs<TI> a, ScanGeom g)
{
    constexpr int CB = kScanThreads / LN, T = kScanChunk, NP = 4 * LN;
    constexpr int QUADS = T * CB / 4, QPT = (QUADS + kScanThreads - 1) / kScanThreads;
    __shared__ float2 s_dx[T][CB];  // delta, and what multiplies the matrix row
    __shared__ __align__(16) float s_m[T * NP], s_c[T * NP];
    __shared__ float s_y[REV ? 1 : T][CB];
    const int tid = threadIdx.x;
    const int64_t nblk = (g.kpg + CB - 1) / CB;
    const int grp = (int)(blockIdx.x / nblk);
    const int64_t c0 = (blockIdx.x - grp * nblk) * CB;       // first channel, within the group
    const int nch = (int)min64(CB, g.kpg - c0);
    const int64_t ch0 = grp * g.kpg + c0;
    const int64_t b = blockIdx.z, seg = a.first_seg + blockIdx.y;
    const int64_t nc = (g.seqlen + T - 1) / T;
    const int64_t cbeg = seg * a.chunks_per_seg, cend = min64(cbeg + a.chunks_per_seg, nc);
    // this thread's states
    const int c = tid / LN, n0 = 4 * (tid % LN);
    const int nn = c < nch ? (int)g.N - n0 : 0;  // live states (may exceed 4)
    const int64_t st = (ch0 + c) * g.N + n0;     // its place in a [dim][N] array
    float h[4] = {0.f, 0.f, 0.f, 0.f}, A2[4] = {0.f, 0.f, 0.f, 0.f}, dsum = 0.f;
    if (nn > 0) {
        load_states(a.A + st, nn, A2);
        if (a.start)
            load_states(a.start + (b * a.n_seg + seg) * g.dim * g.N + st, nn, h);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        A2[i] *= kLog2e;

    for (int64_t k = 0; k < cend - cbeg; ++k) {
        const int64_t chunk = REV ? cend - 1 - k : cbeg + k;
        const int64_t t0 = chunk * T;
        const int nt = (int)min64(T, g.seqlen - t0);
        Raw4<TI> xr[QPT], zr[QPT];
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int q = tid + i * kScanThreads;
            const int t = q / (CB / 4), cq = 4 * (q % (CB / 4));
            if (q >= QUADS)
                break;
            const int n = t < nt ? nch - cq : 0;
            const int64_t tok = b * g.seqlen + t0 + t;
            Raw4<TI> dr{};
            xr[i] = zr[i] = dr;
            if (n > 0) {
                xr[i] = load_raw4(a.x + tok * a.row_x + ch0 + cq, n, a.vec);
                dr = load_raw4(a.dt + tok * g.row_dt + ch0 + cq, n, a.vec);
                if (a.z)
                    zr[i] = load_raw4(a.z + tok * g.row_z + ch0 + cq, n, a.vec);
            }
            float xv[4], dv[4], zv[4];
            unpack<TI, 4>(xr[i], xv);
            unpack<TI, 4>(dr, dv);
            unpack<TI, 4>(zr[i], zv);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float d = 0.f, v = 0.f;
                if (e < n) {
                    d = dv[e] + (a.bias ? a.bias[ch0 + cq + e] : 0.f);
                    d = g.softplus ? softplus(d) : d;
                    v = REV ? (a.z ? xv[e] * fast_silu(zv[e]) : xv[e]) : d * xv[e];
                }
                s_dx[t][cq + e] = make_float2(d, v);
            }
        }
        const int64_t tok0 = b * g.seqlen + t0;
        load_rows<TI, LN>(a.m + tok0 * (REV ? g.row_c : g.row_b) + grp * g.N, REV ? g.row_c : g.row_b, nt,
                          (int)g.N, s_m);
        if (!REV && a.y)
            load_rows<TI, LN>(a.cm + tok0 * g.row_c + grp * g.N, g.row_c, nt, (int)g.N, s_c);
        __syncthreads();
        if (a.kept && nn > 0)
            store_states(a.kept + (b * nc + chunk) * g.dim * g.N + st, nn, h);
        for (int i = 0; i < nt; ++i) {
            const int t = REV ? nt - 1 - i : i;
            const float2 dx = s_dx[t][c];
            const float4 m = *reinterpret_cast<const float4 *>(&s_m[t * NP + n0]);
            const float mv[4] = {m.x, m.y, m.z, m.w};
            dsum += dx.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float d = ex2(dx.x * A2[e]);
                h[e] = REV ? d * fmaf(dx.y, mv[e], h[e]) : fmaf(d, h[e], dx.y * mv[e]);
            }
            if (!REV && a.y) {
                const float4 cv = *reinterpret_cast<const float4 *>(&s_c[t * NP + n0]);
                float s = h[0] * cv.x;
                s = fmaf(h[1], cv.y, s);
                s = fmaf(h[2], cv.z, s);
                s = fmaf(h[3], cv.w, s);
                s = lane_sum<LN>(s);
                if (n0 == 0)
                    s_y[REV ? 0 : t][c] = s;
            }
        }
        __syncthreads();
        if (!REV && a.y) {
#pragma unroll
            for (int i = 0; i < QPT; ++i) {
                const int q = tid + i * kScanThreads;
                const int t = q / (CB / 4), cq = 4 * (q % (CB / 4));
                if (q >= QUADS)
                    break;
                const int n = t < nt ? nch - cq : 0;
                if (n <= 0)
                    continue;
                float xv[4], zv[4], o[4];
                unpack<TI, 4>(xr[i], xv);
                unpack<TI, 4>(zr[i], zv);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    o[e] = s_y[REV ? 0 : t][cq + e];
                    if (a.D && e < n)
                        o[e] = fmaf(a.D[ch0 + cq + e], xv[e], o[e]);
                    if (a.z)
                        o[e] *= fast_silu(zv[e]);
                }
                store4(a.y + (b * g.seqlen + t0 + t) * g.dim + ch0 + cq, o, n, a.vec);
            }
        }
    }
    if (nn > 0) {
        if (a.last && (REV ? cbeg == 0 : cend == nc))
            store_states(a.last + b * g.dim * g.N + st, nn, h);
        if (a.seg_end) {
            store_states(a.seg_end + (b * a.n_seg + seg) * g.dim * g.N + st, nn, h);
            if (n0 == 0)
                a.seg_dsum[(b * a.n_seg + seg) * g.dim + ch0 + c] = dsum;
        }
    }
}

// Segment end states -> segment start states, in place, in the order of the
// pass: start' = exp(A dsum) start + end.
template <bool REV>
__global__ void __launch_bounds__(256)
scan_join_kernel(float *__restrict__ seg, const float *__restrict__ dsum, const float *__restrict__ A,
                 const float *start, int64_t batch, int64_t dim, int64_t N, int64_t n_seg)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t DN = dim * N;
    if (i >= batch * DN)
        return;
    const int64_t b = i / DN, r = i - b * DN, d = r / N;
    const float A2 = A[r] * kLog2e;
    float h = start ? start[i] : 0.f;
    for (int64_t k = 0; k < n_seg; ++k) {
        const int64_t s = b * n_seg + (REV ? n_seg - 1 - k : k);
        float end = 0.f, q = 0.f;
        if (k < n_seg - 1) {  // the last segment's end is not needed (nor computed)
            end = seg[s * DN + r];
            q = dsum[s * dim + d];
        }
        seg[s * DN + r] = h;
        h = fmaf(ex2(A2 * q), h, end);
    }
}

// One token: four states of a channel per thread, LN lanes per channel.
template <typename TI, int LN>
__global__ void __launch_bounds__(256)
scan_step_kernel(const TI *__restrict__ u, const TI *__restrict__ dt, const float *__restrict__ A,
                 const TI *__restrict__ Bm, const TI *__restrict__ Cm, const float *__restrict__ D,
                 const TI *__restrict__ z, const float *__restrict__ bias, const float *state,
                 float *state_out, TI *__restrict__ y, ScanGeom g)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t bd = i / LN;
    const int n0 = 4 * (int)(i % LN);
    const bool live = bd < g.batch * g.dim;
    const int64_t b = live ? bd / g.dim : 0, d = live ? bd - b * g.dim : 0;
    const int nn = live ? (int)g.N - n0 : 0;
    const int64_t grp = d / g.kpg;
    float s = 0.f, uv = 0.f;
    if (nn > 0) {
        float h[4], av[4], bv[4], cv[4];
        load_states(state + bd * g.N + n0, nn, h);
        load_states(A + d * g.N + n0, nn, av);
        uv = to_f32(u[b * g.row_u + d]);
        float dl = to_f32(dt[b * g.row_dt + d]) + (bias ? bias[d] : 0.f);
        dl = g.softplus ? softplus(dl) : dl;
        const TI *bp = Bm + b * g.row_b + grp * g.N + n0, *cp = Cm + b * g.row_c + grp * g.N + n0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bv[e] = e < nn ? to_f32(bp[e]) : 0.f;
            cv[e] = e < nn ? to_f32(cp[e]) : 0.f;
        }
        const float du = dl * uv;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[e] = fmaf(ex2(dl * (av[e] * kLog2e)), h[e], du * bv[e]);
            s = fmaf(h[e], cv[e], s);
        }
        store_states(state_out + bd * g.N + n0, nn, h);
    }
    s = lane_sum<LN>(s);
    if (live && n0 == 0) {
        if (D)
            s = fmaf(D[d], uv, s);
        if (z)
            s *= fast_silu(to_f32(z[b * g.row_z + d]));
        y[bd] = from_f32<TI>(s);
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename TI, bool REV>
cudaError_t launch_pass(const PassArgs<TI> &a, const ScanGeom &g, int64_t segs, cudaStream_t st)
{
    const int LN = scan_lanes(g.N);
    const int64_t CB = kScanThreads / LN;
    const dim3 grid((unsigned)(g.G * ((g.kpg + CB - 1) / CB)), (unsigned)segs, (unsigned)g.batch);
    switch (LN) {
    case 1: scan_pass_kernel<TI, 1, REV><<<grid, kScanThreads, 0, st>>>(a, g); break;
    case 2: scan_pass_kernel<TI, 2, REV><<<grid, kScanThreads, 0, st>>>(a, g); break;
    case 4: scan_pass_kernel<TI, 4, REV><<<grid, kScanThreads, 0, st>>>(a, g); break;
    case 8: scan_pass_kernel<TI, 8, REV><<<grid, kScanThreads, 0, st>>>(a, g); break;
    default: scan_pass_kernel<TI, 16, REV><<<grid, kScanThreads, 0, st>>>(a, g); break;
    }
    note_launch(1);
    return cudaGetLastError();
}

// Runs a pass, in segments where the channels alone cannot fill the GPU: the
// segments' end states from zero, their join, then all segments at once.
template <typename TI, bool REV>
cudaError_t run_pass(PassArgs<TI> a, const float *start, void *ws, const ScanGeom &g, cudaStream_t st)
{
    const ScanSegs sp = scan_segments(g);
    a.chunks_per_seg = sp.chunks_per_seg;
    a.n_seg = sp.n_seg;
    a.first_seg = 0;
    a.seg_end = a.seg_dsum = nullptr;
    a.start = start;
    if (sp.n_seg > 1) {
        float *seg = static_cast<float *>(ws);
        float *dsum = seg + g.batch * sp.n_seg * g.dim * g.N;
        PassArgs<TI> e = a;
        e.start = nullptr;
        e.y = nullptr;
        e.last = e.kept = nullptr;
        e.seg_end = seg;
        e.seg_dsum = dsum;
        e.first_seg = REV ? 1 : 0;
        cudaError_t err = launch_pass<TI, REV>(e, g, sp.n_seg - 1, st);
        if (err != cudaSuccess)
            return err;
        const int64_t n = g.batch * g.dim * g.N;
        scan_join_kernel<REV><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(seg, dsum, a.A, start, g.batch, g.dim,
                                                                         g.N, sp.n_seg);
        note_launch(1);
        err = cudaGetLastError();
        if (err != cudaSuccess)
            return err;
        a.start = seg;
    }
    return launch_pass<TI, REV>(a, g, sp.n_seg, st);
}

bool quads_ok(const ScanGeom &g, const void *x, int64_t row_x, const void *dt, const void *z, const void *y,
              size_t esz)
{
    const size_t a = 4 * esz;
    return (g.kpg % 4 == 0 || g.G == 1) && g.dim % 4 == 0 && row_x % 4 == 0 && g.row_dt % 4 == 0 &&
           (!z || g.row_z % 4 == 0) && aligned(x, a) && aligned(dt, a) && aligned(z, a) && aligned(y, a);
}

template <typename TI>
cudaError_t fwd_t(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                  const float *D, const void *z, const float *bias, const float *init, void *y, float *fin,
                  float *kept, void *ws, const ScanGeom &g, cudaStream_t st)
{
    PassArgs<TI> a{};
    a.x = static_cast<const TI *>(u);
    a.dt = static_cast<const TI *>(dt);
    a.z = y ? static_cast<const TI *>(z) : nullptr;
    a.m = static_cast<const TI *>(Bm);
    a.cm = static_cast<const TI *>(Cm);
    a.A = A;
    a.D = D;
    a.bias = bias;
    a.y = static_cast<TI *>(y);
    a.last = fin;
    a.kept = kept;
    a.row_x = g.row_u;
    a.vec = quads_ok(g, u, g.row_u, dt, a.z, y, sizeof(TI));
    return run_pass<TI, false>(a, init, ws, g, st);
}

template <typename TI>
cudaError_t rev_t(const void *dy, const void *dt, const float *A, const void *Cm, const void *z,
                  const float *bias, const float *dfinal, float *dkept, float *dinit, void *ws,
                  const ScanGeom &g, cudaStream_t st)
{
    PassArgs<TI> a{};
    a.x = static_cast<const TI *>(dy);
    a.dt = static_cast<const TI *>(dt);
    a.z = static_cast<const TI *>(z);
    a.m = static_cast<const TI *>(Cm);
    a.A = A;
    a.bias = bias;
    a.last = dinit;
    a.kept = dkept;
    a.row_x = g.row_dy;
    a.vec = quads_ok(g, dy, g.row_dy, dt, z, nullptr, sizeof(TI));
    return run_pass<TI, true>(a, dfinal, ws, g, st);
}

template <typename TI>
cudaError_t step_t(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *D,
                   const void *z, const float *bias, const float *state, float *state_out, void *y,
                   const ScanGeom &g, cudaStream_t st)
{
    const int LN = scan_lanes(g.N);
    const unsigned blocks = (unsigned)((g.batch * g.dim * LN + 255) / 256);
#define SSD_STEP(LANES)                                                                              \
    scan_step_kernel<TI, LANES><<<blocks, 256, 0, st>>>(                                             \
        static_cast<const TI *>(u), static_cast<const TI *>(dt), A, static_cast<const TI *>(Bm),     \
        static_cast<const TI *>(Cm), D, static_cast<const TI *>(z), bias, state, state_out,          \
        static_cast<TI *>(y), g)
    switch (LN) {
    case 1: SSD_STEP(1); break;
    case 2: SSD_STEP(2); break;
    case 4: SSD_STEP(4); break;
    case 8: SSD_STEP(8); break;
    default: SSD_STEP(16); break;
    }
#undef SSD_STEP
    note_launch(1);
    return cudaGetLastError();
}

}  // namespace

int scan_lanes(int64_t N)
{
    int l = 1;
    while (4 * l < N)
        l *= 2;
    return l;
}

int scan_chunk() { return kScanChunk; }

// Segments of a pass: one where the channel blocks give every SM several
// blocks; else enough segments (of at least four chunks) to do so.
ScanSegs scan_segments(const ScanGeom &g)
{
    const int64_t CB = kScanThreads / scan_lanes(g.N);
    const int64_t blocks = g.G * ((g.kpg + CB - 1) / CB) * g.batch;
    const int64_t nc = (g.seqlen + kScanChunk - 1) / kScanChunk;
    const int64_t want = (int64_t)device_sm_count() * 3;
    ScanSegs s{1, nc};
    if (blocks < want) {
        int64_t n = (2 * want + blocks - 1) / blocks;
        n = min64(n, nc / 4);
        if (n > 1) {
            s.chunks_per_seg = (nc + n - 1) / n;
            s.n_seg = (nc + s.chunks_per_seg - 1) / s.chunks_per_seg;
        }
    }
    return s;
}

size_t scan_pass_workspace(const ScanGeom &g)
{
    const ScanSegs s = scan_segments(g);
    return s.n_seg > 1 ? (size_t)(g.batch * s.n_seg * g.dim * (g.N + 1)) * sizeof(float) : 0;
}

cudaError_t launch_selective_scan(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                                  const float *D, const void *z, const float *bias, const float *init, void *y,
                                  float *fin, float *kept, void *ws, const ScanGeom &g, bool bf16,
                                  cudaStream_t st)
{
    return bf16 ? fwd_t<__nv_bfloat16>(u, dt, A, Bm, Cm, D, z, bias, init, y, fin, kept, ws, g, st)
                : fwd_t<float>(u, dt, A, Bm, Cm, D, z, bias, init, y, fin, kept, ws, g, st);
}

cudaError_t launch_scan_reverse(const void *dy, const void *dt, const float *A, const void *Cm, const void *z,
                                const float *bias, const float *dfinal, float *dkept, float *dinit, void *ws,
                                const ScanGeom &g, bool bf16, cudaStream_t st)
{
    return bf16 ? rev_t<__nv_bfloat16>(dy, dt, A, Cm, z, bias, dfinal, dkept, dinit, ws, g, st)
                : rev_t<float>(dy, dt, A, Cm, z, bias, dfinal, dkept, dinit, ws, g, st);
}

cudaError_t launch_scan_step(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                             const float *D, const void *z, const float *bias, const float *state,
                             float *state_out, void *y, const ScanGeom &g, bool bf16, cudaStream_t st)
{
    return bf16 ? step_t<__nv_bfloat16>(u, dt, A, Bm, Cm, D, z, bias, state, state_out, y, g, st)
                : step_t<float>(u, dt, A, Bm, Cm, D, z, bias, state, state_out, y, g, st);
}

}  // namespace ssd
