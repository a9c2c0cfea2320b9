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
// dB and dC are sums over the group's channels.  A thread owns four states of
// two adjacent channels and walks a chunk in pieces of kPiece tokens, last to
// first: forward through the piece from its start state (kept in shared memory
// by a first walk over the chunk) holding each token's a and a h, then back.  Its
// parts of dB and dC are added over the block's threads in shared memory once
// a piece and written as one partial per channel block; a last kernel adds
// those in a fixed order (no atomics, so results do not depend on scheduling).
// 2 x 4096 tokens of 5120 channels and 16 states take 825 us on a GB300; the
// shared memory pipe (75 passes for a warp's 256 entries a token) is 76% busy,
// issue slots (207) 53%.  With the start states, B, C and the piece's sums in
// registers (255, two blocks an SM instead of three) it took 1010 us, and with
// the pieces unrolled, which overran the instruction cache, 950 us.
#include "scan.cuh"

namespace ssd {
namespace {

constexpr int kPiece = 4;      // tokens whose a and a h a thread holds
constexpr int kGradThreads = 128;

template <typename TI> struct GradArgs {
    const TI *u, *dt, *bm, *cm, *z, *dy;
    const float *A, *D, *bias, *h0, *g1;
    TI *du, *ddt, *dz;
    float *dB, *dC;        // [channel blocks][B * L][N]
    float *dA;             // [B * chunk groups][dim][N]
    float *dD;             // [B * chunk groups][2][dim]: dD, dbias
    ScanEnter enter;
    int64_t chunks_per_group;
    bool vec, vec_bc, vec_st;
};

template <typename TI, int LN> struct GradTile {
    static constexpr int CB = 2 * kGradThreads / LN, NP = 4 * LN;
    static constexpr int CP = kGradThreads / LN;  // channel pairs
    static constexpr int PLANE = kPiece * CB + (LN > 4 ? 4 : 8);
    // One sum's terms are a row of red, CP wide.  Terms are placed by XOR so that
    // a warp's channel pairs and lanes store to different banks, and eight
    // threads' quads of rows are read from different ones.
    static constexpr int PAIRS = 32 / LN, ROWS_SHIFT = LN == 8 ? 1 : LN == 16 ? 2 : 0;
    static __device__ int term(int cp, int lane) { return cp ^ PAIRS * (lane >> ROWS_SHIFT); }
    static __device__ int quad(int i, int row) { return 4 * (i ^ ((row >> ROWS_SHIFT) & (CP / 4 - 1) & 7)); }
    struct Raw {
        TI u[kScanChunk][CB], dt[kScanChunk][CB], z[kScanChunk][CB], dy[kScanChunk][CB];
        TI m[kScanChunk][NP], c[kScanChunk][NP];
    } raw[2];                           // as loaded: this chunk and the next
    float2 dx[kScanChunk][CB];          // delta, delta u
    float dyy[kScanChunk][CB];          // dout silu(z)
    float m[kScanChunk * NP], c[kScanChunk * NP];
    float bias[CB], D[CB];
    float part[3][LN * PLANE];          // each lane's part of sum C h, sum e B, sum q A
    float red[2 * kPiece * NP * CP];    // each channel pair's part of dB, dC
    ulonglong2 hs[kScanChunk / kPiece - 1][2][kGradThreads];  // states entering the pieces but the first
};

// Blocks an SM holds: as shared memory allows, up to three, which leave a
// thread 168 registers.
template <typename TI, int LN> constexpr int grad_blocks()
{
    constexpr int n = 228 * 1024 / (sizeof(GradTile<TI, LN>) + 1024);
    return n < 3 ? n : 3;
}

template <typename TI, int LN>
__global__ void __launch_bounds__(kGradThreads, grad_blocks<TI, LN>()) scan_grad_kernel(GradArgs<TI> a, ScanGeom g)
{
    using Tile = GradTile<TI, LN>;
    constexpr int NT = kGradThreads, CB = Tile::CB, CP = Tile::CP, T = kScanChunk, NP = 4 * LN;
    // elementwise work: columns of four channels, TROWS tokens apart
    constexpr int COLS = CB / 4, TROWS = NT / COLS;
    // a piece's results: PW channels of a token; where a piece has fewer of those
    // than the block threads, TPQ share one and each adds up LN / TPQ lanes' parts
    constexpr int PW = LN <= 2 ? 4 : 2, PCOLS = CB / PW;
    constexpr int TPQ = LN > 4 ? LN / 4 : 1, RROWS = NT / TPQ / PCOLS;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Tile &s = *reinterpret_cast<Tile *>(smem_raw);
    const int tid = threadIdx.x;
    const int64_t nblk = (g.kpg + CB - 1) / CB;
    const int grp = (int)(blockIdx.x / nblk);
    const int64_t c0 = (blockIdx.x - grp * nblk) * CB;
    const int nch = (int)min64(CB, g.kpg - c0);
    const int64_t ch0 = grp * g.kpg + c0;
    const int64_t b = blockIdx.z;
    const int64_t nc = (g.seqlen + T - 1) / T;
    const int64_t cbeg = blockIdx.y * a.chunks_per_group, cend = min64(cbeg + a.chunks_per_group, nc);
    const int N = (int)g.N;
    const int cp = tid / LN, c = 2 * cp, n0 = 4 * (tid % LN);
    const int col = 4 * (tid % COLS), trow = tid / COLS, nq = nch - col;
    const int pcol = PW * (tid / TPQ % PCOLS), prow = tid / TPQ / PCOLS, np = nch - pcol;

    f32x2 A[2][2] = {}, dA[2][2] = {};
    int nn[2];
    const int64_t st = (ch0 + c) * g.N + n0;  // the thread's place in a [dim][N] array
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        nn[j] = c + j < nch ? N - n0 : 0;
        if (nn[j] > 0) {
            float v[4];
            load_states(a.A + st + j * g.N, nn[j], v);
            A[j][0] = pk2(decay_rate(v[0]), decay_rate(v[1]));
            A[j][1] = pk2(decay_rate(v[2]), decay_rate(v[3]));
        }
    }
    float accD[PW] = {}, accb[PW] = {};
    for (int i = tid; i < CB; i += NT) {
        s.bias[i] = a.bias && i < nch ? a.bias[ch0 + i] : 0.f;
        s.D[i] = a.D && i < nch ? a.D[ch0 + i] : 0.f;
    }

    // the chunk's inputs into raw[w]; elements past the tokens, channels and
    // states are zero
    auto fetch = [&](int64_t chunk, int w) {
        const int64_t tok0 = b * g.seqlen + chunk * T;
        const int nt = (int)min64(T, g.seqlen - chunk * T);
        typename Tile::Raw &r = s.raw[w];
#pragma unroll 1
        for (int t = trow; t < T; t += TROWS) {
            const int64_t tok = tok0 + t;
            if (a.vec && nq >= 4 && t < nt) {
                copy_async<4 * sizeof(TI)>(&r.u[t][col], a.u + tok * g.row_u + ch0 + col);
                copy_async<4 * sizeof(TI)>(&r.dt[t][col], a.dt + tok * g.row_dt + ch0 + col);
                copy_async<4 * sizeof(TI)>(&r.dy[t][col], a.dy + tok * g.row_dy + ch0 + col);
                if (a.z)
                    copy_async<4 * sizeof(TI)>(&r.z[t][col], a.z + tok * g.row_z + ch0 + col);
            } else if (nq >= 4 && t < nt) {  // rows off the quads' boundaries
                const Raw4<TI> ur = load_four(a.u + tok * g.row_u + ch0 + col);
                const Raw4<TI> dr = load_four(a.dt + tok * g.row_dt + ch0 + col);
                const Raw4<TI> yr = load_four(a.dy + tok * g.row_dy + ch0 + col);
                if (a.z)
                    *reinterpret_cast<Raw4<TI> *>(&r.z[t][col]) = load_four(a.z + tok * g.row_z + ch0 + col);
                *reinterpret_cast<Raw4<TI> *>(&r.u[t][col]) = ur;
                *reinterpret_cast<Raw4<TI> *>(&r.dt[t][col]) = dr;
                *reinterpret_cast<Raw4<TI> *>(&r.dy[t][col]) = yr;
            } else {
                const int n = t < nt ? nq : 0;
                *reinterpret_cast<Raw4<TI> *>(&r.u[t][col]) = load_raw4(a.u + tok * g.row_u + ch0 + col, n, false);
                *reinterpret_cast<Raw4<TI> *>(&r.dt[t][col]) = load_raw4(a.dt + tok * g.row_dt + ch0 + col, n, false);
                *reinterpret_cast<Raw4<TI> *>(&r.dy[t][col]) = load_raw4(a.dy + tok * g.row_dy + ch0 + col, n, false);
                if (a.z)
                    *reinterpret_cast<Raw4<TI> *>(&r.z[t][col]) =
                        load_raw4(a.z + tok * g.row_z + ch0 + col, n, false);
            }
        }
        for (int i = tid; i < 2 * T * LN; i += NT) {
            const int q = i / (T * LN), t = i / LN % T, n = 4 * (i % LN);
            TI *dst = q ? &r.c[t][n] : &r.m[t][n];
            const TI *src = (q ? a.cm + (tok0 + t) * g.row_c : a.bm + (tok0 + t) * g.row_b) + grp * g.N + n;
            if (a.vec_bc && t < nt && N - n >= 4)
                copy_async<4 * sizeof(TI)>(dst, src);
            else
                *reinterpret_cast<Raw4<TI> *>(dst) = load_raw4(src, t < nt ? N - n : 0, false);
        }
        copy_async_commit();
    };

    // the thread's four states of channel j at p
    auto quad = [&](const float *p, int j, f32x2 (&o)[2]) {
        if (a.vec_st) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(p + j * NP);
            o[0] = v.x;
            o[1] = v.y;
        } else {
            float v[4];
            load_states(p + j * g.N, nn[j], v);
            o[0] = pk2(v[0], v[1]);
            o[1] = pk2(v[2], v[3]);
        }
    };
    const int64_t dn = g.dim * g.N;
    int64_t kept = (b * nc + cbeg) * dn + st;
    fetch(cbeg, 0);
    for (int64_t chunk = cbeg; chunk < cend; ++chunk, kept += dn) {
        const int w = (int)(chunk - cbeg) & 1;
        const int nt = (int)min64(T, g.seqlen - chunk * T);
        const int64_t tok0 = b * g.seqlen + chunk * T;
        // the state entering the chunk and the gradient leaving it
        f32x2 h0[2][2] = {}, e[2][2] = {}, in[2][2] = {};
        float after[2] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (nn[j] > 0) {
                quad(a.h0 + kept, j, h0[j]);
                quad(a.g1 + kept, j, e[j]);
            }
        if (a.enter.state) {  // and what entered the reverse pass's segment, decayed to here
            const float *pe = a.enter.state +
                              (b * a.enter.n_seg + (unsigned)chunk / (unsigned)a.enter.chunks_per_seg) * dn + st;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (nn[j] > 0) {
                    quad(pe, j, in[j]);
                    after[j] = a.enter.after[(b * nc + chunk) * g.dim + ch0 + c + j];
                }
        }
        copy_async_wait<0>();
        __syncthreads();  // raw[w] is complete, and the chunk before is done with everything
        if (chunk + 1 < cend)
            fetch(chunk + 1, w ^ 1);
        const typename Tile::Raw &r = s.raw[w];
#pragma unroll 1
        for (int t = trow; t < T; t += TROWS) {
            float uv[4], dv[4], zv[4], yv[4], bias[4], o[8];
            load_vec<float, 4>(&s.bias[col], bias);
            load_vec<TI, 4>(&r.u[t][col], uv);
            load_vec<TI, 4>(&r.dt[t][col], dv);
            load_vec<TI, 4>(&r.dy[t][col], yv);
            if (a.z)
                load_vec<TI, 4>(&r.z[t][col], zv);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float d0 = dv[i] + bias[i], d1 = dv[i + 1] + bias[i + 1];
                if (g.softplus)
                    softplus2(d0, d1, d0, d1);
                if (nt < T || nq < 4) {
                    d0 = t < nt && i < nq ? d0 : 0.f;
                    d1 = t < nt && i + 1 < nq ? d1 : 0.f;
                }
                o[2 * i] = d0;
                o[2 * i + 2] = d1;
                un2(mul2(pk2(d0, d1), pk2(uv[i], uv[i + 1])), o[2 * i + 1], o[2 * i + 3]);
                if (a.z) {
                    const f32x2 z = pk2(zv[i], zv[i + 1]);
                    un2(mul2(pk2(yv[i], yv[i + 1]), mul2(z, sigmoid2(z))), yv[i], yv[i + 1]);
                }
            }
            *reinterpret_cast<float4 *>(&s.dx[t][col]) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4 *>(&s.dx[t][col + 2]) = make_float4(o[4], o[5], o[6], o[7]);
            store_vec<float, 4>(&s.dyy[t][col], yv);
        }
        for (int i = tid; i < 2 * T * LN; i += NT) {
            const int q = i / (T * LN), k = 4 * (i % (T * LN));
            float v[4];
            load_vec<TI, 4>((q ? &r.c[0][0] : &r.m[0][0]) + k, v);
            store_vec<float, 4>((q ? s.c : s.m) + k, v);
        }
        __syncthreads();

        const f32x2 nudge = dup2(kDecayNudge);
        if (a.enter.state) {
            float x[2][4], most = 0.f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x2 q = dup2(after[j]);
                un2(mul2(q, A[j][0]), x[j][0], x[j][1]);
                un2(mul2(q, A[j][1]), x[j][2], x[j][3]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    most = fmaxf(most, x[j][k]);
            }
            if (most <= kLargeExponent) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    e[j][0] = fma2(pk2(ex2(x[j][0]), ex2(x[j][1])), in[j][0], e[j][0]);
                    e[j][1] = fma2(pk2(ex2(x[j][2]), ex2(x[j][3])), in[j][1], e[j][1]);
                }
            } else {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float v[2], o[2];
                        un2(in[j][k], v[0], v[1]);
                        un2(e[j][k], o[0], o[1]);
                        e[j][k] = pk2(add_scaled(x[j][2 * k], v[0], o[0]), add_scaled(x[j][2 * k + 1], v[1], o[1]));
                    }
            }
        }
        // a walk to each piece's start state
        constexpr int PIECES = T / kPiece;
        {
            f32x2 h[2][2] = {{h0[0][0], h0[0][1]}, {h0[1][0], h0[1][1]}};
#pragma unroll 1
            for (int p = 1; p < PIECES; ++p) {
#pragma unroll
                for (int i = 0; i < kPiece; ++i) {
                    const int t = (p - 1) * kPiece + i;
                    const float4 dx = *reinterpret_cast<const float4 *>(&s.dx[t][c]);
                    const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(&s.m[t * NP + n0]);
                    const f32x2 dl[2] = {dup2(dx.x), dup2(dx.z)}, xv[2] = {dup2(dx.y), dup2(dx.w)};
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        h[j][0] = fma2(ex2_2(fma2(dl[j], A[j][0], nudge)), h[j][0], mul2(xv[j], m.x));
                        h[j][1] = fma2(ex2_2(fma2(dl[j], A[j][1], nudge)), h[j][1], mul2(xv[j], m.y));
                    }
                }
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    s.hs[p - 1][j][tid] = make_ulonglong2(h[j][0], h[j][1]);
            }
        }

#pragma unroll 1
        for (int p = PIECES - 1; p >= 0; --p) {
            const int t0 = p * kPiece;
            f32x2 av[kPiece][2][2], ah[kPiece][2][2];
            f32x2 h[2][2] = {{h0[0][0], h0[0][1]}, {h0[1][0], h0[1][1]}};
            if (p > 0)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const ulonglong2 v = s.hs[p - 1][j][tid];
                    h[j][0] = v.x;
                    h[j][1] = v.y;
                }
            // a token's parts of dB and dC: red[which][token][state % 4][lane][channel pair]
            auto put = [&](int which, int i, f32x2 v0, f32x2 v1) {
                float v[4];
                un2(v0, v[0], v[1]);
                un2(v1, v[2], v[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    s.red[(((which * kPiece + i) * 4 + k) * LN + tid % LN) * CP + Tile::term(cp, tid % LN)] = v[k];
            };
#pragma unroll
            for (int i = 0; i < kPiece; ++i) {
                const int t = t0 + i;
                const float4 dx = *reinterpret_cast<const float4 *>(&s.dx[t][c]);
                const float2 dyy = *reinterpret_cast<const float2 *>(&s.dyy[t][c]);
                const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(&s.m[t * NP + n0]);
                const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(&s.c[t * NP + n0]);
                const f32x2 dl[2] = {dup2(dx.x), dup2(dx.z)}, xv[2] = {dup2(dx.y), dup2(dx.w)};
                const f32x2 yv[2] = {dup2(dyy.x), dup2(dyy.y)};
                float y[2];
                f32x2 dC[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    av[i][j][0] = ex2_2(fma2(dl[j], A[j][0], nudge));
                    av[i][j][1] = ex2_2(fma2(dl[j], A[j][1], nudge));
                    ah[i][j][0] = mul2(av[i][j][0], h[j][0]);
                    ah[i][j][1] = mul2(av[i][j][1], h[j][1]);
                    h[j][0] = fma2(xv[j], m.x, ah[i][j][0]);
                    h[j][1] = fma2(xv[j], m.y, ah[i][j][1]);
                    dC[0] = j ? fma2(yv[j], h[j][0], dC[0]) : mul2(yv[j], h[j][0]);
                    dC[1] = j ? fma2(yv[j], h[j][1], dC[1]) : mul2(yv[j], h[j][1]);
                    y[j] = hsum(fma2(h[j][1], cv.y, mul2(h[j][0], cv.x)));
                }
                put(1, i, dC[0], dC[1]);
                if (a.z)
                    *reinterpret_cast<float2 *>(&s.part[0][(tid % LN) * Tile::PLANE + i * CB + c]) =
                        make_float2(y[0], y[1]);
            }
#pragma unroll
            for (int i = kPiece - 1; i >= 0; --i) {
                const int t = t0 + i;
                const float4 dx = *reinterpret_cast<const float4 *>(&s.dx[t][c]);
                const float2 dyy = *reinterpret_cast<const float2 *>(&s.dyy[t][c]);
                const f32x2 dl[2] = {dup2(dx.x), dup2(dx.z)}, xv[2] = {dup2(dx.y), dup2(dx.w)};
                const f32x2 yv[2] = {dup2(dyy.x), dup2(dyy.y)};
                const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(&s.m[t * NP + n0]);
                const ulonglong2 cv = *reinterpret_cast<const ulonglong2 *>(&s.c[t * NP + n0]);
                float sB[2], sA[2];
                f32x2 dB[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    e[j][0] = fma2(yv[j], cv.x, e[j][0]);
                    e[j][1] = fma2(yv[j], cv.y, e[j][1]);
                    dB[0] = j ? fma2(e[j][0], xv[j], dB[0]) : mul2(e[j][0], xv[j]);
                    dB[1] = j ? fma2(e[j][1], xv[j], dB[1]) : mul2(e[j][1], xv[j]);
                    sB[j] = hsum(fma2(e[j][1], m.y, mul2(e[j][0], m.x)));
                    const f32x2 q0 = mul2(e[j][0], ah[i][j][0]), q1 = mul2(e[j][1], ah[i][j][1]);
                    dA[j][0] = fma2(q0, dl[j], dA[j][0]);
                    dA[j][1] = fma2(q1, dl[j], dA[j][1]);
                    sA[j] = hsum(fma2(q1, A[j][1], mul2(q0, A[j][0])));
                    e[j][0] = mul2(e[j][0], av[i][j][0]);
                    e[j][1] = mul2(e[j][1], av[i][j][1]);
                }
                put(0, i, dB[0], dB[1]);
                const int at = (tid % LN) * Tile::PLANE + i * CB + c;
                *reinterpret_cast<float2 *>(&s.part[1][at]) = make_float2(sB[0], sB[1]);
                *reinterpret_cast<float2 *>(&s.part[2][at]) = make_float2(sA[0], sA[1]);
            }
            __syncthreads();
            for (int o = tid; o < 2 * kPiece * NP; o += NT) {
                const int t = t0 + o / NP % kPiece, n = 4 * (o % LN) + o / LN % 4;
                const float *q = s.red + o * CP;
                f32x2 v0 = 0, v1 = 0;
#pragma unroll
                for (int i = 0; i < CP / 4; ++i) {
                    const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(q + Tile::quad(i, o));
                    v0 = add2(v0, x.x);
                    v1 = add2(v1, x.y);
                }
                if (t < nt && n < N) {
                    float *out = o < kPiece * NP ? a.dB : a.dC;
                    out[((int64_t)blockIdx.x * g.batch * g.seqlen + tok0 + t) * g.N + n] = hsum(add2(v0, v1));
                }
            }
            // per (token, channel) results of the piece
#pragma unroll
            for (int i = prow; i < kPiece; i += RROWS) {
                const int t = t0 + i;
                f32x2 sum[3][PW / 2];
#pragma unroll
                for (int k = 0; k < 3; ++k) {
                    const float *q = &s.part[k][tid % TPQ * Tile::PLANE + i * CB + pcol];
#pragma unroll
                    for (int h = 0; h < PW / 2; ++h)
                        sum[k][h] = 0;
#pragma unroll
                    for (int j = 0; j < LN; j += TPQ) {
                        float v[PW];
                        load_vec<float, PW>(q + j * Tile::PLANE, v);
#pragma unroll
                        for (int h = 0; h < PW / 2; ++h)
                            sum[k][h] = j ? add2(sum[k][h], pk2(v[2 * h], v[2 * h + 1])) : pk2(v[2 * h], v[2 * h + 1]);
                    }
#pragma unroll
                    for (int o = 1; o < TPQ; o *= 2)
#pragma unroll
                        for (int h = 0; h < PW / 2; ++h)
                            sum[k][h] = add2(sum[k][h], __shfl_xor_sync(0xffffffffu, sum[k][h], o));
                }
                if (t >= nt || np <= 0 || tid % TPQ)
                    continue;
                float uv[PW], dv[PW], zv[PW], yv[PW], du[PW], ddt[PW], dz[PW], dyy[PW], bias[PW], Dv[PW], dx[2 * PW];
                load_vec<TI, PW>(&r.u[t][pcol], uv);
                load_vec<TI, PW>(&r.dt[t][pcol], dv);
                load_vec<float, PW>(&s.dyy[t][pcol], dyy);
                load_vec<float, PW>(&s.bias[pcol], bias);
                load_vec<float, PW>(&s.D[pcol], Dv);
                load_vec<float, 4>(&s.dx[t][pcol].x, *reinterpret_cast<float(*)[4]>(dx));
                if constexpr (PW == 4)
                    load_vec<float, 4>(&s.dx[t][pcol + 2].x, *reinterpret_cast<float(*)[4]>(dx + 4));
                if (a.z) {
                    load_vec<TI, PW>(&r.z[t][pcol], zv);
                    load_vec<TI, PW>(&r.dy[t][pcol], yv);
                }
#pragma unroll
                for (int k = 0; k < PW; k += 2) {
                    const f32x2 Dp = pk2(Dv[k], Dv[k + 1]), up = pk2(uv[k], uv[k + 1]);
                    const f32x2 gp = pk2(dyy[k], dyy[k + 1]);
                    const f32x2 sB = sum[1][k / 2];
                    un2(fma2(pk2(dx[2 * k], dx[2 * k + 2]), sB, mul2(Dp, gp)), du[k], du[k + 1]);
                    f32x2 d = fma2(sum[2][k / 2], dup2(kLn2), mul2(up, sB));
                    if (g.softplus)
                        d = mul2(d, sigmoid2(pk2(dv[k] + bias[k], dv[k + 1] + bias[k + 1])));
                    un2(d, ddt[k], ddt[k + 1]);
                    if (a.z) {
                        const f32x2 z = pk2(zv[k], zv[k + 1]);
                        const f32x2 y = fma2(Dp, up, sum[0][k / 2]);
                        un2(mul2(mul2(pk2(yv[k], yv[k + 1]), y), silu_grad2(z, sigmoid2(z))), dz[k], dz[k + 1]);
                    }
                }
#pragma unroll
                for (int k = 0; k < PW; ++k)
                    if (k < np) {
                        accD[k] = fmaf(dyy[k], uv[k], accD[k]);
                        accb[k] += ddt[k];
                    }
                const int64_t at = (tok0 + t) * g.dim + ch0 + pcol;
                store_some<TI, PW>(a.du + at, du, np, a.vec);
                store_some<TI, PW>(a.ddt + at, ddt, np, a.vec);
                if (a.z)
                    store_some<TI, PW>(a.dz + at, dz, np, a.vec);
            }
            __syncthreads();  // red and part may be written again
        }
    }
    // this block's partial sums over its tokens
    const int64_t item = b * gridDim.y + blockIdx.y;
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (nn[j] > 0) {
            float v[4];
            un2(dA[j][0], v[0], v[1]);
            un2(dA[j][1], v[2], v[3]);
            store_states(a.dA + item * g.dim * g.N + st + j * g.N, nn[j], v);
        }
    float *red = s.red;  // [RROWS][2][CB]
    if (tid % TPQ == 0)
#pragma unroll
        for (int k = 0; k < PW; ++k) {
            red[(prow * 2) * CB + pcol + k] = accD[k];
            red[(prow * 2 + 1) * CB + pcol + k] = accb[k];
        }
    __syncthreads();
    for (int i = tid; i < 2 * CB; i += NT) {
        const int which = i / CB, k = i % CB;
        float v = 0.f;
        for (int q = 0; q < RROWS; ++q)
            v += red[(q * 2 + which) * CB + k];
        if (k < nch)
            a.dD[(item * 2 + which) * g.dim + ch0 + k] = v;
    }
}

// Adds the partials in a fixed order.  The first 2 G bc_blocks blocks add the
// groups' channel blocks, out[t][grp][n] = sum_k src[grp nblk + k][t][n] (dB of
// the first group, its dC, dB of the second, ...), four values a thread where
// V = 4 (dstate a multiple of four); the next a_blocks add dA over the items,
// then d_blocks each dD and dbias (nullptr: not wanted), 32 values a block.
template <typename TI> struct ScanSums {
    const float *bc[2], *item[3];
    TI *bc_out[2];
    float *item_out[3];
    int64_t tokens, N, G, nblk, dim, items;
    unsigned bc_blocks, a_blocks, d_blocks;
};
constexpr int kSumThreads = 512;
template <typename TI, int V> __global__ void __launch_bounds__(kSumThreads) scan_sums_kernel(ScanSums<TI> a)
{
    const unsigned first = 2 * (unsigned)a.G * a.bc_blocks;
    if (blockIdx.x < first) {
        const unsigned y = blockIdx.x / a.bc_blocks, x = blockIdx.x - y * a.bc_blocks;
        const int64_t i = ((int64_t)x * kSumThreads + threadIdx.x) * V;
        const int64_t stride = a.tokens * a.N;
        if (i >= stride)
            return;
        const int64_t grp = y / 2;
        const float *p = a.bc[y & 1] + grp * a.nblk * stride + i;
        float s[V] = {};
#pragma unroll 8
        for (int64_t k = 0; k < a.nblk; ++k) {
            float v[V];
            load_vec<float, V>(p + k * stride, v);
#pragma unroll
            for (int e = 0; e < V; ++e)
                s[e] += v[e];
        }
        const int64_t to = a.G == 1 ? i : i / a.N * (a.G * a.N) + grp * a.N + i % a.N;
        store_vec<TI, V>(a.bc_out[y & 1] + to, s);
    } else {  // 32 values a block, a run of items a warp
        constexpr int RUNS = kSumThreads / 32;
        __shared__ float red[RUNS][32];
        unsigned x = blockIdx.x - first;
        int which = 0;
        if (x >= a.a_blocks) {
            x -= a.a_blocks;
            which = 1;
            if (x >= a.d_blocks) {
                x -= a.d_blocks;
                which = 2;
            }
        }
        const int64_t n = which == 0 ? a.dim * a.N : a.dim, stride = which == 0 ? n : 2 * a.dim;
        const int64_t j = (int64_t)x * 32 + threadIdx.x % 32;
        const int run = threadIdx.x / 32;
        if (!a.item_out[which])
            return;
        float s = 0.f;
        if (j < n)
#pragma unroll 16
            for (int64_t k = run; k < a.items; k += RUNS)
                s += a.item[which][k * stride + j];
        red[run][threadIdx.x % 32] = s;
        __syncthreads();
        if (run == 0 && j < n) {
            s = 0.f;
#pragma unroll
            for (int q = 0; q < RUNS; ++q)
                s += red[q][threadIdx.x];
            a.item_out[which][j] = s;
        }
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct GradPlan {
    int64_t nblk, chunks_per_group, n_groups;
};
GradPlan grad_plan(const ScanGeom &g)
{
    GradPlan p;
    const int64_t cb = 2 * kGradThreads / scan_lanes(g.N);
    p.nblk = (g.kpg + cb - 1) / cb;
    const int64_t nc = (g.seqlen + kScanChunk - 1) / kScanChunk;
    // Up to 40 blocks an SM (the last wave's idle slots then cost little; 2 x 4096
    // tokens of 5120 channels, three blocks at a time: 12 blocks an SM 1453 us a
    // training step, 20 1430, 40 1428, 80 1446), each block over a run of chunks so
    // that the sums over tokens leave few partials and a chunk's copies overlap
    // the one before; but no run so long that an SM has less than twelve (1408
    // channels of 64 f32 states, 256 tokens: 117 us a training step with three,
    // 106 with six, 105 with twelve and with 24).
    const int64_t cols = p.nblk * g.G * g.batch, sms = device_sm_count();
    int64_t n = min64(sms * 40 / cols, nc / 4);
    n = n < sms * 12 / cols ? sms * 12 / cols : n;
    n = n < 1 ? 1 : (n > nc ? nc : n);
    p.chunks_per_group = (nc + n - 1) / n;
    p.n_groups = (nc + p.chunks_per_group - 1) / p.chunks_per_group;
    return p;
}

template <typename TI, int LN>
cudaError_t grad_ln(const GradArgs<TI> &a, const ScanGeom &g, const GradPlan &p, cudaStream_t st)
{
    auto k = scan_grad_kernel<TI, LN>;
    static SmemGrant granted;
    const cudaError_t e = allow_smem(reinterpret_cast<const void *>(k), sizeof(GradTile<TI, LN>), &granted);
    if (e != cudaSuccess)
        return e;
    k<<<dim3((unsigned)(g.G * p.nblk), (unsigned)p.n_groups, (unsigned)g.batch), kGradThreads,
        sizeof(GradTile<TI, LN>), st>>>(a, g);
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
                   const void *z, const float *bias, const void *dy, const float *h0, const float *g1,
                   const ScanEnter &enter, void *du, void *ddt, float *dA, void *dB, void *dC, float *dD, void *dz, float *dbias, void *ws,
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
    a.enter = enter;
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
    a.vec_st = g.N == 4 * scan_lanes(g.N) && aligned(h0, 16) && aligned(g1, 16) && aligned(enter.state, 16);
    a.vec_bc = g.N % 4 == 0 && g.row_b % 4 == 0 && g.row_c % 4 == 0 && aligned(Bm, al) && aligned(Cm, al);
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
    ScanSums<TI> sums{};
    sums.bc[0] = w.dB;
    sums.bc[1] = w.dC;
    sums.bc_out[0] = static_cast<TI *>(dB);
    sums.bc_out[1] = static_cast<TI *>(dC);
    sums.item[0] = w.dA;
    sums.item[1] = w.dD;
    sums.item[2] = w.dD + g.dim;
    sums.item_out[0] = dA;
    sums.item_out[1] = dD;
    sums.item_out[2] = dbias;
    sums.tokens = g.batch * g.seqlen;
    sums.G = g.G;
    sums.N = g.N;
    sums.nblk = p.nblk;
    sums.dim = g.dim;
    sums.items = g.batch * p.n_groups;
    const bool quads = g.N % 4 == 0 && aligned(dB, 4 * sizeof(TI)) && aligned(dC, 4 * sizeof(TI));
    const int64_t per_block = kSumThreads * (quads ? 4 : 1);
    sums.bc_blocks = (unsigned)((sums.tokens * g.N + per_block - 1) / per_block);
    sums.a_blocks = (unsigned)((g.dim * g.N + 31) / 32);
    sums.d_blocks = (unsigned)((g.dim + 31) / 32);
    const unsigned grid = (unsigned)(2 * g.G) * sums.bc_blocks + sums.a_blocks + 2 * sums.d_blocks;
    (quads ? scan_sums_kernel<TI, 4> : scan_sums_kernel<TI, 1>)<<<grid, kSumThreads, 0, st>>>(sums);
    note_launch(1);
    return cudaGetLastError();
}

}  // namespace

size_t scan_grad_workspace(const ScanGeom &g) { return grad_layout(g, nullptr).bytes; }

cudaError_t launch_scan_grad(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                             const float *D, const void *z, const float *bias, const void *dy, const float *h0,
                             const float *g1, const ScanEnter &enter, void *du, void *ddt, float *dA, void *dB,
                             void *dC, float *dD, void *dz, float *dbias, void *ws, const ScanGeom &g, bool bf16, cudaStream_t st)
{
    return bf16 ? grad_t<__nv_bfloat16>(u, dt, A, Bm, Cm, D, z, bias, dy, h0, g1, enter, du, ddt, dA, dB, dC, dD, dz,
                                        dbias, ws, g, st)
                : grad_t<float>(u, dt, A, Bm, Cm, D, z, bias, dy, h0, g1, enter, du, ddt, dA, dB, dC, dD, dz, dbias, ws,
                                g, st);
}

}  // namespace ssd
