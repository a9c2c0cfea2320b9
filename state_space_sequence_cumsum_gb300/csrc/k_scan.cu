// Selective scan: the state space recurrence with a decay of its own for
// every channel and state,
//     delta = softplus(dt + dt_bias),
//     h[n] <- exp(delta A[d,n]) h[n] + delta u B[g,n],
//     y = sum_n C[g,n] h[n] + D u,   out = y silu(z)
// for prompts (token tiles with the states in registers), for single tokens,
// and the reverse recurrence the backward starts from,
//     g_t[n] = exp(delta_t A[d,n]) (g_{t+1}[n] + dy_t C_t[n]).
// With no decay shared between states there is no matrix product to form:
// a token costs one exponential and four f32 operations per (channel, state),
// which at 16 states outweigh the HBM traffic (u, dt, z in, out).  On a GB300,
// bf16 with gate, 16 states, 5120 channels:
//     4 x 4096 tokens  517 us; the exponentials alone (32 a clock an SM) take
//                      180 us and the HBM traffic 100 us.  57% of the issue
//                      slots and 72% of the shared memory pipe are busy.
//     reverse pass of 2 x 4096 tokens, states kept: 205 us
//     one token of 128 sequences 18.5 us, 4.8 TB/s (71% of the measured rate)
#include "scan.cuh"

namespace ssd {
namespace {

// One pass over a run of chunks of one sequence and one block of channels.
//   kOut      forward with the output: m = B, c = C, x = u, z gates the output
//   kStates   forward, states only
//   kReverse  m = C, x = dout gated by z, tokens from the last to the first
// A tile is kScanChunk tokens as (delta, delta u) pairs and f32 matrix rows in
// shared memory; there are two, one walked with the states in registers while
// the next is made.
enum PassMode { kOut, kStates, kReverse };

template <typename TI> struct PassArgs {
    const TI *x, *dt, *z, *m, *cm;
    const float *A, *D, *bias;
    const float *start;  // [B][segments][dim][N] (reverse: [B][dim][N], the last segment's), nullptr: zeros
    TI *y;               // forward output
    float *last;         // final state (forward), initial state's gradient (reverse), or nullptr
    float *kept;         // [B][nc][dim][N] state entering each chunk, or nullptr
    float *seg_end;      // [B][segments][dim][N] end state of each segment, or nullptr
    float *seg_dsum;     // [B][segments][dim] sum of delta of each segment
    float *after;        // reverse: [B][nc][dim] sum of delta from a chunk's end to its segment's, or nullptr
    int64_t row_x, row_m;
    int64_t chunks_per_seg, first_seg, n_seg;
    bool vec, vec_bc;
};

// A thread holds four states of two adjacent channels: what a token costs in
// shared memory reads (16 bytes of delta and input, 16 of B, 16 of C a thread)
// then serves eight states.  With one channel a thread those reads, not the
// arithmetic, bounded the walk.
template <int LN> struct PassShape {
    // walking threads of a block: one warp where that gives rows of 16 channels
    // or more; and tile-making ones: as many, or more where a walking thread's
    // few lanes a channel leave them more channels to convert
    static constexpr int NT = LN <= 4 ? 32 : 8 * LN;
    static constexpr int MT = LN == 1 ? 128 : LN == 2 ? 64 : NT;
    static constexpr int CB = 2 * NT / LN;  // channels
    // blocks an SM holds; nine of two warps leave 96 registers a thread, and
    // take the 8.4 blocks an SM of four sequences of 5120 channels in one wave
    // (f32 inputs in flight need more registers: eight)
    static constexpr int BLOCKS = LN == 1 ? 3 : LN == 2 ? 5 : (LN == 4 ? 9 : 72 / (2 * LN));
    static constexpr int blocks(size_t elem) { return elem == 4 && LN == 4 ? 8 : BLOCKS; }
};

template <int LN, int MODE> struct PassTile {
    static constexpr int CB = PassShape<LN>::CB, NP = 4 * LN;
    // y: one plane per lane of a channel, the planes 8 (or 4) banks apart
    static constexpr int YP = kScanChunk * CB + (LN > 4 ? 4 : 8);
    struct Buf {
        float2 dx[kScanChunk][CB];  // delta, and what multiplies the matrix row
        float m[kScanChunk * NP];
        float c[MODE == kOut ? kScanChunk * NP : 4];
        float y[MODE == kOut ? LN * YP : 4];
    } buf[2];
};

// Some of a block's warps walk tiles (the states live in their registers), the
// others make them: per step the walkers go through tile k while the
// makers convert tile k + 1, fetch tile k + 2 and finish the output of tile
// k - 1.  One barrier a step.  A walker alone has too few independent
// instructions to fill its scheduler; the makers fill the gaps.
template <typename TI, int LN, int MODE>
__global__ void __launch_bounds__(PassShape<LN>::NT + PassShape<LN>::MT,
                                  PassShape<LN>::blocks(sizeof(TI))) scan_pass_kernel(PassArgs<TI> a, ScanGeom g)
{
    constexpr int NT = PassShape<LN>::NT, MT = PassShape<LN>::MT, CB = PassShape<LN>::CB, T = kScanChunk, NP = 4 * LN;
    // a thread's quads of a tile: QPT of one column of channels, TROWS tokens
    // apart, and PER of a matrix, BT tokens apart (in the widest and narrowest
    // shapes half the threads have none)
    constexpr int COLS = CB / 4, TROWS = MT / COLS, QPT = TROWS < T ? T / TROWS : 1;
    constexpr int MATS = MODE == kOut ? 2 : 1, BT = MT / LN, PER = BT < T ? T / BT : 1, BQ = MATS * PER;
    constexpr bool REV = MODE == kReverse;
    using Tile = PassTile<LN, MODE>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Tile &sm = *reinterpret_cast<Tile *>(smem_raw);
    // A block's warps go to the SM's schedulers in turn, so with fixed roles all
    // walkers of two-warp blocks would share two of the four: blocks in the
    // upper half of every eight warp slots swap theirs.
    bool walker = threadIdx.x < NT;
    int tid = threadIdx.x < NT ? threadIdx.x : threadIdx.x - NT;
    if constexpr (NT == 32 && MT == 32) {
        __shared__ int s_swap;
        if (threadIdx.x == 0) {
            unsigned slot;
            asm("mov.u32 %0, %%warpid;" : "=r"(slot));
            s_swap = slot >> 2 & 1;
        }
        __syncthreads();
        walker = (threadIdx.x < NT) != (s_swap != 0);
        tid = threadIdx.x % NT;
    }
    const int64_t nblk = (g.kpg + CB - 1) / CB;
    const int grp = (int)(blockIdx.x / nblk);
    const int64_t c0 = (blockIdx.x - grp * nblk) * CB;  // first channel, within the group
    const int nch = (int)min64(CB, g.kpg - c0);
    const int64_t ch0 = grp * g.kpg + c0;
    const int64_t b = blockIdx.z, seg = a.first_seg + blockIdx.y;
    const int64_t nc = (g.seqlen + T - 1) / T;
    const int64_t cbeg = seg * a.chunks_per_seg, cend = min64(cbeg + a.chunks_per_seg, nc);
    const int64_t n_tiles = cend - cbeg;
    const int N = (int)g.N, n0 = 4 * (tid % LN);
    auto at = [&](int64_t k) { return REV ? cend - 1 - k : cbeg + k; };
    auto tokens = [&](int64_t k) { return (int)min64(T, g.seqlen - at(k) * T); };

    if (walker) {
    // ---- walkers
    // this thread's states: h[channel][pair of states]
    const int c = 2 * (tid / LN);
    int nn[2];                                // live states of each channel (may exceed 4)
    const int64_t st = (ch0 + c) * g.N + n0;  // its place in a [dim][N] array
    f32x2 h[2][2] = {}, A[2][2] = {};
    float dsum[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        nn[i] = c + i < nch ? N - n0 : 0;
        if (nn[i] > 0) {
            float v[4];
            load_states(a.A + st + i * g.N, nn[i], v);
            A[i][0] = pk2(decay_rate(v[0]), decay_rate(v[1]));
            A[i][1] = pk2(decay_rate(v[2]), decay_rate(v[3]));
            if (a.start && (!REV || seg == a.n_seg - 1)) {
                load_states(a.start + (REV ? b : b * a.n_seg + seg) * g.dim * g.N + st + i * g.N, nn[i], v);
                h[i][0] = pk2(v[0], v[1]);
                h[i][1] = pk2(v[2], v[3]);
            }
        }
    }
    auto save = [&](float *p) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            if (nn[i] > 0) {
                float v[4];
                un2(h[i][0], v[0], v[1]);
                un2(h[i][1], v[2], v[3]);
                store_states(p + st + i * g.N, nn[i], v);
            }
    };
    __syncthreads();  // tile 0
    for (int64_t k = 0; k < n_tiles; ++k) {
        typename Tile::Buf &s = sm.buf[k & 1];
        if (a.kept)
            save(a.kept + (b * nc + at(k)) * g.dim * g.N);
        if (REV && a.after && n0 == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (nn[i] > 0)
                    a.after[(b * nc + at(k)) * g.dim + ch0 + c + i] = dsum[i];
        // Tokens past the end have delta = x = 0 and change nothing.  A token's
        // decays and inputs do not depend on the states: the next token's are
        // formed before this one's recurrence, which hides their latencies.
        // Each lane stores its part of the output, which the tile's last step
        // adds up.
        const f32x2 nudge = dup2(kDecayNudge);
        f32x2 d[2][2][2], x[2][2][2];
        auto prepare = [&](int i, int w) {
            const int t = REV ? T - 1 - i : i;
            const float4 dx = *reinterpret_cast<const float4 *>(&s.dx[t][c]);
            const ulonglong2 m = *reinterpret_cast<const ulonglong2 *>(&s.m[t * NP + n0]);
            const f32x2 dl[2] = {dup2(dx.x), dup2(dx.z)}, xv[2] = {dup2(dx.y), dup2(dx.w)};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                d[w][j][0] = ex2_2(fma2(dl[j], A[j][0], nudge));
                d[w][j][1] = ex2_2(fma2(dl[j], A[j][1], nudge));
                x[w][j][0] = mul2(xv[j], m.x);
                x[w][j][1] = mul2(xv[j], m.y);
            }
            if (MODE != kOut) {
                dsum[0] += dx.x;
                dsum[1] += dx.z;
            }
        };
        prepare(0, 0);
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int w = i & 1;
            ulonglong2 cv;
            if (MODE == kOut)
                cv = *reinterpret_cast<const ulonglong2 *>(&s.c[i * NP + n0]);
            if (i + 1 < T)
                prepare(i + 1, w ^ 1);
            float part[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    h[j][e] = REV ? mul2(d[w][j][e], add2(x[w][j][e], h[j][e]))
                                  : fma2(d[w][j][e], h[j][e], x[w][j][e]);
                if (MODE == kOut)
                    part[j] = hsum(fma2(h[j][1], cv.y, mul2(h[j][0], cv.x)));
            }
            if (MODE == kOut)
                *reinterpret_cast<float2 *>(&s.y[(tid % LN) * Tile::YP + i * CB + c]) = make_float2(part[0], part[1]);
        }
        __syncthreads();
    }
    if (a.last && (REV ? cbeg == 0 : cend == nc))
        save(a.last + b * g.dim * g.N);
    if (a.seg_end) {
        save(a.seg_end + (b * a.n_seg + seg) * g.dim * g.N);
        if (n0 == 0)
#pragma unroll
            for (int i = 0; i < 2; ++i)
                if (nn[i] > 0)
                    a.seg_dsum[(b * a.n_seg + seg) * g.dim + ch0 + c + i] = dsum[i];
    }
    } else {
    // ---- makers
    // this thread's elementwise work: one column of four channels
    const int cq = 4 * (tid % COLS), nq = nch - cq;
    float bias[4] = {}, Dv[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < nq) {
            bias[e] = a.bias ? a.bias[ch0 + cq + e] : 0.f;
            Dv[e] = MODE == kOut && a.D ? a.D[ch0 + cq + e] : 0.f;
        }

    // where this thread's elements of the next tile to fetch are: its column of
    // the token t_first (then every TROWS-th), and its matrix quads
    Raw4<TI> xr[QPT], dr[QPT], zr[QPT], br[BQ];
    Raw4<TI> xk[3][QPT], zk[3][QPT];  // x and z of tiles k - 1, k, k + 1, for the output
    const int t_first = tid / COLS;
    const int64_t tile0 = REV ? cend - 1 : cbeg;
    const int64_t tok0 = b * g.seqlen + tile0 * T, tok = tok0 + t_first;
    const TI *px = a.x + tok * a.row_x + ch0 + cq, *pd = a.dt + tok * g.row_dt + ch0 + cq;
    const TI *pz = a.z ? a.z + tok * g.row_z + ch0 + cq : nullptr;
    const TI *pm = a.m + (tok0 + tid / LN) * a.row_m + grp * g.N + n0;
    const TI *pc = MODE == kOut ? a.cm + (tok0 + tid / LN) * g.row_c + grp * g.N + n0 : nullptr;
    const bool four = nq >= 4, whole_bc = a.vec_bc && N == NP;
    auto fetch = [&](int nt) {
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int t = t_first + i * TROWS;
            if (TROWS > T && t >= T)
                break;
            const TI *qx = px + i * TROWS * a.row_x, *qd = pd + i * TROWS * g.row_dt, *qz = pz + i * TROWS * g.row_z;
            if (four && nt == T && a.vec) {
                xr[i] = load_ahead_as<Raw4<TI>>(qx);
                dr[i] = load_ahead_as<Raw4<TI>>(qd);
                if (pz)
                    zr[i] = load_ahead_as<Raw4<TI>>(qz);
            } else if (four && nt == T) {  // rows off the quads' boundaries
                xr[i] = load_four(qx);
                dr[i] = load_four(qd);
                if (pz)
                    zr[i] = load_four(qz);
            } else {
                const int n = t < nt ? nq : 0;
                xr[i] = load_raw4(qx, n, a.vec);
                dr[i] = load_raw4(qd, n, a.vec);
                if (pz)
                    zr[i] = load_raw4(qz, n, a.vec);
            }
        }
        px += (REV ? -T : T) * a.row_x;
        pd += (REV ? -T : T) * g.row_dt;
        if (pz)
            pz += (REV ? -T : T) * g.row_z;
#pragma unroll
        for (int i = 0; i < BQ; ++i) {
            const int t = tid / LN + i % PER * BT;
            if (BT > T && t >= T)
                break;
            const TI *q = i < PER ? pm + i % PER * BT * a.row_m : pc + i % PER * BT * g.row_c;
            if (whole_bc && nt == T)
                br[i] = load_ahead_as<Raw4<TI>>(q);
            else
                br[i] = load_raw4(q, t < nt ? N - n0 : 0, a.vec_bc);
        }
        pm += (REV ? -T : T) * a.row_m;
        if (MODE == kOut)
            pc += T * g.row_c;
    };
    auto put = [&](int nt, typename Tile::Buf &s) {
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int t = t_first + i * TROWS;
            if (TROWS > T && t >= T)
                break;
            float xv[4], dv[4], zv[4], o[8];
            unpack<TI, 4>(xr[i], xv);
            unpack<TI, 4>(dr[i], dv);
            if (REV && pz)
                unpack<TI, 4>(zr[i], zv);
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                float d0 = dv[e] + bias[e], d1 = dv[e + 1] + bias[e + 1];
                if (g.softplus)
                    softplus2(d0, d1, d0, d1);
                if (nt < T || nq < 4) {
                    d0 = t < nt && e < nq ? d0 : 0.f;
                    d1 = t < nt && e + 1 < nq ? d1 : 0.f;
                }
                f32x2 v = pk2(xv[e], xv[e + 1]);
                if (!REV) {
                    v = mul2(v, pk2(d0, d1));
                } else if (pz) {
                    const f32x2 z = pk2(zv[e], zv[e + 1]);
                    v = mul2(v, mul2(z, sigmoid2(z)));
                }
                o[2 * e] = d0;
                o[2 * e + 2] = d1;
                un2(v, o[2 * e + 1], o[2 * e + 3]);
            }
            *reinterpret_cast<float4 *>(&s.dx[t][cq]) = make_float4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<float4 *>(&s.dx[t][cq + 2]) = make_float4(o[4], o[5], o[6], o[7]);
        }
#pragma unroll
        for (int i = 0; i < BQ; ++i) {
            float v[4];
            if (BT > T && tid / LN >= T)
                break;
            unpack<TI, 4>(br[i], v);
            store_vec<float, 4>((i < PER ? s.m : s.c) + 4 * (tid + i % PER * MT), v);
        }
    };
    TI *py = MODE == kOut ? a.y + tok * g.dim + ch0 + cq : nullptr;
    auto finish = [&](int nt, const typename Tile::Buf &s, const Raw4<TI> (&xq)[QPT], const Raw4<TI> (&zq)[QPT]) {
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            const int t = t_first + i * TROWS;
            if (t < nt && nq > 0) {
                float xv[4], zv[4], o[4];
                unpack<TI, 4>(xq[i], xv);
                unpack<TI, 4>(zq[i], zv);
                ulonglong2 y = *reinterpret_cast<const ulonglong2 *>(&s.y[t * CB + cq]);
#pragma unroll
                for (int j = 1; j < LN; ++j) {
                    const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(&s.y[j * Tile::YP + t * CB + cq]);
                    y.x = add2(y.x, p.x);
                    y.y = add2(y.y, p.y);
                }
                un2(y.x, o[0], o[1]);
                un2(y.y, o[2], o[3]);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                    f32x2 v = fma2(pk2(Dv[e], Dv[e + 1]), pk2(xv[e], xv[e + 1]), pk2(o[e], o[e + 1]));
                    if (pz) {
                        const f32x2 z = pk2(zv[e], zv[e + 1]);
                        v = mul2(v, mul2(z, sigmoid2(z)));
                    }
                    un2(v, o[e], o[e + 1]);
                }
                store_some<TI, 4>(py + i * TROWS * g.dim, o, nq, a.vec);
            }
        }
        py += T * g.dim;
    };
    // x and z of the tile in the fetch registers, kept for its output
    auto keep = [&](Raw4<TI> (&xq)[QPT], Raw4<TI> (&zq)[QPT]) {
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            xq[i] = xr[i];
            zq[i] = zr[i];
        }
    };
    fetch(tokens(0));
    put(tokens(0), sm.buf[0]);
    keep(xk[1], zk[1]);
    if (n_tiles > 1)
        fetch(tokens(1));
    __syncthreads();  // tile 0
    for (int64_t k = 0; k < n_tiles; ++k) {
        if (k + 1 < n_tiles) {
            put(tokens(k + 1), sm.buf[(k + 1) & 1]);
            keep(xk[2], zk[2]);
            if (k + 2 < n_tiles)
                fetch(tokens(k + 2));
        }
        if (MODE == kOut && k > 0)
            finish(tokens(k - 1), sm.buf[(k - 1) & 1], xk[0], zk[0]);
#pragma unroll
        for (int i = 0; i < QPT; ++i) {
            xk[0][i] = xk[1][i];
            zk[0][i] = zk[1][i];
            xk[1][i] = xk[2][i];
            zk[1][i] = zk[2][i];
        }
        __syncthreads();
    }
    if (MODE == kOut)
        finish(tokens(n_tiles - 1), sm.buf[(n_tiles - 1) & 1], xk[0], zk[0]);
    }
}

// Segment end states -> what enters each segment, in place, in the order of
// the pass: enter' = exp(A dsum) enter + end.  Forward: from the initial
// state, the last segment's end is not there and not needed.  Reverse: the
// last segment's own pass began with what enters it, so from zero; `last`
// receives what leaves the first.  kJoin segments' values are read before the
// first is replaced.
template <bool REV>
__global__ void __launch_bounds__(256)
scan_join_kernel(float *__restrict__ seg, const float *__restrict__ dsum, const float *__restrict__ A,
                 const float *start, float *last, int64_t batch, int64_t dim, int64_t N, int64_t n_seg)
{
    constexpr int kJoin = 24;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t DN = dim * N;
    if (i >= batch * DN)
        return;
    const int64_t b = i / DN, r = i - b * DN, d = r / N;
    const float A2 = decay_rate(A[r]);
    float h = start ? start[i] : 0.f;
    for (int64_t k0 = 0; k0 < n_seg; k0 += kJoin) {
        float end[kJoin], q[kJoin];
#pragma unroll
        for (int j = 0; j < kJoin; ++j) {
            const int64_t k = k0 + j, s = b * n_seg + (REV ? n_seg - 1 - k : k);
            const bool there = REV ? k < n_seg : k < n_seg - 1;
            end[j] = there ? seg[s * DN + r] : 0.f;
            q[j] = there ? dsum[s * dim + d] : 0.f;
        }
        float most = 0.f;
#pragma unroll
        for (int j = 0; j < kJoin; ++j)
            most = fmaxf(most, A2 * q[j]);
        auto walk = [&](auto step) {
#pragma unroll
            for (int j = 0; j < kJoin; ++j) {
                const int64_t k = k0 + j, s = b * n_seg + (REV ? n_seg - 1 - k : k);
                if (k < n_seg) {
                    seg[s * DN + r] = h;
                    h = step(A2 * q[j], h, end[j]);
                }
            }
        };
        if (most <= kLargeExponent)  // decided once: a test at each step holds the loads above apart
            walk([](float x, float v, float e) { return fmaf(ex2(x), v, e); });
        else
            walk(add_scaled);
    }
    if (REV && last)
        last[i] = h;
}

// One token.  A thread holds four states of a channel, LN lanes a channel, for
// R sequences (blockIdx.y: which R).  What a (sequence, channel) needs once --
// its step, input, gate and output -- is the work of one lane: lane r of a
// channel has sequence r's, passes the step to the others and receives the
// sum of their outputs.
//   WHOLE: every lane holds four states and every quad is one access, so all
//   loads are issued before the first is used (threads and sequences past the
//   end load the last one's and store nothing).
template <typename TI, int LN, bool WHOLE>
__global__ void __launch_bounds__(256)
scan_step_kernel(const TI *__restrict__ u, const TI *__restrict__ dt, const float *__restrict__ A,
                 const TI *__restrict__ Bm, const TI *__restrict__ Cm, const float *__restrict__ D,
                 const TI *__restrict__ z, const float *__restrict__ bias, const float *state,
                 float *state_out, TI *__restrict__ y, ScanGeom g)
{
    constexpr int R = LN < 4 ? LN : 4;
    const unsigned i = blockIdx.x * 256u + threadIdx.x;
    const bool live = i / LN < (unsigned)g.dim;
    const unsigned d = live ? i / LN : (unsigned)g.dim - 1;
    const int lane = (int)(i % LN), n0 = 4 * lane;
    const int nn = live ? (int)g.N - n0 : 0;
    const unsigned grp = g.G == 1 ? 0 : d / (unsigned)g.kpg;
    const int64_t b0 = (int64_t)blockIdx.y * R;
    // this lane's sequence
    const int64_t b = min64(b0 + lane % R, g.batch - 1);
    const bool mine = live && lane < R && b0 + lane < g.batch;
    float h[R][4], bv[R][4], cv[R][4], av[4];
    float uv, dl, zv, bs, Dv;
    {
        float4 hr[R], ar;
        Raw4<TI> br[R], cr[R];
        if (WHOLE) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t q = min64(b0 + r, g.batch - 1);
                hr[r] = load_ahead_as<float4>(state + (q * g.dim + d) * g.N + n0);
                br[r] = load_ahead_as<Raw4<TI>>(Bm + q * g.row_b + grp * g.N + n0);
                cr[r] = load_ahead_as<Raw4<TI>>(Cm + q * g.row_c + grp * g.N + n0);
            }
            ar = load_ahead_as<float4>(A + (int64_t)d * g.N + n0);
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int n = b0 + r < g.batch ? nn : 0;
                const int64_t q = b0 + r;
                load_states(state + (q * g.dim + d) * g.N + n0, n, h[r]);
                unpack<TI, 4>(load_raw4(Bm + q * g.row_b + grp * g.N + n0, n, false), bv[r]);
                unpack<TI, 4>(load_raw4(Cm + q * g.row_c + grp * g.N + n0, n, false), cv[r]);
            }
            load_states(A + (int64_t)d * g.N + n0, nn, av);
        }
        const TI ur = u[b * g.row_u + d], dr = dt[b * g.row_dt + d];
        const TI zr = z ? z[b * g.row_z + d] : ur;
        bs = bias ? bias[d] : 0.f;
        Dv = D ? D[d] : 0.f;
        if (WHOLE) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                unpack<float, 4>(hr[r], h[r]);
                unpack<TI, 4>(br[r], bv[r]);
                unpack<TI, 4>(cr[r], cv[r]);
            }
            unpack<float, 4>(ar, av);
        }
        uv = to_f32(ur);
        dl = to_f32(dr) + bs;
        zv = to_f32(zr);
    }
    dl = g.softplus ? softplus(dl) : dl;
#pragma unroll
    for (int e = 0; e < 4; ++e)
        av[e] = decay_rate(av[e]);
    const float du = dl * uv;
    float s[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const float dr = __shfl_sync(0xffffffffu, dl, r, LN), xr = __shfl_sync(0xffffffffu, du, r, LN);
        s[r] = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            h[r][e] = fmaf(ex2(fmaf(dr, av[e], kDecayNudge)), h[r][e], xr * bv[r][e]);
            s[r] = fmaf(h[r][e], cv[r][e], s[r]);
        }
        if (nn > 0 && b0 + r < g.batch)
            store_states(state_out + ((b0 + r) * g.dim + d) * g.N + n0, nn, h[r]);
    }
    // each exchange sends the sums of half the sequences and keeps the other
    // half's; lane r ends with sequence r's
#pragma unroll
    for (int o = 1, n = R; o < R; o *= 2, n /= 2)
#pragma unroll
        for (int k = 0; k < n / 2; ++k) {
            const float keep = lane & o ? s[2 * k + 1] : s[2 * k], send = lane & o ? s[2 * k] : s[2 * k + 1];
            s[k] = keep + __shfl_xor_sync(0xffffffffu, send, o);
        }
#pragma unroll
    for (int o = R; o < LN; o *= 2)
        s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
    if (mine) {
        float out = s[0];
        out = fmaf(Dv, uv, out);
        if (z)
            out *= fast_silu(zv);
        y[b * g.dim + d] = from_f32<TI>(out);
    }
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

template <typename TI, int LN, int MODE>
cudaError_t launch_pass_ln(const PassArgs<TI> &a, const ScanGeom &g, int64_t segs, cudaStream_t st)
{
    constexpr int64_t CB = PassShape<LN>::CB;
    const dim3 grid((unsigned)(g.G * ((g.kpg + CB - 1) / CB)), (unsigned)segs, (unsigned)g.batch);
    constexpr size_t smem = sizeof(PassTile<LN, MODE>);
    auto k = scan_pass_kernel<TI, LN, MODE>;
    static SmemGrant granted;
    const cudaError_t allowed = allow_smem(reinterpret_cast<const void *>(k), smem, &granted);
    if (allowed != cudaSuccess)
        return allowed;
    k<<<grid, PassShape<LN>::NT + PassShape<LN>::MT, smem, st>>>(a, g);
    note_launch(1);
    return cudaGetLastError();
}
template <typename TI, int MODE>
cudaError_t launch_pass(const PassArgs<TI> &a, const ScanGeom &g, int64_t segs, cudaStream_t st)
{
    switch (scan_lanes(g.N)) {
    case 1: return launch_pass_ln<TI, 1, MODE>(a, g, segs, st);
    case 2: return launch_pass_ln<TI, 2, MODE>(a, g, segs, st);
    case 4: return launch_pass_ln<TI, 4, MODE>(a, g, segs, st);
    case 8: return launch_pass_ln<TI, 8, MODE>(a, g, segs, st);
    default: return launch_pass_ln<TI, 16, MODE>(a, g, segs, st);
    }
}

template <bool REV>
cudaError_t launch_join(float *seg, const float *dsum, const float *A, const float *start, float *last,
                        const ScanGeom &g, int64_t n_seg, cudaStream_t st)
{
    const int64_t n = g.batch * g.dim * g.N;
    scan_join_kernel<REV><<<(unsigned)((n + 255) / 256), 256, 0, st>>>(seg, dsum, A, start, last, g.batch, g.dim, g.N,
                                                                     n_seg);
    note_launch(1);
    return cudaGetLastError();
}

struct ScanSegs {
    int64_t n_seg, chunks_per_seg;
};
// A pass's blocks for one segment, and as many as the GPU holds at once.
struct PassFill {
    int64_t blocks, slots;
};
PassFill pass_fill(const ScanGeom &g, size_t elem)
{
    auto fill = [&](auto shape) {
        return PassFill{g.G * ((g.kpg + shape.CB - 1) / shape.CB) * g.batch, shape.blocks(elem) * (int64_t)device_sm_count()};
    };
    switch (scan_lanes(g.N)) {
    case 1: return fill(PassShape<1>());
    case 2: return fill(PassShape<2>());
    case 4: return fill(PassShape<4>());
    case 8: return fill(PassShape<8>());
    default: return fill(PassShape<16>());
    }
}
int64_t chunks(const ScanGeom &g) { return (g.seqlen + kScanChunk - 1) / kScanChunk; }
// As many segments as fit with all their blocks, of four chunks at least.
ScanSegs cut(const PassFill &f, int64_t nc)
{
    const int64_t n = min64(f.slots / f.blocks, nc / 4);
    ScanSegs s{1, nc};
    if (n > 1) {
        s.chunks_per_seg = (nc + n - 1) / n;
        s.n_seg = (nc + s.chunks_per_seg - 1) / s.chunks_per_seg;
    }
    return s;
}

// Segments of a pass: one where the channels alone give the GPU a third of the
// blocks it holds, or the sequence is short.  Measured on 4096 tokens of 5120
// channels, 16 states (nine blocks an SM): one sequence (2.1 blocks an SM) 283
// us whole, 246 us in four segments; two sequences 342 us whole, 389 us in two.
ScanSegs scan_segments(const ScanGeom &g, size_t elem)
{
    const int64_t nc = chunks(g);
    const PassFill f = pass_fill(g, elem);
    return 3 * f.blocks < f.slots && nc >= 32 ? cut(f, nc) : ScanSegs{1, nc};
}

// The reverse pass's segments cost only their join.
ScanSegs scan_reverse_segments(const ScanGeom &g, size_t elem) { return cut(pass_fill(g, elem), chunks(g)); }

size_t segment_bytes(const ScanGeom &g, const ScanSegs &s, int64_t more)
{
    return s.n_seg > 1 ? (size_t)(g.batch * (s.n_seg * g.dim * (g.N + 1) + more)) * sizeof(float) : 0;
}

template <typename TI> void matrix_args(PassArgs<TI> *a, const ScanGeom &g, int64_t row_m)
{
    const size_t al = 4 * sizeof(TI);
    a->row_m = row_m;
    a->vec_bc = g.N % 4 == 0 && g.row_b % 4 == 0 && g.row_c % 4 == 0 && aligned(a->m, al) && aligned(a->cm, al);
}

// The forward, in segments where the channels alone cannot fill the GPU: the
// segments' end states from zero, their join, then all segments at once.
template <typename TI>
cudaError_t run_forward(PassArgs<TI> a, const float *start, void *ws, const ScanGeom &g, cudaStream_t st)
{
    const ScanSegs sp = scan_segments(g, sizeof(TI));
    a.chunks_per_seg = sp.chunks_per_seg;
    a.n_seg = sp.n_seg;
    a.start = start;
    matrix_args(&a, g, g.row_b);
    if (sp.n_seg > 1) {
        float *seg = static_cast<float *>(ws);
        float *dsum = seg + g.batch * sp.n_seg * g.dim * g.N;
        PassArgs<TI> e = a;
        e.start = nullptr;
        e.y = nullptr;
        e.z = nullptr;
        e.last = e.kept = nullptr;
        e.seg_end = seg;
        e.seg_dsum = dsum;
        cudaError_t err = launch_pass<TI, kStates>(e, g, sp.n_seg - 1, st);
        if (err != cudaSuccess)
            return err;
        err = launch_join<false>(seg, dsum, a.A, start, nullptr, g, sp.n_seg, st);
        if (err != cudaSuccess)
            return err;
        a.start = seg;
    }
    return a.y ? launch_pass<TI, kOut>(a, g, sp.n_seg, st) : launch_pass<TI, kStates>(a, g, sp.n_seg, st);
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
    return run_forward<TI>(a, init, ws, g, st);
}

// The reverse pass.  Nothing but the states comes of it, so its segments are
// passed through once, from zero, and the gradients add what entered a
// segment to its chunks' states as they read them.
template <typename TI>
cudaError_t rev_t(const void *dy, const void *dt, const float *A, const void *Cm, const void *z,
                  const float *bias, const float *dfinal, float *dkept, float *dinit, void *ws, ScanEnter *enter,
                  const ScanGeom &g, cudaStream_t st)
{
    const ScanSegs sp = scan_reverse_segments(g, sizeof(TI));
    PassArgs<TI> a{};
    a.x = static_cast<const TI *>(dy);
    a.dt = static_cast<const TI *>(dt);
    a.z = static_cast<const TI *>(z);
    a.m = static_cast<const TI *>(Cm);
    a.A = A;
    a.bias = bias;
    a.start = dfinal;
    a.kept = dkept;
    a.row_x = g.row_dy;
    a.vec = quads_ok(g, dy, g.row_dy, dt, z, nullptr, sizeof(TI));
    a.chunks_per_seg = sp.chunks_per_seg;
    a.n_seg = sp.n_seg;
    matrix_args(&a, g, g.row_c);
    *enter = ScanEnter{nullptr, nullptr, sp.n_seg, sp.chunks_per_seg};
    if (sp.n_seg == 1) {
        a.last = dinit;
        return launch_pass<TI, kReverse>(a, g, 1, st);
    }
    float *seg = static_cast<float *>(ws);
    a.seg_end = seg;
    a.seg_dsum = seg + g.batch * sp.n_seg * g.dim * g.N;
    a.after = a.seg_dsum + g.batch * sp.n_seg * g.dim;
    const cudaError_t err = launch_pass<TI, kReverse>(a, g, sp.n_seg, st);
    if (err != cudaSuccess)
        return err;
    enter->state = seg;
    enter->after = a.after;
    return launch_join<true>(seg, a.seg_dsum, A, nullptr, dinit, g, sp.n_seg, st);
}

template <typename TI>
cudaError_t step_t(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm, const float *D,
                   const void *z, const float *bias, const float *state, float *state_out, void *y,
                   const ScanGeom &g, cudaStream_t st)
{
    const int LN = scan_lanes(g.N);
    const int64_t R = LN < 4 ? LN : 4;
    const dim3 blocks((unsigned)((g.dim * LN + 255) / 256), (unsigned)((g.batch + R - 1) / R));
    const size_t al = 4 * sizeof(TI);
    const bool whole = g.N == 4 * LN && g.row_b % 4 == 0 && g.row_c % 4 == 0 && aligned(Bm, al) && aligned(Cm, al) &&
                       aligned(A, 16) && aligned(state, 16) && aligned(state_out, 16);
#define SSD_STEP(LANES)                                                                              \
    (whole ? scan_step_kernel<TI, LANES, true> : scan_step_kernel<TI, LANES, false>)<<<blocks, 256, 0, st>>>( \
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

// Room for either type.
size_t scan_pass_workspace(const ScanGeom &g)
{
    const size_t a = segment_bytes(g, scan_segments(g, 2), 0), b = segment_bytes(g, scan_segments(g, 4), 0);
    return a > b ? a : b;
}
size_t scan_reverse_workspace(const ScanGeom &g)
{
    const int64_t after = chunks(g) * g.dim;
    const size_t a = segment_bytes(g, scan_reverse_segments(g, 2), after);
    const size_t b = segment_bytes(g, scan_reverse_segments(g, 4), after);
    return a > b ? a : b;
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
                                ScanEnter *enter, const ScanGeom &g, bool bf16, cudaStream_t st)
{
    return bf16 ? rev_t<__nv_bfloat16>(dy, dt, A, Cm, z, bias, dfinal, dkept, dinit, ws, enter, g, st)
                : rev_t<float>(dy, dt, A, Cm, z, bias, dfinal, dkept, dinit, ws, enter, g, st);
}

cudaError_t launch_scan_step(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                             const float *D, const void *z, const float *bias, const float *state,
                             float *state_out, void *y, const ScanGeom &g, bool bf16, cudaStream_t st)
{
    return bf16 ? step_t<__nv_bfloat16>(u, dt, A, Bm, Cm, D, z, bias, state, state_out, y, g, st)
                : step_t<float>(u, dt, A, Bm, Cm, D, z, bias, state, state_out, y, g, st);
}

}  // namespace ssd
