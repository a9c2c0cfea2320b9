// Product of two 8-bit matrices with a scale for each block of 128 along the
// summed dimension, on tensor cores:
//
//     out[m,n] = sum_j sa[m,j] sb[n,j] (sum_{k in block j} a[m,k] b[n,k])
//
// Products of 8-bit floats are exact in f32; a block's inner sum is formed by
// tcgen05.mma (kind::f8f6f4) in a TMEM buffer of its own, and the threads that
// hold the output add it to their registers, times the two scales, in f32.
// Scales are any f32 values, so they cannot go into the MMA.
//
// Operands are K-major tiles of 128 bytes (one block) a row, brought by TMA
// with the 128-byte swizzle; what lies past an edge arrives as zeros.  The MMA's
// 128 rows are rows of `a` or, with few tokens, of the weights (kSwap: the
// output is then written transposed), its BN columns rows of the other matrix.
//
// One CTA: warps 0..4 WG-1 add (thread = MMA row, CW columns), one warp loads,
// one issues MMAs.  BN 256 walks its tiles persistently, so the epilogue of one
// tile runs under the MMAs of the next.  The others take one tile, or with few
// tiles a part of its blocks: the CTAs of a cluster then add their partial
// sums through distributed shared memory, in the order of the parts.
#include <algorithm>

#include "common.cuh"
#include "ssd_internal.h"
#include "tc05.cuh"

namespace ssd {
namespace {
using namespace tc;

constexpr int kRows = 128;                  // MMA rows of a tile
constexpr uint32_t kABytes = kRows * 128;   // one block of them
constexpr int kMostSplits = 8;              // CTAs of a cluster (portable limit)

template <int BN> struct Tile {
    static constexpr int kWG = BN >= 64 ? 2 : 1;  // warpgroups that share the columns
    static constexpr int kCW = BN / kWG;          // columns of a thread
    static constexpr int kAddWarps = 4 * kWG;
    static constexpr int kThreads = kAddWarps * 32 + 64;
    static constexpr bool kPersistent = BN == 256;
    static constexpr int kCtas = kPersistent ? 1 : 2;  // on an SM
    static constexpr int kBuffers = BN >= 128 ? 2 : 4; // in TMEM
    static constexpr uint32_t kStageBytes = kABytes + BN * 128;
    static constexpr int kStages = BN == 256 ? 3 : BN == 128 ? 3 : BN == 64 ? 4 : 5;
    static constexpr uint32_t kStaging = kPersistent ? kAddWarps * 4096 : 0;  // of the output
    static constexpr uint32_t kSmem = kStages * kStageBytes + kStaging + 1024;
};

struct Params {
    const float *sa, *sb;
    int64_t sa_row, sa_block, sb_row, sb_block;  // elements between scales
    int sa_shift, sb_shift;                      // a scale for each 1 << shift rows
    void *out;
    int64_t ld;                                  // elements between rows of out
    int64_t m, n;                                // rows of the MMA's A and B
    int m_tiles, n_tiles, blocks, splits;
    uint32_t idesc;
    bool bf16, vec;                              // vec: out takes 16-byte accesses
    unsigned *status;
};

__device__ __forceinline__ void add_barrier(int threads)
{
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A shared-memory address of this CTA as one of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float4 load_cluster(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr));
    return v;
}

// `count` (1..4) consecutive values of the output from element `at` on.
__device__ __forceinline__ void store4(const Params &p, int64_t at, const float4 &v, int count)
{
    const float e[4] = {v.x, v.y, v.z, v.w};
    if (p.bf16) {
        __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(p.out) + at;
        if (p.vec && count == 4) {
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count)
                o[i] = __float2bfloat16_rn(e[i]);
    } else {
        float *o = static_cast<float *>(p.out) + at;
        if (p.vec && count == 4) {
            *reinterpret_cast<float4 *>(o) = v;
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count)
                o[i] = e[i];
    }
}

// A warp's 32 rows of 128 bytes, staged with the swizzle, to the output: rows
// row0.., `cols` values each from column col on.
template <typename T>
__device__ __forceinline__ void copy_rows(const Params &p, const unsigned char *stage, int64_t row0, int64_t col, int lane)
{
    constexpr int per = 16 / (int)sizeof(T);  // values of a 16-byte chunk
    const int chunk = lane & 7;
    const int64_t c = col + chunk * per;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int r = i * 4 + (lane >> 3);
        if (row0 + r >= p.m || c >= p.n)
            continue;
        const uint4 v = *reinterpret_cast<const uint4 *>(stage + sw128_offset(r, chunk));
        T *o = static_cast<T *>(p.out) + (row0 + r) * p.ld + c;
        if (p.vec && c + per <= p.n) {
            *reinterpret_cast<uint4 *>(o) = v;
        } else {
            const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
            for (int j = 0; j < per; ++j)
                if (c + j < p.n)
                    o[j] = e[j];
        }
    }
}

template <int BN, bool kSwap, bool kRowsB>
__global__ void __launch_bounds__(Tile<BN>::kThreads, Tile<BN>::kCtas)
block_matmul_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const Params p)
{
    using T = Tile<BN>;
    constexpr int ST = T::kStages, NB = T::kBuffers, CW = T::kCW;
    extern __shared__ unsigned char raw[];
    unsigned char *smem = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
    unsigned char *staging = T::kPersistent ? smem + ST * T::kStageBytes : smem;
    __shared__ uint64_t full[ST], empty[ST], done[NB], freed[NB];
    __shared__ uint32_t tmem_slot;
    __shared__ __align__(16) float sb_smem[2][kRowsB ? BN : 4];

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < ST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&done[i], 1);
            mbar_init(&freed[i], T::kAddWarps);
        }
        fence_barrier_init();
    }
    if (warp == T::kAddWarps + 1) {
        tmem_alloc(&tmem_slot, NB * BN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    // this CTA's tiles and, in each, its blocks of the summed dimension
    const int rank = T::kPersistent ? 0 : (int)(blockIdx.x % (unsigned)p.splits);
    const int first = T::kPersistent ? (int)blockIdx.x : (int)(blockIdx.x / (unsigned)p.splits);
    const int step = T::kPersistent ? (int)gridDim.x : p.m_tiles * p.n_tiles;
    const int tiles = p.m_tiles * p.n_tiles;
    const int kb0 = T::kPersistent ? 0 : (int)((int64_t)p.blocks * rank / p.splits);
    const int kb1 = T::kPersistent ? p.blocks : (int)((int64_t)p.blocks * (rank + 1) / p.splits);
    // tiles in groups of kGroup rows of tiles, column after column: what a wave
    // of CTAs reads of both operands stays in L2
    constexpr int kGroup = 16;
    auto place = [&](int t, int &mt, int &nt) {
        const int per = kGroup * p.n_tiles, g = t / per, in = t - g * per;
        const int rows = min(kGroup, p.m_tiles - g * kGroup);
        nt = in / rows;
        mt = g * kGroup + in % rows;
    };

    if (warp == T::kAddWarps) {
        // ---------------------------------------------------------- loads
        if (lane == 0) {
            prefetch_tmap(&ta);
            prefetch_tmap(&tb);
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                int mt, nt;
                place(t, mt, nt);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % ST;
                    if (!mbar_wait(&empty[s], ((it / ST) & 1) ^ 1)) {
                        atomicOr(p.status, 1u);
                        ok = false;
                        break;
                    }
                    unsigned char *a = smem + s * T::kStageBytes;
                    mbar_arrive_expect_tx(&full[s], T::kStageBytes);
                    tma_load_2d(a, &ta, &full[s], kb * 128, mt * kRows);
                    tma_load_2d(a + kABytes, &tb, &full[s], kb * 128, nt * BN);
                }
            }
        }
    } else if (warp == T::kAddWarps + 1) {
        // ----------------------------------------------------------- MMAs
        if (lane == 0) {
            uint32_t it = 0;
            bool ok = true;
            for (int t = first; ok && t < tiles; t += step) {
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const uint32_t s = it % ST, b = it % NB;
                    if (!mbar_wait(&freed[b], ((it / NB) & 1) ^ 1) || !mbar_wait(&full[s], (it / ST) & 1)) {
                        atomicOr(p.status, 1u);
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + s * T::kStageBytes);
                    const uint64_t da = desc_k0(a), db = desc_k0(a + kABytes);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mma_f8_ss(tmem + b * BN, desc_k(da, 0, k), desc_k(db, 0, k), p.idesc, k > 0);
                    mma_commit(&empty[s]);
                    mma_commit(&done[b]);
                }
            }
        }
    } else {
        // ----------------------------------------------- sums and output
        const int wg = warp >> 2, quarter = warp & 3;
        const uint32_t at = tmem + ((uint32_t)(quarter * 32) << 16) + wg * CW;
        uint32_t it = 0;
        bool ok = true;
        for (int t = first; ok && t < tiles; t += step) {
            int mt, nt;
            place(t, mt, nt);
            const int64_t row0 = (int64_t)mt * kRows + quarter * 32, row = row0 + lane;
            const int64_t col0 = (int64_t)nt * BN + wg * CW;
            const float *sa = p.sa + (row < p.m ? row >> p.sa_shift : 0) * p.sa_row;
            const float *sb;
            bool mine = true;
            if (kRowsB) {  // this thread brings one column's scale
                const int64_t c = (int64_t)nt * BN + threadIdx.x;
                mine = threadIdx.x < BN && c < p.n;
                sb = p.sb + (mine ? c >> p.sb_shift : 0) * p.sb_row;
            } else {       // its columns lie in one block of 128
                sb = p.sb + (col0 < p.n ? col0 >> 7 : 0) * p.sb_row;
            }
            uint64_t acc[CW / 2];
#pragma unroll
            for (int i = 0; i < CW / 2; ++i)
                acc[i] = 0;
            float fa = 0.f, fb = 0.f;
            if (kb0 < kb1) {
                fa = sa[kb0 * p.sa_block];
                fb = mine ? sb[kb0 * p.sb_block] : 0.f;
            }
            for (int kb = kb0; kb < kb1; ++kb, ++it) {
                const uint32_t b = it % NB;
                const float wa = fa, wb = fb;
                if (kb + 1 < kb1) {
                    fa = sa[(kb + 1) * p.sa_block];
                    fb = mine ? sb[(kb + 1) * p.sb_block] : 0.f;
                }
                if (kRowsB) {
                    if (threadIdx.x < BN)
                        sb_smem[it & 1][threadIdx.x] = wb;
                    add_barrier(T::kAddWarps * 32);
                }
                if (ok && !mbar_wait(&done[b], (it / NB) & 1)) {
                    atomicOr(p.status, 1u);
                    ok = false;
                }
                if (!ok)
                    continue;
                tc_fence_after();
                const uint32_t f = __float_as_uint(kRowsB ? wa : wa * wb);
                const uint64_t f2 = f2_pack(f, f);
                uint32_t r[2][32];
                tmem_ld32(at + b * BN, r[0]);
#pragma unroll
                for (int c = 0; c < CW / 32; ++c) {
                    tmem_ld_wait_on(r[c & 1]);
                    if (c + 1 < CW / 32) {
                        tmem_ld32(at + b * BN + (c + 1) * 32, r[(c + 1) & 1]);
                    } else {
                        tc_fence_before();
                        warp_arrive(&freed[b]);
                    }
#pragma unroll
                    for (int i = 0; i < 16; i += 2) {
                        uint64_t w0 = f2, w1 = f2;
                        if (kRowsB) {
                            const ulonglong2 s =
                                *reinterpret_cast<const ulonglong2 *>(&sb_smem[it & 1][wg * CW + c * 32 + 2 * i]);
                            w0 = f2_mul(s.x, f2);
                            w1 = f2_mul(s.y, f2);
                        }
                        uint64_t &x = acc[c * 16 + i], &y = acc[c * 16 + i + 1];
                        x = f2_fma(f2_pack(r[c & 1][2 * i], r[c & 1][2 * i + 1]), w0, x);
                        y = f2_fma(f2_pack(r[c & 1][2 * i + 2], r[c & 1][2 * i + 3]), w1, y);
                    }
                }
            }
            auto value = [&](int c) {
                uint32_t lo, hi;
                f2_unpack(acc[c >> 1], lo, hi);
                return __uint_as_float(c & 1 ? hi : lo);
            };
            if (!T::kPersistent && p.splits > 1) {
                // partial sums: rows of BN + 4 (out's rows), or columns of 128 (swapped)
                float *part = reinterpret_cast<float *>(smem);
                const int r = quarter * 32 + lane;
#pragma unroll
                for (int c = 0; c < CW; c += 4) {
                    if (kSwap) {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            part[(wg * CW + c + j) * kRows + r] = value(c + j);
                    } else {
                        *reinterpret_cast<float4 *>(part + r * (BN + 4) + wg * CW + c) =
                            make_float4(value(c), value(c + 1), value(c + 2), value(c + 3));
                    }
                }
            } else if (kSwap) {
                if (row < p.m) {
#pragma unroll
                    for (int c = 0; c < CW; ++c)
                        if (col0 + c < p.n) {
                            const int64_t o = (col0 + c) * p.ld + row;
                            if (p.bf16)
                                static_cast<__nv_bfloat16 *>(p.out)[o] = __float2bfloat16_rn(value(c));
                            else
                                static_cast<float *>(p.out)[o] = value(c);
                        }
                }
            } else {
                unsigned char *stage = staging + warp * 4096;
                if (p.bf16) {
#pragma unroll
                    for (int h = 0; h < CW; h += 64) {
                        constexpr int chunks = (CW < 64 ? CW : 64) / 8;
#pragma unroll
                        for (int j = 0; j < chunks; ++j) {
                            uint32_t v[4];
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                v[q] = pack_bf16x2(value(h + j * 8 + 2 * q), value(h + j * 8 + 2 * q + 1));
                            *reinterpret_cast<uint4 *>(stage + sw128_offset(lane, j)) = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                        __syncwarp();
                        if (CW >= 64 || (lane & 7) < chunks)
                            copy_rows<__nv_bfloat16>(p, stage, row0, col0 + h, lane);
                        __syncwarp();
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < CW; h += 32) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            *reinterpret_cast<float4 *>(stage + sw128_offset(lane, j)) =
                                make_float4(value(h + j * 4), value(h + j * 4 + 1), value(h + j * 4 + 2), value(h + j * 4 + 3));
                        __syncwarp();
                        copy_rows<float>(p, stage, row0, col0 + h, lane);
                        __syncwarp();
                    }
                }
            }
        }
    }
    if (!T::kPersistent && p.splits > 1) {
        // the cluster's partial sums, each CTA every splits-th group of four
        __syncwarp();
        cluster_sync();
        int mt, nt;
        place(first, mt, nt);
        const uint32_t part = smem_u32(smem);
        constexpr int kGroups = kRows * BN / 4;
        for (int i = rank * T::kThreads + (int)threadIdx.x; i < kGroups; i += p.splits * T::kThreads) {
            int64_t outer, inner, n_outer, n_inner;
            uint32_t off;
            if (kSwap) {
                const int c = i / (kRows / 4), r = i % (kRows / 4) * 4;
                outer = (int64_t)nt * BN + c;
                inner = (int64_t)mt * kRows + r;
                n_outer = p.n;
                n_inner = p.m;
                off = (uint32_t)(c * kRows + r) * 4;
            } else {
                const int r = i / (BN / 4), c = i % (BN / 4) * 4;
                outer = (int64_t)mt * kRows + r;
                inner = (int64_t)nt * BN + c;
                n_outer = p.m;
                n_inner = p.n;
                off = (uint32_t)(r * (BN + 4) + c) * 4;
            }
            if (outer >= n_outer || inner >= n_inner)
                continue;
            float4 v = load_cluster(in_cta(part + off, 0));
            for (int k = 1; k < p.splits; ++k) {
                const float4 w = load_cluster(in_cta(part + off, k));
                v.x += w.x;
                v.y += w.y;
                v.z += w.z;
                v.w += w.w;
            }
            store4(p, outer * p.ld + inner, v, (int)min64(4, n_inner - inner));
        }
        cluster_sync();  // nobody leaves while its sums are read
    }
    tc_fence_before();
    __syncthreads();
    if (warp == T::kAddWarps + 1)
        tmem_dealloc(tmem, NB * BN);
}

template <int BN, bool kSwap, bool kRowsB>
cudaError_t launch(const CUtensorMap &ta, const CUtensorMap &tb, const Params &p, int sms, cudaStream_t st)
{
    using T = Tile<BN>;
    static SmemGrant granted;
    const auto kernel = block_matmul_kernel<BN, kSwap, kRowsB>;
    if (cudaError_t e = allow_smem(reinterpret_cast<const void *>(kernel), T::kSmem, &granted))
        return e;
    const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(T::kPersistent ? std::min<int64_t>(tiles, sms) : tiles * p.splits));
    cfg.blockDim = dim3(T::kThreads);
    cfg.dynamicSmemBytes = T::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)p.splits;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = p.splits > 1 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, ta, tb, p);
    if (e == cudaSuccess)
        note_launch(1);
    return e;
}

}  // namespace

cudaError_t launch_block_matmul(const BlockMatrix &a, const BlockMatrix &b, void *out, int64_t m, int64_t n, int64_t k,
                                bool bf16, cudaStream_t st)
{
    const int sms = device_sm_count();
    const int blocks = (int)((k + 127) / 128);
    auto up = [](int64_t v, int64_t to) { return (v + to - 1) / to; };
    // Few tokens: the weights take the MMA's rows, the tokens its columns, so no
    // row of the MMA is idle.
    const bool swap = m <= 128 && n > m;
    const BlockMatrix &ra = swap ? b : a, &rb = swap ? a : b;
    const int64_t rm = swap ? n : m, rn = swap ? m : n;
    int bn = rn <= 32 ? 32 : rn <= 64 ? 64 : 128;
    if (!swap && rn > 128 && up(rm, kRows) * up(rn, 256) * 4 >= 3 * sms)
        bn = 256;
    Params p = {};
    p.m_tiles = (int)up(rm, kRows);
    p.n_tiles = (int)up(rn, bn);
    p.blocks = blocks;
    p.splits = 1;
    if (bn < 256) {
        const int64_t tiles = (int64_t)p.m_tiles * p.n_tiles;
        p.splits = (int)std::max<int64_t>(1, std::min<int64_t>({2 * sms / tiles, (int64_t)kMostSplits, blocks / 2}));
    }
    p.sa = ra.scale;
    p.sa_row = ra.scale_row;
    p.sa_block = ra.scale_block;
    p.sa_shift = ra.tile ? 7 : 0;
    p.sb = rb.scale;
    p.sb_row = rb.scale_row;
    p.sb_block = rb.scale_block;
    p.sb_shift = rb.tile ? 7 : 0;
    p.out = out;
    p.ld = n;
    p.m = rm;
    p.n = rn;
    p.idesc = idesc_f8(kRows, bn, ra.e5m2 ? 1 : 0, rb.e5m2 ? 1 : 0);
    p.bf16 = bf16;
    const int64_t vec = bf16 ? 8 : 4;
    p.vec = n % vec == 0 && (reinterpret_cast<uintptr_t>(out) & 15u) == 0;
    p.status = device_status_word();
    if (!p.status)
        return cudaErrorUnknown;
    CUtensorMap ta, tb;
    if (!make_tmap_bytes(&ta, ra.q, (uint64_t)k, (uint64_t)rm, (uint64_t)ra.row, kRows) ||
        !make_tmap_bytes(&tb, rb.q, (uint64_t)k, (uint64_t)rn, (uint64_t)rb.row, (uint32_t)bn))
        return cudaErrorInvalidValue;
#define SSD_BLOCK_MATMUL(BN, SWAP)                                                            \
    return rb.tile ? launch<BN, SWAP, false>(ta, tb, p, sms, st) : launch<BN, SWAP, true>(ta, tb, p, sms, st)
    if (swap) {
        if (bn == 32)
            SSD_BLOCK_MATMUL(32, true);
        if (bn == 64)
            SSD_BLOCK_MATMUL(64, true);
        SSD_BLOCK_MATMUL(128, true);
    }
    if (bn == 32)
        SSD_BLOCK_MATMUL(32, false);
    if (bn == 64)
        SSD_BLOCK_MATMUL(64, false);
    if (bn == 128)
        SSD_BLOCK_MATMUL(128, false);
    SSD_BLOCK_MATMUL(256, false);
#undef SSD_BLOCK_MATMUL
}

}  // namespace ssd
