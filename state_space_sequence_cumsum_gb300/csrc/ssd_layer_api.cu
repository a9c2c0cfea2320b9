// C ABI of the layer operators around the scan: argument validation and
// workspace layout.  See include/ssd.h for the contract of every entry point.
#include <initializer_list>

#include "common.cuh"
#include "ssd_internal.h"

namespace ssd {

int device_sm_count()
{
    static std::atomic<int> known[kSmemDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();  // sizes are also asked for where there is no device
        return 152;
    }
    if (dev < kSmemDevices && (n = known[dev].load(std::memory_order_relaxed)) > 0)
        return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) {
        cudaGetLastError();
        return 152;
    }
    if (dev < kSmemDevices)
        known[dev].store(n, std::memory_order_relaxed);
    return n;
}

cudaError_t allow_smem(const void *kernel, size_t bytes, SmemGrant *granted)
{
    if (bytes <= 40 * 1024)  // with the kernels' static arrays, within what any kernel may take
        return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    return raise_smem(*granted, dev, bytes, [&](int n) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, n);
    });
}

namespace {

#define SSD_TRY(expr)                                  \
    do {                                               \
        ssd_status_t _s = (expr);                      \
        if (_s != SSD_OK)                              \
            return _s;                                 \
    } while (0)

ssd_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

size_t elem(ssd_dtype_t t) { return t == SSD_BF16 ? 2 : 4; }
bool known(ssd_dtype_t t) { return t == SSD_BF16 || t == SSD_F32; }

// A memory range a call reads or writes.
struct Range {
    const void *p;
    size_t bytes;
    size_t align;
    bool required;
};

ssd_status_t check_range(const Range &r)
{
    if (!r.p)
        return r.required && r.bytes ? SSD_ERR_INVALID_ARG : SSD_OK;
    return reinterpret_cast<uintptr_t>(r.p) % r.align == 0 ? SSD_OK : SSD_ERR_ALIGNMENT;
}

bool overlap(const Range &a, const Range &b)
{
    if (!a.p || !b.p || !a.bytes || !b.bytes)
        return false;
    const char *p = static_cast<const char *>(a.p), *q = static_cast<const char *>(b.p);
    return p < q + b.bytes && q < p + a.bytes;
}

// Pointers present and aligned; no output overlaps an input or another
// output, except that output `out` may be exactly input `in` (may_alias).
ssd_status_t check_all(std::initializer_list<Range> in, std::initializer_list<Range> out, int alias_out = -1,
                       int alias_in = -1)
{
    for (const Range &r : in)
        SSD_TRY(check_range(r));
    for (const Range &r : out)
        SSD_TRY(check_range(r));
    int o = 0;
    for (const Range &a : out) {
        int i = 0;
        for (const Range &b : in) {
            const bool same = o == alias_out && i == alias_in && a.p == b.p;
            if (!same && overlap(a, b))
                return SSD_ERR_INVALID_ARG;
            ++i;
        }
        int k = 0;
        for (const Range &b : out)
            if (k++ < o && overlap(a, b))
                return SSD_ERR_INVALID_ARG;
        ++o;
    }
    return SSD_OK;
}

// Bytes of `rows` rows `row` elements apart, the last one `len` long.
size_t strided(int64_t rows, int64_t row, int64_t len, size_t esz)
{
    return rows > 0 ? (size_t)((rows - 1) * row + len) * esz : 0;
}

ssd_status_t check_ws(const void *ws, size_t have, size_t need)
{
    if (need == 0)
        return SSD_OK;
    return (!ws || have < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) ? SSD_ERR_WORKSPACE : SSD_OK;
}

constexpr double kMostElems = 4e15;

// ------------------------------------------------------------- convolution

ssd_status_t conv_geom(const ssd_conv_dims_t &d, int64_t row, int64_t row_dy, int silu, ConvGeom *g)
{
    if (d.batch < 1 || d.seqlen < 0 || d.dim < 1 || d.width < 1 || row < d.dim || row_dy < d.dim)
        return SSD_ERR_INVALID_ARG;
    if (d.width < 2 || d.width > 4 || d.batch > 65535 || d.dim > (1LL << 24) || d.seqlen > (1LL << 40) ||
        (double)d.batch * (double)(d.seqlen + 4) * (double)row > kMostElems ||
        (double)d.batch * (double)(d.seqlen + 4) * (double)row_dy > kMostElems ||
        // one thread per token in the worst case, 256 a block
        (double)d.batch * (double)d.seqlen * (double)d.dim > 256.0 * 2147483647.0)
        return SSD_ERR_UNSUPPORTED;
    g->batch = d.batch;
    g->seqlen = d.seqlen;
    g->dim = d.dim;
    g->row = row;
    g->row_dy = row_dy;
    g->width = (int)d.width;
    g->silu = silu != 0;
    return SSD_OK;
}

// --------------------------------------------------------------- the scan

ssd_status_t scan_geom(const ssd_scan_dims_t &d, const ssd_scan_rows_t &r, bool has_z, bool has_dy,
                       int softplus, ScanGeom *g)
{
    if (d.batch < 1 || d.seqlen < 0 || d.dim < 1 || d.dstate < 1 || d.ngroups < 1 || d.dim % d.ngroups != 0)
        return SSD_ERR_INVALID_ARG;
    if (d.dstate > 64 || d.batch > 65535 || d.dim > (1LL << 24) || d.seqlen > (1LL << 35))
        return SSD_ERR_UNSUPPORTED;
    const int64_t bc = d.ngroups * d.dstate;
    if (r.u < d.dim || r.dt < d.dim || (has_z && r.z < d.dim) || r.b < bc || r.c < bc || (has_dy && r.dy < d.dim))
        return SSD_ERR_INVALID_ARG;
    const double tokens = (double)d.batch * (double)(d.seqlen + scan_chunk());
    for (int64_t row : {r.u, r.dt, has_z ? r.z : (int64_t)1, r.b, r.c, has_dy ? r.dy : (int64_t)1,
                        d.dim * d.dstate})
        if (tokens * (double)row > kMostElems)
            return SSD_ERR_UNSUPPORTED;
    // one element per thread, 256 a block, in the sums over channel blocks and in the step
    if (2.0 * tokens * (double)bc > 256.0 * 2147483647.0 || (double)d.batch * d.dim * d.dstate * 4 > 256.0 * 2147483647.0)
        return SSD_ERR_UNSUPPORTED;
    g->batch = d.batch;
    g->seqlen = d.seqlen;
    g->dim = d.dim;
    g->N = d.dstate;
    g->G = d.ngroups;
    g->kpg = d.dim / d.ngroups;
    g->row_u = r.u;
    g->row_dt = r.dt;
    g->row_z = r.z;
    g->row_b = r.b;
    g->row_c = r.c;
    g->row_dy = r.dy;
    g->softplus = softplus != 0;
    return SSD_OK;
}

// The geometry of contiguous rows, for the size functions.
bool scan_geom_sizes(const ssd_scan_dims_t &d, ScanGeom *g)
{
    const int64_t bc = d.ngroups * d.dstate;
    const ssd_scan_rows_t r{d.dim, d.dim, d.dim, bc, bc, d.dim};
    return scan_geom(d, r, true, true, 0, g) == SSD_OK;
}

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

int64_t kept_elems(const ScanGeom &g)
{
    return g.batch * ((g.seqlen + scan_chunk() - 1) / scan_chunk()) * g.dim * g.N;
}

// Workspace of the backward: the forward's kept states where the caller has
// none, the reverse pass's, and what the passes and the gradients use.
struct BwdWs {
    float *kept, *dkept;
    void *pass, *grad;
    size_t bytes;
};
BwdWs scan_bwd_layout(const ScanGeom &g, bool have_kept, char *base)
{
    BwdWs w{};
    size_t off = 0;
    auto take = [&](size_t n) {
        char *p = base ? base + off : nullptr;
        off += round256(n);
        return p;
    };
    w.kept = have_kept ? nullptr : reinterpret_cast<float *>(take((size_t)kept_elems(g) * 4));
    w.dkept = reinterpret_cast<float *>(take((size_t)kept_elems(g) * 4));
    const size_t fwd = have_kept ? 0 : scan_pass_workspace(g), rev = scan_reverse_workspace(g);
    w.pass = take(fwd > rev ? fwd : rev);
    w.grad = take(scan_grad_workspace(g));
    w.bytes = off;
    return w;
}

ssd_status_t copy_or_zero(void *dst, const void *src, size_t bytes, cudaStream_t st)
{
    if (!dst || dst == src || !bytes)
        return SSD_OK;
    return cuda_status(src ? cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToDevice, st)
                           : cudaMemsetAsync(dst, 0, bytes, st));
}

// ---------------------------------------------------------------- the norm

ssd_status_t norm_geom(int64_t ntokens, int64_t dim, int64_t gate_rows, float scale, float eps, NormGeom *g)
{
    if (ntokens < 0 || dim < 1 || gate_rows < 0 || !(eps >= 0.f) || eps > 1e30f)
        return SSD_ERR_INVALID_ARG;
    if (gate_rows > 0 && ntokens % gate_rows != 0)
        return SSD_ERR_INVALID_ARG;
    if (dim > 32768 || ntokens > 2147483647LL)
        return SSD_ERR_UNSUPPORTED;
    g->ntokens = ntokens;
    g->dim = dim;
    g->tokens_per_gate = gate_rows > 0 && ntokens > 0 ? ntokens / gate_rows : 1;
    g->scale = scale;
    g->eps = eps;
    g->inv_dim = 1.f / (float)dim;
    return SSD_OK;
}

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

ssd_status_t ssd_causal_conv(const void *x, int64_t row, const float *weight, const float *bias,
                             const void *initial_state, void *y, void *final_state, ssd_conv_dims_t dims,
                             int silu, ssd_dtype_t dtype, void *stream)
{
    ConvGeom g;
    SSD_TRY(conv_geom(dims, row, row, silu, &g));
    if (!known(dtype))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), state = (size_t)(g.batch * (g.width - 1) * g.dim) * e;
    SSD_TRY(check_all({{x, strided(g.batch * g.seqlen, row, g.dim, e), e, true},
                       {weight, (size_t)(g.dim * g.width) * 4, 4, true},
                       {bias, (size_t)g.dim * 4, 4, false},
                       {initial_state, state, e, false}},
                      {{y, (size_t)(g.batch * g.seqlen * g.dim) * e, e, true}, {final_state, state, e, false}}));
    cudaStream_t st = (cudaStream_t)stream;
    if (g.seqlen == 0)
        return copy_or_zero(final_state, initial_state, state, st);
    return cuda_status(launch_conv(x, weight, bias, initial_state, y, final_state, g, dtype == SSD_BF16, st));
}

size_t ssd_causal_conv_bwd_workspace_size(ssd_conv_dims_t dims)
{
    ConvGeom g;
    if (conv_geom(dims, dims.dim, dims.dim, 0, &g) != SSD_OK)
        return 0;
    return round256(conv_bwd_workspace(g));
}

ssd_status_t ssd_causal_conv_bwd(const void *x, int64_t row, const float *weight, const float *bias,
                                 const void *initial_state, const void *dy, int64_t row_dy, const void *dfinal,
                                 void *dx, float *dweight, float *dbias, void *dinit, ssd_conv_dims_t dims,
                                 int silu, ssd_dtype_t dtype, void *workspace, size_t workspace_bytes,
                                 void *stream)
{
    ConvGeom g;
    SSD_TRY(conv_geom(dims, row, row_dy, silu, &g));
    if (!known(dtype))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), state = (size_t)(g.batch * (g.width - 1) * g.dim) * e;
    const size_t need = ssd_causal_conv_bwd_workspace_size(dims);
    SSD_TRY(check_all({{x, strided(g.batch * g.seqlen, row, g.dim, e), e, true},
                       {weight, (size_t)(g.dim * g.width) * 4, 4, true},
                       {bias, (size_t)g.dim * 4, 4, false},
                       {initial_state, state, e, false},
                       {dy, strided(g.batch * g.seqlen, row_dy, g.dim, e), e, true},
                       {dfinal, state, e, false}},
                      {{dx, (size_t)(g.batch * g.seqlen * g.dim) * e, e, true},
                       {dweight, (size_t)(g.dim * g.width) * 4, 4, true},
                       {dbias, (size_t)g.dim * 4, 4, false},
                       {dinit, state, e, false},
                       {workspace, need, 1, false}}));
    SSD_TRY(check_ws(workspace, workspace_bytes, need));
    return cuda_status(launch_conv_bwd(x, weight, bias, initial_state, dy, dfinal, dx, dweight, dbias, dinit,
                                       static_cast<float *>(workspace), g, dtype == SSD_BF16,
                                       (cudaStream_t)stream));
}

ssd_status_t ssd_causal_conv_step(const void *x, int64_t row, const float *weight, const float *bias,
                                  const void *state, void *state_out, void *y, ssd_conv_dims_t dims, int silu,
                                  ssd_dtype_t dtype, void *stream)
{
    ConvGeom g;
    if (dims.seqlen != 1)
        return SSD_ERR_INVALID_ARG;
    SSD_TRY(conv_geom(dims, row, row, silu, &g));
    if (!known(dtype))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), sb = (size_t)(g.batch * (g.width - 1) * g.dim) * e;
    SSD_TRY(check_all({{state, sb, e, true},
                       {x, strided(g.batch, row, g.dim, e), e, true},
                       {weight, (size_t)(g.dim * g.width) * 4, 4, true},
                       {bias, (size_t)g.dim * 4, 4, false}},
                      {{state_out, sb, e, true}, {y, (size_t)(g.batch * g.dim) * e, e, true}}, 0, 0));
    return cuda_status(launch_conv_step(x, weight, bias, state, state_out, y, g, dtype == SSD_BF16,
                                        (cudaStream_t)stream));
}

int ssd_selective_scan_chunk(void) { return scan_chunk(); }

size_t ssd_selective_scan_workspace_size(ssd_scan_dims_t dims)
{
    ScanGeom g;
    return scan_geom_sizes(dims, &g) ? round256(scan_pass_workspace(g)) : 0;
}

ssd_status_t ssd_selective_scan(const void *u, const void *dt, const float *A, const void *Bm, const void *Cm,
                                const float *D, const void *z, const float *dt_bias,
                                const float *initial_state, void *y, float *final_state, float *chunk_states,
                                ssd_scan_dims_t dims, ssd_scan_rows_t rows, int dt_softplus, ssd_dtype_t dtype,
                                void *workspace, size_t workspace_bytes, void *stream)
{
    ScanGeom g;
    SSD_TRY(scan_geom(dims, rows, z != nullptr, false, dt_softplus, &g));
    if (!known(dtype))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), sb = (size_t)(g.batch * g.dim * g.N) * 4;
    const int64_t tokens = g.batch * g.seqlen;
    const size_t need = round256(scan_pass_workspace(g));
    SSD_TRY(check_all({{initial_state, sb, 4, false},
                       {u, strided(tokens, rows.u, g.dim, e), e, true},
                       {dt, strided(tokens, rows.dt, g.dim, e), e, true},
                       {A, (size_t)(g.dim * g.N) * 4, 4, true},
                       {Bm, strided(tokens, rows.b, g.G * g.N, e), e, true},
                       {Cm, strided(tokens, rows.c, g.G * g.N, e), e, true},
                       {D, (size_t)g.dim * 4, 4, false},
                       {z, strided(tokens, rows.z, g.dim, e), e, false},
                       {dt_bias, (size_t)g.dim * 4, 4, false}},
                      {{final_state, sb, 4, false},
                       {y, (size_t)(tokens * g.dim) * e, e, true},
                       {chunk_states, (size_t)kept_elems(g) * 4, 4, false},
                       {workspace, need, 1, false}},
                      0, 0));
    SSD_TRY(check_ws(workspace, workspace_bytes, need));
    cudaStream_t st = (cudaStream_t)stream;
    if (g.seqlen == 0)
        return copy_or_zero(final_state, initial_state, sb, st);
    return cuda_status(launch_selective_scan(u, dt, A, Bm, Cm, D, z, dt_bias, initial_state, y, final_state,
                                             chunk_states, workspace, g, dtype == SSD_BF16, st));
}

size_t ssd_selective_scan_bwd_workspace_size(ssd_scan_dims_t dims, int have_chunk_states)
{
    ScanGeom g;
    if (!scan_geom_sizes(dims, &g) || g.seqlen == 0)
        return 0;
    return scan_bwd_layout(g, have_chunk_states != 0, nullptr).bytes;
}

ssd_status_t ssd_selective_scan_bwd(const void *u, const void *dt, const float *A, const void *Bm,
                                    const void *Cm, const float *D, const void *z, const float *dt_bias,
                                    const float *initial_state, const void *dy, const float *dfinal,
                                    const float *chunk_states, void *du, void *ddt, float *dA, void *dB,
                                    void *dC, float *dD, void *dz, float *ddt_bias, float *dinit,
                                    ssd_scan_dims_t dims, ssd_scan_rows_t rows, int dt_softplus,
                                    ssd_dtype_t dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    ScanGeom g;
    SSD_TRY(scan_geom(dims, rows, z != nullptr, true, dt_softplus, &g));
    if (!known(dtype) || (dD && !D) || (dz && !z))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), sb = (size_t)(g.batch * g.dim * g.N) * 4;
    const int64_t tokens = g.batch * g.seqlen;
    const size_t full = (size_t)(tokens * g.dim) * e, bc = (size_t)(tokens * g.G * g.N) * e;
    const size_t need = ssd_selective_scan_bwd_workspace_size(dims, chunk_states != nullptr);
    SSD_TRY(check_all({{u, strided(tokens, rows.u, g.dim, e), e, true},
                       {dt, strided(tokens, rows.dt, g.dim, e), e, true},
                       {A, (size_t)(g.dim * g.N) * 4, 4, true},
                       {Bm, strided(tokens, rows.b, g.G * g.N, e), e, true},
                       {Cm, strided(tokens, rows.c, g.G * g.N, e), e, true},
                       {D, (size_t)g.dim * 4, 4, false},
                       {z, strided(tokens, rows.z, g.dim, e), e, false},
                       {dt_bias, (size_t)g.dim * 4, 4, false},
                       {initial_state, sb, 4, false},
                       {dy, strided(tokens, rows.dy, g.dim, e), e, true},
                       {dfinal, sb, 4, false},
                       {chunk_states, (size_t)kept_elems(g) * 4, 4, false}},
                      {{du, full, e, true},
                       {ddt, full, e, true},
                       {dA, (size_t)(g.dim * g.N) * 4, 4, true},
                       {dB, bc, e, true},
                       {dC, bc, e, true},
                       {dD, (size_t)g.dim * 4, 4, false},
                       {dz, full, e, z != nullptr},
                       {ddt_bias, (size_t)g.dim * 4, 4, false},
                       {dinit, sb, 4, false},
                       {workspace, need, 1, false}}));
    SSD_TRY(check_ws(workspace, workspace_bytes, need));
    cudaStream_t st = (cudaStream_t)stream;
    if (g.seqlen == 0) {
        SSD_TRY(copy_or_zero(dA, nullptr, (size_t)(g.dim * g.N) * 4, st));
        SSD_TRY(copy_or_zero(dD, nullptr, (size_t)g.dim * 4, st));
        SSD_TRY(copy_or_zero(ddt_bias, nullptr, (size_t)g.dim * 4, st));
        return copy_or_zero(dinit, dfinal, sb, st);
    }
    const bool bf16 = dtype == SSD_BF16;
    const BwdWs w = scan_bwd_layout(g, chunk_states != nullptr, static_cast<char *>(workspace));
    if (!chunk_states) {
        SSD_TRY(cuda_status(launch_selective_scan(u, dt, A, Bm, Cm, D, z, dt_bias, initial_state, nullptr,
                                                  nullptr, w.kept, w.pass, g, bf16, st)));
        chunk_states = w.kept;
    }
    ScanEnter enter;
    SSD_TRY(cuda_status(launch_scan_reverse(dy, dt, A, Cm, z, dt_bias, dfinal, w.dkept, dinit, w.pass, &enter, g, bf16,
                                            st)));
    return cuda_status(launch_scan_grad(u, dt, A, Bm, Cm, D, z, dt_bias, dy, chunk_states, w.dkept, enter, du, ddt,
                                        dA, dB, dC, dD, dz, ddt_bias, w.grad, g, bf16, st));
}

ssd_status_t ssd_selective_scan_step(const void *u, const void *dt, const float *A, const void *Bm,
                                     const void *Cm, const float *D, const void *z, const float *dt_bias,
                                     const float *state, float *state_out, void *y, ssd_scan_dims_t dims,
                                     ssd_scan_rows_t rows, int dt_softplus, ssd_dtype_t dtype, void *stream)
{
    ScanGeom g;
    if (dims.seqlen != 1)
        return SSD_ERR_INVALID_ARG;
    SSD_TRY(scan_geom(dims, rows, z != nullptr, false, dt_softplus, &g));
    if (!known(dtype))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), sb = (size_t)(g.batch * g.dim * g.N) * 4;
    SSD_TRY(check_all({{state, sb, 4, true},
                       {u, strided(g.batch, rows.u, g.dim, e), e, true},
                       {dt, strided(g.batch, rows.dt, g.dim, e), e, true},
                       {A, (size_t)(g.dim * g.N) * 4, 4, true},
                       {Bm, strided(g.batch, rows.b, g.G * g.N, e), e, true},
                       {Cm, strided(g.batch, rows.c, g.G * g.N, e), e, true},
                       {D, (size_t)g.dim * 4, 4, false},
                       {z, strided(g.batch, rows.z, g.dim, e), e, false},
                       {dt_bias, (size_t)g.dim * 4, 4, false}},
                      {{state_out, sb, 4, true}, {y, (size_t)(g.batch * g.dim) * e, e, true}}, 0, 0));
    return cuda_status(launch_scan_step(u, dt, A, Bm, Cm, D, z, dt_bias, state, state_out, y, g,
                                        dtype == SSD_BF16, (cudaStream_t)stream));
}

ssd_status_t ssd_block_norm(const void *y, const void *residual, const float *weight, const float *post_weight,
                            const float *gate, void *out, void *residual_out, int64_t ntokens, int64_t dim,
                            int64_t gate_rows, float scale, float eps, ssd_dtype_t dtype,
                            ssd_dtype_t residual_dtype, void *stream)
{
    NormGeom g;
    SSD_TRY(norm_geom(ntokens, dim, gate_rows, scale, eps, &g));
    if (!known(dtype) || (residual_dtype != dtype && residual_dtype != SSD_F32) || (gate != nullptr) != (gate_rows > 0))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), er = elem(residual_dtype), n = (size_t)(ntokens * dim);
    SSD_TRY(check_all({{residual, n * er, er, false},
                       {y, n * e, e, true},
                       {weight, (size_t)dim * 4, 4, true},
                       {post_weight, (size_t)dim * 4, 4, false},
                       {gate, (size_t)(gate_rows * dim) * 4, 4, false}},
                      {{residual_out, n * er, er, true}, {out, n * e, e, true}}, 0, 0));
    return cuda_status(launch_block_norm(y, residual, weight, post_weight, gate, out, residual_out, g,
                                         dtype == SSD_BF16, residual_dtype == SSD_BF16, (cudaStream_t)stream));
}

size_t ssd_block_norm_bwd_workspace_size(int64_t ntokens, int64_t dim, int64_t gate_rows)
{
    NormGeom g;
    if (norm_geom(ntokens, dim, gate_rows, 1.f, 0.f, &g) != SSD_OK || ntokens == 0)
        return 0;
    return round256(block_norm_bwd_workspace(g, gate_rows > 0));
}

ssd_status_t ssd_block_norm_bwd(const void *y, const void *residual_out, const float *weight,
                                const float *post_weight, const float *gate, const void *dout,
                                const void *dresidual_out, void *dy, void *dresidual, float *dweight,
                                float *dpost_weight, float *dgate, int64_t ntokens, int64_t dim,
                                int64_t gate_rows, float scale, float eps, ssd_dtype_t dtype,
                                ssd_dtype_t residual_dtype, void *workspace, size_t workspace_bytes,
                                void *stream)
{
    NormGeom g;
    SSD_TRY(norm_geom(ntokens, dim, gate_rows, scale, eps, &g));
    if (!known(dtype) || (residual_dtype != dtype && residual_dtype != SSD_F32) ||
        (gate != nullptr) != (gate_rows > 0) || (post_weight != nullptr) != (dpost_weight != nullptr) ||
        (gate != nullptr) != (dgate != nullptr))
        return SSD_ERR_INVALID_ARG;
    const size_t e = elem(dtype), er = elem(residual_dtype), n = (size_t)(ntokens * dim);
    const size_t need = ssd_block_norm_bwd_workspace_size(ntokens, dim, gate_rows);
    SSD_TRY(check_all({{dresidual_out, n * er, er, false},
                       {y, n * e, e, true},
                       {residual_out, n * er, er, true},
                       {weight, (size_t)dim * 4, 4, true},
                       {post_weight, (size_t)dim * 4, 4, false},
                       {gate, (size_t)(gate_rows * dim) * 4, 4, false},
                       {dout, n * e, e, true}},
                      {{dresidual, n * er, er, true},
                       {dy, n * e, e, true},
                       {dweight, (size_t)dim * 4, 4, true},
                       {dpost_weight, (size_t)dim * 4, 4, false},
                       {dgate, (size_t)(gate_rows * dim) * 4, 4, false},
                       {workspace, need, 1, false}},
                      0, 0));
    SSD_TRY(check_ws(workspace, workspace_bytes, need));
    cudaStream_t st = (cudaStream_t)stream;
    if (ntokens == 0) {
        SSD_TRY(copy_or_zero(dweight, nullptr, (size_t)dim * 4, st));
        SSD_TRY(copy_or_zero(dpost_weight, nullptr, (size_t)dim * 4, st));
        return copy_or_zero(dgate, nullptr, (size_t)(gate_rows * dim) * 4, st);
    }
    return cuda_status(launch_block_norm_bwd(y, residual_out, weight, post_weight, gate, dout, dresidual_out, dy,
                                             dresidual, dweight, dpost_weight, dgate,
                                             static_cast<float *>(workspace), g, dtype == SSD_BF16,
                                             residual_dtype == SSD_BF16, st));
}

}  // extern "C"
