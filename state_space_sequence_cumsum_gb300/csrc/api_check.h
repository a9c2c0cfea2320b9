// Argument checks of the layer operators' entry points.
#pragma once
#include <cstdint>
#include <initializer_list>

#include "ssd_internal.h"

namespace ssd {

#define SSD_TRY(expr)                                  \
    do {                                               \
        ssd_status_t _s = (expr);                      \
        if (_s != SSD_OK)                              \
            return _s;                                 \
    } while (0)

inline ssd_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

inline size_t elem(ssd_dtype_t t) { return t == SSD_BF16 ? 2 : 4; }
inline bool known(ssd_dtype_t t) { return t == SSD_BF16 || t == SSD_F32; }

// A memory range a call reads or writes.
struct Range {
    const void *p;
    size_t bytes;
    size_t align;
    bool required;
};

inline ssd_status_t check_range(const Range &r)
{
    if (!r.p)
        return r.required && r.bytes ? SSD_ERR_INVALID_ARG : SSD_OK;
    return reinterpret_cast<uintptr_t>(r.p) % r.align == 0 ? SSD_OK : SSD_ERR_ALIGNMENT;
}

inline bool overlap(const Range &a, const Range &b)
{
    if (!a.p || !b.p || !a.bytes || !b.bytes)
        return false;
    const char *p = static_cast<const char *>(a.p), *q = static_cast<const char *>(b.p);
    return p < q + b.bytes && q < p + a.bytes;
}

// Pointers present and aligned; no output overlaps an input or another
// output, except that output `out` may be exactly input `in` (may_alias).
inline ssd_status_t check_all(std::initializer_list<Range> in, std::initializer_list<Range> out, int alias_out = -1,
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
inline size_t strided(int64_t rows, int64_t row, int64_t len, size_t esz)
{
    return rows > 0 ? (size_t)((rows - 1) * row + len) * esz : 0;
}

inline ssd_status_t check_ws(const void *ws, size_t have, size_t need)
{
    if (need == 0)
        return SSD_OK;
    return (!ws || have < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) ? SSD_ERR_WORKSPACE : SSD_OK;
}

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace ssd
