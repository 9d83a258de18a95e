// Checks of arguments that the operators' C entry points share (host side).
#pragma once
#include <cstdint>

#include "gg_ops.h"

namespace gg {

constexpr int64_t kMaxSize = ((int64_t)1 << 31) - 1;

// A rows x cols matrix argument of a call (element size es, pitch in elements).
struct Mat {
    const char *name;
    const void *p;
    int64_t rows, cols, ld, es;

    uint64_t begin() const { return reinterpret_cast<uint64_t>(p); }
    uint64_t bytes() const
    {
        return rows > 0 && cols > 0 ? (uint64_t)((rows - 1) * ld + cols) * (uint64_t)es : 0;
    }
};

// Whether two matrices share an element's bytes.  Matrices of one pitch may
// interleave (column ranges of one buffer): their rows are compared then.
inline bool share(const Mat &a, const Mat &b)
{
    if (!a.p || !b.p || a.bytes() == 0 || b.bytes() == 0)
        return false;
    if (a.begin() + a.bytes() <= b.begin() || b.begin() + b.bytes() <= a.begin())
        return false;
    const uint64_t pa = (uint64_t)(a.ld * a.es), pb = (uint64_t)(b.ld * b.es);
    if (pa != pb || a.rows < 2 || b.rows < 2)
        return true;
    const Mat &lo = a.begin() <= b.begin() ? a : b, &hi = a.begin() <= b.begin() ? b : a;
    const uint64_t shift = (hi.begin() - lo.begin()) % pa;  // hi's first column within lo's row
    const uint64_t wl = (uint64_t)(lo.cols * lo.es), wh = (uint64_t)(hi.cols * hi.es);
    return !(shift >= wl && shift + wh <= pa);
}

inline bool same(const Mat &a, const Mat &b) { return a.p == b.p && a.ld == b.ld; }

inline gg_status check_mat(const Mat &m, bool needed)
{
    if (m.rows == 0 || m.cols == 0)
        return GG_OK;
    if (!m.p)
        return needed ? op_fail(GG_ERR_INVALID_ARG, "%s must be non-NULL", m.name) : GG_OK;
    if (m.ld < m.cols)
        return op_fail(GG_ERR_INVALID_ARG, "%s: the pitch %lld is below the row length %lld", m.name,
                       (long long)m.ld, (long long)m.cols);
    if (m.ld > INT64_MAX / 16 / (m.rows > 0 ? m.rows : 1))
        return op_fail(GG_ERR_UNSUPPORTED, "%s: its extent passes 2^59 bytes", m.name);
    if (m.begin() % (uint64_t)m.es != 0)
        return op_fail(GG_ERR_ALIGNMENT, "%s must be aligned to its %lld-byte elements", m.name,
                       (long long)m.es);
    return GG_OK;
}

// Matrices that tensor maps (or 16-byte loads) read.
inline gg_status check_tma(const Mat &m)
{
    if (m.rows == 0 || m.cols == 0)
        return GG_OK;
    if (m.begin() % 16 != 0 || m.ld % 8 != 0)
        return op_fail(GG_ERR_ALIGNMENT, "%s must be 16-byte aligned with a pitch that is a multiple "
                                         "of 8", m.name);
    if (m.ld >= (int64_t)1 << 39)  // a tensor map's strides are below 2^40 bytes
        return op_fail(GG_ERR_UNSUPPORTED, "%s: its pitch must be below 2^39 elements", m.name);
    return GG_OK;
}

inline gg_status check_apart(const Mat &out, const Mat &other)
{
    return share(out, other) ? op_fail(GG_ERR_INVALID_ARG, "%s overlaps %s", out.name, other.name)
                             : GG_OK;
}

inline gg_status check_sizes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0)
        return op_fail(GG_ERR_INVALID_ARG, "sizes must be >= 0");
    if (M > kMaxSize || N > kMaxSize || K > kMaxSize)
        return op_fail(GG_ERR_UNSUPPORTED, "sizes must be below 2^31");
    return GG_OK;
}

inline gg_status check_types(gg_dtype dtype, gg_activation act, const char *what)
{
    if (dtype != GG_F16 && dtype != GG_BF16)
        return op_fail(GG_ERR_UNSUPPORTED, "%s takes GG_F16 or GG_BF16", what);
    if (act < GG_ACT_NONE || act > GG_ACT_SILU)
        return op_fail(GG_ERR_INVALID_ARG, "unknown activation %d", (int)act);
    return GG_OK;
}

inline gg_status check_route(gg_weight_layout layout, gg_linear_path path)
{
    if (layout != GG_WEIGHT_KN && layout != GG_WEIGHT_NK)
        return op_fail(GG_ERR_INVALID_ARG, "unknown weight layout %d", (int)layout);
    if (path != GG_LINEAR_AUTO && path != GG_LINEAR_SPLIT && path != GG_LINEAR_PAIR)
        return op_fail(GG_ERR_INVALID_ARG, "unknown linear path %d", (int)path);
    return GG_OK;
}

}  // namespace gg

#define GG_TRY(x)                  \
    do {                           \
        const gg_status st_ = (x); \
        if (st_ != GG_OK)          \
            return st_;            \
    } while (0)
