// checks.hpp -- the argument checks that the C entry points on token rows
// share (internal): what a call reads and writes, rows and flat buffers, counts.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "errors.hpp"
#include "gdnq.h"

namespace gdnq {
namespace checks {

constexpr size_t HUGE_SPAN = (size_t)1 << 60;

// What a call reads and writes, to check that nothing written overlaps
// anything else.
struct Spans {
    static constexpr int MAX = 16;
    Span s[MAX];
    bool out[MAX];
    int n = 0;

    int add(const Span &x, bool written)
    {
        if (x.n >= HUGE_SPAN) return fail(GDNQ_EINVAL, "%s is larger than any memory", x.name);
        for (int i = 0; i < n; i++)
            if ((written || out[i]) && gdnq::overlap(x, s[i]))
                return fail(GDNQ_EINVAL, "%s overlaps %s", x.name, s[i].name);
        s[n] = x;
        out[n++] = written;
        return GDNQ_OK;
    }
};

enum Use { READ, WRITE };

// Product of sizes, HUGE_SPAN where it would reach that.
inline size_t bytes(size_t a, size_t b, size_t c = 1, size_t d = 1)
{
    const size_t f[3] = {b, c, d};
    for (size_t x : f) {
        if (x && a >= HUGE_SPAN / x) return HUGE_SPAN;
        a *= x;
    }
    return a;
}

// A contiguous buffer of n bytes.
inline int flat(Spans &sp, const void *p, size_t n, const char *name, Use use = READ, bool nullable = false)
{
    if (!p) return nullable ? GDNQ_OK : fail(GDNQ_EINVAL, "%s is NULL", name);
    if (!gdnq::aligned16(p)) return fail(GDNQ_EINVAL, "%s is not 16-byte aligned", name);
    return sp.add(Span{p, n, name}, use == WRITE);
}

// n >= 1 rows of `len` elements of es bytes, ld apart (0: len; the distance is
// filled in).
inline int rows(Spans &sp, const void *p, long long n, long long len, int64_t &ld, int es, const char *name,
                Use use = READ, bool nullable = false)
{
    if (ld == 0) ld = len;
    if (!p) return nullable ? GDNQ_OK : fail(GDNQ_EINVAL, "%s is NULL", name);
    if (ld < len)
        return fail(GDNQ_EINVAL, "rows of %s are %lld elements long but %lld apart", name, len, (long long)ld);
    if (reinterpret_cast<uintptr_t>(p) % (unsigned)es)
        return fail(GDNQ_EINVAL, "%s is not aligned to its element size", name);
    return sp.add(Span{p, bytes((size_t)(n - 1), (size_t)ld, es) + bytes((size_t)len, es), name}, use == WRITE);
}

#define TRY(call)              \
    do {                       \
        const int rc_ = (call); \
        if (rc_) return rc_;   \
    } while (0)

inline int check_io_dtype(int io)
{
    if (io != GDNQ_IO_F32 && io != GDNQ_IO_BF16)
        return fail(GDNQ_EINVAL, "io_dtype must be GDNQ_IO_F32 or GDNQ_IO_BF16 (got %d)", io);
    return GDNQ_OK;
}

inline int check_counts(int32_t n, int32_t T)
{
    if (n < 0) return fail(GDNQ_EINVAL, "n_seqs must be >= 0 (got %d)", n);
    if (T < 0) return fail(GDNQ_EINVAL, "T must be >= 0 (got %d)", T);
    return GDNQ_OK;
}

// Work items of one call; the kernels number them in 31 bits.
inline int check_grid(unsigned long long items, const char *what)
{
    if (items > 0x7ffffff0ULL) return fail(GDNQ_EINVAL, "%s too large", what);
    return GDNQ_OK;
}

inline int check_rows(int32_t n)
{
    if (n < 0) return fail(GDNQ_EINVAL, "rows must be >= 0 (got %d)", n);
    return GDNQ_OK;
}

inline hipStream_t stream_of(void *s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace checks
}  // namespace gdnq
