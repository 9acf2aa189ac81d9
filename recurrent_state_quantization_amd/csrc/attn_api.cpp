// attn_api.cpp -- the C ABI of include/gdnq_attn.h: argument checks on the
// host, then the launches of the call on the caller's stream.  Nothing is
// allocated and nothing is synchronized.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "attn_launchers.hpp"
#include "checks.hpp"
#include "gdnq_attn.h"

namespace {

using namespace gdnq::checks;
using gdnq::fail;
using gdnq::launched;
using gdnq::ok;
using gdnq::Span;

// By the exponent's bits: the sources are compiled for arithmetic without NaN.
bool finite(double x)
{
    uint64_t u;
    std::memcpy(&u, &x, 8);
    return (u >> 52 & 0x7FF) != 0x7FF;
}

bool positive(double x) { return finite(x) && x > 0.0; }

int item(int io) { return io == GDNQ_IO_BF16 ? 2 : 4; }

// The descriptor with its defaults filled in.
int check_rope(const gdnq_rope_desc *desc, gdnq_rope_desc &d)
{
    if (!desc) return fail(GDNQ_EINVAL, "desc is NULL");
    d = *desc;
    if (d.d < 2 || d.d > 1024 || d.d % 2) return fail(GDNQ_EUNSUPPORTED, "d must be even, 2 to 1024 (got %d)", d.d);
    if (d.rot == 0) d.rot = d.d;
    if (d.rot < 2 || d.rot > d.d || d.rot % 2)
        return fail(GDNQ_EINVAL, "rot must be even, 2 to d (0 means d; got rot=%d, d=%d)", d.rot, d.d);
    TRY(check_io_dtype(d.io_dtype));
    if (d.flags & ~(GDNQ_ROPE_INTERLEAVED | GDNQ_ROPE_INVERSE))
        return fail(GDNQ_EINVAL, "unknown flag bits 0x%x", d.flags);
    if (!positive(d.amp)) return fail(GDNQ_EINVAL, "amp must be > 0 (got %g)", (double)d.amp);
    return GDNQ_OK;
}

int check_freqs(const gdnq_rope_freqs *f, int rot)
{
    if (!f) return fail(GDNQ_EINVAL, "freqs is NULL");
    if (f->kind < GDNQ_ROPE_PLAIN || f->kind > GDNQ_ROPE_RAMP_INDEX)
        return fail(GDNQ_EINVAL, "unknown kind %d of frequencies", f->kind);
    if (!finite(f->base) || f->base <= 1.0) return fail(GDNQ_EINVAL, "base must be > 1 (got %g)", f->base);
    if (f->kind != GDNQ_ROPE_PLAIN && !positive(f->factor))
        return fail(GDNQ_EINVAL, "factor must be > 0 (got %g)", f->factor);
    if (f->kind >= GDNQ_ROPE_RAMP_TURNS) {
        if (!positive(f->orig_len)) return fail(GDNQ_EINVAL, "orig_len must be > 0 (got %g)", f->orig_len);
        if (!positive(f->lo) || !finite(f->hi) || f->lo >= f->hi)
            return fail(GDNQ_EINVAL, "0 < lo < hi is needed (got %g, %g)", f->lo, f->hi);
    }
    for (int i = 0; f->divisors && i < rot / 2; i++)
        if (!positive(f->divisors[i])) return fail(GDNQ_EINVAL, "divisors[%d] must be > 0", i);
    return GDNQ_OK;
}

// The descriptor with its defaults filled in.
int check_attn(const gdnq_attn_desc *desc, gdnq_attn_desc &d)
{
    if (!desc) return fail(GDNQ_EINVAL, "desc is NULL");
    d = *desc;
    if (d.H < 1) return fail(GDNQ_EINVAL, "H must be >= 1 (got %d)", d.H);
    if (d.hk < 0 || (d.hk > 0 && d.H % d.hk != 0))
        return fail(GDNQ_EINVAL, "hk must divide H (0 means H; got hk=%d, H=%d)", d.hk, d.H);
    if (d.hk == 0) d.hk = d.H;
    if (d.d != 64 && d.d != 128 && d.d != 256)
        return fail(GDNQ_EUNSUPPORTED, "d must be 64, 128 or 256 (got %d)", d.d);
    TRY(check_io_dtype(d.io_dtype));
    if (d.page < 8 || d.page > 65536 || (d.page & (d.page - 1)))
        return fail(GDNQ_EUNSUPPORTED, "page must be a power of two, 8 to 65536 (got %d)", d.page);
    if (d.window < 0) return fail(GDNQ_EINVAL, "window must be >= 0 (got %d)", d.window);
    if (!finite(d.scale) || d.scale < 0.0f)
        return fail(GDNQ_EINVAL, "scale must be >= 0 (got %g)", (double)d.scale);
    if (d.scale == 0.0f) d.scale = (float)(1.0 / std::sqrt((double)d.d));
    if (!finite(d.acc_decay) || d.acc_decay < 0.0f || d.acc_decay > 1.0f)
        return fail(GDNQ_EINVAL, "acc_decay must be in 0..1 (got %g)", (double)d.acc_decay);
    return GDNQ_OK;
}

// The cache's sizes, with the row distances filled in.
int check_sizes(const gdnq_attn_desc &d, const gdnq_kv *cache, gdnq_kv &kv)
{
    if (!cache) return fail(GDNQ_EINVAL, "kv is NULL");
    kv = *cache;
    if (kv.n_pages < 1) return fail(GDNQ_EINVAL, "n_pages must be >= 1 (got %d)", kv.n_pages);
    if (kv.n_slots < 1) return fail(GDNQ_EINVAL, "n_slots must be >= 1 (got %d)", kv.n_slots);
    if (kv.max_pages < 1) return fail(GDNQ_EINVAL, "max_pages must be >= 1 (got %d)", kv.max_pages);
    if ((long long)kv.max_pages * d.page > (1LL << 30))
        return fail(GDNQ_EUNSUPPORTED, "a slot holds at most 2^30 rows (got %d pages of %d)", kv.max_pages, d.page);
    if (kv.ldp == 0 && kv.ldh == 0 && kv.ldr == 0) {
        kv.ldr = d.d;
        kv.ldh = (int64_t)d.page * d.d;
        kv.ldp = d.hk * kv.ldh;
    }
    const int es = item(d.io_dtype);
    const int64_t far = (int64_t)1 << 48;
    if (kv.ldp < 0 || kv.ldh < 0 || kv.ldr < 0 || kv.ldp > far || kv.ldh > far || kv.ldr > far)
        return fail(GDNQ_EINVAL, "ldp, ldh and ldr must be in 0..2^48");
    if (kv.ldp * es % 16 || kv.ldh * es % 16 || kv.ldr * es % 16)
        return fail(GDNQ_EINVAL, "ldp, ldh and ldr must be multiples of 16 bytes");
    // heads around rows, or rows around heads, in pages; in 128 bits, which no product leaves
    const __int128 heads = d.hk - 1, rows = d.page - 1;
    if (rows && heads && kv.ldh >= (int64_t)1 << 40 && kv.ldr >= (int64_t)1 << 40)
        return fail(GDNQ_EINVAL, "ldh and ldr are both larger than any page");
    const bool hr = kv.ldr >= d.d && (!heads || kv.ldh >= rows * kv.ldr + d.d);
    const bool rh = (!heads || kv.ldh >= d.d) && kv.ldr >= heads * kv.ldh + d.d;
    if (!hr && !rh) return fail(GDNQ_EINVAL, "the rows of a page overlap (ldh=%lld, ldr=%lld)", (long long)kv.ldh,
                                (long long)kv.ldr);
    if (kv.n_pages > 1 && kv.ldp < heads * kv.ldh + rows * kv.ldr + d.d)
        return fail(GDNQ_EINVAL, "pages overlap (ldp=%lld)", (long long)kv.ldp);
    return GDNQ_OK;
}

// n copies of what the next level describes, ld bytes apart (at least as far as one of them reaches).
struct Level {
    int64_t n, ld;
};

// Whether two arrangements of rows of `len` bytes, the second x bytes behind the first, share no byte.
bool copies_apart(const Level *level, int levels, int64_t x, int64_t len)
{
    if (levels == 0) return x >= len || x <= -len;
    if (level->n == 1) return copies_apart(level + 1, levels - 1, x, len);
    // a copy reaches only those of the other arrangement that begin at most ld before or behind it
    const int64_t below = x / level->ld - (x % level->ld < 0);
    for (int64_t a = below; a <= below + 1; a++)
        if (a > -level->n && a < level->n && !copies_apart(level + 1, levels - 1, x - a * level->ld, len)) return false;
    return true;
}

// Whether no row of k shares a byte with one of v (the two of them in one pool, by pages, heads or rows).
bool rows_apart(const gdnq_attn_desc &d, const gdnq_kv &kv)
{
    const int es = item(d.io_dtype);
    const Level heads{d.hk, kv.ldh * es}, rows{d.page, kv.ldr * es};
    const bool outer = d.hk == 1 || kv.ldh >= (d.page - 1) * kv.ldr + d.d;   // heads around rows
    const Level level[3] = {{kv.n_pages, kv.ldp * es}, outer ? heads : rows, outer ? rows : heads};
    const int64_t x = reinterpret_cast<intptr_t>(kv.v) - reinterpret_cast<intptr_t>(kv.k);
    return copies_apart(level, 3, x, (int64_t)d.d * es);
}

// The cache's buffers and their uses (`use` of k and v).
int check_cache(const gdnq_attn_desc &d, const gdnq_kv &kv, Use use, Use acc, Use pos, Spans &sp)
{
    const int es = item(d.io_dtype);
    size_t n = bytes((size_t)(kv.n_pages - 1), (size_t)kv.ldp, es);
    n += bytes((size_t)(d.hk - 1), (size_t)kv.ldh, es) + bytes((size_t)(d.page - 1), (size_t)kv.ldr, es) +
         (size_t)d.d * es;
    Spans others = sp;
    TRY(flat(sp, kv.k, n, "kv.k", use));
    if (use == WRITE && kv.v && gdnq::overlap(Span{kv.k, n, ""}, Span{kv.v, n, ""}) && rows_apart(d, kv)) {
        TRY(flat(others, kv.v, n, "kv.v", use));
        sp.s[sp.n] = others.s[others.n - 1];
        sp.out[sp.n++] = true;
    } else
        TRY(flat(sp, kv.v, n, "kv.v", use));
    const size_t m = bytes(kv.n_pages, d.hk, d.page, 4);
    TRY(flat(sp, kv.acc, m, "kv.acc", acc, true));
    TRY(flat(sp, kv.pos, m, "kv.pos", pos, true));
    TRY(flat(sp, kv.table, bytes(kv.n_slots, kv.max_pages, 4), "kv.table"));
    return flat(sp, kv.lens, (size_t)kv.n_slots * 4, "kv.lens");
}

int check_slots(const gdnq_kv &kv, const int32_t *slots, int32_t n, Spans &sp)
{
    if (!slots && kv.n_slots < n) return fail(GDNQ_EINVAL, "slots is NULL with %d slots for %d entries", kv.n_slots, n);
    return flat(sp, slots, (size_t)n * 4, "slots", READ, true);
}

int check_entries(int32_t n)
{
    if (n < 0) return fail(GDNQ_EINVAL, "n must be >= 0 (got %d)", n);
    return GDNQ_OK;
}

int check_budget(int32_t budget)
{
    if (budget < 1) return fail(GDNQ_EINVAL, "budget must be >= 1 (got %d)", budget);
    return GDNQ_OK;
}

// Sizes that the workspaces are counted with.
int check_step_sizes(const gdnq_attn_desc &d, const gdnq_kv &kv, int32_t n)
{
    TRY(check_grid((unsigned long long)n * d.H, "n*H"));
    if (kv.acc && bytes(kv.n_pages, d.page, d.H, 4) >= HUGE_SPAN)
        return fail(GDNQ_EINVAL, "the scores of H heads over the pool's rows are larger than any memory");
    return GDNQ_OK;
}

int check_evict_sizes(const gdnq_attn_desc &d, int32_t n)
{
    return check_grid((unsigned long long)n * d.hk * 16, "n*hk");
}

int check_workspace(void *p, size_t got, size_t need, Spans &sp)
{
    if (got < need) return fail(GDNQ_EINVAL, "workspace of %zu bytes is too small (%zu are needed)", got, need);
    if (need) TRY(flat(sp, p, need, "workspace", WRITE));
    return GDNQ_OK;
}

// Whether n rows of two operands, ld elements apart in both, are columns of the same rows that
// share no element (the parts of a fused projection's output).
bool apart(const void *a, long long na, const void *b, long long nb, int64_t ld, int es)
{
    const uint64_t row = (uint64_t)ld * es, x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const uint64_t d = y >= x ? (y - x) % row : (row - (x - y) % row) % row;   // from a to the next b
    return d >= (uint64_t)na * es && d + (uint64_t)nb * es <= row;
}

// x turned into y, or in place
int check_turned(Spans &sp, const void *x, int64_t &ldx, void *y, int64_t &ldy, long long n, long long len, int es,
                 const char *xn, const char *yn)
{
    if (x == y && x) {
        if ((ldx ? ldx : len) != (ldy ? ldy : len))
            return fail(GDNQ_EINVAL, "%s is %s but its rows are another distance apart", yn, xn);
        TRY(rows(sp, y, n, len, ldy, es, yn, WRITE));
        ldx = ldy;
        return GDNQ_OK;
    }
    TRY(rows(sp, x, n, len, ldx, es, xn));
    return rows(sp, y, n, len, ldy, es, yn, WRITE);
}

}  // namespace

extern "C" {

int gdnq_rope_table(const gdnq_rope_desc *desc, const gdnq_rope_freqs *freqs, uint64_t *table)
{
    gdnq_rope_desc d;
    TRY(check_rope(desc, d));
    TRY(check_freqs(freqs, d.rot));
    if (!table) return fail(GDNQ_EINVAL, "table is NULL");
    // in the host's 64-bit mantissas: the table's units are 2^-64 turns
    typedef long double real;
    const real two_pi = 6.283185307179586476925286766559005768L;
    const int rot = d.rot;
    real base = freqs->base;
    if (freqs->kind == GDNQ_ROPE_BASE && rot > 2) base *= powl(freqs->factor, (real)rot / (rot - 2));
    real i0 = 0, i1 = 0;
    if (freqs->kind == GDNQ_ROPE_RAMP_INDEX) {
        i0 = floorl((real)rot / 2 * logl(freqs->orig_len / (two_pi * freqs->hi)) / logl(base));
        i1 = ceill((real)rot / 2 * logl(freqs->orig_len / (two_pi * freqs->lo)) / logl(base));
        i0 = i0 < 0 ? 0 : i0;
        i1 = i1 > rot - 1 ? rot - 1 : i1;
        if (i0 == i1) i1 += 0.001L;
    }
    for (int i = 0; i < rot / 2; i++) {
        real t = powl(base, (real)(-2 * i) / rot), g = 1;
        if (freqs->kind == GDNQ_ROPE_LINEAR) g = 0;
        if (freqs->kind == GDNQ_ROPE_RAMP_TURNS)
            g = (freqs->orig_len * t / two_pi - freqs->lo) / ((real)freqs->hi - freqs->lo);
        if (freqs->kind == GDNQ_ROPE_RAMP_INDEX) g = 1 - (i - i0) / (i1 - i0);
        g = g < 0 ? 0 : g > 1 ? 1 : g;
        if (g < 1) t = g * t + (1 - g) * t / freqs->factor;
        if (freqs->divisors) t /= freqs->divisors[i];
        real turns = t / two_pi;
        turns -= floorl(turns);
        const real units = roundl(ldexpl(turns, 64));
        table[i] = units >= 0x1p64L ? 0 : (uint64_t)units;
    }
    return ok();
}

int gdnq_rope(const gdnq_rope_desc *desc, const uint64_t *table, const void *x, int64_t ldx, int32_t H,
              const int32_t *pos, void *y, int64_t ldy, int32_t n_rows, void *stream)
{
    gdnq_rope_desc d;
    TRY(check_rope(desc, d));
    if (H < 1) return fail(GDNQ_EINVAL, "H must be >= 1 (got %d)", H);
    TRY(check_rows(n_rows));
    if (n_rows == 0) return ok();
    Spans sp;
    TRY(flat(sp, table, (size_t)d.rot / 2 * 8, "table"));
    TRY(flat(sp, pos, (size_t)n_rows * 4, "pos"));
    TRY(check_turned(sp, x, ldx, y, ldy, n_rows, (long long)H * d.d, item(d.io_dtype), "x", "y"));
    TRY(check_grid((unsigned long long)n_rows * H, "rows*H"));
    const gdnq::RopeCall c{x, y, table, pos, ldx, ldy, H, n_rows};
    return launched(gdnq::launch_rope(d, c, stream_of(stream)));
}

int gdnq_kv_append(const gdnq_attn_desc *desc, const gdnq_rope_desc *rope, const uint64_t *table, const gdnq_kv *cache,
                   const void *q, int64_t ldq, void *q_out, int64_t ldqo, const void *k, int64_t ldk, const void *v,
                   int64_t ldv, const int32_t *pos, const int32_t *slots, const int32_t *cu_seqlens, int32_t n,
                   int32_t T, void *stream)
{
    gdnq_attn_desc d;
    gdnq_rope_desc r;
    gdnq_kv kv;
    TRY(check_attn(desc, d));
    if (rope) {
        TRY(check_rope(rope, r));
        if (r.d != d.d || r.io_dtype != d.io_dtype)
            return fail(GDNQ_EINVAL, "rope is for heads of another size or type (d=%d, io_dtype=%d) than desc's", r.d,
                        r.io_dtype);
    }
    TRY(check_sizes(d, cache, kv));
    TRY(check_counts(n, T));
    if (!cu_seqlens && n != T) return fail(GDNQ_EINVAL, "cu_seqlens is NULL with %d tokens for %d entries", T, n);
    if (n == 0 || T == 0) return ok();
    const int es = item(d.io_dtype);
    Spans sp;
    if (rope) TRY(flat(sp, table, (size_t)r.rot / 2 * 8, "table"));
    TRY(check_slots(kv, slots, n, sp));
    TRY(flat(sp, cu_seqlens, ((size_t)n + 1) * 4, "cu_seqlens", READ, true));
    TRY(flat(sp, pos, (size_t)T * 4, "pos", READ, true));
    TRY(check_cache(d, kv, WRITE, WRITE, WRITE, sp));
    const long long nq = (long long)d.H * d.d, nk = (long long)d.hk * d.d;
    Spans queries = sp;
    TRY(rows(sp, k, T, nk, ldk, es, "k"));
    TRY(rows(sp, v, T, nk, ldv, es, "v"));
    if (!q != !q_out) return fail(GDNQ_EINVAL, "q and q_out must both be there, or neither");
    if (q) {
        TRY(check_turned(queries, q, ldq, q_out, ldqo, T, nq, es, "q", "q_out"));
        // k and v may be other columns of the same rows
        if (ldk != ldqo || !apart(q_out, nq, k, nk, ldk, es)) TRY(rows(queries, k, T, nk, ldk, es, "k"));
        if (ldv != ldqo || !apart(q_out, nq, v, nk, ldv, es)) TRY(rows(queries, v, T, nk, ldv, es, "v"));
    }
    TRY(check_grid(((unsigned long long)T + n) * 4, "T"));
    const gdnq::AppendCall c{kv, q, k, v, q_out, table, pos, slots, cu_seqlens, ldq, ldqo, ldk, ldv, n, T};
    if (!gdnq::kv_append_numbers(d, rope ? &r : nullptr, c))
        return fail(GDNQ_EINVAL, "too many heads for one row (H=%d, hk=%d)", d.H, d.hk);
    return launched(gdnq::launch_kv_append(d, rope ? &r : nullptr, c, stream_of(stream)));
}

int gdnq_attn_workspace(const gdnq_attn_desc *desc, const gdnq_kv *cache, int32_t n, size_t *bytes_out)
{
    gdnq_attn_desc d;
    gdnq_kv kv;
    TRY(check_attn(desc, d));
    TRY(check_sizes(d, cache, kv));
    TRY(check_entries(n));
    if (!bytes_out) return fail(GDNQ_EINVAL, "bytes_out is NULL");
    TRY(check_step_sizes(d, kv, n));
    *bytes_out = n == 0 ? 0 : gdnq::attn_workspace(d, kv, n);
    return ok();
}

int gdnq_attn_step(const gdnq_attn_desc *desc, const gdnq_kv *cache, const void *q, int64_t ldq, void *o, int64_t ldo,
                   const int32_t *slots, int32_t n, void *workspace, size_t workspace_bytes, void *stream)
{
    gdnq_attn_desc d;
    gdnq_kv kv;
    TRY(check_attn(desc, d));
    TRY(check_sizes(d, cache, kv));
    TRY(check_entries(n));
    if (n == 0) return ok();
    const int es = item(d.io_dtype);
    Spans sp;
    TRY(check_slots(kv, slots, n, sp));
    TRY(check_cache(d, kv, READ, WRITE, READ, sp));
    TRY(rows(sp, q, n, (long long)d.H * d.d, ldq, es, "q"));
    TRY(rows(sp, o, n, (long long)d.H * d.d, ldo, es, "o", WRITE));
    TRY(check_step_sizes(d, kv, n));
    TRY(check_workspace(workspace, workspace_bytes, gdnq::attn_workspace(d, kv, n), sp));
    const gdnq::AttnCall c{kv, q, o, slots, ldq, ldo, n, workspace};
    return launched(gdnq::launch_attn_step(d, c, stream_of(stream)));
}

int gdnq_kv_evict_workspace(const gdnq_attn_desc *desc, const gdnq_kv *cache, int32_t budget, int32_t n,
                            size_t *bytes_out)
{
    gdnq_attn_desc d;
    gdnq_kv kv;
    TRY(check_attn(desc, d));
    TRY(check_sizes(d, cache, kv));
    TRY(check_budget(budget));
    TRY(check_entries(n));
    if (!bytes_out) return fail(GDNQ_EINVAL, "bytes_out is NULL");
    TRY(check_evict_sizes(d, n));
    *bytes_out = n == 0 ? 0 : gdnq::kv_evict_workspace(d, kv, budget, n);
    return ok();
}

int gdnq_kv_evict(const gdnq_attn_desc *desc, const gdnq_kv *cache, int32_t budget, int32_t sink, int32_t recent,
                  const int32_t *slots, int32_t n, void *workspace, size_t workspace_bytes, void *stream)
{
    gdnq_attn_desc d;
    gdnq_kv kv;
    TRY(check_attn(desc, d));
    TRY(check_sizes(d, cache, kv));
    TRY(check_budget(budget));
    if (sink < 0 || recent < 0 || (long long)sink + recent > budget)
        return fail(GDNQ_EINVAL, "sink and recent must be >= 0 and at most budget together (got %d, %d, %d)", sink,
                    recent, budget);
    TRY(check_entries(n));
    if (n == 0) return ok();
    if (!kv.acc || !kv.pos) return fail(GDNQ_EINVAL, "%s is NULL", kv.acc ? "kv.pos" : "kv.acc");
    Spans sp;
    TRY(check_slots(kv, slots, n, sp));
    TRY(check_cache(d, kv, WRITE, WRITE, WRITE, sp));
    TRY(check_evict_sizes(d, n));
    TRY(check_workspace(workspace, workspace_bytes, gdnq::kv_evict_workspace(d, kv, budget, n), sp));
    const gdnq::EvictCall c{kv, slots, budget, sink, recent, n, workspace};
    return launched(gdnq::launch_kv_evict(d, c, stream_of(stream)));
}

}  // extern "C"
