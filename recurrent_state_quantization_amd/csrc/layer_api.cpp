// layer_api.cpp -- the C ABI of include/gdnq_layer.h: argument checks on the
// host, then the launches of the call on the caller's stream.  Nothing is
// allocated and nothing is synchronized.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "checks.hpp"
#include "gdnq_layer.h"
#include "layer_launchers.hpp"

namespace {

using namespace gdnq::checks;
using gdnq::fail;
using gdnq::launched;
using gdnq::ok;
using gdnq::Span;

int check_pool(int32_t n_slots, const int32_t *slots, int32_t n, Spans &sp)
{
    if (n_slots < 1) return fail(GDNQ_EINVAL, "n_slots must be >= 1 (got %d)", n_slots);
    if (!slots && n_slots < n) return fail(GDNQ_EINVAL, "slots is NULL with %d slots for %d entries", n_slots, n);
    return flat(sp, slots, (size_t)n * 4, "slots", READ, true);
}

int check_packed(const int32_t *cont, const int32_t *cu, int32_t n, Spans &sp)
{
    TRY(flat(sp, cont, (size_t)n * 4, "cont", READ, true));
    return flat(sp, cu, ((size_t)n + 1) * 4, "cu_seqlens");
}

// ------------------------------------------------------------ convolution
int check_conv(const gdnq_conv_desc *d)
{
    if (!d) return fail(GDNQ_EINVAL, "desc is NULL");
    if (d->C < 1) return fail(GDNQ_EINVAL, "C must be >= 1 (got %d)", d->C);
    if (d->width < 2 || d->width > 4) return fail(GDNQ_EUNSUPPORTED, "width must be 2, 3 or 4 (got %d)", d->width);
    TRY(check_io_dtype(d->io_dtype));
    if (d->flags & ~GDNQ_CONV_SILU) return fail(GDNQ_EINVAL, "unknown flag bits 0x%x", d->flags);
    return GDNQ_OK;
}

int check_conv_call(const gdnq_conv_desc &d, gdnq::ConvCall &c, long long n_rows, Spans &sp)
{
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4;
    int64_t ldx = c.ldx, ldy = c.ldy;
    TRY(rows(sp, c.x, n_rows, d.C, ldx, es, "x"));
    TRY(flat(sp, c.w, (size_t)d.width * d.C * 4, "w"));
    TRY(flat(sp, c.bias, (size_t)d.C * 4, "bias", READ, true));
    TRY(check_pool(c.n_slots, c.slots, c.n, sp));
    TRY(flat(sp, c.state, bytes(c.n_slots, d.width - 1, d.C, es), "state", WRITE));
    TRY(rows(sp, c.y, n_rows, d.C, ldy, es, "y", WRITE));
    c.ldx = ldx;
    c.ldy = ldy;
    return GDNQ_OK;
}

// ------------------------------------------------------------------- scan
int check_ssm(const gdnq_ssm_desc *d)
{
    if (!d) return fail(GDNQ_EINVAL, "desc is NULL");
    if (d->H < 1) return fail(GDNQ_EINVAL, "H must be >= 1 (got %d)", d->H);
    if ((d->dk != 64 && d->dk != 128) || (d->dv != 64 && d->dv != 128))
        return fail(GDNQ_EUNSUPPORTED, "dk and dv must each be 64 or 128 (got dk=%d dv=%d)", d->dk, d->dv);
    if (d->hk < 0 || (d->hk > 0 && d->H % d->hk != 0))
        return fail(GDNQ_EINVAL, "hk must divide H (0 means H; got hk=%d, H=%d)", d->hk, d->H);
    TRY(check_io_dtype(d->io_dtype));
    if (d->flags & ~GDNQ_SSM_SOFTPLUS) return fail(GDNQ_EINVAL, "unknown flag bits 0x%x", d->flags);
    if (!(d->dt_min >= 0.0f) || !(d->dt_max >= d->dt_min))
        return fail(GDNQ_EINVAL, "0 <= dt_min <= dt_max is needed (got %g, %g)", (double)d->dt_min, (double)d->dt_max);
    return GDNQ_OK;
}

int check_ssm_call(const gdnq_ssm_desc &d, gdnq::SsmCall &c, long long n_rows, Spans &sp)
{
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4;
    const long long hk = d.hk ? d.hk : d.H;
    gdnq_ssm_io &io = c.io;
    TRY(rows(sp, io.x, n_rows, (long long)d.H * d.dv, io.ldx, es, "x"));
    TRY(rows(sp, io.B, n_rows, hk * d.dk, io.ldb, es, "B"));
    TRY(rows(sp, io.C, n_rows, hk * d.dk, io.ldc, es, "C"));
    TRY(rows(sp, io.dt, n_rows, d.H, io.lddt, es, "dt"));
    TRY(flat(sp, io.A, (size_t)d.H * 4, "A"));
    TRY(flat(sp, io.D, (size_t)d.H * 4, "D", READ, true));
    TRY(flat(sp, io.dt_bias, (size_t)d.H * 4, "dt_bias", READ, true));
    TRY(check_pool(c.n_slots, c.slots, c.n, sp));
    TRY(flat(sp, c.S, bytes(c.n_slots, d.H, (size_t)d.dk * d.dv, 4), "S", WRITE));
    return rows(sp, io.y, n_rows, (long long)d.H * d.dv, io.ldy, es, "y", WRITE);
}

// ------------------------------------------------------------------ norms
int check_norm(const gdnq_norm_desc *d, uint32_t flags)
{
    if (!d) return fail(GDNQ_EINVAL, "desc is NULL");
    if (d->D < 1) return fail(GDNQ_EINVAL, "D must be >= 1 (got %d)", d->D);
    if (d->D > 32768) return fail(GDNQ_EUNSUPPORTED, "D must be at most 32768 (got %d)", d->D);
    if (d->group < 0 || (d->group > 0 && d->D % d->group != 0))
        return fail(GDNQ_EINVAL, "group must divide D (0 means D; got group=%d, D=%d)", d->group, d->D);
    TRY(check_io_dtype(d->io_dtype));
    if (d->flags & ~flags) return fail(GDNQ_EINVAL, "flag bits 0x%x are unknown here", d->flags & ~flags);
    if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return fail(GDNQ_EINVAL, "eps must be > 0 (got %g)", (double)d->eps);
    if (!std::isfinite(d->w_offset)) return fail(GDNQ_EINVAL, "w_offset must be finite");
    return GDNQ_OK;
}

}  // namespace

extern "C" {

int gdnq_conv_prefill(const gdnq_conv_desc *desc, const void *x, int64_t ldx, const float *w, const float *bias,
                      void *state, int32_t n_slots, const int32_t *slots, const int32_t *cont,
                      const int32_t *cu_seqlens, int32_t n_seqs, int32_t T, void *y, int64_t ldy, void *stream)
{
    TRY(check_conv(desc));
    TRY(check_counts(n_seqs, T));
    if (n_seqs == 0 || T == 0) return ok();
    gdnq::ConvCall c{x, w, bias, state, y, slots, cont, cu_seqlens, ldx, ldy, n_slots, n_seqs, T};
    Spans sp;
    TRY(check_packed(cont, cu_seqlens, n_seqs, sp));
    TRY(check_conv_call(*desc, c, T, sp));
    TRY(check_grid(((unsigned long long)T / 16 + n_seqs) * (((unsigned long long)desc->C + 63) / 64), "T*C"));
    return launched(gdnq::launch_conv_prefill(*desc, c, stream_of(stream)));
}

int gdnq_conv_step(const gdnq_conv_desc *desc, const void *x, int64_t ldx, const float *w, const float *bias,
                   void *state, int32_t n_slots, const int32_t *slots, int32_t n, void *y, int64_t ldy, void *stream)
{
    TRY(check_conv(desc));
    TRY(check_rows(n));
    if (n == 0) return ok();
    gdnq::ConvCall c{x, w, bias, state, y, slots, nullptr, nullptr, ldx, ldy, n_slots, n, n};
    Spans sp;
    TRY(check_conv_call(*desc, c, n, sp));
    TRY(check_grid((unsigned long long)n * (((unsigned long long)desc->C + 63) / 64), "n*C"));
    return launched(gdnq::launch_conv_step(*desc, c, stream_of(stream)));
}

int gdnq_ssm_workspace(const gdnq_ssm_desc *desc, int32_t n_seqs, int32_t T, size_t *bytes_out)
{
    TRY(check_ssm(desc));
    TRY(check_counts(n_seqs, T));
    if (!bytes_out) return fail(GDNQ_EINVAL, "bytes_out is NULL");
    *bytes_out = n_seqs == 0 || T == 0 ? 0 : gdnq::ssm_workspace(*desc, n_seqs, T);
    return ok();
}

int gdnq_ssm_prefill(const gdnq_ssm_desc *desc, const gdnq_ssm_io *io, float *S, int32_t n_slots, const int32_t *slots,
                     const int32_t *cont, const int32_t *cu_seqlens, int32_t n_seqs, int32_t T, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    TRY(check_ssm(desc));
    if (desc->io_dtype != GDNQ_IO_BF16) return fail(GDNQ_EUNSUPPORTED, "gdnq_ssm_prefill takes bf16 rows");
    TRY(check_counts(n_seqs, T));
    if (n_seqs == 0 || T == 0) return ok();
    if (!io) return fail(GDNQ_EINVAL, "io is NULL");
    gdnq::SsmCall c{*io, S, slots, cont, cu_seqlens, n_slots, n_seqs, T, workspace};
    Spans sp;
    TRY(check_packed(cont, cu_seqlens, n_seqs, sp));
    TRY(check_ssm_call(*desc, c, T, sp));
    const int64_t far = 1 << 22;   // a chunk's rows are addressed by 32-bit offsets
    if (c.io.ldx > far || c.io.ldb > far || c.io.ldc > far || c.io.ldy > far || c.io.lddt > far)
        return fail(GDNQ_EUNSUPPORTED, "gdnq_ssm_prefill takes rows at most 2^22 elements apart");
    const size_t need = gdnq::ssm_workspace(*desc, n_seqs, T);
    if (workspace_bytes < need)
        return fail(GDNQ_EINVAL, "workspace of %zu bytes is too small (%zu are needed)", workspace_bytes, need);
    if (need) TRY(flat(sp, workspace, need, "workspace", WRITE));
    TRY(check_grid(((unsigned long long)T / 128 + n_seqs + 8) * desc->H * 16, "T*H"));
    if (T <= gdnq::SSM_WHOLE)   // 2 dv threads for every sequence and head, in one dimension of a grid
        TRY(check_grid((unsigned long long)n_seqs * desc->H * desc->dv, "n_seqs*H"));
    return launched(gdnq::launch_ssm_prefill(*desc, c, stream_of(stream)));
}

int gdnq_ssm_step(const gdnq_ssm_desc *desc, const gdnq_ssm_io *io, float *S, int32_t n_slots, const int32_t *slots,
                  int32_t n, void *stream)
{
    TRY(check_ssm(desc));
    TRY(check_rows(n));
    if (n == 0) return ok();
    if (!io) return fail(GDNQ_EINVAL, "io is NULL");
    gdnq::SsmCall c{*io, S, slots, nullptr, nullptr, n_slots, n, n, nullptr};
    Spans sp;
    TRY(check_ssm_call(*desc, c, n, sp));
    TRY(check_grid((unsigned long long)n * desc->H, "n*H"));
    return launched(gdnq::launch_ssm_step(*desc, c, stream_of(stream)));
}

int gdnq_norm_gated(const gdnq_norm_desc *desc, const void *x, int64_t ldx, const void *z, int64_t ldz, const float *w,
                    void *y, int64_t ldy, int32_t n_rows, void *stream)
{
    TRY(check_norm(desc, GDNQ_NORM_GATE_SIGMOID | GDNQ_NORM_GATE_FIRST | GDNQ_NORM_GROUP_WEIGHT));
    TRY(check_rows(n_rows));
    if (n_rows == 0) return ok();
    const gdnq_norm_desc &d = *desc;
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4, group = d.group ? d.group : d.D;
    Spans sp;
    TRY(rows(sp, x, n_rows, d.D, ldx, es, "x"));
    TRY(rows(sp, z, n_rows, d.D, ldz, es, "z", READ, true));
    TRY(flat(sp, w, ((d.flags & GDNQ_NORM_GROUP_WEIGHT) ? group : d.D) * (size_t)4, "w"));
    TRY(rows(sp, y, n_rows, d.D, ldy, es, "y", WRITE));
    TRY(check_grid((unsigned long long)n_rows * (d.D / group), "rows*groups"));
    const gdnq::NormCall c{x, z, nullptr, y, nullptr, w, nullptr, ldx, ldz, 0, 0, ldy, 1.0f, n_rows};
    return launched(gdnq::launch_norm_gated(d, c, stream_of(stream)));
}

int gdnq_norm_residual(const gdnq_norm_desc *desc, const void *x, int64_t ldx, const float *post_w, float scale,
                       const void *res, int64_t ldr, void *res_out, int64_t ldro, const float *w, void *y, int64_t ldy,
                       int32_t n_rows, void *stream)
{
    TRY(check_norm(desc, GDNQ_NORM_RES_F32));
    TRY(check_rows(n_rows));
    const gdnq_norm_desc &d = *desc;
    if (d.group != 0 && d.group != d.D)
        return fail(GDNQ_EUNSUPPORTED, "gdnq_norm_residual norms whole rows (got group=%d, D=%d)", d.group, d.D);
    if (!std::isfinite(scale)) return fail(GDNQ_EINVAL, "scale must be finite");
    if (n_rows == 0) return ok();
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4, rs = (d.flags & GDNQ_NORM_RES_F32) ? 4 : es;
    Spans sp;
    TRY(rows(sp, x, n_rows, d.D, ldx, es, "x"));
    TRY(flat(sp, post_w, (size_t)d.D * 4, "post_w", READ, true));
    TRY(flat(sp, w, (size_t)d.D * 4, "w", READ, !y));
    if (res_out == res && res) {   // in place: one buffer, one distance
        if ((ldr ? ldr : d.D) != (ldro ? ldro : d.D))
            return fail(GDNQ_EINVAL, "res_out is res but its rows are another distance apart");
        TRY(rows(sp, res_out, n_rows, d.D, ldro, rs, "res_out", WRITE));
        ldr = ldro;
    } else {
        TRY(rows(sp, res, n_rows, d.D, ldr, rs, "res"));
        TRY(rows(sp, res_out, n_rows, d.D, ldro, rs, "res_out", WRITE));
    }
    TRY(rows(sp, y, n_rows, d.D, ldy, es, "y", WRITE, true));
    TRY(check_grid((unsigned long long)n_rows, "rows"));
    const gdnq::NormCall c{x, nullptr, res, y, res_out, w, post_w, ldx, 0, ldr, ldro, ldy, scale, n_rows};
    return launched(gdnq::launch_norm_residual(d, c, stream_of(stream)));
}

}  // extern "C"
