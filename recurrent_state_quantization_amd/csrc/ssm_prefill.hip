// ssm_prefill.hip -- the selective state space scan over packed prompts on
// the matrix cores (gdnq_ssm_prefill): per head, with
// delta = clamp(softplus(dt + bias)),
//   S <- e^{delta A} S + B (delta x)^T,   y = S^T C + D x.
// LinQuant, appendix Table 3, Mamba-2 row, in the dk x dv orientation.
//
// The recurrence unrolled over a chunk of 64 tokens, with cs_i the running
// sum of delta A inside the chunk and S the state at its start:
//   M_ij = (C_i . B_j) e^{cs_i - cs_j} delta_j   (j <= i, else 0)
//   Y    = M X + diag(e^{cs}) C S + D X
//   S   <- e^{cs_63} S + B^T diag(e^{cs_63 - cs} delta) X.
// Exponents are kept in base 2 and are never positive, so nothing overflows;
// e^{cs_63 - cs_j} comes from a sum over the tokens behind j, which keeps it
// exact where it is near one.
//
// Precision: the products run on v_mfma_f32_32x32x16_bf16 with fp32 sums.
// B, C and x are bf16, so C B^T is exact up to the sum; the fp32 operands M
// and S of the outputs are split into two bf16 parts (off by 2^-18), the
// weighted x of the state's update into three (2^-26), so that states stay
// as exact as fp32.
//
// A wave owns 32 value columns of one head for the whole segment: its state
// (dk x 32) stays in accumulators, which feed C S directly as the B operand
// when the contraction index is taken in the accumulators' row order (slots
// 0..3 of lane half h are rows 16t + 4h .. + 3, slots 4..7 rows 16t + 8 + 4h
// .. + 3).  The transposed product B C^T likewise leaves M in the layout of
// an A operand.  x and B are read by columns with the transposing LDS read.
// A workgroup holds up to 8 waves: HPW heads that share B and C.
//
// Long sequences are cut into segments of 2^SH tokens (launch_ssm_prefill
// says when): a first kernel forms each segment's own state and decay from
// zero, a second runs along the segments of each sequence and leaves the
// state at every segment's start, and the main kernel starts from those.
#include "layer_launchers.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int CH = 64;   // tokens per chunk

struct SsmArgs {
    SsmCall c;
    int H, hk;
    int sh;              // log2 of a segment's tokens
    unsigned ids;        // segment numbers
    float dt_min, dt_max;
    bool sp, wide;
    Divisor byHB;        // head blocks per segment
    float *ws;           // [ids][H][dk*dv] states, then [ids][H] base-2 decay exponents
};

__device__ __forceinline__ floatx16 mma(bf16x8 a, bf16x8 b, floatx16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// Inclusive prefix sum over the 64 lanes of a wave: shifts within rows of 16
// lanes, then the last lane of rows 0 and 2 into rows 1 and 3, then lane 31
// into rows 2 and 3.
__device__ __forceinline__ float scan64(float x)
{
#define GDNQ_DPP(x, ctrl, rmask) \
    __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, rmask, 0xf, true))
    x += GDNQ_DPP(x, 0x111, 0xf);
    x += GDNQ_DPP(x, 0x112, 0xf);
    x += GDNQ_DPP(x, 0x114, 0xf);
    x += GDNQ_DPP(x, 0x118, 0xf);
    x += GDNQ_DPP(x, 0x142, 0xa);
    x += GDNQ_DPP(x, 0x143, 0xc);
#undef GDNQ_DPP
    return x;
}

__device__ __forceinline__ float lane_of(float x, int lane)
{
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// h + l = x up to 2^-18 of x
__device__ __forceinline__ void split2(const float (&x)[8], bf16x8 &h, bf16x8 &l)
{
#pragma unroll
    for (int e = 0; e < 8; e++) {
        h[e] = (__bf16)x[e];
        l[e] = (__bf16)(x[e] - (float)h[e]);
    }
}

// h + m + l = x up to 2^-26 of x
__device__ __forceinline__ void split3(const float (&x)[8], bf16x8 &h, bf16x8 &m, bf16x8 &l)
{
#pragma unroll
    for (int e = 0; e < 8; e++) {
        h[e] = (__bf16)x[e];
        const float r = x[e] - (float)h[e];
        m[e] = (__bf16)r;
        l[e] = (__bf16)(r - (float)m[e]);
    }
}

// Columns of a row-major LDS tile as an operand: lane (c, h) gets column c of
// rows 4h .. 4h + 3 and 8 + 4h .. + 3 behind p.  p is the lane's own address:
// row 4h + (lane % 16) / 4, column 16 (c / 16) + 4 (lane % 4).
__device__ __forceinline__ bf16x8 ld_cols(const __bf16 *p, int stride)
{
    using lds_p = __attribute__((address_space(3))) shortx4 *;
    const shortx4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(p));
    const shortx4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(p + 8 * stride));
    typedef short shortx8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// 4 values at p, then 4 at p + 8: a row as an operand in the accumulators' order
__device__ __forceinline__ bf16x8 ld_rows(const __bf16 *p)
{
    const bf16x4 a = *reinterpret_cast<const bf16x4 *>(p);
    const bf16x4 b = *reinterpret_cast<const bf16x4 *>(p + 8);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 8 consecutive bf16 values of a token row
__device__ __forceinline__ u32x4 ld_global8(const void *base, size_t off, bool wide)
{
    const uint16_t *p = reinterpret_cast<const uint16_t *>(base) + off;
    if (wide) return *reinterpret_cast<const u32x4 *>(p);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return r;
}

// Row strides in elements.  B is read by rows (C B^T) and by columns (the
// state's update): a stride of 20 banks more than a multiple of 64 keeps the
// row reads at two lanes per bank and the column reads below that.  C is
// read by rows in 16-byte pieces (4 banks more), x by columns only (16 more).
template <int DK, int DV, int HPW>
struct SsmGeom {
    static constexpr int SL = DV / 32;           // waves per head
    static constexpr int NW = HPW * SL;
    static constexpr int NT = NW * 64;
    static constexpr int SB = DK + 40, SC = DK + 8, SX = HPW * DV + (HPW * DV == 64 ? 40 : 32);
    static constexpr int NB = CH * DK / 8 / NT;         // 16-byte pieces of B (and of C) per thread
    static constexpr int NX = CH * HPW * DV / 8 / NT;   // and of x
    static constexpr int NBLK = DK / 32;
};

enum { V_CS, V_E, V_W, V_D, V_VE, V_N };   // per-token vectors in LDS

template <class G>
struct SsmLds {
    __bf16 b[CH * G::SB];
    __bf16 c[CH * G::SC];
    __bf16 x[CH * G::SX];
    alignas(16) float v[G::NW / G::SL][V_N][CH];
    float tot[G::NW / G::SL];
};

// STATE: only the segment's own state and decay, from zero.
template <int DK, int DV, int HPW, bool STATE>
__global__ __launch_bounds__((SsmGeom<DK, DV, HPW>::NT)) void ssm_chunk_kernel(SsmArgs A)
{
    using G = SsmGeom<DK, DV, HPW>;
    __shared__ SsmLds<G> L;
    const int t = (int)__builtin_amdgcn_workitem_id_x(), lane = t & 63;
    const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
    const int hw = wv / G::SL, slice = wv % G::SL;
    const unsigned g = __builtin_amdgcn_workgroup_id_x();
    const unsigned id = __builtin_amdgcn_readfirstlane(div_by(g, A.byHB));
    const int h0 = (int)(g - id * A.byHB.d) * HPW, head = h0 + hw;
    const int hb = h0 / (A.H / A.hk);
    const gdnq_ssm_io &io = A.c.io;
    SeqTile q;
    if (!seq_tile(A.c.cu, A.c.slots, A.c.n, (int)id, A.sh, A.c.T, A.c.n_slots, q)) return;
    const bool multi = q.len > (1 << A.sh), last = ((long long)(q.k + 1) << A.sh) >= q.len;
    if (STATE && last) return;
    const size_t row0 = (size_t)q.start + ((size_t)q.k << A.sh);
    const int ntok = min(1 << A.sh, q.len - (q.k << A.sh));

    const int c = lane & 31, hh = lane >> 5;
    // the wave's state: accumulator r of block nb is row 32 nb + 8 (r/4) + 4 hh + r % 4, column 32 slice + c
    floatx16 S[G::NBLK];
    const size_t soff = (size_t)(4 * hh) * DV + slice * 32 + c;
    float *const pool = A.c.S + ((size_t)q.slot * A.H + head) * DK * DV + soff;
    float *const seg = A.ws + ((size_t)id * A.H + head) * DK * DV + soff;   // touched only if multi
    {
        const float *from = multi ? seg : pool;
        const bool load = !STATE && (multi || (A.c.cont && A.c.cont[q.seq]));
#pragma unroll
        for (int nb = 0; nb < G::NBLK; nb++)
#pragma unroll
            for (int r = 0; r < 16; r++) S[nb][r] = load ? from[(size_t)(32 * nb + 8 * (r / 4) + r % 4) * DV] : 0.0f;
    }
    const float Ah = io.A[head] * 1.44269504f, bias = io.dt_bias ? io.dt_bias[head] : 0.0f;
    const float Dh = io.D ? io.D[head] : 0.0f;
    float seglog = 0.0f;

    for (int c0 = 0; c0 < ntok; c0 += CH) {
        const int nv = min(CH, ntok - c0);
        const size_t row = row0 + c0;
        __syncthreads();   // the previous chunk's reads are done
        // ---- stage the chunk; rows behind the end repeat the last one (their weights are zero)
#pragma unroll
        for (int i = 0; i < G::NB; i++) {
            const int p = t + i * G::NT, r = p / (DK / 8), k8 = p % (DK / 8);
            const size_t src = row + min(r, nv - 1);
            const u32x4 vb = ld_global8(io.B, src * io.ldb + (size_t)hb * DK + k8 * 8, A.wide);
            *reinterpret_cast<u32x4 *>(&L.b[r * G::SB + k8 * 8]) = vb;
            if constexpr (!STATE) {
                const u32x4 vc = ld_global8(io.C, src * io.ldc + (size_t)hb * DK + k8 * 8, A.wide);
                // columns of each 16 in the order 0-3, 8-11, 4-7, 12-15
                __bf16 *d = &L.c[r * G::SC + (k8 & ~1) * 8 + (k8 & 1) * 4];
                *reinterpret_cast<uint2 *>(d) = make_uint2(vc[0], vc[1]);
                *reinterpret_cast<uint2 *>(d + 8) = make_uint2(vc[2], vc[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < G::NX; i++) {
            constexpr int PR = HPW * DV / 8;
            const int p = t + i * G::NT, r = p / PR, k8 = p % PR;
            const u32x4 vx = ld_global8(io.x, (row + min(r, nv - 1)) * io.ldx + (size_t)h0 * DV + k8 * 8, A.wide);
            *reinterpret_cast<u32x4 *>(&L.x[r * G::SX + k8 * 8]) = vx;
        }
        // ---- decays: one wave per head, one token per lane
        if (slice == 0) {
            float d = load1<true>(io.dt, (row + min(lane, nv - 1)) * io.lddt + head) + bias;
            if (A.sp) d = softplus(d);
            d = lane < nv ? fminf(fmaxf(d, A.dt_min), A.dt_max) : 0.0f;
            const float la = d * Ah;
            const float cs = scan64(la);
            const float suf = __shfl(scan64(__shfl(la, 63 - lane)), 63 - lane) - la;   // the tokens behind this one
            const float mid = lane_of(cs, 31), tot = lane_of(cs, 63);
            const float lr = exp2f(lane < 32 ? mid - cs : cs - mid);
            L.v[hw][V_CS][lane] = cs;
            L.v[hw][V_E][lane] = exp2f(cs);
            L.v[hw][V_W][lane] = exp2f(suf) * d;
            L.v[hw][V_D][lane] = d;
            L.v[hw][V_VE][lane] = lane < 32 ? lr * d : lr;
            seglog += tot;
            if (lane == 0) L.tot[hw] = exp2f(tot);
        }
        __syncthreads();

        const int l16 = lane & 15;
        const int tr_r = 4 * hh + l16 / 4, tr_c = 16 * (c / 16) + 4 * (l16 & 3);
        const float *vec = &L.v[hw][0][0];
        bf16x8 xf[4];   // x rows 16 f .. + 15, the wave's columns
#pragma unroll
        for (int f = 0; f < 4; f++)
            xf[f] = ld_cols(&L.x[(16 * f + tr_r) * G::SX + hw * DV + slice * 32 + tr_c], G::SX);

        if constexpr (!STATE) {
            floatx16 Y[2], Gt[3];   // Gt: (j, i) blocks (0,0), (0,1), (1,1) of B C^T
#pragma unroll
            for (int r = 0; r < 16; r++) Y[0][r] = Y[1][r] = Gt[0][r] = Gt[1][r] = Gt[2][r] = 0.0f;
#pragma unroll
            for (int s = 0; s < DK / 16; s++) {
                const bf16x8 ca = *reinterpret_cast<const bf16x8 *>(&L.c[c * G::SC + 16 * s + 8 * hh]);
                const bf16x8 cb = *reinterpret_cast<const bf16x8 *>(&L.c[(32 + c) * G::SC + 16 * s + 8 * hh]);
                const bf16x8 ba = ld_rows(&L.b[c * G::SB + 16 * s + 4 * hh]);
                const bf16x8 bb = ld_rows(&L.b[(32 + c) * G::SB + 16 * s + 4 * hh]);
                float sv[8];
#pragma unroll
                for (int e = 0; e < 8; e++) sv[e] = S[s / 2][8 * (s & 1) + e];
                bf16x8 sh, sl;
                split2(sv, sh, sl);
                Gt[0] = mma(ba, ca, Gt[0]);
                Gt[1] = mma(ba, cb, Gt[1]);
                Gt[2] = mma(bb, cb, Gt[2]);
                Y[0] = mma(ca, sh, Y[0]);
                Y[1] = mma(cb, sh, Y[1]);
                Y[0] = mma(ca, sl, Y[0]);
                Y[1] = mma(cb, sl, Y[1]);
            }
#pragma unroll
            for (int ib = 0; ib < 2; ib++)
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float4 e = *reinterpret_cast<const float4 *>(&vec[V_E * CH + 32 * ib + 8 * k + 4 * hh]);
                    const float ev[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                    for (int r = 0; r < 4; r++) Y[ib][4 * k + r] *= ev[r];
                }
            // ---- Y += M X, block by block
#pragma unroll
            for (int b = 0; b < 3; b++) {
                const int jb = b == 2, ib = b > 0;
                const bool diag = b != 1;
                const float ci = vec[(diag ? V_CS : V_VE) * CH + 32 * ib + c];
#pragma unroll
                for (int tt = 0; tt < 2; tt++) {
                    float m[8];
#pragma unroll
                    for (int k = 0; k < 2; k++) {
                        const int j0 = 32 * jb + 16 * tt + 8 * k + 4 * hh;
                        const float4 dj = *reinterpret_cast<const float4 *>(&vec[(diag ? V_D : V_VE) * CH + j0]);
                        const float dv[4] = {dj.x, dj.y, dj.z, dj.w};
                        float cj[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                        if (diag) {
                            const float4 cv = *reinterpret_cast<const float4 *>(&vec[V_CS * CH + j0]);
                            cj[0] = cv.x, cj[1] = cv.y, cj[2] = cv.z, cj[3] = cv.w;
                        }
#pragma unroll
                        for (int r = 0; r < 4; r++) {
                            const float gv = Gt[b][8 * tt + 4 * k + r] * dv[r];
                            if (diag)
                                m[4 * k + r] = j0 + r <= 32 * ib + c
                                                   ? gv * __builtin_amdgcn_exp2f(ci - cj[r]) : 0.0f;
                            else
                                m[4 * k + r] = gv * ci;
                        }
                    }
                    bf16x8 mh, ml;
                    split2(m, mh, ml);
                    Y[ib] = mma(mh, xf[2 * jb + tt], Y[ib]);
                    Y[ib] = mma(ml, xf[2 * jb + tt], Y[ib]);
                }
            }
            // ---- y = Y + D x; neighbouring lanes trade halves so that each stores two columns of one row
            const uint32_t sel = (lane & 1) ? 0x03020706u : 0x05040100u;
            uint16_t *const yp = reinterpret_cast<uint16_t *>(io.y) + (size_t)head * DV + slice * 32 + (c & ~1);
#pragma unroll
            for (int ib = 0; ib < 2; ib++)
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
                    const bf16x8 &xr = xf[2 * ib + r / 8];
                    const float y0 = fmaf(Dh, (float)xr[r % 8], Y[ib][r]);
                    const float y1 = fmaf(Dh, (float)xr[r % 8 + 1], Y[ib][r + 1]);
                    const uint32_t u = __builtin_bit_cast(uint32_t, (bf16x2{(__bf16)y0, (__bf16)y1}));
                    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, DPP_XOR1, 0xF, 0xF, true);
                    const uint32_t w = __builtin_amdgcn_perm(o, u, sel);
                    const int i = 32 * ib + 8 * (r / 4) + 4 * hh + r % 4 + (lane & 1);
                    if (i < nv) {
                        uint16_t *d = yp + (row + i) * io.ldy;
                        if (A.wide) *reinterpret_cast<uint32_t *>(d) = w;
                        else d[0] = (uint16_t)w, d[1] = (uint16_t)(w >> 16);
                    }
                }
        }

        // ---- S <- e^{cs_63} S + B^T (w x)
        const float tot = L.tot[hw];
#pragma unroll
        for (int nb = 0; nb < G::NBLK; nb++)
#pragma unroll
            for (int r = 0; r < 16; r++) S[nb][r] *= tot;
#pragma unroll
        for (int f = 0; f < 4; f++) {
            float wx[8];
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float4 w = *reinterpret_cast<const float4 *>(&vec[V_W * CH + 16 * f + 8 * k + 4 * hh]);
                const float wv4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int r = 0; r < 4; r++) wx[4 * k + r] = wv4[r] * (float)xf[f][4 * k + r];
            }
            bf16x8 xh, xm, xl;
            split3(wx, xh, xm, xl);
#pragma unroll
            for (int nb = 0; nb < G::NBLK; nb++) {
                const bf16x8 bt = ld_cols(&L.b[(16 * f + tr_r) * G::SB + 32 * nb + tr_c], G::SB);
                S[nb] = mma(bt, xh, S[nb]);
                S[nb] = mma(bt, xm, S[nb]);
                S[nb] = mma(bt, xl, S[nb]);
            }
        }
    }
    if (STATE || last) {
        float *to = STATE ? seg : pool;
#pragma unroll
        for (int nb = 0; nb < G::NBLK; nb++)
#pragma unroll
            for (int r = 0; r < 16; r++) to[(size_t)(32 * nb + 8 * (r / 4) + r % 4) * DV] = S[nb][r];
    }
    if (STATE && slice == 0 && lane == 0) A.ws[(size_t)A.ids * A.H * DK * DV + (size_t)id * A.H + head] = seglog;
}

// Along each sequence of several segments: the state at every segment's
// start, in the place of the segment's own state.  One thread per 4 values.
template <int E>
__global__ __launch_bounds__(256) void ssm_join_kernel(SsmArgs A, Divisor byPart, Divisor byH)
{
    const unsigned g = __builtin_amdgcn_workgroup_id_x();
    const unsigned bh = div_by(g, byPart), part = g - bh * byPart.d;
    const unsigned b = div_by(bh, byH), h = bh - b * byH.d;
    SeqTile q;
    if (!seq_rows(A.c.cu, A.c.slots, (int)b, A.c.T, A.c.n_slots, q)) return;
    const int n = (int)(((long long)q.len + (1 << A.sh) - 1) >> A.sh);
    if (n < 2) return;
    const size_t at = (size_t)part * 256 + __builtin_amdgcn_workitem_id_x();
    const size_t id0 = (size_t)(q.start >> A.sh) + b, step = (size_t)A.H * E / 4;
    float4 *ws = reinterpret_cast<float4 *>(A.ws) + (id0 * A.H + h) * (E / 4) + at;
    const float *lg = A.ws + (size_t)A.ids * A.H * E + id0 * A.H + h;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (A.c.cont && A.c.cont[b]) v = reinterpret_cast<const float4 *>(A.c.S)[((size_t)q.slot * A.H + h) * (E / 4) + at];
    for (int k = 0; k < n; k++) {
        const size_t o = (size_t)k * step;
        if (k + 1 < n) {
            const float4 l = ws[o];
            const float a = exp2f(lg[(size_t)k * A.H]);
            ws[o] = v;
            v.x = fmaf(a, v.x, l.x);
            v.y = fmaf(a, v.y, l.y);
            v.z = fmaf(a, v.z, l.z);
            v.w = fmaf(a, v.w, l.w);
        } else
            ws[o] = v;
    }
}

int heads_per_group(const gdnq_ssm_desc &d)
{
    const int per = d.hk ? d.H / d.hk : 1, most = d.dv == 64 ? 4 : 2;
    for (int n = most; n > 1; n /= 2)
        if (per % n == 0) return n;
    return 1;
}

// log2 of a segment's tokens: the longest that still gives the chip 2048
// waves of 32 columns each, if the T tokens were one sequence; from 256 tokens.
int segment_shift(const gdnq_ssm_desc &d, int T)
{
    const long long per = (long long)d.H * (d.dv / 32);
    int sh = 8;
    while (sh < 30 && ((long long)T >> (sh + 1)) * per >= 2048) sh++;
    return sh;
}

unsigned segment_ids(int n, int T, int sh) { return (unsigned)(T >> sh) + (unsigned)n; }

}  // namespace

size_t ssm_workspace(const gdnq_ssm_desc &d, int n, int T)
{
    const int sh = segment_shift(d, T);
    if (T <= 1 << sh) return 0;
    return (size_t)segment_ids(n, T, sh) * (size_t)d.H * ((size_t)d.dk * d.dv + 1) * 4;
}

hipError_t launch_ssm_prefill(const gdnq_ssm_desc &d, const SsmCall &c, hipStream_t st)
{
    const int hk = d.hk ? d.hk : d.H, hpw = heads_per_group(d), sh = segment_shift(d, c.T);
    const unsigned ids = segment_ids(c.n, c.T, sh), blocks = (unsigned)(d.H / hpw);
    const gdnq_ssm_io &io = c.io;
    const bool wide = wide_rows(io.x, io.ldx, 2) && wide_rows(io.B, io.ldb, 2) && wide_rows(io.C, io.ldc, 2) &&
                      wide_rows(io.y, io.ldy, 2);
    const SsmArgs A{c, d.H, hk, sh, ids, d.dt_min, d.dt_max, (d.flags & GDNQ_SSM_SOFTPLUS) != 0, wide,
                    make_divisor(blocks), reinterpret_cast<float *>(c.ws)};
    return with_dims(d.dk, d.dv, [&](auto DK, auto DV) {
        const auto go = [&](auto HPW) {
            using G = SsmGeom<DK.value, DV.value, HPW.value>;
            if (c.T > 1 << sh) {
                hipLaunchKernelGGL((ssm_chunk_kernel<DK.value, DV.value, HPW.value, true>), dim3(ids * blocks),
                                   dim3(G::NT), 0, st, A);
                constexpr unsigned parts = DK.value * DV.value / 1024;
                hipLaunchKernelGGL((ssm_join_kernel<DK.value * DV.value>), dim3((unsigned)c.n * d.H * parts), dim3(256),
                                   0, st, A, make_divisor(parts), make_divisor((unsigned)d.H));
            }
            hipLaunchKernelGGL((ssm_chunk_kernel<DK.value, DV.value, HPW.value, false>), dim3(ids * blocks),
                               dim3(G::NT), 0, st, A);
            return hipGetLastError();
        };
        if constexpr (DV.value == 64)
            if (hpw == 4) return go(std::integral_constant<int, 4>{});
        if (hpw >= 2) return go(std::integral_constant<int, 2>{});
        return go(std::integral_constant<int, 1>{});
    });
}

}  // namespace gdnq
