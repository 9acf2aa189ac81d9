// ssm_prefill.hip -- the selective state space scan over packed prompts
// (gdnq_ssm_prefill): per head, with delta = clamp(softplus(dt + bias))
//   S <- e^{delta A} S + B (delta x)^T,   y = S^T C + D x.
// LinQuant, appendix Table 3, Mamba-2 row, in the dk x dv orientation.
//
// One workgroup per (sequence, head) walks the tokens; a thread owns 4
// columns of every RP-th row of the fp32 state for the whole sequence.
#include "layer_launchers.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

struct SsmArgs {
    SsmCall c;
    int H, hk;
    float dt_min, dt_max;
    bool sp;
    Divisor byH, byG;
};

template <int DK, int DV>
__global__ __launch_bounds__(256) void ssm_scan_kernel(SsmArgs A)
{
    constexpr int QL = DV / 4, RP = 256 / QL, NP = DK / RP;
    __shared__ float bl[DK], cl[DK], red[4][DV];
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const unsigned g = __builtin_amdgcn_workgroup_id_x();
    const unsigned b = __builtin_amdgcn_readfirstlane(div_by(g, A.byH));
    const unsigned h = __builtin_amdgcn_readfirstlane(g - b * (unsigned)A.H);
    const unsigned hb = div_by(h, A.byG);
    const gdnq_ssm_io &io = A.c.io;
    SeqTile q;
    if (!seq_rows(A.c.cu, A.c.slots, (int)b, A.c.T, A.c.n_slots, q)) return;
    const int cq = t % QL, r0 = t / QL;
    float4 *S = reinterpret_cast<float4 *>(A.c.S + ((size_t)q.slot * A.H + h) * DK * DV) + (size_t)r0 * QL + cq;
    const bool kept = A.c.cont && A.c.cont[b];
    float4 s[NP];
#pragma unroll
    for (int p = 0; p < NP; p++) s[p] = kept ? S[(size_t)p * RP * QL] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int n = 0; n < q.len; n++) {
        const size_t i = (size_t)q.start + n;
        if (t < DK) bl[t] = load1<true>(io.B, i * io.ldb + (size_t)hb * DK + t);
        else if (t < 2 * DK) cl[t - DK] = load1<true>(io.C, i * io.ldc + (size_t)hb * DK + t - DK);
        float dl = load1<true>(io.dt, i * io.lddt + h) + (io.dt_bias ? io.dt_bias[h] : 0.0f);
        if (A.sp) dl = softplus(dl);
        dl = fminf(fmaxf(dl, A.dt_min), A.dt_max);
        const float a = expf(dl * io.A[h]);
        float u[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; j++) {
            u[j] = dl * load1<true>(io.x, i * io.ldx + (size_t)h * DV + cq * 4 + j);
            y[j] = 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int p = 0; p < NP; p++) {
            const float bb = bl[p * RP + r0], c = cl[p * RP + r0];
            s[p].x = fmaf(bb, u[0], a * s[p].x);
            s[p].y = fmaf(bb, u[1], a * s[p].y);
            s[p].z = fmaf(bb, u[2], a * s[p].z);
            s[p].w = fmaf(bb, u[3], a * s[p].w);
            y[0] = fmaf(c, s[p].x, y[0]);
            y[1] = fmaf(c, s[p].y, y[1]);
            y[2] = fmaf(c, s[p].z, y[2]);
            y[3] = fmaf(c, s[p].w, y[3]);
        }
#pragma unroll
        for (int j = 0; j < 4; j++) {
            float p = y[j], r = y[j];
            swap32(p, r);
            p += r;
            if constexpr (QL == 16) {
                r = p;
                swap16(p, r);
                p += r;
            }
            if ((t & 63) < QL) red[t >> 6][cq * 4 + j] = p;
        }
        __syncthreads();
        if (t < DV) {
            const float x = load1<true>(io.x, i * io.ldx + (size_t)h * DV + t);
            const float o = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]);
            store1<true>(io.y, i * io.ldy + (size_t)h * DV + t, io.D ? fmaf(io.D[h], x, o) : o);
        }
    }
#pragma unroll
    for (int p = 0; p < NP; p++) S[(size_t)p * RP * QL] = s[p];
}

}  // namespace

size_t ssm_workspace(const gdnq_ssm_desc &, int, int) { return 0; }

hipError_t launch_ssm_prefill(const gdnq_ssm_desc &d, const SsmCall &c, hipStream_t st)
{
    const int hk = d.hk ? d.hk : d.H;
    const SsmArgs A{c, d.H, hk, d.dt_min, d.dt_max, (d.flags & GDNQ_SSM_SOFTPLUS) != 0,
                    make_divisor((unsigned)d.H), make_divisor((unsigned)(d.H / hk))};
    return with_dims(d.dk, d.dv, [&](auto DK, auto DV) {
        hipLaunchKernelGGL((ssm_scan_kernel<decltype(DK)::value, decltype(DV)::value>),
                           dim3((unsigned)c.n * (unsigned)d.H), dim3(256), 0, st, A);
        return hipGetLastError();
    });
}

}  // namespace gdnq
