// ssm_step.hip -- one token of the selective state space scan for a pool of
// states (gdnq_ssm_step): per head, with delta = clamp(softplus(dt + bias))
//   S <- e^{delta A} S + B (delta x)^T,   y = S^T C + D x.
// LinQuant, appendix Table 3, Mamba-2 row, in the dk x dv orientation.
//
// The fp32 state is read and written once (8 dk dv bytes per head) against
// 5 operations per element: bound by HBM.  One workgroup per (entry, head);
// a thread owns 4 columns of every RP-th row, so each wave's accesses are
// 1 KiB of consecutive memory.  1024 entries of 32 heads of 128 x 128: 832 us
// (5.1 TB/s, the rate of a large copy).
#include "layer_launchers.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

struct SsmStepArgs {
    SsmCall c;
    int H, hk;
    float dt_min, dt_max;
    bool sp;
    Divisor byH, byG;
    unsigned nx;   // width of the grid
};

template <bool BF16, int DK, int DV>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmStepArgs A)
{
    constexpr int QL = DV / 4;        // lanes per row
    constexpr int RP = 256 / QL;      // rows per pass
    constexpr int NP = DK / RP;
    __shared__ float bl[DK], cl[DK], red[4][DV];
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const unsigned g = block_id(A.nx);
    const unsigned i = __builtin_amdgcn_readfirstlane(div_by(g, A.byH));
    const unsigned h = __builtin_amdgcn_readfirstlane(g - i * (unsigned)A.H);
    const unsigned hb = div_by(h, A.byG);
    const gdnq_ssm_io &io = A.c.io;
    if (i >= (unsigned)A.c.n) return;
    const int slot = A.c.slots ? A.c.slots[i] : (int)i;
    if (slot < 0 || slot >= A.c.n_slots) return;   // uniform, before the barriers
    const int cq = t % QL, r0 = t / QL;
    float4 *S = reinterpret_cast<float4 *>(A.c.S + ((size_t)slot * A.H + h) * DK * DV) + (size_t)r0 * QL + cq;
    float4 s[NP];
#pragma unroll
    for (int p = 0; p < NP; p++) s[p] = S[(size_t)p * RP * QL];
    if (t < DK) bl[t] = load1<BF16>(io.B, (size_t)i * io.ldb + (size_t)hb * DK + t);
    else if (t < 2 * DK) cl[t - DK] = load1<BF16>(io.C, (size_t)i * io.ldc + (size_t)hb * DK + t - DK);
    float dl = load1<BF16>(io.dt, (size_t)i * io.lddt + h) + (io.dt_bias ? io.dt_bias[h] : 0.0f);
    if (A.sp) dl = softplus(dl);
    dl = fminf(fmaxf(dl, A.dt_min), A.dt_max);
    const float a = expf(dl * io.A[h]);
    float u[4];
#pragma unroll
    for (int j = 0; j < 4; j++)
        u[j] = dl * load1<BF16>(io.x, (size_t)i * io.ldx + (size_t)h * DV + cq * 4 + j);
    __syncthreads();
    float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < NP; p++) {
        const float b = bl[p * RP + r0], c = cl[p * RP + r0];
        s[p].x = fmaf(b, u[0], a * s[p].x);
        s[p].y = fmaf(b, u[1], a * s[p].y);
        s[p].z = fmaf(b, u[2], a * s[p].z);
        s[p].w = fmaf(b, u[3], a * s[p].w);
        y[0] = fmaf(c, s[p].x, y[0]);
        y[1] = fmaf(c, s[p].y, y[1]);
        y[2] = fmaf(c, s[p].z, y[2]);
        y[3] = fmaf(c, s[p].w, y[3]);
        S[(size_t)p * RP * QL] = s[p];
    }
    // sum over the row groups: the wave's by lane swaps, then the four waves'
#pragma unroll
    for (int j = 0; j < 4; j++) {
        float p = y[j], q = y[j];
        swap32(p, q);
        p += q;
        if constexpr (QL == 16) {
            q = p;
            swap16(p, q);
            p += q;
        }
        if ((t & 63) < QL) red[t >> 6][cq * 4 + j] = p;
    }
    __syncthreads();
    if (t < DV) {
        const float x = load1<BF16>(io.x, (size_t)i * io.ldx + (size_t)h * DV + t);
        const float o = (red[0][t] + red[1][t]) + (red[2][t] + red[3][t]);
        store1<BF16>(io.y, (size_t)i * io.ldy + (size_t)h * DV + t, io.D ? fmaf(io.D[h], x, o) : o);
    }
}

}  // namespace

hipError_t launch_ssm_step(const gdnq_ssm_desc &d, const SsmCall &c, hipStream_t st)
{
    const int hk = d.hk ? d.hk : d.H;
    const dim3 grid = grid_of((unsigned)c.n * (unsigned)d.H, 256);
    const SsmStepArgs A{c, d.H, hk, d.dt_min, d.dt_max, (d.flags & GDNQ_SSM_SOFTPLUS) != 0,
                        make_divisor((unsigned)d.H), make_divisor((unsigned)(d.H / hk)), grid.x};
    return with_dims(d.dk, d.dv, [&](auto DK, auto DV) {
        return with_bool(d.io_dtype == GDNQ_IO_BF16, [&](auto bf) {
            hipLaunchKernelGGL((ssm_step_kernel<decltype(bf)::value, decltype(DK)::value, decltype(DV)::value>),
                               grid, dim3(256), 0, st, A);
            return hipGetLastError();
        });
    });
}

}  // namespace gdnq
