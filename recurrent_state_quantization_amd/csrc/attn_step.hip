// attn_step.hip -- the attention of one new token of each entry over its rows
// in the paged cache (gdnq_attn_step): per query head
//   s_r = scale q . k_r,  w_r = e^{s_r - m} / sum e^{s - m},  o = sum w_r v_r
// with one pass over the rows, which keeps the running maximum m, the sum and
// the output, all in fp32.
#include "attn_launchers.hpp"
#include "paged.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

constexpr float LOG2E = 1.44269504f, LOWEST = -3.4028234e38f;

struct AttnArgs {
    AttnCall c;
    int H, hk, shift, window;
    float scale2, decay;   // scale log2(e): weights are powers of two
    Divisor byHk;
    unsigned nx;
};

template <bool BF16, int D>
__global__ __launch_bounds__(256) void attn_simple_kernel(AttnArgs A)
{
    constexpr int E = D / 64;
    __shared__ float mj[4], lj[4], oj[4][D];
    const AttnCall &c = A.c;
    const unsigned id = block_id(A.nx);
    const unsigned i = div_by(id, A.byHk), h = id - i * (unsigned)A.hk;
    if (i >= (unsigned)c.n) return;
    SlotRows s;
    if (!slot_rows(c.kv, c.slots, (int)i, A.shift, s)) return;
    const int t = (int)__builtin_amdgcn_workitem_id_x(), lane = t & 63, w = t >> 6;
    const int first = A.window ? max(0, s.len - A.window) : 0, G = A.H / A.hk;
    for (int g = 0; g < G; g++) {
        const size_t hq = (size_t)(h * G + g) * D + lane * E;
        float q[E], o[E], m = LOWEST, l = 0.0f;
#pragma unroll
        for (int e = 0; e < E; e++) {
            q[e] = load1<BF16>(c.q, (size_t)i * c.ldq + hq + e) * A.scale2;
            o[e] = 0.0f;
        }
        auto score = [&](int r, size_t &at, size_t &sum) {
            const int p = s.table[r >> A.shift], off = r & ((1 << A.shift) - 1);
            if (p < 0 || p >= c.kv.n_pages) return -INFINITY;
            at = row_at(c.kv, p, (int)h, off) + lane * E;
            sum = sum_at(A.hk, A.shift, p, (int)h, off);
            float x = 0.0f;
#pragma unroll
            for (int e = 0; e < E; e++) x = fmaf(q[e], load1<BF16>(c.kv.k, at + e), x);
            return lanes_sum<64>(x);
        };
        size_t at = 0, sum = 0;
        for (int r = first + w; r < s.len; r += 4) {
            const float x = score(r, at, sum);
            if (x == -INFINITY) continue;
            const float mn = fmaxf(m, x), f = __builtin_amdgcn_exp2f(m - mn), p = __builtin_amdgcn_exp2f(x - mn);
            m = mn;
            l = fmaf(l, f, p);
#pragma unroll
            for (int e = 0; e < E; e++) o[e] = fmaf(p, load1<BF16>(c.kv.v, at + e), o[e] * f);
        }
        __syncthreads();
        mj[w] = m;
        lj[w] = l;
#pragma unroll
        for (int e = 0; e < E; e++) oj[w][lane * E + e] = o[e];
        __syncthreads();
        const float M = fmaxf(fmaxf(mj[0], mj[1]), fmaxf(mj[2], mj[3]));
        float L = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; k++) L = fmaf(lj[k], __builtin_amdgcn_exp2f(mj[k] - M), L);
        if (w == 0) {
#pragma unroll
            for (int e = 0; e < E; e++) {
                float x = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; k++) x = fmaf(oj[k][lane * E + e], __builtin_amdgcn_exp2f(mj[k] - M), x);
                store1<BF16>(c.o, (size_t)i * c.ldo + hq + e, L > 0.0f ? x / L : 0.0f);
            }
        }
        if (c.kv.acc)
            for (int r = first + w; r < s.len; r += 4) {
                const float x = score(r, at, sum);
                if (x == -INFINITY || lane != 0) continue;
                const float was = c.kv.acc[sum];
                c.kv.acc[sum] = (g == 0 ? A.decay * was : was) + __builtin_amdgcn_exp2f(x - M) / L;
            }
    }
}

}  // namespace

size_t attn_workspace(const gdnq_attn_desc &, const gdnq_kv &, int) { return 0; }

hipError_t launch_attn_step(const gdnq_attn_desc &d, const AttnCall &c, hipStream_t st)
{
    const dim3 grid = grid_of((unsigned long long)c.n * d.hk, 256);
    const AttnArgs A{c, d.H, d.hk, __builtin_ctz((unsigned)d.page), d.window, d.scale * LOG2E, d.acc_decay,
                     make_divisor((unsigned)d.hk), grid.x};
    return with_bool(d.io_dtype == GDNQ_IO_BF16, [&](auto bf) {
        constexpr bool B = decltype(bf)::value;
        if (d.d == 64) hipLaunchKernelGGL((attn_simple_kernel<B, 64>), grid, dim3(256), 0, st, A);
        else if (d.d == 128) hipLaunchKernelGGL((attn_simple_kernel<B, 128>), grid, dim3(256), 0, st, A);
        else hipLaunchKernelGGL((attn_simple_kernel<B, 256>), grid, dim3(256), 0, st, A);
        return hipGetLastError();
    });
}

}  // namespace gdnq
