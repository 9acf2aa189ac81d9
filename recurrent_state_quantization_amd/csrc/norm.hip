// norm.hip -- RMS norms around a recurrent block: behind it with its gate
// (gdnq_norm_gated), and in front of the next one with the residual sum
// (gdnq_norm_residual).
//
// Each input is read once and each output written once, so both kernels are
// bound by HBM; the row (or group) stays in registers between its sum of
// squares and its output.  NT threads hold one group, K pieces of V values
// each, piece k of thread t at (k NT + t) V, so every access of a wave is
// consecutive.  NT and K grow with the group (norm_dispatch).  Measured in
// bf16: 32768 rows of 4096 gated in groups of 512 135 us (6.0 TB/s; a large
// copy reaches 5.0), 32768 x 4096 on an fp32 residual stream with a norm
// behind the block 297 us (5.4 TB/s).  Small groups leave lanes idle (16 a
// group at least: 32768 x 4096 in groups of 64 186 us, 4.3 TB/s; 4080 in groups
// of 24 429 us), and rows that are not multiples of 16 bytes take one value a
// lane (32768 x 4097 369 us, 2.2 TB/s; residual 526 us, 3.1 TB/s).
#include "layer_launchers.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

struct NormArgs {
    NormCall c;
    int D, group;
    unsigned groups;   // rows times groups per row
    Divisor byGroups;  // groups per row
    uint32_t flags;
    float eps, w_offset, inv_n;
    unsigned nx;       // width of the grid
};

// Sum over a group's NT threads, in each of them.  `slot` numbers the sums
// of a kernel, so that one's partials are not overwritten by the next's.
template <int NT>
__device__ __forceinline__ float group_sum(float x, float (*part)[16], int slot)
{
    x = lanes_sum<(NT < 64 ? NT : 64)>(x);
    if constexpr (NT > 64) {
        const int t = (int)__builtin_amdgcn_workitem_id_x();
        if ((t & 63) == 0) part[slot][t >> 6] = x;
        __syncthreads();
        x = part[slot][0];
#pragma unroll
        for (int i = 1; i < NT / 64; i++) x += part[slot][i];
    }
    return x;
}

// 1 / sqrt(mean square + eps).  The instruction takes normal arguments only;
// a smaller one (eps below 2^-126 and a row as small) goes through it 2^48
// times as large.
__device__ __forceinline__ float inv_rms(float ss, const NormArgs &A)
{
    const float m = fmaf(ss, A.inv_n, A.eps);
    const bool small = m < 0x1p-126f;
    const float r = __builtin_amdgcn_rsqf(small ? m * 0x1p48f : m);
    return small ? r * 0x1p24f : r;
}

template <bool BF16, int V, int NT, int K>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void norm_gated_kernel(NormArgs A)
{
    constexpr int WG = NT < 256 ? 256 : NT;
    using P = Pack<BF16, V>;
    __shared__ float part[1][16];
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const unsigned gi = block_id(A.nx) * (WG / NT) + (unsigned)t / NT;
    if (gi >= A.groups) return;   // whole groups of lanes; a group of several waves has its workgroup to itself
    const unsigned row = div_by(gi, A.byGroups);
    const int c0 = (int)(gi - row * A.byGroups.d) * A.group, l = t % NT;
    const size_t xo = (size_t)row * A.c.ldx + c0, zo = (size_t)row * A.c.ldz + c0, yo = (size_t)row * A.c.ldy + c0;
    const float *wp = A.c.w + ((A.flags & GDNQ_NORM_GROUP_WEIGHT) ? 0 : c0);
    const bool first = (A.flags & GDNQ_NORM_GATE_FIRST) != 0;
    typename P::raw xr[K], zr[K];
    float u[K][V], g[K][V];
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int at = (k * NT + l) * V;
        if (at < A.group) {
            xr[k] = P::load(A.c.x, xo + at);
            if (A.c.z) zr[k] = P::load(A.c.z, zo + at);
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < K; k++) {
        if ((k * NT + l) * V < A.group) {
            P::widen(xr[k], u[k]);
            if (A.c.z) P::widen(zr[k], g[k]);
#pragma unroll
            for (int v = 0; v < V; v++) {
                if (A.c.z) {
                    const float s = sigmoid<!BF16>(g[k][v]);
                    g[k][v] = (A.flags & GDNQ_NORM_GATE_SIGMOID) ? s : g[k][v] * s;
                } else
                    g[k][v] = 1.0f;
                if (first) u[k][v] *= g[k][v];
                ss = fmaf(u[k][v], u[k][v], ss);
            }
        }
    }
    const float r = inv_rms(group_sum<NT>(ss, part, 0), A);
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int at = (k * NT + l) * V;
        if (at < A.group) {
            float w[V], y[V];
            load_weights<V>(wp + at, w);
#pragma unroll
            for (int v = 0; v < V; v++) {
                y[v] = u[k][v] * r * (w[v] + A.w_offset);
                if (!first) y[v] *= g[k][v];
            }
            store_vec<BF16, V>(A.c.y, yo + at, y);
        }
    }
}

// V residual values, fp32 or of the io type
template <bool R32, bool BF16, int V>
__device__ __forceinline__ void load_res(const void *base, size_t off, float (&out)[V])
{
    if constexpr (R32) load_weights<V>(reinterpret_cast<const float *>(base) + off, out);
    else load_vec<BF16, V>(base, off, out);
}

template <bool R32, bool BF16, int V>
__device__ __forceinline__ void store_res(void *base, size_t off, const float (&v)[V])
{
    if constexpr (!R32) store_vec<BF16, V>(base, off, v);
    else if constexpr (V == 1) reinterpret_cast<float *>(base)[off] = v[0];
    else
#pragma unroll
        for (int i = 0; i < V / 4; i++)
            reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + off)[i] =
                make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

template <bool BF16, bool R32, int V, int NT, int K>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void norm_residual_kernel(NormArgs A)
{
    constexpr int WG = NT < 256 ? 256 : NT;
    __shared__ float part[2][16];
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const unsigned row = block_id(A.nx) * (WG / NT) + (unsigned)t / NT;
    if (row >= A.groups) return;
    const int l = t % NT;
    float p[K][V], r[K][V];
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int at = (k * NT + l) * V;
        if (at < A.D) {
            load_vec<BF16, V>(A.c.x, (size_t)row * A.c.ldx + at, p[k]);
            load_res<R32, BF16, V>(A.c.res, (size_t)row * A.c.ldr + at, r[k]);
        }
    }
    if (A.c.post_w) {
        float ss = 0.0f;
#pragma unroll
        for (int k = 0; k < K; k++)
            if ((k * NT + l) * V < A.D)
#pragma unroll
                for (int v = 0; v < V; v++) ss = fmaf(p[k][v], p[k][v], ss);
        const float q = inv_rms(group_sum<NT>(ss, part, 0), A);
#pragma unroll
        for (int k = 0; k < K; k++) {
            const int at = (k * NT + l) * V;
            if (at < A.D) {
                float w[V];
                load_weights<V>(A.c.post_w + at, w);
#pragma unroll
                for (int v = 0; v < V; v++) p[k][v] *= q * (w[v] + A.w_offset);
            }
        }
    }
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int at = (k * NT + l) * V;
        if (at < A.D) {
#pragma unroll
            for (int v = 0; v < V; v++) {
                r[k][v] = fmaf(A.c.scale, p[k][v], r[k][v]);
                ss = fmaf(r[k][v], r[k][v], ss);
            }
            store_res<R32, BF16, V>(A.c.res_out, (size_t)row * A.c.ldro + at, r[k]);
        }
    }
    if (!A.c.y) return;
    const float q = inv_rms(group_sum<NT>(ss, part, 1), A);
#pragma unroll
    for (int k = 0; k < K; k++) {
        const int at = (k * NT + l) * V;
        if (at < A.D) {
            float w[V], y[V];
            load_weights<V>(A.c.w + at, w);
#pragma unroll
            for (int v = 0; v < V; v++) y[v] = r[k][v] * q * (w[v] + A.w_offset);
            store_vec<BF16, V>(A.c.y, (size_t)row * A.c.ldy + at, y);
        }
    }
}

// f(NT, K) for a group of n values: 16 lanes up to 32 pieces of V values, a
// wave up to 128, four waves up to 1024, sixteen above.
template <int V, class F>
hipError_t norm_dispatch(int n, F &&f)
{
    const int m = (n + V - 1) / V;
#define GDNQ_NORM_CASE(nt, k) \
    if (m <= nt * k) return f(std::integral_constant<int, nt>{}, std::integral_constant<int, k>{})
    GDNQ_NORM_CASE(16, 1);
    GDNQ_NORM_CASE(16, 2);
    GDNQ_NORM_CASE(64, 1);
    GDNQ_NORM_CASE(64, 2);
    GDNQ_NORM_CASE(256, 1);
    GDNQ_NORM_CASE(256, 2);
    GDNQ_NORM_CASE(256, 4);
    GDNQ_NORM_CASE(1024, 4);
    if constexpr (V <= 4) GDNQ_NORM_CASE(1024, 8);
    if constexpr (V == 1) GDNQ_NORM_CASE(1024, 32);
#undef GDNQ_NORM_CASE
    return hipErrorInvalidValue;
}

NormArgs norm_args(const gdnq_norm_desc &d, const NormCall &c)
{
    const int group = d.group ? d.group : d.D;
    const unsigned per = (unsigned)(d.D / group);
    return NormArgs{c, d.D, group, (unsigned)c.rows * per, make_divisor(per), d.flags, d.eps, d.w_offset,
                    1.0f / (float)group, 0};
}

}  // namespace

hipError_t launch_norm_gated(const gdnq_norm_desc &d, const NormCall &c, hipStream_t st)
{
    NormArgs A = norm_args(d, c);
    const bool bf = d.io_dtype == GDNQ_IO_BF16;
    const int es = bf ? 2 : 4;
    const bool wide = A.group % (16 / es) == 0 && wide_rows(c.x, c.ldx, es) && wide_rows(c.y, c.ldy, es) &&
                      (!c.z || wide_rows(c.z, c.ldz, es));
    return with_bool(bf, [&](auto BF) {
        return with_bool(wide, [&](auto WIDE) {
            constexpr int V = decltype(WIDE)::value ? (decltype(BF)::value ? 8 : 4) : 1;
            return norm_dispatch<V>(A.group, [&](auto NT, auto K) {
                constexpr int WG = NT.value < 256 ? 256 : NT.value, per = WG / NT.value;
                const dim3 grid = grid_of((A.groups + per - 1) / per, WG);
                A.nx = grid.x;
                hipLaunchKernelGGL((norm_gated_kernel<decltype(BF)::value, V, NT.value, K.value>),
                                   grid, dim3(WG), 0, st, A);
                return hipGetLastError();
            });
        });
    });
}

hipError_t launch_norm_residual(const gdnq_norm_desc &d, const NormCall &c, hipStream_t st)
{
    NormArgs A = norm_args(d, c);
    const bool bf = d.io_dtype == GDNQ_IO_BF16, r32 = bf && (d.flags & GDNQ_NORM_RES_F32);
    const int es = bf ? 2 : 4, rs = r32 ? 4 : es;
    const bool wide = d.D % (16 / es) == 0 && wide_rows(c.x, c.ldx, es) && wide_rows(c.res, c.ldr, rs) &&
                      wide_rows(c.res_out, c.ldro, rs) && (!c.y || wide_rows(c.y, c.ldy, es));
    const auto go = [&](auto BF, auto R32, auto WIDE) {
        constexpr int V = decltype(WIDE)::value ? (decltype(BF)::value ? 8 : 4) : 1;
        return norm_dispatch<V>(d.D, [&](auto NT, auto K) {
            constexpr int WG = NT.value < 256 ? 256 : NT.value, per = WG / NT.value;
            const dim3 grid = grid_of((A.groups + per - 1) / per, WG);
            A.nx = grid.x;
            hipLaunchKernelGGL((norm_residual_kernel<decltype(BF)::value, decltype(R32)::value, V, NT.value, K.value>),
                               grid, dim3(WG), 0, st, A);
            return hipGetLastError();
        });
    };
    return with_bool(wide, [&](auto WIDE) {
        if (!bf) return go(std::false_type{}, std::false_type{}, WIDE);
        return with_bool(r32, [&](auto R32) { return go(std::true_type{}, R32, WIDE); });
    });
}

}  // namespace gdnq
