// conv.hip -- short causal depthwise convolution of a recurrent layer's
// inputs (gdnq_conv_prefill, gdnq_conv_step):
//   y_t,c = act(bias_c + sum_{k < W} w_k,c x_{t-(W-1)+k,c}),
// inputs before the sequence taken from the slot's state or zero.
//
// Every input is read once and every output written once; about 2 W + 10
// vector operations per element leave both kernels bound by HBM.  A lane
// owns V channels (16 bytes of a row; one channel where pointers, distances
// or the channel count are not multiples of 16 bytes: 32701 x 4097 178 us, 3.0
// TB/s, where 4096 take 107 us, 5.0 TB/s), a wave 64 V of them,
// and the taps slide along the tokens in registers.
#include "layer_launchers.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

struct ConvArgs {
    ConvCall c;
    int C;
    unsigned waves;   // channel blocks times tiles (prompts) or entries (single tokens)
    Divisor byCb;     // channel blocks per row
    unsigned nx;      // width of the grid
};

// act(bias + taps), one fused multiply-add per tap
template <bool BF16, int V, int W, bool SILU>
__device__ __forceinline__ void conv_taps(const float (&win)[W][V], const float (&w)[W][V], const float (&b)[V],
                                          float (&y)[V])
{
#pragma unroll
    for (int v = 0; v < V; v++) {
        float a = b[v];
#pragma unroll
        for (int k = 0; k < W; k++) a = fmaf(w[k][v], win[k][v], a);
        y[v] = SILU ? a * sigmoid<!BF16>(a) : a;
    }
}

template <int V, int W>
__device__ __forceinline__ void conv_weights(const ConvArgs &A, int c0, float (&w)[W][V], float (&b)[V])
{
#pragma unroll
    for (int k = 0; k < W; k++) load_weights<V>(A.c.w + (size_t)k * A.C + c0, w[k]);
#pragma unroll
    for (int v = 0; v < V; v++) b[v] = 0.0f;
    if (A.c.bias) load_weights<V>(A.c.bias + c0, b);
}

// address of element `off` of an io-dtype array
template <bool BF16>
__device__ __forceinline__ const char *row_ptr(const void *base, size_t off)
{
    return reinterpret_cast<const char *>(base) + off * (BF16 ? 2 : 4);
}

// One wave: 64 V channels of one tile of 2^SH tokens.  The wave of a
// sequence's first tile also stores the new state: it alone reads the old
// one, so no other wave can see it replaced.
template <bool BF16, int V, int W, bool SILU, int SH>
__global__ __launch_bounds__(256) void conv_prefill_kernel(ConvArgs A)
{
    using P = Pack<BF16, V>;
    constexpr int TT = 1 << SH, U = 8;
    const int lane = (int)(__builtin_amdgcn_workitem_id_x() & 63u);
    const unsigned wave = __builtin_amdgcn_readfirstlane(block_id(A.nx) * 4u +
                                                         (__builtin_amdgcn_workitem_id_x() >> 6));
    if (wave >= A.waves) return;
    const unsigned id = div_by(wave, A.byCb);
    const int c0 = ((int)(wave - id * A.byCb.d) * 64 + lane) * V;
    SeqTile q;
    if (!seq_tile(A.c.cu, A.c.slots, A.c.n, (int)id, SH, A.c.T, A.c.n_slots, q)) return;
    if (c0 >= A.C) return;

    float w[W][V], b[V], win[W][V], old[W - 1][V];
    conv_weights<V, W>(A, c0, w, b);
    const size_t t0 = (size_t)q.start + ((size_t)q.k << SH);
    const int nt = min(TT, q.len - (q.k << SH));
    const size_t hist = (size_t)q.slot * (W - 1) * A.C + c0;
    const bool kept = A.c.cont && A.c.cont[q.seq];
    if (q.k == 0) {
#pragma unroll
        for (int j = 0; j < W - 1; j++) {
#pragma unroll
            for (int v = 0; v < V; v++) old[j][v] = 0.0f;
            if (kept) load_vec<BF16, V>(A.c.state, hist + (size_t)j * A.C, old[j]);
#pragma unroll
            for (int v = 0; v < V; v++) win[j][v] = old[j][v];
        }
    } else {   // a tile holds more tokens than the taps reach back
#pragma unroll
        for (int j = 0; j < W - 1; j++) load_vec<BF16, V>(A.c.x, (t0 - (W - 1) + j) * A.c.ldx + c0, win[j]);
    }
    // U rows at a time, the next U on their way meanwhile
    const char *xp = row_ptr<BF16>(A.c.x, t0 * A.c.ldx + c0);
    char *yp = const_cast<char *>(row_ptr<BF16>(A.c.y, t0 * A.c.ldy + c0));
    const size_t dx = (size_t)A.c.ldx * sizeof(typename P::elem), dy = (size_t)A.c.ldy * sizeof(typename P::elem);
    const auto load = [&](typename P::raw(&in)[U], int m) {
#pragma unroll
        for (int u = 0; u < U; u++, xp += dx)
            if (u < m) in[u] = P::load(xp, 0);
    };
    const auto emit = [&](const typename P::raw &in) {
        float y[V];
        P::widen(in, win[W - 1]);
        conv_taps<BF16, V, W, SILU>(win, w, b, y);
        store_vec<BF16, V>(yp, 0, y);
        yp += dy;
#pragma unroll
        for (int j = 0; j < W - 1; j++)
#pragma unroll
            for (int v = 0; v < V; v++) win[j][v] = win[j + 1][v];
    };
    typename P::raw in[2][U];
    load(in[0], nt);
    int t = 0;
    for (; t + 2 * U <= nt; t += 2 * U) {
        load(in[1], U);
#pragma unroll
        for (int u = 0; u < U; u++) emit(in[0][u]);
        load(in[0], nt - t - 2 * U);
#pragma unroll
        for (int u = 0; u < U; u++) emit(in[1][u]);
    }
    if (t < nt) {
        load(in[1], nt - t - U);
#pragma unroll
        for (int u = 0; u < 2 * U; u++)
            if (t + u < nt) emit(in[u / U][u % U]);
    }
    if (q.k == 0) {
        float s[W - 1][V];
#pragma unroll
        for (int r = 0; r < W - 1; r++) {
            const int at = q.len - (W - 1) + r;   // the row's token, or one of the old state's
            if (at >= 0) {
                load_vec<BF16, V>(A.c.x, ((size_t)q.start + at) * A.c.ldx + c0, s[r]);
            } else {
#pragma unroll
                for (int j = 0; j < W - 1; j++)
                    if (j == W - 1 + at)
#pragma unroll
                        for (int v = 0; v < V; v++) s[r][v] = old[j][v];
            }
        }
#pragma unroll
        for (int r = 0; r < W - 1; r++) store_vec<BF16, V>(A.c.state, hist + (size_t)r * A.C, s[r]);
    }
}

// One wave: 64 V channels of one entry (1024 entries x 8192 channels in bf16:
// 23 us, 5.8 TB/s with part of it in the last-level cache).
template <bool BF16, int V, int W, bool SILU>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs A)
{
    const int lane = (int)(__builtin_amdgcn_workitem_id_x() & 63u);
    const unsigned wave = __builtin_amdgcn_readfirstlane(block_id(A.nx) * 4u +
                                                         (__builtin_amdgcn_workitem_id_x() >> 6));
    if (wave >= A.waves) return;
    const unsigned i = div_by(wave, A.byCb);
    const int c0 = ((int)(wave - i * A.byCb.d) * 64 + lane) * V;
    if (c0 >= A.C) return;
    float w[W][V], b[V], win[W][V], y[V];
    load_vec<BF16, V>(A.c.x, (size_t)i * A.c.ldx + c0, win[W - 1]);
    conv_weights<V, W>(A, c0, w, b);
    const int slot = A.c.slots ? A.c.slots[i] : (int)i;
    if (slot < 0 || slot >= A.c.n_slots) return;
    const size_t hist = (size_t)slot * (W - 1) * A.C + c0;
#pragma unroll
    for (int j = 0; j < W - 1; j++) load_vec<BF16, V>(A.c.state, hist + (size_t)j * A.C, win[j]);
    conv_taps<BF16, V, W, SILU>(win, w, b, y);
    store_vec<BF16, V>(A.c.y, (size_t)i * A.c.ldy + c0, y);
#pragma unroll
    for (int j = 0; j < W - 1; j++) store_vec<BF16, V>(A.c.state, hist + (size_t)j * A.C, win[j + 1]);
}

// f(BF16, V, W, SILU) as compile-time constants
template <class F>
hipError_t conv_dispatch(const gdnq_conv_desc &d, const ConvCall &c, F &&f)
{
    const bool bf = d.io_dtype == GDNQ_IO_BF16;
    const int es = bf ? 2 : 4, v = 16 / es;
    const bool wide = d.C % v == 0 && wide_rows(c.x, c.ldx, es) && wide_rows(c.y, c.ldy, es);
    return with_bool(bf, [&](auto BF) {
        return with_bool(wide, [&](auto WIDE) {
            constexpr int V = decltype(WIDE)::value ? (decltype(BF)::value ? 8 : 4) : 1;
            return with_bool((d.flags & GDNQ_CONV_SILU) != 0, [&](auto SILU) {
                const std::integral_constant<int, V> vc{};
                if (d.width == 2) return f(BF, vc, std::integral_constant<int, 2>{}, SILU);
                if (d.width == 3) return f(BF, vc, std::integral_constant<int, 3>{}, SILU);
                return f(BF, vc, std::integral_constant<int, 4>{}, SILU);
            });
        });
    });
}

}  // namespace

hipError_t launch_conv_prefill(const gdnq_conv_desc &d, const ConvCall &c, hipStream_t st)
{
    return conv_dispatch(d, c, [&](auto BF, auto V, auto W, auto SILU) {
        constexpr int SH = 4;   // 32 and 8 tokens a tile: 201 and 197 us for 32768 x 8192 bf16, 16: 190
        const unsigned ncb = (unsigned)((d.C + 64 * V.value - 1) / (64 * V.value));
        const unsigned waves = ncb * ((unsigned)(c.T >> SH) + (unsigned)c.n);
        const dim3 grid = grid_of((waves + 3) / 4, 256);
        const ConvArgs A{c, d.C, waves, make_divisor(ncb), grid.x};
        hipLaunchKernelGGL((conv_prefill_kernel<decltype(BF)::value, V.value, W.value, decltype(SILU)::value, SH>),
                           grid, dim3(256), 0, st, A);
        return hipGetLastError();
    });
}

hipError_t launch_conv_step(const gdnq_conv_desc &d, const ConvCall &c, hipStream_t st)
{
    return conv_dispatch(d, c, [&](auto BF, auto V, auto W, auto SILU) {
        const unsigned ncb = (unsigned)((d.C + 64 * V.value - 1) / (64 * V.value));
        const unsigned waves = ncb * (unsigned)c.n;
        const dim3 grid = grid_of((waves + 3) / 4, 256);
        const ConvArgs A{c, d.C, waves, make_divisor(ncb), grid.x};
        hipLaunchKernelGGL((conv_step_kernel<decltype(BF)::value, V.value, W.value, decltype(SILU)::value>),
                           grid, dim3(256), 0, st, A);
        return hipGetLastError();
    });
}

}  // namespace gdnq
