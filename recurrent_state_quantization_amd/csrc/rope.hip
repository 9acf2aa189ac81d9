// rope.hip -- rotary positions of every head of a batch of token rows
// (gdnq_rope).
//
// A workgroup takes some rows: it forms the (cos, sin) pairs of each row once,
// in LDS, and turns all heads with them.  Bound by HBM, once these are paid for
// all heads together: 32768 rows of 40 heads of 128 in bf16 105 us (6.4 TB/s; 113
// through the caches), 8191 of 24 heads in fp32 37 us (5.4 TB/s).
#include <algorithm>

#include "attn_launchers.hpp"
#include "rotate.hpp"

namespace gdnq {
namespace {

constexpr int MAX_CS = 2048;   // (cos, sin) pairs of a workgroup's rows: 16 KB

struct RopeArgs {
    RopeCall c;
    HeadPieces p;
    int d, rows, heads;   // rows and heads per workgroup
    float amp;
    bool inverse;
    Divisor byRow, byPairs, bySplit;   // pieces per row, pairs per row, groups of heads
    unsigned nx;              // width of the grid
};

template <bool BF16, bool INTER, bool STREAM>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs A)
{
    __shared__ float2 cs[MAX_CS];
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const unsigned id = block_id(A.nx), rb = div_by(id, A.bySplit);
    const long long first = (long long)rb * A.rows;
    if (first >= A.c.rows) return;
    const int r0 = (int)first, h0 = (int)(id - rb * A.bySplit.d) * A.heads;
    const int nr = min(A.rows, A.c.rows - r0), nh = min(A.heads, A.c.H - h0);
    const int pairs = A.p.rot / 2;
    for (int i = t; i < nr * pairs; i += 256) {
        const int r = (int)div_by((unsigned)i, A.byPairs);
        const long long pos = A.c.pos[r0 + r];
        unsigned long long f = A.c.table[i - r * pairs] * (unsigned long long)pos;
        if (A.inverse) f = 0ull - f;
        cs[i] = turn(f, A.amp);
    }
    __syncthreads();
    const int per = A.heads * A.p.ni;
    for (int i = t; i < nr * per; i += 256) {
        const int r = (int)div_by((unsigned)i, A.byRow), in_row = i - r * per;
        const int h = (int)div_by((unsigned)in_row, A.p.byNi);
        if (h >= nh) continue;
        const size_t at = (size_t)(h0 + h) * A.d;
        const size_t row = (size_t)(r0 + r);
        turn_piece<BF16, INTER, STREAM>(A.c.x, row * A.c.ldx + at, A.c.y, row * A.c.ldy + at, in_row - h * A.p.ni,
                                           cs + r * pairs, A.p);
    }
}

}  // namespace

hipError_t launch_rope(const gdnq_rope_desc &d, const RopeCall &c, hipStream_t st)
{
    const bool bf16 = d.io_dtype == GDNQ_IO_BF16, inter = d.flags & GDNQ_ROPE_INTERLEAVED;
    const int es = bf16 ? 2 : 4;
    RopeArgs A{c, head_pieces(d.d, d.rot, inter, bf16), d.d, 1, c.H, d.amp,
               (d.flags & GDNQ_ROPE_INVERSE) != 0, {}, {}, {}, 0};
    // Whole rows, some 512 pieces in a workgroup (three rows of 40 heads of 128 in bf16 instead of one:
    // 124 us instead of 113), or, of few rows, the heads that give each thread a piece.
    A.heads = c.rows >= 512 ? c.H : std::min(c.H, std::max(1, 256 / A.p.ni));
    A.rows = A.heads < c.H ? 1 : std::max(1, std::min(512 / (c.H * A.p.ni), MAX_CS / (d.rot / 2)));
    A.byRow = make_divisor((unsigned)(A.heads * A.p.ni));
    A.byPairs = make_divisor((unsigned)(d.rot / 2));
    const unsigned split = (unsigned)((c.H + A.heads - 1) / A.heads);
    A.bySplit = make_divisor(split);
    const dim3 grid = grid_of((unsigned long long)((c.rows + A.rows - 1) / A.rows) * split, 256);
    A.nx = grid.x;
    // rows off 16 bytes share cache lines between lanes: 140 us through the caches, 150 past them
    const bool stream = streams(2ull * c.rows * c.H * d.d * es) && wide_rows(c.x, c.ldx, es) &&
                        wide_rows(c.y, c.ldy, es);
    return with_bool(bf16, [&](auto b) {
        return with_bool(inter, [&](auto n) {
            return with_bool(stream, [&](auto o) {
                constexpr bool B = decltype(b)::value, N = decltype(n)::value, S = decltype(o)::value;
                hipLaunchKernelGGL((rope_kernel<B, N, S>), grid, dim3(256), 0, st, A);
                return hipGetLastError();
            });
        });
    });
}

}  // namespace gdnq
