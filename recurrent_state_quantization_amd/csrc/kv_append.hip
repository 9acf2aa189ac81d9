// kv_append.hip -- new tokens into the paged cache (gdnq_kv_append): queries
// and keys turned by their positions, keys and values stored behind the rows
// that their slot holds.
//
// One pass over the tokens' rows.  A workgroup takes a few tokens of a sequence:
// their (cos, sin) pairs and places are formed once in LDS and serve all heads,
// whose pieces it deals out over its threads in one order: queries, keys, values.
// Bound by HBM: 20011 tokens of 13 prompts, 32 query and 8 cache heads of 128,
// 99 us (5.0 TB/s, the rate of a large copy), 88 where a part of the rows is still
// in the memory's cache.  Of long calls the queries go past the caches, both ways
// (111 us through them); keys and values do not: they are read next.
#include "attn_launchers.hpp"
#include "paged.hpp"
#include "rotate.hpp"

namespace gdnq {
namespace {

constexpr int NT = 256, MAX_ROWS = 4;

struct AppendArgs {
    AppendCall c;
    HeadPieces p;
    int H, hk, d, shift;
    int rows;         // log2 of a workgroup's tokens
    int nv, pieces;   // pieces of a head of values, of a token
    float amp;
    bool turn, inverse;
    Divisor byPieces, byNv;
    unsigned nx;      // width of the grid
};

template <bool BF16, bool INTER, bool STREAM>
__global__ __launch_bounds__(NT) void kv_append_kernel(AppendArgs A)
{
    constexpr int V = Row16<BF16, STREAM>::V;
    __shared__ float2 cs[MAX_ROWS][128];
    __shared__ int page[MAX_ROWS], at[MAX_ROWS], position[MAX_ROWS];
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const int id = (int)block_id(A.nx);
    const AppendCall &c = A.c;
    // the first token, its sequence's tokens, and those from this one to the last
    int tok, entry, count, behind;
    if (c.cu) {
        if ((long long)id >= (long long)(c.T >> A.rows) + c.n) return;
        SeqTile x;
        if (!seq_tile(c.cu, nullptr, c.n, id, A.rows, c.T, 0x7FFFFFFF, x)) return;
        tok = x.start + (x.k << A.rows);
        entry = x.seq;
        count = x.len;
        behind = x.len - (x.k << A.rows);
    } else {
        if (id >= c.n) return;
        tok = entry = id;
        count = behind = 1;
    }
    SlotRows s;
    if (!slot_rows(c.kv, c.slots, entry, A.shift, s) || s.len < count) return;
    const int nr = min(1 << A.rows, behind), row0 = s.len - behind;
    if (t < nr) {
        const int row = row0 + t;
        page[t] = s.table[row >> A.shift];
        at[t] = row & ((1 << A.shift) - 1);
        position[t] = c.pos ? c.pos[tok + t] : row;
    }
    const int pairs = A.turn ? A.p.rot / 2 : 0;
    for (int i = t; i < nr * 128; i += NT) {
        const int r = i >> 7, x = i & 127;
        if (x >= pairs) continue;
        const unsigned long long f = c.table[x] * (unsigned long long)(long long)(c.pos ? c.pos[tok + r] : row0 + r);
        cs[r][x] = turn(A.inverse ? 0ull - f : f, A.amp);
    }
    __syncthreads();
    const int nq = c.q ? A.H * A.p.ni : 0, nk = A.hk * A.p.ni;
    for (int i = t; i < nr * A.pieces; i += NT) {
        const int r = (int)div_by((unsigned)i, A.byPieces), x = i - r * A.pieces;
        const bool query = x < nq, key = !query && x < nq + nk;
        const size_t row = (size_t)(tok + r);
        if (query) {
            const int h = (int)div_by((unsigned)x, A.p.byNi);
            turn_piece<BF16, INTER, STREAM>(c.q, row * c.ldq + (size_t)h * A.d, c.q_out,
                                               row * c.ldqo + (size_t)h * A.d, x - h * A.p.ni, cs[r], A.p);
            continue;
        }
        if (page[r] < 0 || page[r] >= c.kv.n_pages) continue;
        if (key) {
            const int y = x - nq, h = (int)div_by((unsigned)y, A.p.byNi);
            turn_piece<BF16, INTER, false>(c.k, row * c.ldk + (size_t)h * A.d, c.kv.k,
                                              row_at(c.kv, page[r], h, at[r]), y - h * A.p.ni, cs[r], A.p);
        } else {
            const int y = x - nq - nk, h = (int)div_by((unsigned)y, A.byNv), j = (y - h * A.nv) * V;
            const uint4 v = Row16<BF16, STREAM>::load(c.v, row * c.ldv + (size_t)h * A.d + j);
            Row16<BF16, false>::store(c.kv.v, row_at(c.kv, page[r], h, at[r]) + j, v);
        }
    }
    for (int i = t; i < nr * A.hk; i += NT) {
        const int r = i / A.hk, h = i - r * A.hk;
        if (page[r] < 0 || page[r] >= c.kv.n_pages) continue;
        if (c.kv.acc) c.kv.acc[sum_at(A.hk, A.shift, page[r], h, at[r])] = 0.0f;
        if (c.kv.pos) c.kv.pos[sum_at(A.hk, A.shift, page[r], h, at[r])] = position[r];
    }
}

// log2 of the tokens of a workgroup: four of a prompt, whose rows of a head lie together (the same call 95 us
// with one token where four take 88, 115 with eight; from memory 98, 99)
int log_rows(const AppendCall &c) { return c.cu && c.T >= 1024 ? 2 : 0; }

HeadPieces pieces_of(const gdnq_attn_desc &d, const gdnq_rope_desc *r)
{
    const bool inter = r && (r->flags & GDNQ_ROPE_INTERLEAVED);
    return head_pieces(d.d, r ? r->rot : 0, inter, d.io_dtype == GDNQ_IO_BF16);
}

long long pieces_of_token(const gdnq_attn_desc &d, const AppendCall &c, int ni, int nv)
{
    return ((c.q ? (long long)d.H : 0) + d.hk) * ni + (long long)d.hk * nv;
}

}  // namespace

bool kv_append_numbers(const gdnq_attn_desc &d, const gdnq_rope_desc *r, const AppendCall &c)
{
    const int nv = d.d / (d.io_dtype == GDNQ_IO_BF16 ? 8 : 4);
    return pieces_of_token(d, c, pieces_of(d, r).ni, nv) <= (0x7FFFFFFF - NT) >> log_rows(c);
}

hipError_t launch_kv_append(const gdnq_attn_desc &d, const gdnq_rope_desc *r, const AppendCall &c, hipStream_t st)
{
    const bool bf16 = d.io_dtype == GDNQ_IO_BF16, inter = r && (r->flags & GDNQ_ROPE_INTERLEAVED);
    const int es = bf16 ? 2 : 4;
    AppendArgs A{c, pieces_of(d, r), d.H, d.hk, d.d, __builtin_ctz((unsigned)d.page), log_rows(c),
                 d.d / (16 / es), 0, r ? r->amp : 1.0f, r != nullptr, r && (r->flags & GDNQ_ROPE_INVERSE), {}, {}, 0};
    A.pieces = (int)pieces_of_token(d, c, A.p.ni, A.nv);
    A.byPieces = make_divisor((unsigned)A.pieces);
    A.byNv = make_divisor((unsigned)A.nv);
    const dim3 grid = grid_of(c.cu ? (unsigned long long)(c.T >> A.rows) + c.n : c.n, NT);
    A.nx = grid.x;
    // rows off 16 bytes share cache lines between lanes: 128 us through the caches, 211 past them
    const bool stream = streams(2ull * c.T * ((c.q ? d.H : 0) + 2 * d.hk) * d.d * es) && wide_rows(c.k, c.ldk, es) &&
                        wide_rows(c.v, c.ldv, es) &&
                        (!c.q || (wide_rows(c.q, c.ldq, es) && wide_rows(c.q_out, c.ldqo, es)));
    return with_bool(bf16, [&](auto b) {
        return with_bool(inter, [&](auto n) {
            return with_bool(stream, [&](auto o) {
                constexpr bool B = decltype(b)::value, N = decltype(n)::value, S = decltype(o)::value;
                hipLaunchKernelGGL((kv_append_kernel<B, N, S>), grid, dim3(NT), 0, st, A);
                return hipGetLastError();
            });
        });
    });
}

}  // namespace gdnq
