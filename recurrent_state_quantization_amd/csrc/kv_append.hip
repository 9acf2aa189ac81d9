// kv_append.hip -- new tokens into the paged cache (gdnq_kv_append): queries
// and keys turned by their positions, keys and values stored behind the rows
// that their slot holds.
//
// One pass over the tokens' rows.  A workgroup takes a token: its (cos, sin)
// pairs are formed once in LDS and serve the query and the key heads.
#include "attn_launchers.hpp"
#include "paged.hpp"
#include "rotate.hpp"

namespace gdnq {
namespace {

struct AppendArgs {
    AppendCall c;
    HeadPieces p;
    int H, hk, d, shift;
    float amp;
    bool turn, inverse;
    unsigned nx;   // width of the grid
};

template <bool BF16, int V, bool INTER>
__global__ __launch_bounds__(256) void kv_append_kernel(AppendArgs A)
{
    using P = Pack<BF16, V>;
    __shared__ float2 cs[128];
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const int id = (int)block_id(A.nx);
    const AppendCall &c = A.c;
    // the token, its sequence's last row and the rows behind it
    int tok, entry, behind;
    if (c.cu) {
        if ((long long)id >= (long long)c.T + c.n) return;
        SeqTile x;
        if (!seq_tile(c.cu, nullptr, c.n, id, 0, c.T, 0x7FFFFFFF, x)) return;
        tok = x.start + x.k;
        entry = x.seq;
        behind = x.len - x.k;
    } else {
        if (id >= c.n) return;
        tok = entry = id;
        behind = 1;
    }
    SlotRows s;
    if (!slot_rows(c.kv, c.slots, entry, A.shift, s)) return;
    const int count = c.cu ? c.cu[entry + 1] - c.cu[entry] : 1, row = s.len - behind;
    if (s.len < count) return;
    const int pos = c.pos ? c.pos[tok] : row;
    for (int i = t; i < A.p.rot / 2; i += 256) {
        unsigned long long f = A.turn ? c.table[i] * (unsigned long long)(long long)pos : 0ull;
        cs[i] = turn(A.inverse ? 0ull - f : f, A.amp);
    }
    __syncthreads();
    if (c.q)
        for (int i = t; i < A.H * A.p.ni; i += 256) {
            const int h = (int)div_by((unsigned)i, A.p.byNi);
            turn_piece<BF16, V, INTER>(c.q, (size_t)tok * c.ldq + (size_t)h * A.d, c.q_out,
                                       (size_t)tok * c.ldqo + (size_t)h * A.d, i - h * A.p.ni, cs, A.p);
        }
    const int page = s.table[row >> A.shift], off = row & ((1 << A.shift) - 1);
    if (page < 0 || page >= c.kv.n_pages) return;
    for (int i = t; i < A.hk * A.p.ni; i += 256) {
        const int h = (int)div_by((unsigned)i, A.p.byNi);
        turn_piece<BF16, V, INTER>(c.k, (size_t)tok * c.ldk + (size_t)h * A.d, c.kv.k, row_at(c.kv, page, h, off),
                                   i - h * A.p.ni, cs, A.p);
    }
    const int nv = A.d / V;
    for (int i = t; i < A.hk * nv; i += 256) {
        const int h = i / nv, j = (i - h * nv) * V;
        P::store(c.kv.v, row_at(c.kv, page, h, off) + j, P::load(c.v, (size_t)tok * c.ldv + (size_t)h * A.d + j));
    }
    for (int h = t; h < A.hk; h += 256) {
        if (c.kv.acc) c.kv.acc[sum_at(A.hk, A.shift, page, h, off)] = 0.0f;
        if (c.kv.pos) c.kv.pos[sum_at(A.hk, A.shift, page, h, off)] = pos;
    }
}

}  // namespace

hipError_t launch_kv_append(const gdnq_attn_desc &d, const gdnq_rope_desc *r, const AppendCall &c, hipStream_t st)
{
    const bool bf16 = d.io_dtype == GDNQ_IO_BF16, inter = r && (r->flags & GDNQ_ROPE_INTERLEAVED);
    const int es = bf16 ? 2 : 4, rot = r ? r->rot : 0;
    const bool wide = wide_pieces(d.d, rot, inter, es) && wide_rows(c.k, c.ldk, es) && wide_rows(c.v, c.ldv, es) &&
                      (!c.q || (wide_rows(c.q, c.ldq, es) && wide_rows(c.q_out, c.ldqo, es)));
    AppendArgs A{c, head_pieces(d.d, rot, inter, wide ? 16 / es : 1), d.H, d.hk, d.d, __builtin_ctz((unsigned)d.page),
                 r ? r->amp : 1.0f, r != nullptr, r && (r->flags & GDNQ_ROPE_INVERSE), 0};
    const dim3 grid = grid_of(c.cu ? (unsigned long long)c.T + c.n : c.n, 256);
    A.nx = grid.x;
    return with_bool(bf16, [&](auto b) {
        return with_bool(wide, [&](auto w) {
            return with_bool(inter, [&](auto n) {
                constexpr bool B = decltype(b)::value;
                constexpr int V = decltype(w)::value ? (B ? 8 : 4) : 1;
                hipLaunchKernelGGL((kv_append_kernel<B, V, decltype(n)::value>), grid, dim3(256), 0, st, A);
                return hipGetLastError();
            });
        });
    });
}

}  // namespace gdnq
