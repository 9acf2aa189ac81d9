// kv_evict.hip -- rows of least accumulated weight leave the paged cache
// (gdnq_kv_evict).
//
// One workgroup per entry and head.  The sums become whole numbers of the same
// order, the protected rows the largest; four rounds of counting by 8 bits find
// the largest number that leaves, and how many rows of that number leave (the
// lower ones).  Then the rows before the budget that leave (holes) and the rows
// behind it that stay, equally many, are numbered in order by prefix counts;
// the k-th of these moves into the k-th hole.  Sources lie behind the budget
// and destinations before it, so the moves are independent.
#include <algorithm>

#include "attn_launchers.hpp"
#include "paged.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

struct EvictArgs {
    EvictCall c;
    int hk, shift, most;   // moves of a head at most
    int pieces;            // 16-byte pieces of a row; ldp, ldh and ldr count such pieces here
    Divisor byHk;
    unsigned nx;
};

// Whole numbers in the order of the sums (both zeros alike).
__device__ __forceinline__ unsigned order_of(float x)
{
    const unsigned u = __float_as_uint(x + 0.0f);
    return (int)u < 0 ? ~u : u | 0x80000000u;
}

constexpr int NT = 256;

// Counts of the set flags of lower threads and of all, over the workgroup.
__device__ __forceinline__ int count_before(bool f, int *part, int &total)
{
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const unsigned long long b = __ballot(f);
    const int in_wave = __popcll(b & ((1ull << (t & 63)) - 1));
    __syncthreads();
    if ((t & 63) == 0) part[t >> 6] = __popcll(b);
    __syncthreads();
    int before = in_wave;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; w++) {
        if (w < (t >> 6)) before += part[w];
        total += part[w];
    }
    return before;
}

__global__ __launch_bounds__(NT) void kv_evict_kernel(EvictArgs A)
{
    __shared__ int hist[256], part[NT / 64], chosen[2], top;
    const EvictCall &c = A.c;
    const unsigned id = block_id(A.nx);
    const int i = (int)div_by(id, A.byHk), h = (int)(id - (unsigned)i * (unsigned)A.hk);
    if (i >= c.n) return;
    SlotRows s;
    if (!slot_rows(c.kv, c.slots, i, A.shift, s) || s.len <= c.budget) return;
    const int t = (int)__builtin_amdgcn_workitem_id_x(), mask = (1 << A.shift) - 1, n = s.len;
    auto page_of = [&](int r) { return s.table[r >> A.shift]; };
    auto at = [&](int r) { return sum_at(A.hk, A.shift, page_of(r), h, r & mask); };

    bool bad = false;
    for (int p = t; p << A.shift < n; p += NT) bad |= s.table[p] < 0 || s.table[p] >= c.kv.n_pages;
    if (t == 0) top = INT32_MIN;
    if (__syncthreads_or(bad)) return;
    int newest = INT32_MIN;
    for (int r = t; r < n; r += NT) newest = max(newest, c.kv.pos[at(r)]);
    atomicMax(&top, newest);
    __syncthreads();
    const long long recent = (long long)top - c.recent;
    auto key = [&](int r) {
        const size_t a = at(r);
        const int p = c.kv.pos[a];
        return p < c.sink || p > recent ? 0xFFFFFFFFu : order_of(c.kv.acc[a]);
    };

    // the number of the last row to leave: `prefix` fills from the top; `need` rows of those with it leave
    unsigned prefix = 0;
    int need = n - c.budget;
    for (int bits = 24; bits >= 0; bits -= 8) {
        hist[t] = 0;
        __syncthreads();
        const unsigned above = bits == 24 ? 0u : ~0u << (bits + 8);
        for (int r = t; r < n; r += NT) {
            const unsigned k = key(r);
            if ((k & above) == prefix) atomicAdd(&hist[(k >> bits) & 255u], 1);
        }
        __syncthreads();
        if (t == 0) {
            int b = 0, left = need;
            while (left > hist[b]) left -= hist[b++];
            chosen[0] = b;
            chosen[1] = left;
        }
        __syncthreads();
        prefix |= (unsigned)chosen[0] << bits;
        need = chosen[1];
    }

    int *dst = (int *)c.ws + (size_t)id * 2 * A.most, *src = dst + A.most;
    int ties = 0, holes = 0, kept = 0;
    for (int r0 = 0; r0 < n; r0 += NT) {
        const int r = r0 + t;
        const unsigned k = r < n ? key(r) : 0xFFFFFFFFu;
        const bool tie = r < n && k == prefix;
        int all;
        const int tb = ties + count_before(tie, part, all);
        ties += all;
        const bool gone = r < n && (k < prefix || (tie && tb < need));
        const bool hole = gone && r < c.budget, keep = r < n && !gone && r >= c.budget;
        const int hb = holes + count_before(hole, part, all);
        holes += all;
        const int kb = kept + count_before(keep, part, all);
        kept += all;
        if (hole && hb < A.most) dst[hb] = r;
        if (keep && kb < A.most) src[kb] = r;
    }
    __syncthreads();
    uint4 *K = reinterpret_cast<uint4 *>(c.kv.k), *V = reinterpret_cast<uint4 *>(c.kv.v);
    for (int x = t; x < holes * A.pieces; x += NT) {
        const int m = x / A.pieces, j = x - m * A.pieces, a = src[m], b = dst[m];
        const size_t from = row_at(c.kv, page_of(a), h, a & mask) + j, to = row_at(c.kv, page_of(b), h, b & mask) + j;
        K[to] = K[from];
        V[to] = V[from];
    }
    for (int m = t; m < holes; m += NT) {
        const size_t a = at(src[m]), b = at(dst[m]);
        c.kv.acc[b] = c.kv.acc[a];
        c.kv.pos[b] = c.kv.pos[a];
    }
}

}  // namespace

namespace {

// Moves of a head at most: rows that leave before the budget, rows that stay behind it.
int most_moves(const gdnq_attn_desc &d, const gdnq_kv &kv, int budget)
{
    const int rows = kv.max_pages * d.page;
    return rows <= budget ? 0 : std::min(budget, rows - budget);
}

}  // namespace

size_t kv_evict_workspace(const gdnq_attn_desc &d, const gdnq_kv &kv, int budget, int n)
{
    return (size_t)n * d.hk * most_moves(d, kv, budget) * 8;
}

hipError_t launch_kv_evict(const gdnq_attn_desc &d, const EvictCall &c, hipStream_t st)
{
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4, per = 16 / es, most = most_moves(d, c.kv, c.budget);
    if (most == 0) return hipSuccess;   // no slot holds more than the budget
    const dim3 grid = grid_of((unsigned long long)c.n * d.hk, NT);
    EvictArgs A{c, d.hk, __builtin_ctz((unsigned)d.page), most, d.d / per, make_divisor((unsigned)d.hk), grid.x};
    A.c.kv.ldp /= per;
    A.c.kv.ldh /= per;
    A.c.kv.ldr /= per;
    hipLaunchKernelGGL(kv_evict_kernel, grid, dim3(NT), 0, st, A);
    return hipGetLastError();
}

}  // namespace gdnq
