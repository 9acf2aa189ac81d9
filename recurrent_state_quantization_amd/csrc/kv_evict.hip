// kv_evict.hip -- rows of least accumulated weight leave the paged cache
// (gdnq_kv_evict).
//
// One workgroup per entry and head chooses.  The sums become whole numbers of
// the same order, the protected rows the largest, and stay in registers; four
// rounds of counting by 8 bits find the largest number that leaves, and how
// many rows of that number leave (the lower ones).  Then the rows before the
// budget that leave (holes) and the rows behind it that stay, equally many, are
// numbered in order by prefix counts; the k-th of these moves into the k-th
// hole.  Sources lie behind the budget and destinations before it, so the moves
// are independent: a few of them are made at once, more of them by a second
// kernel with many workgroups for each head.
#include <algorithm>

#include "attn_launchers.hpp"
#include "paged.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

constexpr int FEW = 64;   // moves that the choosing workgroup makes itself

// A row's page and its place in it, before and behind a move.
struct Move {
    int from, from_off, to, to_off;
};

struct EvictArgs {
    EvictCall c;
    int hk, shift, most;   // moves of a head at most
    int pieces;            // 16-byte pieces of a row; ldp, ldh and ldr count such pieces here
    int *count;            // [n hk]: moves left to the second kernel
    Move *moves;           // [n hk][most]
    Divisor byHk, bySplit;
    unsigned nx;
};

// Whole numbers in the order of the sums (both zeros alike).
__device__ __forceinline__ unsigned order_of(float x)
{
    const unsigned u = __float_as_uint(x + 0.0f);
    return (int)u < 0 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ void move_sums(const EvictArgs &A, int h, const Move &m)
{
    const size_t from = sum_at(A.hk, A.shift, m.from, h, m.from_off), to = sum_at(A.hk, A.shift, m.to, h, m.to_off);
    A.c.kv.acc[to] = A.c.kv.acc[from];
    A.c.kv.pos[to] = A.c.kv.pos[from];
}

__device__ __forceinline__ void move_piece(const EvictArgs &A, int h, const Move &m, int j)
{
    const size_t from = row_at(A.c.kv, m.from, h, m.from_off) + j, to = row_at(A.c.kv, m.to, h, m.to_off) + j;
    uint4 *K = reinterpret_cast<uint4 *>(A.c.kv.k), *V = reinterpret_cast<uint4 *>(A.c.kv.v);
    const uint4 k = K[from], v = V[from];
    K[to] = k;
    V[to] = v;
}

// NT threads of K consecutive rows each; more rows than that (MANY) in several
// rounds, whose numbers are formed again in every pass.
template <int NT, int K, bool MANY>
__global__ __launch_bounds__(NT) void kv_evict_kernel(EvictArgs A)
{
    constexpr int NW = NT / 64, COPIES = NW < 4 ? NW : 4;
    __shared__ int hist[COPIES][256];
    __shared__ unsigned long long part[NW];
    __shared__ int chosen[3], top;
    __shared__ Move few[FEW];
    const EvictCall &c = A.c;
    const unsigned id = block_id(A.nx);
    const int i = (int)div_by(id, A.byHk), h = (int)(id - (unsigned)i * (unsigned)A.hk);
    if (i >= c.n) return;
    const int t = (int)__builtin_amdgcn_workitem_id_x(), lane = t & 63, w = t >> 6, mask = (1 << A.shift) - 1;
    if (t == 0 && A.count) A.count[id] = 0;
    SlotRows s;
    if (!slot_rows(c.kv, c.slots, i, A.shift, s) || s.len <= c.budget) return;
    const int n = s.len, rounds = MANY ? (n + NT * K - 1) / (NT * K) : 1;

    unsigned key[K];
    int pos[K];
    // the sums and positions of the thread's rows in a round; false: a page does not exist
    auto load = [&](int round) {
        const int r0 = (round * NT + t) * K;
        bool all = true;
#pragma unroll
        for (int g = 0; g < K; g += 8) {   // eight rows lie in one page
            const int r = r0 + g;
            int p = r < n ? s.table[r >> A.shift] : 0;
            if (p < 0 || p >= c.kv.n_pages) {
                all = false;
                p = 0;
            }
            const size_t at = sum_at(A.hk, A.shift, p, h, r & mask);
            const uint4 *a = reinterpret_cast<const uint4 *>(c.kv.acc + at);
            const int4 *q = reinterpret_cast<const int4 *>(c.kv.pos + at);
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            int4 u = make_int4(INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN), v = u;
            if (r < n) {
                x = a[0];
                y = a[1];
                u = q[0];
                v = q[1];
            }
            key[g] = x.x; key[g + 1] = x.y; key[g + 2] = x.z; key[g + 3] = x.w;
            key[g + 4] = y.x; key[g + 5] = y.y; key[g + 6] = y.z; key[g + 7] = y.w;
            pos[g] = u.x; pos[g + 1] = u.y; pos[g + 2] = u.z; pos[g + 3] = u.w;
            pos[g + 4] = v.x; pos[g + 5] = v.y; pos[g + 6] = v.z; pos[g + 7] = v.w;
        }
        return all;
    };
    long long recent = 0;
    // their numbers; rows behind the last are the largest and come behind the protected ones
    auto number = [&](int round) {
        const int r0 = (round * NT + t) * K;
#pragma unroll
        for (int k = 0; k < K; k++) {
            const bool stay = pos[k] < c.sink || pos[k] > recent || r0 + k >= n;
            key[k] = stay ? 0xFFFFFFFFu : order_of(__uint_as_float(key[k]));
        }
    };
    auto again = [&](int round) {
        if constexpr (MANY) {
            load(round);
            number(round);
        }
    };

    if (t == 0) top = INT32_MIN;
    for (int x = t; x < COPIES * 256; x += NT) (&hist[0][0])[x] = 0;
    int newest = INT32_MIN;
    bool bad = false;
    for (int round = 0; round < rounds; round++) {
        bad |= !load(round);
#pragma unroll
        for (int k = 0; k < K; k++)
            if ((round * NT + t) * K + k < n) newest = max(newest, pos[k]);
    }
    if (__syncthreads_or(bad)) return;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) newest = max(newest, __shfl_xor(newest, d));
    if (lane == 0) atomicMax(&top, newest);
    __syncthreads();
    recent = (long long)top - c.recent;
    number(0);

    // the number of the last row to leave: `prefix` fills from the top; `need` rows of those with it leave
    unsigned prefix = 0;
    int need = n - c.budget, ties = 0;
    for (int bits = 24; bits >= 0; bits -= 8) {
        const unsigned above = bits == 24 ? 0u : ~0u << (bits + 8);
        for (int round = 0; round < rounds; round++) {
            again(round);
#pragma unroll
            for (int k = 0; k < K; k++) {
                const bool in = (key[k] & above) == prefix;
                const int digit = (int)((key[k] >> bits) & 255u);
                // sums are alike: lanes of one digit count together
                const unsigned long long b = __ballot(in);
                if (b == 0) continue;
                const int d0 = __builtin_amdgcn_readlane(digit, (int)__ffsll((long long)b) - 1);
                const unsigned long long same = __ballot(in && digit == d0);
                if (lane == 0) atomicAdd(&hist[w % COPIES][d0], __popcll(same));
                if (in && digit != d0) atomicAdd(&hist[w % COPIES][digit], 1);
            }
        }
        __syncthreads();
        if (w == 0) {   // four digits a lane
            int cnt[4], sum = 0;
#pragma unroll
            for (int x = 0; x < 4; x++) {
                cnt[x] = 0;
#pragma unroll
                for (int y = 0; y < COPIES; y++) {
                    cnt[x] += hist[y][4 * lane + x];
                    hist[y][4 * lane + x] = 0;
                }
                sum += cnt[x];
            }
            int before = sum;
#pragma unroll
            for (int d = 1; d < 64; d *= 2) {
                const int y = __shfl_up(before, d);
                if (lane >= d) before += y;
            }
            before -= sum;
#pragma unroll
            for (int x = 0; x < 4; x++) {
                if (need > before && need <= before + cnt[x]) {
                    chosen[0] = 4 * lane + x;
                    chosen[1] = need - before;
                    chosen[2] = cnt[x];
                }
                before += cnt[x];
            }
        }
        __syncthreads();
        prefix |= (unsigned)chosen[0] << bits;
        need = chosen[1];
        ties = chosen[2];
        __syncthreads();
    }

    // sums over the lower threads, and over all
    auto sum_before = [&](unsigned long long x, unsigned long long &all) {
        unsigned long long in = x;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const unsigned long long y = __shfl_up(in, d);
            if (lane >= d) in += y;
        }
        if (lane == 63) part[w] = in;
        __syncthreads();
        unsigned long long before = in - x;
        all = 0;
#pragma unroll
        for (int k = 0; k < NW; k++) {
            if (k < w) before += part[k];
            all += part[k];
        }
        __syncthreads();
        return before;
    };

    int tied = 0, moved = 0, kept = 0;
    Move *list = A.moves ? A.moves + (size_t)id * A.most : nullptr;
    for (int round = 0; round < rounds; round++) {
        again(round);
        const int r0 = (round * NT + t) * K;
        int tb = 0;
        unsigned long long all;
        if (ties > need) {   // some of the equal ones stay: number them
            int mine = 0;
#pragma unroll
            for (int k = 0; k < K; k++) mine += key[k] == prefix && r0 + k < n;
            tb = tied + (int)sum_before((unsigned)mine, all);
            tied += (int)all;
        }
        unsigned gone = 0, in = 0;   // flags of the thread's rows
        static_assert(K <= 32, "a flag for each row of a thread");
#pragma unroll
        for (int k = 0; k < K; k++) {
            const bool tie = key[k] == prefix && r0 + k < n;
            if (key[k] < prefix || (tie && (ties <= need || tb < need))) gone |= 1u << k;
            tb += tie;
            if (r0 + k < n) in |= 1u << k;
        }
        const unsigned front = r0 >= c.budget ? 0u : c.budget - r0 >= 32 ? ~0u : (1u << (c.budget - r0)) - 1;
        const unsigned holes = gone & front, keeps = in & ~gone & ~front;
        const unsigned long long b =
            sum_before((unsigned long long)__popc(holes) << 32 | (unsigned)__popc(keeps), all);
        int hb = moved + (int)(b >> 32), kb = kept + (int)(unsigned)b;
        moved += (int)(all >> 32);
        kept += (int)(unsigned)all;
        // rows in order: the same numbers on both sides make a move
        auto note = [&](int x, int r, bool to) {
            if (x >= A.most) return;
            const int p = s.table[r >> A.shift];
            if (x < FEW) {
                (to ? few[x].to : few[x].from) = p;
                (to ? few[x].to_off : few[x].from_off) = r & mask;
            }
            if (list) {
                (to ? list[x].to : list[x].from) = p;
                (to ? list[x].to_off : list[x].from_off) = r & mask;
            }
        };
        for (unsigned f = holes; f; f &= f - 1) note(hb++, r0 + __ffs(f) - 1, true);
        for (unsigned f = keeps; f; f &= f - 1) note(kb++, r0 + __ffs(f) - 1, false);
    }
    if (moved > FEW) {
        if (t == 0) A.count[id] = moved;
        return;
    }
    __syncthreads();
    for (int x = t; x < moved * A.pieces; x += NT) {
        const int m = x / A.pieces;
        move_piece(A, h, few[m], x - m * A.pieces);
    }
    if (t < moved) move_sums(A, h, few[t]);
}

// The moves of a head, by `split` workgroups.
__global__ __launch_bounds__(256) void kv_move_kernel(EvictArgs A)
{
    const unsigned id = block_id(A.nx), pair = div_by(id, A.bySplit), part = id - pair * A.bySplit.d;
    if (pair >= (unsigned)A.c.n * (unsigned)A.hk) return;
    const int t = (int)__builtin_amdgcn_workitem_id_x(), count = A.count[pair];
    const int h = (int)(pair - div_by(pair, A.byHk) * (unsigned)A.hk);
    const Move *list = A.moves + (size_t)pair * A.most;
    const int rows = 256 / A.pieces, j = t % A.pieces, step = rows * (int)A.bySplit.d;
    for (int m = (int)part * rows + t / A.pieces; m < count; m += step) {
        const Move x = list[m];
        move_piece(A, h, x, j);
        if (j == 0) move_sums(A, h, x);
    }
}

// Moves of a head at most: rows that leave before the budget, rows that stay behind it.
int most_moves(const gdnq_attn_desc &d, const gdnq_kv &kv, int budget)
{
    const int rows = kv.max_pages * d.page;
    return rows <= budget ? 0 : std::min(budget, rows - budget);
}

size_t up16(size_t x) { return (x + 15) / 16 * 16; }

}  // namespace

size_t kv_evict_workspace(const gdnq_attn_desc &d, const gdnq_kv &kv, int budget, int n)
{
    const size_t heads = (size_t)n * d.hk, most = (size_t)most_moves(d, kv, budget);
    return most <= FEW ? 0 : up16(heads * 4) + heads * most * sizeof(Move);
}

hipError_t launch_kv_evict(const gdnq_attn_desc &d, const EvictCall &c, hipStream_t st)
{
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4, per = 16 / es, most = most_moves(d, c.kv, c.budget);
    if (most == 0) return hipSuccess;   // no slot holds more than the budget
    const unsigned long long heads = (unsigned long long)c.n * d.hk;
    const int rows = c.kv.max_pages * d.page;
    EvictArgs A{c, d.hk, __builtin_ctz((unsigned)d.page), most, d.d / per, nullptr, nullptr,
                make_divisor((unsigned)d.hk), {}, 0};
    A.c.kv.ldp /= per;
    A.c.kv.ldh /= per;
    A.c.kv.ldr /= per;
    if (most > FEW) {
        A.count = static_cast<int *>(c.ws);
        A.moves = reinterpret_cast<Move *>(static_cast<char *>(c.ws) + up16(heads * 4));
    }
    auto choose = [&](auto nt, auto k, auto many) {
        constexpr int NT = decltype(nt)::value;
        const dim3 grid = grid_of(heads, NT);
        A.nx = grid.x;
        hipLaunchKernelGGL((kv_evict_kernel<NT, decltype(k)::value, decltype(many)::value>), grid, dim3(NT), 0, st, A);
    };
    using std::integral_constant;
    if (rows <= 256 * 16) choose(integral_constant<int, 256>{}, integral_constant<int, 16>{}, std::false_type{});
    else if (rows <= 1024 * 16) choose(integral_constant<int, 1024>{}, integral_constant<int, 16>{}, std::false_type{});
    else if (rows <= 1024 * 32) choose(integral_constant<int, 1024>{}, integral_constant<int, 32>{}, std::false_type{});
    else choose(integral_constant<int, 1024>{}, integral_constant<int, 16>{}, std::true_type{});
    if (most > FEW) {
        const int at_once = 256 / A.pieces;
        const unsigned long long split =
            std::min<unsigned long long>((most + at_once - 1) / at_once, std::max(1ull, 4096 / heads));
        A.bySplit = make_divisor((unsigned)split);
        const dim3 grid = grid_of(heads * split, 256);
        A.nx = grid.x;
        hipLaunchKernelGGL(kv_move_kernel, grid, dim3(256), 0, st, A);
    }
    return hipGetLastError();
}

}  // namespace gdnq
