// kv_evict.hip -- rows of least accumulated weight leave the paged cache
// (gdnq_kv_evict).
//
// One workgroup per entry and head chooses.  The sums become whole numbers of
// the same order, the protected rows the largest, and stay in registers.  The
// range of the others is cut into 1024 parts and the rows in each counted; the
// part in which the last row to leave lies is cut again, until it leaves as a
// whole (mostly after two rounds) or holds one number, of which the lower rows
// leave.  Then the rows before the budget that leave (holes) and the rows behind
// it that stay, equally many, are numbered in order by prefix counts; the k-th
// of these moves into the k-th hole.  Sources lie behind the budget and
// destinations before it, so the moves are independent: a few of them are made
// at once, more of them by a second kernel with many workgroups for each head.
// Where one row leaves, as decoding goes on over a full cache, it is the
// smallest of all, and the last row takes its place.
#include <algorithm>

#include "attn_launchers.hpp"
#include "paged.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

constexpr int FEW = 64;   // moves that the choosing workgroup makes itself
constexpr int HELD = 1024 * 32;   // rows whose numbers a workgroup holds in registers
constexpr unsigned STAYS = 0xFFFFFFFFu;   // the number of protected rows, above all others

// A row's numbers before and behind a move.
struct Move {
    int from, to;
};

struct EvictArgs {
    EvictCall c;
    int hk, shift, most;   // moves of a head at most
    int pieces;            // 16-byte pieces of a row; ldp, ldh and ldr count such pieces here
    int *count;            // [n hk]: moves left to the second kernel
    Move *moves;           // [n hk][most]
    unsigned *keys;        // [n hk][rows of a slot]: the rows' numbers, where registers do not hold them
    int rows;
    Divisor byHk, bySplit;
    unsigned nx;
};

typedef uint32_t words __attribute__((ext_vector_type(4)));   // a 16-byte piece

// Whole numbers in the order of the sums (both zeros alike).
__device__ __forceinline__ unsigned order_of(float x)
{
    const unsigned u = __float_as_uint(x + 0.0f);
    return (int)u < 0 ? ~u : u | 0x80000000u;
}

// Piece j of a row's key and value; with the first, its sum and position.  Rows
// are read past the caches, which the old ones would only fill (8 prompts to 2048
// rows 52 us instead of 56).
__device__ __forceinline__ void move_piece(const EvictArgs &A, const int32_t *table, int h, const Move &m, int j)
{
    const int mask = (1 << A.shift) - 1, pf = table[m.from >> A.shift], pt = table[m.to >> A.shift];
    const size_t from = row_at(A.c.kv, pf, h, m.from & mask) + j, to = row_at(A.c.kv, pt, h, m.to & mask) + j;
    words *K = reinterpret_cast<words *>(A.c.kv.k), *V = reinterpret_cast<words *>(A.c.kv.v);
    const words k = __builtin_nontemporal_load(K + from), v = __builtin_nontemporal_load(V + from);
    if (j == 0) {
        const size_t sf = sum_at(A.hk, A.shift, pf, h, m.from & mask), st = sum_at(A.hk, A.shift, pt, h, m.to & mask);
        A.c.kv.acc[st] = A.c.kv.acc[sf];
        A.c.kv.pos[st] = A.c.kv.pos[sf];
    }
    K[to] = k;
    V[to] = v;
}

// Sum over the lanes up to this one.
__device__ __forceinline__ int lanes_before(int x)
{
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);    // row_shr:1
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);    // row_shr:2
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);    // row_shr:4
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);    // row_shr:8
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, true);    // row_bcast:15
    return x + __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, true);   // row_bcast:31
}

// NT threads of K rows each, four consecutive ones (16 bytes, in one page) of
// every NT * 4 rows; more rows than NT K (MANY) in several rounds, whose numbers
// go to the workspace once they are formed (2 entries of 70000 rows down to 30000
// 153 us; formed again in every pass 181).
template <int NT, int K, bool MANY>
__global__ __launch_bounds__(NT) void kv_evict_kernel(EvictArgs A)
{
    constexpr int NW = NT / 64, BITS = 10, BINS = 1 << BITS, BT = BINS / NT, Q = K / 4;
    constexpr int PARTS = Q * NW;      // waves' parts of a round, in the order of their rows
    static_assert(PARTS <= 128 && NT * K <= 65535, "two parts a lane, counts of 16 bits");
    __shared__ int hist[BINS], part[PARTS], chosen[3], top, open, last, sum;
    __shared__ unsigned least, most;
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
    // f(k) for the thread's rows k of a round, four at a time, as far as there are any
    auto each = [&](int round, auto &&f) {
        const int fours = (n - round * NT * K + 4 * NT - 1) / (4 * NT);
#pragma unroll
        for (int q = 0; q < Q; q++)
            if (q < fours)
#pragma unroll
                for (int k = 4 * q; k < 4 * q + 4; k++) f(k);
    };
    auto row = [&](int round, int k) { return ((round * Q + k / 4) * NT + t) * 4 + k % 4; };
    // the sums and positions of the thread's rows in a round; false: a page does not exist
    auto load = [&](int round) {
        bool all = true;
        each(round, [&](int g) {
            if (g % 4) return;
            const int r = row(round, g);
            int p = r < n ? s.table[r >> A.shift] : 0;
            if (p < 0 || p >= c.kv.n_pages) {
                all = false;
                p = 0;
            }
            const size_t at = sum_at(A.hk, A.shift, p, h, r & mask);
            uint4 x = make_uint4(0, 0, 0, 0);
            int4 u = make_int4(INT32_MIN, INT32_MIN, INT32_MIN, INT32_MIN);
            if (r < n) {
                x = *reinterpret_cast<const uint4 *>(c.kv.acc + at);
                u = *reinterpret_cast<const int4 *>(c.kv.pos + at);
            }
            key[g] = x.x; key[g + 1] = x.y; key[g + 2] = x.z; key[g + 3] = x.w;
            if (r + 3 >= n) {   // rows behind the last: protected (a sink is never below zero)
                if (r + 1 >= n) u.y = INT32_MIN;
                if (r + 2 >= n) u.z = INT32_MIN;
                u.w = INT32_MIN;
            }
            pos[g] = u.x; pos[g + 1] = u.y; pos[g + 2] = u.z; pos[g + 3] = u.w;
        });
        return all;
    };
    int newest = INT32_MIN;
    // the rows' numbers: rows behind the last are among the protected ones, behind them
    auto number = [&](int round) {
        each(round, [&](int k) {
            const bool stay = pos[k] < c.sink || (unsigned)newest - (unsigned)pos[k] < (unsigned)c.recent;
            key[k] = stay ? STAYS : order_of(__uint_as_float(key[k]));
        });
    };
    unsigned *const keys = MANY ? A.keys + (size_t)id * A.rows : nullptr;
    auto form = [&](int round) {
        if constexpr (MANY) {
            load(round);
            number(round);
            each(round, [&](int k) {
                if (k % 4 == 3 && row(round, k - 3) < n)
                    *reinterpret_cast<uint4 *>(keys + row(round, k - 3)) =
                        make_uint4(key[k - 3], key[k - 2], key[k - 1], key[k]);
            });
        }
    };
    auto again = [&](int round) {
        if constexpr (MANY)
            each(round, [&](int k) {
                if (k % 4) return;
                uint4 x = make_uint4(STAYS, STAYS, STAYS, STAYS);
                if (row(round, k) < n) x = *reinterpret_cast<const uint4 *>(keys + row(round, k));
                key[k] = x.x; key[k + 1] = x.y; key[k + 2] = x.z; key[k + 3] = x.w;
            });
    };

    if (t == 0) {
        top = INT32_MIN;
        least = STAYS;
        most = 0;
        open = 0;
        last = INT32_MAX;
    }
    for (int x = t; x < BINS; x += NT) hist[x] = 0;
    bool bad = false;
    for (int round = 0; round < rounds; round++) {
        bad |= !load(round);
        each(round, [&](int k) { newest = max(newest, pos[k]); });
    }
    if (__syncthreads_or(bad)) return;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) newest = max(newest, __shfl_xor(newest, d));
    if (lane == 0) atomicMax(&top, newest);
    __syncthreads();
    newest = top;
    if constexpr (!MANY) number(0);

    // the range of the rows that are not protected (hi: one more), and how many these are
    unsigned lo = STAYS, hi = 0;
    int free = 0;
    for (int round = 0; round < rounds; round++) {
        form(round);
        each(round, [&](int k) {
            lo = min(lo, key[k]);
            hi = max(hi, key[k] + 1);   // 0 of a protected row
            free += key[k] != STAYS;
        });
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        lo = min(lo, (unsigned)__shfl_xor((int)lo, d));
        hi = max(hi, (unsigned)__shfl_xor((int)hi, d));
        free += __shfl_xor(free, d);
    }
    if (lane == 0) {
        atomicMin(&least, lo);
        atomicMax(&most, hi);
        atomicAdd(&open, free);
    }
    __syncthreads();
    lo = least;
    hi = most - 1;
    free = open;

    int need = n - c.budget;
    if (need == 1) {   // the lowest row of the smallest number; the last row takes its place
        int r = INT32_MAX;
        for (int round = 0; round < rounds; round++) {
            again(round);
            each(round, [&](int k) {
                if (key[k] == lo) r = min(r, row(round, k));
            });
        }
#pragma unroll
        for (int d = 1; d < 64; d *= 2) r = min(r, __shfl_xor(r, d));
        if (lane == 0) atomicMin(&last, r);
        __syncthreads();
        r = last;
        if (r == n - 1) return;
        if (t < A.pieces) move_piece(A, s.table, h, Move{n - 1, r}, t);
        return;
    }

    // the rows below `lo` leave, and `need` of the `ties` rows of that number, the lower ones
    int ties = n - free;
    if (need > free) {   // and some of the protected ones
        need -= free;
        lo = STAYS;
    } else {
        int shift = lo == hi ? 0 : max(0, 32 - BITS - __clz((int)(hi - lo)));
        for (;;) {
            int same = 0;   // of `lo` itself, say rows that never had any weight, there may be many
            for (int round = 0; round < rounds; round++) {
                again(round);
                each(round, [&](int k) {
                    // numbers below `lo`, where there are some, are 2^24 from its other side, and shift is
                    // at most 12 then
                    const unsigned d = (key[k] - lo) >> shift;
                    same += key[k] == lo;
                    if (d < BINS && key[k] != STAYS && key[k] != lo) atomicAdd(&hist[d], 1);
                });
            }
            same = lanes_before(same);
            if (lane == 63) atomicAdd(&hist[0], same);
            __syncthreads();
            int cnt[BT], sum = 0;
#pragma unroll
            for (int x = 0; x < BT; x++) {
                cnt[x] = hist[t * BT + x];
                hist[t * BT + x] = 0;
                sum += cnt[x];
            }
            const int in = lanes_before(sum);
            if (lane == 63) part[w] = in;
            __syncthreads();
            int before = in - sum;
#pragma unroll
            for (int k = 0; k < NW; k++)
                if (k < w) before += part[k];
#pragma unroll
            for (int x = 0; x < BT; x++) {
                if (need > before && need <= before + cnt[x]) {
                    chosen[0] = t * BT + x;
                    chosen[1] = need - before;
                    chosen[2] = cnt[x];
                }
                before += cnt[x];
            }
            __syncthreads();
            lo += (unsigned)chosen[0] << shift;
            need = chosen[1];
            ties = chosen[2];
            if (ties == need) {   // all of the part
                lo += 1u << shift;
                need = ties = 0;
                break;
            }
            if (shift == 0) break;
            shift = max(0, shift - BITS);
            __syncthreads();   // before the counts and the choice of the next round
        }
    }

    // x[q]: counts (two of 16 bits) of the thread's rows of quarter q of a round, made the counts
    // of all rows of the round before them; returns those of the whole round
    auto count_before = [&](unsigned (&x)[Q]) {
        unsigned in[Q];
#pragma unroll
        for (int q = 0; q < Q; q++) {
            in[q] = (unsigned)lanes_before((int)x[q]);
            if (lane == 63) part[q * NW + w] = (int)in[q];
        }
        __syncthreads();
        if (w == 0) {
            const int a = 2 * lane < PARTS ? part[2 * lane] : 0, b = 2 * lane + 1 < PARTS ? part[2 * lane + 1] : 0;
            const int all = lanes_before(a + b);
            if (2 * lane < PARTS) part[2 * lane] = all - a - b;
            if (2 * lane + 1 < PARTS) part[2 * lane + 1] = all - b;
            if (lane == 63) sum = all;
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < Q; q++) x[q] = (unsigned)part[q * NW + w] + in[q] - x[q];
        const unsigned all = (unsigned)sum;
        __syncthreads();
        return all;
    };

    int tied = 0, moved = 0, kept = 0;
    Move *list = A.moves ? A.moves + (size_t)id * A.most : nullptr;
    // rows in order: the same numbers on both sides make a move
    auto note = [&](int x, int r, bool to) {
        if (x < FEW) (to ? few[x].to : few[x].from) = r;
        if (list && x < A.most) (to ? list[x].to : list[x].from) = r;
    };
    for (int round = 0; round < rounds; round++) {
        again(round);
        unsigned before[Q] = {}, flags[Q] = {};
        if (ties > need) {   // some of the equal ones stay: number them
            each(round, [&](int k) { before[k / 4] += key[k] == lo && row(round, k) < n; });
            const int all = (int)count_before(before);
            each(round, [&](int k) {
                if (key[k] == lo && row(round, k) < n && tied + (int)before[k / 4]++ < need) key[k] = 0;
            });
            tied += all;
#pragma unroll
            for (int q = 0; q < Q; q++) before[q] = 0;
        }
        // what is below `lo` leaves now
        each(round, [&](int k) {
            const int r = row(round, k);
            const bool gone = key[k] < lo, hole = gone && r < c.budget, keep = !gone && r >= c.budget && r < n;
            before[k / 4] += (hole ? 0x10000u : 0u) + (keep ? 1u : 0u);
            flags[k / 4] |= (hole ? 1u : 0u) << (k % 4) | (keep ? 16u : 0u) << (k % 4);
        });
        const unsigned all = count_before(before);
#pragma unroll
        for (int q = 0; q < Q; q++) {
            int hb = moved + (int)(before[q] >> 16), kb = kept + (int)(before[q] & 0xFFFFu);
            for (unsigned f = flags[q] & 15u; f; f &= f - 1) note(hb++, row(round, 4 * q) + __ffs(f) - 1, true);
            for (unsigned f = flags[q] >> 4; f; f &= f - 1) note(kb++, row(round, 4 * q) + __ffs(f) - 1, false);
        }
        moved += (int)(all >> 16);
        kept += (int)(all & 0xFFFFu);
    }
    if (moved > FEW) {
        if (t == 0) A.count[id] = moved;
        return;
    }
    __syncthreads();
    for (int x = t; x < moved * A.pieces; x += NT) {
        const int m = x / A.pieces;
        move_piece(A, s.table, h, few[m], x - m * A.pieces);
    }
}

// The moves of a head, by `split` workgroups.
__global__ __launch_bounds__(256) void kv_move_kernel(EvictArgs A)
{
    const unsigned id = block_id(A.nx), pair = div_by(id, A.bySplit), part = id - pair * A.bySplit.d;
    if (pair >= (unsigned)A.c.n * (unsigned)A.hk) return;
    const int t = (int)__builtin_amdgcn_workitem_id_x(), count = A.count[pair];
    const int i = (int)div_by(pair, A.byHk), h = (int)(pair - (unsigned)i * (unsigned)A.hk);
    SlotRows s;
    if (count == 0 || !slot_rows(A.c.kv, A.c.slots, i, A.shift, s)) return;
    const Move *list = A.moves + (size_t)pair * A.most;
    const int rows = 256 / A.pieces, j = t % A.pieces, step = rows * (int)A.bySplit.d;
    for (int m = (int)part * rows + t / A.pieces; m < count; m += step) move_piece(A, s.table, h, list[m], j);
}

// Moves of a head at most: rows that leave before the budget, rows that stay behind it.
int most_moves(const gdnq_attn_desc &d, const gdnq_kv &kv, int budget)
{
    const int rows = kv.max_pages * d.page;
    return rows <= budget ? 0 : std::min(budget, rows - budget);
}

size_t up16(size_t x) { return (x + 15) / 16 * 16; }

// The moves' part of the workspace, behind which the numbers are.
size_t moves_bytes(size_t heads, size_t most)
{
    return most <= FEW ? 0 : up16(heads * 4) + up16(heads * most * sizeof(Move));
}

}  // namespace

size_t kv_evict_workspace(const gdnq_attn_desc &d, const gdnq_kv &kv, int budget, int n)
{
    const size_t heads = (size_t)n * d.hk, rows = (size_t)kv.max_pages * d.page;
    const size_t most = (size_t)most_moves(d, kv, budget);
    return most == 0 ? 0 : moves_bytes(heads, most) + (rows > HELD ? heads * rows * 4 : 0);
}

hipError_t launch_kv_evict(const gdnq_attn_desc &d, const EvictCall &c, hipStream_t st)
{
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4, per = 16 / es, most = most_moves(d, c.kv, c.budget);
    if (most == 0) return hipSuccess;   // no slot holds more than the budget
    const unsigned long long heads = (unsigned long long)c.n * d.hk;
    const int rows = c.kv.max_pages * d.page;
    EvictArgs A{c, d.hk, __builtin_ctz((unsigned)d.page), most, d.d / per, nullptr, nullptr, nullptr, rows,
                make_divisor((unsigned)d.hk), {}, 0};
    A.c.kv.ldp /= per;
    A.c.kv.ldh /= per;
    A.c.kv.ldr /= per;
    if (most > FEW) {
        A.count = static_cast<int *>(c.ws);
        A.moves = reinterpret_cast<Move *>(static_cast<char *>(c.ws) + up16(heads * 4));
    }
    if (rows > HELD)
        A.keys = reinterpret_cast<unsigned *>(static_cast<char *>(c.ws) + moves_bytes(heads, (size_t)most));
    auto choose = [&](auto nt, auto k, auto many) {
        constexpr int NT = decltype(nt)::value;
        const dim3 grid = grid_of(heads, NT);
        A.nx = grid.x;
        hipLaunchKernelGGL((kv_evict_kernel<NT, decltype(k)::value, decltype(many)::value>), grid, dim3(NT), 0, st, A);
    };
    using std::integral_constant;
    if (rows <= 256 * 16) choose(integral_constant<int, 256>{}, integral_constant<int, 16>{}, std::false_type{});
    else if (rows <= 1024 * 16) choose(integral_constant<int, 1024>{}, integral_constant<int, 16>{}, std::false_type{});
    // 24 rows of a thread are what its registers hold; with 32, 15 of them go to memory (8 prompts of up to
    // 20000 rows 51 and 53 us), which is still less than to form the numbers again
    else if (rows <= 1024 * 24) choose(integral_constant<int, 1024>{}, integral_constant<int, 24>{}, std::false_type{});
    else if (rows <= HELD) choose(integral_constant<int, 1024>{}, integral_constant<int, 32>{}, std::false_type{});
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
