// attn_step.hip -- the attention of one new token of each entry over its rows
// in the paged cache (gdnq_attn_step): per query head
//   s_r = scale q . k_r,  w_r = e^{s_r - m} / sum e^{s - m},  o = sum w_r v_r
// with one pass over the rows, which keeps the running maximum m, the sum and
// the output, all in fp32.
//
// Keys and values are read once, 4 d H rows operations against them: bound by
// HBM, so the kernel is made of loads in flight.  The query heads of a cache
// head are the columns of a matrix product (16 at a time, the missing ones
// repeats), so a row is read once for all of them:
//
//   S [rows x heads] = K Q^T,  then  O^T [d x heads] += V^T W^T
//
// The instruction's accumulator has a head per lane and four rows of a lane in
// its registers, which is how its second operand wants the weights if the sum
// over rows is taken in that order: the weights never leave their lane.  The
// other operand wants for one column of V eight rows in one lane: a lane loads
// 16 bytes of each of its rows and picks the columns apart with byte
// permutes, so neither K nor V goes through LDS.  In bf16 a weight is split
// into two bf16 parts, which leave 2^-17 of it (one part would leave 2^-9,
// and the matrix cores have nothing else to do); in fp32 the products are fp32.
//
// Work is dealt out in units of 4 steps (one per wave) of an entry and a cache
// head, entry after entry, in equal shares over a fixed number of workgroups,
// whatever the entries' lengths: every workgroup finds its share from all
// lengths by a prefix sum.  An entry and head inside one share is finished there;
// the pieces of the others (maximum, sum, output) go to the workspace, and a
// second kernel joins them.
//
// 64 entries of 512 to 32768 rows, 8 cache heads of 128, 4 query heads each, in
// bf16: 367 us (6.5 TB/s; a large copy reaches 4.9); one entry of 131071 rows 92
// us, 5 to 7 of them the join; 24 entries of about 15000 rows of 8 heads of 64 in
// fp32 385 us (5.9 TB/s).  Sums of weights cost their scores, which are written
// among the reads and read again: 192 entries to 2100 rows, 8 query heads each,
// 180 us instead of 126.
#include <algorithm>

#include "attn_launchers.hpp"
#include "paged.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

constexpr float LOG2E = 1.44269504f, LOWEST = -3.4028234e38f;
constexpr int NT = 256, NW = NT / 64;
constexpr int SHARES = 512;   // workgroups at most: two for each compute unit; half as many for heads of
                              // 256, whose registers leave room for one
constexpr int JOIN_HEADS = 16;     // workgroups at most that join a pair's heads
constexpr int SUM_ROWS = NT * 4;   // rows of which a workgroup adds up the weights at a time

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned long long u64;

// Where a share begins: entry, pair (cache head and up to 64 of its query heads),
// unit of the pair, and the pair's units; and the units of all entries (0: the share has
// none).
struct Start {
    int i, p, u, units;
    u64 all;
};

// The workspace's parts.
struct Space {
    Start *start;       // [shares], for the second kernel
    float *part_ml;     // [2 shares][16 tw][2]: maximum and sum of a share's first and last piece
    float *part_o;      // [2 shares][gt][D]
    u64 *before;        // [n]: units of the entries before, for the sums of weights, as are
    float *whole_ml;    // [n P][16 tw][2]
    float *scores;      // [n_pages][hk][G][page], and four more
    size_t spare;       // where these are, for rows on no page
};

struct StepArgs {
    AttnCall c;
    Space w;
    int H, hk, G;              // query heads per cache head,
    int gt, nt, P;             // per pair; pairs per cache head, per entry
    int tw;                    // groups of 16 heads in a pair, each with its own waves
    int nt16;                  // groups of 16 heads per cache head
    int shift, window;
    int shares, splits;        // 0: a wave for each pair; workgroups for the sums of an entry and cache head
    int lg;                    // log2 of the most shares
    float scale2, decay;       // scale log2(e): weights are powers of two
    bool wide_q, wide_o;
    Divisor bySplits, byHk, byGroups;
    unsigned nx;               // width of the grid, where it is not the shares
};

template <bool BF16, int D>
struct Geo {
    static constexpr int J = BF16 ? 2 : 1, ROWS = 16 * J;      // rows of a step
    static constexpr int ES = BF16 ? 2 : 4, E = 16 / ES;       // values in 16 bytes
    static constexpr int KP = D / (4 * E);                     // 16-byte pieces of a key row in a lane
    static constexpr int VW = D / 16;                          // values of a value row in a lane,
    static constexpr int VP = VW * ES > 16 ? VW * ES / 16 : 1; // in pieces
    static constexpr int VE = VW / VP;                         // of 16 bytes (8 for 64 bf16)
};

// Rows [first, len) of an entry, in steps [t0, t1) and units.
struct Entry {
    SlotRows s;
    int first, t0, t1, units;   // units 0: skipped; an entry without rows has one, without steps
};

template <int ROWS>
__device__ __forceinline__ Entry entry_of(const StepArgs &A, const SlotRows &s)
{
    Entry e{};
    e.s = s;
    e.first = A.window ? max(0, e.s.len - A.window) : 0;
    e.t0 = e.first / ROWS;
    e.t1 = (e.s.len + ROWS - 1) / ROWS;
    e.units = max(1, (e.t1 - e.t0 + NW - 1) / NW);
    return e;
}

template <int ROWS>
__device__ __forceinline__ Entry entry_of(const StepArgs &A, int i)
{
    SlotRows s;
    return slot_rows(A.c.kv, A.c.slots, i, A.shift, s) ? entry_of<ROWS>(A, s) : Entry{};
}

// `all` units in shares: one unit each, or 2^lg shares.  (A call has fewer workgroups
// than that only where its units cannot be more than these.)
struct Deal {
    u64 all;
    int lg;

    __device__ __forceinline__ bool single() const { return all <= (1ull << lg); }
    __device__ __forceinline__ int shares() const { return single() ? (int)all : 1 << lg; }
    // first unit of share b; the share that holds unit x
    __device__ __forceinline__ u64 begin(int b) const
    {
        return single() ? (u64)(unsigned)b : (all * (unsigned)b) >> lg;
    }
    __device__ __forceinline__ int holds(u64 x) const
    {
        return single() ? (int)x : (int)((((x + 1) << lg) - 1) / all);
    }
};

// Sum over the lower threads, and over all, of the workgroup.
__device__ __forceinline__ u64 sum_before(u64 x, u64 *part, u64 &all)
{
    const int t = (int)__builtin_amdgcn_workitem_id_x(), lane = t & 63;
    u64 in = x;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const u64 y = __shfl_up(in, d);
        if (lane >= d) in += y;
    }
    if (lane == 63) part[t >> 6] = in;
    __syncthreads();
    u64 before = in - x;
    all = 0;
#pragma unroll
    for (int w = 0; w < NW; w++) {
        if (w < (t >> 6)) before += part[w];
        all += part[w];
    }
    return before;
}

// The units [x, end) of a share, and where it begins.
struct Share {
    u64 x, end;
    Start at;

    __device__ __forceinline__ void bounds(int lg, int b)
    {
        const Deal d{at.all, lg};
        x = d.begin(b);
        end = d.begin(b + 1);
    }
};

// Workgroup b's share and the rows of its first entry; false: none.
template <int ROWS>
__device__ __forceinline__ bool find_share(const StepArgs &A, int b, Share &sh, Entry &e)
{
    __shared__ u64 part[NW];
    __shared__ int at[4];
    __shared__ SlotRows rows;
    const int t = (int)__builtin_amdgcn_workitem_id_x();
    const int per = (A.c.n + NT - 1) / NT, lo = min(t * per, A.c.n), hi = min(lo + per, A.c.n);
    u64 mine = 0;
#pragma unroll 4
    for (int i = lo; i < hi; i++) mine += (unsigned)entry_of<ROWS>(A, i).units;
    const u64 before = sum_before(mine, part, sh.at.all) * (unsigned)A.P;
    if (b == 0 && A.w.before) {
        u64 x = before;
        for (int i = lo; i < hi; i++) {
            A.w.before[i] = x;
            x += (u64)(unsigned)entry_of<ROWS>(A, i).units * (unsigned)A.P;
        }
    }
    sh.at.all *= (unsigned)A.P;
    mine *= (unsigned)A.P;
    if (b >= Deal{sh.at.all, A.lg}.shares()) {
        sh.at.all = 0;
        return false;
    }
    sh.bounds(A.lg, b);
    if (sh.x >= before && sh.x < before + mine) {
        int i = lo;
        u64 x = sh.x - before;
        Entry f;
        for (;; i++) {
            f = entry_of<ROWS>(A, i);
            if (x < (u64)(unsigned)f.units * (unsigned)A.P || i + 1 >= hi) break;
            x -= (u64)(unsigned)f.units * (unsigned)A.P;
        }
        const int p = (int)(x / (unsigned)f.units);
        at[0] = i;
        at[1] = p;
        at[2] = (int)(x - (u64)p * (unsigned)f.units);
        at[3] = f.units;
        rows = f.s;
    }
    __syncthreads();
    sh.at.i = __builtin_amdgcn_readfirstlane(at[0]);
    sh.at.p = __builtin_amdgcn_readfirstlane(at[1]);
    sh.at.u = __builtin_amdgcn_readfirstlane(at[2]);
    sh.at.units = __builtin_amdgcn_readfirstlane(at[3]);
    e = entry_of<ROWS>(A, rows);
    return true;
}

// Every piece of the share: f(entry number, entry, pair, first and last unit).
template <int ROWS, class F>
__device__ __forceinline__ void for_pieces(const StepArgs &A, const Share &sh, Entry e, F &&f)
{
    u64 x = sh.x;
    int i = sh.at.i, p = sh.at.p, u = sh.at.u;
    while (x < sh.end) {
        const int ue = (int)min((u64)e.units, u + (sh.end - x));
        f(i, e, p, u, ue);
        x += (unsigned)(ue - u);
        u = 0;
        if (++p == A.P && x < sh.end) {
            p = 0;
            do e = entry_of<ROWS>(A, ++i);   // units are left, so an entry with some follows
            while (e.units == 0 && i + 1 < A.c.n);
            if (e.units == 0) return;        // (unless the lengths change under the call)
        }
    }
}

__device__ __forceinline__ float across_rows_max(float x)
{
    float a = x, b = x;
    swap16(a, b);
    x = fmaxf(a, b);
    a = b = x;
    swap32(a, b);
    return fmaxf(a, b);
}

__device__ __forceinline__ float across_rows_sum(float x)
{
    float a = x, b = x;
    swap16(a, b);
    x = a + b;
    a = b = x;
    swap32(a, b);
    return a + b;
}

// A sum of weights as a divisor: of no rows, where there is nothing to divide, not 0; of others, whose largest
// weight is 1, as it is.  A NaN stays one: a comparison, compiled for arithmetic without NaN, may make it no rows.
__device__ __forceinline__ float divisor(float l) { return l + 0x1p-100f; }

// 16 bytes.  What is read once is kept out of the caches' way (64 requests to 32768
// rows 410 -> 366 us, 5.8 -> 6.5 TB/s); what several waves read (AGAIN) is not (32
// requests to 20000 rows, 64 query heads to a cache head, 145 -> 106 us).
template <bool AGAIN>
__device__ __forceinline__ uint4 read16(const char *p)
{
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
    u32x4 x;
    if constexpr (AGAIN) x = *q;
    else x = __builtin_nontemporal_load(q);
    return make_uint4(x.x, x.y, x.z, x.w);
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, (bf16x2{(__bf16)a, (__bf16)b}));
}

// One wave's steps over a piece, `stride` apart.  Lane = (head or row or column n = lane & 15, group g = lane >> 4).
template <bool BF16, int D, bool SUMS, bool WIDE>
struct Steps {
    using X = Geo<BF16, D>;
    static constexpr int J = X::J;

    const StepArgs &A;
    const Entry &e;
    int h, n, g;
    const int stride;
    size_t head;                 // of the cache, in elements
    uint4 q[X::KP], k[J][X::KP];
    uint4 v[J * 4][X::VP];       // row 16 j + 4 g + i at 4 j + i
    f32x4 o[X::VP][X::VE];
    float m, l;
    int page_k[J], page_v[J];    // of the step loaded next,
    int then_k[J], then_v[J];    // and of the one after it
    bool edge;                   // the loaded step has rows that do not count,
    bool ok[J];                  // or whose page does not exist (of this lane's rows of V and scores)
    int at_v[J];                 // (with SUMS) their pages

    __device__ __forceinline__ Steps(const StepArgs &A_, const Entry &e_, int h_, int stride_)
        : A(A_), e(e_), h(h_), stride(stride_)
    {
        const int lane = (int)(__builtin_amdgcn_workitem_id_x() & 63u);
        n = lane & 15;
        g = lane >> 4;
        head = (size_t)h * A.c.kv.ldh;
    }

    __device__ __forceinline__ const char *at(const void *base, int page, int r) const
    {
        const size_t off = (size_t)page * A.c.kv.ldp + head + (size_t)(r & ((1 << A.shift) - 1)) * A.c.kv.ldr;
        return reinterpret_cast<const char *>(base) + off * X::ES;
    }

    __device__ __forceinline__ void load_q(int i, int hq, int heads)
    {
#pragma unroll
        for (int c = 0; c < X::KP; c++) {
            const size_t off = (size_t)i * A.c.ldq + (size_t)(hq + n % heads) * D + c * 4 * X::E + g * X::E;
            if (A.wide_q) q[c] = Pack<BF16, X::E>::load(A.c.q, off);
            else {
                float x[X::E];
#pragma unroll
                for (int w = 0; w < X::E; w++) x[w] = load1<BF16>(A.c.q, off + w);
                q[c] = Pack<BF16, X::E>::narrow(x);
            }
        }
    }

    // a row's page; rows behind the last take its page
    __device__ __forceinline__ int page_of(int r) const { return e.s.table[min(r, e.s.len - 1) >> A.shift]; }

    __device__ __forceinline__ void load_pages(int t, int (&k)[J], int (&v)[J]) const
    {
#pragma unroll
        for (int j = 0; j < J; j++) {
            k[j] = page_of(t * X::ROWS + 16 * j + n);
            v[j] = page_of(t * X::ROWS + 16 * j + 4 * g);
        }
    }

    __device__ __forceinline__ bool there(int page) const { return page >= 0 && page < A.c.kv.n_pages; }

    __device__ __forceinline__ void load_k(int t)
    {
#pragma unroll
        for (int j = 0; j < J; j++) {
            const char *p = at(A.c.kv.k, there(page_k[j]) ? page_k[j] : 0, t * X::ROWS + 16 * j + n) + g * 16;
#pragma unroll
            for (int c = 0; c < X::KP; c++) k[j][c] = read16<WIDE>(p + c * 64);
        }
    }

    __device__ __forceinline__ void load_v(int t)
    {
        const int r0 = t * X::ROWS;
        bool bad = false;
#pragma unroll
        for (int j = 0; j < J; j++) {
            ok[j] = there(page_v[j]);
            bad |= !ok[j];
            at_v[j] = ok[j] ? page_v[j] : 0;
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const char *p = at(A.c.kv.v, at_v[j], r0 + 16 * j + 4 * g + i) + n * (X::VE * X::ES);
#pragma unroll
                for (int c = 0; c < X::VP; c++) {
                    if constexpr (X::VE * X::ES == 16)
                        v[4 * j + i][c] = read16<WIDE>(p + c * 256);
                    else {
                        const uint2 x = load_nt8(reinterpret_cast<const int8_t *>(p));
                        v[4 * j + i][c] = make_uint4(x.x, x.y, 0, 0);
                    }
                }
            }
        }
        edge = r0 < e.first || r0 + X::ROWS > e.s.len || __any(bad);
    }

    __device__ __forceinline__ f32x4 scores(int j) const
    {
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < X::KP; c++) {
            if constexpr (BF16)
                s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[j][c]),
                                                            __builtin_bit_cast(bf16x8, q[c]), s, 0, 0, 0);
            else {
                const f32x4 a = __builtin_bit_cast(f32x4, k[j][c]), b = __builtin_bit_cast(f32x4, q[c]);
#pragma unroll
                for (int w = 0; w < 4; w++) s = __builtin_amdgcn_mfma_f32_16x16x4f32(a[w], b[w], s, 0, 0, 0);
            }
        }
        return s;
    }

    // column w of piece c of the eight rows
    __device__ __forceinline__ bf16x8 column(int c, int w) const
    {
        uint32_t x[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint4 &a = v[2 * i][c], &b = v[2 * i + 1][c];
            const uint32_t lo = w / 2 == 0 ? a.x : w / 2 == 1 ? a.y : w / 2 == 2 ? a.z : a.w;
            const uint32_t hi = w / 2 == 0 ? b.x : w / 2 == 1 ? b.y : w / 2 == 2 ? b.z : b.w;
            x[i] = __builtin_amdgcn_perm(hi, lo, w & 1 ? 0x07060302u : 0x05040100u);
        }
        return __builtin_bit_cast(bf16x8, make_uint4(x[0], x[1], x[2], x[3]));
    }

    __device__ __forceinline__ void add_values(const float (&p)[4 * J])
    {
        if constexpr (BF16) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; i++) {
                const float a = p[2 * i], b = p[2 * i + 1];
                hi[i] = pack_bf16(a, b);
                lo[i] = pack_bf16(a - __uint_as_float(hi[i] << 16), b - __uint_as_float(hi[i] & 0xFFFF0000u));
            }
            const bf16x8 ph = __builtin_bit_cast(bf16x8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            const bf16x8 pl = __builtin_bit_cast(bf16x8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
#pragma unroll
            for (int c = 0; c < X::VP; c++)
#pragma unroll
                for (int w = 0; w < X::VE; w++) {
                    const bf16x8 col = column(c, w);
                    o[c][w] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(col, ph, o[c][w], 0, 0, 0);
                    o[c][w] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(col, pl, o[c][w], 0, 0, 0);
                }
        } else {
#pragma unroll
            for (int i = 0; i < 4; i++)
#pragma unroll
                for (int c = 0; c < X::VP; c++) {
                    const f32x4 a = __builtin_bit_cast(f32x4, v[i][c]);
#pragma unroll
                    for (int w = 0; w < X::VE; w++)
                        o[c][w] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[w], p[i], o[c][w], 0, 0, 0);
                }
        }
    }

    // Step t, which is loaded; with MORE the next is loaded meanwhile.  Loads return in order, so
    // a wait for one is a wait for those before it: the pages come before the rows, and no
    // condition stands around either (a wait would be one for all of them then).
    template <bool MORE>
    __device__ __forceinline__ void step(int t)
    {
        float s[4 * J], top = LOWEST;
        if constexpr (MORE) load_pages(t + 2 * stride, then_k, then_v);
#pragma unroll
        for (int j = 0; j < J; j++) {
            const f32x4 x = scores(j);
#pragma unroll
            for (int i = 0; i < 4; i++) s[4 * j + i] = x[i] * A.scale2;
        }
        if constexpr (MORE) load_k(t + stride);
        float4 raw[J];
        size_t to[J];
        if constexpr (SUMS) {
#pragma unroll
            for (int j = 0; j < J; j++) {
                raw[j] = make_float4(s[4 * j], s[4 * j + 1], s[4 * j + 2], s[4 * j + 3]);
                // rows before a window or behind the last may lie on pages that are another entry's by now
                const int r = t * X::ROWS + 16 * j + 4 * g, off = r & ((1 << A.shift) - 1);
                const bool mine = ok[j] && r + 3 >= e.first && r < e.s.len;
                to[j] = mine ? ((((size_t)at_v[j] * A.hk + h) * A.G + sum_head) << A.shift) + off : A.w.spare;
            }
        }
        if (edge) {
#pragma unroll
            for (int j = 0; j < J; j++)
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const int r = t * X::ROWS + 16 * j + 4 * g + i;
                    const bool in = ok[j] && r >= e.first && r < e.s.len;
                    s[4 * j + i] = in ? s[4 * j + i] : -INFINITY;
#pragma unroll
                    for (int c = 0; c < X::VP; c++) {   // whatever lies there, 0 x NaN among it
                        v[4 * j + i][c].x = in ? v[4 * j + i][c].x : 0u;
                        v[4 * j + i][c].y = in ? v[4 * j + i][c].y : 0u;
                        v[4 * j + i][c].z = in ? v[4 * j + i][c].z : 0u;
                        v[4 * j + i][c].w = in ? v[4 * j + i][c].w : 0u;
                    }
                }
        }
#pragma unroll
        for (int i = 0; i < 4 * J; i++) top = fmaxf(top, s[i]);
        const float mn = fmaxf(m, across_rows_max(top)), f = __builtin_amdgcn_exp2f(m - mn);
        m = mn;
        l *= f;
#pragma unroll
        for (int i = 0; i < 4 * J; i++) {
            s[i] = __builtin_amdgcn_exp2f(s[i] - mn);
            l += s[i];
        }
#pragma unroll
        for (int c = 0; c < X::VP; c++)
#pragma unroll
            for (int w = 0; w < X::VE; w++) o[c][w] *= f;
        add_values(s);
        if constexpr (MORE) {
            load_v(t + stride);
#pragma unroll
            for (int j = 0; j < J; j++) {
                page_k[j] = then_k[j];
                page_v[j] = then_v[j];
            }
        }
        if constexpr (SUMS) {   // behind the loads: a wait for these is none for the stores
#pragma unroll
            for (int j = 0; j < J; j++) *reinterpret_cast<float4 *>(A.w.scores + to[j]) = raw[j];
        }
    }

    // The steps from t on below `end`, for `heads` query heads from hq on (of none, nothing).
    __device__ __forceinline__ void run(int i, int hq, int heads, int t, int end)
    {
        m = LOWEST;
        l = 0.0f;
#pragma unroll
        for (int c = 0; c < X::VP; c++)
#pragma unroll
            for (int w = 0; w < X::VE; w++) o[c][w] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (t >= end || heads <= 0) return;
        sum_head = hq - h * A.G + n % heads;
        load_q(i, hq, heads);
        load_pages(t, page_k, page_v);
        load_pages(t + stride, then_k, then_v);
        load_k(t);
        load_v(t);
#pragma unroll
        for (int j = 0; j < J; j++) {
            page_k[j] = then_k[j];
            page_v[j] = then_v[j];
        }
        for (; t + stride < end; t += stride) step<true>(t);
        step<false>(t);
        l = across_rows_sum(l);
    }

    int sum_head;   // (with SUMS) the lane's head within the cache head's
};

template <bool BF16, int D, bool SUMS, bool WIDE>
__global__ __launch_bounds__(NT, D == 256 ? 1 : 2) void attn_kernel(StepArgs A)
{
    using X = Geo<BF16, D>;
    const int tw = WIDE ? A.tw : 1;
    constexpr int DC = D < 128 ? D : 128;             // columns joined at a time
    constexpr int PC = DC / (16 * X::VE);             // in pieces of a lane
    __shared__ float mj[NW][16], lj[NW][16];
    __shared__ float oj[NW][16][DC + 4];              // heads 4 banks apart
    const int t = (int)__builtin_amdgcn_workitem_id_x(), w = __builtin_amdgcn_readfirstlane(t >> 6);
    const int b = (int)__builtin_amdgcn_workgroup_id_x();
    Share sh{};
    Entry first;
    const bool some = find_share<X::ROWS>(A, b, sh, first);
    if (t == 0 && A.w.start) A.w.start[b] = sh.at;
    if (!some) return;
    u64 done = sh.x;
    for_pieces<X::ROWS>(A, sh, first, [&](int i, const Entry &e, int p, int u, int ue) {
        // wave w: every tw-th of the pair's groups of 16 heads, and of the steps those of its group's waves
        const int h = p / A.nt, first_head = (p - h * A.nt) * A.gt, heads = min(A.gt, A.G - first_head);
        const int hq = h * A.G + first_head, group = w & (tw - 1), waves = NW / tw;
        const int mine = min(16, heads - 16 * group);
        Steps<BF16, D, SUMS, WIDE> st(A, e, h, waves);
        st.run(i, hq + 16 * group, mine, e.t0 + u * NW + w / tw, min(e.t0 + ue * NW, e.t1));
        const bool whole = u == 0 && ue == e.units;
        const size_t slot = 2 * (size_t)b + (done != sh.x);
        done += (unsigned)(ue - u);
        __syncthreads();   // the last piece's sums have been read
        if (st.g == 0) {
            mj[w][st.n] = st.m;
            lj[w][st.n] = st.l;
        }
#pragma unroll
        for (int c0 = 0; c0 < X::VP; c0 += PC) {
            if (c0) __syncthreads();
            if (st.n < mine)
#pragma unroll
                for (int c = 0; c < PC; c++)
#pragma unroll
                    for (int r = 0; r < 4; r++)
#pragma unroll
                        for (int x = 0; x < X::VE; x += 4)
                            *reinterpret_cast<float4 *>(
                                &oj[w][st.n][c * 16 * X::VE + (4 * st.g + r) * X::VE + x]) =
                                make_float4(st.o[c0 + c][x][r], st.o[c0 + c][x + 1][r], st.o[c0 + c][x + 2][r],
                                            st.o[c0 + c][x + 3][r]);
            __syncthreads();
            for (int x = t; x < heads * DC; x += NT) {
                const int hd = x / DC, col = x - hd * DC, n = hd & 15;
                float M = LOWEST, L = 0.0f, y = 0.0f;
                const int k0 = WIDE ? hd >> 4 : 0;   // its group's waves
#pragma unroll
                for (int k = k0; k < NW; k += tw) M = fmaxf(M, mj[k][n]);
#pragma unroll
                for (int k = k0; k < NW; k += tw) {
                    const float f = __builtin_amdgcn_exp2f(mj[k][n] - M);
                    L = fmaf(lj[k][n], f, L);
                    y = fmaf(oj[k][n][col], f, y);
                }
                const int at = c0 / PC * DC + col;
                if (whole)
                    store1<BF16>(A.c.o, (size_t)i * A.c.ldo + (size_t)(hq + hd) * D + at, y / divisor(L));
                else
                    A.w.part_o[(slot * A.gt + hd) * D + at] = y;
                if (c0 == 0 && col == 0 && (SUMS || !whole)) {
                    float *ml = whole ? A.w.whole_ml + ((size_t)i * A.P + p) * 32 * tw : A.w.part_ml + slot * 32 * tw;
                    ml[2 * hd] = M;
                    ml[2 * hd + 1] = L;
                }
            }
        }
    });
}

// Short caches: a wave for each group of 16 heads of an entry's cache heads,
// without shares, pieces or join.
template <bool BF16, int D, bool SUMS>
__global__ __launch_bounds__(NT, D == 256 ? 1 : 2) void attn_short_kernel(StepArgs A)
{
    using X = Geo<BF16, D>;
    const int w = __builtin_amdgcn_readfirstlane((int)__builtin_amdgcn_workitem_id_x() >> 6);
    const int groups = A.hk * A.nt16;
    const unsigned id = block_id(A.nx) * NW + (unsigned)w, i = div_by(id, A.byGroups), p = id - i * (unsigned)groups;
    if (i >= (unsigned)A.c.n) return;
    const Entry e = entry_of<X::ROWS>(A, (int)i);
    if (e.units == 0) return;
    const int h = (int)p / A.nt16, group = (int)p - h * A.nt16, heads = min(16, A.G - group * 16);
    const int hq = h * A.G + group * 16;
    Steps<BF16, D, SUMS, false> st(A, e, h, 1);
    st.run((int)i, hq, heads, e.t0, e.t1);
    if (st.n >= heads) return;
    if (SUMS && st.g == 0) {
        const size_t pair = ((size_t)i * A.hk + h) * A.nt + group / A.tw;
        float *ml = A.w.whole_ml + (pair * A.tw + group % A.tw) * 32 + 2 * st.n;
        ml[0] = st.m;
        ml[1] = st.l;
    }
    const float f = 1.0f / divisor(st.l);
#pragma unroll
    for (int c = 0; c < X::VP; c++)
#pragma unroll
        for (int r = 0; r < 4; r++) {
            const size_t to = (size_t)i * A.c.ldo + (size_t)(hq + st.n) * D + (c * 16 + 4 * st.g + r) * X::VE;
            float y[X::VE];
#pragma unroll
            for (int x = 0; x < X::VE; x++) y[x] = st.o[c][x][r] * f;
            if constexpr (X::VE == X::E) {
                if (A.wide_o) {
                    store_vec<BF16, X::E>(A.c.o, to, y);
                    continue;
                }
            }
#pragma unroll
            for (int x = 0; x < X::VE; x++) store1<BF16>(A.c.o, to + x, y[x]);
        }
}

// A pair whose units begin at unit `begin`: the shares that hold pieces of it, and
// the place of a share's piece.
struct Pieces {
    int b0, b1;
    bool inside;   // it begins inside share b0

    __device__ __forceinline__ Pieces(int f, int l, bool in) : b0(f), b1(l), inside(in) {}
    __device__ __forceinline__ Pieces(const Deal &d, u64 begin, int units)
    {
        b0 = d.holds(begin);
        b1 = d.holds(begin + (unsigned)units - 1);
        inside = d.begin(b0) != begin;
    }

    __device__ __forceinline__ size_t slot(int b) const { return 2 * (size_t)b + (b == b0 && inside); }
};

// Joins the pieces of the pairs that lie in several shares: workgroups (b, first),
// for every JOIN_HEADS-th head, that of the pair which share b begins inside of, if
// no share before it does so too.
template <bool BF16, int D>
__device__ __forceinline__ void join_pieces(const StepArgs &A, const Share &sh, int b, int first)
{
    constexpr int COLS = D / 4, PARTS = NT / COLS;   // threads on four columns each
    __shared__ float f[SHARES + 1], red[2][NW];
    __shared__ float4 oj[PARTS][COLS];
    const int t = (int)__builtin_amdgcn_workitem_id_x(), col = t % COLS, part = t / COLS;
    if (b == 0 || sh.at.u == 0) return;
    const u64 begin = sh.x - (unsigned)sh.at.u;
    const Pieces pc(Deal{sh.at.all, A.lg}, begin, sh.at.units);
    if (pc.b0 != b - 1) return;
    const int h = sh.at.p / A.nt, first_head = (sh.at.p - h * A.nt) * A.gt, heads = min(A.gt, A.G - first_head);
    const int np = pc.b1 - pc.b0 + 1, stride = 32 * A.tw;
    for (int hd = first; hd < heads; hd += JOIN_HEADS) {
        const float *ml = A.w.part_ml + 2 * hd;
        if (hd != first) __syncthreads();   // the last head's sums have been read
        float M = LOWEST;
        for (int k = t; k < np; k += NT) {
            f[k] = ml[pc.slot(pc.b0 + k) * stride];
            M = fmaxf(M, f[k]);
        }
        M = fmaxf(M, __shfl_xor(M, 1));
        M = fmaxf(M, __shfl_xor(M, 2));
        M = fmaxf(M, __shfl_xor(M, 4));
        M = fmaxf(M, __shfl_xor(M, 8));
        M = across_rows_max(M);
        if ((t & 63) == 0) red[0][t >> 6] = M;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NW; k++) M = fmaxf(M, red[0][k]);
        float L = 0.0f;
        for (int k = t; k < np; k += NT) {
            f[k] = __builtin_amdgcn_exp2f(f[k] - M);
            L = fmaf(ml[pc.slot(pc.b0 + k) * stride + 1], f[k], L);
        }
        L = lanes_sum<64>(L);
        if ((t & 63) == 0) red[1][t >> 6] = L;
        __syncthreads();
        L = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
        float4 y = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
        for (int k = part; k < np; k += PARTS) {
            const float4 x =
                *reinterpret_cast<const float4 *>(A.w.part_o + (pc.slot(pc.b0 + k) * A.gt + hd) * D + 4 * col);
            y.x = fmaf(x.x, f[k], y.x);
            y.y = fmaf(x.y, f[k], y.y);
            y.z = fmaf(x.z, f[k], y.z);
            y.w = fmaf(x.w, f[k], y.w);
        }
        oj[part][col] = y;
        __syncthreads();
        if (t < COLS) {
#pragma unroll
            for (int k = 1; k < PARTS; k++) {
                const float4 x = oj[k][t];
                y.x += x.x; y.y += x.y; y.z += x.z; y.w += x.w;
            }
            const float r = 1.0f / divisor(L);
            const size_t to = (size_t)sh.at.i * A.c.ldo + (size_t)(h * A.G + first_head + hd) * D + 4 * t;
            store1<BF16>(A.c.o, to, y.x * r);
            store1<BF16>(A.c.o, to + 1, y.y * r);
            store1<BF16>(A.c.o, to + 2, y.z * r);
            store1<BF16>(A.c.o, to + 3, y.w * r);
        }
    }
}

// acc of an entry's rows in a cache head, from the stored scores and the pairs'
// maxima and sums: four rows (16 bytes, in one page) of a thread, SUM_ROWS at a
// time by one of `splits` workgroups.
template <int ROWS>
__device__ __forceinline__ void add_weights(const StepArgs &A, unsigned id)
{
    __shared__ float M[64], R[64], mj[NW][16], lj[NW][16];
    const int t = (int)__builtin_amdgcn_workitem_id_x(), n = t & 15, k0 = t >> 4;
    const unsigned ih = div_by(id, A.bySplits);
    const int which = (int)(id - ih * (unsigned)A.splits), i = (int)div_by(ih, A.byHk), h = (int)ih - i * A.hk;
    const int p = h * A.nt;
    const u64 all = A.shares ? A.w.start[0].all : 0, before = A.shares ? A.w.before[i] : 0;
    const Entry e = entry_of<ROWS>(A, i);
    if (e.units == 0) return;
    const int lo = e.t0 * ROWS, hi = e.s.len, stride = 32 * A.tw;
    bool known = false;   // M and R are the pair's
    for (int r0 = lo + which * SUM_ROWS; r0 < hi; r0 += A.splits * SUM_ROWS) {
        const int r = r0 + 4 * t, off = r & ((1 << A.shift) - 1);
        const int page = r < hi ? e.s.table[r >> A.shift] : -1;
        const bool in = page >= 0 && page < A.c.kv.n_pages;
        float w[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int tile = 0; tile < A.nt; tile++) {
            const int heads = min(A.gt, A.G - tile * A.gt);
            // eight heads at a time: of the first ones before the maximum and the sum are known
            const size_t first = in ? ((((size_t)page * A.hk + h) * A.G + tile * A.gt) << A.shift) + off : 0;
            const float *from = A.w.scores + first;
            float4 s[8];
            auto load = [&](int x0) {
#pragma unroll
                for (int x = 0; x < 8; x++)
                    if (x0 + x < heads && in)
                        s[x] = *reinterpret_cast<const float4 *>(from + ((size_t)(x0 + x) << A.shift));
            };
            load(0);
            if (A.nt > 1 || !known) {   // the pair's maximum and sum
                Pieces pc{0, 0, false};
                if (A.shares) pc = Pieces(Deal{all, A.lg}, before + (u64)(p + tile) * (unsigned)e.units, e.units);
                __syncthreads();
                if (pc.b0 == pc.b1) {
                    if (t < heads) {
                        const float *ml = A.w.whole_ml + ((size_t)i * A.P + p + tile) * stride + 2 * t;
                        M[t] = ml[0];
                        R[t] = 1.0f / divisor(ml[1]);
                    }
                } else
                    for (int g0 = 0; g0 < heads; g0 += 16) {
                        float m = LOWEST, l = 0.0f;
                        if (g0 + n < heads)
                            for (int b = pc.b0 + k0; b <= pc.b1; b += 16) {
                                const float *ml = A.w.part_ml + pc.slot(b) * stride + 2 * (g0 + n);
                                const float mn = fmaxf(m, ml[0]);
                                l = l * __builtin_amdgcn_exp2f(m - mn) + ml[1] * __builtin_amdgcn_exp2f(ml[0] - mn);
                                m = mn;
                            }
                        const float mw = across_rows_max(m);
                        const float lw = across_rows_sum(l * __builtin_amdgcn_exp2f(m - mw));
                        if ((t & 63) < 16) {
                            mj[t >> 6][n] = mw;
                            lj[t >> 6][n] = lw;
                        }
                        __syncthreads();
                        if (t < 16) {
                            float mm = mj[0][t], ll = 0.0f;
#pragma unroll
                            for (int k = 1; k < NW; k++) mm = fmaxf(mm, mj[k][t]);
#pragma unroll
                            for (int k = 0; k < NW; k++) ll = fmaf(lj[k][t], __builtin_amdgcn_exp2f(mj[k][t] - mm), ll);
                            M[g0 + t] = mm;
                            R[g0 + t] = 1.0f / divisor(ll);
                        }
                        __syncthreads();
                    }
                __syncthreads();
                known = true;
            }
            for (int x0 = 0; x0 < heads; x0 += 8) {
                if (x0) load(x0);
#pragma unroll
                for (int x = 0; x < 8; x++)
                    if (x0 + x < heads) {
                        const float m = M[x0 + x], f = R[x0 + x];
                        w[0] = fmaf(__builtin_amdgcn_exp2f(s[x].x - m), f, w[0]);
                        w[1] = fmaf(__builtin_amdgcn_exp2f(s[x].y - m), f, w[1]);
                        w[2] = fmaf(__builtin_amdgcn_exp2f(s[x].z - m), f, w[2]);
                        w[3] = fmaf(__builtin_amdgcn_exp2f(s[x].w - m), f, w[3]);
                    }
            }
        }
        if (!in) continue;
        float *acc = A.c.kv.acc + sum_at(A.hk, A.shift, page, h, off);
        if (r >= e.first && r + 4 <= e.s.len) {
            float4 a = A.decay == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *reinterpret_cast<const float4 *>(acc);
            a.x = fmaf(A.decay, a.x, w[0]);
            a.y = fmaf(A.decay, a.y, w[1]);
            a.z = fmaf(A.decay, a.z, w[2]);
            a.w = fmaf(A.decay, a.w, w[3]);
            *reinterpret_cast<float4 *>(acc) = a;
        } else
#pragma unroll
            for (int x = 0; x < 4; x++)
                if (r + x >= e.first && r + x < e.s.len)
                    acc[x] = A.decay == 0.0f ? w[x] : fmaf(A.decay, acc[x], w[x]);
    }
}

template <bool BF16, int D, bool SUMS>
__global__ __launch_bounds__(NT) void attn_join_kernel(StepArgs A)
{
    using X = Geo<BF16, D>;
    // the sums' workgroups first: they have more to do
    unsigned id = block_id(A.nx);
    if constexpr (SUMS) {
        const unsigned sums = (unsigned)A.c.n * (unsigned)A.hk * (unsigned)A.splits;
        if (id < sums) {
            add_weights<X::ROWS>(A, id);
            return;
        }
        id -= sums;
    }
    const int joins = min(A.gt, JOIN_HEADS), b = (int)(id / (unsigned)joins), first = (int)id - b * joins;
    if (b >= A.shares) return;
    Share sh{};
    sh.at = A.w.start[b];
    if (sh.at.all == 0) return;
    sh.bounds(A.lg, b);
    join_pieces<BF16, D>(A, sh, b, first);
}

size_t up16(size_t x) { return (x + 15) / 16 * 16; }

// How a call is dealt out, and its workspace.
struct Plan {
    int G, tw, gt, nt, nt16, P, lg, shares, splits;
    bool brief, join, sums;   // brief: the kernel of short caches (the workspace has room for shares
                              // all the same: it does not shrink with more entries)
    size_t start, part_ml, part_o, before, whole_ml, scores, bytes;   // offsets

    Plan(const gdnq_attn_desc &d, const gdnq_kv &kv, int n)
    {
        const int rows = d.io_dtype == GDNQ_IO_BF16 ? 32 : 16;
        G = d.H / d.hk;
        const long long held = (long long)kv.max_pages * d.page;
        const long long most = d.window ? std::min<long long>(held, d.window) : held;   // rows attended to
        const long long steps = most / rows + 2;   // one more at each end of a window
        const long long units = (steps + NW - 1) / NW;
        lg = d.d == 256 ? 8 : 9;
        static_assert(SHARES == 1 << 9, "");
        const long long cap = 1LL << lg, few = std::min(units, cap);
        nt16 = (G + 15) / 16;
        // More than 16 query heads to a cache head: two or four groups of 16 in a workgroup, which share
        // the rows in the caches, or a workgroup for each, where there are not several units for each
        // share: its piece of 64 heads is half as large as a unit (32 requests to 20000 rows, 64 heads,
        // 106 us against 156; one of 30000, 128 heads, 48 against 30).
        const bool wide = nt16 > 1 && (long long)n * d.hk * few >= 4 * cap;
        tw = !wide ? 1 : nt16 == 2 ? 2 : 4;
        gt = std::min(G, 16 * tw);
        nt = (nt16 + tw - 1) / tw;
        P = d.hk * nt;
        shares = (int)std::min(cap, (long long)n * P * few);
        join = units > 1;
        sums = kv.acc != nullptr;
        // A wave for each pair, or shares.  8 heads of 128 in bf16, us, waves and shares: one entry of
        // 128 rows 8.9 and 8.8, of 256 14.5 and 10.4; 32 entries to 256 16.3 and 14.1; 128 to 128 11.7
        // and 17.2, to 256 19.6 and 27.5, to 512 35 and 41, to 1024 66 and 62; 2000 to 64 80 and 132,
        // to 512 409 and 480.
        brief = steps - 2 <= 4 || (steps - 2 <= 16 && (long long)n * d.hk * nt16 >= 1024);
        // enough workgroups to fill the compute units, and none without rows
        const long long parts = (most + SUM_ROWS - 1) / SUM_ROWS;
        splits = (int)std::max(1LL, std::min(parts, 4096 / ((long long)n * d.hk)));
        const size_t u = (size_t)shares;
        start = 0;
        part_ml = up16(join || sums ? u * sizeof(Start) : 0);
        part_o = part_ml + (join ? u * 2 * 32 * tw * 4 : 0);
        before = part_o + up16(join ? u * 2 * gt * d.d * 4 : 0);
        whole_ml = before + up16(sums ? (size_t)n * 8 : 0);
        scores = whole_ml + (sums ? (size_t)n * P * 32 * tw * 4 : 0);
        bytes = scores + (sums ? (size_t)kv.n_pages * d.page * d.H * 4 + 16 : 0);
    }
};

}  // namespace

size_t attn_workspace(const gdnq_attn_desc &d, const gdnq_kv &kv, int n) { return Plan(d, kv, n).bytes; }

hipError_t launch_attn_step(const gdnq_attn_desc &d, const AttnCall &c, hipStream_t st)
{
    const Plan p(d, c.kv, c.n);
    char *ws = static_cast<char *>(c.ws);
    const int es = d.io_dtype == GDNQ_IO_BF16 ? 2 : 4;
    Space w{};
    const int shares = p.brief ? 0 : p.shares;
    if (shares && (p.join || p.sums)) w.start = reinterpret_cast<Start *>(ws + p.start);
    if (shares && p.join) {
        w.part_ml = reinterpret_cast<float *>(ws + p.part_ml);
        w.part_o = reinterpret_cast<float *>(ws + p.part_o);
    }
    if (p.sums) {
        if (shares) w.before = reinterpret_cast<u64 *>(ws + p.before);
        w.whole_ml = reinterpret_cast<float *>(ws + p.whole_ml);
        w.scores = reinterpret_cast<float *>(ws + p.scores);
        w.spare = (size_t)c.kv.n_pages * d.page * d.H;
    }
    const unsigned long long groups = (unsigned long long)c.n * d.hk * p.nt16;
    const dim3 waves = grid_of((groups + NW - 1) / NW, NT);
    const unsigned long long second = (p.join ? (unsigned long long)shares * std::min(p.gt, JOIN_HEADS) : 0) +
                                      (p.sums ? (unsigned long long)c.n * d.hk * p.splits : 0);
    const dim3 joins = second ? grid_of(second, NT) : dim3(0);
    StepArgs A{c, w, d.H, d.hk, p.G, p.gt, p.nt, p.P, p.tw, p.nt16, __builtin_ctz((unsigned)d.page), d.window, shares,
               p.splits, p.lg, d.scale * LOG2E, d.acc_decay, wide_rows(c.q, c.ldq, es), wide_rows(c.o, c.ldo, es),
               make_divisor((unsigned)p.splits), make_divisor((unsigned)d.hk),
               make_divisor((unsigned)(d.hk * p.nt16)), 0};
    return with_bool(d.io_dtype == GDNQ_IO_BF16, [&](auto bf) {
        return with_bool(p.sums, [&](auto sm) {
            auto go = [&](auto dd) {
                constexpr bool B = decltype(bf)::value, S = decltype(sm)::value;
                constexpr int D = decltype(dd)::value;
                if (shares && p.tw > 1)
                    hipLaunchKernelGGL((attn_kernel<B, D, S, true>), dim3((unsigned)shares), dim3(NT), 0, st, A);
                else if (shares)
                    hipLaunchKernelGGL((attn_kernel<B, D, S, false>), dim3((unsigned)shares), dim3(NT), 0, st, A);
                else {
                    A.nx = waves.x;
                    hipLaunchKernelGGL((attn_short_kernel<B, D, S>), waves, dim3(NT), 0, st, A);
                }
                A.nx = joins.x;
                if (second)
                    hipLaunchKernelGGL((attn_join_kernel<B, D, S>), joins, dim3(NT), 0, st, A);
                return hipGetLastError();
            };
            if (d.d == 64) return go(std::integral_constant<int, 64>{});
            if (d.d == 128) return go(std::integral_constant<int, 128>{});
            return go(std::integral_constant<int, 256>{});
        });
    });
}

}  // namespace gdnq
