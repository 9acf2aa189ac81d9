// ssm_prefill.hip -- the selective state space scan over packed prompts on
// the matrix cores (gdnq_ssm_prefill): per head, with
// delta = clamp(softplus(dt + bias)),
//   S <- e^{delta A} S + B (delta x)^T,   y = S^T C + D x.
// LinQuant, appendix Table 3, Mamba-2 row, in the dk x dv orientation.
//
// The recurrence unrolled over a chunk of 64 tokens, with cs_i the running
// sum of delta A inside the chunk, w_j = e^{cs_63 - cs_j} delta_j, S the state
// at the chunk's start and S' = e^{cs_63} S, takes all decays out of the
// token-by-token product:
//   Y = diag(e^{cs_i - cs_63}) (tril(C B^T) (w X) + C S') + D X,
//   S <- S' + B^T (w X).
// tril(C B^T) is the same for all heads that share B and C, so a workgroup
// forms it once, and w X serves both lines.  With exponents in base 2 and
// cs_63 > -RANGE every factor is in range; cs_63 - cs_j is summed over the
// tokens behind j, which keeps it exact where it is small.  A head whose
// chunk decays further, to -2 RANGE, counts the exponents from a whole number
// h near cs_63 / 2 instead of 0 and decays S by 2^{cs_63 - h} before and by
// 2^h after, which loses no digits; beyond that its outputs are formed from
// factors that are all at most one:
//   Y = (tril(C B^T) . e^{cs_i - cs_j} delta_j) X + diag(e^{cs_i}) C S + D X.
//
// Precision: the products run on the bf16 matrix instructions with fp32
// sums.  B, C and x are bf16, so C B^T is exact up to the sum.  The fp32
// operands of the outputs, tril(C B^T), S' and w X, are taken in two bf16
// parts (off by at most 2^-16 of an operand; by a model of one chunk 4e-6 of
// an output row in norm, where the outputs' own rounding is 1.7e-3, so that 3
// outputs in 1000 round to a neighbour; a third part would be a third more
// products).  An output's decays come from sums over a chunk of at most 160 in
// base 2, each off by up to 8 2^-24 of that.  The state's update takes w X in
// three (2^-24), so that states stay as exact as fp32 (with two they measured
// 1.7e-6 off in norm, and the call took 0.86 of the time).
//
// A wave owns 32 value columns of one head for a whole piece of a sequence: its
// state (dk x 32) stays in accumulators, which feed C S directly as the B operand
// when the contraction index is taken in the accumulators' row order (slots
// 0..3 of lane half h are rows 16t + 4h .. + 3, slots 4..7 rows 16t + 8 + 4h
// .. + 3).  x and B are read by columns with the transposing LDS read.  A
// workgroup holds up to 8 waves: HPW heads that share B and C.
//
// While chunk c is computed, the next one is prepared: its rows of B and C are
// on their way into registers in the first half (C S) and go to the other
// half of their LDS buffers before a barrier in the middle, behind which the
// waves form its tril(C B^T) and load its x; the heads' first waves form its
// decays.  x and y pass through LDS within each wave.
//
// The packed tokens are dealt out in equal shares over the compute units
// (shares() says how many), wherever that cuts a sequence: a first kernel forms
// the state and decay of each share's last piece, if its sequence goes on in
// the next, from the sequence's own start or from zero, a second runs along
// the shares of each sequence and leaves the state at every later one's start,
// and the main kernel starts from those.
#include <algorithm>
#include <cmath>

#include "layer_launchers.hpp"
#include "rows.hpp"

namespace gdnq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef short shortx4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

constexpr int CH = 64;   // tokens per chunk

// Places of the packed axis that is dealt out in shares: sequence b holds its
// tokens' places from cu[b] + PAD b on and PAD more, the price of beginning a
// sequence (a chunk and a half, and half a chunk at its end) and of many in
// one share. 9 sequences, 32731 tokens of 32 heads of 128 x 128: 372 us with
// 96, 367 with 128, 364 with 192.
constexpr long long PAD = 192;

struct SsmArgs {
    SsmCall c;
    int H, hk;
    long long len;       // places of a share at most (share_len()); 0: one share per sequence, its whole length
    unsigned ids;        // shares
    double per_chunk;    // 1 / (CH ids)
    float dt_min, dt_max;
    bool sp;
    Divisor byHB;        // head blocks per share
    // [ids][H][dk*dv] states where a share begins inside a sequence (at first
    // that of the piece before), as many where a share's last sequence begins
    // inside it and does not end there, then [ids][H] base-2 decay exponents
    float *ws;
};

__device__ __forceinline__ floatx16 mma(bf16x8 a, bf16x8 b, floatx16 c)
{
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

template <class T>
__device__ __forceinline__ T lane_of(T x, int lane)
{
    return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}

// A row of a chunk times a distance below 2^24 bytes; the masks tell the
// compiler that the 24-bit multiplier does.
__device__ __forceinline__ uint32_t row_bytes(uint32_t row, uint32_t ld) { return (row & 63u) * (ld & 0xFFFFFFu); }

// a value that is the same in every lane, in a scalar register
__device__ __forceinline__ float uniform(float x)
{
    return __int_as_float(__builtin_amdgcn_readfirstlane(__float_as_int(x)));
}

// Sum over the lanes behind this one (exclusive), and over all: shifts down
// within rows of 16 lanes, then the totals of the rows behind.
template <class T>
__device__ __forceinline__ T suffix64(T x, int lane, T &total)
{
#define GDNQ_DPP(x, ctrl) \
    __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), ctrl, 0xf, 0xf, true))
    T s = GDNQ_DPP(x, 0x101);   // row_shl:1
    s += GDNQ_DPP(s, 0x101);
    s += GDNQ_DPP(s, 0x102);
    s += GDNQ_DPP(s, 0x104);
    s += GDNQ_DPP(s, 0x108);
#undef GDNQ_DPP
    const T t = s + x;   // lane 16 r: the total of row r
    const T t3 = lane_of(t, 48), t2 = lane_of(t, 32) + t3, t1 = lane_of(t, 16) + t2;
    total = lane_of(t, 0) + t1;
    return s + (lane < 32 ? (lane < 16 ? t1 : t2) : (lane < 48 ? t3 : T(0)));
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// two values rounded to bf16 in one instruction, the first in the low half
__device__ __forceinline__ uint32_t pack2(float a, float b)
{
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((floatx2{a, b}), bf16x2));
}
__device__ __forceinline__ float low_of(uint32_t p) { return __uint_as_float(p << 16); }
__device__ __forceinline__ float high_of(uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); }

// x[0..N) as the sum of P bf16 parts, off by at most 2^-(8 P) of x
template <int P, int N>
__device__ __forceinline__ void split(float (&x)[N], uint32_t (&part)[P][N / 2])
{
#pragma unroll
    for (int p = 0; p < P; p++)
#pragma unroll
        for (int i = 0; i < N / 2; i++) {
            part[p][i] = pack2(x[2 * i], x[2 * i + 1]);
            if (p + 1 < P) {
                x[2 * i] -= low_of(part[p][i]);
                x[2 * i + 1] -= high_of(part[p][i]);
            }
        }
}

__device__ __forceinline__ bf16x8 operand(const uint32_t (&p)[4])
{
    return __builtin_bit_cast(bf16x8, (u32x4{p[0], p[1], p[2], p[3]}));
}

// Columns of a row-major LDS tile as an operand: lane (c, h) gets column c of
// rows 4h .. 4h + 3 and 8 + 4h .. + 3 behind p.  p is the lane's own address:
// row 4h + (lane % 16) / 4, column 16 (c / 16) + 4 (lane % 4).
__device__ __forceinline__ bf16x8 ld_cols(const __bf16 *p, int stride)
{
    using lds_p = __attribute__((address_space(3))) shortx4 *;
    const shortx4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(p));
    const shortx4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_p)(p + 8 * stride));
    typedef short shortx8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// 4 values at p, then 4 at p + 8: a row as an operand in the accumulators' order
__device__ __forceinline__ bf16x8 ld_rows(const __bf16 *p)
{
    const bf16x4 a = *reinterpret_cast<const bf16x4 *>(p);
    const bf16x4 b = *reinterpret_cast<const bf16x4 *>(p + 8);
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// 8 consecutive bf16 values `off` bytes behind a uniform base, in one access
// where rows are WIDE
template <bool WIDE>
__device__ __forceinline__ u32x4 ld_global8(const char *base, uint32_t off)
{
    if constexpr (WIDE) return *reinterpret_cast<const u32x4 *>(base + off);
    const uint16_t *p = reinterpret_cast<const uint16_t *>(base + off);
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 4; i++) r[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
    return r;
}

template <bool WIDE>
__device__ __forceinline__ void st_global8(char *base, uint32_t off, u32x4 v)
{
    if constexpr (WIDE) *reinterpret_cast<u32x4 *>(base + off) = v;
    else {
        uint16_t *p = reinterpret_cast<uint16_t *>(base + off);
#pragma unroll
        for (int i = 0; i < 4; i++) p[2 * i] = (uint16_t)v[i], p[2 * i + 1] = (uint16_t)(v[i] >> 16);
    }
}

// Row strides in elements.  B is read by rows (C B^T) and by columns (the
// state's update): a stride of 20 banks more than a multiple of 64 keeps the
// row reads at two lanes per bank and the column reads below that.  C is
// read by rows in 16-byte pieces (4 banks more).  A wave's x tile has rows of
// 16 banks, which its column reads cover without a pad.
template <int DK, int DV, int HPW>
struct SsmGeom {
    static constexpr int SL = DV / 32;           // waves per head
    static constexpr int NW = HPW * SL;
    static constexpr int NT = NW * 64;
    static constexpr int SB = DK + 40, SC = DK + 8, SX = 32;
    static constexpr int NB = CH * DK / 8 / NT;  // 16-byte pieces of B (and of C) per thread
    static constexpr int NBLK = DK / 32;
};

// Per-token vectors of a head in LDS: w, the outputs' row factor, and for the
// other form delta, cs, and cs as a whole number of 2^-23, modulo 2^32.
//
// Between two tokens that are close, cs_i - cs_j is small while both may be as
// far as -2^14 (64 tokens that forget everything), where fp32 sums are off by
// 2^-10.  Whole numbers add exactly: the difference is right as long as it is
// less than 2^8, off by the rounding of each token's exponent (2^-24) only.
// The sums in fp32 tell where it is not; there the factor is zero.
enum { V_W, V_F, V_D, V_CS, V_Q, V_N };
constexpr float QUANTUM = 1.0f / (1 << 23), GONE = -200.0f;   // 2^-200 is zero in fp32

// 2^(cs_i - cs_j) from the difference in fp32 and the one in whole numbers
__device__ __forceinline__ float decay_between(float far, uint32_t q)
{
    return far < GONE ? 0.0f : __builtin_amdgcn_exp2f(fminf((float)(int)q * QUANTUM, 0.0f));
}

// 2^RANGE and 2^-RANGE times any usual value, and its second bf16 part, are
// normal numbers.
constexpr float RANGE = 80.0f;
enum { NEAR, FAR, APART };   // cs_63 above -RANGE, above -2 RANGE, below

template <class G, bool STATE>
struct SsmLds {
    static constexpr int HEADS = G::NW / G::SL;
    __bf16 b[2][CH * G::SB];
    __bf16 c[STATE ? 1 : 2][STATE ? 8 : CH * G::SC];
    __bf16 x[G::NW][CH * G::SX];
    // tril(C B^T) as operands: rows 0..31 by tokens 0..15, 16..31, rows 32..63
    // by tokens 0..15, .., 48..63; each in two parts of 8 values per lane
    alignas(16) __bf16 g[STATE ? 1 : 2][STATE ? 1 : 6][2][STATE ? 8 : 64 * 8];
    static constexpr int VN = STATE ? 1 : V_N;
    alignas(16) float v[2][HEADS][VN][CH];
    float tot[2][HEADS], after[2][HEADS];   // the decay of S before the chunk's products, and (of FAR) behind them
    int mode[2][HEADS];
};

// The last of the numbers 0 .. n - 1 for which `in` holds, where it holds up to
// one and not behind (0 is taken to): a probe per lane, 64 numbers a round, in
// [0, n) whatever `in` says.
template <class In>
__device__ __forceinline__ int last_of(int n, In &&in)
{
    const int lane = (int)(__builtin_amdgcn_workitem_id_x() & 63u);
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int step = (hi - lo + 63) / 64;
        const long long p = lo + (long long)lane * step;
        bool yes = lane == 0;
        if (p < hi && lane) yes = in(p);
        const int k = __popcll(__ballot(yes));
        lo += (k - 1) * step;
        if (lo + step < hi) hi = lo + step;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

// The last sequence that begins at place `at` or before it (sequence b begins
// at cu[b] + PAD b).
__device__ __forceinline__ int seq_at(const int32_t *cu, int n, long long at)
{
    return last_of(n, [&](long long p) { return (long long)cu[p] + PAD * p <= at; });
}

// Places of a share.  The host's length deals out all T rows and n sequences;
// where rows behind the last sequence, or sequences without tokens at the end,
// pad the call, the shares are cut from the places before them (4096 tokens in
// one of 512 sequences 96 us, 380 with the host's; 2048 of 16384 rows 54, 145).
// total and before are the last two bounds, which a kernel reads first of all.
__device__ __forceinline__ long long share_len(const SsmArgs &A, int total, int before)
{
    const int n = A.c.n;
    const bool empty = n > 1 && before == total;
    if (total < 0 || total > A.c.T || (total == A.c.T && !empty)) return A.len;
    const int used = empty ? last_of(n, [&](long long p) { return A.c.cu[p] < total; }) : n - 1;
    const long long chunks = (long long)((double)(total + PAD * used) * A.per_chunk) + 1;
    return min(max(chunks, 2ll) * CH, A.len);
}

// A share: the pieces of sequences on its places of share_len(), one after another.
// STATE: only the state and decay of its last piece, if that piece's sequence
// goes on behind it.  MANY: a share may hold more than one piece; one alone
// spares the loop's registers (16384 tokens of 64 heads of 128 x 64 191 us,
// 195 with it, 300 tokens 32, 34).
template <int DK, int DV, int HPW, bool STATE, bool MANY, bool WIDE>
__global__ __launch_bounds__((SsmGeom<DK, DV, HPW>::NT)) void ssm_chunk_kernel(SsmArgs A)
{
    using G = SsmGeom<DK, DV, HPW>;
    __shared__ SsmLds<G, STATE> L;
    using Vectors = float[SsmLds<G, STATE>::VN][CH];
    const int t = (int)__builtin_amdgcn_workitem_id_x(), lane = t & 63;
    const int wv = __builtin_amdgcn_readfirstlane(t >> 6);
    const int hw = wv % HPW, slice = wv / HPW;   // a head's first wave on each SIMD
    // head blocks of a share are neighbours (and so on all XCDs: giving them
    // one XCD's numbers spread the work unevenly and was no faster)
    const unsigned g = __builtin_amdgcn_workgroup_id_x();
    const unsigned id = __builtin_amdgcn_readfirstlane(div_by(g, A.byHB));
    if (id + (STATE ? 1 : 0) >= A.ids) return;
    const int h0 = (int)(g - id * A.byHB.d) * HPW, head = h0 + hw;
    const int hb = h0 / (A.H / A.hk);
    const gdnq_ssm_io &io = A.c.io;
    const int c = lane & 31, hh = lane >> 5;
    // accumulator r of the state's block nb is row 32 nb + 8 (r/4) + 4 hh + r % 4, column 32 slice + c
    const size_t soff = (size_t)(4 * hh) * DV + slice * 32 + c;
    const int total = A.c.cu[A.c.n], before = A.c.cu[A.c.n - 1];
    const float Ah = uniform(io.A[head] * 1.44269504f), bias = uniform(io.dt_bias ? io.dt_bias[head] : 0.0f);
    const float Dh = uniform(io.D ? io.D[head] : 0.0f);
    if constexpr (!STATE) {   // the blocks above the diagonal stay zero
        for (int i = t; i < 2 * 6 * 2 * 64; i += G::NT)
            *reinterpret_cast<uint4 *>(&L.g[0][0][0][i * 8]) = make_uint4(0, 0, 0, 0);
    }
    const long long len = A.len ? share_len(A, total, before) : 0, from = len * id, to = from + len;
    const int b0 = len == 0 ? (int)id : seq_at(A.c.cu, A.c.n, STATE ? to - 1 : from);
    for (int sq = b0; sq < A.c.n; sq++) {
        if (MANY && sq > b0) {   // a bound out of range ends nothing: its sequences are skipped below
            const int at = A.c.cu[sq];
            if (at >= 0 && at <= A.c.T && at + PAD * sq >= to) return;
        }
        SeqTile q{};
        const bool is = seq_rows(A.c.cu, A.c.slots, sq, A.c.T, A.c.n_slots, q);
        // the piece's first token and the one behind its last, in the sequence
        const long long v0 = q.start + PAD * sq;
        const int t0 = len && from > v0 ? (int)min(from - v0, (long long)q.len) : 0;
        const int t1 = len ? (int)max(min(to - v0, (long long)q.len), 0ll) : q.len;
        const bool last = t1 == q.len;
        if (!is || t0 >= t1 || (STATE && last)) {
            if constexpr (MANY) continue;
            return;
        }
        const size_t row0 = (size_t)q.start + t0;
        const int ntok = t1 - t0;
        floatx16 S[G::NBLK];   // the wave's state
        float *const pool = A.c.S + ((size_t)q.slot * A.H + head) * DK * DV + soff;
        const size_t one = (size_t)A.H * DK * DV, all = A.ids * one;
        float *const mid = A.ws + id * one + (size_t)head * DK * DV + soff, *const begin = mid + all;   // if it is cut
        {
            const bool load = t0 > 0 ? !STATE : A.c.cont && A.c.cont[sq];
            const float *src = t0 > 0 ? mid : STATE || last ? pool : begin;
#pragma unroll
            for (int nb = 0; nb < G::NBLK; nb++)
#pragma unroll
                for (int r = 0; r < 16; r++) S[nb][r] = load ? src[(size_t)(32 * nb + 8 * (r / 4) + r % 4) * DV] : 0.0f;
            if (STATE && load) {   // the main kernel's last piece replaces it while the first is still to read it
#pragma unroll
                for (int nb = 0; nb < G::NBLK; nb++)
#pragma unroll
                    for (int r = 0; r < 16; r++) begin[(size_t)(32 * nb + 8 * (r / 4) + r % 4) * DV] = S[nb][r];
            }
        }
        float seglog = 0.0f;

        // the thread's 16-byte pieces of a chunk's rows, B and C dealt out over
        // the workgroup, x's 32 columns over the wave; rows behind the piece's
        // end repeat its last one, with weights of zero.  Byte offsets from the
        // chunk's first row: a row number below 64 times a distance below 2^24.
        u32x4 rb[G::NB], rc[G::NB], rx[4];
        constexpr int PK = DK / 8, RPI = G::NT / PK;   // pieces per row, rows per turn
        const int br = t / PK;
        const uint32_t bcol = (uint32_t)(hb * DK + t % PK * 8) * 2u;
        const uint32_t xcol = (uint32_t)(head * DV + slice * 32 + lane % 4 * 8) * 2u;
        // each of these advances by a chunk with every call
        const uint32_t ldb = (uint32_t)io.ldb * 2u, ldc = (uint32_t)io.ldc * 2u, ldx = (uint32_t)io.ldx * 2u,
                       ldy = (uint32_t)io.ldy * 2u, ldt = (uint32_t)io.lddt * 2u;
        const char *pb = reinterpret_cast<const char *>(io.B) + row0 * ldb;
        const char *pc = reinterpret_cast<const char *>(io.C) + row0 * ldc;
        const char *px = reinterpret_cast<const char *>(io.x) + row0 * ldx;
        const char *pt = reinterpret_cast<const char *>(io.dt) + row0 * ldt + (size_t)head * 2;
        char *py = reinterpret_cast<char *>(io.y) + row0 * ldy;
        const auto fetch = [&](int nv) {
#pragma unroll
            for (int i = 0; i < G::NB; i++) {
                const uint32_t r = (uint32_t)min(br + i * RPI, nv - 1);
                rb[i] = ld_global8<WIDE>(pb, row_bytes(r, ldb) + bcol);
                if constexpr (!STATE) rc[i] = ld_global8<WIDE>(pc, row_bytes(r, ldc) + bcol);
            }
            pb += (size_t)CH * ldb;
            pc += (size_t)CH * ldc;
        };
        const auto fetch_x = [&](int nv) {
#pragma unroll
            for (int i = 0; i < 4; i++)
                rx[i] = ld_global8<WIDE>(px, row_bytes((uint32_t)min(16 * i + lane / 4, nv - 1), ldx) + xcol);
            px += (size_t)CH * ldx;
        };
        uint32_t dt_in = 0;
        const auto fetch_dt = [&](int nv) {   // widened at its use, or it would be waited for here
            if (slice == 0) dt_in = *reinterpret_cast<const uint16_t *>(pt + row_bytes((uint32_t)min(lane, nv - 1), ldt));
            pt += (size_t)CH * ldt;
        };
        const auto stage = [&](int buf) {
#pragma unroll
            for (int i = 0; i < G::NB; i++) {
                const int r = br + i * RPI, k8 = t % PK;
                *reinterpret_cast<u32x4 *>(&L.b[buf][r * G::SB + k8 * 8]) = rb[i];
                if constexpr (!STATE) {
                    // columns of each 16 in the order 0-3, 8-11, 4-7, 12-15
                    __bf16 *d = &L.c[buf][r * G::SC + (k8 & ~1) * 8 + (k8 & 1) * 4];
                    *reinterpret_cast<uint2 *>(d) = make_uint2(rc[i][0], rc[i][1]);
                    *reinterpret_cast<uint2 *>(d + 8) = make_uint2(rc[i][2], rc[i][3]);
                }
            }
        };
        // decays of a chunk: one wave per head, one token per lane
        const auto decays = [&](uint32_t dt, int nv, int buf) {
            float d = low_of(dt) + bias;
            if (A.sp) d = softplus(d);
            d = lane < nv ? fminf(fmaxf(d, A.dt_min), A.dt_max) : 0.0f;
            // 2^-256 is zero in fp32; the bound keeps the sums over tokens that forget
            // everything from growing without end
            const float la = fmaxf(d * Ah, -256.0f);
            float tot;
            const float suf = suffix64(la, lane, tot);   // cs_63 - cs
            const int mode = STATE || tot > -RANGE ? NEAR : tot > -2.0f * RANGE ? FAR : APART;
            // a whole number, taken out of the exponents' own whole part: suf - h in
            // fp32 would lose the digits of a small suf (2^-19, 13 times fp32's rounding)
            const int h = mode == FAR ? (int)rintf(0.5f * tot) : 0;
            const float whole = rintf(suf), part = suf - whole;
            Vectors &v = L.v[buf][hw];
            v[V_W][lane] = ldexpf(__builtin_amdgcn_exp2f(part) * d, (int)whole - h);
            if constexpr (!STATE) {
                v[V_F][lane] = ldexpf(__builtin_amdgcn_exp2f(-part), h - (int)whole);   // of APART: below
                v[V_D][lane] = d;
                if (mode == APART) {
                    uint32_t qtot;
                    const uint32_t qs = suffix64((uint32_t)(int)rintf(la * (1.0f / QUANTUM)), lane, qtot);
                    v[V_F][lane] = decay_between(tot - suf, qtot - qs);
                    v[V_CS][lane] = tot - suf;
                    v[V_Q][lane] = __uint_as_float(qtot - qs);
                }
            }
            seglog += tot;
            if (lane == 0) {
                L.tot[buf][hw] = __builtin_amdgcn_exp2f(tot - (float)h);
                if constexpr (!STATE) L.after[buf][hw] = ldexpf(1.0f, h);
                L.mode[buf][hw] = mode;
            }
        };

        // tril(C B^T) of the chunk in buf: block n of the 10 blocks of 16 x 16 tokens
        // on and below the diagonal, transposed, and its way into the operands
        const int l16 = lane & 15, qd = lane >> 4;
        const auto tri_i = [](int n) { return (int)((0x3333222110ull >> (4 * n)) & 15u); };
        const auto tri_j = [](int n) { return (int)((0x3210210100ull >> (4 * n)) & 15u); };
        const auto triangle = [&](int buf, int n) {
            const __bf16 *pb = &L.b[buf][(16 * tri_j(n) + l16) * G::SB + 16 * (qd / 2) + 4 * (qd & 1)];
            const __bf16 *pc = &L.c[buf][(16 * tri_i(n) + l16) * G::SC + 8 * qd];
            floatx4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int s = 0; s < DK / 32; s++)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ld_rows(pb + 32 * s),
                                                              *reinterpret_cast<const bf16x8 *>(pc + 32 * s), acc, 0, 0, 0);
            return acc;
        };
        const auto put_triangle = [&](int buf, int n, floatx4 acc) {
            const int I = tri_i(n), J = tri_j(n);   // row 4 qd + r of the block is token j, lane l16 token i
            float m[4];
            uint32_t part[2][2];
#pragma unroll
            for (int r = 0; r < 4; r++) m[r] = I > J || 4 * qd + r <= l16 ? acc[r] : 0.0f;
            split<2, 4>(m, part);
            const int f = I < 2 ? J : 2 + J, at = ((qd & 1) * 32 + 16 * (I & 1) + l16) * 8 + 4 * (qd / 2);
#pragma unroll
            for (int p = 0; p < 2; p++)
                *reinterpret_cast<uint2 *>(&L.g[buf][f][p][at]) = make_uint2(part[p][0], part[p][1]);
        };
        const int n0 = wv;   // the wave's first block; the others follow NW apart

        fetch_dt(min(CH, ntok));
        fetch(min(CH, ntok));
        fetch_x(min(CH, ntok));
        if (MANY && sq > b0) __syncthreads();   // the buffers of the piece before are free
        if (slice == 0) decays(dt_in, min(CH, ntok), 0);
        stage(0);
        if (CH < ntok) fetch_dt(min(CH, ntok - CH));
        if constexpr (!STATE) {
            __syncthreads();
            for (int n = n0; n < 10; n += G::NW) put_triangle(0, n, triangle(0, n));
        }
        // a chunk's outputs wait in the wave's x tile until the next chunk begins:
        // there the loads of a chunk ago have long arrived, so that nothing waits for the stores
        __bf16 *const xt = L.x[wv];
        u32x4 yo[4];
        const auto load_y = [&] {
#pragma unroll
            for (int n = 0; n < 4; n++) yo[n] = *reinterpret_cast<const u32x4 *>(&xt[(64 * n + lane) * 8]);
        };
        const auto store_y = [&](int nv) {
#pragma unroll
            for (int n = 0; n < 4; n++)
                if (nv == CH || 16 * n + lane / 4 < nv)
                    st_global8<WIDE>(py, row_bytes((uint32_t)(16 * n + lane / 4), ldy) + xcol, yo[n]);
            py += (size_t)CH * ldy;
        };
        int buf = 0;
        for (int left = ntok; left > 0; left -= CH, buf ^= 1) {
            const bool more = left > CH;
            __syncthreads();   // the chunk is staged, and the previous one's buffers are free
            if constexpr (!STATE) load_y();
            wave_lds_sync();
#pragma unroll
            for (int i = 0; i < 4; i++) *reinterpret_cast<u32x4 *>(&xt[(64 * i + lane) * 8]) = rx[i];
            uint32_t dt_now = dt_in;
            asm volatile("" : "+v"(dt_now));   // arrived as well, before stores and new loads are on their way
            if (!STATE && left < ntok) store_y(CH);
            if (more) fetch(min(CH, left - CH));
            if (slice == 0 && more) decays(dt_now, min(CH, left - CH), buf ^ 1);
            wave_lds_sync();

            const int tr_r = 4 * hh + l16 / 4, tr_c = 16 * (c / 16) + 4 * (l16 & 3);
            const Vectors &vec = L.v[buf][hw];
            const float tot = uniform(L.tot[buf][hw]), after = STATE ? 1.0f : uniform(L.after[buf][hw]);
            const int mode = STATE ? NEAR : __builtin_amdgcn_readfirstlane(L.mode[buf][hw]);
            const bool apart = mode == APART;
            bf16x8 xf[4];   // x rows 16 f .. + 15, the wave's columns
#pragma unroll
            for (int f = 0; f < 4; f++)
                xf[f] = ld_cols(&xt[(16 * f + tr_r) * G::SX + tr_c], G::SX);

            const auto decay_state = [&](float by) {
#pragma unroll
                for (int nb = 0; nb < G::NBLK; nb++)
#pragma unroll
                    for (int r = 0; r < 16; r++) S[nb][r] *= by;
            };
            floatx16 Y[2];
            const auto scale_rows = [&] {   // Y rows by V_F
                float4 e[8];
#pragma unroll
                for (int k = 0; k < 8; k++) e[k] = *reinterpret_cast<const float4 *>(&vec[V_F][8 * k + 4 * hh]);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < 8; k++) {
                    floatx16 &y = Y[k / 4];
                    const int r = 4 * (k % 4);
                    y[r] *= e[k].x, y[r + 1] *= e[k].y, y[r + 2] *= e[k].z, y[r + 3] *= e[k].w;
                }
            };
            const auto output = [&] {
                // y = Y + D x to the wave's x tile; neighbouring lanes trade halves so
                // that each writes two columns of a row
                const uint32_t sel = (lane & 1) ? 0x03020706u : 0x05040100u;
                wave_lds_sync();
#pragma unroll
                for (int ib = 0; ib < 2; ib++)
#pragma unroll
                    for (int r = 0; r < 16; r += 2) {
                        const uint32_t xr = __builtin_bit_cast(u32x4, xf[2 * ib + r / 8])[r % 8 / 2];
                        const uint32_t u = pack2(fmaf(Dh, low_of(xr), Y[ib][r]), fmaf(Dh, high_of(xr), Y[ib][r + 1]));
                        const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u, DPP_XOR1, 0xF, 0xF, true);
                        const int i = 32 * ib + 8 * (r / 4) + r % 4 + 4 * hh + (lane & 1);
                        *reinterpret_cast<uint32_t *>(&xt[i * G::SX + (c & ~1)]) = __builtin_amdgcn_perm(o, u, sel);
                    }
            };
            if (!apart) decay_state(tot);
            if constexpr (!STATE) {
#pragma unroll
                for (int r = 0; r < 16; r++) Y[0][r] = Y[1][r] = 0.0f;
#pragma unroll
                for (int s = 0; s < DK / 16; s++) {
                    const bf16x8 ca = *reinterpret_cast<const bf16x8 *>(&L.c[buf][c * G::SC + 16 * s + 8 * hh]);
                    const bf16x8 cb = *reinterpret_cast<const bf16x8 *>(&L.c[buf][(32 + c) * G::SC + 16 * s + 8 * hh]);
                    float sv[8];
                    uint32_t part[2][4];
#pragma unroll
                    for (int e = 0; e < 8; e++) sv[e] = S[s / 2][8 * (s & 1) + e];
                    split<2, 8>(sv, part);
                    Y[0] = mma(ca, operand(part[0]), Y[0]);
                    Y[1] = mma(cb, operand(part[0]), Y[1]);
                    Y[0] = mma(ca, operand(part[1]), Y[0]);
                    Y[1] = mma(cb, operand(part[1]), Y[1]);
                }
                if (apart) {
                    scale_rows();
#pragma unroll
                    for (int fr = 0; fr < 6; fr++) {
                        const int ib = fr >= 2, f = ib ? fr - 2 : fr;
                        __builtin_amdgcn_sched_barrier(0);   // one operand's values at a time: registers
                        const u32x4 gh = *reinterpret_cast<const u32x4 *>(&L.g[buf][fr][0][lane * 8]);
                        const u32x4 gl = *reinterpret_cast<const u32x4 *>(&L.g[buf][fr][1][lane * 8]);
                        const float ci = vec[V_CS][32 * ib + c];
                        const uint32_t qi = __float_as_uint(vec[V_Q][32 * ib + c]);
                        float m[8];
                        uint32_t part[2][4];
#pragma unroll
                        for (int e = 0; e < 8; e++) {
                            const int j = 16 * f + 8 * (e / 4) + 4 * hh + e % 4;
                            const float gv = (e & 1) ? high_of(gh[e / 2]) + high_of(gl[e / 2])
                                                     : low_of(gh[e / 2]) + low_of(gl[e / 2]);
                            // above the diagonal gv is zero and the factor at most one
                            m[e] = gv * (vec[V_D][j] * decay_between(ci - vec[V_CS][j], qi - __float_as_uint(vec[V_Q][j])));
                        }
                        split<2, 8>(m, part);
                        Y[ib] = mma(operand(part[0]), xf[f], Y[ib]);
                        Y[ib] = mma(operand(part[1]), xf[f], Y[ib]);
                    }
                    output();
                    decay_state(tot);
                }
            }
            floatx4 tri = {};
            if constexpr (!STATE) {
                if (more) stage(buf ^ 1);
                __syncthreads();   // the next chunk is staged (if there is one: the blocks of a chunk behind the last are not used)
            }
            if (left > 2 * CH) fetch_dt(min(CH, left - 2 * CH));
            if (more) fetch_x(min(CH, left - CH));
            if constexpr (!STATE) tri = triangle(buf ^ 1, n0);
            // ---- S' + B^T (w x), and tril(C B^T) (w x) (not used of a chunk set APART)
#pragma unroll
            for (int f = 0; f < 4; f++) {
                const u32x4 xr = __builtin_bit_cast(u32x4, xf[f]);
                float wx[8];
                uint32_t part[3][4];
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const float4 w = *reinterpret_cast<const float4 *>(&vec[V_W][16 * f + 8 * k + 4 * hh]);
                    wx[4 * k] = w.x * low_of(xr[2 * k]);
                    wx[4 * k + 1] = w.y * high_of(xr[2 * k]);
                    wx[4 * k + 2] = w.z * low_of(xr[2 * k + 1]);
                    wx[4 * k + 3] = w.w * high_of(xr[2 * k + 1]);
                }
                split<3, 8>(wx, part);
                const bf16x8 xh = operand(part[0]), xm = operand(part[1]), xl = operand(part[2]);
                if constexpr (!STATE) {
#pragma unroll
                    for (int ib = f / 2; ib < 2; ib++) {
                        const int fr = ib ? 2 + f : f;
                        const bf16x8 gh = *reinterpret_cast<const bf16x8 *>(&L.g[buf][fr][0][lane * 8]);
                        const bf16x8 gl = *reinterpret_cast<const bf16x8 *>(&L.g[buf][fr][1][lane * 8]);
                        Y[ib] = mma(gh, xh, Y[ib]);
                        Y[ib] = mma(gl, xh, Y[ib]);
                        Y[ib] = mma(gh, xm, Y[ib]);
                    }
                }
#pragma unroll
                for (int nb = 0; nb < G::NBLK; nb++) {
                    const bf16x8 bt = ld_cols(&L.b[buf][(16 * f + tr_r) * G::SB + 32 * nb + tr_c], G::SB);
                    S[nb] = mma(bt, xh, S[nb]);
                    S[nb] = mma(bt, xm, S[nb]);
                    S[nb] = mma(bt, xl, S[nb]);
                }
            }
            if (STATE && more) stage(buf ^ 1);
            if constexpr (!STATE) {
                put_triangle(buf ^ 1, n0, tri);
                for (int n = n0 + G::NW; n < 10; n += G::NW) put_triangle(buf ^ 1, n, triangle(buf ^ 1, n));
            }
            if (mode == FAR) decay_state(after);
            if constexpr (!STATE)
                if (!apart) {
                    scale_rows();
                    output();
                }
        }
        if constexpr (!STATE) {
            wave_lds_sync();
            load_y();
            store_y((ntok - 1) % CH + 1);
        }
        if (STATE || last) {
            float *end = STATE ? mid + one : pool;   // STATE: in the next share's place, whose start it leads to
#pragma unroll
            for (int nb = 0; nb < G::NBLK; nb++)
#pragma unroll
                for (int r = 0; r < 16; r++) end[(size_t)(32 * nb + 8 * (r / 4) + r % 4) * DV] = S[nb][r];
        }
        if (STATE && slice == 0 && lane == 0) A.ws[2 * all + (size_t)id * A.H + head] = seglog;
        if constexpr (!MANY) return;
    }
}

// Along each sequence of several pieces: the state at every later piece's
// start, in the place of the state of the piece before.  One thread per 4
// values of a sequence, or of a share that a sequence of several pieces begins
// in (`shared`), whichever are fewer.
template <int E>
__global__ __launch_bounds__(256) void ssm_join_kernel(SsmArgs A, Divisor byPart, Divisor byH, bool shared)
{
    const unsigned g = __builtin_amdgcn_workgroup_id_x();
    const unsigned bh = div_by(g, byPart), part = g - bh * byPart.d;
    const unsigned nr = __builtin_amdgcn_readfirstlane(div_by(bh, byH)), h = bh - nr * byH.d;
    const long long len = share_len(A, A.c.cu[A.c.n], A.c.cu[A.c.n - 1]);
    const int b = shared ? seq_at(A.c.cu, A.c.n, len * (nr + 1) - 1) : (int)nr;
    SeqTile q;
    if (!seq_rows(A.c.cu, A.c.slots, b, A.c.T, A.c.n_slots, q)) return;
    const long long v0 = q.start + PAD * b;
    // the shares it is in (bounds that break the rules may put it behind the last)
    const size_t first = (size_t)(v0 / len), end = min((size_t)((v0 + q.len - 1) / len), (size_t)A.ids - 1);
    if (first >= end || (shared && first != nr)) return;
    const size_t at = (size_t)part * 256 + __builtin_amdgcn_workitem_id_x(), step = (size_t)A.H * E / 4;
    float4 *ws = reinterpret_cast<float4 *>(A.ws) + (size_t)h * (E / 4) + at;
    const float *lg = A.ws + 2 * (size_t)A.ids * A.H * E + h;
    float4 v = ws[(first + 1) * step];
    for (size_t k = first + 2; k <= end; k++) {
        const float4 l = ws[k * step];
        const float a = exp2f(lg[(k - 1) * A.H]);
        v.x = fmaf(a, v.x, l.x);
        v.y = fmaf(a, v.y, l.y);
        v.z = fmaf(a, v.z, l.z);
        v.w = fmaf(a, v.w, l.w);
        ws[k * step] = v;
    }
}

// Heads per workgroup: as many as share B and C and fit its 8 waves, a power
// of two; rows that need narrow accesses take one.  Fewer waves have nothing
// to overlap their splits with: 16384 tokens of 60 heads of 128 x 64 take 246
// us at H / hk = 6, 451 at 3; 64 heads 218 at 4, 464 at 1, 435 with y alone
// unaligned.
int heads_per_group(const gdnq_ssm_desc &d)
{
    const int per = d.hk ? d.H / d.hk : 1;
    for (int n = d.dv == 64 ? 4 : 2; n > 1; n /= 2)
        if (per % n == 0) return n;
    return 1;
}

struct Shares {
    long long len;   // SsmArgs::len
    unsigned ids;
};

// f(n) for the numbers of shares that a call may be dealt out in, growing: an
// eighth to six rounds of one workgroup per compute unit, more than one round
// only where that fills the last one better by a hundredth (by the estimate
// below a call loses 1.5% to this at most, and 1 in 100 loses any; the
// workspace is up to 6 times smaller for it).
template <class F>
void share_counts(double blocks, F &&f)
{
    double fill = 0.0;
    for (const double r : {0.125, 0.25, 0.5, 1.0, 2.0, 3.0, 4.0, 6.0}) {
        const long long n = (long long)(r * 256.0 / blocks);
        if (n < 2) continue;
        if (r >= 1.0) {
            const double x = (double)n * blocks / (r * 256.0);
            if (x <= 1.01 * fill) continue;
            fill = x;
        }
        f(n);
    }
}

long long places_of(int n, int T) { return T + PAD * (n - 1); }

// How a call is dealt out.  Up to SSM_WHOLE tokens a share is a whole sequence: the
// two other kernels cost more than they save (300 tokens of 64 heads of
// 128 x 64: 32 us; 39 when cut at 128).  Above, equal shares of the places,
// one or as many as share_counts() says, whichever has the least estimated time: 6.0 us
// a chunk and half as much again to begin in the main kernel, 3.4 us a chunk
// and one more in the states' kernel, and the joined states at 5 TB/s (dk =
// 128; with dk = 64 all three are about half).  Measured in us for half a
// round, one, two, three: 16384 tokens of 64 heads of 128 x 64 290, 194, 224,
// 257; 32731 tokens in 9 sequences of 32 heads of 128 x 128 566, 368, 404, 423;
// 32768 in 4 of 80 heads of 128 x 64 1196, 635, 634, 633; 6000 in 20 of 24
// heads 79, 63, 78, 79.  The prices are those of workgroups of 8 waves, and
// narrow rows are dealt out as wide ones are.
Shares shares(const gdnq_ssm_desc &d, int n, int T)
{
    if (T <= SSM_WHOLE) return {0, (unsigned)n};
    const double blocks = d.H / heads_per_group(d), join = (double)d.H * 128 * d.dv * 8 / 5e6;
    const long long places = places_of(n, T);
    Shares best{places, 1};
    double least = std::ceil(blocks / 256.0) * ((double)places / CH + 1.5) * 6.0;
    share_counts(blocks, [&](long long want) {
        const long long len = std::max(((places + want - 1) / want + CH - 1) / CH * CH, 2ll * CH);
        const double ids = (double)((places + len - 1) / len), chunks = (double)len / CH;
        const double us = std::ceil(ids * blocks / 256.0) * (chunks + 1.5) * 6.0 +
                          std::ceil((ids - 1.0) * blocks / 256.0) * (chunks + 1.0) * 3.4 + (ids - 1.0) * join;
        if (us < least) {
            best = {len, (unsigned)ids};
            least = us;
        }
    });
    return best;
}

}  // namespace

// Room for the most shares of any call with as many sequences and rows or
// fewer (a share has 2 CH places at least), not for this call's own number,
// which is the least of an estimate and may be larger for a shorter call.
size_t ssm_workspace(const gdnq_ssm_desc &d, int n, int T)
{
    long long most = 0;
    if (T > SSM_WHOLE) share_counts((double)(d.H / heads_per_group(d)), [&](long long want) { most = want; });
    most = std::min(most, (places_of(n, T) + 2 * CH - 1) / (2 * CH));
    return (size_t)most * (size_t)d.H * (2 * (size_t)d.dk * d.dv + 1) * 4;
}

hipError_t launch_ssm_prefill(const gdnq_ssm_desc &d, const SsmCall &c, hipStream_t st)
{
    const gdnq_ssm_io &io = c.io;
    const bool wide = wide_rows(io.x, io.ldx, 2) && wide_rows(io.B, io.ldb, 2) && wide_rows(io.C, io.ldc, 2) &&
                      wide_rows(io.y, io.ldy, 2);
    const int hk = d.hk ? d.hk : d.H, hpw = wide ? heads_per_group(d) : 1;
    const Shares sh = shares(d, c.n, c.T);
    const unsigned ids = sh.ids, blocks = (unsigned)(d.H / hpw);
    const SsmArgs A{c, d.H, hk, sh.len, ids, 1.0 / ((double)CH * ids), d.dt_min, d.dt_max,
                    (d.flags & GDNQ_SSM_SOFTPLUS) != 0, make_divisor(blocks), reinterpret_cast<float *>(c.ws)};
    return with_dims(d.dk, d.dv, [&](auto DK, auto DV) {
        const auto go = [&](auto HPW, auto WIDE) {
            using G = SsmGeom<DK.value, DV.value, HPW.value>;
            constexpr bool W = decltype(WIDE)::value;
            if (sh.len && ids > 1) {
                hipLaunchKernelGGL((ssm_chunk_kernel<DK.value, DV.value, HPW.value, true, false, W>),
                                   dim3((ids - 1) * blocks), dim3(G::NT), 0, st, A);
                constexpr unsigned parts = DK.value * DV.value / 1024;
                const unsigned nr = std::min((unsigned)c.n, ids - 1);
                hipLaunchKernelGGL((ssm_join_kernel<DK.value * DV.value>), dim3(nr * d.H * parts), dim3(256), 0, st, A,
                                   make_divisor(parts), make_divisor((unsigned)d.H), nr < (unsigned)c.n);
            }
            if (sh.len && c.n > 1)
                hipLaunchKernelGGL((ssm_chunk_kernel<DK.value, DV.value, HPW.value, false, true, W>), dim3(ids * blocks),
                                   dim3(G::NT), 0, st, A);
            else
                hipLaunchKernelGGL((ssm_chunk_kernel<DK.value, DV.value, HPW.value, false, false, W>),
                                   dim3(ids * blocks), dim3(G::NT), 0, st, A);
            return hipGetLastError();
        };
        if (!wide) return go(std::integral_constant<int, 1>{}, std::false_type{});
        if constexpr (DV.value == 64)
            if (hpw == 4) return go(std::integral_constant<int, 4>{}, std::true_type{});
        if (hpw >= 2) return go(std::integral_constant<int, 2>{}, std::true_type{});
        return go(std::integral_constant<int, 1>{}, std::true_type{});
    });
}

}  // namespace gdnq
