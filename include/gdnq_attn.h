/*
 * gdnq_attn.h -- the operators of the softmax attention layer that hybrid
 * models keep beside their recurrent ones, around its paged cache of keys and
 * values, for AMD Instinct MI355X (gfx950), in the same library as gdnq.h:
 *
 *  - rotary positions of query and key rows, and their gradient (gdnq_rope,
 *    with the frequencies of gdnq_rope_table);
 *  - storing new tokens in the cache, with their rotary positions, for packed
 *    prompts and single tokens (gdnq_kv_append);
 *  - the attention of one new token of each entry over its rows in the cache
 *    (gdnq_attn_step), which can sum up the weights that every row received;
 *  - eviction: the rows of least accumulated weight leave the cache, head by
 *    head (gdnq_kv_evict).
 *
 * The conventions of gdnq.h and of gdnq_layer.h hold: token tensors (x, q, k,
 * v, o) are rows one token each, ld* elements apart (0: their length), with
 * their element's alignment only; per-entry arrays, tables and workspaces are
 * contiguous and 16-byte aligned; nothing written may overlap anything else of
 * the call; packed sequences and slots work as there.  In bf16, products are
 * formed from the values as they are, sums, softmax statistics and weights in
 * fp32, and each output is rounded once.
 */
#ifndef GDNQ_ATTN_H
#define GDNQ_ATTN_H

#include "gdnq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* --------------------------------------------------- rotary positions */
#define GDNQ_ROPE_INTERLEAVED 1u /* pairs (2i, 2i+1); else (i, i + rot/2)        */
#define GDNQ_ROPE_INVERSE 2u     /* turn the other way: the gradient of the call
                                    without it                                   */

typedef struct {
    int32_t d;        /* values per head, even, 2..1024                          */
    int32_t rot;      /* the first rot values of a head turn, the others are
                         copied: even, 2..d (0 means d)                          */
    int32_t io_dtype; /* GDNQ_IO_F32 or GDNQ_IO_BF16 for x and y                 */
    uint32_t flags;
    float amp;        /* factor of the turned values, > 0 (1; the attention
                         factor of scaled contexts)                              */
} gdnq_rope_desc;

/* How the angles per position theta_i = base^(-2i/rot) of the pairs i < rot/2
   are scaled for long contexts; n_i = orig_len theta_i / 2 pi is the number of
   turns of a pair over the contexts that the model was trained on. */
enum {
    GDNQ_ROPE_PLAIN = 0,      /* theta_i                                         */
    GDNQ_ROPE_LINEAR = 1,     /* theta_i / factor                                */
    GDNQ_ROPE_BASE = 2,       /* base factor^(rot/(rot-2)) as the base: the last
                                 pair is slower by factor, the first as it was   */
    GDNQ_ROPE_RAMP_TURNS = 3, /* g_i theta_i + (1-g_i) theta_i / factor with
                                 g_i = (n_i - lo) / (hi - lo), within [0, 1]     */
    GDNQ_ROPE_RAMP_INDEX = 4  /* the same with 1 - g_i = (i - i0) / (i1 - i0)
                                 within [0, 1], where i(n) = rot/2
                                 ln(orig_len / (2 pi n)) / ln(base), i0 =
                                 max(floor(i(hi)), 0), i1 = min(ceil(i(lo)),
                                 rot-1) (i0 + 0.001 where that is i0)            */
};

typedef struct {
    int32_t kind;
    double base;            /* > 1                                               */
    double factor;          /* > 0; kinds other than GDNQ_ROPE_PLAIN             */
    double orig_len;        /* > 0; the ramps                                    */
    double lo, hi;          /* 0 < lo < hi; the ramps                            */
    const double *divisors; /* host [rot/2], each > 0: every theta_i is divided by
                               its own, after the above; or NULL                 */
} gdnq_rope_freqs;

/*
 * The frequencies as the calls below take them: table is HOST memory of rot/2
 * values, to be copied to the device once.  table[i] = theta_i / 2 pi in units
 * of 2^-64 turns (modulo one turn, which whole positions do not see), so that
 * the product with a position modulo 2^64 is the angle, without a rounding that
 * grows with the position.
 */
int gdnq_rope_table(const gdnq_rope_desc *desc, const gdnq_rope_freqs *freqs, uint64_t *table);

/*
 * Every head of every row by its row's position:
 *   (y_a, y_b) = amp (x_a cos t - x_b sin t, x_b cos t + x_a sin t),
 *   t = pos theta_i, for the head's pairs (a, b); the values from rot on are
 *   copied.  With GDNQ_ROPE_INVERSE t is -pos theta_i.
 *   table  device uint64 [rot/2];  pos  device int32 [rows] (any value)
 *   x      device io_dtype [rows, H*d]; y likewise, or x itself (with the same
 *          row distance).  The query and key heads of a fused projection are
 *          adjacent columns: one call turns both.
 * rows == 0 is a no-op.
 */
int gdnq_rope(const gdnq_rope_desc *desc, const uint64_t *table, const void *x, int64_t ldx, int32_t H,
              const int32_t *pos, void *y, int64_t ldy, int32_t rows, void *stream);

/* ---------------------------------------------------------- the cache */
typedef struct {
    int32_t H;        /* query heads                                             */
    int32_t hk;       /* heads of the cache, dividing H (0 means H): query head hh
                         reads cache head hh / (H / hk)                          */
    int32_t d;        /* values per head: 64, 128 or 256                         */
    int32_t io_dtype; /* GDNQ_IO_F32 or GDNQ_IO_BF16 for q, k, v, o and the cache */
    int32_t page;     /* rows per page, a power of two, 8..65536                 */
    int32_t window;   /* attention over the last `window` rows (0: all)          */
    float scale;      /* of the scores, > 0 (0: 1/sqrt(d))                       */
    float acc_decay;  /* of the sums of weights, 0..1 (0: replaced unread)       */
} gdnq_attn_desc;

/*
 * A pool of pages with the tables of its slots.  Row r of a slot is row
 * r % page of page table[slot][r / page]; its keys (values) of head h are d
 * consecutive elements at
 *   k + p ldp + h ldh + (r % page) ldr.
 * ldp, ldh and ldr are multiples of 16 bytes; all 0: [n_pages,hk,page,d].
 * k and v may be one pool, between each other's pages, heads or rows (such as
 * [n_pages,2,hk,page,d]), where no row of the one shares a byte with one of the
 * other.
 * acc and pos belong to rows and heads too: [n_pages,hk,page] each.
 *   acc  the attention weight that the row has received, or NULL: gdnq_kv_append
 *        sets it to 0 and gdnq_attn_step adds to it; that of a prompt's own
 *        attention, which is not a call of this library, is the caller's to add
 *   pos  the position of its token, or NULL
 * An entry whose slot is outside [0, n_slots), or whose lens is outside
 * [0, max_pages page], is skipped on the device (nothing read or written for
 * it).  A row whose page number is outside [0, n_pages) does not exist: nothing
 * is stored for it and no attention goes to it; eviction skips its entry.
 * Pages may be shared by slots where a call only reads them.
 */
typedef struct {
    void *k, *v;           /* device, 16-byte aligned                            */
    float *acc;
    int32_t *pos;
    const int32_t *table;  /* device [n_slots,max_pages]                         */
    const int32_t *lens;   /* device [n_slots]: rows that the slot holds         */
    int32_t n_pages, n_slots, max_pages; /* max_pages page <= 2^30               */
    int64_t ldp, ldh, ldr; /* elements                                           */
} gdnq_kv;

/*
 * Stores new tokens: cu_seqlens as in gdnq_layer.h, or NULL with T == n: one
 * token for each of the n entries.  Sequence i's m tokens become the last rows of its
 * slot, lens - m .. lens - 1 (lens counts them already; one shorter than m is
 * skipped).
 *   k, v    device io_dtype [T, hk*d]: keys, turned as in gdnq_rope, and values
 *   q       device io_dtype [T, H*d], turned into q_out (or q itself, with the
 *           same row distance); both NULL: only k and v.  q_out may be other
 *           columns of the rows that k and v are columns of, with their row
 *           distance: a fused projection's output is turned where it is
 *   rope    with d and io_dtype of desc and its table; NULL: nothing turns
 *   pos     device int32 [T], or NULL: each token's row is its position
 * kv->acc, if there, is set to 0 and kv->pos, if there, to the position in the
 * new rows.  Rows of q_out of skipped entries and of no sequence are left as
 * they were.  n == 0 or T == 0 is a no-op.
 */
int gdnq_kv_append(const gdnq_attn_desc *desc, const gdnq_rope_desc *rope, const uint64_t *table, const gdnq_kv *kv,
                   const void *q, int64_t ldq, void *q_out, int64_t ldqo, const void *k, int64_t ldk, const void *v,
                   int64_t ldv, const int32_t *pos, const int32_t *slots, const int32_t *cu_seqlens, int32_t n,
                   int32_t T, void *stream);

/*
 * Bytes of device workspace that gdnq_attn_step needs for this descriptor, cache
 * (its sizes, and whether it has acc) and number of entries.  Never less for
 * more entries.  With acc it has room for the scores of every row of the pool,
 * n_pages page H 4 bytes, whatever the entries hold.
 */
int gdnq_attn_workspace(const gdnq_attn_desc *desc, const gdnq_kv *kv, int32_t n, size_t *bytes_out);

/*
 * The attention of one token for each of n entries over its slot's rows (all
 * lens of them, or the last `window`; the token's own row is there already):
 *   w_r = softmax_r(scale q . k_r),   o = sum_r w_r v_r.
 *   q, o  device io_dtype [n, H*d].  An entry without rows gives zeros.
 * NaN in a query, or in a key that is attended to, makes the outputs and sums of
 * its heads NaN, whatever else is in the call.
 * With kv->acc, for every row that was attended: acc = acc_decay acc + the sum
 * of w_r over the query heads of its cache head.  No page may then be attended to
 * twice in a call, by two entries or by one whose table names it twice.  (Pages
 * that lie before every row of a window are not attended to: their table entries
 * may be anything.)
 * workspace: device, 16-byte aligned, at least gdnq_attn_workspace bytes, free
 * for other use once the call has run; calls that may run at the same time need
 * one each.  n == 0 is a no-op.
 * The work is dealt out by the rows that a slot may hold, max_pages page or the
 * window, before the lens are known: batches of short caches (up to some hundred
 * rows) take up to 1.8 times as long in a table that is wider than they need.
 */
int gdnq_attn_step(const gdnq_attn_desc *desc, const gdnq_kv *kv, const void *q, int64_t ldq, void *o, int64_t ldo,
                   const int32_t *slots, int32_t n, void *workspace, size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace that gdnq_kv_evict needs; never less for more entries.
 * It follows the rows that a slot may hold, max_pages page: above the budget 8
 * bytes for each row that could move (the lesser of the budget and the rows behind
 * it, none up to 64), and above 32768 rows 4 more for every row, for each entry and
 * head.
 */
int gdnq_kv_evict_workspace(const gdnq_attn_desc *desc, const gdnq_kv *kv, int32_t budget, int32_t n,
                            size_t *bytes_out);

/*
 * Cuts every entry that holds more than `budget` rows down to that many, each
 * head by itself.  The lens - budget rows of least acc leave, of equal ones the
 * lower row first.  Rows whose pos is below `sink`, or above the head's largest
 * minus `recent`, stay (sink + recent <= budget; where more rows than the
 * budget are such, the lower of them leave).  Kept rows behind the budget move,
 * in order, into the rows before it that became free, in order: K, V, acc and
 * pos.  Rows from the budget on are left as they were.
 * The entry then holds min(lens, budget) rows: lens is the caller's to lower.
 * Keys carry their positions already, so attention does not see the order (a
 * window would: it counts rows).  kv->acc and kv->pos must be there, acc without
 * NaN.  Behind prompts acc is 0 everywhere unless the caller has added their
 * attention's weights: the lowest unprotected rows would leave.  Slots of one call
 * must be distinct, and so must their pages.  workspace as for gdnq_attn_step.
 * n == 0 is a no-op.  A table that is wider than the rows held costs time here too
 * (64 entries of 2049 rows, 8 heads, one row of each leaving: 16 us in tables of
 * 2080 rows, 22 of 20000, 23 of 131072).
 */
int gdnq_kv_evict(const gdnq_attn_desc *desc, const gdnq_kv *kv, int32_t budget, int32_t sink, int32_t recent,
                  const int32_t *slots, int32_t n, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDNQ_ATTN_H */
