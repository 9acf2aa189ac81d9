/*
 * gdnq_layer.h -- the operators around a recurrent state in its layer, for
 * AMD Instinct MI355X (gfx950), in the same library as gdnq.h:
 *
 *  - the short causal convolution in front of the recurrence, for packed
 *    prompts (gdnq_conv_prefill) and single tokens (gdnq_conv_step);
 *  - the selective state space scan, the recurrence without the delta rule
 *    (LinQuant, appendix Table 3, Mamba-2 row), for packed prompts
 *    (gdnq_ssm_prefill) and single tokens (gdnq_ssm_step).  Its fp32 states
 *    have the layout of the GDN / KDA states, so gdn_state_quantize and
 *    gdn_state_dequantize store and restore them in 8, 6 or 4 bits;
 *  - the RMS norm behind the block with its gate (gdnq_norm_gated), and the
 *    residual sum with the norm in front of the next block
 *    (gdnq_norm_residual).
 *
 * The conventions of gdnq.h hold (asynchronous on `stream`, nothing
 * allocated or kept between calls, argument errors found on the host before
 * any launch, NaN or infinite inputs undefined), and these besides:
 *
 *  - Token tensors (x, y, z, B, C, dt, residuals) are rows of contiguous
 *    values, one row per token; ld* is the distance between rows in
 *    elements, at least the row's length (0 means the row's length), so a
 *    call reads its columns straight out of a projection's wider output.
 *    These pointers need their element's alignment only; rows whose pointers
 *    and distances are all multiples of 16 bytes take wide loads.
 *    Weights, states, per-entry arrays (slots, cont, cu_seqlens) and
 *    workspaces are contiguous and 16-byte aligned.
 *  - Outputs and states must not overlap any input (the address range from
 *    the first to the last row counts) or each other.
 *  - Packed sequences: T token rows hold n_seqs sequences, sequence i in rows
 *    cu_seqlens[i] .. cu_seqlens[i+1]-1 (device int32 [n_seqs+1],
 *    non-decreasing, from >= 0 to <= T).  Rows that belong to no sequence are
 *    left as they were.  A sequence whose bounds are outside 0 <= start <=
 *    end <= T is skipped on the device; one of zero tokens leaves its slot as
 *    it was.  Where cu_seqlens decreases, rows and slots of other sequences
 *    may be left as they were too, or in part; nothing else is touched.
 *  - State pools: sequence or token i uses slot slots[i] (device int32; NULL:
 *    slot i, which needs n_slots >= n) of the n_slots in the pool.  An entry
 *    whose slot is outside [0, n_slots) is skipped on the device (nothing
 *    read or written for it).  Slots of one call must be distinct: two
 *    entries on one slot race.
 *  - cont (device int32 [n_seqs], NULL: all zero): nonzero continues from the
 *    slot's state, zero starts from zeros without reading the slot.
 *  - In bf16, sums, states, decays and norms are formed in fp32, and each
 *    output is rounded once.
 */
#ifndef GDNQ_LAYER_H
#define GDNQ_LAYER_H

#include "gdnq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------- short causal convolution */
#define GDNQ_CONV_SILU 1u   /* y = s / (1 + e^{-s}) of the sum s */

typedef struct {
    int32_t C;         /* channels, >= 1                                       */
    int32_t width;     /* taps, 2..4                                           */
    int32_t io_dtype;  /* GDNQ_IO_F32 or GDNQ_IO_BF16 for x, y and the state   */
    uint32_t flags;    /* GDNQ_CONV_SILU or 0                                  */
} gdnq_conv_desc;

/*
 * Depthwise causal convolution of every sequence:
 *   y_t,c = act(bias_c + sum_{k < width} w_k,c x_{t-(width-1)+k,c})
 *   x      device io_dtype [T,C] (rows ldx apart); y likewise (rows ldy apart)
 *   w      device fp32 [width,C], the newest token's tap last
 *   bias   device fp32 [C], or NULL
 *   state  device io_dtype [n_slots,width-1,C]: the last width-1 inputs,
 *          oldest first, exactly as they were read; replaced at the end of
 *          each sequence.
 * T == 0 or n_seqs == 0 is a no-op.
 */
int gdnq_conv_prefill(const gdnq_conv_desc *desc, const void *x, int64_t ldx, const float *w,
                      const float *bias, void *state, int32_t n_slots, const int32_t *slots,
                      const int32_t *cont, const int32_t *cu_seqlens, int32_t n_seqs, int32_t T,
                      void *y, int64_t ldy, void *stream);

/*
 * One token for each of n entries: row i of x [n,C] and y, state of slot
 * slots[i] read, shifted by one token and stored.  n == 0 is a no-op.
 */
int gdnq_conv_step(const gdnq_conv_desc *desc, const void *x, int64_t ldx, const float *w,
                   const float *bias, void *state, int32_t n_slots, const int32_t *slots, int32_t n,
                   void *y, int64_t ldy, void *stream);

/* --------------------------------------- selective state space scan */
#define GDNQ_SSM_SOFTPLUS 1u   /* delta = softplus(dt + dt_bias), else dt + dt_bias */

typedef struct {
    int32_t H;             /* heads                                             */
    int32_t dk, dv;        /* state and value channels per head, each 64 or 128 */
    int32_t hk;            /* heads of B and C, dividing H (0 means H): head hh
                              reads B and C of head hh / (H / hk)               */
    int32_t io_dtype;      /* GDNQ_IO_F32 or GDNQ_IO_BF16 for x, B, C, dt, y    */
    uint32_t flags;        /* GDNQ_SSM_SOFTPLUS or 0                            */
    float dt_min, dt_max;  /* delta is clamped to [dt_min, dt_max], 0 <= dt_min */
} gdnq_ssm_desc;

/*
 * The inputs and the output of a call, rows of one token each:
 *   x, y  [T, H*dv], B, C  [T, hk*dk], dt  [T, H], io_dtype, rows ldx, ldy,
 *   ldb, ldc, lddt elements apart
 *   A        device fp32 [H], finite and <= 0
 *   D        device fp32 [H] or NULL (no skip term)
 *   dt_bias  device fp32 [H] or NULL
 * With delta_t = clamp(softplus(dt_t + dt_bias), dt_min, dt_max) and
 * a_t = e^{delta_t A}, per head:
 *   S_t = a_t S_{t-1} + B_t (delta_t x_t)^T,   y_t = S_t^T C_t + D x_t.
 */
typedef struct {
    const void *x, *B, *C, *dt;
    void *y;
    const float *A, *D, *dt_bias;
    int64_t ldx, ldb, ldc, lddt, ldy;
} gdnq_ssm_io;

/*
 * Bytes of device workspace that gdnq_ssm_prefill needs for this descriptor,
 * number of sequences and number of token rows (0: none).  Never less for more
 * sequences or more rows: the workspace of a program's largest call serves the
 * others.
 */
int gdnq_ssm_workspace(const gdnq_ssm_desc *desc, int32_t n_seqs, int32_t T, size_t *bytes_out);

/*
 * Packed prompts.  S: device fp32 [n_slots,H,dk,dv], the pool of states (the
 * layout of gdnq.h's fp32 states); each sequence's slot is replaced by its
 * state after the last token.  io_dtype must be GDNQ_IO_BF16 and rows at most
 * 2^22 elements apart (GDNQ_EUNSUPPORTED otherwise).  Runs chunk by chunk on
 * the matrix cores, fp32 operands split into bf16 parts (two for outputs, three
 * for states).
 * Range: inside a chunk values carry factors from 2^-80 to 2^80, so a head's
 * states and its sums of delta x and B (delta x)^T must stay below 2^40 in
 * magnitude (larger ones may overflow), and y takes values that are not far
 * above 2^-30 with an absolute error of up to 2^-46 (sum |C| + 64 max |B C|).
 * workspace: device, 16-byte aligned, at least gdnq_ssm_workspace bytes
 * (NULL where that is 0), free for other use once the call has run; calls
 * that may run at the same time need one each.
 * T == 0 or n_seqs == 0 is a no-op.
 */
int gdnq_ssm_prefill(const gdnq_ssm_desc *desc, const gdnq_ssm_io *io, float *S, int32_t n_slots,
                     const int32_t *slots, const int32_t *cont, const int32_t *cu_seqlens,
                     int32_t n_seqs, int32_t T, void *workspace, size_t workspace_bytes, void *stream);

/* One token for each of n entries (rows of x, B, C, dt, y).  n == 0 is a no-op. */
int gdnq_ssm_step(const gdnq_ssm_desc *desc, const gdnq_ssm_io *io, float *S, int32_t n_slots,
                  const int32_t *slots, int32_t n, void *stream);

/* ------------------------------------------------- norms around a block */
#define GDNQ_NORM_GATE_SIGMOID 1u   /* gate act(z) = 1/(1+e^{-z}); else z/(1+e^{-z}) */
#define GDNQ_NORM_GATE_FIRST 2u     /* norm(x act(z)); else norm(x) act(z)           */
#define GDNQ_NORM_GROUP_WEIGHT 4u   /* w has `group` values, shared by the groups    */
#define GDNQ_NORM_RES_F32 8u        /* the residual stream is fp32 whatever io_dtype */

typedef struct {
    int32_t D;         /* values per row, 1..32768                             */
    int32_t group;     /* values normalised together, dividing D (0 means D)   */
    int32_t io_dtype;  /* GDNQ_IO_F32 or GDNQ_IO_BF16                          */
    uint32_t flags;
    float eps;         /* > 0                                                  */
    float w_offset;    /* the weight is w_offset + w (0, or 1 for weights
                          kept around zero)                                    */
} gdnq_norm_desc;

/*
 * After a block, with N(u)_c = u_c / sqrt(mean over c's group of u^2 + eps):
 *   y = (w_offset + w) N(x) act(z),  or  (w_offset + w) N(x act(z)) with
 *   GDNQ_NORM_GATE_FIRST.  z NULL: no gate.
 *   x, z, y  device io_dtype [rows,D]; w device fp32 [D] ([group] with
 *   GDNQ_NORM_GROUP_WEIGHT).  rows == 0 is a no-op.
 */
int gdnq_norm_gated(const gdnq_norm_desc *desc, const void *x, int64_t ldx, const void *z, int64_t ldz,
                    const float *w, void *y, int64_t ldy, int32_t rows, void *stream);

/*
 * Before a block (group must be 0 or D; only GDNQ_NORM_RES_F32 as a flag):
 *   p = x, or (w_offset + post_w) N(x) when post_w is not NULL (a norm behind
 *   the block that x comes from);
 *   r = res + scale p, stored to res_out;   y = (w_offset + w) N(r), from r
 *   before it is rounded.
 *   x, y  device io_dtype [rows,D]; res, res_out  io_dtype or, with
 *   GDNQ_NORM_RES_F32, fp32 [rows,D]; res_out may be res itself (with the same
 *   row distance), and y may be NULL (the sum alone).  w, post_w fp32 [D].
 */
int gdnq_norm_residual(const gdnq_norm_desc *desc, const void *x, int64_t ldx, const float *post_w,
                       float scale, const void *res, int64_t ldr, void *res_out, int64_t ldro,
                       const float *w, void *y, int64_t ldy, int32_t rows, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDNQ_LAYER_H */
