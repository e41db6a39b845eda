/*
 * tp_block.h -- C ABI of libtp_linear.so, second part: 8-bit block-scaled
 * linear layers and the norm at the boundary between two transformer blocks.
 *
 * The conventions of tp_linear.h hold (layout, device pointers, streams,
 * errors and tp_last_error(), no device memory allocated, M == 0 a no-op),
 * with the types and alignments given here.
 *
 * Quantized rows
 * --------------
 * A matrix of K features per row is held as
 *   codes   [rows, K8]  e4m3 (OCP: finite, largest 448, 0x7f/0xff NaN), one
 *                       byte each, K8 = K rounded up to a multiple of 128; the
 *                       codes past K are zero;
 *   scales  [rows, K8 / 128]  e8m0, one byte each: byte s stands for
 *                       2^(s - 127), 255 for NaN.
 * Feature k of row r stands for codes[r, k] * 2^(scales[r, k / 128] - 127).  The products keep the
 * values that fp32 holds as normal numbers, 2^-126 to below 2^128; smaller ones may count as zero,
 * larger ones as infinite.
 * Scales are powers of two: the CDNA4 matrix cores apply them inside the
 * product, and scaling by one is exact.  Both operands of a product carry a
 * scale for each 128 features of each row, so a shard of quantized rows is cut
 * like any other (rows anywhere, features at multiples of 128, and at multiples of
 * 512 where the cut is used in place: scale rows start at 4-byte addresses).
 */
#ifndef TP_BLOCK_H
#define TP_BLOCK_H

#include "tp_linear.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * tp_quantize_fp8 -- rows of x to codes and scales.
 *
 *   x       [M, K]        bf16 or fp32 (x_dtype), row stride ldx >= K elements;
 *                         element alignment suffices
 *   codes   [M, K8]       row stride ldc >= K8 bytes, base and ldc multiples of 16
 *   scales  [M, K8/128]   row stride lds >= K8/128 bytes, base and lds multiples of 4;
 *                         bytes past K8/128 are not written
 *
 * Scale of a block: the least 2^e, e >= -126, with max |x| <= 448 * 2^e; 1 for an
 * all-zero block.  Codes: x / 2^e (exact) rounded to e4m3, nearest even.  A block
 * that holds an infinity or a NaN gets the scale NaN (255) and codes 0x7f, so
 * every product with it is NaN.
 * Errors: TP_ERR_INVALID_ARG (pointers, strides, dtype, K < 1, M < 0),
 * TP_ERR_UNSUPPORTED (dimensions above 2^30, strides above 2^31).
 */
tp_status tp_quantize_fp8(const void *x, int64_t ldx, tp_dtype x_dtype, void *codes, int64_t ldc,
                          void *scales, int64_t lds, int64_t M, int64_t K, hipStream_t stream);

/*
 * tp_linear_colwise_fp8 -- tp_linear_colwise on quantized rows:
 * Y_r = act(X . W_r^T + b_r).
 *
 *   x, x_scale  [M, K] codes (row stride ldx bytes) and [M, K/128] scales (ldxs)
 *   w, w_scale  [n_shard, K] codes (ldw) and [n_shard, K/128] scales (ldws);
 *               2 n_shard rows [gate; up] with TP_ACT_SWIGLU
 *   bias        [n_shard] (2 n_shard with TP_ACT_SWIGLU) bf16, or NULL; 8-byte aligned
 *   y           [M, n_shard]  bf16 or fp32 (y_dtype), row stride ldy elements
 *   act         as tp_linear_colwise
 *
 * Arithmetic: bias and activation in fp32, one rounding to y_dtype, and products and sums
 * as exact as that rounding asks for.  fp32 output, and up to 96 rows: the codes are widened
 * to bf16 (exact) and multiplied exactly, fp32 accumulation.  bf16 output of more rows: where the
 * output is large, the 8-bit matrix cores, which accumulate in fp32 but drop, among the products of
 * each 8 consecutive features, what lies 2^13 and more below the largest of them (about 2e-5 of the
 * result, a hundredth of the bf16 rounding).
 * Requires K % 128 == 0 (the padded K of the quantized rows), n_shard % 16 == 0;
 * code pointers 16-byte aligned and their strides multiples of 16; scale pointers
 * 4-byte aligned and their strides multiples of 4 (>= K/128; the product may read,
 * and ignores, the bytes between K/128 and the next multiple of 4 of each row);
 * y 16-byte aligned, ldy a multiple of 16 bytes; each operand view below 2 GiB, row
 * strides of at most 2^31, at most 2^22 output tiles of 192 x 256
 * (TP_ERR_UNSUPPORTED otherwise).
 */
tp_status tp_linear_colwise_fp8(const void *x, int64_t ldx, const void *x_scale, int64_t ldxs,
                                const void *w, int64_t ldw, const void *w_scale, int64_t ldws,
                                const void *bias, void *y, int64_t ldy, tp_dtype y_dtype, tp_act act,
                                int64_t M, int64_t n_shard, int64_t K, hipStream_t stream);

/*
 * tp_linear_rowwise_fp8 -- tp_linear_rowwise on quantized rows: the fp32 partial
 * P_r = X_r . W_r^T, no bias.  Operands and requirements as tp_linear_colwise_fp8;
 * partial [M, N] fp32, row stride ldp (a multiple of 4).
 */
tp_status tp_linear_rowwise_fp8(const void *x, int64_t ldx, const void *x_scale, int64_t ldxs,
                                const void *w, int64_t ldw, const void *w_scale, int64_t ldws,
                                float *partial, int64_t ldp, int64_t M, int64_t N, int64_t k_shard,
                                hipStream_t stream);

/*
 * tp_linear_fp8_tile_shape -- host-only query of how the two products above run a problem of this
 * shape (K input features; for TP_ACT_SWIGLU, N counts the outputs) on the current device:
 * *tile_rows and *tile_cols receive the output tile of the tiled kernels (rows 256, 224, 192, 128, 96
 * or 64; columns 256, 192 or 128, half of that with SwiGLU), or, where the split-K kernel runs (up to
 * 96 rows, and beyond when one round of its workgroups covers the output), the rows that a workgroup holds
 * (a multiple of 16, up to 96) and the run of output columns (4 to 48, at most 32 with SwiGLU) that
 * it owns.
 * Errors: TP_ERR_INVALID_ARG for a null output pointer, an unknown act or y_dtype, or sizes
 * outside 0 <= M, 0 < N, 0 < K, all at most 2^30.
 */
tp_status tp_linear_fp8_tile_shape(int64_t M, int64_t N, int64_t K, tp_act act, tp_dtype y_dtype,
                                   int64_t *tile_rows, int64_t *tile_cols);

/*
 * tp_block_norm -- the boundary between two blocks in one pass over the rows.
 *
 *   y = ((parts[0] + parts[1]) + ...) + bias          the block's output (the SUM of
 *                                                     tp_partial_combine, fp32 adds)
 *   h = residual_scale * x + gate_g * post(y)         the residual stream
 *   z = pre(h) * (1 + scale_g) + shift_g              the next block's input
 *
 * post and pre are TP_NORM_NONE, TP_NORM_LAYER ((v - mean) / sqrt(var + eps), biased
 * variance) or TP_NORM_RMS (v / sqrt(mean(v^2) + eps)), then * weight + bias where
 * given ([D] bf16).  All arithmetic is fp32; h and z are each rounded once, and
 * z is computed from the unrounded h.
 *
 * Without parts (num_parts 0) there is no block output: h is x, it is not written
 * (h, gate and bias NULL, post_norm NONE, residual_scale 1) and z = pre(x) ....
 * With pre_norm NONE there is no z (z, scale, shift NULL).
 *
 * Rows take their modulation (gate, scale, shift: rows of [groups, D] tables) from
 * group r / group_rows, or, with group_index (int32 [M], device), from group
 * group_index[r].  An index outside [0, groups) names no group: scale and shift are
 * then 0 and the gated branch is left out (h = residual_scale * x), whatever its
 * values.  A gate, scale or shift that is NULL does not take part (1, 0, 0).
 *
 * Aliasing: h may be x (same pointer, stride and dtype).  Otherwise outputs overlap
 * nothing.  Element alignment suffices for every input, h and z.  Quantized z: as
 * tp_quantize_fp8's outputs.
 * D at most 32768 (TP_ERR_UNSUPPORTED above), num_parts at most 16.
 */
typedef enum { TP_NORM_NONE = 0, TP_NORM_LAYER = 1, TP_NORM_RMS = 2 } tp_norm;
typedef enum { TP_ROWS_BF16 = 0, TP_ROWS_F32 = 1, TP_ROWS_FP8 = 2 } tp_rows;

typedef struct tp_block_norm_args {
    int64_t M, D;
    const void *x;              /* [M, D] the residual stream */
    int64_t ldx;
    tp_dtype x_dtype;
    tp_dtype part_dtype;
    const void *const *parts;   /* HOST array of num_parts device pointers, each [M, D] */
    int64_t ld_part;
    int num_parts;              /* 0 .. 16 */
    tp_norm post_norm;
    const void *bias;           /* [D] bf16 or NULL */
    const void *post_weight;    /* [D] bf16 or NULL */
    const void *post_bias;
    void *h;                    /* [M, D]; NULL exactly if num_parts == 0 */
    int64_t ldh;
    tp_dtype h_dtype;
    tp_norm pre_norm;
    const void *pre_weight;     /* [D] bf16 or NULL */
    const void *pre_bias;
    void *z;                    /* [M, D]; NULL exactly if pre_norm is TP_NORM_NONE */
    int64_t ldz;                /* elements (bytes for codes) */
    void *z_scale;              /* TP_ROWS_FP8: the scales; NULL otherwise */
    int64_t ldzs;
    tp_rows z_rows;
    tp_dtype mod_dtype;         /* of gate, scale and shift */
    const void *gate;           /* [groups, D] or NULL */
    const void *scale;
    const void *shift;
    int64_t ld_gate, ld_scale, ld_shift;
    int64_t groups;             /* >= 1 where a table is given */
    int64_t group_rows;         /* >= 1; groups * group_rows >= M (without group_index) */
    const int32_t *group_index; /* int32 [M] or NULL */
    float residual_scale;
    float eps;                  /* finite, >= 0 */
} tp_block_norm_args;

tp_status tp_block_norm(const tp_block_norm_args *args, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TP_BLOCK_H */
