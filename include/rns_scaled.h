/*
 * rns_scaled.h -- block-scaled 8-bit floating-point operands on gfx950: the
 * quantiser that makes them, the matrix product that takes them, and a
 * mixture-of-experts layer for a few tokens on weights held in them.
 *
 * The exact products of rns_gemm.h answer what a product is; these answer it
 * at the matrix cores' 8-bit rate, and rns_enclose.h tells how far such an
 * answer can be off: a block-scaled operand's entries (value times scale, up
 * to 28 significant bits) are binary64 numbers, which the enclosure takes as
 * they are.
 *
 * Conventions of rns_gemm.h: device pointers owned by the caller, launches
 * asynchronous on the caller's stream, no allocation, 0 or a negative RNS_E_*
 * code, nothing written on a validation error.  Arrays of binary32 and int32
 * lie on 4-byte boundaries.
 *
 * The format
 * ----------
 * Values.  RNS_T_E4M3 (4 exponent bits, 3 mantissa bits, largest 448, NaN but
 *   no infinity) or RNS_T_E5M2 (largest 57344, infinities and NaN), one byte
 *   each, rows of `ld` bytes.
 * Scales.  One per block of 128 columns (the contraction axis; the last block
 *   may be narrower), shared by block_rows = 1 row or block_rows = 128 rows.
 *   RNS_T_F32: any binary32 factor.  RNS_T_E8M0: a byte e standing for
 *   2^(e - 127), 255 for NaN.  The scale of row r, column block b is element
 *   (r / block_rows) * s_row + b * s_blk of the scale array.
 * Meaning.  Entry (r, c) is value(r, c) * scale(r / block_rows, c / 128).
 */
#ifndef RNS_SCALED_H
#define RNS_SCALED_H

#include "rns_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RNS_SCALE_BLOCK 128

enum rns_type {
    RNS_T_F32 = 0,
    RNS_T_BF16 = 1,
    RNS_T_F16 = 2,
    RNS_T_E4M3 = 3,
    RNS_T_E5M2 = 4,
    RNS_T_E8M0 = 5
};

/* sizes above these are refused (RNS_E_ARG): element indices inside one tile are 32-bit */
#define RNS_SCALED_DIM_MAX ((int64_t)1 << 31)
#define RNS_SCALED_LD_MAX ((int64_t)1 << 22)

typedef struct rns_scaled {
    const void *values;      /* [rows][ld] bytes */
    const void *scales;
    int64_t ld;              /* bytes between rows, >= the row's columns */
    int64_t s_row, s_blk;    /* scale strides, in elements */
    int32_t type;            /* RNS_T_E4M3 or RNS_T_E5M2 */
    int32_t scale_type;      /* RNS_T_F32 or RNS_T_E8M0 */
    int32_t block_rows;      /* 1 or 128 */
    int32_t readable;        /* 1: every row may be read to the next multiple of 16 bytes */
} rns_scaled_t;

/*
 * rns_block_quantize -- q, s from x [R][C] (x_type RNS_T_F32, BF16 or F16;
 * ldx elements between rows), and, where qt is not null, qt, st from its
 * transpose [C][R], quantised along R, from the same read of x.
 *
 * With amax the largest finite magnitude of a block and FMAX the type's
 * largest value:
 *   scale_type RNS_T_F32:  s = max(fl(amax / FMAX), 2^-126), 1 if amax is 0
 *   scale_type RNS_T_E8M0: s = the smallest power of two with amax <= FMAX s,
 *                          clamped to 2^-127 .. 2^127, 1 if amax is 0
 *   value = x / s, rounded to binary32 and then to the nearest value of the
 *           type, ties to even (with a power of two the first is exact).
 * NaN stays NaN; an infinity becomes NaN in E4M3 and stays one in E5M2; both
 * leave the block's other entries as they would be without them.
 *
 * Rows of q are ldq bytes apart, ldq a multiple of 128 and at least C: columns
 * C .. up to the next multiple of 128 are written as zeros.  Scale (r, b) is
 * at element b * s_ld + r, s_ld at least the scale rows (R, or ceil(R / 128)
 * for block_rows 128).  qt has C rows ldqt bytes apart (a multiple of 128, at
 * least R), st the scale stride st_ld likewise for C rows.
 * Returns RNS_OK, RNS_E_ARG or RNS_E_HIP.  R == 0 or C == 0 is a no-op.
 */
int rns_block_quantize(int64_t R, int64_t C, const void *x, int32_t x_type, int64_t ldx,
                       int32_t type, int32_t block_rows, int32_t scale_type,
                       void *q, int64_t ldq, void *s, int64_t s_ld,
                       void *qt, int64_t ldqt, void *st, int64_t st_ld, hipStream_t stream);

/*
 * rns_scaled_mm_nt -- Y[m][n] = sum_k a(m, k) b(n, k): a is [M][K], b is
 * [N][K], both contracted along their columns, with
 *   Y[m][n] = sum_blocks sa(m, blk) sb(n, blk) sum_{k in blk} va(m, k) vb(n, k),
 * the scaled total in binary32, rounded once to y_type (RNS_T_F32, BF16 or F16;
 * ldy elements between rows).  Scales may be as far from one as they can be
 * written: nothing overflows before a block's scaled product does, and one below
 * 2^-120 is kept to 2^-144.  For y_type RNS_T_F32 the inner sums are binary32
 * sums of exact products; for the 16-bit types they are the 8-bit matrix
 * instructions', which keep each product to about 2^-14 of the largest of the
 * 64 or 128 added at a time (sums whose terms cancel to less than that want y
 * in binary32).  b's values are
 * RNS_T_E4M3, a's either type; both scale arrays are of one type.
 *
 * Operands are read in place.  Rows on 16-byte boundaries, readable to the next
 * one (what rns_block_quantize writes is), take the fast kernels.  The
 * workspace (16-byte aligned) holds the partial sums of products that are split
 * along K (rns_scaled_workspace_size; mostly 0, then ws may be null).
 * K == 0 writes zeros; M == 0 or N == 0 is a no-op.
 * Returns RNS_OK, RNS_E_ARG, RNS_E_WORKSPACE or RNS_E_HIP.
 */
int rns_scaled_workspace_size(int64_t M, int64_t N, int64_t K, const rns_scaled_t *a, const rns_scaled_t *b,
                              size_t *bytes);
int rns_scaled_mm_nt(int64_t M, int64_t N, int64_t K, const rns_scaled_t *a, const rns_scaled_t *b,
                     void *y, int32_t y_type, int64_t ldy, void *ws, size_t ws_bytes, hipStream_t stream);

/*
 * rns_moe_layer -- a mixture-of-experts layer for up to RNS_MOE_MAX_TOKENS
 * tokens.  x is bfloat16 [T][H], router [E][H] (RNS_T_BF16 or RNS_T_F32):
 *   l = x router^T                      (binary32)
 *   the top_k experts of a token: largest l first, the lower index first
 *     among equals, NaN below every number
 *   p_e = exp(l_e - max l) / sum over the chosen experts (renormalize != 0)
 *     or over all experts (renormalize == 0)
 *   y = sum_e p_e W_out[e] (silu(W_in[e][0] x) * (W_in[e][1] x))
 * with silu(g) = g / (1 + exp(-g)).  Weights are RNS_T_E4M3 with 128 x 128
 * blocks: w_in [E][2][I][H], w_out [E][H][I], contiguous, 16-byte aligned, H
 * and I multiples of 16.  Scale strides are in elements: w_in's scale of
 * expert e, part p, row block r, column block b is at e * si[0] + p * si[1] +
 * r * si[2] + b * si[3], w_out's at e * so[0] + r * so[1] + b * so[2].
 * Sums are binary32; the hidden activation is carried with 16 mantissa bits.
 * A token's result does not depend on what the other tokens of the call hold.
 * y is bfloat16 [T][H], x and y contiguous and 16-byte aligned.
 * ids (int32 [T][top_k]) and probs (binary32 [T][top_k]) receive the routing
 * where they are not null.  ws: rns_moe_workspace_size bytes, 256-byte aligned.
 * T == 0 is a no-op.  Returns RNS_OK, RNS_E_ARG, RNS_E_WORKSPACE or RNS_E_HIP.
 */
#define RNS_MOE_MAX_TOKENS 64
#define RNS_MOE_MAX_EXPERTS 256
#define RNS_MOE_MAX_TOP_K 16

typedef struct rns_moe {
    int32_t T, E, H, I, top_k, renormalize;
    int32_t router_type;     /* RNS_T_BF16 or RNS_T_F32 */
    int32_t scale_type;      /* RNS_T_F32 or RNS_T_E8M0, of both weights */
    const void *x, *router, *w_in, *w_in_scales, *w_out, *w_out_scales;
    int64_t si[4], so[3];
    void *y;
    int32_t *ids;
    float *probs;
} rns_moe_t;

int rns_moe_workspace_size(int32_t T, int32_t E, int32_t H, int32_t I, int32_t top_k, size_t *bytes);
int rns_moe_layer(const rns_moe_t *args, void *ws, size_t ws_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* RNS_SCALED_H */
