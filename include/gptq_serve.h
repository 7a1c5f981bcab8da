/*
 * gptq_serve.h — the quantized forms a model is served in (part of libgptq.so).
 *
 * gptq.h quantizes the weights of a layer. Next to the integer codes it writes, a model is
 * served with activations and weights in 8-bit floating point, and with a quantized cache of
 * keys and values:
 *
 *   gptq_fp8_quantize   a matrix to e4m3 codes with one scale for each block of 128
 *   gptq_fp8_matmul     the product of two such matrices on the 8-bit tensor cores
 *   gptq_cache_write    rows of keys and values quantized into the slots of a cache
 *   gptq_cache_read     rows of the cache read back in 16 or 32 bits
 *
 * The conventions of gptq.h hold: device pointers of the current device, work enqueued on
 * `stream` only, argument errors returned at once with nothing enqueued, errors that the device
 * finds kept in the status word that gptq_sync_status reads. None of these entry points needs a
 * workspace, allocates, or keeps anything between calls; all of them can be captured into a CUDA
 * graph, and run at once on several streams as long as they do not write the same memory.
 *
 * Arrays start on a multiple of their element's size (more where it is said); others are refused.
 *
 * e4m3: 1 sign, 4 exponent and 3 mantissa bits, largest value 448, no infinity, one NaN.
 */
#ifndef GPTQ_SERVE_H
#define GPTQ_SERVE_H

#include "gptq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The entry points of this header also take 16-bit IEEE floats, next to the types of gptq_dtype
 * (GPTQ_BF16 = 0, GPTQ_F32 = 1). */
typedef enum { GPTQ_F16 = 2 } gptq_serve_dtype;

/* Columns that share a scale. */
#define GPTQ_FP8_BLOCK 128

/*
 * codes, scales = X in 8-bit floating point, one scale per block of block_rows x 128:
 *   a = max |x| over the block;  s = max(a / 448, 2^-126);  r = 1 / s (both fp32, nearest);
 *   code = the e4m3 value nearest to x r (the exact product, rounded once, ties to even).
 * The value a code stands for is s * code.
 *   X           device, rows x cols, x_dtype GPTQ_BF16, GPTQ_F16 or GPTQ_F32, rows ldx elements
 *               apart (ldx >= cols; any alignment of the type).
 *   block_rows  1 (activations: one scale per row and 128 columns) or 128 (weights).
 *   codes       device, rows x cols bytes, rows ldc bytes apart (ldc >= cols). gptq_fp8_matmul
 *               needs rows that start on 16-byte boundaries. Bytes between cols and ldc are left.
 *   scales      device, ceil(rows / block_rows) x ceil(cols / 128) fp32, row-major.
 * Ragged last blocks take the values they have. rows == 0 or cols == 0 is a no-op.
 * Limits: rows * ceil(cols / 128) < 2^31, cols < 2^31.
 * Device errors: GPTQ_ERR_NONFINITE (info = row of a NaN or an infinity in X). Such a value gets
 * the e4m3 NaN, and its block's scale comes from the block's finite values.
 */
GPTQ_API int gptq_fp8_quantize(const void *X, int x_dtype, int64_t rows, int64_t cols, int64_t ldx,
                               int block_rows, void *codes, int64_t ldc, float *scales,
                               gptq_stream_t stream);

/*
 * Y = A B^T of two matrices in 8-bit floating point with block scales:
 *   Y[i][j] = sum_b sA[i][b] sB[j / 128][b] sum_{l in block b} A[i][l] B[j][l]
 * over the blocks b of 128 of the k common columns. The inner sums run on the tensor cores with
 * fp32 accumulation; each is scaled by the fp32 product of its two scales and added in fp32; Y is
 * rounded once, to y_dtype.
 *   A, sA   device, m x k e4m3 codes, rows lda bytes apart; m x ceil(k / 128) fp32 (activations,
 *           as gptq_fp8_quantize writes them with block_rows 1).
 *   B, sB   device, n x k e4m3 codes, rows ldb bytes apart; ceil(n / 128) x ceil(k / 128) fp32
 *           (a layer's weight, one neuron per row, block_rows 128).
 *   Y       device, m x n, y_dtype GPTQ_BF16, GPTQ_F16 or GPTQ_F32, rows ldy elements apart
 *           (ldy >= n). Must not overlap the inputs.
 * A and B must start on 16-byte boundaries, and lda and ldb be multiples of 16, at least k (the
 * pitch of a single row is not looked at). m, n and k are otherwise free (k == 0 writes zeros, m == 0 or n == 0 is a no-op), each < 2^31 - 256.
 * A call gives the same bits each time it is made on a device of the same number of multiprocessors
 * (no atomics). m, n, k and that number choose how the sum over the blocks is split, so the same row or
 * column can differ in its last bits between products of other sizes, or between devices.
 * A code that is NaN makes its row (A) or column (B) of Y NaN. Scales are taken as they are.
 */
GPTQ_API int gptq_fp8_matmul(const void *A, int64_t lda, const float *sA, const void *B,
                             int64_t ldb, const float *sB, int64_t m, int64_t n, int64_t k,
                             void *Y, int y_dtype, int64_t ldy, gptq_stream_t stream);

/* What a cache holds for each group of values. */
typedef enum {
    GPTQ_CACHE_INT4 = 0, /* 4-bit min-max grid: packed codes, a scale, a zero-point */
    GPTQ_CACHE_INT8 = 1, /* 8-bit min-max grid */
    GPTQ_CACHE_E4M3 = 2  /* e4m3 codes and a scale, no zero-point */
} gptq_cache_format;

/* Added to the format of gptq_cache_read: rows without a slot are set to zero. */
#define GPTQ_CACHE_CLEAR 16

/* Most tokens of one gptq_cache_write call that need no `claims`. */
#define GPTQ_CACHE_UNCLAIMED 512

/*
 * Quantize rows of keys and values into slots of a cache. A cache has n_slots slots; slot i of a
 * paged cache is entry i % page_size of page i / page_size. K and V each have three arrays (V's
 * arrays and V itself are NULL for a cache of one kind of row):
 *   codes   n_slots x heads x head_dim codes: two 4-bit codes per byte (the even element in the
 *           low half, as gptq_quantize_layer packs them), else one byte each; 8-byte aligned.
 *   scales  n_slots x heads x G fp32, G = head_dim / group_size (1 if group_size is 0).
 *   zeros   n_slots x heads x G uint8; NULL for GPTQ_CACHE_E4M3.
 * Each group of group_size consecutive values of a head (0: the head) gets its own grid:
 *   4 and 8 bits: the min-max rule of gptq_quantize_layer: mn = min(0, min x), mx = max(0, max x),
 *     a zero range widened to [-1, 1]; s = max((mx - mn) / maxq, 2^-126); z = the whole number
 *     nearest to -mn maxq / (mx - mn); code = clamp(rint(x r + z), 0, maxq) with r = 1 / s (fp32;
 *     x r + z is rounded once). Ties go to the even number. The value is s (code - z).
 *   e4m3: as gptq_fp8_quantize, with the group as the block.
 *   K, V        device, tokens x heads x head_dim values of x_dtype (GPTQ_BF16, GPTQ_F16 or
 *               GPTQ_F32): element (t, h, d) at t * token stride + h * head stride + d (strides in
 *               elements, e.g. of views into a fused projection).
 *   slots       device, tokens int64. A negative slot skips its token: nothing of it is read into
 *               the cache or checked. If several tokens of the call name the same slot, the last
 *               one stays, whole.
 *   claims      device, n_slots int32 that belong to the cache and are zero: scratch that finds
 *               such tokens, zero again when the call is done. May be NULL for up to
 *               GPTQ_CACHE_UNCLAIMED tokens. Two calls that run at once on one cache must not
 *               write the same slot.
 * head_dim and group_size are multiples of 8, head_dim % group_size == 0, group_size <= 1024 (and
 * head_dim <= 1024 where group_size is 0), heads * head_dim <= 65536. tokens < 2^31.
 * Device errors: GPTQ_ERR_ARG (info = token whose slot is not below n_slots; it is skipped),
 * GPTQ_ERR_NONFINITE (info = token with a NaN or an infinity, or a group whose range overflows
 * fp32). With min-max grids such a group reads back as NaN; with e4m3 the value alone does.
 */
GPTQ_API int gptq_cache_write(const void *K, int64_t k_token_stride, int64_t k_head_stride,
                              const void *V, int64_t v_token_stride, int64_t v_head_stride,
                              int x_dtype, int64_t tokens, int heads, int head_dim,
                              const int64_t *slots, int64_t n_slots, int format, int group_size,
                              void *codes_k, float *scales_k, uint8_t *zeros_k, void *codes_v,
                              float *scales_v, uint8_t *zeros_v, int32_t *claims,
                              gptq_stream_t stream);

/*
 * Read rows of a cache back: K[t], V[t] = the values of slot slots[t], each the product s (code - z)
 * (e4m3: s times the code's value) rounded to fp32 and, where y_dtype has 16 bits, rounded to it next.
 * Arguments as in gptq_cache_write, K and V written (no two heads may overlap). A slot may be named
 * any number of times. A negative slot leaves its row of K and V as it was, and so does a slot not
 * below n_slots, which is reported (GPTQ_ERR_ARG, info = token); with format + GPTQ_CACHE_CLEAR
 * both rows are set to zero instead.
 */
GPTQ_API int gptq_cache_read(const int64_t *slots, int64_t tokens, int64_t n_slots, int heads,
                             int head_dim, int format, int group_size, const void *codes_k,
                             const float *scales_k, const uint8_t *zeros_k, const void *codes_v,
                             const float *scales_v, const uint8_t *zeros_v, void *K,
                             int64_t k_token_stride, int64_t k_head_stride, void *V,
                             int64_t v_token_stride, int64_t v_head_stride, int y_dtype,
                             gptq_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GPTQ_SERVE_H */
