/*
 * qlin, between the projections of a decoder layer: the RMS norm that adds the
 * residual and rounds for the next projection, rotary positions, a paged
 * key-value cache in 8 bits, and the attention of one new token over it.
 *
 * The conventions of qlin.h hold for every entry point here (device pointers
 * owned by the caller, no allocation and no synchronization, work enqueued on
 * `stream`, which belongs to the current device, arguments checked before any
 * launch, bf16 as uint16 bit patterns, errors returned as qlin_status), with
 * these additions:
 *
 *  - Heads are `dim` channels long, a multiple of 16 from 16 to 256.  Heads of
 *    one token are contiguous, [heads, dim]; a stride between tokens is counted
 *    in elements, is a multiple of 8 and at least heads * dim, so that q, k and
 *    v may be parts of the rows of one projection's output.
 *  - Positions, slots, lengths and page numbers are int32 arrays on the device
 *    and are not known to the host: what they name outside its range is skipped
 *    as stated, never accessed.
 *  - Codes of values t with absmax a and range Q (127: int8, 448: E4M3) are
 *    those of the activation quantizers of qlin.h but for the last bit of inv,
 *    which is a reciprocal and a product here:
 *      inv = fl32(Q * fl32(1 / a)) (0 if a == 0),
 *      code = round_half_even(fl32(t * inv)), saturated to -Q .. Q,
 *    with t and a scaled by 2^64 first for a < 2^-64; the scale is a / Q.
 *  - Sums, softmax statistics and angles are f32 or f64.  Results do not depend
 *    on what else runs: the same call gives the same bits.
 *  - Inputs that are not finite, or past 2^55 in magnitude, give unspecified
 *    values in the rows (heads, sequences) that contain them and nowhere else.
 *    They do not vanish in 8 bits: the scale of a head (token, group) that is
 *    rounded with a NaN or an infinity in it is NaN, and so is all that is read
 *    of it.
 */
#ifndef QLIN_LAYER_H_
#define QLIN_LAYER_H_

#include "qlin.h"

#ifdef __cplusplus
extern "C" {
#endif

#define QLIN_MAX_HEADS 1024
#define QLIN_MAX_HEAD_DIM 256

/* ---------------------------------------------------------------------- */
/* Norm                                                                   */
/* ---------------------------------------------------------------------- */

/* For each row of x (bf16 [M, K], K as for the products of qlin.h):
 *   r = bf16(x + residual), written to sum      (residual null: r = x, sum null)
 *   t[k] = r[k] * gamma[k]                      (exact in f32)
 *   d = 1 / sqrt(mean_k r[k]^2 + eps)
 *   qlin_norm_bf16: y[k] = bf16(t[k] * d)
 *   qlin_norm_int8: per token, the codes q[k] of t[k] as stated above for
 *                   Q = 127, a = max_k |t[k]|, and s = a * d / 127
 *   qlin_norm_fp8:  the same with E4M3 codes and Q = 448, per token (group 0)
 *                   or per 128 inputs (group 128, aligned at k = 128 g)
 * (the codes are those of the normalised row t * d, before any rounding to
 * bf16: d cancels out of them).  q and s feed qlin_gemm_* as the activation
 * quantizers' do; y feeds the calls that do not round their input.
 * gamma bf16 [K]; residual and sum bf16 [M, K], both or neither; sum may be
 * residual or x itself (an update in place) and overlaps nothing otherwise.
 * x, residual, gamma, sum, y and q 16-byte aligned, s 4.  eps from 1e-20 to 1
 * (QLIN_ERR_UNSUPPORTED).  M == 0 is a no-op. */
qlin_status qlin_norm_bf16(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, int64_t M, int64_t K,
                           float eps, uint16_t* sum, uint16_t* y, hipStream_t stream);
qlin_status qlin_norm_int8(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, int64_t M, int64_t K,
                           float eps, uint16_t* sum, int8_t* q, float* s, hipStream_t stream);
qlin_status qlin_norm_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, int64_t M, int64_t K,
                          float eps, int32_t group, uint16_t* sum, uint8_t* q, float* s, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Rotary positions                                                       */
/* ---------------------------------------------------------------------- */

/* Channels 0..dims of a head form dims / 2 pairs; pair i (channels i and
 * i + dims / 2, or 2 i and 2 i + 1 where interleaved) is rotated by the angle
 * position * frequencies[i] and multiplied by strength:
 *   (a, b) -> strength * (a cos - b sin, b cos + a sin)
 * The other channels stay.  Angles are formed and reduced in f64: a position of
 * 10^6 is as exact as one of 10. */
typedef struct qlin_rotation {
    const double* frequencies; /* device, f64 [dims / 2], 8-byte aligned */
    int32_t dims;              /* a multiple of 16, at most dim */
    int32_t interleaved;       /* 0: halves, 1: neighbours */
    float strength;            /* factor of cosine and sine, 1 where there is none */
} qlin_rotation;

/* y[t, h] = the rotation of x[t, h] by positions[t], rounded once to bf16.
 * gamma (bf16 [dim], or null): the head is first divided by its root mean
 * square and multiplied by gamma, h / sqrt(mean h^2 + eps) * gamma.
 * x [T, heads, dim] and y with their strides; y may be x (same stride), and
 * overlaps nothing otherwise.  x, y and gamma 16-byte aligned, positions 4. */
qlin_status qlin_rope(const uint16_t* x, int64_t x_stride, const int32_t* positions, int64_t T, int32_t heads, int32_t dim,
                      const qlin_rotation* rope, const uint16_t* gamma, float eps, uint16_t* y, int64_t y_stride,
                      hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Cache                                                                  */
/* ---------------------------------------------------------------------- */

typedef enum qlin_cache_kind {
    QLIN_CACHE_BF16 = 0, /* not rounded further, no scales */
    QLIN_CACHE_INT8 = 1, /* int8 codes and one f32 scale per token and head, absmax / 127 */
    QLIN_CACHE_FP8 = 2   /* E4M3 codes and one f32 scale per token and head, absmax / 448 */
} qlin_cache_kind;

/* Keys and values of one layer, [pages, kv_heads, page_size, dim], 16-byte
 * aligned; scales [pages, kv_heads, page_size], 16-byte aligned (null for bf16).
 * Slot p * page_size + i is place i of page p.  A page holds consecutive tokens
 * of one sequence (a prefix's pages may be read by several): token j of a
 * sequence is in place j % page_size of the page that its table names at
 * j / page_size.  page_size is a multiple of 16; pages * page_size at most
 * 2^31 - 1 (QLIN_ERR_SHAPE). */
typedef struct qlin_kv_cache {
    void* k;
    void* v;
    float* k_scale;
    float* v_scale;
    int64_t pages;
    int32_t kv_heads;
    int32_t page_size;
    int32_t dim;
    int32_t kind; /* qlin_cache_kind */
} qlin_kv_cache;

/* The queries of a qlin_cache_write. */
typedef struct qlin_queries {
    const uint16_t* q; /* bf16 [T, heads, dim], 16-byte aligned */
    int64_t stride;
    const uint16_t* gamma; /* as k_gamma, or null */
    uint16_t* out;         /* bf16 [T, heads, dim], 16-byte aligned; may be q (same stride) */
    int64_t out_stride;
    int32_t heads;
} qlin_queries;

/* Writes token t's keys and values (bf16 [T, kv_heads, dim], 16-byte aligned,
 * with their strides) to slots[t], and rotates its queries, in one launch:
 *   keys: as qlin_rope with k_gamma (bf16 [dim], or null) and rope (null: no
 *     rotation), not rounded in between, then rounded as the cache's kind says,
 *     with one scale for the dim values of a head;
 *   values: rounded as the cache's kind says;
 *   queries (null: none; needs rope or a gamma, QLIN_ERR_NULL): as qlin_rope.
 * A slot outside 0..pages * page_size - 1 (-1 for rows that pad a batch) is not
 * written; that token's queries are rotated all the same.  The slots of a call
 * differ: a slot that is named twice holds a mixture of its tokens.
 * positions int32 [T], read where rope is given (null otherwise). */
qlin_status qlin_cache_write(const qlin_kv_cache* cache, const int32_t* slots, int64_t T, const uint16_t* k, int64_t k_stride,
                             const uint16_t* v, int64_t v_stride, const int32_t* positions, const qlin_rotation* rope,
                             const uint16_t* k_gamma, float eps, const qlin_queries* queries, hipStream_t stream);

/* k[i], v[i] = bf16(code * scale) of slots[i], for i < n: bf16
 * [n, kv_heads, dim], 16-byte aligned.  Rows whose slot is outside the cache
 * are left as they were. */
qlin_status qlin_cache_read(const qlin_kv_cache* cache, const int32_t* slots, int64_t n, uint16_t* k, uint16_t* v,
                            hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Attention of one new token                                             */
/* ---------------------------------------------------------------------- */

/* Bytes of the workspace of qlin_attn_decode (0 for sizes out of range): the
 * same for any number of sequences and any lengths. */
int64_t qlin_attn_decode_workspace(int32_t heads, int32_t kv_heads, int32_t dim);

/* For each of S sequences and each of its heads (head h reads kv head
 * h / (heads / kv_heads)):
 *   out[s, h] = bf16( sum_j p_j v_j ),  p = softmax_j(scale * q[s, h] . k_j)
 * over its tokens j < n = lengths[s], of these the last `window` where window
 * is not 0.  The new token's own key and value are written before the call
 * (qlin_cache_write) and counted in lengths.
 *   lengths[s] == 0: out[s] is zero; negative: out[s] is left as it was (rows
 *     that pad a batch); past page_columns * page_size: taken as that;
 *   pages int32 [S, page_columns]: page of tokens i * page_size .. of a
 *     sequence; entries behind its length (or before its window) are not used;
 *     tokens of a page outside the cache are left out of the softmax (none
 *     left: zero).
 * q, out bf16 [S, heads, dim], 16-byte aligned, out overlapping nothing.
 * Products q . k are exact, sums f32; p * v_scale (p of at most 1, before it is
 * divided by its sum) is a matrix-core operand and kept as two bf16 parts: off
 * by 2^-17 of it or by 2^-134, which is more below 2^-117.
 * page_columns * page_size is at most 2^30.
 * workspace: qlin_attn_decode_workspace bytes, 16-byte aligned; its contents
 * before and after a call mean nothing.  Calls that may run at the same time
 * need workspaces of their own. */
qlin_status qlin_attn_decode(const uint16_t* q, const qlin_kv_cache* cache, const int32_t* pages, int64_t S, int32_t heads,
                             int64_t page_columns, const int32_t* lengths, int64_t window, float scale, uint16_t* out,
                             void* workspace, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_LAYER_H_ */
