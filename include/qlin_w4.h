/*
 * qlin, 4-bit weights and experts: projections on 4-bit weights with group
 * scales, routing to experts, and the experts' gated MLP on 4-bit weights.
 *
 * The conventions of qlin.h hold for every entry point here (device pointers
 * owned by the caller, no allocation and no synchronization, work enqueued on
 * `stream`, which belongs to the current device, arguments checked before any
 * launch, bf16 as uint16 bit patterns, errors returned as qlin_status), with
 * these additions:
 *
 *  - A 4-bit weight matrix [N, K] has one code 0..15 per weight, one bf16 scale
 *    per `group` consecutive inputs of a row (group 32, 64 or 128; K a multiple
 *    of it) and either one zero point (uint8) per scale or 8 for all of them:
 *        w[n, k] = (code[n, k] - zero[n, k / group]) * scale[n, k / group]
 *    K is a multiple of 32 and at most QLIN_MAX_K; the rows N of a call's
 *    matrices (of the two of a gate/up pair together) are any number up to
 *    QLIN_MAX_MN, its outputs (the experts': T * k rows of the longer of H and I)
 *    up to 2^40 (QLIN_ERR_SHAPE).
 *  - The activations are bf16 and not rounded (the numerics of
 *    qlin_linear_weight_only): products of inputs and codes are exact, sums are
 *    f32 per group, scaled in f32 and added in f32.
 *  - Results do not depend on what else runs: the same call gives the same bits.
 *  - A row of x with an infinity or NaN, or with values past 2^112 in magnitude
 *    (whose sums, or the experts' h, leave f32), gives values that are not finite, or unspecified, in
 *    its own rows of the result and nowhere else.
 */
#ifndef QLIN_W4_H_
#define QLIN_W4_H_

#include "qlin.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------------- */
/* Layout                                                                 */
/* ---------------------------------------------------------------------- */

/* Bytes of the codes of one matrix [N, K] in the packed order: rows are padded
 * to a multiple of 16, inputs to a multiple of 128 (0 for sizes out of range). */
int64_t qlin_w4_packed_bytes(int64_t N, int64_t K);
/* Scales (and zero points) of one matrix in the packed order. */
int64_t qlin_w4_packed_scales(int64_t N, int64_t K, int32_t group);

/* E matrices of row-major codes q_w [E, N, K / 2] (byte i of a row: input 2 i
 * in the low four bits, 2 i + 1 in the high four), scales s_w and zero points
 * z_w [E, N, K / group] (z_w null: none) into the order that the matrix cores
 * read, one matrix after the other.  A block is 16 rows x 128 inputs; block
 * (n / 16) * ceil(K / 128) + k / 128 of a matrix holds
 *   codes, 1024 bytes: dword j < 4 of lane l < 64, at byte 16 l + 4 j, has row
 *     l % 16, inputs 32 j + 8 (l / 16) + 0..7 of the block: its byte b has input b
 *     of those in the low four bits and input 4 + b in the high four;
 *   scales and zero points, 16 * (128 / group) entries each: row by row.
 * Padding is written as zeros.  q_w and q_w_packed are 16-byte aligned, s_w 2,
 * s_w_packed 8, z_w_packed 4; nothing overlaps; z_w and z_w_packed are both
 * null or neither.  Every call below reads this one layout, for one token as
 * for long inputs: the row-major weights need not be kept. */
qlin_status qlin_pack_w4(const uint8_t* q_w, const uint16_t* s_w, const uint8_t* z_w, int64_t E, int64_t N, int64_t K,
                         int32_t group, uint8_t* q_w_packed, uint16_t* s_w_packed, uint8_t* z_w_packed,
                         hipStream_t stream);

/* A packed matrix, or E of them one after the other. */
typedef struct qlin_w4_weight {
    const uint8_t* q_w;   /* packed codes, 16-byte aligned */
    const uint16_t* s_w;  /* packed scales, 8-byte aligned */
    const uint8_t* z_w;   /* packed zero points, 4-byte aligned, or null: every zero point is 8 */
    int64_t n;            /* rows N of each matrix */
} qlin_w4_weight;

/* ---------------------------------------------------------------------- */
/* Projections                                                            */
/* ---------------------------------------------------------------------- */

/* y[i][m, n] = sum_k x[m, k] w_i[n, k] for the nw (1..QLIN_MAX_SEGMENTS)
 * matrices that read the same input: x bf16 [M, K], 16-byte aligned; y[i]
 * [M, weights[i].n], 16-byte aligned, in the type `out` (QLIN_OUT_BF16, rounded
 * to nearest even, or QLIN_OUT_F32).  Any M; one launch.  M == 0 or no rows: no-op.
 * Outputs may not overlap each other or any input (QLIN_ERR_ALIAS).  Both
 * arrays are read during the call only. */
qlin_status qlin_linear_w4(const uint16_t* x, int64_t M, int64_t K, int32_t group, const qlin_w4_weight* weights,
                           void* const* y, int32_t nw, qlin_out out, hipStream_t stream);

/* Gate/up pair of a gated MLP: h[m, j] = bf16(silu(g) * u), g = x W_gate^T and
 * u = x W_up^T in f32, rounded once (qlin_linear_swiglu rounds g, u and silu(g)
 * to bf16 as well; here nothing but h is).  Both matrices [I, K] (equal n);
 * h bf16 [M, I], 16-byte aligned.  Otherwise as qlin_linear_w4. */
qlin_status qlin_linear_swiglu_w4(const uint16_t* x, int64_t M, int64_t K, int32_t group, const qlin_w4_weight* gate,
                                  const qlin_w4_weight* up, uint16_t* h, hipStream_t stream);

/* ---------------------------------------------------------------------- */
/* Experts                                                                */
/* ---------------------------------------------------------------------- */

#define QLIN_MAX_EXPERTS 1024
#define QLIN_MAX_CHOICES 32
#define QLIN_MAX_GROUPS 64

typedef enum qlin_score {
    QLIN_SCORE_SOFTMAX = 0,  /* over the token's E logits */
    QLIN_SCORE_SIGMOID = 1   /* of each logit; 0 below a logit of -708, where f64 ends */
} qlin_score;

/* Chooses k of E experts for each of T tokens.
 *   logits [T, E], bf16 (logits_type QLIN_OUT_BF16) or f32 (QLIN_OUT_F32);
 *   score[e]: softmax or sigmoid of the token's logits;
 *   choice[e] = score[e] + bias[e] (bias f32 [E], or null);
 *   groups > 1: the experts form `groups` runs of E / groups; a run's worth is
 *     the sum of the group_best (1 or 2) largest choices of its experts that are
 *     not masked out (one alone counts alone), the top_groups runs of the largest
 *     worth stay and no expert of another run is chosen; a run whose experts are
 *     all masked out comes after every other run;
 *   ids[t, 0..k): the experts with the k largest choices, largest first;
 *   weights[t, j] = scale * score[ids[t, j]], divided by the sum of the token's
 *     k chosen scores if renormalize (0 where that sum is 0).
 * Equal choices or worths: the lowest index first.  Scores and choices are
 * evaluated in f64, and where the order of the choices is that of the logits
 * (no bias; no groups, or group_best 1) they are compared as logits: the choice
 * does not depend on rounding.  An expert whose logit is -infinity or NaN is
 * masked out: score 0, its bias counts for nothing, and it comes after every
 * other expert of the runs that stay (in index order, so ids are always k
 * different experts); +infinity counts as the largest finite value, a bias of
 * +infinity or -infinity as the largest or smallest one, a bias of NaN as the
 * smallest.  A token whose experts are all masked out gets weights 0.
 * 1 <= k <= min(QLIN_MAX_CHOICES, top_groups * E / groups), E <= QLIN_MAX_EXPERTS,
 * groups <= QLIN_MAX_GROUPS a divisor of E, 1 <= top_groups <= groups
 * (QLIN_ERR_SHAPE).  logits aligned to their type, ids and weights to 4 bytes.
 * T == 0 is a no-op. */
qlin_status qlin_route(const void* logits, qlin_out logits_type, int64_t T, int64_t E, int32_t k, qlin_score score,
                       const float* bias, int32_t groups, int32_t top_groups, int32_t group_best, int32_t renormalize,
                       float scale, int32_t* ids, float* weights, hipStream_t stream);

/* Bytes of the workspace of qlin_experts_w4 (0 for sizes out of range and for no tokens).  They
 * grow with T: a workspace for T tokens serves any fewer. */
int64_t qlin_experts_w4_workspace(int64_t T, int32_t k, int64_t E, int64_t H, int64_t I);

/* The gated MLP of the chosen experts, summed with the router's weights:
 *   y[t] = bf16( sum_j weights[t, j] * W_down[e] h_j ),  e = ids[t, j],
 *   h_j = silu(W_gate[e] x_t) * (W_up[e] x_t)
 * over the slots j whose ids[t, j] is in [0, E); any other id (e.g. -1 for
 * tokens that pad a batch, or experts that live elsewhere) adds nothing, and a
 * token without experts gets zeros.  An expert may be chosen twice.  h is the
 * only value rounded on the way (it is a matrix-core operand): to bf16 where
 * many rows share an expert's weights and the matrix cores bound the call, to
 * two bf16 parts (16 bits) where they do not.  The sums are f32 in a fixed order:
 * that over the experts in the order of j, but for few tokens, whose slots are
 * multiplied one by one: there consecutive shares of the (j, input) pairs are
 * summed with the weights applied, and then added in order.
 *   x bf16 [T, H]; ids [T, k], weights f32 [T, k] (qlin_route writes both);
 *   gate, up: E matrices [I, H]; down: E matrices [H, I]; one group size for
 *   all three (H and I multiples of it); y bf16 [T, H].
 *   workspace: qlin_experts_w4_workspace bytes, 16-byte aligned; its contents
 *   before and after a call mean nothing.  Calls that may run at the same time
 *   need workspaces of their own.
 * T * k is at most QLIN_MAX_MN.  T == 0 is a no-op. */
qlin_status qlin_experts_w4(const uint16_t* x, int64_t T, int64_t H, int64_t I, int64_t E, int32_t k, int32_t group,
                            const int32_t* ids, const float* weights, const qlin_w4_weight* gate,
                            const qlin_w4_weight* up, const qlin_w4_weight* down, uint16_t* y, void* workspace,
                            hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_W4_H_ */
