// Launchers of the norm, rotary, cache and attention kernels.  All arguments
// are validated by the caller (layer_api.hip) before a launch.  Host
// declarations only.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/qlin_layer.h"

namespace qlin {

// The status of a launch; records the HIP error for qlin_last_hip_error (qlin_api.hip).
qlin_status hip_status(hipError_t e);

enum NormOut : int { kNormBf16 = 0, kNormInt8 = 1, kNormFp8 = 2, kNormFp8Block = 3 };
struct NormCall {
    const uint16_t* x;
    const uint16_t* residual;   // or null
    const uint16_t* gamma;
    uint16_t* sum;              // null where residual is
    void* y;                    // bf16 values or codes
    float* s;
    int64_t M, K;
    float eps;
};
hipError_t launch_norm(NormOut out, const NormCall& c, hipStream_t st);

// Queries, keys and values of T tokens; a part that a call lacks has no heads.
struct HeadsCall {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    uint16_t* q_out;
    int64_t q_out_stride;
    const uint16_t *q_gamma, *k_gamma;   // or null
    float eps, inv_dim;
    const int* positions;
    const int* slots;
    qlin_rotation rope;                  // frequencies null: no rotation
    qlin_kv_cache cache;
    int heads, kv_heads, dim;
    int64_t T;
};
hipError_t launch_heads(const HeadsCall& c, hipStream_t st);
hipError_t launch_cache_read(const qlin_kv_cache& cache, const int* slots, int64_t n, uint16_t* k, uint16_t* v, hipStream_t st);

struct AttnCall {
    const uint16_t* q;
    qlin_kv_cache cache;
    const int* pages;
    const int* lengths;
    uint16_t* out;
    void* workspace;
    int S, heads, columns, window;
    float scale;
};
constexpr int kAttnHeads = 16;   // query heads of one kv head that a workgroup takes: columns of the matrix instruction
struct AttnShape {
    int tiles;      // groups of query heads per kv head
    int rows;       // query heads of a group (of the last one: at most)
    int workers;    // workgroups that share the tokens of a group of heads
};
AttnShape attn_shape(int heads, int kv_heads, int dim);
int64_t attn_workspace(int heads, int kv_heads, int dim);
hipError_t launch_attn(const AttnCall& c, hipStream_t st);

}  // namespace qlin
