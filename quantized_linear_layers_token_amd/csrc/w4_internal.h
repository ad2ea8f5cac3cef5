// Launchers of the 4-bit products, the router and the experts' MLP.  All
// arguments are validated by the caller (w4_api.hip) before a launch.
// Host declarations only.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/qlin_w4.h"

namespace qlin {

// The status of a launch; records the HIP error for qlin_last_hip_error (qlin_api.hip).
qlin_status hip_status(hipError_t e);

// Packed 4-bit weights: one matrix [N, K] is ceil(N / 16) row tiles, each
// ceil(K / 128) blocks of 1 KiB (16 rows x 128 inputs), see qlin_pack_w4.
constexpr int kW4Rows = 16;
constexpr int kW4K = 128;
constexpr int kW4Block = 1024;
inline int64_t w4_row_tiles(int64_t N) { return (N + kW4Rows - 1) / kW4Rows; }
inline int64_t w4_k_tiles(int64_t K) { return (K + kW4K - 1) / kW4K; }

constexpr int kW4Segments = 4;

// One product launch.  Dense: up to four weight matrices reading the same M
// rows of x.  Experts: one matrix (or a gate/up pair) per expert and the
// routed rows of the items below.
struct W4Call {
    const uint16_t* x;                 // bf16 [rows, K]
    const uint8_t* w[kW4Segments];     // packed codes (experts: [E] matrices)
    const uint16_t* s[kW4Segments];    // packed scales
    const uint8_t* z[kW4Segments];     // packed zero points, or null (8)
    void* y[kW4Segments];
    int n[kW4Segments];                // output rows of each matrix
    int nseg;
    int mode;                          // OutMode of y
    int group;                         // inputs per scale: 32, 64 or 128
    int64_t M, K;
    // experts
    const int* ids;                    // expert of each slot (slot = token * k + choice)
    int* order;                        // slots in the order of their experts
    int* items;                        // {expert, first place in order, rows}; null: item i is slot i alone
    int* nitems;
    int slots;                         // > 0 (gate/up, streamed): these many ids are not sorted yet: the workgroups find
                                       // their items themselves and write order, items and nitems
    int E;
    int xdiv;                          // row of x of a slot: slot / xdiv
    int64_t max_items;                 // bound of *nitems (slots where items is null)
};

hipError_t launch_pack_w4(const uint8_t* q, const uint16_t* s, const uint8_t* z, int64_t E, int64_t N, int64_t K, int group,
                          uint8_t* qp, uint16_t* sp, uint8_t* zp, hipStream_t st);

// Forms of a product, by the part of the output that a workgroup takes: rows
// of x (of one expert) times row tiles of 16 weight rows.  The first five
// stream the weights (w4_stream.hip: its eight, or four, wavefronts split the
// inputs), the last two tile (w4_tiled.hip).  In gate/up pairs half of the row
// tiles are the gate's, so the first is for single matrices only.
enum W4Form : int { kW4Stream16x1 = 0, kW4Stream16x2, kW4Stream16x4, kW4Stream16x4W4, kW4Stream32x4, kW4Tiled64x8, kW4Tiled64x16, kW4Forms };
constexpr int kW4FormRows[kW4Forms] = {16, 16, 16, 16, 32, 64, 64};
constexpr int kW4FormTiles[kW4Forms] = {1, 2, 4, 4, 4, 8, 16};
constexpr int kW4FormThreads[kW4Forms] = {512, 512, 512, 256, 512, 512, 256};
// The forms that the library holds: no row tile for the second matrix of a pair
// in the first; and with groups of 128, 16 x 4 by eight wavefronts is slower than
// by four at any size (6.0 / 5.8 against 5.9 / 5.6 in the cost table).
constexpr bool w4_form_built(int form, int group, bool pair) {
    return !(form == kW4Stream16x1 && pair) && !(form == kW4Stream16x4 && group == 128);
}

// y (or, with pair, h = silu(x w[0]^T) * (x w[1]^T)) in the given form.  Between
// the two products of the experts, the streaming forms write and read h as two
// bf16 parts, [rows][2][n]: h rounded to bf16, and what that left (16 bits of
// h; the matrix cores have the time).  The tiled forms keep the first alone.
hipError_t launch_w4_stream(int form, const W4Call& c, bool pair, bool experts, hipStream_t st);
hipError_t launch_w4_tiled(int form, const W4Call& c, bool pair, bool experts, hipStream_t st);

// Workgroups of a launch: token blocks (items) times parts of the row tiles.
inline int64_t w4_units(int form, const W4Call& c, bool pair) {
    const int per = kW4FormTiles[form] / (pair ? 2 : 1);
    int64_t u = 0;
    for (int i = 0; i < (pair ? 1 : c.nseg); ++i) u += (w4_row_tiles(c.n[i]) + per - 1) / per;
    return u;
}
inline int64_t w4_blocks(int form, const W4Call& c, bool experts) {
    return experts ? c.max_items : (c.M + kW4FormRows[form] - 1) / kW4FormRows[form];
}

hipError_t launch_route(const void* logits, bool f32, int64_t T, int E, int k, int score, const float* bias, int groups,
                        int top_groups, int group_best, bool renorm, float scale, int32_t* ids, float* weights,
                        hipStream_t st);

// The streaming forms of gate and up find their items by themselves up to these sizes.
constexpr int kOwnItemSlots = 512, kOwnItemExperts = 256;

// The routed rows sorted by expert and cut into items of at most block_rows
// rows of one expert.  order [T * k], items [3 * max_items], nitems [1].
hipError_t launch_experts_plan(const int32_t* ids, int64_t slots, int E, int block_rows, int* order, int* items,
                               int* nitems, hipStream_t st);
// y[t] = sum_j weights[t, j] * rows[t * k + j] over the slots with an expert.
hipError_t launch_experts_combine(const float* rows, const int32_t* ids, const float* weights, int64_t T, int k, int E,
                                  int64_t H, uint16_t* y, hipStream_t st);
// The down projection and the weighted sum of few tokens in one launch.
hipError_t launch_experts_down_direct(const W4Call& c, const float* weights, int64_t T, int k, uint16_t* y,
                                      hipStream_t st);

}  // namespace qlin
