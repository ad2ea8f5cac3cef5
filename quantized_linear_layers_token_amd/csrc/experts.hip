// The experts' MLP around its two products: the routed rows sorted by expert
// (few of them are sorted inside the gate and up product instead), and the
// weighted sum of each token's rows.
#include "w4_device.h"

namespace qlin {

namespace {

// One workgroup counts the slots of each expert, places the experts one after
// the other, and writes the slots in that order, those of one expert in the
// order of their tokens: the same for every run.  Each wavefront owns a
// contiguous share of the slots, kept in registers between the two passes
// where 1024 per wavefront hold it (16384 slots: 14.2 us; 28 with half the
// wavefronts and the ids read again, 8 loads in flight; bound by latencies).
// The counts are integer sums (LDS atomics: any order gives the same); for the
// places, lanes with equal experts find each other by one ballot per bit of
// the expert.
constexpr int kPlanWaves = 16;
constexpr int kPlanBatch = 16;       // loads in flight per lane
template <int BITS>
__global__ __launch_bounds__(kPlanWaves * 64) void experts_plan_kernel(const int32_t* __restrict__ ids, int64_t slots, int E,
                                                                      int block_rows, int* __restrict__ order,
                                                                      int* __restrict__ items, int* __restrict__ nitems) {
    constexpr int EP = 1 << BITS;
    __shared__ int count[kPlanWaves][EP];
    __shared__ int first[EP + 1], item0[EP + 1];
    __shared__ int wsum[2][kPlanWaves];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t chunks = (slots + 63) / 64, per = (chunks + kPlanWaves - 1) / kPlanWaves;
    const int64_t c0 = wave * per, c1 = c0 + per < chunks ? c0 + per : chunks;
    int id[kPlanBatch];
    auto load = [&](int64_t c) {
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) {
            const int64_t i = (c + b) * 64 + lane;
            id[b] = c + b < c1 && i < slots ? ids[i] : -1;
        }
    };
    load(c0);
    for (int i = tid; i < kPlanWaves * EP; i += kPlanWaves * 64) (&count[0][0])[i] = 0;
    __syncthreads();
    for (int64_t c = c0; c < c1; c += kPlanBatch) {
        if (c > c0) load(c);
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b)
            if ((unsigned)id[b] < (unsigned)E) atomicAdd(&count[wave][id[b]], 1);
    }
    __syncthreads();

    // per expert: rows and items, then their sums over the experts before it
    constexpr int PT = EP / (kPlanWaves * 64) > 0 ? EP / (kPlanWaves * 64) : 1;   // experts per thread
    int rows[PT], its[PT], rsum = 0, isum = 0;
#pragma unroll
    for (int p = 0; p < PT; ++p) {
        const int e = tid * PT + p;
        rows[p] = 0;
        if (e < EP)
            for (int w = 0; w < kPlanWaves; ++w) {
                const int n = count[w][e];
                count[w][e] = rows[p];
                rows[p] += n;
            }
        its[p] = (rows[p] + block_rows - 1) / block_rows;
        rsum += rows[p];
        isum += its[p];
    }
    int rpre = rsum, ipre = isum;
    for (int d = 1; d < 64; d <<= 1) {
        const int a = __shfl_up(rpre, d), b = __shfl_up(ipre, d);
        if (lane >= d) {
            rpre += a;
            ipre += b;
        }
    }
    if (lane == 63) {
        wsum[0][wave] = rpre;
        wsum[1][wave] = ipre;
    }
    __syncthreads();
    for (int w = 0; w < wave; ++w) {
        rpre += wsum[0][w];
        ipre += wsum[1][w];
    }
    int at = rpre - rsum, it = ipre - isum;
#pragma unroll
    for (int p = 0; p < PT; ++p) {
        const int e = tid * PT + p;
        if (e < EP) {
            first[e] = at;
            item0[e] = it;
        }
        at += rows[p];
        it += its[p];
    }
    if (tid == kPlanWaves * 64 - 1) {   // the last thread's sums are the totals
        first[EP] = at;
        item0[EP] = it;
        *nitems = it;
    }
    __syncthreads();
    for (int i = tid; i < item0[EP]; i += kPlanWaves * 64) {
        int e = 0;                       // the last expert with item0[e] <= i
#pragma unroll
        for (int step = EP / 2; step > 0; step >>= 1)
            if (item0[e + step] <= i) e += step;
        const int begin = first[e] + (i - item0[e]) * block_rows;
        items[3 * i] = e;
        items[3 * i + 1] = begin;
        items[3 * i + 2] = min(block_rows, first[e + 1] - begin);
    }

    for (int64_t c = c0; c < c1; c += kPlanBatch) {
        if (per > kPlanBatch) load(c);
#pragma unroll
        for (int b = 0; b < kPlanBatch; ++b) {
            const int e = id[b];
            const bool live = (unsigned)e < (unsigned)E;
            uint64_t same = __ballot(live);
            if (!same) continue;
#pragma unroll
            for (int bit = 0; bit < BITS; ++bit) {
                const bool on = (e >> bit) & 1;
                const uint64_t v = __ballot(on);
                same &= on ? v : ~v;
            }
            if (live) {
                const int before = count[wave][e];
                order[first[e] + before + __popcll(same & ((uint64_t(1) << lane) - 1))] = (int)((c + b) * 64 + lane);
                // the count moves on after every lane of the group has read it
                __builtin_amdgcn_wave_barrier();
                if (lane == __builtin_ctzll(same)) count[wave][e] = before + __popcll(same);
            }
            __builtin_amdgcn_wave_barrier();
            __threadfence_block();
        }
    }
}

// y[t] = sum_j weights[t, j] * rows[t * k + j]: four outputs per thread, the
// slots in order.  Bound by reading the f32 rows (they stay f32: one rounding
// of the sum instead of one per expert): 134 MB in 22 us.  Eight rows are read
// at once; those of slots without an expert hold anything and are dropped
// after the read.
__global__ __launch_bounds__(256) void experts_combine_kernel(const float* __restrict__ rows, const int32_t* __restrict__ ids,
                                                             const float* __restrict__ weights, int64_t T, int k, int E,
                                                             int64_t H, uint16_t* __restrict__ y) {
    const int64_t quads = H / 4, n = T * quads;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
        const int64_t t = i / quads, h = (i % quads) * 4;
        float v[4] = {};
        for (int j0 = 0; j0 < k; j0 += 8) {
            v4f r[8];
            float w[8];
            bool live[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int64_t s = t * k + min(j0 + j, k - 1);
                r[j] = *reinterpret_cast<const v4f*>(rows + s * H + h);
                w[j] = weights[s];
                live[j] = j0 + j < k && (unsigned)ids[s] < (unsigned)E;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (live[j])
#pragma unroll
                    for (int c = 0; c < 4; ++c) v[c] = __builtin_fmaf(w[j], r[j][c], v[c]);
        }
        store4_f32(y, t * H + h, v, OUT_BF16);
    }
}

}  // namespace

hipError_t launch_experts_plan(const int32_t* ids, int64_t slots, int E, int block_rows, int* order, int* items,
                               int* nitems, hipStream_t st) {
    if (E <= 64) experts_plan_kernel<6><<<1, kPlanWaves * 64, 0, st>>>(ids, slots, E, block_rows, order, items, nitems);
    else if (E <= 256) experts_plan_kernel<8><<<1, kPlanWaves * 64, 0, st>>>(ids, slots, E, block_rows, order, items, nitems);
    else experts_plan_kernel<10><<<1, kPlanWaves * 64, 0, st>>>(ids, slots, E, block_rows, order, items, nitems);
    return hipGetLastError();
}

hipError_t launch_experts_combine(const float* rows, const int32_t* ids, const float* weights, int64_t T, int k, int E,
                                  int64_t H, uint16_t* y, hipStream_t st) {
    const int64_t want = (T * (H / 4) + 255) / 256;
    experts_combine_kernel<<<(unsigned)(want < 65536 ? want : 65536), 256, 0, st>>>(rows, ids, weights, T, k, E, H, y);
    return hipGetLastError();
}

}  // namespace qlin
