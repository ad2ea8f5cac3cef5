// Products of few rows on 4-bit weights: every weight byte is read once per
// block of tokens, straight into the matrix-core operand registers.
//
//   y[m, n] = sum_g s[n, g] * ( sum_{k in g} x[m, k] * code[n, k]  -  z[n, g] * sum_{k in g} x[m, k] )
//
// Bound by HBM at few tokens (half a byte per weight).  One wavefront takes R
// tiles of 16 weight rows and a share of the inputs; the NW wavefronts of a
// workgroup split the inputs and add their partial sums through LDS in a fixed
// order.  The packed order makes every weight load 1 KiB contiguous per
// wavefront, and lets one 16x16x32 bf16 product take eight codes of a lane
// after seven instructions of widening.  The matrix cores are idle otherwise,
// so the sums of x that the zero points need are a product with a constant
// operand: of -8 where there are no zero points, and its result is then the
// start value of every tile's sum.  Groups are summed in f32 and scaled in f32.
// One token, 2 x 14336 x 4096: 12.5 us, 4.8 TB/s (a large copy's rate); 4096 x
// 4096: 4.4 us, where an empty kernel takes 2.8.
// With more tokens x weighs too, which every workgroup reads whole: 4096 x 14336
// takes 9.9 us for one token, 13.4 - 15 for 13, 17 for 16.  The L1s set the pace
// there: 0.82 accesses per CU and clock at 13 rows, 0.84 at 16, 0.49 at one (each
// line of x is asked of the L2s once per workgroup, no more).
#include "w4_device.h"

namespace qlin {

namespace {

constexpr int kAux = 2;   // buffer-load cache policy: streaming

// Sum over the lanes up to and with this one: shifts by 1, 2, 4, 8 in the rows
// of 16 lanes, then the last lane of a row added to the rows after it.
__device__ __forceinline__ int lane_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
    return v;
}

// The item `block` of the ids (rows of one expert, ROWS at most, experts and
// slots in order), found by one wavefront for itself: the experts counted in
// `hist` (64 * ceil(E / 64) ints), items and rows summed over the lanes, which
// own ceil(E / 64) consecutive experts each, and the slots of the item's expert
// found by ballots, into `list`.  rows = 0: no such item.  total: their number;
// place: rows before this item.  (About 1 us per workgroup; a launch that sorts
// costs 3.9 us and three loads in turn to read what it found.  Done again by the
// second product it gains nothing: that one reads what the first wrote down.)
template <int ROWS>
__device__ __forceinline__ void own_item(const int* __restrict__ ids, int slots, int E, int block, int lane, int* hist, int* list,
                                         int& expert, int& rows, int& place, int& total) {
    constexpr int B = kOwnItemSlots / 64;
    const int per = (E + 63) >> 6;
    int id[B];
#pragma unroll
    for (int b = 0; b < B; ++b) id[b] = b * 64 + lane < slots ? ids[b * 64 + lane] : -1;
    for (int p = 0; p < per; ++p) hist[p * 64 + lane] = 0;
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
#pragma unroll
    for (int b = 0; b < B; ++b)
        if ((unsigned)id[b] < (unsigned)E) atomicAdd(&hist[id[b]], 1);
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
    int mine = 0;                         // items in the upper half, rows in the lower
    for (int p = 0; p < per; ++p) {
        const int n = hist[lane * per + p];
        mine += ((n + ROWS - 1) / ROWS << 16) + n;
    }
    const int upto = lane_scan(mine);
    const uint64_t past = __ballot((upto >> 16) > block);
    total = __builtin_amdgcn_readlane(upto, 63) >> 16;
    rows = expert = place = 0;
    if (past == 0) return;
    const int who = __builtin_ctzll(past);
    const int before = __builtin_amdgcn_readlane(upto - mine, who);
    int base = before >> 16, count = 0;
    place = before & 0xFFFF;
    for (int p = 0; p < per; ++p) {       // (ends at the item's expert: it is one of this lane's)
        expert = who * per + p;
        count = __builtin_amdgcn_readfirstlane(hist[expert]);
        const int items = (count + ROWS - 1) / ROWS;
        if (block < base + items) break;
        base += items;
        place += count;
    }
    const int begin = (block - base) * ROWS;
    place += begin;
    rows = min(ROWS, count - begin);
    int seen = -begin;
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const uint64_t same = __ballot(id[b] == expert);
        const int at = seen + __popcll(same & ((uint64_t(1) << lane) - 1));
        if (id[b] == expert && at >= 0 && at < ROWS) list[at] = b * 64 + lane;
        seen += __popcll(same);
    }
    __builtin_amdgcn_wave_barrier();
    __threadfence_block();
}

// D: blocks of 128 inputs whose loads are in flight per wavefront.
template <int G, int MT, int R, int NW, int D, bool ZP, bool PAIR, bool EXPERTS>
__global__ __launch_bounds__(NW * 64, 2) void w4_stream_kernel(W4Call c, int KT, int units, int units0, int units1, int units2) {
    constexpr int SUB = kW4K / G;                 // groups in a 128-input block
    constexpr int SL = G / 32;                    // 32-input slices of a group
    constexpr int T = MT * 16;
    constexpr int RM = PAIR ? R / 2 : R;          // row tiles of each matrix
    constexpr int P = EXPERTS && !PAIR ? 2 : 1;   // bf16 parts of an input (the experts' h comes in two)
    __shared__ __attribute__((aligned(16))) float red[NW * R * T * 16];
    __shared__ int own[PAIR && EXPERTS ? NW : 1][T];   // the rows of an item that the wavefronts found

    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int q = lane >> 4, col = lane & 15;

    // the matrix and its first row tile
    const int block = (int)(blockIdx.x / (unsigned)units);   // token block or item
    int unit = (int)(blockIdx.x % (unsigned)units), seg = 0;
    if constexpr (!PAIR && !EXPERTS) {
        if (unit >= units0) { unit -= units0; seg = 1; }
        if (seg == 1 && unit >= units1) { unit -= units1; seg = 2; }
        if (seg == 2 && unit >= units2) { unit -= units2; seg = 3; }
    }
    const int N = PAIR || EXPERTS ? c.n[0] : pick_int(c.n, seg);
    const int tiles = (N + 15) >> 4;
    const int tile0 = unit * RM;
    const int K = (int)c.K;

    // the rows of x
    int e = 0, begin = 0, rows;
    int64_t m0 = 0;
    if constexpr (EXPERTS) {
        if (PAIR && c.slots > 0) {
            // counted in this wavefront's part of `red`, which it writes only at the end; those of the
            // first row tiles write the item down for the second product
            static_assert(R * T * 16 >= kOwnItemExperts, "counts fit the wavefront's sums");
            int total;
            own_item<T>(c.ids, c.slots, c.E, block, lane, reinterpret_cast<int*>(red) + wave * (R * T * 16), own[wave], e, rows, begin,
                        total);
            if (unit == 0 && wave == 0) {
                if (block == 0 && lane == 0) *c.nitems = total;
                if (rows > 0 && lane < 3) c.items[3 * block + lane] = lane == 0 ? e : lane == 1 ? begin : rows;
                if (lane < rows) c.order[begin + lane] = own[0][lane];
            }
            if (rows == 0) return;
        } else if (!PAIR || c.items) {            // (the down product of single slots is another kernel)
            if (block >= *c.nitems) return;
            e = c.items[3 * block];
            begin = c.items[3 * block + 1];
            rows = c.items[3 * block + 2];
        } else {
            e = c.ids[block];
            if ((unsigned)e >= (unsigned)c.E) return;
            rows = 1;
        }
    } else {
        m0 = (int64_t)block * T;
        rows = (int)min((int64_t)T, c.M - m0);
    }
    auto row_of = [&](int t) -> int64_t {         // output row of the block's row t
        if constexpr (EXPERTS) return PAIR && c.slots > 0 ? (int64_t)own[wave][t] : !PAIR || c.items ? (int64_t)c.order[begin + t] : (int64_t)block;
        else return m0 + t;
    };
    Global<uint16_t> xp[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int64_t r = row_of(min(mt * 16 + col, rows - 1));
        xp[mt] = (Global<uint16_t>)c.x + (PAIR && EXPERTS ? r / c.xdiv : r) * (P * K) + q * 8;
    }

    // this wavefront's share of the inputs: n blocks from k0.  Descriptors that
    // cover just those: blocks past them read as zeros, codes and scales.
    const int per = (KT + NW - 1) / NW;
    const int k0 = min(wave * per, KT), n = min(per, KT - k0);
    __amdgpu_buffer_rsrc_t dw[R], ds[R], dz[R];
    uint32_t z_fill[R];                           // added to what was read: 0, or 8 for every group
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int m = PAIR ? r / RM : seg, tile = min(tile0 + r % RM, tiles - 1);
        const int64_t at = ((int64_t)e * tiles + tile) * KT + k0;
        dw[r] = uniform_rsrc(pick_ptr(c.w, m) + at * kW4Block, n * kW4Block);
        ds[r] = uniform_rsrc(pick_ptr(c.s, m) + at * 16 * SUB, n * 32 * SUB);
        if constexpr (ZP) {
            const uint8_t* z = pick_ptr(c.z, m);
            z_fill[r] = z ? 0u : 0x08080808u;
            dz[r] = uniform_rsrc(z ? z + at * 16 * SUB : nullptr, z ? n * 16 * SUB : 0);
        }
    }
    const int last = K / 32 - 1;                  // the last slice of 32 inputs
    const v8bf ones = bf16_const(ZP ? -1.0f : -8.0f);
    v4f tot[R][MT] = {};

    v4u w[D][R];
    v8bf a[D][MT][P][4];
    W4Scales<SUB> s[D][R];
    uint32_t z[D][R];
    auto load = [&](int d, int i) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[d][r] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(dw[r], i * kW4Block + lane * 16, 0, kAux));
            s[d][r].load(ds[r], (i * 16 + col) * 2 * SUB, 0);
            if constexpr (ZP) z[d][r] = w4_zeros<SUB>(dz[r], (i * 16 + col) * SUB, 0);   // without zero points: 0
        }
        __builtin_amdgcn_sched_barrier(0);        // the weights first: they come from HBM
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int p = 0; p < P; ++p) a[d][mt][p][j] = *(Global<v8bf>)(xp[mt] + p * K + 32 * min(4 * (k0 + i) + j, last));
    };
    auto multiply = [&](int d) {
#pragma unroll
        for (int g = 0; g < SUB; ++g) {           // (groups past K have scales of zero)
            v4f c0[MT] = {};
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int p = 0; p < P; ++p)
#pragma unroll
                    for (int j = 0; j < SL; ++j) c0[mt] = mfma_bf16(a[d][mt][p][g * SL + j], ones, c0[mt]);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                v4f acc[MT];
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    acc[mt] = c0[mt];
                    if constexpr (ZP) {
                        const float zf = (float)(((again(z[d][r]) + z_fill[r]) >> (8 * g)) & 255u);
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[mt][i] *= zf;
                    }
                }
#pragma unroll
                for (int j = 0; j < SL; ++j) {
                    const v8bf b = w4_codes(w[d][r][g * SL + j]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int p = 0; p < P; ++p) acc[mt] = mfma_bf16(a[d][mt][p][g * SL + j], b, acc[mt]);
                }
                W4Scales<SUB> t = s[d][r];
                if constexpr (SUB > 1) t.v[g >> 1] = again(t.v[g >> 1]);
                const float sf = t.at(g);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) tot[r][mt][i] = __builtin_fmaf(sf, acc[mt][i], tot[r][mt][i]);
            }
            // one group at a time: else the start values of all of them take registers at once
            if constexpr (SUB > 1) __builtin_amdgcn_sched_barrier(0);
        }
    };
    // one loop exit: with one after every block the compiler waits for every
    // load in flight at the top of the loop
#pragma unroll
    for (int d = 0; d < D; ++d) {
        load(d, d);
        __builtin_amdgcn_sched_barrier(0);
    }
    int i = 0;
    for (; i + D < n; i += D) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            multiply(d);
            __builtin_amdgcn_sched_barrier(0);
            load(d, i + D + d);
            __builtin_amdgcn_sched_barrier(0);
        }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
        if (i + d < n) multiply(d);

#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = mt * 16 + 4 * q + i;
                if (t < rows) red[(wave * R + r) * (T * 16) + t * 16 + col] = tot[r][mt][i];
            }
    __syncthreads();
    auto sum = [&](int r, int at) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) v += red[(i * R + r) * (T * 16) + at];
        return v;
    };
    constexpr int W = 16 * RM;                    // outputs of one row
    for (int idx = tid; idx < rows * W; idx += NW * 64) {
        const int t = idx / W, n = idx % W, r = n / 16;
        const int nn = tile0 * 16 + n;
        if (nn >= N) continue;
        const int at = t * 16 + (n & 15);
        const int64_t o = row_of(t) * (PAIR && EXPERTS ? 2 * (int64_t)N : (int64_t)N) + nn;
        if constexpr (PAIR) {
            const float h = swiglu_f32(sum(r, at), sum(r + RM, at));
            uint16_t* y = static_cast<uint16_t*>(c.y[0]);
            const uint16_t hi = f32_to_bf16(h);
            y[o] = hi;
            if constexpr (EXPERTS) y[o + N] = f32_to_bf16(h - bf16_lo(hi));
        } else store_f32(EXPERTS ? c.y[0] : pick_ptr(c.y, seg), o, sum(r, at), c.mode);
    }
}

// The down projection of few tokens with the weighted sum over their experts:
//   y[t, n] = sum_j weights[t, j] * sum_k h[t * k + j, k] * w[ids[t, j]][n, k].
// A workgroup takes one token and 16 output rows; its wavefronts share out the
// (slot, 128-input block) pairs, so that a single token still keeps every load
// of its 16 rows in flight, and no row of a slot passes through memory.  The
// operand's 16 rows are the two parts of h in turn: the sums of rows 0 and 1
// are those of one part each.  Eight slots of 2048 x 1024: 8.0 us (7.1 at
// best, 1.2 TB/s: one round of workgroups, so the latency of its loads bounds it).
template <int G, int NW, bool ZP>
__global__ __launch_bounds__(NW * 64) void w4_down_direct_kernel(W4Call c, int KT, int units, const float* __restrict__ weights,
                                                                 int k, uint16_t* __restrict__ y) {
    constexpr int SUB = kW4K / G, SL = G / 32, U = 4;
    __shared__ float red[NW * 16];
    const int tid = threadIdx.x;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lane = tid & 63;
    const int q = lane >> 4, col = lane & 15;
    const int64_t t = blockIdx.x / (unsigned)units;
    const int tile = (int)(blockIdx.x % (unsigned)units);
    const int N = c.n[0], K = (int)c.K, NG = K / G, slices = K >> 5;
    const int id = lane < k ? c.ids[t * k + lane] : -1;
    const float wt = lane < k ? weights[t * k + lane] : 0.0f;

    const int all = k * KT, per = (all + NW - 1) / NW;
    const int f0 = wave * per, f1 = min(all, f0 + per);
    const v8bf ones = bf16_const(ZP ? -1.0f : -8.0f);
    float tot = 0.0f;
    for (int f = f0; f < f1; f += U) {
        v4u w[U];
        v8bf a[U][4];
        W4Scales<SUB> s[U];
        uint32_t z[U];
        float wu[U];
        int kb[U];
        bool live[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = min(f + u, f1 - 1), j = at / KT;
            kb[u] = at - j * KT;
            const int e = __builtin_amdgcn_readlane(id, j);
            wu[u] = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(wt), j));
            live[u] = (unsigned)e < (unsigned)c.E && f + u < f1;
            const int64_t ee = live[u] ? e : 0;    // a slot without an expert reads expert 0 and is dropped
            w[u] = __builtin_nontemporal_load(
                reinterpret_cast<const v4u*>(c.w[0] + ((ee * units + tile) * KT + kb[u]) * kW4Block + lane * 16));
            const uint16_t* xr = c.x + ((t * k + j) * 2 + (col & 1)) * (int64_t)K + q * 8;
#pragma unroll
            for (int i = 0; i < 4; ++i) a[u][i] = *reinterpret_cast<const v8bf*>(xr + 32 * min(4 * kb[u] + i, slices - 1));
            const int64_t sat = (((ee * units + tile) * KT + kb[u]) * 16 + col) * SUB;
            s[u].load((Global<uint16_t>)c.s[0] + sat);
            if constexpr (ZP) z[u] = w4_zeros<SUB>((Global<uint8_t>)c.z[0] + sat);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!live[u]) continue;
            float part = 0.0f;
#pragma unroll
            for (int g = 0; g < SUB; ++g) {
                if (kb[u] * SUB + g >= NG) break;
                v4f acc = {};
#pragma unroll
                for (int j = 0; j < SL; ++j) acc = mfma_bf16(a[u][g * SL + j], ones, acc);
                if constexpr (ZP) acc *= (float)((z[u] >> (8 * g)) & 255u);
#pragma unroll
                for (int j = 0; j < SL; ++j) acc = mfma_bf16(a[u][g * SL + j], w4_codes(w[u][g * SL + j]), acc);
                part = __builtin_fmaf(s[u].at(g), acc[0] + acc[1], part);
            }
            tot = __builtin_fmaf(wu[u], part, tot);
        }
    }
    if (q == 0) red[wave * 16 + col] = tot;
    __syncthreads();
    if (tid < 16 && tile * 16 + tid < N) {
        float v = 0.0f;
#pragma unroll
        for (int i = 0; i < NW; ++i) v += red[i * 16 + tid];
        y[t * N + tile * 16 + tid] = f32_to_bf16(v);
    }
}

template <int G>
hipError_t run_down_direct(const W4Call& c, const float* weights, int64_t T, int k, uint16_t* y, hipStream_t st) {
    constexpr int NW = 16;
    const int KT = (int)w4_k_tiles(c.K), units = (int)w4_row_tiles(c.n[0]);
    const unsigned grid = (unsigned)(T * units);
    if (c.z[0]) w4_down_direct_kernel<G, NW, true><<<grid, NW * 64, 0, st>>>(c, KT, units, weights, k, y);
    else w4_down_direct_kernel<G, NW, false><<<grid, NW * 64, 0, st>>>(c, KT, units, weights, k, y);
    return hipGetLastError();
}

template <int G, int FORM, int NW, int D, bool PAIR, bool EXPERTS>
hipError_t run(const W4Call& c, hipStream_t st) {
    constexpr int MT = kW4FormRows[FORM] / 16, R = kW4FormTiles[FORM], RM = PAIR ? R / 2 : R;
    static_assert(NW * 64 == kW4FormThreads[FORM], "threads of the form");
    const int KT = (int)w4_k_tiles(c.K);
    const int64_t units = w4_units(FORM, c, PAIR);
    int u[kW4Segments] = {0, 0, 0, 0};
    bool zp = false;
    for (int i = 0; i < c.nseg; ++i) {
        u[i] = (int)((w4_row_tiles(c.n[i]) + RM - 1) / RM);
        zp |= c.z[i] != nullptr;
    }
    const unsigned grid = (unsigned)(w4_blocks(FORM, c, EXPERTS) * units);
    if (zp)
        w4_stream_kernel<G, MT, R, NW, D, true, PAIR, EXPERTS><<<grid, NW * 64, 0, st>>>(c, KT, (int)units, u[0], u[1], u[2]);
    else
        w4_stream_kernel<G, MT, R, NW, D, false, PAIR, EXPERTS><<<grid, NW * 64, 0, st>>>(c, KT, (int)units, u[0], u[1], u[2]);
    return hipGetLastError();
}

template <int G, bool PAIR, bool EXPERTS>
hipError_t by_form(int form, const W4Call& c, hipStream_t st) {
    constexpr int D4 = 2;   // two blocks of four row tiles: too many registers with more scales
    if constexpr (w4_form_built(kW4Stream16x1, G, PAIR))
        if (form == kW4Stream16x1) return run<G, kW4Stream16x1, 8, 2, PAIR, EXPERTS>(c, st);
    if (form <= kW4Stream16x2) return run<G, kW4Stream16x2, 8, 2, PAIR, EXPERTS>(c, st);
    if constexpr (w4_form_built(kW4Stream16x4, G, PAIR))
        if (form == kW4Stream16x4) return run<G, kW4Stream16x4, 8, 1, PAIR, EXPERTS>(c, st);
    if (form == kW4Stream16x4W4) return run<G, kW4Stream16x4W4, 4, D4, PAIR, EXPERTS>(c, st);
    return run<G, kW4Stream32x4, 8, 1, PAIR, EXPERTS>(c, st);
}

template <bool PAIR, bool EXPERTS>
hipError_t by_group(int form, const W4Call& c, hipStream_t st) {
    if (c.group == 32) return by_form<32, PAIR, EXPERTS>(form, c, st);
    if (c.group == 64) return by_form<64, PAIR, EXPERTS>(form, c, st);
    return by_form<128, PAIR, EXPERTS>(form, c, st);
}

// Row-major weights to the packed order: one thread per packed dword of
// codes, then one per scale.
__global__ __launch_bounds__(256) void pack_w4_kernel(const uint8_t* __restrict__ q, const uint16_t* __restrict__ s,
                                                      const uint8_t* __restrict__ z, int64_t N, int64_t K, int G, int tiles,
                                                      int KT, int64_t blocks, uint32_t* __restrict__ qp,
                                                      uint16_t* __restrict__ sp, uint8_t* __restrict__ zp) {
    const int64_t first = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
    for (int64_t i = first; i < blocks * 256; i += step) {
        const int j = (int)(i & 3), lane = (int)(i >> 2) & 63;
        const int64_t blk = i >> 8, rest = blk / KT;
        const int64_t n = (rest % tiles) * 16 + (lane & 15);
        const int64_t k = (blk % KT) * 128 + 32 * j + 8 * (lane >> 4);
        uint32_t out = 0;
        if (n < N && k < K) {   // K % 32 == 0: the eight inputs are there together
            const uint8_t* src = q + ((rest / tiles) * N + n) * (K / 2) + k / 2;
            uint32_t in = 0;
#pragma unroll
            for (int b = 0; b < 4; ++b) in |= (uint32_t)src[b] << (8 * b);
#pragma unroll
            for (int b = 0; b < 4; ++b) {
                out |= ((in >> (4 * b)) & 15u) << (8 * b);
                out |= ((in >> (16 + 4 * b)) & 15u) << (8 * b + 4);
            }
        }
        qp[i] = out;
    }
    const int sub = 128 / G;
    for (int64_t i = first; i < blocks * 16 * sub; i += step) {
        const int64_t blk = i / (16 * sub), rest = blk / KT;
        const int64_t n = (rest % tiles) * 16 + (i / sub) % 16, g = (blk % KT) * sub + i % sub;
        const bool in = n < N && g < K / G;
        const int64_t at = ((rest / tiles) * N + n) * (K / G) + g;
        sp[i] = in ? s[at] : 0;
        if (zp) zp[i] = in ? z[at] : 0;
    }
}

}  // namespace

hipError_t launch_pack_w4(const uint8_t* q, const uint16_t* s, const uint8_t* z, int64_t E, int64_t N, int64_t K, int group,
                          uint8_t* qp, uint16_t* sp, uint8_t* zp, hipStream_t st) {
    const int64_t blocks = E * w4_row_tiles(N) * w4_k_tiles(K);   // one thread block per block at most
    pack_w4_kernel<<<(unsigned)(blocks < 65536 ? blocks : 65536), 256, 0, st>>>(
        q, s, z, N, K, group, (int)w4_row_tiles(N), (int)w4_k_tiles(K), blocks, reinterpret_cast<uint32_t*>(qp), sp, zp);
    return hipGetLastError();
}

hipError_t launch_w4_stream(int form, const W4Call& c, bool pair, bool experts, hipStream_t st) {
    if (pair) return experts ? by_group<true, true>(form, c, st) : by_group<true, false>(form, c, st);
    return experts ? by_group<false, true>(form, c, st) : by_group<false, false>(form, c, st);
}

hipError_t launch_experts_down_direct(const W4Call& c, const float* weights, int64_t T, int k, uint16_t* y,
                                      hipStream_t st) {
    if (c.group == 32) return run_down_direct<32>(c, weights, T, k, y, st);
    if (c.group == 64) return run_down_direct<64>(c, weights, T, k, y, st);
    return run_down_direct<128>(c, weights, T, k, y, st);
}

}  // namespace qlin
