// Products of many rows on 4-bit weights, tiled for the matrix cores, in two
// forms of 64 rows of x (BM) by 64 RT weight rows per workgroup:
//   64 x 16 row tiles (RT = 4, KG = 1): four wavefronts, 256 weight rows;
//   64 x 8 row tiles (RT = 2, KG = 2): two groups of four wavefronts, 128 weight
//     rows; each group takes half of the input blocks with copies of x of its
//     own, and the groups' sums are added through those copies at the end.  Half
//     of the reuse of x and of the widened codes, for twice the workgroups: it is
//     for sizes whose 64 x 16 tiles leave CUs idle.
//
// Bound by the matrix cores, next by the vector instructions that widen the
// codes (seven per eight codes) and scale the group sums (four per 16 x 16
// tile and group): both are shared by more tiles the larger a wavefront's part
// is.  A wavefront takes 16 RT weight rows and all rows of x: its codes come
// straight from the packed order into registers, are widened once per
// 128-input block and used for every row of x; the rows of x pass through LDS,
// copied there in operand order without passing through registers, so that a
// read is 16 contiguous bytes per lane.  The sums of x that the zero points
// need are products with a constant operand, one token tile per wavefront,
// shared through LDS.  64 x 16, 2048 x 4096 x 14336: 233 - 246 us, 1.0 PFLOP/s, the
// matrix cores busy for half of the cycles at the 1.8 GHz that their power allows
// (the library's bf16 product of that shape: 224 us); 64 experts of 2048 x 1024 with
// 16384 rows: 166 - 187 us for gate and up, 109 - 117 for down.
#include "w4_device.h"

namespace qlin {

namespace {

constexpr int kPanelGroup = 8;   // panels that take turns on the same rows of x (their weights stay in the XCD's L2)

constexpr int kItemGroup = 4;    // items that take turns on the same panel

template <int G, int RT, int KG, bool ZP, bool PAIR, bool EXPERTS>
__global__ __launch_bounds__(256 * KG, 2) void w4_tiled_kernel(W4Call c, int KT, int panels, int panels0, int panels1, int panels2,
                                                          int row_blocks) {
    constexpr int SUB = kW4K / G, SL = G / 32;
    constexpr int MT = 4, BM = MT * 16;
    static_assert(KG == 1 || RT <= 2, "a group's sums fit its copies of x");
    // two distinct arrays: the compiler then knows which one a copy writes
    __shared__ __attribute__((aligned(1024))) uint8_t x0[KG * BM * 256], x1[KG * BM * 256];
    __shared__ __attribute__((aligned(16))) float cs_all[KG * SUB * BM];

    const int tid = threadIdx.x;
    const int grp = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
    const int wave = __builtin_amdgcn_readfirstlane((tid >> 6) & 3);   // in its group
    const int lane = tid & 63;
    const int q = lane >> 4, col = lane & 15;

    // Workgroup b runs on XCD b % 8.  Dense: each XCD takes a contiguous part of
    // the tiles, ordered so that kPanelGroup panels run over the same rows of x.
    // Experts: kItemGroup items in a row (most often one expert's) to an XCD, so
    // that they read its weights there once, and the XCDs in turn, so that each
    // has its share however many items there are.
    const int b = blockIdx.x;
    int panel, block, seg = 0;
    if constexpr (EXPERTS) {
        const int at = b >> 3, group = at / (kItemGroup * panels), in_group = at - group * (kItemGroup * panels);
        panel = __builtin_amdgcn_readfirstlane(in_group / kItemGroup);
        block = __builtin_amdgcn_readfirstlane((group * 8 + (b & 7)) * kItemGroup + in_group % kItemGroup);
        if (block >= *c.nitems) return;
    } else {
        const int ntiles = row_blocks * panels;
        const int per = ntiles >> 3, extra = ntiles & 7, xcd = b & 7;
        const int t = xcd * per + min(xcd, extra) + (b >> 3);
        const int band = t / (kPanelGroup * row_blocks);
        const int width = min(kPanelGroup, panels - band * kPanelGroup);
        const int in_band = t - band * kPanelGroup * row_blocks;
        block = __builtin_amdgcn_readfirstlane(in_band / width);
        panel = __builtin_amdgcn_readfirstlane(band * kPanelGroup + in_band % width);
    }
    if constexpr (!PAIR && !EXPERTS) {
        if (panel >= panels0) { panel -= panels0; seg = 1; }
        if (seg == 1 && panel >= panels1) { panel -= panels1; seg = 2; }
        if (seg == 2 && panel >= panels2) { panel -= panels2; seg = 3; }
    }
    const int N = PAIR || EXPERTS ? c.n[0] : pick_int(c.n, seg);
    const int tiles = (N + 15) >> 4;
    const int K = (int)c.K, slices = K >> 5;

    int e = 0, begin = 0, rows;
    int64_t m0 = 0;
    if constexpr (EXPERTS) {
        e = c.items[3 * block];
        begin = c.items[3 * block + 1];
        rows = c.items[3 * block + 2];
    } else {
        m0 = (int64_t)block * BM;
        rows = (int)min((int64_t)BM, c.M - m0);
    }
    auto row_of = [&](int r) -> int64_t {
        if constexpr (EXPERTS) return (int64_t)c.order[begin + r];
        else return m0 + r;
    };

    // the rows of x that this wavefront copies: one token tile
    const int64_t xr = row_of(min(wave * 16 + col, rows - 1));
    const uint16_t* xp = c.x + (EXPERTS ? xr / c.xdiv : xr) * K + q * 8;
    // this group's copies, sums and blocks of inputs
    float* cs = cs_all + grp * (SUB * BM);
    const int share = (KT + KG - 1) / KG;
    const int kb0 = min(grp * share, KT - 1), nb = max(0, min(share, KT - grp * share));
    // this wavefront's row tiles (SwiGLU: two of the gate, the same two of up);
    // those past the matrix read its last tile and are not stored.  The offset
    // of a block goes into the scalar offset of a buffer load, which the
    // descriptor does not check: it stays inside the matrix by itself.
    constexpr int NM = PAIR ? 2 : 1, RM = RT / NM;   // matrices, row tiles of each
    const int tile0 = (panel * 4 + wave) * RM;
    const int first = min(tile0, tiles - 1), last = min(RM, tiles - first) - 1;
    __amdgpu_buffer_rsrc_t dw[NM], ds[NM], dz[NM];
    uint32_t z_fill[NM];         // added to what was read: 0, or 8 for every group
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        const int64_t at = ((int64_t)e * tiles + first) * KT;
        const int blocks = (last + 1) * KT;
        const int i = PAIR ? m : seg;
        dw[m] = uniform_rsrc(pick_ptr(c.w, i) + at * kW4Block, blocks * kW4Block);
        ds[m] = uniform_rsrc(pick_ptr(c.s, i) + at * 16 * SUB, blocks * 32 * SUB);
        if constexpr (ZP) {
            const uint8_t* z = pick_ptr(c.z, i);
            z_fill[m] = z ? 0u : 0x08080808u;
            dz[m] = uniform_rsrc(z ? z + at * 16 * SUB : nullptr, z ? blocks * 16 * SUB : 0);
        }
    }

    auto copy_x = [&](int kb, uint8_t* xs) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            __builtin_amdgcn_global_load_lds(
                (const __attribute__((address_space(1))) void*)(xp + 32 * min(4 * kb + j, slices - 1)),
                (__attribute__((address_space(3))) void*)(xs + grp * (BM * 256) + (wave * 4 + j) * 1024), 16, 0, 0);
    };
    // scales and zero points stay packed until they are used
    v4u w[RT];
    W4Scales<SUB> s[RT], sn[RT];
    uint32_t z[RT], zn[RT];
    auto load_w = [&](int kb) {
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            const int m = r / RM, b = min(r % RM, last) * KT + kb;
            w[r] = __builtin_bit_cast(v4u, __builtin_amdgcn_raw_buffer_load_b128(dw[m], lane * 16, b * kW4Block, 0));
            sn[r].load(ds[m], col * 2 * SUB, b * 32 * SUB);
            if constexpr (ZP) zn[r] = w4_zeros<SUB>(dz[m], col * SUB, b * 16 * SUB);   // without zero points: 0
        }
    };
    auto x_at = [&](const uint8_t* xs, int mt, int j) {
        return *reinterpret_cast<const v8bf*>(xs + grp * (BM * 256) + (mt * 4 + j) * 1024 + lane * 16);
    };

    const v8bf ones = bf16_const(ZP ? -1.0f : -8.0f);
    v4f tot[RT][MT] = {};
    v8bf codes[RT][4], a[2][SL];
    v4f c0[2], acc[RT];
    // A unit is one group of one token tile.  While its products run, the next
    // unit's operands are read from LDS and the previous unit's sums are scaled.
    constexpr int UNITS = MT * SUB;
    auto read = [&](const uint8_t* xs, int u) {
        const int mt = u / SUB, g = u % SUB;
#pragma unroll
        for (int j = 0; j < SL; ++j) a[u & 1][j] = x_at(xs, mt, g * SL + j);
        c0[u & 1] = *reinterpret_cast<const v4f*>(cs + g * BM + mt * 16 + 4 * q);
    };
    auto multiply = [&](int u) {
        const int g = u % SUB;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            acc[r] = c0[u & 1];
            if constexpr (ZP) {
                const float zf = (float)((again(z[r]) >> (8 * g)) & 255u);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[r][i] *= zf;
            }
        }
#pragma unroll
        for (int j = 0; j < SL; ++j)
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r] = mfma_bf16(a[u & 1][j], codes[r][g * SL + j], acc[r]);
    };
    auto scale = [&](int u) {
        const int mt = u / SUB, g = u % SUB;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            W4Scales<SUB> t = s[r];
            if constexpr (SUB > 1) t.v[g >> 1] = again(t.v[g >> 1]);
            const float sf = t.at(g);
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[r][mt][i] = __builtin_fmaf(sf, acc[r][i], tot[r][mt][i]);
        }
    };
    // block i of the group's share
    auto step = [&](int i, const uint8_t* xs, uint8_t* xn) {
        const int next = kb0 + max(0, min(i + 1, nb - 1));   // the copies past the share go unused
        __builtin_amdgcn_sched_barrier(0);
        // this block's copies and weights have landed, and nobody reads xn any more
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        // the sums of x of this wavefront's token tile
#pragma unroll
        for (int g = 0; g < SUB; ++g) {
            v4f v = {};
#pragma unroll
            for (int j = 0; j < SL; ++j) v = mfma_bf16(x_at(xs, wave, g * SL + j), ones, v);
            if (col == 0) *reinterpret_cast<v4f*>(cs + g * BM + wave * 16 + 4 * q) = v;
        }
        __builtin_amdgcn_sched_barrier(0);
        copy_x(next, xn);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
#pragma unroll
            for (int j = 0; j < 4; ++j) codes[r][j] = w4_codes(w[r][j]);
            s[r] = sn[r];
            if (i >= nb) s[r] = W4Scales<SUB>{};   // steps past the share add nothing
            if constexpr (ZP) z[r] = zn[r] + z_fill[r / RM];
        }
        __builtin_amdgcn_sched_barrier(0);
        load_w(next);
        // the sums are in LDS; the copies stay in flight
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        __builtin_amdgcn_sched_barrier(0);
        read(xs, 0);
#pragma unroll
        for (int u = 0; u < UNITS; ++u) {
            if (u + 1 < UNITS) read(xs, u + 1);
            __builtin_amdgcn_sched_barrier(0);
            multiply(u);
            scale(u);
            __builtin_amdgcn_sched_barrier(0);
        }
        // the sums are done here: left to itself, the compiler moves their last
        // additions past the next barrier and keeps every product until then
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) asm volatile("" : "+v"(tot[r][mt]));
    };
    copy_x(kb0, x0);
    load_w(kb0);
    // one loop exit: with one after every step the compiler drains every load
    // in flight at the top of the loop
    for (int i = 0; i < share; i += 2) {
        step(i, x0, x1);
        step(i + 1, x1, x0);
    }
    __builtin_amdgcn_s_waitcnt(0x0F70);           // the copies past the last block have landed

    // the groups' sums, in their order, each group for a part of the token tiles
    if constexpr (KG > 1) {
        __syncthreads();
        auto at = [&](int g, int r, int mt) {
            return reinterpret_cast<v4f*>((r ? x1 : x0) + g * (BM * 256) + (wave * MT + mt) * 1024 + lane * 16);
        };
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) *at(grp, r, mt) = tot[r][mt];
        __syncthreads();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (mt % KG != grp) continue;
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                v4f v = *at(0, r, mt);
#pragma unroll
                for (int g = 1; g < KG; ++g) {
                    const v4f o = *at(g, r, mt);
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += o[i];
                }
                tot[r][mt] = v;
            }
        }
    }

    __attribute__((address_space(1))) void* y = (__attribute__((address_space(1))) void*)pick_ptr(c.y, seg);
    auto store = [&](auto put) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            if (KG > 1 && mt % KG != grp) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r0 = mt * 16 + 4 * q + i;
                if (r0 >= rows) continue;
                const int64_t o = row_of(r0) * N;
#pragma unroll
                for (int r = 0; r < RM; ++r) {
                    const int n = (tile0 + r) * 16 + col;
                    if (n < N) put(o + n, r, mt, i);
                }
            }
        }
    };
    // The experts' h is rounded to one bf16 here (2^-8 of it; y's error against 64
    // bits 1.7e-3 -> 2.3e-3): a second part would double the matrix products of down.
    if constexpr (PAIR)
        store([&](int64_t at, int r, int mt, int i) {
            ((__attribute__((address_space(1))) uint16_t*)y)[at] =
                f32_to_bf16(swiglu_f32(tot[r][mt][i], tot[r + RM][mt][i]));
        });
    else if (c.mode == OUT_F32)
        store([&](int64_t at, int r, int mt, int i) { ((__attribute__((address_space(1))) float*)y)[at] = tot[r][mt][i]; });
    else
        store([&](int64_t at, int r, int mt, int i) { ((__attribute__((address_space(1))) uint16_t*)y)[at] = f32_to_bf16(tot[r][mt][i]); });
}

template <int G, int FORM, bool PAIR, bool EXPERTS>
hipError_t run(const W4Call& c, hipStream_t st) {
    constexpr int RT = kW4FormTiles[FORM] / 4, KG = kW4FormThreads[FORM] / 256, PT = kW4FormTiles[FORM] / (PAIR ? 2 : 1);
    const int KT = (int)w4_k_tiles(c.K), panels = (int)w4_units(FORM, c, PAIR), blocks = (int)w4_blocks(FORM, c, EXPERTS);
    int p[kW4Segments] = {0, 0, 0, 0};
    bool zp = false;
    for (int i = 0; i < c.nseg; ++i) {
        p[i] = (int)((w4_row_tiles(c.n[i]) + PT - 1) / PT);
        zp |= c.z[i] != nullptr;
    }
    constexpr int64_t round = 8 * kItemGroup;
    const unsigned grid = (unsigned)((EXPERTS ? (blocks + round - 1) / round * round : (int64_t)blocks) * panels);
    if (zp) w4_tiled_kernel<G, RT, KG, true, PAIR, EXPERTS><<<grid, 256 * KG, 0, st>>>(c, KT, panels, p[0], p[1], p[2], blocks);
    else w4_tiled_kernel<G, RT, KG, false, PAIR, EXPERTS><<<grid, 256 * KG, 0, st>>>(c, KT, panels, p[0], p[1], p[2], blocks);
    return hipGetLastError();
}

template <bool PAIR, bool EXPERTS, int G>
hipError_t by_form(int form, const W4Call& c, hipStream_t st) {
    if (form == kW4Tiled64x8) return run<G, kW4Tiled64x8, PAIR, EXPERTS>(c, st);
    return run<G, kW4Tiled64x16, PAIR, EXPERTS>(c, st);
}

template <bool PAIR, bool EXPERTS>
hipError_t by_group(int form, const W4Call& c, hipStream_t st) {
    if (c.group == 32) return by_form<PAIR, EXPERTS, 32>(form, c, st);
    if (c.group == 64) return by_form<PAIR, EXPERTS, 64>(form, c, st);
    return by_form<PAIR, EXPERTS, 128>(form, c, st);
}

}  // namespace

hipError_t launch_w4_tiled(int form, const W4Call& c, bool pair, bool experts, hipStream_t st) {
    if (pair) return experts ? by_group<true, true>(form, c, st) : by_group<true, false>(form, c, st);
    return experts ? by_group<false, true>(form, c, st) : by_group<false, false>(form, c, st);
}

}  // namespace qlin
