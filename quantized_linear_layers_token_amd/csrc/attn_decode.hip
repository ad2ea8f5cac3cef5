// Attention of one new token per sequence over the paged cache, split over the
// tokens and joined.
//
// The cache is read once and bounds the call; everything else is arranged
// around a steady stream of its rows.  A step of a wavefront takes 32 tokens
// of one kv head and all query heads that read it (up to 16):
//   S^T = K q^T   on 16x16x32 bf16 matrix instructions, K's rows straight from
//                 memory as the first operand (codes widened to bf16, exactly),
//                 so that a lane gets the scores of one head and 8 tokens;
//   p = 2^(s - m) with the running maximum m of the head, in f32;
//   O^T += V^T p^T  with the lane's own 8 tokens as its share of the inner
//                 index: p never leaves the lane, and V's transpose is a
//                 permutation of bytes within the lane (8 tokens x 4, 8 or 16
//                 channels), done while its codes are widened.
// The scale of a key multiplies its scores, that of a value its p.  p is split
// in two bf16 parts (the matrix cores have the time: about a tenth of theirs
// is used), which leaves 2^-17 of it.
//
// Work is cut in items (attn_index.h), one to a workgroup, so that they are
// about even whatever the lengths: a workgroup finds its own by a scan of the
// lengths.  A sequence of one item is finished by it; of one of several each
// item writes a partial sum, and a second launch joins them.  So the launches do
// not depend on the lengths and can be captured.  Where no sequence can be long,
// or there are a great many, an item is a sequence and there is one launch.
//
// Measured: 206744 tokens of 8 sequences (32 / 8 heads of 128, E4M3, 436 MB)
// 85.9 us, 5.1 TB/s, the rate of a large copy; equal lengths 5.4 TB/s, bf16 5.7.
// What is left of the time is fixed: 5 us for a short sequence in one launch
// (lengths, page table and rows are three dependent loads), 2 for the second
// launch, 1.5 to 2 more where it joins something.  A sequence of 777 tokens takes
// 9.5 to 10 us (its kernels 7.2 and 3.0), 37 ragged ones in bf16 (57 MB) 17.
// In earlier states of the loop two units of every wavefront under way instead
// of one changed nothing (101.3 -> 101.5 us for 8 x 32768 tokens) or cost up to
// a fifth (128 x 1024 tokens of 4 kv heads of 64: 16.8 -> 20.8), and eight
// wavefronts to a workgroup instead of four 40 % of 64 x 256 tokens.
#include <type_traits>

#include "attn_index.h"
#include "layer_device.h"
#include "layer_forms.h"

namespace qlin {

namespace {

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef unsigned v8u __attribute__((ext_vector_type(8)));

constexpr int kWaves = kAttnWaves;
constexpr int kThreads = kWaves * kWave;
constexpr int kTries = 4;                     // for a size of items that fits the card
constexpr float kNone = -__builtin_inff();    // score of no token

struct AttnArgs {
    const uint16_t* q;
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const int *pages, *lengths;
    uint16_t* out;
    float* sums;      // partial sums [group of heads][2 workers][rows][dim]: those of a split sequence follow each other
    float* stats;     // their maxima and sums of p [group of heads][2 workers][rows][2]
    int* joins;       // [group of heads]: 4 ints, the number of partial sums first, then for each {sequence, its first, their number, 0}
    int64_t npages;
    int S, heads, kv_heads, shared_by, dim, columns, page_size, page_shift, window;   // shared_by: query heads of a kv head
    int tiles, rows, workers;
    int least;        // items are not cut below so many units
    float scale;      // times log2 e
};

// Page tables and lengths are read through the scalar cache: a vector load
// between those of the tiles would wait for all that were issued before it.
typedef const __attribute__((address_space(4))) int* Table;
__device__ __forceinline__ Table table_of(const int* p) { return (Table)(uintptr_t)p; }

__device__ __forceinline__ AttnSpan span_of(int length, const AttnArgs& a) {
    return attn_span(length, a.columns, a.page_size, a.window);
}

__device__ __forceinline__ v4f mfma(v8bf a, v8bf b, v4f c) { return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0); }

// Slots between the last matrix instruction and the first read of its result
// (one more than the four passes of a 16x16x32 need on this machine).
__device__ __forceinline__ void settle() {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// Maximum and sum over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float column_max(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float column_sum(float v) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

__device__ __forceinline__ uint32_t bits(v2bf v) { return __builtin_bit_cast(uint32_t, v); }
__device__ __forceinline__ v8bf operand(uint32_t a, uint32_t b, uint32_t c, uint32_t d) { return __builtin_bit_cast(v8bf, v4u{a, b, c, d}); }

// Byte I of w, a signed integer, as f32 (one instruction; the compiler takes two or three).
template <int I>
__device__ __forceinline__ float signed_byte(uint32_t w) {
    float f;
    if constexpr (I == 0) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_0" : "=v"(f) : "v"(w));
    if constexpr (I == 1) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_1" : "=v"(f) : "v"(w));
    if constexpr (I == 2) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_2" : "=v"(f) : "v"(w));
    if constexpr (I == 3) asm("v_cvt_f32_i32_sdwa %0, sext(%1) dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:BYTE_3" : "=v"(f) : "v"(w));
    return f;
}

// Codes as bf16, exactly: a pair of bytes of w (E4M3: by one instruction;
// int8: by way of f32, whose upper halves are the bf16 values).
template <int KIND, bool HI>
__device__ __forceinline__ uint32_t widen_pair(uint32_t w) {
    if constexpr (KIND == QLIN_CACHE_FP8) {
        return bits(__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
    } else {
        const float a = signed_byte<HI ? 2 : 0>(w), b = signed_byte<HI ? 3 : 1>(w);
        return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302);
    }
}

// 8 channels of a row as an operand of S^T.
template <int KIND>
__device__ __forceinline__ v8bf key_operand(uint32_t a, uint32_t b) {
    return operand(widen_pair<KIND, false>(a), widen_pair<KIND, true>(a), widen_pair<KIND, false>(b), widen_pair<KIND, true>(b));
}

// Head length DP = 64, 128 or 256 in registers; heads of dim < DP channels
// read some channels twice, against zeros of q and without a place in out.
template <int KIND, int DP>
struct Tiles {
    static constexpr int kBytes = KIND == QLIN_CACHE_BF16 ? 2 : 1;
    static constexpr int kKeyChunks = DP / 4 * kBytes / 16;    // 16-byte chunks of a row per lane
    static constexpr int kValueDwords = DP / 16 * kBytes / 4;  // dwords of a row per lane
    v4u key[2][kKeyChunks];
    uint32_t value[8][kValueDwords];
    v4f key_scale[2], value_scale[2];
};

template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t (&to)[N]) {
    if constexpr (N == 1) {
        to[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (N == 2) {
        const v2u t = *reinterpret_cast<const v2u*>(p);
        to[0] = t.x, to[1] = t.y;
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const v4u t = reinterpret_cast<const v4u*>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) to[4 * i + j] = t[j];
        }
    }
}

// Inclusive sums over the wavefront's lanes (each at most 2^25: no overflow).
__device__ __forceinline__ unsigned scan(unsigned v) {
    auto add = [](unsigned v, unsigned o) { return v + o; };
    v = add(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));
    v = add(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
    v = add(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
    v = add(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
    v = add(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));   // lane 15 (47) to the next row
    v = add(v, (unsigned)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));   // lane 31 to the upper rows
    return v;
}
__device__ __forceinline__ unsigned lane_of(unsigned v, int lane) { return (unsigned)__builtin_amdgcn_readlane((int)v, lane); }

// Wavefronts of a SIMD that the registers are bounded to; no form spills.  Heads
// of 256 channels with two and with one, 16 x 4096 tokens of 16 / 8 heads: int8
// 57.5 and 59.8 us, E4M3 56.9 and 56.3, bf16 108 (19 registers spilled) and 99.
constexpr int waves_per_simd(int dp, bool bf16) { return dp == 64 ? 4 : dp == 128 ? 3 : bf16 ? 1 : 2; }

// ALONE: a workgroup takes a whole sequence, and nothing is joined.
template <int KIND, int DP, int WAVES, bool ALONE>
__global__ __launch_bounds__(WAVES * kWave, waves_per_simd(DP, KIND == QLIN_CACHE_BF16)) void attn_kernel(AttnArgs a) {
    using T = Tiles<KIND, DP>;
    constexpr int kTiles = DP / 16, kSteps = DP / 32;
    constexpr int kPad = DP + 4;
    constexpr int kSlots = WAVES / 2 < 4 ? WAVES / 2 : 4;
    __shared__ float joined[kSlots][kAttnHeads * kPad];
    __shared__ float stats[kSlots][2][kAttnHeads];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int n = lane & 15, g = lane >> 4;
    const int group = blockIdx.x, worker = blockIdx.y;
    const int kv_head = a.tiles == 1 ? group : group / a.tiles, tile = a.tiles == 1 ? 0 : group % a.tiles;
    const int head0 = kv_head * a.shared_by + tile * kAttnHeads;
    const int rows = min(a.rows, a.shared_by - tile * kAttnHeads);
    AttnSpan span = {};
    int s = 0, first = 0, last = 0, record = -1;   // the item: a sequence and its units; its partial sum (-1: the whole sequence)
    if constexpr (ALONE) {
        s = worker;
        span = span_of(table_of(a.lengths)[s], a);
        last = (int)span.units;
    } else {
        auto length_at = [&](int c) { return c + lane < a.S ? a.lengths[c + lane] : -1; };
        AttnSpan of_lane = span_of(length_at(0), a);
        int64_t total = lane_of(scan(of_lane.units), kWave - 1);
        for (int c = kWave; c < a.S; c += kWave) total += lane_of(scan(span_of(length_at(c), a).units), kWave - 1);
        unsigned most = attn_most(total, a.workers, a.least);
        if (a.S <= kWave && a.S < a.workers) {   // as many items as workers at most: even on the CUs
            for (int k = 0; k < kTries; ++k) {
                const unsigned n = lane_of(scan(attn_items(of_lane.units, most)), kWave - 1);
                if (n <= (unsigned)a.workers) break;
                most = attn_larger(most, n, a.workers);
            }
        }
        unsigned items = 0, split = 0;   // of the sequences before a chunk of 64: items, and those of split sequences
        bool found = false;
        for (int c = 0; c < a.S; c += kWave) {
            if (c) of_lane = span_of(length_at(c), a);
            const unsigned n = attn_items(of_lane.units, most), upto = scan(n), split_upto = scan(n > 1 ? n : 0);
            const uint64_t past = __ballot(items + upto > (unsigned)worker);
            if (past) {
                const int at = __builtin_ctzll(past);
                const unsigned of = lane_of(n, at), i = worker - (items + lane_of(upto, at) - of);
                s = c + at;
                span = AttnSpan{(int)lane_of(of_lane.n, at), (int)lane_of(of_lane.start, at), lane_of(of_lane.units, at)};
                first = (int)attn_first_unit(span.units, of, i), last = (int)attn_first_unit(span.units, of, i + 1);
                if (of > 1) {
                    const int begin = (int)(split + lane_of(split_upto, at) - of);
                    record = begin + (int)i;
                    if (threadIdx.x == 0)
                        *reinterpret_cast<v4i*>(a.joins + 4 * ((int64_t)group * (2 * a.workers + 1) + 1 + record)) = v4i{s, begin, (int)of, 0};
                }
                found = true;
                break;
            }
            items += lane_of(upto, kWave - 1), split += lane_of(split_upto, kWave - 1);
        }
        // the first workgroup without an item has seen them all
        if (!found && items == (unsigned)worker && threadIdx.x == 0) a.joins[4 * (int64_t)group * (2 * a.workers + 1)] = (int)split;
    }

    const int64_t row_bytes = (int64_t)a.dim * T::kBytes;
    // byte offsets in a row: the lane's 16-byte chunks (keys: every fourth, so that four lanes read 64 bytes at once),
    // its DP / 16 channels (values)
    int key_at[T::kKeyChunks];
#pragma unroll
    for (int i = 0; i < T::kKeyChunks; ++i) {
        const int at = 16 * (4 * i + g);
        key_at[i] = n * (int)row_bytes + (at < row_bytes ? at : 0);
    }
    const int value_piece = n * (DP / 16 * T::kBytes);
    const int value_at = 4 * g * (int)row_bytes + (value_piece < row_bytes ? value_piece : 0);

    if (first < last) {
        // the wavefront's units of the item
        const int mine = first + (last - first) * wave / WAVES, end = first + (last - first) * (wave + 1) / WAVES;

        v8bf q[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
            // the channels of the key chunks: 8 to a chunk in bf16, 16 (two operands) in 8 bits
            const int d = KIND == QLIN_CACHE_BF16 ? 8 * (4 * i + g) : 16 * (4 * (i / 2) + g) + 8 * (i % 2);
            v4u w = v4u{0, 0, 0, 0};
            if (n < rows && d < a.dim) w = *reinterpret_cast<const v4u*>(a.q + ((int64_t)s * a.heads + head0 + n) * a.dim + d);
            q[i] = __builtin_bit_cast(v8bf, w);
        }

        const Table table = table_of(a.pages + (int64_t)s * a.columns);
        struct Places {
            AttnPlace at[2];
        };
        auto where = [&](int unit) {
            Places p;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                p.at[j] = attn_place(span, unit, j, table, (int)a.npages, a.kv_heads, kv_head, a.page_size, a.page_shift);
            return p;
        };
        auto load_keys = [&](const Places& p, T& t) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint8_t* base = a.k + p.at[j].row * row_bytes;
#pragma unroll
                for (int i = 0; i < T::kKeyChunks; ++i) t.key[j][i] = *reinterpret_cast<const v4u*>(base + key_at[i]);
                if constexpr (KIND != QLIN_CACHE_BF16) t.key_scale[j] = reinterpret_cast<const v4f*>(a.k_scale + p.at[j].row)[g];
            }
        };
        auto load_values = [&](const Places& p, T& t) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint8_t* base = a.v + p.at[j].row * row_bytes;
#pragma unroll
                for (int i = 0; i < 4; ++i) load_dwords(base + value_at + i * row_bytes, t.value[4 * j + i]);
                if constexpr (KIND != QLIN_CACHE_BF16) t.value_scale[j] = reinterpret_cast<const v4f*>(a.v_scale + p.at[j].row)[g];
            }
        };

        float m = kNone, l = 0.0f;
        v4f acc[kTiles];
#pragma unroll
        for (int r = 0; r < kTiles; ++r) acc[r] = v4f{0, 0, 0, 0};

        T t = {};
        Places here = {}, next = {};
        if (mine < end) {
            here = where(mine);
            load_keys(here, t);
            load_values(here, t);
        }
        for (int unit = mine; unit < end; ++unit) {
            const bool more = unit + 1 < end;
            if (more) next = where(unit + 1);
            v4f score[2] = {v4f{0, 0, 0, 0}, v4f{0, 0, 0, 0}};
#pragma unroll
            for (int i = 0; i < kSteps; ++i) {
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    v8bf k;
                    if constexpr (KIND == QLIN_CACHE_BF16) k = __builtin_bit_cast(v8bf, t.key[j][i]);
                    else k = key_operand<KIND>(t.key[j][i / 2][2 * (i % 2)], t.key[j][i / 2][2 * (i % 2) + 1]);
                    score[j] = mfma(k, q[i], score[j]);
                }
            }
            v4f key_scale[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) key_scale[j] = KIND == QLIN_CACHE_BF16 ? v4f{1, 1, 1, 1} : t.key_scale[j];
            if (more) load_keys(next, t);
            settle();
            float p[8], top = kNone;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = 4 * g + i;
                    const float x = score[j][i] * (KIND == QLIN_CACHE_BF16 ? a.scale : key_scale[j][i] * a.scale);
                    p[4 * j + i] = at >= here.at[j].lo && at < here.at[j].hi ? x : kNone;
                    top = fmaxf(top, p[4 * j + i]);
                }
            }
            top = column_max(top);
            if (__any(top > m)) {
                const float now = fmaxf(m, top);
                const float by = m == kNone ? 0.0f : __builtin_amdgcn_exp2f(m - now);
                m = now;
                l *= by;
#pragma unroll
                for (int r = 0; r < kTiles; ++r) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) acc[r][i] *= by;
                }
            }
            const float zero_at = m == kNone ? 0.0f : m;
            const bool whole = here.at[0].lo == 0 && here.at[1].lo == 0 && here.at[0].hi == 16 && here.at[1].hi == 16;
            if (!whole) {   // what lies in masked places may be anything
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int at = 4 * g + i;
                        const bool live = at >= here.at[j].lo && at < here.at[j].hi;
#pragma unroll
                        for (int w = 0; w < T::kValueDwords; ++w) t.value[4 * j + i][w] = live ? t.value[4 * j + i][w] : 0;
                        if constexpr (KIND != QLIN_CACHE_BF16) t.value_scale[j][i] = live ? t.value_scale[j][i] : 0.0f;
                    }
                }
            }
            // Single registers from here on.  Without this clang 22 (ROCm 7.2) compiled an earlier state of this loop, in the
            // three one-launch forms for bf16, so that loaded registers were given to p before their last use: 6, 16 and 16
            // reads of them, an excerpt in tests/test_attn_lost_registers.py.  The loop as it is compiles to none either way,
            // in the same time (no case by more than 0.2 %).
#pragma unroll
            for (int i = 0; i < 8; ++i) {
#pragma unroll
                for (int w = 0; w < T::kValueDwords; ++w) asm("" : "+v"(t.value[i][w]));
            }
            v8bf high, low;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float e = __builtin_amdgcn_exp2f(p[4 * j + i] - zero_at);
                    l += e;
                    const float x = KIND == QLIN_CACHE_BF16 ? e : e * t.value_scale[j][i];
                    high[4 * j + i] = (__bf16)x;
                    low[4 * j + i] = (__bf16)(x - (float)high[4 * j + i]);
                }
            }
#pragma unroll
            for (int w = 0; w < T::kValueDwords; ++w) {
                // dword w of the 8 tokens: channels (of the lane) 4 w .. 4 w + 3, or 2 w, 2 w + 1 in bf16
                if constexpr (KIND == QLIN_CACHE_BF16) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint32_t pick = h ? 0x07060302u : 0x05040100u;
                        uint32_t d[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) d[i] = __builtin_amdgcn_perm(t.value[2 * i + 1][w], t.value[2 * i][w], pick);
                        const v8bf v = operand(d[0], d[1], d[2], d[3]);
                        acc[2 * w + h] = mfma(v, high, acc[2 * w + h]);
                        acc[2 * w + h] = mfma(v, low, acc[2 * w + h]);
                    }
                } else {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {   // bytes 2 h and 2 h + 1 of two tokens: {a, b, a', b'}
                        const uint32_t pick = h ? 0x07030602u : 0x05010400u;
                        uint32_t x[4], y[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t both = __builtin_amdgcn_perm(t.value[2 * i + 1][w], t.value[2 * i][w], pick);
                            x[i] = widen_pair<KIND, false>(both);
                            y[i] = widen_pair<KIND, true>(both);
                        }
                        const v8bf v0 = operand(x[0], x[1], x[2], x[3]), v1 = operand(y[0], y[1], y[2], y[3]);
                        acc[4 * w + 2 * h] = mfma(v0, high, acc[4 * w + 2 * h]);
                        acc[4 * w + 2 * h + 1] = mfma(v1, high, acc[4 * w + 2 * h + 1]);
                        acc[4 * w + 2 * h] = mfma(v0, low, acc[4 * w + 2 * h]);
                        acc[4 * w + 2 * h + 1] = mfma(v1, low, acc[4 * w + 2 * h + 1]);
                    }
                }
            }
            if (more) {
                load_values(next, t);
                here = next;
            }
        }
        settle();
        l = column_sum(l);

        // The wavefronts' sums, joined in pairs: the upper half hands its to the
        // lower, and so on.  acc[r][i] is channel (DP / 16) (4 g + i) + r of head n.
        auto give = [&](int slot) {
            if (n < rows) {
                float* to = joined[slot] + n * kPad + 4 * g * kTiles;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int r = 0; r < kTiles; ++r) to[i * kTiles + r] = acc[r][i];
                }
                if (g == 0) stats[slot][0][n] = m, stats[slot][1][n] = l;
            }
        };
        auto take = [&](int slot) {
            if (n < rows) {
                const float om = stats[slot][0][n], now = fmaxf(m, om), zero_at = now == kNone ? 0.0f : now;
                const float by = __builtin_amdgcn_exp2f(m - zero_at), other = __builtin_amdgcn_exp2f(om - zero_at);
                const float* from = joined[slot] + n * kPad + 4 * g * kTiles;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int r = 0; r < kTiles; ++r) acc[r][i] = acc[r][i] * by + from[i * kTiles + r] * other;
                }
                l = l * by + stats[slot][1][n] * other;
                m = now;
            }
        };
#pragma unroll
        for (int half = WAVES / 2; half >= 1; half /= 2) {
#pragma unroll
            for (int w = 0; w < half; w += kSlots) {   // wavefronts w .. of the lower half take from those of the upper
                __syncthreads();   // the buffers are free
                if (wave >= half + w && wave < half + min(w + kSlots, half)) give(wave - half - w);
                __syncthreads();
                if (wave >= w && wave < min(w + kSlots, half)) take(wave - w);
            }
        }

        if (wave == 0 && n < rows) {
            const int d0 = 4 * g * kTiles;
            if (ALONE || record < 0) {
                const float by = l > 0.0f || l != l ? 1.0f / l : 0.0f;
                uint16_t* to = a.out + ((int64_t)s * a.heads + head0 + n) * a.dim + d0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int r = 0; r < kTiles; r += 2)
                        if (d0 + i * kTiles + r < a.dim)
                            *reinterpret_cast<uint32_t*>(to + i * kTiles + r) = bf16_pair(acc[r][i] * by, acc[r + 1][i] * by);
                }
            } else {
                const int64_t at = ((int64_t)group * 2 * a.workers + record) * a.rows + n;
                float* to = a.sums + at * a.dim + d0;
                if (g == 0) *reinterpret_cast<v2f*>(a.stats + 2 * at) = v2f{m, l};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int r = 0; r < kTiles; r += 4)
                        if (d0 + i * kTiles + r < a.dim)
                            *reinterpret_cast<v4f*>(to + i * kTiles + r) = v4f{acc[r][i], acc[r + 1][i], acc[r + 2][i], acc[r + 3][i]};
                }
            }
        }
    }

    // sequences without tokens: zeros
    auto clear = [&](int e) {
        const int length = table_of(a.lengths)[e];
        if (length == 0 || (length > 0 && a.columns == 0))
            for (int i = lane; i < rows * a.dim / 2; i += kWave)
                reinterpret_cast<uint32_t*>(a.out + ((int64_t)e * a.heads + head0) * a.dim)[i] = 0;
    };
    if constexpr (ALONE) {
        if (wave == 0) clear(s);
    } else {   // a share of them for each workgroup
        for (int e = worker * WAVES + wave; e < a.S; e += (a.workers + a.S + 1) * WAVES) clear(e);
    }
}

// A head's running maximum, sum of p and (unnormalised) output: lane l of the
// wavefront holds channels 2 l, 2 l + 1, 128 + 2 l and 129 + 2 l.
struct Joined {
    float m, l, o[4];
};

// The partial sums first, first + step, .. (count of them) of one query head:
// lane p has the maximum and sum of the p-th, and the values of 16, or of the
// last 4, are under way together.
__device__ __forceinline__ Joined join_parts(const AttnArgs& a, int group, int row, int first, int step, int count) {
    const int lane = threadIdx.x % kWave;
    auto at = [&](int p) { return ((int64_t)group * 2 * a.workers + first + step * p) * a.rows + row; };
    Joined r = {kNone, 0.0f, {0, 0, 0, 0}};
    for (int p0 = 0; p0 < count; p0 += kWave) {
        const int here = min(count - p0, kWave);
        v2f stat = v2f{kNone, 0.0f};
        if (lane < here) stat = *reinterpret_cast<const v2f*>(a.stats + 2 * at(p0 + lane));
        float weight = 0.0f;
        auto batch = [&](auto size, int p) {
            constexpr int kSize = decltype(size)::value;
            v2f x[kSize][2];
#pragma unroll
            for (int u = 0; u < kSize; ++u) {
                const float* from = a.sums + at(p0 + min(p + u, here - 1)) * a.dim;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int d = 2 * lane + 128 * i;
                    x[u][i] = d < a.dim ? *reinterpret_cast<const v2f*>(from + d) : v2f{0, 0};
                }
            }
            if (p == 0) {
                const float top = fmaxf(r.m, column_max(lanes_max<16>(stat.x))), zero_at = top == kNone ? 0.0f : top;
                const float by = __builtin_amdgcn_exp2f(r.m - zero_at);
                weight = __builtin_amdgcn_exp2f(stat.x - zero_at);
                r.l = r.l * by + column_sum(lanes_sum<16>(stat.y * weight));
                r.m = top;
#pragma unroll
                for (int i = 0; i < 4; ++i) r.o[i] *= by;
            }
#pragma unroll
            for (int u = 0; u < kSize; ++u) {
                const float w = p + u < here ? __uint_as_float(lane_of(__float_as_uint(weight), min(p + u, kWave - 1))) : 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) r.o[i] = __builtin_fmaf(x[u][i / 2][i % 2], w, r.o[i]);
            }
        };
        int p = 0;
        for (; here - p > 4; p += 16) batch(std::integral_constant<int, 16>{}, p);
        if (p < here) batch(std::integral_constant<int, 4>{}, p);
    }
    return r;
}

// Joins the partial sums of split sequences.  The n workgroups of a sequence's
// n partial sums share its query heads: of up to kFew partial sums a wavefront
// joins those of a head, of more the four wavefronts of a workgroup do, a
// quarter each.
__global__ __launch_bounds__(kThreads) void attn_join_kernel(AttnArgs a) {
    constexpr int kFew = 4;
    __shared__ float part_max[kWaves], part_sum[kWaves];
    __shared__ float part_out[kWaves][QLIN_MAX_HEAD_DIM];
    const int lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int group = blockIdx.x, record = blockIdx.y;
    const Table joins = table_of(a.joins + 4 * ((int64_t)group * (2 * a.workers + 1)));
    const int records = joins[0], s = joins[4 * (1 + record)], begin = joins[4 * (1 + record) + 1], parts = joins[4 * (1 + record) + 2];
    if (record >= records) return;
    const int tile = group % a.tiles;
    const int rows = min(a.rows, a.shared_by - tile * kAttnHeads);
    const int64_t head0 = (int64_t)s * a.heads + group / a.tiles * a.shared_by + tile * kAttnHeads;
    if (parts <= kFew) {
        for (int row = kWaves * (record - begin) + wave; row < rows; row += kWaves * parts) {
            const Joined r = join_parts(a, group, row, begin, 1, parts);
            const float by = r.l > 0.0f || r.l != r.l ? 1.0f / r.l : 0.0f;
            uint16_t* to = a.out + (head0 + row) * a.dim;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int d = 2 * lane + 128 * i;
                if (d < a.dim) *reinterpret_cast<uint32_t*>(to + d) = bf16_pair(r.o[2 * i] * by, r.o[2 * i + 1] * by);
            }
        }
        return;
    }
    for (int row = record - begin; row < rows; row += parts) {
        const Joined r = join_parts(a, group, row, begin + wave, kWaves, (parts - wave + kWaves - 1) / kWaves);
        __syncthreads();   // the buffers are free
        if (lane == 0) part_max[wave] = r.m, part_sum[wave] = r.l;
#pragma unroll
        for (int i = 0; i < 4; ++i) part_out[wave][2 * lane + 128 * (i / 2) + i % 2] = r.o[i];
        __syncthreads();
        const int d = threadIdx.x;
        if (d < a.dim) {
            float top = kNone, sum = 0.0f, out = 0.0f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) top = fmaxf(top, part_max[w]);
            top = top == kNone ? 0.0f : top;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) {
                const float by = __builtin_amdgcn_exp2f(part_max[w] - top);
                sum += part_sum[w] * by;
                out += part_out[w][d] * by;
            }
            a.out[(head0 + row) * a.dim + d] = f32_to_bf16(sum > 0.0f || sum != sum ? out / sum : 0.0f);
        }
    }
}

template <int KIND, int DP>
void launch_dim(const AttnArgs& a, bool alone, dim3 grid, hipStream_t st) {
    constexpr int kAlone = DP == 64 ? 8 : kWaves;
    if (alone) hipLaunchKernelGGL((attn_kernel<KIND, DP, kAlone, true>), grid, dim3(kAlone * kWave), 0, st, a);
    else hipLaunchKernelGGL((attn_kernel<KIND, DP, kWaves, false>), grid, dim3(kThreads), 0, st, a);
}
template <int KIND>
void launch_kind(const AttnArgs& a, bool alone, dim3 grid, hipStream_t st) {
    switch (attn_channels(a.dim)) {
        case 64: return launch_dim<KIND, 64>(a, alone, grid, st);
        case 128: return launch_dim<KIND, 128>(a, alone, grid, st);
        default: launch_dim<KIND, 256>(a, alone, grid, st);
    }
}

constexpr int kMaxSequences = 4096;   // of a launch: up to 1024 groups of heads and 2^32 threads

}  // namespace

AttnShape attn_shape(int heads, int kv_heads, int dim) {
    // Two workgroups to a CU (one of 256 channels), though the registers hold more.  8 x 32768 tokens of 32 / 8 heads of
    // 128 with one, two and three to a CU: E4M3 120, 103 and 106 us, int8 135, 106 and 109, bf16 188 each time.  16 x 4096
    // of 256 channels in E4M3: 57.8, 57.6 and 63.0.  The room that is left takes the items beyond `workers`, of which there
    // are up to S.
    const int share = kCus * (dim <= 128 ? 2 : 1);
    const int shared_by = heads / kv_heads, tiles = (shared_by + kAttnHeads - 1) / kAttnHeads;
    const int groups = kv_heads * tiles;
    return AttnShape{tiles, shared_by < kAttnHeads ? shared_by : kAttnHeads, groups >= share ? 1 : share / groups};
}

int64_t attn_workspace(int heads, int kv_heads, int dim) {
    const AttnShape s = attn_shape(heads, kv_heads, dim);
    const int64_t groups = (int64_t)kv_heads * s.tiles, records = groups * 2 * s.workers;
    return 16 * (groups + records) + records * s.rows * (dim + 2) * 4;
}

hipError_t launch_attn(const AttnCall& c, hipStream_t st) {
    const AttnShape shape = attn_shape(c.heads, c.cache.kv_heads, c.cache.dim);
    const int groups = c.cache.kv_heads * shape.tiles;
    AttnArgs a{};
    a.q = c.q;
    a.k = static_cast<const uint8_t*>(c.cache.k);
    a.v = static_cast<const uint8_t*>(c.cache.v);
    a.k_scale = c.cache.k_scale;
    a.v_scale = c.cache.v_scale;
    a.pages = c.pages;
    a.lengths = c.lengths;
    a.out = c.out;
    const int64_t records = (int64_t)groups * 2 * shape.workers;
    a.joins = static_cast<int*>(c.workspace);
    a.stats = reinterpret_cast<float*>(a.joins + 4 * (groups + records));
    a.sums = a.stats + records * shape.rows * 2;
    a.npages = c.cache.pages;
    a.S = c.S;
    a.heads = c.heads;
    a.kv_heads = c.cache.kv_heads;
    a.shared_by = c.heads / c.cache.kv_heads;
    a.dim = c.cache.dim;
    a.columns = c.columns;
    a.page_size = c.cache.page_size;
    a.page_shift = a.page_size & (a.page_size - 1) ? -1 : __builtin_ctz((unsigned)a.page_size);
    a.window = c.window;
    a.tiles = shape.tiles;
    a.rows = shape.rows;
    a.workers = shape.workers;
    // Where the sequences are many, one of 512 tokens is not cut.  Since an item's size is looked for this matters little:
    // 32 / 8 heads of 128 in E4M3 whole and cut down to 128 tokens, 64 x 256 tokens 13.2 us either way, 40 x 300 to 512
    // 16.0 and 16.3, 63 x 1 to 512 15.8 and 16.2, 70 x 1 to 512 18.4 and 16.9.
    a.least = c.S <= shape.workers / 2 ? kAttnWaves : 4 * kAttnWaves;
    a.scale = c.scale * 1.44269504088896340736f;
    const bool alone = attn_alone(c.S, (int64_t)c.columns * c.cache.page_size, groups, c.cache.dim);
    if (c.S > kMaxSequences) {   // one half of the sequences after the other
        AttnCall part = c;
        part.S = c.S / 2;
        const hipError_t e = launch_attn(part, st);
        if (e != hipSuccess) return e;
        const int64_t done = part.S;
        part.S = c.S - part.S;
        part.q += done * c.heads * c.cache.dim;
        part.out += done * c.heads * c.cache.dim;
        if (c.columns) part.pages += done * c.columns;
        part.lengths += done;
        return launch_attn(part, st);
    }
    const dim3 grid((unsigned)groups, (unsigned)(alone ? c.S : shape.workers + c.S + 1));
    if (c.cache.kind == QLIN_CACHE_BF16) launch_kind<QLIN_CACHE_BF16>(a, alone, grid, st);
    else if (c.cache.kind == QLIN_CACHE_INT8) launch_kind<QLIN_CACHE_INT8>(a, alone, grid, st);
    else launch_kind<QLIN_CACHE_FP8>(a, alone, grid, st);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && !alone) {
        hipLaunchKernelGGL(attn_join_kernel, dim3((unsigned)groups, (unsigned)(2 * shape.workers)), dim3(kThreads), 0, st, a);
        e = hipGetLastError();
    }
    return e;
}

}  // namespace qlin
