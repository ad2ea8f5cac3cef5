// Which tokens a workgroup of the attention takes and where they lie: the
// integer part of attn_decode.hip, in functions that host code can run too
// (constexpr: for either side), so that every bound is tested on the CPU.
#pragma once

#include <stdint.h>

namespace qlin {

constexpr int kAttnUnit = 32;    // tokens of a wavefront's step
constexpr int kAttnHalf = 16;    // tokens that lie in one page: page_size is a multiple of it
constexpr int kAttnWaves = 4;    // wavefronts of a workgroup

constexpr int attn_min(int a, int b) { return a < b ? a : b; }
constexpr int attn_max(int a, int b) { return a > b ? a : b; }

// The tokens start .. n - 1 of a sequence (those of its window) and the units
// that hold them.  columns * page_size is at most 2^30.
struct AttnSpan {
    int n, start;
    unsigned units;
};
constexpr AttnSpan attn_span(int length, int columns, int page_size, int window) {
    const int n = attn_min(attn_max(length, 0), columns * page_size);
    const int start = window > 0 ? attn_max(0, n - window) : 0;
    return AttnSpan{n, start, (unsigned)((n + kAttnUnit - 1) / kAttnUnit - start / kAttnUnit)};
}

// Units of one workgroup: an even share, but one for each wavefront at least.
constexpr int64_t attn_share(int64_t total, int workers) {
    const int64_t even = (total + workers - 1) / workers;
    return even > kAttnWaves ? even : kAttnWaves;
}

// The part of a workgroup's partial sums that a sequence takes whose first unit
// is `before` and that the workgroup, whose first unit is `lo`, does not hold
// whole: 0 for the one that lies over the workgroup's first unit, 1 for one
// that begins later (and goes on past its last).
constexpr int attn_part(int64_t before, int64_t lo) { return before > lo ? 1 : 0; }
// The workgroup that holds a sequence's last unit.
constexpr int attn_last_worker(int64_t before, unsigned units, int64_t share) { return (int)((before + units - 1) / share); }

// One half of a unit: the row of the cache (page, kv head, place) of its first
// token and which of its 16 tokens are live, lo <= i < hi.  A half without any
// (behind the length, before the window, of a page outside the cache) has the
// rows of page 0, which its loads may read and nothing uses.
struct AttnPlace {
    int64_t row;
    int lo, hi;
};
template <class Table>
constexpr AttnPlace attn_place(const AttnSpan& span, int unit, int half, Table table, int pages, int kv_heads, int kv_head, int page_size) {
    const int t = (span.start / kAttnUnit + unit) * kAttnUnit + kAttnHalf * half;
    const int column = t / page_size, place = t - column * page_size;
    int page = t < span.n && t + kAttnHalf > span.start ? table[column] : -1;
    const bool live = page >= 0 && page < pages;
    page = live ? page : 0;
    return AttnPlace{((int64_t)page * kv_heads + kv_head) * page_size + place, live ? attn_max(span.start - t, 0) : kAttnHalf,
                     live ? attn_min(span.n - t, kAttnHalf) : 0};
}

}  // namespace qlin
