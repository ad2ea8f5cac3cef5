// Which tokens a workgroup of the attention takes and where they lie: the
// integer part of attn_decode.hip, in functions that host code can run too
// (constexpr: for either side), so that every bound is tested on the CPU.
//
// A sequence's tokens are cut in units of 32, and the units in items, one to a
// workgroup: a sequence of up to `most` units is one item, a longer one
// ceil(units / most) of about equal size.  With most = ceil(total / workers)
// or more there are at most workers + S items,
// whatever the lengths, and at most 2 workers of them belong to sequences of
// several (whose partial sums are written down and joined): n > 1 means
// units > most, so n < 2 units / most.
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

// Units of an item at most, a multiple of the wavefronts (which share them
// evenly then); `least` (a multiple too) where the shares are smaller.
constexpr unsigned attn_most(int64_t total, int workers, int least) {
    const int64_t even = ((total + workers - 1) / workers + kAttnWaves - 1) / kAttnWaves * kAttnWaves;
    return even < least ? (unsigned)least : even > 0x7ffffff0 ? 0x7ffffff0u : (unsigned)even;
}
// The next try where that gave `items`, more than workers: a multiple of the
// wavefronts again, and larger.
constexpr unsigned attn_larger(unsigned most, unsigned items, int workers) {
    const int64_t scaled = ((int64_t)most * items / workers + kAttnWaves) / kAttnWaves * kAttnWaves;
    return scaled > 0x7ffffff0 ? 0x7ffffff0u : scaled > most ? (unsigned)scaled : most + kAttnWaves;
}
// Items of a sequence.
constexpr unsigned attn_items(unsigned units, unsigned most) { return (units + most - 1) / most; }
// Of these, the first unit of item i of n (the end of the last: i = n).
constexpr unsigned attn_first_unit(unsigned units, unsigned n, unsigned i) {
    const unsigned each = units / n, more = units - each * n;
    return i * each + (i < more ? i : more);
}

// One half of a unit: the row of the cache (page, kv head, place) of its first
// token and which of its 16 tokens are live, lo <= i < hi.  A half without any
// (behind the length, before the window, of a page outside the cache) has the
// rows of page 0, which its loads may read and nothing uses.
// page_shift: log2 of page_size, or -1 (a division of its own would wait some
// 40 instructions before every step's loads).
struct AttnPlace {
    int64_t row;
    int lo, hi;
};
template <class Table>
constexpr AttnPlace attn_place(const AttnSpan& span, int unit, int half, Table table, int pages, int kv_heads, int kv_head, int page_size,
                               int page_shift) {
    const int t = (span.start / kAttnUnit + unit) * kAttnUnit + kAttnHalf * half;
    const int column = page_shift >= 0 ? t >> page_shift : t / page_size, place = t - column * page_size;
    int page = t < span.n && t + kAttnHalf > span.start ? table[column] : -1;
    const bool live = page >= 0 && page < pages;
    page = live ? page : 0;
    return AttnPlace{((int64_t)page * kv_heads + kv_head) * page_size + place, live ? attn_max(span.start - t, 0) : kAttnHalf,
                     live ? attn_min(span.n - t, kAttnHalf) : 0};
}

}  // namespace qlin
