// Which form of its kernel a call takes, in functions that host code can run
// too (constexpr: for either side): the tests see by them that every form that
// is built is taken by some call, and take each.
#pragma once

#include <stdint.h>

namespace qlin {

constexpr int kHeadsThreads = 256;

// Lanes that hold a head, eight channels each.
constexpr int heads_lanes(int dim) { return dim <= 64 ? 8 : dim <= 128 ? 16 : 32; }

// Tokens of a workgroup, `heads` of each (queries, keys and values): several
// where its threads hold their heads at once and the workgroups are still many.
// 32768 tokens of one kv head of 64 channels written: 4.7 us with 16, 32.0 with
// one.
constexpr int heads_tokens(int lanes, int heads, int64_t T) {
    return 16 * heads * lanes <= kHeadsThreads && T >= 8192 ? 16 : 4 * heads * lanes <= kHeadsThreads && T >= 1024 ? 4 : 1;
}

// Whether that can be: a token has one head at least where queries alone are
// rotated (in bf16), a key and a value otherwise.
constexpr bool heads_fit(int tokens, int lanes, bool alone) { return tokens * lanes * (alone ? 1 : 2) <= kHeadsThreads; }

}  // namespace qlin
