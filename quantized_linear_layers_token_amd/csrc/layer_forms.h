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

constexpr int kCus = 256;

// Channels of a head in the attention's registers.
constexpr int attn_channels(int dim) { return dim <= 64 ? 64 : dim <= 128 ? 128 : 256; }

// An item is a sequence, and there is one launch, where no sequence of the
// table's `tokens` can be longer than two steps of a workgroup's wavefronts, or
// than kAttnMedium and the sequences' groups of heads fill half of the CUs; and
// for more sequences than a workgroup can scan.
constexpr int64_t kAttnMedium = 2048;
constexpr int kAttnScanned = 1024;
constexpr bool attn_alone(int64_t sequences, int64_t tokens, int groups, int dim) {
    return tokens <= (dim <= 64 ? 512 : 256) || (tokens <= kAttnMedium && sequences * groups >= kCus / 2) || sequences > kAttnScanned;
}

}  // namespace qlin
