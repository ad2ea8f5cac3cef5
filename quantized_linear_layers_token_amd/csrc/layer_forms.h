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
// Several and one, us: 32768 tokens of one kv head of 64 channels written 5.7
// and 32.0; rotations of 32768 tokens, one head of 64 6.3 and 28.2, one of 128
// 8.4 and 29.2, two of 256 18.7 and 30.6, eight of 64 15.0 and 29.6; of 8192
// tokens 5.7 to 7.1 and 8.6 to 9.7; of 1024 and 2048 the call's time either way.
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
// for more sequences than a workgroup can scan.  One launch and two, us, equal
// lengths of 16 / 8 heads of 128 in E4M3: 16 sequences of 512, 1024 and 2048
// tokens 10.2 and 12.3, 15.5 and 14.8, 26.2 and 19.6; 32 of them 10.8 and 14.5,
// 16.3 and 19.6, 33.6 and 33.1; 64 of them 15.6 and 18.1, 29.5 and 31.8, 52.6
// and 55.0.  Heads of 64 9.5 and 11.4 (16 of 1024) to 29.7 and 34.7 (64 of 2048),
// of 256 14.2 and 15.5 (16 of 512), 41.5 and 34.1 (16 of 2048), 99 and 102 (64 of
// 2048).  So the few sequences at the rule's edge lose by it, ragged ones most
// (16 of 1 to 2048: 25.8 and 16.5).
constexpr int64_t kAttnMedium = 2048;
constexpr int kAttnScanned = 1024;
constexpr bool attn_alone(int64_t sequences, int64_t tokens, int groups, int dim) {
    return tokens <= (dim <= 64 ? 512 : 256) || (tokens <= kAttnMedium && sequences * groups >= kCus / 2) || sequences > kAttnScanned;
}

}  // namespace qlin
