// The attention's integer part (attn_index.h) on the CPU: over random batches, every live token is taken exactly once,
// every row that is loaded lies in the cache, every table entry that is read lies in the table, and the partial sums that
// are written are those that are joined.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <vector>

#include "../../quantized_linear_layers_token_amd/csrc/attn_index.h"

using namespace qlin;

#define CHECK(x) \
    do { \
        if (!(x)) { std::printf("line %d: %s (round %d)\n", __LINE__, #x, round); std::exit(1); } \
    } while (0)

struct Row {   // a table row that knows its bounds
    const int* p;
    int columns;
    int operator[](int i) const {
        if (i < 0 || i >= columns) { std::printf("table read out of range: %d of %d\n", i, columns); std::exit(1); }
        return p[i];
    }
};

int main() {
    std::mt19937 rng(7);
    auto draw = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
    long units_seen = 0, joined_seen = 0, live_seen = 0;
    for (int round = 0; round < 4000; ++round) {
        const int page_size = 16 * draw(1, 6), columns = draw(0, 40), pages = draw(1, 60), kv_heads = draw(1, 4);
        const int S = draw(1, 200) / draw(1, 20) + 1, workers = draw(1, 3) == 1 ? draw(1, 6) : draw(1, 64);
        const int window = draw(0, 2) ? 0 : draw(1, columns * page_size + 40);
        std::vector<int> length(S), table((size_t)S * columns);
        for (int& v : length) v = draw(0, 5) == 0 ? draw(-2, 1) : draw(0, columns * page_size + 20);
        for (int& v : table) v = draw(0, 30) == 0 ? draw(-3, pages + 3) : draw(0, pages - 1);
        std::vector<AttnSpan> span(S);
        std::vector<int64_t> before(S);
        int64_t total = 0;
        for (int s = 0; s < S; ++s) {
            span[s] = attn_span(length[s], columns, page_size, window);
            before[s] = total;
            total += span[s].units;
            CHECK((span[s].units == 0) == (length[s] <= 0 || columns == 0));
        }
        const int64_t share = attn_share(total, workers);
        CHECK(share * workers >= total);
        std::map<std::pair<int, int>, std::set<std::pair<int, int>>> parts;   // (worker, part) -> sequences that write it
        std::map<int, std::set<std::pair<int, int>>> of_sequence;             // sequence -> its parts
        std::map<int, std::vector<int>> join;                                 // worker -> sequence, last, part
        std::vector<std::vector<int>> taken(S);
        for (int s = 0; s < S; ++s) taken[s].assign((size_t)span[s].n, 0);
        for (int w = 0; w < workers; ++w) {
            const int64_t lo = w * share, hi = lo + share < total ? lo + share : total;
            if (lo >= total) continue;
            for (int s = 0; s < S; ++s) {
                if (span[s].units == 0 || before[s] >= hi || before[s] + span[s].units <= lo) continue;
                const int first = (int)((lo > before[s] ? lo : before[s]) - before[s]);
                const int64_t stop = before[s] + span[s].units;
                const int last = (int)((hi < stop ? hi : stop) - before[s]);
                int reached = first;
                for (int wave = 0; wave < kAttnWaves; ++wave) {
                    const int mine = first + (int)((int64_t)(last - first) * wave / kAttnWaves);
                    const int end = first + (int)((int64_t)(last - first) * (wave + 1) / kAttnWaves);
                    CHECK(mine == reached);
                    reached = end;
                    for (int u = mine; u < end; ++u) {
                        ++units_seen;
                        for (int half = 0; half < 2; ++half) {
                            const AttnPlace p = attn_place(span[s], u, half, Row{table.data() + (size_t)s * columns, columns}, pages, kv_heads,
                                                           kv_heads - 1, page_size);
                            const int64_t rows = (int64_t)pages * kv_heads * page_size;
                            CHECK(p.row >= 0 && p.row % kAttnHalf == 0 && p.row + kAttnHalf <= rows);
                            const int t = (span[s].start / kAttnUnit + u) * kAttnUnit + kAttnHalf * half;
                            for (int i = 0; i < kAttnHalf; ++i) {
                                if (i < p.lo || i >= p.hi) continue;
                                CHECK(t + i >= span[s].start && t + i < span[s].n);
                                const int page = table[(size_t)s * columns + (t + i) / page_size];
                                CHECK(p.row + i == ((int64_t)page * kv_heads + kv_heads - 1) * page_size + (t + i) % page_size);
                                ++taken[s][t + i];
                                ++live_seen;
                            }
                        }
                    }
                }
                CHECK(reached == last);
                const bool starts = before[s] >= lo, ends = stop <= hi;
                if (starts && ends) continue;
                const int part = attn_part(before[s], lo);
                parts[{w, part}].insert({s, w});
                of_sequence[s].insert({w, part});
                if (starts) {
                    CHECK(!join.count(w));
                    join[w] = {s, attn_last_worker(before[s], span[s].units, share), part};
                }
            }
        }
        for (const auto& p : parts) CHECK(p.second.size() == 1);
        std::set<int> begun;
        for (const auto& j : join) {
            std::set<std::pair<int, int>> read;
            for (int w = j.first; w <= j.second[1]; ++w) read.insert({w, w == j.first ? j.second[2] : 0});
            CHECK(read == of_sequence[j.second[0]]);
            CHECK(j.second[1] < workers);
            begun.insert(j.second[0]);
            ++joined_seen;
        }
        CHECK(begun.size() == of_sequence.size());
        for (int s = 0; s < S; ++s) {
            for (int t = 0; t < span[s].n; ++t) {
                const int page = table[(size_t)s * columns + t / page_size];
                CHECK(taken[s][t] == (t >= span[s].start && page >= 0 && page < pages ? 1 : 0));
            }
        }
    }
    // the largest sizes: nothing wraps
    int round = -1;
    const AttnSpan most = attn_span(0x7fffffff, 1 << 26, 16, 0);
    CHECK(most.n == 1 << 30 && most.units == 1u << 25);
    const AttnSpan windowed = attn_span(0x7fffffff, 1 << 26, 16, 1);
    CHECK(windowed.units == 1 && windowed.start == (1 << 30) - 1);
    const int64_t total = (int64_t)(1 << 24) << 25;
    CHECK(attn_last_worker(total - (1 << 25), 1u << 25, attn_share(total, 512)) == 511);
    std::printf("%ld units, %ld joins, %ld tokens: every bound held\n", units_seen, joined_seen, live_seen);
    return 0;
}
