// The attention's integer part (attn_index.h) on the CPU: over random batches, every live token is taken exactly once,
// every row that is loaded lies in the cache, every table entry that is read lies in the table, and there is a
// workgroup for every item and room for every partial sum.
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include <random>
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
        const int shift = page_size & (page_size - 1) ? -1 : __builtin_ctz(page_size);
        std::vector<AttnSpan> span(S);
        int64_t total = 0;
        for (int s = 0; s < S; ++s) {
            span[s] = attn_span(length[s], columns, page_size, window);
            total += span[s].units;
            CHECK((span[s].units == 0) == (length[s] <= 0 || columns == 0));
        }
        unsigned most = attn_most(total, workers, kAttnWaves * draw(1, 4));
        for (int k = S < workers ? draw(0, 6) : 0; k > 0; --k) {       // (as the workgroups look for a size that fits)
            unsigned n = 0;
            for (int s = 0; s < S; ++s) n += attn_items(span[s].units, most);
            if (n <= (unsigned)workers) break;
            const unsigned next = attn_larger(most, n, workers);
            CHECK(next > most && next % kAttnWaves == 0);
            most = next;
        }
        unsigned items = 0, split = 0;
        std::vector<std::vector<int>> taken(S);
        for (int s = 0; s < S; ++s) {
            taken[s].assign((size_t)span[s].n, 0);
            const unsigned n = attn_items(span[s].units, most);
            CHECK((n == 0) == (span[s].units == 0));
            items += n;
            split += n > 1 ? n : 0;
            unsigned reached = 0;
            for (unsigned i = 0; i < n; ++i) {
                const unsigned first = attn_first_unit(span[s].units, n, i), last = attn_first_unit(span[s].units, n, i + 1);
                CHECK(first == reached && last > first && last - first <= most);
                reached = last;
                int wave_reached = (int)first;
                for (int wave = 0; wave < kAttnWaves; ++wave) {
                    const int mine = first + (int)(last - first) * wave / kAttnWaves, end = first + (int)(last - first) * (wave + 1) / kAttnWaves;
                    CHECK(mine == wave_reached);
                    wave_reached = end;
                    for (int u = mine; u < end; ++u) {
                        ++units_seen;
                        for (int half = 0; half < 2; ++half) {
                            const AttnPlace p = attn_place(span[s], u, half, Row{table.data() + (size_t)s * columns, columns}, pages, kv_heads,
                                                           kv_heads - 1, page_size, shift);
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
                CHECK(wave_reached == (int)last);
            }
            CHECK(reached == span[s].units);
            joined_seen += n > 1;
        }
        CHECK(items <= (unsigned)(workers + S));     // a workgroup for each, and one more that has none
        CHECK(split <= (unsigned)(2 * workers));     // room for each partial sum
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
    for (int workers : {1, 2, 96, 1024})
        for (int64_t total : {(int64_t)1 << 25, (int64_t)1 << 30, (int64_t)1024 << 25}) {
            const unsigned m = attn_most(total, workers, kAttnWaves), units = 1u << 25, n = attn_items(units, m);
            CHECK(n >= 1 && (int64_t)n * (total >> 25) <= 2 * (int64_t)workers + (total >> 25));
            CHECK(attn_first_unit(units, n, 0) == 0 && attn_first_unit(units, n, n) == units);
            for (unsigned i = 0; i < n; ++i) CHECK(attn_first_unit(units, n, i) < attn_first_unit(units, n, i + 1));
        }
    std::printf("%ld units, %ld joins, %ld tokens: every bound held\n", units_seen, joined_seen, live_seen);
    return 0;
}
