// C ABI of the 4-bit products, the router and the experts' MLP: argument
// validation and dispatch.  No allocation, no synchronization; every check
// runs before the first launch.
#include <stdint.h>

#include <algorithm>
#include <cmath>

#include "../../include/qlin_w4.h"
#include "qlin_internal.h"
#include "w4_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;
};
Range rng(const void* p, int64_t bytes) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return Range{b, b + (uintptr_t)bytes};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

bool valid_mn(int64_t v) { return v >= 0 && v <= QLIN_MAX_MN; }
bool valid_k(int64_t K) { return K > 0 && K % 32 == 0 && K <= QLIN_MAX_K; }
bool valid_group(int32_t g, int64_t K) { return (g == 32 || g == 64 || g == 128) && K % g == 0; }

// Ranges that a weight of E matrices [n, K] covers.
struct WeightRanges {
    Range q, s, z;
};
WeightRanges ranges(const qlin_w4_weight& w, int64_t E, int64_t K, int32_t group) {
    const int64_t scales = E * qlin_w4_packed_scales(w.n, K, group);
    return WeightRanges{rng(w.q_w, E * qlin_w4_packed_bytes(w.n, K)), rng(w.s_w, 2 * scales), rng(w.z_w, w.z_w ? scales : 0)};
}
bool overlap(Range a, const WeightRanges& w) { return overlap(a, w.q) || overlap(a, w.s) || overlap(a, w.z); }

qlin_status check_pointers(const qlin_w4_weight& w) {
    if (!w.q_w || !w.s_w) return QLIN_ERR_NULL;
    if (!aligned(w.q_w, 16) || !aligned(w.s_w, 8) || !aligned(w.z_w, 4)) return QLIN_ERR_ALIGN;
    return QLIN_OK;
}

// Outputs and inputs of one call stay within what an address space holds, so
// that no size computed from them overflows.
constexpr int64_t kMaxElements = int64_t(1) << 40;

// Choice of a product's form: the one with the least estimated time, from the
// number w of workgroups per CU.  {first, more}: us per 4096 inputs of one
// workgroup on every CU, and of each further one, measured at 1488 x 2048,
// 4096 x 4096, 14336 x 4096 and 4096 x 14336 with 1 to 2048 rows (group 128
// without zero points, group 32 with them; 64 lies between).  The streaming
// forms' workgroups share a CU (a second one costs half of the first at
// least); the tiled forms run one (64 x 8) or two (64 x 16) at a time.
// Examples of both sides, us at 4096 x 4096 in the order of the forms: 64 rows
// 19.6, 12.5, 9.74, 9.69, 13.4, 29.1, 47.3 (16 x 4 with four wavefronts chosen);
// 512 rows 125, 72, 48, 46, 40, 31.6, 47.6 (64 x 8 chosen); 2048 rows 489, 268,
// 179, 181, 145, 117, 73.6 (64 x 16 chosen).  Over 130 shapes off these the
// choice was 5 % slower than the best form, in the geometric mean.  (16 x 4 by
// eight wavefronts is not built for groups of 128: its costs there serve the mean.)
struct FormCost {
    double first, more;
};
constexpr FormCost kCost128[qlin::kW4Forms] = {{4.0, 3.8}, {4.5, 4.5}, {6.0, 5.8}, {5.9, 5.6}, {10.2, 10.2}, {27, 29}, {44, 68}};
constexpr FormCost kCost32[qlin::kW4Forms] = {{4.5, 4.3}, {5.5, 5.2}, {9.3, 7.8}, {10, 7.4}, {13.6, 14.5}, {44, 37}, {92, 126}};

double form_cost(int form, const qlin::W4Call& c, bool pair, int64_t blocks) {
    const double w = (double)(blocks * qlin::w4_units(form, c, pair)) / 256.0;
    FormCost f = kCost128[form];
    const FormCost g = kCost32[form];
    if (c.group == 32) f = g;
    if (c.group == 64) f = FormCost{(f.first + g.first) / 2, (f.more + g.more) / 2};
    if (w <= 1.0) return f.first;
    if (form == qlin::kW4Tiled64x8) return std::ceil(w) * f.more;
    if (form == qlin::kW4Tiled64x16) {           // pairs, and what is left after them
        const double pairs = std::floor(w / 2), rest = w - 2 * pairs;
        return pairs * f.more + (rest > 1.0 ? f.more : rest > 0.0 ? f.first : 0.0);
    }
    return std::max(1.5 * f.first, w * f.more);
}
// The grid of one launch holds fewer than 2^32 threads.
bool form_fits(int form, const qlin::W4Call& c, bool pair, int64_t blocks) {
    return blocks * qlin::w4_units(form, c, pair) < (int64_t(1) << 32) / qlin::kW4FormThreads[form];
}
// The cheapest form for items (token blocks) of `rows` rows of x at most, or any where rows is 0; -1: none fits.
int choose_form(const qlin::W4Call& c, bool pair, bool experts, int rows) {
    int best = -1;
    double least = 0;
    for (int f = 0; f < qlin::kW4Forms; ++f) {
        if (!qlin::w4_form_built(f, c.group, pair) || (rows && qlin::kW4FormRows[f] != rows)) continue;
        const int64_t blocks = qlin::w4_blocks(f, c, experts);
        if (!form_fits(f, c, pair, blocks)) continue;
        const double cost = form_cost(f, c, pair, blocks);
        if (best < 0 || cost < least) {
            best = f;
            least = cost;
        }
    }
    return best;
}
hipError_t product(int form, const qlin::W4Call& c, bool pair, bool experts, hipStream_t st) {
    return form >= qlin::kW4Tiled64x8 ? qlin::launch_w4_tiled(form, c, pair, experts, st)
                                      : qlin::launch_w4_stream(form, c, pair, experts, st);
}

}  // namespace

extern "C" {

int64_t qlin_w4_packed_bytes(int64_t N, int64_t K) {
    if (!valid_mn(N) || !valid_k(K)) return 0;
    return qlin::w4_row_tiles(N) * qlin::w4_k_tiles(K) * qlin::kW4Block;
}

int64_t qlin_w4_packed_scales(int64_t N, int64_t K, int32_t group) {
    if (!valid_mn(N) || !valid_k(K) || !valid_group(group, K)) return 0;
    return qlin::w4_row_tiles(N) * qlin::w4_k_tiles(K) * qlin::kW4Rows * (qlin::kW4K / group);
}

qlin_status qlin_pack_w4(const uint8_t* q_w, const uint16_t* s_w, const uint8_t* z_w, int64_t E, int64_t N, int64_t K,
                         int32_t group, uint8_t* q_w_packed, uint16_t* s_w_packed, uint8_t* z_w_packed,
                         hipStream_t stream) {
    if (E < 0 || E > QLIN_MAX_EXPERTS || !valid_mn(N) || !valid_k(K) || !valid_group(group, K)) return QLIN_ERR_SHAPE;
    if (E == 0 || N == 0) return QLIN_OK;
    if (!q_w || !s_w || !q_w_packed || !s_w_packed || (z_w == nullptr) != (z_w_packed == nullptr)) return QLIN_ERR_NULL;
    if (!aligned(q_w, 16) || !aligned(s_w, 2) || !aligned(q_w_packed, 16) || !aligned(s_w_packed, 8) || !aligned(z_w_packed, 4))
        return QLIN_ERR_ALIGN;
    const int64_t scales = E * N * (K / group), packed = E * qlin_w4_packed_scales(N, K, group);
    const Range in[3] = {rng(q_w, E * N * (K / 2)), rng(s_w, 2 * scales), rng(z_w, z_w ? scales : 0)};
    const Range out[3] = {rng(q_w_packed, E * qlin_w4_packed_bytes(N, K)), rng(s_w_packed, 2 * packed),
                          rng(z_w_packed, z_w ? packed : 0)};
    for (int i = 0; i < 3; ++i)
        for (int j = 0; j < 3; ++j)
            if (overlap(out[i], in[j]) || (i != j && overlap(out[i], out[j]))) return QLIN_ERR_ALIAS;
    return qlin::hip_status(qlin::launch_pack_w4(q_w, s_w, z_w, E, N, K, group, q_w_packed, s_w_packed, z_w_packed, stream));
}

qlin_status qlin_linear_w4(const uint16_t* x, int64_t M, int64_t K, int32_t group, const qlin_w4_weight* weights,
                           void* const* y, int32_t nw, qlin_out out, hipStream_t stream) {
    if (!weights || !y) return QLIN_ERR_NULL;
    if (nw < 1 || nw > QLIN_MAX_SEGMENTS) return QLIN_ERR_SHAPE;
    if (!valid_mn(M) || !valid_k(K) || !valid_group(group, K)) return QLIN_ERR_SHAPE;
    if (out != QLIN_OUT_BF16 && out != QLIN_OUT_F32) return QLIN_ERR_UNSUPPORTED;
    int64_t rows = 0;
    for (int i = 0; i < nw; ++i) {
        if (!valid_mn(weights[i].n)) return QLIN_ERR_SHAPE;
        rows += weights[i].n;
    }
    if (rows > QLIN_MAX_MN || M * rows > kMaxElements) return QLIN_ERR_SHAPE;
    if (M == 0 || rows == 0) return QLIN_OK;
    if (!x) return QLIN_ERR_NULL;
    if (!aligned(x, 16)) return QLIN_ERR_ALIGN;
    qlin::W4Call c{};
    c.x = x;
    c.mode = (int)out;
    c.group = group;
    c.M = M;
    c.K = K;
    const Range rx = rng(x, 2 * M * K);
    const int64_t size = out == QLIN_OUT_F32 ? 4 : 2;
    for (int i = 0; i < nw; ++i) {
        if (weights[i].n == 0) continue;
        const qlin_status st = check_pointers(weights[i]);
        if (st != QLIN_OK) return st;
        if (!y[i]) return QLIN_ERR_NULL;
        if (!aligned(y[i], 16)) return QLIN_ERR_ALIGN;
        const Range ry = rng(y[i], size * M * weights[i].n);
        if (overlap(ry, rx)) return QLIN_ERR_ALIAS;
        for (int j = 0; j < nw; ++j) {
            if (weights[j].n == 0) continue;
            if (overlap(ry, ranges(weights[j], 1, K, group))) return QLIN_ERR_ALIAS;
            if (j != i && y[j] && overlap(ry, rng(y[j], size * M * weights[j].n))) return QLIN_ERR_ALIAS;
        }
        c.w[c.nseg] = weights[i].q_w;
        c.s[c.nseg] = weights[i].s_w;
        c.z[c.nseg] = weights[i].z_w;
        c.y[c.nseg] = y[i];
        c.n[c.nseg] = (int)weights[i].n;
        ++c.nseg;
    }
    const int form = choose_form(c, false, false, 0);
    if (form < 0) return QLIN_ERR_SHAPE;
    return qlin::hip_status(product(form, c, false, false, stream));
}

qlin_status qlin_linear_swiglu_w4(const uint16_t* x, int64_t M, int64_t K, int32_t group, const qlin_w4_weight* gate,
                                  const qlin_w4_weight* up, uint16_t* h, hipStream_t stream) {
    if (!gate || !up) return QLIN_ERR_NULL;
    if (!valid_mn(M) || !valid_k(K) || !valid_group(group, K)) return QLIN_ERR_SHAPE;
    const int64_t I = gate->n;
    if (!valid_mn(I) || up->n != I || 2 * I > QLIN_MAX_MN || M * I > kMaxElements) return QLIN_ERR_SHAPE;
    if (M == 0 || I == 0) return QLIN_OK;
    if (!x || !h) return QLIN_ERR_NULL;
    for (const qlin_w4_weight* w : {gate, up}) {
        const qlin_status st = check_pointers(*w);
        if (st != QLIN_OK) return st;
    }
    if (!aligned(x, 16) || !aligned(h, 16)) return QLIN_ERR_ALIGN;
    const Range rh = rng(h, 2 * M * I);
    if (overlap(rh, rng(x, 2 * M * K)) || overlap(rh, ranges(*gate, 1, K, group)) || overlap(rh, ranges(*up, 1, K, group)))
        return QLIN_ERR_ALIAS;
    qlin::W4Call c{};
    c.x = x;
    c.w[0] = gate->q_w, c.w[1] = up->q_w;
    c.s[0] = gate->s_w, c.s[1] = up->s_w;
    c.z[0] = gate->z_w, c.z[1] = up->z_w;
    c.y[0] = h;
    c.n[0] = c.n[1] = (int)I;
    c.nseg = 2;
    c.mode = QLIN_OUT_BF16;
    c.group = group;
    c.M = M;
    c.K = K;
    const int form = choose_form(c, true, false, 0);
    if (form < 0) return QLIN_ERR_SHAPE;
    return qlin::hip_status(product(form, c, true, false, stream));
}

qlin_status qlin_route(const void* logits, qlin_out logits_type, int64_t T, int64_t E, int32_t k, qlin_score score,
                       const float* bias, int32_t groups, int32_t top_groups, int32_t group_best, int32_t renormalize,
                       float scale, int32_t* ids, float* weights, hipStream_t stream) {
    if (logits_type != QLIN_OUT_BF16 && logits_type != QLIN_OUT_F32) return QLIN_ERR_UNSUPPORTED;
    if (score != QLIN_SCORE_SOFTMAX && score != QLIN_SCORE_SIGMOID) return QLIN_ERR_UNSUPPORTED;
    if (!valid_mn(T) || E < 1 || E > QLIN_MAX_EXPERTS) return QLIN_ERR_SHAPE;
    if (groups < 1 || groups > QLIN_MAX_GROUPS || E % groups != 0 || top_groups < 1 || top_groups > groups) return QLIN_ERR_SHAPE;
    if (group_best < 1 || group_best > 2) return QLIN_ERR_SHAPE;
    if (k < 1 || k > QLIN_MAX_CHOICES || k > top_groups * (E / groups)) return QLIN_ERR_SHAPE;
    if (T == 0) return QLIN_OK;
    if (!logits || !ids || !weights) return QLIN_ERR_NULL;
    if (!aligned(logits, logits_type == QLIN_OUT_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return QLIN_ERR_ALIGN;
    const Range rl = rng(logits, T * E * (logits_type == QLIN_OUT_F32 ? 4 : 2)), rb = rng(bias, bias ? 4 * E : 0);
    const Range ri = rng(ids, 4 * T * k), rw = rng(weights, 4 * T * k);
    if (overlap(ri, rl) || overlap(rw, rl) || overlap(ri, rb) || overlap(rw, rb) || overlap(ri, rw)) return QLIN_ERR_ALIAS;
    return qlin::hip_status(qlin::launch_route(logits, logits_type == QLIN_OUT_F32, T, (int)E, k, (int)score, bias, groups,
                                               top_groups, group_best, renormalize != 0, scale, ids, weights, stream));
}

}  // extern "C"

namespace {

// The experts' workspace, every part 16-byte aligned.
struct Workspace {
    int64_t order, items, nitems, h, rows, bytes;
};
// Few ids: the workgroups of gate and up find the rows of their item themselves
// (w4_stream.hip), with no launch for the sorting: 37 tokens of 6 choices among
// 40 experts 43.4 -> 40.5 us, 16 tokens of 2 among 8: 18.8 -> 15.6.
bool own_items(int64_t slots, int64_t E) { return slots <= qlin::kOwnItemSlots && E <= qlin::kOwnItemExperts; }
// Few tokens: multiply each slot by its own expert's weights, with no sorting
// and the weighted sum inside the down product (two launches), or sort the slots
// by expert and read the weights of each expert once (three or four)?  Estimates
// in us.  Direct: one round of the 256 CUs per 256 / (H / 16) tokens, which each
// take the k * I / 128 blocks of a row tile with 16 wavefronts (half a round or
// less takes three quarters of one).  Sorted: the launches, and the expected
// number of different experts times their bytes at 5.6 TB/s.  Measured, direct
// and sorted: 64 experts of 2048 x 1024, 8 choices, 1, 2, 4 and 8 tokens: 13.7 and
// 16.1, 17.8 and 21.2, 30.0 and 28.6, 52 and 37; 8 such experts, 2 choices, 2, 4
// and 8 tokens: 11.8 and 12.4, 19.2 and 14.8, 31 and 14.9; 16 experts of
// 1024 x 512, 2 choices, 4, 8 and 16 tokens: 9.0 and 11.6, 13.3 and 12.4, 20.9 and
// 12.9; 300 of 512 x 256, 4 choices, 8 tokens: 9.7 and 19.1.
bool direct_is_faster(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    const int64_t groups = T * qlin::w4_row_tiles(H);
    if (groups >= (int64_t(1) << 22)) return false;   // 1024 threads each, below 2^32 of one launch
    const double rounds = groups <= 128 ? 0.75 : std::ceil((double)groups / 256.0);
    const double direct = 5.5 + rounds * (4.0 + 1.5 * (double)(k * qlin::w4_k_tiles(I)) / 16.0);
    const double different = (double)E * (1.0 - std::pow(1.0 - 1.0 / (double)E, (double)(T * k)));
    return direct < (own_items(T * k, E) ? 11.0 : 14.0) + different * 1.4 * (double)H * (double)I / 5.2e6;
}

// Items of at most `rows` rows that the routed rows of E experts can need.
int64_t max_items(int64_t slots, int64_t E, int rows) { return (slots < E ? slots : E) + slots / rows; }

Workspace layout(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    const int64_t slots = T * k;
    auto pad = [](int64_t b) { return (b + 255) & ~int64_t(255); };
    // laid out alike whether the slots are sorted or not: the size grows with T
    Workspace w{};
    w.order = 0;
    w.items = w.order + pad(4 * slots);
    w.nitems = w.items + pad(12 * max_items(slots, E, 16));
    w.h = w.nitems + 256;
    w.rows = w.h + pad(4 * slots * I);   // two bf16 parts
    w.bytes = w.rows + pad(4 * slots * H);
    return w;
}

bool experts_sizes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I) {
    if (!valid_mn(T) || k < 1 || k > QLIN_MAX_CHOICES || T * k > QLIN_MAX_MN) return false;
    if (E < 1 || E > QLIN_MAX_EXPERTS || !valid_k(H) || !valid_k(I)) return false;
    return T * k * (H > I ? H : I) <= kMaxElements;
}

}  // namespace

extern "C" {

int64_t qlin_experts_w4_workspace(int64_t T, int32_t k, int64_t E, int64_t H, int64_t I) {
    if (!experts_sizes(T, k, E, H, I) || T == 0) return 0;   // no tokens: nothing is launched
    return layout(T, k, E, H, I).bytes;
}

qlin_status qlin_experts_w4(const uint16_t* x, int64_t T, int64_t H, int64_t I, int64_t E, int32_t k, int32_t group,
                            const int32_t* ids, const float* weights, const qlin_w4_weight* gate,
                            const qlin_w4_weight* up, const qlin_w4_weight* down, uint16_t* y, void* workspace,
                            hipStream_t stream) {
    if (!gate || !up || !down) return QLIN_ERR_NULL;
    if (!experts_sizes(T, k, E, H, I) || !valid_group(group, H) || !valid_group(group, I)) return QLIN_ERR_SHAPE;
    if (gate->n != I || up->n != I || down->n != H) return QLIN_ERR_SHAPE;
    if (T == 0) return QLIN_OK;
    if (!x || !ids || !weights || !y || !workspace) return QLIN_ERR_NULL;
    for (const qlin_w4_weight* w : {gate, up, down}) {
        const qlin_status st = check_pointers(*w);
        if (st != QLIN_OK) return st;
    }
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(workspace, 16) || !aligned(ids, 4) || !aligned(weights, 4))
        return QLIN_ERR_ALIGN;
    const int64_t slots = T * k;
    const Workspace l = layout(T, k, E, H, I);
    const Range ry = rng(y, 2 * T * H), rw = rng(workspace, l.bytes);
    if (overlap(ry, rw)) return QLIN_ERR_ALIAS;
    for (Range written : {ry, rw}) {
        if (overlap(written, rng(x, 2 * T * H)) || overlap(written, rng(ids, 4 * slots)) ||
            overlap(written, rng(weights, 4 * slots)))
            return QLIN_ERR_ALIAS;
        if (overlap(written, ranges(*gate, E, H, group)) || overlap(written, ranges(*up, E, H, group)) ||
            overlap(written, ranges(*down, E, I, group)))
            return QLIN_ERR_ALIAS;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    int* order = reinterpret_cast<int*>(ws + l.order);
    int* items = reinterpret_cast<int*>(ws + l.items);
    int* nitems = reinterpret_cast<int*>(ws + l.nitems);
    uint16_t* h = reinterpret_cast<uint16_t*>(ws + l.h);
    float* rows = reinterpret_cast<float*>(ws + l.rows);

    // gate and up, then down
    qlin::W4Call a{}, b{};
    a.group = b.group = group;
    a.ids = b.ids = ids;
    a.E = b.E = (int)E;
    a.x = x;
    a.w[0] = gate->q_w, a.w[1] = up->q_w;
    a.s[0] = gate->s_w, a.s[1] = up->s_w;
    a.z[0] = gate->z_w, a.z[1] = up->z_w;
    a.y[0] = h;
    a.n[0] = a.n[1] = (int)I;
    a.nseg = 2;
    a.mode = QLIN_OUT_BF16;
    a.K = H;
    a.xdiv = k;
    b.x = h;
    b.w[0] = down->q_w;
    b.s[0] = down->s_w;
    b.z[0] = down->z_w;
    b.y[0] = rows;
    b.n[0] = (int)H;
    b.nseg = 1;
    b.mode = QLIN_OUT_F32;
    b.K = I;
    b.xdiv = 1;
    a.max_items = b.max_items = slots;
    const int one_by_one = direct_is_faster(T, k, E, H, I) ? choose_form(a, true, true, 16) : -1;
    if (one_by_one >= 0) {
        const hipError_t e = product(one_by_one, a, true, true, stream);
        if (e != hipSuccess) return qlin::hip_status(e);
        return qlin::hip_status(qlin::launch_experts_down_direct(b, weights, T, k, y, stream));
    }
    // the rows of an item: those of the cheapest pair of forms
    int form_a = -1, form_b = -1, item_rows = 0;
    double least = 0;
    for (int r = 16; r <= 64; r *= 2) {
        a.max_items = b.max_items = max_items(slots, E, r);
        const int fa = choose_form(a, true, true, r), fb = choose_form(b, false, true, r);
        if (fa < 0 || fb < 0) continue;
        const double cost = form_cost(fa, a, true, a.max_items) * (double)H + form_cost(fb, b, false, b.max_items) * (double)I;
        if (item_rows == 0 || cost < least) {
            form_a = fa, form_b = fb, item_rows = r;
            least = cost;
        }
    }
    if (item_rows == 0) return QLIN_ERR_SHAPE;
    a.max_items = b.max_items = max_items(slots, E, item_rows);
    a.order = b.order = order;
    a.items = b.items = items;
    a.nitems = b.nitems = nitems;
    hipError_t e = hipSuccess;
    if (item_rows < 64 && own_items(slots, E)) a.slots = (int)slots;
    else e = qlin::launch_experts_plan(ids, slots, (int)E, item_rows, order, items, nitems, stream);
    if (e == hipSuccess) e = product(form_a, a, true, true, stream);
    if (e == hipSuccess) e = product(form_b, b, false, true, stream);
    if (e == hipSuccess) e = qlin::launch_experts_combine(rows, ids, weights, T, k, (int)E, H, y, stream);
    return qlin::hip_status(e);
}

}  // extern "C"
