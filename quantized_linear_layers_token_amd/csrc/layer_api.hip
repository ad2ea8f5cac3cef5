// C ABI of the norm, rotary, cache and attention calls: argument validation
// and dispatch.  No allocation, no synchronization; every check runs before the
// first launch.
#include <stdint.h>

#include <cmath>
#include <initializer_list>

#include "../../include/qlin_layer.h"
#include "layer_internal.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;
};
Range rng(const void* p, int64_t bytes) {
    const uintptr_t b = reinterpret_cast<uintptr_t>(p);
    return p ? Range{b, b + (uintptr_t)bytes} : Range{0, 0};
}
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
bool any_overlap(std::initializer_list<Range> outputs, std::initializer_list<Range> inputs) {
    for (const Range* o = outputs.begin(); o != outputs.end(); ++o) {
        for (const Range& i : inputs)
            if (overlap(*o, i)) return true;
        for (const Range* p = outputs.begin(); p != o; ++p)
            if (overlap(*o, *p)) return true;
    }
    return false;
}

// The heads of T tokens: `width` elements of bf16 every `stride`.
struct Heads {
    const uint16_t* p;
    int64_t T, stride, width;
    Range range() const { return rng(p, 2 * ((T - 1) * stride + width)); }
};
bool overlap(const Heads& a, const Heads& b) {
    if (!a.p || !b.p || !overlap(a.range(), b.range())) return false;
    if (a.stride != b.stride) return true;
    // parts of the same rows: apart where one ends before the other begins, in every row
    const int64_t bytes = 2 * a.stride;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    const int64_t off = y >= x ? (int64_t)((y - x) % (uintptr_t)bytes) : (bytes - (int64_t)((x - y) % (uintptr_t)bytes)) % bytes;
    return off < 2 * a.width || off + 2 * b.width > bytes;
}

bool valid_count(int64_t v) { return v >= 0 && v <= QLIN_MAX_MN; }
bool valid_heads(int32_t v) { return v >= 1 && v <= QLIN_MAX_HEADS; }
bool valid_dim(int32_t v) { return v >= 16 && v <= QLIN_MAX_HEAD_DIM && v % 16 == 0; }
bool valid_stride(int64_t v, int64_t width) { return v >= width && v % 8 == 0 && v <= (int64_t(1) << 31); }
bool valid_eps(float e) { return e >= 1e-20f && e <= 1.0f; }

qlin_status check_rotation(const qlin_rotation& r, int32_t dim) {
    if (!r.frequencies) return QLIN_ERR_NULL;
    if (r.dims < 16 || r.dims > dim || r.dims % 16) return QLIN_ERR_SHAPE;
    if (!aligned(r.frequencies, 8)) return QLIN_ERR_ALIGN;
    if (r.interleaved != 0 && r.interleaved != 1) return QLIN_ERR_UNSUPPORTED;
    return std::isfinite(r.strength) ? QLIN_OK : QLIN_ERR_UNSUPPORTED;
}

qlin_status check_cache(const qlin_kv_cache& c) {
    if (c.kind != QLIN_CACHE_BF16 && c.kind != QLIN_CACHE_INT8 && c.kind != QLIN_CACHE_FP8) return QLIN_ERR_UNSUPPORTED;
    if (!valid_heads(c.kv_heads) || !valid_dim(c.dim) || c.page_size < 16 || c.page_size % 16) return QLIN_ERR_SHAPE;
    if (c.pages < 1 || c.pages > 0x7fffffff / c.page_size) return QLIN_ERR_SHAPE;
    if (!c.k || !c.v) return QLIN_ERR_NULL;
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return QLIN_ERR_ALIGN;
    if (c.kind != QLIN_CACHE_BF16) {
        if (!c.k_scale || !c.v_scale) return QLIN_ERR_NULL;
        if (!aligned(c.k_scale, 16) || !aligned(c.v_scale, 16)) return QLIN_ERR_ALIGN;
    }
    return QLIN_OK;
}
struct CacheRanges {
    Range k, v, ks, vs;
};
CacheRanges ranges(const qlin_kv_cache& c) {
    const int64_t rows = c.pages * c.kv_heads * c.page_size, bytes = rows * c.dim * (c.kind == QLIN_CACHE_BF16 ? 2 : 1);
    const int64_t scales = c.kind == QLIN_CACHE_BF16 ? 0 : 4 * rows;
    return CacheRanges{rng(c.k, bytes), rng(c.v, bytes), rng(c.k_scale, scales), rng(c.v_scale, scales)};
}

qlin_status norm(qlin::NormOut out, const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, int64_t M, int64_t K,
                 float eps, uint16_t* sum, void* y, float* s, hipStream_t stream) {
    if (!valid_count(M) || K <= 0 || K % 16 || K > QLIN_MAX_K) return QLIN_ERR_SHAPE;
    if (out == qlin::kNormFp8Block && K % 128) return QLIN_ERR_SHAPE;
    if (!valid_eps(eps)) return QLIN_ERR_UNSUPPORTED;
    if (M == 0) return QLIN_OK;
    const bool codes = out != qlin::kNormBf16;
    if (!x || !gamma || !y || (codes && !s) || !residual != !sum) return QLIN_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(gamma, 16) || !aligned(sum, 16) || !aligned(y, 16) || !aligned(s, 4))
        return QLIN_ERR_ALIGN;
    const int64_t rows = 2 * M * K;
    const Range yr = rng(y, codes ? M * K : rows), sr = rng(s, codes ? 4 * M * (out == qlin::kNormFp8Block ? K / 128 : 1) : 0);
    const Range xr = rng(x, rows), rr = rng(residual, rows), gr = rng(gamma, 2 * K), tr = rng(sum, rows);
    if (any_overlap({yr, sr, tr}, {gr}) || any_overlap({yr, sr}, {xr, rr})) return QLIN_ERR_ALIAS;
    if ((sum != x && overlap(tr, xr)) || (sum != residual && overlap(tr, rr))) return QLIN_ERR_ALIAS;
    return qlin::hip_status(qlin::launch_norm(out, qlin::NormCall{x, residual, gamma, sum, y, s, M, K, eps}, stream));
}

}  // namespace

extern "C" {

qlin_status qlin_norm_bf16(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, int64_t M, int64_t K, float eps,
                           uint16_t* sum, uint16_t* y, hipStream_t stream) {
    return norm(qlin::kNormBf16, x, residual, gamma, M, K, eps, sum, y, nullptr, stream);
}

qlin_status qlin_norm_int8(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, int64_t M, int64_t K, float eps,
                           uint16_t* sum, int8_t* q, float* s, hipStream_t stream) {
    return norm(qlin::kNormInt8, x, residual, gamma, M, K, eps, sum, q, s, stream);
}

qlin_status qlin_norm_fp8(const uint16_t* x, const uint16_t* residual, const uint16_t* gamma, int64_t M, int64_t K, float eps,
                          int32_t group, uint16_t* sum, uint8_t* q, float* s, hipStream_t stream) {
    if (group != 0 && group != 128) return QLIN_ERR_SHAPE;
    return norm(group ? qlin::kNormFp8Block : qlin::kNormFp8, x, residual, gamma, M, K, eps, sum, q, s, stream);
}

qlin_status qlin_rope(const uint16_t* x, int64_t x_stride, const int32_t* positions, int64_t T, int32_t heads, int32_t dim,
                      const qlin_rotation* rope, const uint16_t* gamma, float eps, uint16_t* y, int64_t y_stride, hipStream_t stream) {
    if (!valid_count(T) || !valid_heads(heads) || !valid_dim(dim)) return QLIN_ERR_SHAPE;
    const int64_t width = (int64_t)heads * dim;
    if (!valid_stride(x_stride, width) || !valid_stride(y_stride, width)) return QLIN_ERR_SHAPE;
    if (!rope) return QLIN_ERR_NULL;
    const qlin_status r = check_rotation(*rope, dim);
    if (r != QLIN_OK) return r;
    if (gamma && !valid_eps(eps)) return QLIN_ERR_UNSUPPORTED;
    if (T == 0) return QLIN_OK;
    if (!x || !positions || !y) return QLIN_ERR_NULL;
    if (!aligned(x, 16) || !aligned(y, 16) || !aligned(gamma, 16) || !aligned(positions, 4)) return QLIN_ERR_ALIGN;
    const Heads in{x, T, x_stride, width}, out{y, T, y_stride, width};
    if (!(x == y && x_stride == y_stride) && overlap(in, out)) return QLIN_ERR_ALIAS;
    if (any_overlap({out.range()}, {rng(positions, 4 * T), rng(rope->frequencies, 4 * rope->dims), rng(gamma, 2 * dim)})) return QLIN_ERR_ALIAS;
    qlin::HeadsCall c{};
    c.q = x;
    c.q_stride = x_stride;
    c.q_out = y;
    c.q_out_stride = y_stride;
    c.q_gamma = gamma;
    c.eps = eps;
    c.positions = positions;
    c.rope = *rope;
    c.heads = heads;
    c.dim = dim;
    c.inv_dim = 1.0f / (float)dim;
    c.T = T;
    return qlin::hip_status(qlin::launch_heads(c, stream));
}

qlin_status qlin_cache_write(const qlin_kv_cache* cache, const int32_t* slots, int64_t T, const uint16_t* k, int64_t k_stride,
                             const uint16_t* v, int64_t v_stride, const int32_t* positions, const qlin_rotation* rope,
                             const uint16_t* k_gamma, float eps, const qlin_queries* queries, hipStream_t stream) {
    if (!cache) return QLIN_ERR_NULL;
    qlin_status r = check_cache(*cache);
    if (r != QLIN_OK) return r;
    if (!valid_count(T)) return QLIN_ERR_SHAPE;
    const int32_t dim = cache->dim;
    const int64_t width = (int64_t)cache->kv_heads * dim;
    if (!valid_stride(k_stride, width) || !valid_stride(v_stride, width)) return QLIN_ERR_SHAPE;
    if (rope && (r = check_rotation(*rope, dim)) != QLIN_OK) return r;
    int64_t q_width = 0;
    if (queries) {
        if (!valid_heads(queries->heads)) return QLIN_ERR_SHAPE;
        q_width = (int64_t)queries->heads * dim;
        if (!valid_stride(queries->stride, q_width) || !valid_stride(queries->out_stride, q_width)) return QLIN_ERR_SHAPE;
        if (!rope && !queries->gamma) return QLIN_ERR_NULL;   // nothing to do with them
    }
    const uint16_t* q_gamma = queries ? queries->gamma : nullptr;
    if ((k_gamma || q_gamma) && !valid_eps(eps)) return QLIN_ERR_UNSUPPORTED;
    if (T == 0) return QLIN_OK;
    if (!slots || !k || !v || (rope && !positions) || (queries && (!queries->q || !queries->out))) return QLIN_ERR_NULL;
    if (!aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16) || !aligned(positions, 4) || !aligned(k_gamma, 16) || !aligned(q_gamma, 16))
        return QLIN_ERR_ALIGN;
    if (queries && (!aligned(queries->q, 16) || !aligned(queries->out, 16))) return QLIN_ERR_ALIGN;
    const Heads kh{k, T, k_stride, width}, vh{v, T, v_stride, width};
    const Heads qh{queries ? queries->q : nullptr, T, queries ? queries->stride : 0, q_width};
    const Heads oh{queries ? queries->out : nullptr, T, queries ? queries->out_stride : 0, q_width};
    const bool in_place = queries && qh.p == oh.p && qh.stride == oh.stride;
    if (overlap(oh, kh) || overlap(oh, vh) || (!in_place && overlap(oh, qh))) return QLIN_ERR_ALIAS;
    const CacheRanges cr = ranges(*cache);
    const Range small[] = {rng(slots, 4 * T), rng(rope ? positions : nullptr, 4 * T), rng(rope ? rope->frequencies : nullptr, rope ? 4 * rope->dims : 0),
                           rng(k_gamma, 2 * dim), rng(q_gamma, 2 * dim)};
    if (any_overlap({cr.k, cr.v, cr.ks, cr.vs, oh.p ? oh.range() : Range{0, 0}}, {small[0], small[1], small[2], small[3], small[4]}))
        return QLIN_ERR_ALIAS;
    if (any_overlap({cr.k, cr.v, cr.ks, cr.vs}, {kh.range(), vh.range(), qh.p ? qh.range() : Range{0, 0}})) return QLIN_ERR_ALIAS;
    qlin::HeadsCall c{};
    if (queries) {
        c.q = queries->q;
        c.q_stride = queries->stride;
        c.q_out = queries->out;
        c.q_out_stride = queries->out_stride;
        c.q_gamma = queries->gamma;
        c.heads = queries->heads;
    }
    c.k = k;
    c.v = v;
    c.k_stride = k_stride;
    c.v_stride = v_stride;
    c.k_gamma = k_gamma;
    c.eps = eps;
    c.positions = positions;
    c.slots = slots;
    if (rope) c.rope = *rope;
    c.cache = *cache;
    c.kv_heads = cache->kv_heads;
    c.dim = dim;
    c.inv_dim = 1.0f / (float)dim;
    c.T = T;
    return qlin::hip_status(qlin::launch_heads(c, stream));
}

qlin_status qlin_cache_read(const qlin_kv_cache* cache, const int32_t* slots, int64_t n, uint16_t* k, uint16_t* v, hipStream_t stream) {
    if (!cache) return QLIN_ERR_NULL;
    const qlin_status r = check_cache(*cache);
    if (r != QLIN_OK) return r;
    if (!valid_count(n)) return QLIN_ERR_SHAPE;
    if (n == 0) return QLIN_OK;
    if (!slots || !k || !v) return QLIN_ERR_NULL;
    if (!aligned(slots, 4) || !aligned(k, 16) || !aligned(v, 16)) return QLIN_ERR_ALIGN;
    const int64_t bytes = 2 * n * cache->kv_heads * cache->dim;
    const CacheRanges cr = ranges(*cache);
    if (any_overlap({rng(k, bytes), rng(v, bytes)}, {rng(slots, 4 * n), cr.k, cr.v, cr.ks, cr.vs})) return QLIN_ERR_ALIAS;
    return qlin::hip_status(qlin::launch_cache_read(*cache, slots, n, k, v, stream));
}

int64_t qlin_attn_decode_workspace(int32_t heads, int32_t kv_heads, int32_t dim) {
    if (!valid_heads(heads) || !valid_heads(kv_heads) || heads % kv_heads || !valid_dim(dim)) return 0;
    return qlin::attn_workspace(heads, kv_heads, dim);
}

qlin_status qlin_attn_decode(const uint16_t* q, const qlin_kv_cache* cache, const int32_t* pages, int64_t S, int32_t heads,
                             int64_t page_columns, const int32_t* lengths, int64_t window, float scale, uint16_t* out,
                             void* workspace, hipStream_t stream) {
    if (!cache) return QLIN_ERR_NULL;
    const qlin_status r = check_cache(*cache);
    if (r != QLIN_OK) return r;
    if (!valid_count(S) || !valid_heads(heads) || heads % cache->kv_heads) return QLIN_ERR_SHAPE;
    if (page_columns < 0 || page_columns > (int64_t(1) << 30) / cache->page_size || window < 0) return QLIN_ERR_SHAPE;
    if (!std::isfinite(scale)) return QLIN_ERR_UNSUPPORTED;
    if (S == 0) return QLIN_OK;
    if (!q || (page_columns && !pages) || !lengths || !out || !workspace) return QLIN_ERR_NULL;
    if (!aligned(q, 16) || !aligned(pages, 4) || !aligned(lengths, 4) || !aligned(out, 16) || !aligned(workspace, 16)) return QLIN_ERR_ALIGN;
    const int64_t rows = 2 * S * heads * cache->dim;
    const CacheRanges cr = ranges(*cache);
    if (any_overlap({rng(out, rows), rng(workspace, qlin::attn_workspace(heads, cache->kv_heads, cache->dim))},
                    {rng(q, rows), rng(pages, 4 * S * page_columns), rng(lengths, 4 * S), cr.k, cr.v, cr.ks, cr.vs}))
        return QLIN_ERR_ALIAS;
    qlin::AttnCall c{};
    c.q = q;
    c.cache = *cache;
    c.pages = pages;
    c.lengths = lengths;
    c.out = out;
    c.workspace = workspace;
    c.S = (int)S;
    c.heads = heads;
    c.columns = (int)page_columns;
    c.window = window > (int64_t(1) << 30) ? 0 : (int)window;   // (no sequence is longer)
    c.scale = scale;
    return qlin::hip_status(qlin::launch_attn(c, stream));
}

}  // extern "C"
