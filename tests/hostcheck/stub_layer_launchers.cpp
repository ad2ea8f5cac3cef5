// Host-only stand-ins for the launchers of the norm, rotary, cache and attention calls, linked with their C-ABI layer
// (layer_api.hip) into a sanitizer build that runs on a CPU: every launcher counts and returns success without touching
// memory.  Test infrastructure: never part of libqlin.so.
#include "../../quantized_linear_layers_token_amd/csrc/layer_internal.h"

namespace {
int g_launches = 0;
bool g_bad = false;   // arguments that a kernel does not take
hipError_t reached() {
    ++g_launches;
    return hipSuccess;
}
bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
void cache_ok(const qlin_kv_cache& c) {
    g_bad |= !c.k || !c.v || c.page_size % 16 || c.page_size <= 0 || c.pages < 1 || c.pages * c.page_size > 0x7fffffff;
    g_bad |= c.dim % 16 || c.dim < 16 || c.dim > 256 || c.kv_heads < 1;
    g_bad |= c.kind != QLIN_CACHE_BF16 && (!aligned(c.k_scale, 16) || !c.k_scale || !c.v_scale);
}
}  // namespace

extern "C" int layer_launches(void) { return g_launches; }
extern "C" int layer_bad(void) { return g_bad; }

namespace qlin {
qlin_status hip_status(hipError_t e) { return e == hipSuccess ? QLIN_OK : QLIN_ERR_HIP; }
hipError_t launch_norm(NormOut out, const NormCall& c, hipStream_t) {
    g_bad |= c.K % 16 || (out == kNormFp8Block && c.K % 128) || c.M < 1 || !c.residual != !c.sum || (out != kNormBf16 && !c.s) || !(c.eps > 0);
    return reached();
}
hipError_t launch_heads(const HeadsCall& c, hipStream_t) {
    g_bad |= c.dim % 16 || c.dim < 16 || c.dim > 256 || c.T < 1 || c.heads + c.kv_heads < 1;
    g_bad |= c.rope.frequencies && (c.rope.dims % 16 || c.rope.dims > c.dim || !c.positions);
    if (c.kv_heads) {
        cache_ok(c.cache);
        g_bad |= c.cache.dim != c.dim || c.cache.kv_heads != c.kv_heads || !c.slots || !c.k || !c.v;
    }
    if (c.heads) g_bad |= !c.q || !c.q_out || (!c.rope.frequencies && !c.q_gamma);
    return reached();
}
hipError_t launch_cache_read(const qlin_kv_cache& cache, const int* slots, int64_t n, uint16_t* k, uint16_t* v, hipStream_t) {
    cache_ok(cache);
    g_bad |= !slots || n < 1 || !k || !v;
    return reached();
}
int64_t attn_workspace(int heads, int kv_heads, int dim) { return (int64_t)heads / kv_heads * dim * 1024; }
hipError_t launch_attn(const AttnCall& c, hipStream_t) {
    cache_ok(c.cache);
    g_bad |= c.S < 1 || c.heads % c.cache.kv_heads || (int64_t)c.columns * c.cache.page_size > (1 << 30) || c.window < 0 || (c.columns && !c.pages);
    return reached();
}
}  // namespace qlin
