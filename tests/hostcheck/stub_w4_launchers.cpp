// Host-only stand-ins for the launchers of the 4-bit products, the router and
// the experts, linked with their C-ABI layer (w4_api.hip) into a sanitizer
// build that runs on a CPU: every launcher records what it was asked for and
// returns success without touching memory.  Test infrastructure: never part of
// libqlin.so.
#include "../../quantized_linear_layers_token_amd/csrc/qlin_internal.h"
#include "../../quantized_linear_layers_token_amd/csrc/w4_internal.h"

namespace {
int g_launches = 0;
int g_form = -1, g_pair_form = -1;
long long g_items = 0;
bool g_bad = false;   // a form that its launch does not fit
hipError_t reached() {
    ++g_launches;
    return hipSuccess;
}
hipError_t product(int form, const qlin::W4Call& c, bool pair, bool experts) {
    (pair ? g_pair_form : g_form) = form;
    g_items = c.max_items;
    const bool tiled = form >= qlin::kW4Tiled64x8;
    const int64_t groups = qlin::w4_blocks(form, c, experts) * qlin::w4_units(form, c, pair);
    g_bad |= groups <= 0 || groups * qlin::kW4FormThreads[form] >= (int64_t(1) << 32);
    g_bad |= experts && tiled && !c.items;            // the tiled kernel goes by items
    g_bad |= pair && form == qlin::kW4Stream16x1;
    // items found by the workgroups: streamed gate and up only, within the sizes that fit, with room to write them down
    g_bad |= c.slots > 0 && (!experts || !pair || tiled || !c.items || !c.order || !c.nitems ||
                             c.slots > qlin::kOwnItemSlots || c.E > qlin::kOwnItemExperts);
    return reached();
}
}  // namespace

extern "C" int w4_launches(void) { return g_launches; }
extern "C" int w4_form(void) { return g_form; }
extern "C" int w4_pair_form(void) { return g_pair_form; }
extern "C" long long w4_items(void) { return g_items; }
extern "C" int w4_bad(void) { return g_bad; }

namespace qlin {
qlin_status hip_status(hipError_t e) { return e == hipSuccess ? QLIN_OK : QLIN_ERR_HIP; }
hipError_t launch_pack_w4(const uint8_t*, const uint16_t*, const uint8_t*, int64_t, int64_t, int64_t, int, uint8_t*,
                          uint16_t*, uint8_t*, hipStream_t) {
    return reached();
}
hipError_t launch_w4_stream(int form, const W4Call& c, bool pair, bool experts, hipStream_t) {
    g_bad |= form >= kW4Tiled64x8;
    return product(form, c, pair, experts);
}
hipError_t launch_w4_tiled(int form, const W4Call& c, bool pair, bool experts, hipStream_t) {
    g_bad |= form < kW4Tiled64x8;
    return product(form, c, pair, experts);
}
hipError_t launch_route(const void*, bool, int64_t, int, int, int, const float*, int, int, int, bool, float, int32_t*,
                        float*, hipStream_t) {
    return reached();
}
hipError_t launch_experts_plan(const int32_t*, int64_t, int, int, int*, int*, int*, hipStream_t) { return reached(); }
hipError_t launch_experts_combine(const float*, const int32_t*, const float*, int64_t, int, int, int64_t, uint16_t*,
                                  hipStream_t) {
    return reached();
}
hipError_t launch_experts_down_direct(const W4Call&, const float*, int64_t, int, uint16_t*, hipStream_t) {
    return reached();
}
}  // namespace qlin
