// The corrected division by 127 and 448 (scale_of in layer_device.h) on the CPU, over every f32 mantissa: the correctly
// rounded a / Q.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <initializer_list>

static float of(uint32_t b) { float f; std::memcpy(&f, &b, 4); return f; }
static uint32_t bits(float f) { uint32_t b; std::memcpy(&b, &f, 4); return b; }

int main() {
    long bad = 0;
    for (uint32_t m = 0; m < (1u << 23); ++m) {
        const float a = of(0x3F800000u | m);
        for (float q : {127.0f, 448.0f}) {
            const float inv = 1.0f / q, x = a * inv;
            bad += bits(std::fmaf(std::fmaf(-q, x, a), inv, x)) != bits(a / q);
        }
    }
    std::printf("%ld differ\n", bad);
    return bad != 0;
}
