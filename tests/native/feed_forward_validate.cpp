// feed_forward_validate.cpp -- runs the argument checks of the feed-forward
// operators (validate.hpp) on a seeded sample of boundary values, built with
// the host sanitizers: any signed overflow or other undefined behaviour in
// the checks aborts the run.  Test infrastructure only.
#include <stdint.h>
#include <stdio.h>

#include "../../fp8_fine_grained_x128_amd/csrc/validate.hpp"

using namespace fp8q::check;

static uint64_t state = 7;
static uint64_t rnd() {
    uint64_t z = (state += 0x9e3779b97f4a7c15ULL);
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ULL;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebULL;
    return z ^ (z >> 31);
}
static int64_t n() {
    static const int64_t v[] = {-1, 0, 1, 2, 4, 16, 64, 65, 128, 129, 256, 1024, 7168, 16384, 16385, (1LL << 24) - 1, 1LL << 24,
                                1LL << 32, (1LL << 32) + 16, 1LL << 50, 1LL << 62, INT64_MAX, INT64_MIN, -128};
    return v[rnd() % (sizeof(v) / sizeof(v[0]))];
}
static int64_t usual() { return rnd() % 3 ? 256 : n(); }  // so that some calls come through
static int i() { static const int v[] = {-1, 0, 1, 2, 1024, 1025, 0x7fffffff}; return rnd() % 2 ? (int)(rnd() % 2) : v[rnd() % 7]; }
static const void* p() {
    static const uintptr_t v[] = {0, 1u << 20, (1u << 20) + 2, (1u << 20) + 8};
    return reinterpret_cast<const void*>(rnd() % 4 ? uintptr_t(1u << 20) : v[rnd() % 4]);
}
static float e() { static const float v[] = {0.0f, 1e-5f, -1.0f, 1.0f / 0.0f}; return v[rnd() % 4]; }

int main() {
    long long launched = 0;
    for (int k = 0; k < 2000000; ++k) {
        int r = 0;
        switch (k % 6) {
            case 0: r = layernorm(p(), i(), usual(), usual(), usual(), p(), p(), i(), e(), i(), p(), i(), usual(), p(), usual(),
                                  p(), usual(), i(), p(), p()); break;
            case 1: r = layernorm_backward(p(), usual(), p(), usual(), i(), usual(), usual(), p(), i(), p(), p(), i(), p(),
                                           usual(), p(), usual(), p(), p(), i(), n(), p(), n()); break;
            case 2: r = swiglu_quantize(p(), p(), i(), usual(), usual(), usual(), p(), usual(), p(), usual(), p(), p(), usual(),
                                        p(), p(), usual(), i()); break;
            case 3: r = swiglu_backward(p(), p(), usual(), p(), p(), usual(), p(), i(), usual(), usual(), usual(), p(), p(),
                                        usual()); break;
            case 4: r = swiglu_backward_quantize(p(), p(), usual(), p(), p(), usual(), p(), i(), usual(), usual(), usual(), p(),
                                                 p(), usual(), p(), p(), usual(), p(), p(), usual(), p(), p(), usual(), p(),
                                                 usual(), p(), usual(), i()); break;
            default: r = moe_decode(p(), usual(), rnd() % 2 ? 4 : n(), usual(), p(), usual(), i(), i(), usual(), p(), usual(),
                                    rnd() % 2 ? 1 << 20 : n(), p(), usual(), rnd() % 2 ? 1 << 20 : n(), p(), usual(),
                                    rnd() % 2 ? 1 << 20 : n(), p(), usual(), rnd() % 2 ? 1 << 20 : n(), p(), i(), usual(), n(),
                                    p(), n()); break;
        }
        if (r == kLaunch) ++launched;
        if (r < kLaunch || r > FP8Q_EHIP) { printf("status %d out of range\n", r); return 1; }
    }
    printf("%lld of 2000000 sampled calls valid\n", launched);
    return launched > 1000 ? 0 : 1;
}
