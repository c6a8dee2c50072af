// experts_validate.cpp -- runs the argument checks of the experts' weight
// gradients, their operands and the AdamW step (validate.hpp) on a seeded
// sample of boundary values, built with the host sanitizers: any signed
// overflow or other undefined behaviour in the checks aborts the run.  Test
// infrastructure only.
#include <stdint.h>
#include <stdio.h>

#include "../../fp8_fine_grained_x128_amd/csrc/validate.hpp"

using namespace fp8q::check;

static uint64_t state = 11;
static uint64_t rnd() {
    uint64_t z = (state += 0x9e3779b97f4a7c15ULL);
    z = (z ^ (z >> 30)) * 0xbf58476d1ce4e5b9ULL;
    z = (z ^ (z >> 27)) * 0x94d049bb133111ebULL;
    return z ^ (z >> 31);
}
static int64_t n() {
    static const int64_t v[] = {-1, 0, 1, 2, 16, 127, 128, 129, 256, 1024, 7168, 128 * 65535, (1LL << 24) - 1, 1LL << 24, 1LL << 30,
                                (1LL << 31) - 1, 1LL << 31, 1LL << 32, 1LL << 33, 1LL << 50, 1LL << 62, INT64_MAX, INT64_MIN};
    return v[rnd() % (sizeof(v) / sizeof(v[0]))];
}
static int64_t usual() { return rnd() % 4 ? 256 : n(); }  // so that some calls come through
static int64_t wide() { return rnd() % 4 ? 1 << 20 : n(); }
static int i() { static const int v[] = {-1, 0, 1, 2, 8, 32, 1024, 1025, 0x7fffffff, -0x7fffffff - 1}; return rnd() % 2 ? (int)(rnd() % 2) : v[rnd() % 10]; }
static int groups_() { return rnd() % 3 ? 4 : i(); }
static uintptr_t a() {
    static const uintptr_t v[] = {0, 1u << 20, (1u << 20) + 2, (1u << 20) + 8};
    return rnd() % 8 ? uintptr_t(1u << 20) : v[rnd() % 4];
}
static const void* p() { return reinterpret_cast<const void*>(a()); }
static double d() { static const double v[] = {0.0, 0.9, 1.0, -1.0, 1e-8, 1.0 / 0.0, 0.0 / 0.0}; return rnd() % 4 ? 0.5 : v[rnd() % 7]; }

int main() {
    long long launched[4] = {0, 0, 0, 0};
    for (int k = 0; k < 2000000; ++k) {
        int r = 0;
        const int which = k % 4;
        if (which == 0) {
            r = grouped_quantize_act(p(), i(), usual(), usual(), usual(), p(), groups_(), p(), wide(), p(), usual(), i());
        } else if (which == 1) {
            r = grouped_requant(p(), usual(), usual(), usual(), p(), usual(), p(), groups_(), p(), wide(), p(), usual(), i());
        } else if (which == 2) {
            const int64_t rows = usual(), N = usual(), K = usual();
            const int G = groups_();
            r = wgrad_sizes(rows, G, N, K);
            if (r == kLaunch)
                r = grouped_wgrad(p(), wide(), p(), usual(), p(), wide(), p(), usual(), p(), G, rows, N, K, p(), i(), usual(),
                                  wide(), i(), (unsigned)i(), rnd() % 2 ? 0 : 4096, p(), n());
        } else {
            fp8q_adamw_tensor t[2];
            for (auto& x : t) {
                const bool coded = rnd() % 2;
                x = fp8q_adamw_tensor{};
                x.n = rnd() % 3 ? 1 << 16 : n();
                x.p = (float*)a(), x.g = p(), x.m = (void*)a(), x.v = (void*)a(), x.sm = (float*)a(), x.sv = (float*)a();
                if (coded) x.N = usual(), x.K = usual(), x.q = (uint8_t*)a(), x.s = (float*)a();
                if (coded && rnd() % 2) x.qt = (uint8_t*)a(), x.st = (float*)a();
            }
            fp8q_adamw_config c{d(), d(), d(), d(), d(), usual(), nullptr, nullptr, nullptr, 0};
            if (rnd() % 4 == 0) c.lr_dev = (const float*)a(), c.step_dev = (const int64_t*)a(), c.grad_scale = (const float*)a();
            r = adamw(t, rnd() % 8 ? 2 : -(int)(rnd() % 2), i(), rnd() % 2 ? 8 : 32, &c, i());
        }
        if (r == kLaunch) ++launched[which];
        if (r < kLaunch || r > FP8Q_EHIP) { printf("status %d out of range\n", r); return 1; }
    }
    printf("%lld, %lld, %lld and %lld of 500000 sampled calls each valid\n", launched[0], launched[1], launched[2], launched[3]);
    for (long long l : launched)
        if (l < 1000) return 1;
    return 0;
}
