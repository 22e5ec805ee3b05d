// Host checks of csrc/narrow.h under UndefinedBehaviorSanitizer (conversions
// out of an int's range included).  Exit status 0 = pass.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <limits>
#include <random>
#include <vector>

#include "narrow.h"

static int failures = 0;

#define CHECK(cond, ...)                                              \
    do {                                                              \
        if (!(cond)) {                                                \
            std::fprintf(stderr, "FAIL line %d: %s: ", __LINE__, #cond); \
            std::fprintf(stderr, __VA_ARGS__);                        \
            std::fprintf(stderr, "\n");                               \
            ++failures;                                               \
        }                                                             \
    } while (0)

// Rows between low and first, from equal values over subnormal spreads to the
// whole range: every part lies in the histogram, and parts do not fall with
// the value.
static void parts() {
    const float big = std::numeric_limits<float>::max();
    std::vector<float> firsts = {0.f, 1.f, -1.f, 90.f, 1e-37f, -1e-37f, 1e-44f, 1000.f, 1e20f, -1e20f, big, -9e29f};
    int cut = 0;
    for (float first : firsts)
        for (int e = -149; e <= 128; ++e)
            for (float m : {1.f, 1.37f, 1.99f}) {
                const float low = first - (float)std::fmin(std::ldexp((double)m, e), 3.4e38);
                if (!std::isfinite(low) || !(low <= first) || !moe::can_narrow(low, first)) continue;
                const float per = moe::parts_per_unit(low, first);
                CHECK(std::isfinite(per) && per > 0.f, "first %g low %g", first, low);
                ++cut;
                int last = -1;
                for (int i = 0; i <= 64; ++i) {
                    float x = i == 64 ? low : i == 0 ? first : (float)(first + ((double)low - first) * i / 64);
                    if (i == 1) x = std::nextafter(first, low);
                    const int part = moe::part_at(first, x, per);
                    CHECK(part >= 0 && part < moe::kParts, "first %g low %g x %g part %d", first, low, x, part);
                    if (i != 1) {
                        CHECK(part >= last, "first %g low %g x %g part %d after %d", first, low, x, part, last);
                        last = part;
                    }
                }
                CHECK(moe::part_at(first, first, per) == 0, "first %g low %g", first, low);
            }
    CHECK(cut > 1000, "%d", cut);
    // outside of the range, and no number
    const float inf = std::numeric_limits<float>::infinity();
    for (float x : {-inf, -big, std::nanf("")}) {
        const int part = moe::part_at(1.f, x, moe::parts_per_unit(0.f, 1.f));
        CHECK(part >= 0 && part < moe::kParts, "x %g part %d", x, part);
    }
}

// Bins of every distance and temperature, masks of the lowest value among them.
static void bins() {
    const float big = std::numeric_limits<float>::max();
    for (float first : {big, 1e30f, 90.f, 1.f, 0.f, -7.f, -1e38f})
        for (float scale : {1e30f, 6.4e7f, 64.f, 0.9f, 1e-30f, 0.f}) {
            int last = 0;
            std::vector<float> xs = {first, first - 1e-6f * std::fabs(first), first - 0.01f, first - 1.f, first - 31.9f, first - 33.f,
                                     first - 1e9f, first - 1e30f, -3.3895313892515355e38f, -big};
            std::sort(xs.begin(), xs.end(), [](float a, float b) { return a > b; });
            for (float x : xs) {
                if (!(x <= first)) continue;
                const int bin = moe::bin_of(x, first, scale);
                CHECK(bin >= last && bin < moe::kBins, "first %g x %g scale %g bin %d after %d", first, x, scale, bin, last);
                last = bin;
            }
        }
}

// Running sums of a row's weights, largest first, in units of the narrowing:
// off by less than the slack from the exact ones, for tails that hold most of
// the row, rows of one value and thresholds next to 1.
static void sums() {
    std::mt19937_64 rng(1);
    std::normal_distribution<float> normal;
    double worst = 0;
    for (int n : {2049, 4096, 20000, 32768})
        for (float spread : {0.f, 1e-3f, 1.f, 4.f, 12.f})
            for (float first : {0.f, 20.f, -3000.f})
                for (double invt : {1.0, 1 / 0.7, 0.1, 3.0}) {
                    std::vector<float> x(n);
                    for (float &v : x) v = first - std::fmin(std::fabs(normal(rng)) * spread, (float)(27.0 / invt));
                    x[0] = first;
                    std::sort(x.begin(), x.end(), [](float a, float b) { return a > b; });
                    double all = 0;
                    for (float v : x) all += std::exp(((double)v - first) * invt);
                    const float unit = (float)(moe::kNarrowMass / all), scale = (float)(invt * 1.4426950408889634);
                    unsigned long long got = 0;
                    double run = 0;
                    for (float v : x) {
                        got += moe::narrow_mass(unit, std::exp2((v - first) * scale));
                        run += std::exp(((double)v - first) * invt);
                        worst = std::fmax(worst, std::fabs((double)got - run / all * moe::kNarrowMass) / moe::narrow_slack(n));
                    }
                    CHECK(got < 1ull << 31, "%llu", got);
                }
    CHECK(worst < 1, "%g of the slack", worst);
    std::printf("sums: %g of the slack\n", worst);
}

int main() {
    parts();
    bins();
    sums();
    if (failures) return 1;
    std::puts("all checks passed");
    return 0;
}
