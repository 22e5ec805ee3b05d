// Host checks of csrc/narrow.h under UndefinedBehaviorSanitizer (conversions
// out of an int's range included).  Exit status 0 = pass.
#include <cmath>
#include <cstdio>
#include <limits>
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

int main() {
    parts();
    if (failures) return 1;
    std::puts("all checks passed");
    return 0;
}
