// Arithmetic of the search for a row's threshold (sample.hip): the bins of
// hist_kernel and gather_kernel, and the narrowing in small_kernel, where among
// equal parts of [low, first] a row's token falls and what it weighs.
// constexpr, so that the same functions run in the kernels and in the host's
// tests.
#pragma once

namespace moe {

// Bin of a token's distance from the first, in float32: all that is asked of
// it is that it never falls while the value does.  The last bin holds all that
// lies beyond: masks of the lowest value are an infinite distance away.
constexpr int kBins = 2048;
constexpr int bin_of(float x, float first, float scale) {
    const float d = (first - x) * scale;
    return (int)(d < (float)(kBins - 1) ? d : (float)(kBins - 1));
}

constexpr int kParts = 2048;

// Whether [low, first] is cut into parts.  A spread below 1e-30 has no finite
// number of parts to a unit, and values of -1e30 and below are masks.
constexpr bool can_narrow(float low, float first) { return low > -1e30f && first - low >= 1e-30f; }

// Parts to a unit; the value `low` itself falls into the last part.
constexpr float parts_per_unit(float low, float first) { return (kParts - 0.1f) / (first - low); }

// The part of x in [low, first], from the first down; the last one for
// whatever lies outside or is no number.
constexpr int part_at(float first, float x, float per) {
    const float d = (first - x) * per;
    return (int)(d < (float)(kParts - 1) ? d : (float)(kParts - 1));
}

// Weights of a top-p narrowing, float32 numbers relative to the first, are
// added as integers in units of 1 / kNarrowMass of the row's sum: a tail's
// tokens hold units however far below the first they lie, and whole rows stay
// below 2^31.
constexpr double kNarrowMass = 2.13e9;
constexpr unsigned narrow_mass(float unit, float w) { return (unsigned)(unit * w + 0.5f); }

// What a sum of n of them may be off by.  Half a unit each; and of the sum
// 3 * 2^-24 * 40 * ln 2 = 5.0e-6 for the exponents (three roundings, at most 40
// bits: the least token counted weighs (1 - top_p) / 2V, 2^-40, of the sum),
// 1.2e-7 for exp2 and 2.4e-7 for the products and the comparison's
// conversions, 11500 units in all.
constexpr float narrow_slack(int n) { return 14000.f + 0.5f * (float)n; }

}  // namespace moe
