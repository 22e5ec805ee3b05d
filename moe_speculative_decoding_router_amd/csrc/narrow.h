// Arithmetic of the narrowing in small_kernel (sample.hip): where among equal
// parts of [low, first] a row's token falls.  constexpr, so that the same
// functions run in the kernels and in the host's tests.
#pragma once

namespace moe {

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
    return d < (float)(kParts - 1) ? (int)d : kParts - 1;
}

}  // namespace moe
