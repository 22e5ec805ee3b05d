// The 4-bit K/V cache's tile and its codes, for the kernels that read or write
// them.  Layout in include/moe_verify.h.
#pragma once

#include "common.h"

namespace moe {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Bytes of a row's 17 D / 16 share: a tile holds 16 rows of K, its scales, V and its scales.
template <int D>
struct Tile {
    static constexpr int kK = 0, kKs = 8 * D, kV = 17 * D / 2, kVs = 33 * D / 2, kBytes = 17 * D;
};

// 2^(e - 127) of a scale byte.
__device__ __forceinline__ float scale_of(unsigned e) { return __uint_as_float(e << 23); }

// Eight codes as bf16 and as float32, exactly (2 significant bits and a power of two).
__device__ __forceinline__ bf16x8 dequant8(unsigned w, float s) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } o;
    o.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    o.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    o.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    o.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return o.v;
}

__device__ __forceinline__ void dequant8_f32(unsigned w, float s, f32x4 &lo, f32x4 &hi) {
    const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0), y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const f32x2 y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2), y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    lo = f32x4{y0[0], y0[1], y1[0], y1[1]};
    hi = f32x4{y2[0], y2[1], y3[0], y3[1]};
}

}  // namespace moe
