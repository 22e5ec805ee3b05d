// The experts of prompts: the choice of each token's experts from its router
// logits, and the experts' products over any number of tokens.
#include "common.h"
#include "prompt.h"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Route.  One wave a token, E / 64 logits a lane as integers whose order is the
// floats'; k rounds of a wave maximum, each taking the lowest index that holds
// it, so that lane r ends with rank r.
// ---------------------------------------------------------------------------
constexpr int kRouteThreads = 256;

// Monotone image of a float: NaN as -inf, +inf as the largest, both zeros the
// same.  0 is below every image and stands for a logit that is taken or not there.
__device__ __forceinline__ unsigned image(float v) {
    v = v == v ? fminf(v, 3.402823466e38f) + 0.f : -__builtin_inff();
    const unsigned u = __float_as_uint(v);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ float from_image(unsigned u) {
    return __uint_as_float((u >> 31) ? u & 0x7fffffffu : ~u);
}

__device__ __forceinline__ unsigned wave_max_u(unsigned v) {
    v = max(v, (unsigned)dpp_ror<8>((int)v));
    v = max(v, (unsigned)dpp_ror<4>((int)v));
    v = max(v, (unsigned)dpp_ror<2>((int)v));
    v = max(v, (unsigned)dpp_ror<1>((int)v));
    return max(max((unsigned)__builtin_amdgcn_readlane((int)v, 0), (unsigned)__builtin_amdgcn_readlane((int)v, 16)),
               max((unsigned)__builtin_amdgcn_readlane((int)v, 32), (unsigned)__builtin_amdgcn_readlane((int)v, 48)));
}

template <int N>
__global__ __launch_bounds__(kRouteThreads) void route_tokens_kernel(const float *logits, int64_t stride, int T, int E, int k,
                                                                     int32_t *idx, float *w) {
    const int lane = threadIdx.x & 63;
    const int t = blockIdx.x * (kRouteThreads / 64) + (threadIdx.x >> 6);
    if (t >= T) return;
    const float *row = logits + (size_t)t * stride;
    unsigned v[N];
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = j * 64 + lane < E ? image(row[j * 64 + lane]) : 0u;
    unsigned first = 0, val = 0;
    int mine = 0;
    for (int r = 0; r < k; ++r) {
        unsigned m = v[0];
#pragma unroll
        for (int j = 1; j < N; ++j) m = max(m, v[j]);
        m = wave_max_u(m);
        if (r == 0) first = m;
        bool done = false;  // the same in every lane
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const uint64_t at = __ballot(v[j] == m);
            if (!done && at) {
                const int l = __ffsll((unsigned long long)at) - 1;
                if (lane == r) mine = j * 64 + l, val = m;
                if (lane == l) v[j] = 0;
                done = true;
            }
        }
    }
    // softmax over the chosen: nothing where even the first is -inf
    const float top = from_image(first);
    const float e = lane < k && top > -__builtin_inff() ? expf(from_image(val) - top) : 0.f;
    const float z = wave_sum(e);
    if (lane < k) {
        idx[(size_t)t * k + lane] = mine;
        w[(size_t)t * k + lane] = z > 0.f ? e / z : 0.f;
    }
}

}  // namespace

hipError_t launch_route_tokens(const float *logits, int64_t stride, int T, int E, int k, int32_t *idx, float *w,
                               hipStream_t s) {
    const int n = (E + 63) / 64;
    auto kern = n == 1 ? route_tokens_kernel<1> : n == 2 ? route_tokens_kernel<2> : n <= 4 ? route_tokens_kernel<4> : route_tokens_kernel<8>;
    hipLaunchKernelGGL(kern, dim3((T + kRouteThreads / 64 - 1) / (kRouteThreads / 64)), dim3(kRouteThreads), 0, s, logits, stride,
                       T, E, k, idx, w);
    return hipGetLastError();
}

}  // namespace moe
