// Internal declarations of the serving operators around the verify layer:
// the 4-bit K/V cache (kv4.hip) and the drawing and acceptance of draft
// tokens (sample.hip).  Host side in serve.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

#include "internal.h"

namespace moe {

// Allows a kernel `lds` bytes of dynamic LDS, once per device.  (Doing it
// twice is harmless, so two threads need no order.)
template <auto Kernel>
hipError_t allow_lds(int lds) {
    static std::atomic<uint64_t> done{0};  // a bit a device
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev) & 1) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel), hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e == hipSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_relaxed);
    return e;
}

// The cache and the rows of one call, by value in the kernel arguments.
struct KvRows {
    uint8_t *data;
    const int32_t *table, *len;
    int num_pages, page_shift, Hkv, D, max_pages, nseq;
    int off[kMaxSegments + 1];
};

struct KvAppendArgs {
    KvRows r;
    const void *k, *v;
    int64_t ks, vs;  // elements between tokens
    const int32_t *path, *count;
    void *k_out, *v_out;
    int T, f32;
};
hipError_t launch_kv4_append(const KvAppendArgs &a, hipStream_t s);

struct KvAttendArgs {
    KvRows r;
    const void *q;
    int64_t qs;  // elements between tokens
    void *out;
    float *part;  // partial results of split units
    float scale;
    int T, Hq, G, f32;
    int mt, nwg;                 // 16-row tiles of a row block, workgroups
    uint64_t anc[kMaxTokens];    // rows of its own sequence that each call row sees
};
// Fills mt and nwg from the shape; returns the workspace bytes.
size_t kv4_attend_plan(KvAttendArgs &a, int n_cu);
hipError_t launch_kv4_attend(const KvAttendArgs &a, hipStream_t s);

struct SampleArgs {
    const void *logits;
    int64_t stride;
    int T, V, f32;
    const float *temperature, *top_p, *min_p;
    const int32_t *top_k;
    void *ws;
};
size_t sample_ws_bytes(int T, int V);
hipError_t launch_sample(const SampleArgs &a, const float *u, int32_t *token, float *prob, float *probs,
                         hipStream_t s);

struct AcceptArgs {
    const int32_t *tokens;
    const float *q, *u, *u_final;
    int32_t *out, *path, *count;
    int nseq;
    int off[kMaxSegments + 1];
    int8_t parent[kMaxTokens];  // row of the call, -1 for roots
};
hipError_t launch_accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t s);

}  // namespace moe
