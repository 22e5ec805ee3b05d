// Internal declarations of the operators for prompts: the prompts' attention
// (prompt.hip), the experts' products over many tokens (experts.hip) and the
// cache's rows and pages (pages.hip).  Host side in prompt.cpp.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "serve.h"

namespace moe {

struct KvReadArgs {
    KvRows r;
    void *k, *v;
    int T, f32;
};
hipError_t launch_kv4_read(const KvReadArgs &a, hipStream_t s);

// Page tables and reference counts; a list of n <= kMaxSegments sequences.
struct PoolArgs {
    int32_t *refs, *table;
    int num_pages, page_shift, nseq, max_pages, n;
    const int32_t *src, *dst, *rows;
    int32_t *pairs, *ok;
};
hipError_t launch_reserve(const PoolArgs &a, hipStream_t s);
hipError_t launch_fork(const PoolArgs &a, hipStream_t s);
hipError_t launch_release(const PoolArgs &a, hipStream_t s);

struct CompactArgs {
    int32_t *refs, *table;
    int num_pages, nseq, max_pages, max_moves;
    int32_t *pairs;
    // set by the launch
    int most, chunks;
    int32_t *chunk, *low, *high, *rank;
};
size_t compact_ws_bytes(int num_pages, int max_moves);
hipError_t launch_compact(CompactArgs a, int32_t *ws, hipStream_t s);

struct CopyArgs {
    uint8_t *data;
    size_t page_bytes;
    const int32_t *pairs;
    int num_pages, n;
    int pieces;  // set by the launch
};
hipError_t launch_copy_pages(CopyArgs a, hipStream_t s);

// Attention of prompts.  Offsets by value; row j of a sequence's n sees its
// first j + 1 + (m - n) keys.
struct PromptArgs {
    const void *q, *k, *v;
    int64_t qs, ks, vs;  // elements between tokens
    void *out;
    void *ws;
    float scale;
    int nseq, Hq, Hkv, G, D, f32;
    int q_off[kMaxSegments + 1], k_off[kMaxSegments + 1];
    // plan
    int parts;              // shares of a unit's keys
    int units;              // row blocks of all sequences and heads
    int blocks[kMaxSegments + 1];  // row blocks before each sequence
    size_t part_at;  // of the shares in the workspace
};
// Fills the plan; returns the workspace bytes.
size_t prompt_plan(PromptArgs &a, int n_cu);
hipError_t launch_prompt(const PromptArgs &a, hipStream_t s);

hipError_t launch_route_tokens(const float *logits, int64_t stride, int T, int E, int k, int32_t *idx, float *w,
                               hipStream_t s);

// The experts' products over T tokens.  Rows of the products are the (token,
// rank) pairs grouped by expert, then every token once for the shared expert.
struct ExpertArgs {
    int T, H, I, E, k, fp8, f32, shared;
    const void *x;
    int64_t xs;  // elements between tokens
    const int32_t *idx;
    const float *w;
    void *y;
    const void *W_gu, *W_d, *Wsh_gu, *Wsh_d;
    const float *s_gu, *s_d, *ssh_gu, *ssh_d;
    void *ws;
};
bool experts_fit(const ExpertArgs &a);  // whether the grids of a call are below HIP's limit
size_t experts_ws_bytes(const ExpertArgs &a);
hipError_t launch_experts(const ExpertArgs &a, hipStream_t s);

}  // namespace moe
