// Host-side checks of the operators for prompts (csrc/prompt.cpp) under
// AddressSanitizer and UndefinedBehaviorSanitizer (g++), with recorders in
// place of the kernel launchers.  The arrays that the ABI marks (host) are heap
// blocks of exactly the documented size; device pointers are addresses that nothing
// dereferences.  Exit status 0 = pass.
#include <algorithm>
#include <cstdio>
#include <limits>
#include <memory>
#include <string>
#include <vector>

#include "moe_verify.h"
#include "prompt.h"

static int failures = 0, launches = 0;
static std::string error;
static moe::PromptArgs prompt_args;
static moe::ExpertArgs expert_args;
static moe::KvReadArgs read_args;
static moe::PoolArgs pool_args;
static moe::CompactArgs compact_args;
static moe::CopyArgs copy_args;

namespace moe {
int set_error(int code, const char *msg) {
    error = msg;
    return code;
}
int device_cu_count() { return 256; }
int verify_needs(const ::moe_layer *layer, int T, const ::moe_bias *, size_t *need) {
    *need = 1;
    return layer && T == 1 ? MOE_OK : MOE_EINVAL;
}
hipError_t launch_kv4_read(const KvReadArgs &a, hipStream_t) { return ++launches, read_args = a, hipSuccess; }
hipError_t launch_reserve(const PoolArgs &a, hipStream_t) { return ++launches, pool_args = a, hipSuccess; }
hipError_t launch_fork(const PoolArgs &a, hipStream_t) { return ++launches, pool_args = a, hipSuccess; }
hipError_t launch_release(const PoolArgs &a, hipStream_t) { return ++launches, pool_args = a, hipSuccess; }
size_t compact_ws_bytes(int num_pages, int max_moves) { return (size_t)num_pages * 4 + max_moves; }
hipError_t launch_compact(CompactArgs a, int32_t *, hipStream_t) { return ++launches, compact_args = a, hipSuccess; }
hipError_t launch_copy_pages(CopyArgs a, hipStream_t) { return ++launches, copy_args = a, hipSuccess; }
size_t prompt_plan(PromptArgs &a, int) { return a.units = 7, (size_t)1024; }
hipError_t launch_prompt(const PromptArgs &a, hipStream_t) { return ++launches, prompt_args = a, hipSuccess; }
hipError_t launch_route_tokens(const float *, int64_t, int, int, int, int32_t *, float *, hipStream_t) { return ++launches, hipSuccess; }
bool experts_fit(const ExpertArgs &a) { return a.T < 1 << 20; }
size_t experts_ws_bytes(const ExpertArgs &a) { return 4096 + (size_t)a.T; }
hipError_t launch_experts(const ExpertArgs &a, hipStream_t) { return ++launches, expert_args = a, hipSuccess; }
}  // namespace moe

#define CHECK(cond)                                                                                       \
    do {                                                                                                  \
        if (!(cond)) {                                                                                    \
            std::fprintf(stderr, "FAIL %s:%d: %s (%s)\n", __FILE__, __LINE__, #cond, error.c_str());      \
            ++failures;                                                                                   \
        }                                                                                                 \
    } while (0)

static std::unique_ptr<int32_t[]> block(const std::vector<int32_t> &v) {
    std::unique_ptr<int32_t[]> b(new int32_t[v.size()]);
    std::copy(v.begin(), v.end(), b.get());
    return b;
}

int main() {
    void *const P = reinterpret_cast<void *>(4096);
    int32_t *const I = static_cast<int32_t *>(P);
    float *const F = static_cast<float *>(P);
    const int64_t low = std::numeric_limits<int64_t>::min();
    const int big = std::numeric_limits<int32_t>::max();

    // ---- attention of prompts ----
    std::vector<int32_t> many(65);
    for (int i = 0; i <= 64; ++i) many[i] = 3 * i;
    const auto q64 = block(many), q2 = block({0, 4, 9}), k2 = block({0, 0, 1 << 22}), bad = block({0, 5, 4}), none = block({0, 0});
    CHECK(prompt_attend_workspace_bytes(2, q2.get(), k2.get(), 8, 2, 128, MOE_BF16) == 1024);
    CHECK(prompt_attend(P, P, P, 1024, 256, 1 << 24, 2, q2.get(), k2.get(), 8, 2, 128, MOE_BF16, 0.5f, P, P, 1024, nullptr) == MOE_OK);
    CHECK(launches == 1 && prompt_args.q_off[2] == 9 && prompt_args.k_off[2] == 1 << 22 && prompt_args.G == 4 && prompt_args.vs == 1 << 24);
    CHECK(prompt_attend(P, P, P, 1024, 256, 256, 64, q64.get(), q64.get(), 8, 2, 128, MOE_F32, 0.5f, P, P, 1024, nullptr) == MOE_OK);
    CHECK(launches == 2 && prompt_args.q_off[64] == 192 && prompt_args.f32);
    CHECK(prompt_attend(P, P, P, 1024, 256, 256, 65, q64.get(), q64.get(), 8, 2, 128, MOE_F32, 0.5f, P, P, 1024, nullptr) == MOE_EINVAL);
    CHECK(prompt_attend(P, P, P, 1024, 256, 256, 2, q2.get(), bad.get(), 8, 2, 128, MOE_F32, 0.5f, P, P, 1024, nullptr) == MOE_EINVAL);
    CHECK(prompt_attend(P, P, P, low, 256, 256, 2, q2.get(), q2.get(), 8, 2, 128, MOE_F32, 0.5f, P, P, 1024, nullptr) == MOE_EINVAL);
    CHECK(prompt_attend(P, P, P, 1024, 256, 256, 2, q2.get(), q2.get(), 8, 2, 128, MOE_F32, 0.5f, P, P, 1023, nullptr) == MOE_EWORKSPACE);
    CHECK(prompt_attend(P, P, P, 1024, 256, 256, 2, q2.get(), q2.get(), big, 1, 128, MOE_F32, 0.5f, P, P, 1024, nullptr) == MOE_EINVAL);
    CHECK(prompt_attend(nullptr, nullptr, nullptr, 1024, 256, 256, 1, none.get(), none.get(), 8, 2, 128, MOE_F32, 0.5f, nullptr, nullptr, 0,
                        nullptr) == MOE_OK);
    CHECK(launches == 2);

    // ---- experts ----
    moe_layer L{};
    L.H = 256, L.I = 128, L.E = 8, L.k = 2, L.wdtype = MOE_BF16, L.W_gu = P, L.W_d = P, L.Wr = F;
    CHECK(moe_experts_workspace_bytes(&L, 100, MOE_F32) == 4196);
    CHECK(moe_experts(&L, P, 256, 100, MOE_F32, I, F, P, P, 4196, nullptr) == MOE_OK && launches == 3 && expert_args.f32 && !expert_args.shared);
    CHECK(moe_experts(&L, P, 256, 100, MOE_F32, I, F, P, P, 4195, nullptr) == MOE_EWORKSPACE);
    CHECK(moe_experts(&L, P, low, 100, MOE_F32, I, F, P, P, 4196, nullptr) == MOE_EINVAL);
    CHECK(moe_experts(&L, P, 256, big, MOE_F32, I, F, P, P, 4196, nullptr) == MOE_EINVAL);
    CHECK(moe_experts(&L, P, 256, 1 << 20, MOE_F32, I, F, P, P, 1u << 30, nullptr) == MOE_ENOTSUP);
    CHECK(moe_experts(nullptr, P, 256, 100, MOE_F32, I, F, P, P, 4196, nullptr) == MOE_EINVAL);
    CHECK(route_tokens(F, 300, 1 << 24, 300, 32, I, F, nullptr) == MOE_OK && launches == 4);
    CHECK(route_tokens(F, low, 4, 300, 32, I, F, nullptr) == MOE_EINVAL && launches == 4);

    // ---- rows and pages ----
    moe_kv4_cache c{P, 100, 64, 2, 128};
    moe_kv4_rows r2{I, 10, I, 2, q2.get()};
    CHECK(kv4_read(&c, &r2, P, P, 9, MOE_F32, nullptr) == MOE_OK && launches == 5 && read_args.r.off[2] == 9 && read_args.r.page_shift == 6);
    CHECK(kv4_read(&c, &r2, P, P, 8, MOE_F32, nullptr) == MOE_EINVAL && kv4_read(nullptr, &r2, P, P, 9, MOE_F32, nullptr) == MOE_EINVAL);
    moe_kv4_pool p{I, I, 1 << 24, 4096, 1, 523263};
    CHECK(kv4_reserve(&p, I, I, 64, I, nullptr) == MOE_OK && pool_args.page_shift == 12 && pool_args.n == 64 && launches == 6);
    CHECK(kv4_fork(&p, I, I, I, 64, I, I, nullptr) == MOE_OK && kv4_release(&p, I, I, 1, nullptr) == MOE_OK && launches == 8);
    moe_kv4_pool wide = p;
    wide.max_pages = big;
    CHECK(kv4_reserve(&wide, I, I, 1, I, nullptr) == MOE_EINVAL && kv4_fork(&wide, I, I, I, 1, I, I, nullptr) == MOE_EINVAL);
    CHECK(kv4_reserve(nullptr, I, I, 1, I, nullptr) == MOE_EINVAL && kv4_reserve(&p, I, I, big, I, nullptr) == MOE_EINVAL && launches == 8);
    const size_t need = kv4_compact_workspace_bytes(&p, 1 << 24);
    CHECK(need == ((size_t)5 << 24) && kv4_compact(&p, 1 << 24, I, P, need, nullptr) == MOE_OK && compact_args.max_moves == 1 << 24);
    CHECK(kv4_compact(&p, 1 << 24, I, P, need - 1, nullptr) == MOE_EWORKSPACE && kv4_compact_workspace_bytes(&p, -1) == 0);
    moe_kv4_cache huge{P, big, 4096, 1024, 256};
    CHECK(kv4_copy_pages(&huge, I, 1 << 24, nullptr) == MOE_OK && copy_args.page_bytes == (size_t)1024 * 256 * 17 * 256);
    CHECK(kv4_copy_pages(&huge, I, big, nullptr) == MOE_EINVAL && launches == 10);
    if (failures == 0) std::puts("all checks passed");
    return failures != 0;
}
