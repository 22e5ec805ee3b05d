// Host-side checks of the serving operators (csrc/serve.cpp) under
// AddressSanitizer and UndefinedBehaviorSanitizer (g++), with recorders in
// place of the kernel launchers.  The arrays that the ABI marks (host) are heap
// blocks of exactly the documented size, so that a read past one is seen;
// device pointers are addresses that nothing dereferences.  Exit status 0 = pass.
#include <cstdio>
#include <limits>
#include <memory>
#include <string>
#include <vector>

#include "moe_verify.h"
#include "serve.h"

static int failures = 0, appends = 0, attends = 0, samples = 0, accepts = 0;
static std::string error;
static moe::KvAppendArgs append_args;
static moe::KvAttendArgs attend_args;
static moe::SampleArgs sample_args;
static moe::AcceptArgs accept_args;

namespace moe {
int set_error(int code, const char *msg) {
    error = msg;
    return code;
}
int device_cu_count() { return 256; }
hipError_t launch_kv4_append(const KvAppendArgs &a, hipStream_t) {
    ++appends;
    append_args = a;
    return hipSuccess;
}
size_t kv4_attend_plan(KvAttendArgs &a, int n_cu) {
    a.mt = 1;
    a.nwg = n_cu;
    return 4096;
}
hipError_t launch_kv4_attend(const KvAttendArgs &a, hipStream_t) {
    ++attends;
    attend_args = a;
    return hipSuccess;
}
size_t sample_ws_bytes(int T, int V) { return (size_t)T * 256 + (size_t)V; }
hipError_t launch_sample(const SampleArgs &a, const float *, int32_t *, float *, float *, hipStream_t) {
    ++samples;
    sample_args = a;
    return hipSuccess;
}
hipError_t launch_accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t) {
    ++accepts;
    sample_args = a;
    accept_args = c;
    return hipSuccess;
}
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
    moe_kv4_cache c{P, 100, 64, 2, 128};
    std::vector<int32_t> one(65);
    for (int i = 0; i <= 64; ++i) one[i] = i;
    const auto off64 = block(one), off3 = block({0, 4, 4, 9}), bad = block({0, 5, 4, 9});
    moe_kv4_rows r3{I, 10, I, 3, off3.get()}, r64{I, 10, I, 64, off64.get()}, rb{I, 10, I, 3, bad.get()};

    // ---- append ----
    CHECK(kv4_append(&c, &r3, P, P, 256, 1024, 9, MOE_BF16, nullptr, nullptr, P, P, nullptr) == MOE_OK);
    CHECK(appends == 1 && append_args.r.page_shift == 6 && append_args.r.off[3] == 9 && append_args.vs == 1024 && !append_args.f32);
    CHECK(kv4_append(&c, &r64, P, P, 256, 256, 64, MOE_F32, I, I, nullptr, nullptr, nullptr) == MOE_OK && append_args.r.off[64] == 64);
    const auto all = block({0, 1 << 20});
    moe_kv4_rows ra{I, 10, I, 1, all.get()};
    CHECK(kv4_append(&c, &ra, P, P, 256, 256, 1 << 20, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) == MOE_OK);
    const int before = appends;
    CHECK(kv4_append(&c, &ra, P, P, 256, 256, (1 << 20) + 1, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) == MOE_EINVAL);
    CHECK(kv4_append(&c, &rb, P, P, 256, 256, 9, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) == MOE_EINVAL);
    CHECK(kv4_append(&c, &r3, P, P, 255, 256, 9, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) == MOE_EINVAL);
    CHECK(kv4_append(&c, &r3, P, P, std::numeric_limits<int64_t>::min(), 256, 9, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) ==
          MOE_EINVAL);
    CHECK(kv4_append(nullptr, &r3, P, P, 256, 256, 9, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) == MOE_EINVAL);
    CHECK(kv4_append(&c, nullptr, P, P, 256, 256, 9, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) == MOE_EINVAL);
    moe_kv4_rows wide = r3;
    wide.max_pages = std::numeric_limits<int32_t>::max();
    CHECK(kv4_append(&c, &wide, P, P, 256, 256, 9, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr) == MOE_EINVAL);
    CHECK(appends == before);

    // ---- attend: what each row sees ----
    const auto tree = block({-1, 0, 0, 1, -1, 0, 1, 0, 3});
    CHECK(kv4_attend_workspace_bytes(&c, &r3, 9, 8, MOE_BF16) == 4096);
    CHECK(kv4_attend(&c, &r3, P, 1024, 9, 8, MOE_BF16, 0.5f, tree.get(), P, P, 4096, nullptr) == MOE_OK && attends == 1);
    const uint64_t want[9] = {1, 3, 5, 11, 1, 3, 7, 9, 25};
    for (int t = 0; t < 9; ++t) CHECK(attend_args.anc[t] == want[t]);
    const auto whole = block({0, 64});
    moe_kv4_rows rw{I, 10, I, 1, whole.get()};
    CHECK(kv4_attend(&c, &rw, P, 1024, 64, 8, MOE_F32, 0.5f, nullptr, P, P, 4096, nullptr) == MOE_OK);
    CHECK(attend_args.anc[0] == 1 && attend_args.anc[62] == ~0ull >> 1 && attend_args.anc[63] == ~0ull && attend_args.G == 4);
    const auto late = block({-1, 0, 2, 1, -1, 0, 1, 0, 3});
    CHECK(kv4_attend(&c, &r3, P, 1024, 9, 8, MOE_BF16, 0.5f, late.get(), P, P, 4096, nullptr) == MOE_EINVAL);
    CHECK(kv4_attend(&c, &r3, P, 1024, 9, 8, MOE_BF16, std::numeric_limits<float>::infinity(), nullptr, P, P, 4096, nullptr) == MOE_EINVAL);
    CHECK(kv4_attend(&c, &r3, P, 1024, 9, 8, MOE_BF16, 0.5f, nullptr, P, P, 4095, nullptr) == MOE_EWORKSPACE);
    CHECK(kv4_attend_workspace_bytes(&c, &r3, 9, 7, MOE_BF16) == 0 && kv4_attend_workspace_bytes(&c, &rb, 9, 8, MOE_BF16) == 0);
    CHECK(attends == 2);

    // ---- draws and acceptance ----
    moe_sampling f{F, nullptr, F, nullptr};
    CHECK(sample_workspace_bytes(3, 1000) == 1768 && sample_workspace_bytes(65536, 10) == 0 && sample_workspace_bytes(1, (1 << 18) + 1) == 0);
    CHECK(sample_tokens(P, 1000, 3, 1000, MOE_F32, &f, F, I, nullptr, nullptr, P, 1768, nullptr) == MOE_OK && samples == 1);
    CHECK(sample_args.temperature == F && !sample_args.top_k && sample_args.top_p == F && !sample_args.min_p);
    CHECK(sample_tokens(P, 1000, 3, 1000, MOE_BF16, nullptr, F, I, nullptr, nullptr, P, 1768, nullptr) == MOE_OK && !sample_args.top_p);
    CHECK(sample_tokens(nullptr, 0, 0, 1000, MOE_F32, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, 0, nullptr) == MOE_OK && samples == 2);
    CHECK(sample_tokens(P, 999, 3, 1000, MOE_F32, &f, F, I, nullptr, nullptr, P, 1768, nullptr) == MOE_EINVAL);
    CHECK(accept_drafts(P, 1000, 9, 1000, MOE_F32, &f, I, 3, off3.get(), tree.get(), nullptr, F, nullptr, I, I, I, P, 1 << 16, nullptr) ==
          MOE_OK);
    const int parents[9] = {-1, 0, 0, 1, -1, 4, 5, 4, 7};
    for (int t = 0; t < 9; ++t) CHECK(accept_args.parent[t] == parents[t]);
    CHECK(accept_drafts(P, 1000, 64, 1000, MOE_F32, nullptr, I, 1, whole.get(), nullptr, F, F, F, I, I, I, P, 1 << 16, nullptr) == MOE_OK);
    CHECK(accept_args.parent[0] == -1 && accept_args.parent[63] == 62 && accepts == 2);
    CHECK(accept_drafts(P, 1000, 9, 1000, MOE_F32, &f, I, 3, off3.get(), tree.get(), F, F, F, I, I, I, P, 1 << 16, nullptr) == MOE_ENOTSUP);
    CHECK(accept_drafts(P, 1000, 9, 1000, MOE_F32, &f, I, 3, off3.get(), nullptr, F, F, nullptr, I, I, I, P, 1 << 16, nullptr) == MOE_EINVAL);
    CHECK(accept_drafts(P, 1000, 9, 1000, MOE_F32, &f, I, 65, off64.get(), nullptr, nullptr, F, nullptr, I, I, I, P, 1 << 16, nullptr) ==
          MOE_EINVAL);
    CHECK(accepts == 2);
    if (failures == 0) std::puts("all checks passed");
    return failures != 0;
}
