// Host checks of csrc/plan.h (tile sizes, grids, workspace layouts of the
// operators for prompts) under AddressSanitizer and UndefinedBehaviorSanitizer.
// Lines "T k E I f32" on stdin are answered by the rows of a product tile, one
// a line, on stdout.  Exit status 0 = pass.
#include <cstdio>
#include <random>
#include <utility>
#include <vector>

#include "moe_verify.h"
#include "plan.h"

using namespace moe;

static int failures = 0;

#define CHECK(cond)                                                       \
    do {                                                                  \
        if (!(cond)) {                                                    \
            std::fprintf(stderr, "FAIL line %d: %s\n", __LINE__, #cond);  \
            ++failures;                                                   \
        }                                                                 \
    } while (0)

static ExpertArgs call(int T, int k, int E, int H, int I, bool f32, bool shared) {
    ExpertArgs a{};
    a.T = T, a.k = k, a.E = E, a.H = H, a.I = I, a.f32 = f32, a.shared = shared;
    return a;
}

// The arrays of a call lie behind each other, aligned, inside the workspace.
static void layout(const ExpertArgs &a) {
    const plan::Experts q = plan::experts(a);
    const size_t pairs = (size_t)a.T * a.k, rows = pairs + (a.shared ? a.T : 0);
    CHECK((size_t)q.pairs == pairs && (size_t)q.rows == rows);
    CHECK((int64_t)q.chunk * q.chunks >= q.pairs && q.chunks <= plan::kMaxChunks && (q.pairs == 0 || q.chunks >= 1));
    CHECK(q.Ip >= a.I && q.Ip % 64 == 0);
    const std::pair<size_t, size_t> parts[] = {
        {q.counts, (size_t)q.chunks * a.E * 4}, {q.first, (size_t)(a.E + 2) * 4}, {q.tile, (size_t)(a.E + 2) * 4}, {q.row_token, rows * 4},
        {q.row_of, pairs * 4}, {q.x, a.f32 ? (size_t)a.T * a.H * 6 : 0}, {q.h, (a.f32 ? 3 : 1) * rows * q.Ip * 2}, {q.out, rows * a.H * 4}};
    size_t end = 0;
    for (const auto &p : parts) {
        CHECK(p.first >= end && p.first % 256 == 0);
        end = p.first + p.second;
    }
    CHECK(end <= q.bytes);
}

// A product's grid holds the tiles of any division of the pairs among the experts.
static void grid(std::mt19937 &rng, const ExpertArgs &a) {
    const int TN = plan::tile_rows(a), TM = TN == 32 ? 64 : TN;
    for (int trial = 0; trial < 4; ++trial) {
        std::vector<int64_t> n(a.E);
        const int used = trial == 0 ? 1 : 1 + (int)(rng() % a.E);
        for (int64_t i = 0; i < (int64_t)a.T * a.k; ++i) ++n[trial == 3 ? i % a.E : rng() % used];
        int64_t tiles = a.shared ? (a.T + TN - 1) / TN : 0;
        for (int64_t c : n) tiles += (c + TN - 1) / TN;
        CHECK(tiles * ((2 * (int64_t)a.I + TM - 1) / TM) <= plan::product_grid(a, true, TM, TN));
        CHECK(tiles * ((a.H + TM - 1) / TM) <= plan::product_grid(a, false, TM, TN));
    }
}

static void prompt(const std::vector<int> &n, const std::vector<int> &m, int Hq, int Hkv, int D, bool f32, int n_cu) {
    PromptArgs a{};
    a.nseq = (int)n.size(), a.Hq = Hq, a.Hkv = Hkv, a.G = Hq / Hkv, a.D = D, a.f32 = f32;
    int64_t blocks = 0;
    int keys = 0;
    for (int s = 0; s < a.nseq; ++s) {
        a.q_off[s + 1] = a.q_off[s] + n[s];
        a.k_off[s + 1] = a.k_off[s] + m[s];
        blocks += (n[s] + plan::kRows - 1) / plan::kRows;
        if (n[s] > 0) keys = std::max(keys, m[s]);
    }
    const size_t ws = plan::prompt(a, n_cu), terms = f32 ? (size_t)a.k_off[a.nseq] * Hkv * D * 12 : 0;
    CHECK(a.blocks[a.nseq] == blocks && (a.units == blocks * Hq || (a.units == INT32_MAX && blocks * Hq >= INT32_MAX)));
    CHECK(a.parts >= 1 && a.parts <= 64 && (a.parts == 1 || a.parts <= keys / 256));
    CHECK(a.part_at >= terms && a.part_at % 256 == 0 && a.part_at < terms + 256);
    CHECK(ws == a.part_at + (a.parts > 1 ? (size_t)a.units * a.parts * plan::kRows * (D + 2) * 4 : 0));
}

int main() {
    std::mt19937 rng(5);
    for (int T : {0, 1, 63, 4099, 1 << 20})
        for (int k : {1, 8, 32})
            for (int E : {32, 512})
                for (int H : {64, 8320, 16384})
                    for (int I : {32, 1 << 20})
                        for (int flags = 0; flags < 4; ++flags) layout(call(T, k, E, H, I, flags & 1, flags & 2));
    for (int i = 0; i < 300; ++i) {
        const int E = 1 + rng() % 512, k = 1 + rng() % std::min(E, 32), T = 1 + rng() % (rng() % 2 ? 40 : 3000);
        grid(rng, call(T, k, E, 64 * (1 + rng() % 64), 32 * (1 + rng() % 64), rng() % 2, rng() % 2));
    }
    CHECK(!plan::experts_fit(call(1 << 20, 32, 512, 16384, 256, false, false)));  // 2^34 elements
    CHECK(plan::experts_fit(call(4099, 4, 32, 2880, 2880, false, false)));
    CHECK(!plan::experts_fit(call(1 << 20, 1, 1, 64, 1 << 20, false, false)));    // a grid of 2^25

    const int most = 1 << 22;
    for (int D : {64, 128, 256})
        for (int f32 = 0; f32 < 2; ++f32) {
            prompt({0}, {0}, 1, 1, D, f32, 256);
            prompt({most}, {most}, 8192, 1, D, f32, 256);
            prompt({1}, {most}, 1024, 1024, D, f32, 256);
            prompt({515}, {60516}, 32, 8, D, f32, 256);
            prompt(std::vector<int>(64, most / 64), std::vector<int>(64, most / 64), 8, 8, D, f32, 1);
            for (int i = 0; i < 200; ++i) {
                std::vector<int> n(1 + rng() % 64), m(n.size());
                for (size_t s = 0; s < n.size(); ++s) n[s] = rng() % 4 ? rng() % 700 : 0, m[s] = rng() % 4 ? rng() % 50000 : 0;
                const int Hkv = 1 + rng() % 16;
                prompt(n, m, Hkv * (1 + rng() % 8), Hkv, D, f32, 256);
            }
        }

    for (int P : {1, 2, 4095, 4096, 4097, 1 << 24})
        for (int moves : {1, 3, 4096, 1 << 24}) {
            const size_t lists = std::min(moves, P / 2);
            CHECK(plan::compact_bytes(P, moves) == 4 * ((size_t)(P + 4095) / 4096 + 1 + 2 * lists + P));
        }

    int T, k, E, I, f32;
    while (std::scanf("%d %d %d %d %d", &T, &k, &E, &I, &f32) == 5) std::printf("%d\n", plan::tile_rows(call(T, k, E, 64, I, f32, false)));
    if (failures == 0) std::puts("all checks passed");
    return failures != 0;
}
