// Host-side planning of the operators for prompts: tile sizes, grids and
// workspace layouts from sizes alone, so that a host program can check them.
// Included by the sources that launch the kernels.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "prompt.h"

namespace moe {
namespace plan {

// Hands out 256-byte aligned places one behind the other.
struct Places {
    size_t end = 0;
    size_t take(size_t bytes) {
        const size_t at = end;
        end += (bytes + 255) & ~(size_t)255;
        return at;
    }
};

// ---- prompt_attend ----
constexpr int kRows = 128;  // query rows of a workgroup

inline size_t prompt(PromptArgs &a, int n_cu) {
    int blocks = 0, keys = 0;
    a.blocks[0] = 0;
    for (int s = 0; s < a.nseq; ++s) {
        const int n = a.q_off[s + 1] - a.q_off[s], m = a.k_off[s + 1] - a.k_off[s];
        blocks += (n + kRows - 1) / kRows;
        a.blocks[s + 1] = blocks;
        if (n > 0 && m > keys) keys = m;
    }
    a.units = (int64_t)blocks * a.Hq < INT32_MAX ? blocks * a.Hq : INT32_MAX;
    a.parts = 1;
    // Units that fill the workgroups that run at once a few times over at most leave some idle in the
    // last round.  Their keys are cut into as many shares of at least 256 as take the least time, by
    // what a step of 64 keys costs a workgroup (1.6 us at D = 128 where two share a compute unit) and
    // the join of a share's rows.  (515 rows, 32 heads, 60516 keys: 570 us with three shares, 680 with
    // the four that fill every workgroup, 571 with sixteen.)
    const int slots = n_cu * (a.f32 ? 1 : 2);
    if (a.units > 0 && a.units < 4 * slots) {
        const double step = 1.6 * a.D / 128 * (a.f32 ? 3 : 1), join = (double)a.units * kRows * (a.D + 2) * 8 / 4.5e6;
        double best = 1e30;
        for (int p = 1; p <= 64 && (p == 1 || p <= keys / 256); ++p) {
            const int64_t rounds = ((int64_t)a.units * p + slots - 1) / slots;
            const double cost = rounds * (keys / 64.0 / p) * step + (p > 1 ? 4 + join * p : 0);
            if (cost < 0.98 * best) best = cost, a.parts = p;
        }
    }
    size_t ws = a.f32 ? (size_t)a.k_off[a.nseq] * a.Hkv * a.D * 12 : 0;
    ws = (ws + 255) & ~(size_t)255;
    a.part_at = ws;
    if (a.parts > 1) ws += (size_t)a.units * a.parts * kRows * (a.D + 2) * 4;
    return ws;
}

// ---- moe_experts ----
constexpr int kMinChunk = 2048;  // pairs of a workgroup of the list kernels at least
constexpr int kMaxChunks = 256;

// Rows of a product tile: large ones where experts have some rows on average and
// their tiles are enough to fill half the card, small ones (32 rows by 64
// weight rows) else.  us a call, small and large: 32 experts of 2048 x 1024, bf16, 24
// rows each 90 and 89, 48 rows 110 and 94, 128 rows 196 and 109 (float32 111 and 101, 142
// and 111, 287 and 215); 60 of 1024 x 512, 24 rows 45.6 and 46.3, 32 rows 50.9 and 47.8;
// 8 of 1024 x 512 (32 large tiles), 32 rows 21.2 and 24.6, 160 rows 28.1 and 42.7.
// (The 403 MB of weights of the first take 62 us at the rate of a streaming read.)
inline int tile_rows(const ExpertArgs &a) {
    const int64_t pairs = (int64_t)a.T * a.k;
    const int large = a.f32 ? 128 : 256;
    const int64_t tiles = std::max(pairs / large, (int64_t)a.E) * ((2 * (int64_t)a.I + large - 1) / large);
    return pairs / a.E < 28 || tiles < 128 ? 32 : large;
}

// Workgroups of a product: tiles at most, since every used expert's last one is filled in part.
inline int64_t product_grid(const ExpertArgs &a, bool gate_up, int TM, int TN) {
    const int64_t M = gate_up ? 2 * (int64_t)a.I : a.H, mblocks = (M + TM - 1) / TM, pairs = (int64_t)a.T * a.k;
    const int64_t used = a.E < pairs ? a.E : pairs;
    const int64_t tiles = pairs / TN + used + (a.shared ? (a.T + TN - 1) / TN : 0);
    return (tiles * mblocks + 7) / 8 * 8;
}

inline bool experts_fit(const ExpertArgs &a) {
    const int TN = tile_rows(a), TM = TN == 32 ? 64 : TN == 128 ? 128 : 256;
    const int64_t grid = std::max(product_grid(a, true, TM, TN), product_grid(a, false, TM, TN));
    return grid < 1 << 22 && (int64_t)a.T * a.H < (int64_t)1 << 33;
}

// Sizes of a call, and where its arrays lie in the workspace.
struct Experts {
    int pairs, rows;    // T k, and with the shared expert's
    int chunk, chunks;  // pairs of a workgroup of the list kernels
    int tn;             // rows of a product tile
    int Ip;             // elements of a hidden row
    size_t counts, first, tile, row_token, row_of, x, h, out, bytes;
};

inline Experts experts(const ExpertArgs &a) {
    Experts q{};
    q.pairs = a.T * a.k;
    q.rows = q.pairs + (a.shared ? a.T : 0);
    q.chunk = std::max((q.pairs + kMaxChunks - 1) / kMaxChunks, kMinChunk);
    q.chunks = (q.pairs + q.chunk - 1) / q.chunk;
    q.tn = tile_rows(a);
    q.Ip = (a.I + 63) / 64 * 64;
    const int NT = a.f32 ? 3 : 1;
    Places p;
    q.counts = p.take((size_t)q.chunks * a.E * 4);
    q.first = p.take((a.E + 2) * 4);
    q.tile = p.take((a.E + 2) * 4);
    q.row_token = p.take((size_t)q.rows * 4);
    q.row_of = p.take((size_t)q.pairs * 4);
    q.x = p.take(a.f32 ? (size_t)a.T * a.H * 6 : 0);
    q.h = p.take((size_t)NT * q.rows * q.Ip * 2);
    q.out = p.take((size_t)q.rows * a.H * 4);
    q.bytes = p.end;
    return q;
}

// ---- kv4_compact ----
constexpr int kCompactChunk = 4096;  // pages of a workgroup

inline int compact_most(int num_pages, int max_moves) { return std::min(max_moves, num_pages / 2); }

// Workspace: used pages of each chunk and of all, the lowest free and the
// highest used pages, the used pages' ranks.
inline size_t compact_bytes(int num_pages, int max_moves) {
    return 4 * ((size_t)(num_pages + kCompactChunk - 1) / kCompactChunk + 1 + 2 * (size_t)compact_most(num_pages, max_moves) + num_pages);
}

}  // namespace plan
}  // namespace moe
