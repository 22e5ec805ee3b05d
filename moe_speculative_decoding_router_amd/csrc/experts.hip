// The experts of prompts: the choice of each token's experts from its router
// logits, and the experts' products over any number of tokens.
#include "common.h"
#include "dma.h"
#include "plan.h"

#include <type_traits>

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Route.  One wave a token, E / 64 logits a lane as integers whose order is the
// floats'; k rounds of a wave maximum, each taking the lowest index that holds
// it, so that lane r ends with rank r.
// ---------------------------------------------------------------------------
// Latency bounds it: 65 tokens of 128 experts take 3.7 us, 16384 of 256 (17 MB) 10.
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

// ---------------------------------------------------------------------------
// The experts' products.  The (token, rank) pairs are grouped by expert (rows
// of the products); gate-up makes the hidden activations of every row, down
// their outputs, combine the tokens' weighted sums in rank order.
//
// Weights are the A operand of v_mfma_f32_16x16x32_bf16: the packed tiles come
// into LDS as they are and are read from it 16 bytes a lane, without a bank met
// twice; activations are the B operand, gathered by row straight into LDS, 128 bytes
// a row and load.  An fp8 tile is converted to bf16 in registers, exactly, times
// the power of two of its block's scale; what is left of the scale, a factor in
// [1, 2), is kept out of the sums, which are multiplied by the quotient of two
// blocks' factors when the block changes, every 128 k: no second set of
// accumulators, and no quotient that overflows.
//
// What is rounded in bf16 calls: the hidden activations (each by at most 2^-8) and
// the result.  The experts' outputs stay float32 until they are added: as bf16
// they would save 90 MB of the 378 that 16396 rows of 2880 write and read, but the
// results would be off by 0.0029 of their norm instead of 0.0023 (plain float32 ones that
// are rounded once: 0.0017).
//
// What bounds it: 4099 tokens, 4 of 32 experts of 2880 x 2880 (816 GFLOP) take 877 to
// 930 us, of which gate-up 543 (1000 TFLOP/s) and down 325 (835), where a large bf16
// product reaches 1352; 40 go to adding 190 MB of outputs, 9 to the lists.  Matrix
// instructions are under way 52% of the cycles: compute units idle 20% of the
// time behind the last of their six or seven tiles, and the clock falls to 1.9 GHz.
// fp8, 1024 tokens, 8 of 32 experts of 7168 x 2048 and a shared one (812 GFLOP): 960 to 1040.
// Tried and slower: workgroups that stay and draw tiles by ticket (bf16 964), tiles
// of half the rows at the end of the list (958), 128 x 512 tiles (1055; the
// activations no longer stay in the L2), v_mfma_f32_32x32x16_bf16 (940), row blocks
// dealt to the XCDs in turn (908), outputs stored past the caches (962).
// ---------------------------------------------------------------------------
constexpr int kListThreads = 256;
constexpr int kPerRound = 8;  // pairs of a thread at a time

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));

// The workspace, and what every kernel of a call needs.
struct Plan {
    ExpertArgs a;
    int pairs, rows;     // T k, and with the shared expert's
    int chunk, chunks;   // pairs of a workgroup of the list kernels
    int tn;              // rows of a product tile
    int Ip;              // elements of a hidden row
    int *counts;         // [chunks][E]
    int *first;          // [E + 2] first row of each expert (E: the shared one)
    int *tile;           // [E + 2] product tiles before each expert
    int *row_token;      // [rows]
    int *row_of;         // [pairs] row of each pair, -1 for entries that name no expert
    __bf16 *x;           // [3][T][H] terms of float32 activations
    __bf16 *h;           // [NT][rows][Ip] hidden activations
    float *out;          // [rows][H] outputs
};

__global__ __launch_bounds__(kListThreads) void count_pairs_kernel(Plan p) {
    __shared__ int n[kMaxExperts];
    for (int e = threadIdx.x; e < p.a.E; e += kListThreads) n[e] = 0;
    __syncthreads();
    const int64_t end = min((int64_t)(blockIdx.x + 1) * p.chunk, (int64_t)p.pairs);
    for (int64_t i = (int64_t)blockIdx.x * p.chunk + threadIdx.x; i < end; i += kPerRound * kListThreads) {
        int e[kPerRound];
#pragma unroll
        for (int j = 0; j < kPerRound; ++j) e[j] = i + j * kListThreads < end ? p.a.idx[i + j * kListThreads] : -1;
#pragma unroll
        for (int j = 0; j < kPerRound; ++j)
            if (e[j] >= 0 && e[j] < p.a.E) atomicAdd(&n[e[j]], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.a.E; e += kListThreads) p.counts[(size_t)blockIdx.x * p.a.E + e] = n[e];
}

// Places the pairs.  A row's products do not depend on where it lies in its
// expert's list, so the order in which the atomics hand out places is free.
__global__ __launch_bounds__(kListThreads) void place_pairs_kernel(Plan p) {
    __shared__ int at[kMaxExperts], all[kMaxExperts], sum[2];
    const int E = p.a.E, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int e = tid; e < E; e += kListThreads) {
        int before = 0, n = 0;
        if (p.chunks > 1) {
#pragma unroll 8
            for (int c = 0; c < p.chunks; ++c) {
                const int v = p.counts[(size_t)c * E + e];
                before += c < (int)blockIdx.x ? v : 0;
                n += v;
            }
        }
        at[e] = before;
        all[e] = n;
    }
    __syncthreads();
    const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min(begin + p.chunk, (int64_t)p.pairs);
    if (p.chunks == 1) {
        for (int64_t i = tid; i < end; i += kListThreads) {
            const int e = p.a.idx[i];
            if (e >= 0 && e < E) atomicAdd(&all[e], 1);
        }
        __syncthreads();
    }
    if (wave == 0) {  // first rows and tiles of the experts, 64 at a time
        int rows = 0, tiles = 0;
        for (int e0 = 0; e0 < E; e0 += 64) {
            const int e = e0 + lane, n = e < E ? all[e] : 0, t = (n + p.tn - 1) / p.tn;
            const int ri = wave_incl_scan(n), ti = wave_incl_scan(t);
            if (e < E) {
                at[e] += rows + ri - n;
                if (blockIdx.x == 0) p.first[e] = rows + ri - n, p.tile[e] = tiles + ti - t;
            }
            rows += __builtin_amdgcn_readlane(ri, 63);
            tiles += __builtin_amdgcn_readlane(ti, 63);
        }
        if (lane == 0) {
            sum[0] = rows;
            if (blockIdx.x == 0) {
                const int own = p.a.shared ? p.a.T : 0;
                p.first[E] = rows, p.tile[E] = tiles;
                p.first[E + 1] = rows + own, p.tile[E + 1] = tiles + (own + p.tn - 1) / p.tn;
            }
        }
    }
    __syncthreads();
    for (int64_t i = begin + tid; i < end; i += kPerRound * kListThreads) {
        int e[kPerRound];
#pragma unroll
        for (int j = 0; j < kPerRound; ++j) e[j] = i + j * kListThreads < end ? p.a.idx[i + j * kListThreads] : -1;
#pragma unroll
        for (int j = 0; j < kPerRound; ++j) {
            const int64_t at_pair = i + j * kListThreads;
            if (at_pair >= end) break;
            int r = -1;
            if (e[j] >= 0 && e[j] < E) {
                r = atomicAdd(&at[e[j]], 1);
                p.row_token[r] = (int)((unsigned)at_pair / (unsigned)p.a.k);
            }
            p.row_of[at_pair] = r;
        }
    }
    if (p.a.shared)
        for (int64_t t = (int64_t)blockIdx.x * kListThreads + tid; t < p.a.T; t += (int64_t)gridDim.x * kListThreads)
            p.row_token[sum[0] + t] = (int)t;
}

// float32 activations as three planes of bf16 terms.
__global__ __launch_bounds__(kListThreads) void split_x_kernel(Plan p) {
    const int64_t i = ((int64_t)blockIdx.x * kListThreads + threadIdx.x) * 4, n = (int64_t)p.a.T * p.a.H;
    if (i >= n) return;
    const int64_t t = i / p.a.H;
    f32x4 v = *reinterpret_cast<const f32x4 *>((const float *)p.a.x + t * p.a.xs + (i - t * p.a.H));
#pragma unroll
    for (int y = 0; y < 3; ++y) {
        bf16x4 z;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = (__bf16)v[e], v[e] -= (float)z[e];
        *reinterpret_cast<bf16x4 *>(p.x + y * n + i) = z;
    }
}

// Rows of a tile lie in LDS as 8 chunks of 16 bytes (64 k), chunk c of row r at
// c ^ swizzle(r), so that 16 lanes that read one chunk of 16 rows meet no bank twice.
__device__ __forceinline__ int swizzle(int r) { return ((r >> 1) ^ ((r & 1) << 2)) & 7; }

// 8 e4m3 codes as bf16, times the power of two `scale`: exact (4 significant bits).
__device__ __forceinline__ bf16x8 decode8(unsigned lo, unsigned hi, float scale) {
    union {
        bf16x2v h[4];
        bf16x8 v;
    } o;
    o.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
    o.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
    o.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
    o.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
    return o.v;
}

// A block scale as a power of two and a factor in [1, 2) with its sign (1 for 0).
struct Scale {
    float power, factor;
};
__device__ __forceinline__ Scale parts_of(float s) {
    const unsigned u = __float_as_uint(s), e = u & 0x7f800000u;
    return {__uint_as_float(e), e ? __uint_as_float((u & 0x807fffffu) | 0x3f800000u) : 1.f};
}

// Shape of a product tile: TM weight rows by TN activation rows, WM x WN waves,
// FP8 weights, NT activation terms.  A wave's columns are 16 of every 16 WN
// activation rows, so that a tile with few rows costs all waves less; the loop
// is compiled for each number JN of such steps, with as many buffers of 64 k as
// LDS holds.
template <bool GU, bool FP8_, int NT_, int TM_, int TN_, int WM_, int WN_, int LDS_>
struct Shape {
    static constexpr bool kGateUp = GU, FP8 = FP8_;
    static constexpr int NT = NT_, TM = TM_, TN = TN_, WM = WM_, WN = WN_, kLds = LDS_;
    static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
    static constexpr int kStep = 16 * WN;  // activation rows of a step
    static constexpr int A = TM * (FP8 ? 64 : 128);  // bytes of a buffer
    static constexpr int PA = A / 1024 / kWaves;     // loads of a wave
    static constexpr int MT = TM / WM / 16, NC = TN / kStep;  // 16 x 16 tiles of a wave
    // loads of a wave for an activation term, 8 rows each: every wave has as many, so that
    // their counts tell which buffers are there
    static constexpr int PB(int jn) { return (jn * kStep + 8 * kWaves - 1) / (8 * kWaves); }
    static constexpr int B(int jn) { return NT * PB(jn) * kWaves * 1024; }
    // Buffers of activations and of weights: up to four of both, and one more of
    // the weights, which come from further away, where LDS still holds it.
    static constexpr int NB(int jn) {
        const int n = LDS_ / (A + B(jn));
        return n > 4 ? 4 : n;
    }
    static constexpr int NA(int jn) { return NB(jn) < 4 && NB(jn) * (A + B(jn)) + A <= LDS_ ? NB(jn) + 1 : NB(jn); }
    static_assert(A % (1024 * kWaves) == 0 && NB(NC) >= 2 && LDS_ <= 163840, "");
};

// What a workgroup works on.
struct Job {
    const uint8_t *W;
    const float *sc, *sc_up;  // fp8: scales of the result rows (gate-up: of the gate rows and the up rows)
    int mb, row0, rows, M, K;
};

// A wave's operands of one step of 32 k.
template <typename S, int JN>
struct Frags {
    typedef unsigned u32xa __attribute__((ext_vector_type(S::FP8 ? 2 : 4)));
    u32xa a[S::MT];
    bf16x8 b[S::NT][JN];
};

template <typename S, int JN>
__device__ __forceinline__ void multiply(const Plan &p, const Job &job, uint8_t *lds) {
    // A row's place among its expert's tiles, and so the loop that it goes through, is left to the order
    // of atomics: all loops have to round alike, so none may fuse a product into the rest it leaves.
#pragma clang fp contract(off)
    constexpr bool GU = S::kGateUp, FP8 = S::FP8;
    constexpr int NT = S::NT, MT = S::MT, NA = S::NA(JN), NB = S::NB(JN), PA = S::PA, PB = S::PB(JN), kLoads = PA + PB * NT;
    constexpr int kPlane = PB * S::kWaves * 1024, kB0 = NA * S::A;  // the activations' buffers lie behind the weights'
    static_assert((NB - 1) * PB * NT + (NA - 1) * PA < 63, "");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave / S::WN, wn = wave % S::WN, g = lane >> 4, c = lane & 15;
    const int K = job.K;

    // ---- loads: weights in pieces of 1 KB (16 rows x 32 or 64 k), activations of 8 rows x 64 k ----
    const int rts = job.M / 16, nkt = K / (FP8 ? 64 : 32), steps = (K + 63) / 64;
    const unsigned lds0 = lds_address(lds);
    const __bf16 *brow[PB];
    const size_t plane = GU ? (size_t)p.a.T * p.a.H : (size_t)p.rows * p.Ip;
#pragma unroll
    for (int j = 0; j < PB; ++j) {
        const int r = (j * S::kWaves + wave) * 8 + (lane >> 3);
        const int row = job.row0 + min(r, job.rows - 1);  // rows behind the last are copies of it
        if constexpr (GU) {
            const size_t t = p.row_token[row];
            brow[j] = NT > 1 ? p.x + t * p.a.H : (const __bf16 *)p.a.x + t * p.a.xs;
        } else {
            brow[j] = p.h + (size_t)row * p.Ip;
        }
        brow[j] += ((lane & 7) ^ swizzle(r)) * 8;
    }
    // load i of a wave's kLoads: the activations of a step, then the weights of a step
    auto load = [&](int i, int step_b, int buf_b, int step_a, int buf_a) {
        if (i >= PB * NT) {
            // piece of the buffer: row tile, then its k tiles
            const int piece = wave * PA + i - PB * NT, rt = FP8 ? piece : piece >> 1;
            const int kt = FP8 ? step_a : min(2 * step_a + (piece & 1), nkt - 1);
            const int grt = min(job.mb * (S::TM / 16) + rt, rts - 1);
            const size_t kb = GU ? (size_t)grt * nkt + kt : ((size_t)(grt >> 2) * nkt + kt) * 4 + (grt & 3);
            dma16(job.W + kb * 1024, lane * 16, lds0 + buf_a * S::A + piece * 1024);
        } else {
            const int j = i / NT, y = i % NT;
            dma16v(brow[j] + y * plane + step_b * 64, lds0 + kB0 + buf_b * (NT * kPlane) + y * kPlane + (j * S::kWaves + wave) * 1024);
        }
    };

    f32x4 acc[MT][JN];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < JN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // read i of a step's kReads: the activations first, every product needs them
    typedef Frags<S, JN> F;
    constexpr int kReads = NT * JN + MT;
    auto read = [&](F &f, int i, int buf_a, int buf_b, int s) {
        const uint8_t *A = lds + buf_a * S::A, *B = lds + kB0 + buf_b * (NT * kPlane);
        if (i < NT * JN) {
            const int y = NT - 1 - i / JN, j = i % JN, ch = FP8 ? 2 * g + s : 4 * s + g;
            f.b[y][j] = *reinterpret_cast<const bf16x8 *>(B + y * kPlane + ((j * S::WN + wn) * 16 + c) * 128 + ((ch ^ swizzle(c)) << 4));
        } else {
            const int m = wm * MT + i - NT * JN;
            const uint8_t *at = FP8 ? A + m * 1024 + lane * 16 + 8 * s : A + (m * 2 + s) * 1024 + lane * 16;
            f.a[i - NT * JN] = *reinterpret_cast<const typename F::u32xa *>(at);
        }
    };
    // The products of one step of 32 k, row tile by row tile; between them the reads of the next step
    // (`with`, if READ) and the loads of the buffer that has become free (if LOAD), in this order.
    float operand = 1.f, factor = 1.f, ratio = 1.f;
    int ba = 0, bb = 0;  // the buffers in use
    auto products = [&](const F &f, F &with, int at_a, int at_b, int at_s, int st, auto READ, auto LOAD, auto SCALE) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            if constexpr (LOAD.value) {
#pragma unroll
                for (int x = i * kLoads / MT; x < (i + 1) * kLoads / MT; ++x) load(x, min(st + NB, steps - 1), bb, min(st + NA, steps - 1), ba);
            }
            if constexpr (READ.value) {  // done with the last but one row tile
                constexpr int n = MT > 1 ? MT - 1 : 1;
#pragma unroll
                for (int x = min(i * kReads / n, kReads); x < min((i + 1) * kReads / n, kReads); ++x) read(with, x, at_a, at_b, at_s);
            }
            if constexpr (SCALE.value) {
#pragma unroll
                for (int j = 0; j < JN; ++j) acc[i][j] *= ratio;
            }
            bf16x8 a;
            if constexpr (FP8) a = decode8(f.a[i][0], f.a[i][1], operand);
            else a = __builtin_bit_cast(bf16x8, f.a[i]);
#pragma unroll
            for (int y = NT - 1; y >= 0; --y)  // the smaller terms first
#pragma unroll
                for (int j = 0; j < JN; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, f.b[y][j], acc[i][j], 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    // fp8: a new block of 128 k: its power of two goes into the codes, its factor into the sums.
    // A lane holds the scales of every 64th block; they are waited for where they are
    // loaded, since a wait where they are used would be for the buffers' loads as well.
    float scale_x = 0.f, scale_y = 0.f;
    auto rescale = [&](int st) {
        if constexpr (FP8) {
            const int block = st >> 1;
            if ((block & 63) == 0) {
                const int at = min(block + lane, K / 128 - 1);
                scale_x = job.sc[at];
                if (GU) scale_y = job.sc_up[at];
                asm volatile("" : "+v"(scale_x), "+v"(scale_y));
            }
            const Scale x = parts_of(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale_x), block & 63)));
            const Scale y = GU ? parts_of(__int_as_float(__builtin_amdgcn_readlane(__float_as_int(scale_y), block & 63))) : x;
            operand = GU && c >= 8 ? y.power : x.power;
            const float f = GU && lane >= 32 ? y.factor : x.factor;
            ratio = factor / f;
            factor = f;
        }
    };

    // Buffers behind the last step hold copies of it, so that all waits count the same loads.
#pragma unroll
    for (int i = 0; i < NA; ++i)
#pragma unroll
        for (int x = i < NB ? 0 : PB * NT; x < kLoads; ++x) load(x, min(i, steps - 1), i, min(i, steps - 1), i);
    dma_wait<(NB - 1) * PB * NT + (NA - 1) * PA>();
    dma_barrier();
    F f0, f1;
#pragma unroll
    for (int i = 0; i < kReads; ++i) read(f0, i, 0, 0, 0);
    auto step = [&](int st, auto SCALE) {
        products(f0, f1, ba, bb, 1, 0, yes, no, SCALE);
        const int na = ba + 1 == NA ? 0 : ba + 1, nb = bb + 1 == NB ? 0 : bb + 1;
        dma_wait<(NB - 2) * kLoads + (NA > NB ? PA : 0)>();  // the next buffers are there,
        dma_barrier();                                       // and these were read by all
        products(f1, f0, na, nb, 0, st, yes, yes, no);
        ba = na;
        bb = nb;
    };
    if constexpr (FP8) {  // an even number of steps
        int st = 0;
        for (; st + 2 < steps; st += 2) {
            rescale(st);
            step(st, yes);
            step(st + 1, no);
        }
        rescale(st);
        step(st, yes);
        products(f0, f1, ba, bb, 1, 0, yes, no, no);
        products(f1, f0, 0, 0, 0, 0, no, no, no);
    } else {
        for (int st = 0; st + 1 < steps; ++st) step(st, no);
        products(f0, f1, ba, bb, 1, 0, yes, no, no);
        if (GU || nkt % 2 == 0) products(f1, f0, 0, 0, 0, 0, no, no, no);  // else the last 32 k of an odd number
    }
    dma_wait<0>();

    // ---- results: lane (g, c) holds weight rows 4 g .. 4 g + 3 of its tiles for activation row c ----
    if constexpr (FP8) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < JN; ++j) acc[i][j] *= factor;
    }
    const int rt0 = job.mb * (S::TM / 16) + wm * MT;
#pragma unroll
    for (int j = 0; j < JN; ++j) {
        const int r = (j * S::WN + wn) * 16 + c;
        if constexpr (GU) {
            // a row tile is 8 gate rows (lanes below 32) and the same 8 up rows; two tiles exchange
            // halves, so that every lane holds both of one element
#pragma unroll
            for (int i = 0; i < MT; i += 2) {
                float hid[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const unsigned a0 = __float_as_uint(acc[i][j][x]), a1 = __float_as_uint(acc[MT > 1 ? i + 1 : i][j][x]);
                    const auto sw = __builtin_amdgcn_permlane32_swap(a0, a1, false, false);
                    const float gate = __uint_as_float(sw[0]), u = __uint_as_float(sw[1]);
                    hid[x] = gate * __builtin_amdgcn_rcpf(1.f + __expf(-gate)) * u;
                }
                const int rt = rt0 + i + (lane >> 5);
                if (r < job.rows && rt < rts && (MT > 1 || lane < 32)) {
                    __bf16 *to = p.h + (size_t)(job.row0 + r) * p.Ip + rt * 8 + 4 * (g & 1);
#pragma unroll
                    for (int y = 0; y < NT; ++y) {
                        bf16x4 z;
#pragma unroll
                        for (int x = 0; x < 4; ++x) z[x] = (__bf16)hid[x], hid[x] -= (float)z[x];
                        *reinterpret_cast<bf16x4 *>(to + (size_t)y * p.rows * p.Ip) = z;
                    }
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                if (r >= job.rows || rt0 + i >= rts) continue;
                *reinterpret_cast<f32x4 *>(p.out + (size_t)(job.row0 + r) * p.a.H + (rt0 + i) * 16 + 4 * g) = acc[i][j];
            }
        }
    }
}

template <typename S>
__global__ __launch_bounds__(S::kThreads, 2) void product_kernel(Plan p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // [NA][A], [NB][B]
    constexpr bool GU = S::kGateUp, FP8 = S::FP8;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int E = p.a.E;
    Job job;
    job.K = GU ? p.a.H : p.a.I;
    job.M = GU ? 2 * p.a.I : p.a.H;
    const int mblocks = (job.M + S::TM - 1) / S::TM;

    // ---- the workgroup's tile: each XCD takes a run of neighbours, an expert's row blocks
    // one after the other and all its tiles beside each other ----
    const int64_t items = (int64_t)p.tile[E + 1] * mblocks, run = (items + 7) >> 3;
    const int64_t item = (blockIdx.x & 7) * run + (blockIdx.x >> 3);
    if ((int64_t)(blockIdx.x >> 3) >= run || item >= items) return;
    int e = 0;
    for (int e0 = 0; e0 <= E; e0 += 64) {
        const int x = min(e0 + (int)(threadIdx.x & 63), E);
        const uint64_t at = __ballot(item >= (int64_t)p.tile[x] * mblocks && item < (int64_t)p.tile[x + 1] * mblocks);
        if (at) e = min(e0 + __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)at)) - 1, E);
    }
    const int t0 = p.tile[e], nt = p.tile[e + 1] - t0;
    const int in = (int)(item - (int64_t)t0 * mblocks), tile = in % nt;
    job.mb = in / nt;
    job.row0 = p.first[e] + tile * S::TN;
    job.rows = min(S::TN, p.first[e + 1] - job.row0);
    const bool own = e == E;  // the shared expert
    job.W = (const uint8_t *)(GU ? (own ? p.a.Wsh_gu : p.a.W_gu) : (own ? p.a.Wsh_d : p.a.W_d)) +
            (own ? 0 : (size_t)e * job.M * job.K * (FP8 ? 1 : 2));
    if constexpr (FP8) {  // a wave's weight rows lie in one block of 128, gate and up rows in one each
        const float *s = GU ? (own ? p.a.ssh_gu : p.a.s_gu) : (own ? p.a.ssh_d : p.a.s_d);
        const int kbs = job.K / 128;
        const int block = GU ? job.mb * (S::TM / 2) / 128 : min((job.mb * S::TM + wave / S::WN * (S::TM / S::WM)) / 128, job.M / 128 - 1);
        job.sc = s + (own ? 0 : (size_t)e * (job.M / 128) * kbs) + (size_t)block * kbs;
        job.sc_up = job.sc + (size_t)(p.a.I / 128) * kbs;
    }
    const int jn = (job.rows + S::kStep - 1) / S::kStep;
    if constexpr (S::NC >= 4) {
        if (jn == 4) return multiply<S, 4>(p, job, lds);
        if (jn == 3) return multiply<S, 3>(p, job, lds);
    }
    if constexpr (S::NC >= 2) {
        if (jn == 2) return multiply<S, 2>(p, job, lds);
    }
    multiply<S, 1>(p, job, lds);
}

// y[t] = sum of the token's rows in rank order, times their weights, and of the
// shared expert's.  8 elements a thread.
template <bool F32>
__global__ __launch_bounds__(kListThreads) void combine_rows_kernel(Plan p) {
    const int t = blockIdx.x, H = p.a.H;
    const int own = p.a.shared ? p.first[p.a.E] + t : -1;
    for (int i = (blockIdx.y * kListThreads + threadIdx.x) * 8; i < H; i += gridDim.y * kListThreads * 8) {
        float y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] = 0.f;
        auto add = [&](int row, float w) {
            const f32x4 *v = reinterpret_cast<const f32x4 *>(p.out + (size_t)row * H + i);
            const f32x4 a = v[0], b = v[1];
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = fmaf(w, a[e], y[e]), y[4 + e] = fmaf(w, b[e], y[4 + e]);
        };
        for (int j = 0; j < p.a.k; ++j) {
            const int row = p.row_of[(size_t)t * p.a.k + j];
            if (row >= 0) add(row, p.a.w[(size_t)t * p.a.k + j]);
        }
        if (own >= 0) add(own, 1.f);
        if constexpr (F32) {
            f32x4 *d = reinterpret_cast<f32x4 *>((float *)p.a.y + (size_t)t * H + i);
            d[0] = f32x4{y[0], y[1], y[2], y[3]};
            d[1] = f32x4{y[4], y[5], y[6], y[7]};
        } else {
            bf16x8 z;
#pragma unroll
            for (int e = 0; e < 8; ++e) z[e] = (__bf16)y[e];
            *reinterpret_cast<bf16x8 *>((__bf16 *)p.a.y + (size_t)t * H + i) = z;
        }
    }
}

template <typename S>
hipError_t launch_product(const Plan &p, hipStream_t s) {
    if (S::kLds > 65536) {
        const hipError_t e = allow_lds<product_kernel<S>>(S::kLds);
        if (e != hipSuccess) return e;
    }
    const int64_t grid = plan::product_grid(p.a, S::kGateUp, S::TM, S::TN);
    hipLaunchKernelGGL(product_kernel<S>, dim3((unsigned)grid), dim3(S::kThreads), S::kLds, s, p);
    return hipGetLastError();
}

template <bool FP8, int NT, int TM, int TN, int WM, int WN, int LDS>
hipError_t launch_both(const Plan &p, hipStream_t s) {
    const hipError_t e = launch_product<Shape<true, FP8, NT, TM, TN, WM, WN, LDS>>(p, s);
    if (e != hipSuccess) return e;
    return launch_product<Shape<false, FP8, NT, TM, TN, WM, WN, LDS>>(p, s);
}

template <bool FP8>
hipError_t launch_products(const Plan &p, hipStream_t s) {
    if (p.a.f32) {
        if (p.tn == 32) return launch_both<FP8, 3, 64, 32, 4, 1, 81920>(p, s);
        return launch_both<FP8, 3, 128, 128, 2, 4, 163840>(p, s);
    }
    if (p.tn == 32) return launch_both<FP8, 1, 64, 32, 4, 1, 81920>(p, s);
    return launch_both<FP8, 1, 256, 256, 2, 4, 163840>(p, s);
}

Plan lay_out(const ExpertArgs &a) {
    const plan::Experts q = plan::experts(a);
    uint8_t *ws = (uint8_t *)a.ws;
    Plan p{};
    p.a = a;
    p.pairs = q.pairs;
    p.rows = q.rows;
    p.chunk = q.chunk;
    p.chunks = q.chunks;
    p.tn = q.tn;
    p.Ip = q.Ip;
    p.counts = (int *)(ws + q.counts);
    p.first = (int *)(ws + q.first);
    p.tile = (int *)(ws + q.tile);
    p.row_token = (int *)(ws + q.row_token);
    p.row_of = (int *)(ws + q.row_of);
    p.x = (__bf16 *)(ws + q.x);
    p.h = (__bf16 *)(ws + q.h);
    p.out = (float *)(ws + q.out);
    return p;
}

}  // namespace

bool experts_fit(const ExpertArgs &a) { return plan::experts_fit(a); }

size_t experts_ws_bytes(const ExpertArgs &a) { return plan::experts(a).bytes; }

hipError_t launch_experts(const ExpertArgs &a, hipStream_t s) {
    const Plan p = lay_out(a);
    if (p.chunks > 1) hipLaunchKernelGGL(count_pairs_kernel, dim3(p.chunks), dim3(kListThreads), 0, s, p);
    hipLaunchKernelGGL(place_pairs_kernel, dim3(p.chunks), dim3(kListThreads), 0, s, p);
    if (a.f32) {
        const int64_t n = ((int64_t)a.T * a.H / 4 + kListThreads - 1) / kListThreads;
        hipLaunchKernelGGL(split_x_kernel, dim3((unsigned)n), dim3(kListThreads), 0, s, p);
    }
    hipError_t e = hipGetLastError();
    if (e == hipSuccess) e = a.fp8 ? launch_products<true>(p, s) : launch_products<false>(p, s);
    if (e != hipSuccess) return e;
    const dim3 grid(a.T, (a.H + kListThreads * 8 - 1) / (kListThreads * 8));
    if (a.f32) hipLaunchKernelGGL(combine_rows_kernel<true>, grid, dim3(kListThreads), 0, s, p);
    else hipLaunchKernelGGL(combine_rows_kernel<false>, grid, dim3(kListThreads), 0, s, p);
    return hipGetLastError();
}

hipError_t launch_route_tokens(const float *logits, int64_t stride, int T, int E, int k, int32_t *idx, float *w,
                               hipStream_t s) {
    const int n = (E + 63) / 64;
    auto kern = n == 1 ? route_tokens_kernel<1> : n == 2 ? route_tokens_kernel<2> : n <= 4 ? route_tokens_kernel<4> : route_tokens_kernel<8>;
    hipLaunchKernelGGL(kern, dim3((T + kRouteThreads / 64 - 1) / (kRouteThreads / 64)), dim3(kRouteThreads), 0, s, logits, stride,
                       T, E, k, idx, w);
    return hipGetLastError();
}

}  // namespace moe
