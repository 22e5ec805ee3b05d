// Drawing and accepting draft tokens.  The filtered distribution of a row of
// logits is defined in include/moe_verify.h.
//
// Every filter keeps a prefix of the row's ranking (value desc, index asc),
// so a row's filter is one threshold: the last kept value and, among equal
// values, the last kept index.  Weights w = exp(-(first - l) / temperature)
// are computed in float64 and summed as integers in units of 2^-45: a sum
// does not depend on its order, and 2^18 weights of at most 1 fit 63 bits.
// (Two sums of long rows are joined from the chunks' in float64 instead: the
// row's in join_kernel and in row_mass.)
//
// A row is cut into chunks of 4096 tokens, a workgroup each.  Without
// filters two launches draw: part_kernel (each chunk's largest value and its
// sum relative to it, one pass over the logits) and join_kernel (a workgroup
// a row: the chunk that holds the draw, then the token).  With filters:
//   max_kernel      the row's largest value
//   hist_kernel     a histogram of the distance from it (1 / 64 nat a bin): the
//                   bins above which every token is kept, and the few that
//                   the thresholds lie in (top-k, top-p)
//   gather_kernel   sums of the kept, a list of the tokens in those few bins
//   resolve_kernel  a workgroup a row: sorts the list, fixes the threshold and
//                   draws
// A row whose list would be too long is resolved by a radix descent over the
// whole row instead: where the threshold lies among too many equal or close
// values (a mask of one finite value too, if top_k counts more than the allowed
// tokens), and for a top_k above the list.  Rows of up to 32768 tokens take one
// launch, small_kernel.
//
// The logits are few bytes (64 rows of 150001 bf16: 19 MB, 4 us): what takes
// time is the chain of dependent steps, each some latencies of memory and LDS
// long, and for large batches the float64 exponentials.  float64 costs as much
// as float32 here; a weight with its units takes about 25 instructions.
#include <type_traits>

#include "common.h"
#include "narrow.h"
#include "serve.h"

namespace moe {
namespace {

constexpr int kThreads = 256;            // of the kernels with a workgroup a chunk
constexpr int kRowThreads = 512;         // of those with a workgroup a row
constexpr int kChunk = 4096;             // tokens
constexpr int kMaxChunks = 64;           // of a row of 2^18 tokens: a lane each
constexpr int kHistThreads = 1024;       // of hist_kernel, which takes kHistChunks chunks
constexpr int kHistChunks = 4;
constexpr double kBinsPerNat = 64.0;
constexpr int kGroups = kChunk / 256;
constexpr int kList = 8192;              // tokens in the bins of the thresholds
constexpr int kBatchChunks = 16384;      // of the rows that are worked on together; bounds the workspace
constexpr double kUnit = 35184372088832.0;         // 2^45
constexpr double kUnitP = 2251799813685248.0;       // 2^51, of probabilities (their sum is 1)

// What a row's filter comes to.
struct RowState {
    double invt, minp;
    float first;      // the largest value
    unsigned key;     // last kept value, as an ordered key
    int last;         // last kept index among values of that key
    int token;        // the draw (-1: no token)
    double sum;       // weights kept, in units
};

// Value of a row's token; NaN becomes -inf, +inf the largest float, -0 +0.  The
// sum makes -0 +0 and a signalling NaN quiet; the median of a NaN and two
// numbers is the smaller number.  (Written out: the compiler folds a clamp by
// comparisons on the ground that no NaN reaches it, and one that tells NaN
// apart takes five instructions.)
__device__ __forceinline__ float clean(float x) {
    float y;
    asm("v_med3_f32 %0, %1, %2, %3" : "=v"(y) : "v"(x + 0.f), "v"(-INFINITY), "s"(3.402823466e38f));
    return y;
}

template <bool F32>
__device__ __forceinline__ float value(const void *row, int i) {
    return clean(F32 ? ((const float *)row)[i] : bf16_to_f32(((const uint16_t *)row)[i]));
}

// Order-preserving key; 0 for -inf, which is never kept.
__device__ __forceinline__ unsigned key_of(float x) {
    const unsigned b = __float_as_uint(x);
    return x == -INFINITY ? 0u : b ^ ((unsigned)((int)b >> 31) | 0x80000000u);
}

__device__ __forceinline__ float of_key(unsigned k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// a * b + c with c in scalar registers (the compiler copies such a constant
// into the result's registers first, which costs as much as the product).
__device__ __forceinline__ double fma_sc(double a, double b, double c) {
    double d;
    asm("v_fma_f64 %0, %1, %2, %3" : "=v"(d) : "v"(a), "v"(b), "s"(c));
    return d;
}

// 2^(t / 128) for t <= 0: 2^(j / 128) from a table in LDS and the exponent, and
// the series of 2^(f / 128), |f| <= 1 / 2, to f^4 (the next term is 1e-15 of
// the result).  j comes out of the low bits of a sum with 1.5 2^52.  Far
// arguments, -inf and NaN give e^-700, which is 0 in every use.
struct ExpTable {
    double t[128];
    __device__ void fill() {  // a barrier follows
        if (threadIdx.x < 128) t[threadIdx.x] = exp2((double)threadIdx.x / 128.0);
    }
    __device__ __forceinline__ double operator()(double x) const {
        constexpr double l = 0.69314718055994530942 / 128.0;
        x = fmax(x, -129262.0);
        const double s = x + 6755399441055744.0;
        const int i = (int)__double_as_longlong(s);
        const double f = x - (s - 6755399441055744.0);
        const double e = fma_sc(f, fma_sc(f, fma_sc(f, l * l * l * l / 24.0 * f + l * l * l / 6.0, l * l / 2.0), l), 1.0) * t[i & 127];
        return __hiloint2double(__double2hiint(e) + ((i & ~127) << 13), __double2loint(e));
    }
};

__device__ __forceinline__ double weight(const ExpTable &et, float x, float first, double invt) {
    return et(((double)x - (double)first) * (invt * (128.0 * 1.4426950408889634074)));
}

// w 2^45 rounded to an integer: the low bits of 2^52 + w 2^45.  Sums are taken
// of the raw bits, and what n of them hold too much is taken off at the end.
__device__ __forceinline__ uint64_t raw_units(double w) {
    return (uint64_t)__double_as_longlong(fma_sc(w, kUnit, 4503599627370496.0));
}
__device__ __forceinline__ uint64_t off_units(int n) { return (uint64_t)n * 0x4330000000000000ull; }
__device__ __forceinline__ uint64_t units(double w) { return raw_units(w) - off_units(1); }

// A kept token's weight, 0 for the others.
__device__ __forceinline__ double kept_weight(const ExpTable &et, const RowState &st, float x, int i) {
    const unsigned k = key_of(x);
    if (k == 0 || k < st.key || (k == st.key && i > st.last)) return 0.0;
    const double w = weight(et, x, st.first, st.invt);
    return w >= st.minp ? w : 0.0;
}

template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u64(uint64_t v) {  // 0 where the source lane is outside the row
    const int lo = __builtin_amdgcn_update_dpp(0, (int)(unsigned)v, CTRL, 0xF, 0xF, false);
    const int hi = __builtin_amdgcn_update_dpp(0, (int)(v >> 32), CTRL, 0xF, 0xF, false);
    return ((uint64_t)(unsigned)hi << 32) | (unsigned)lo;
}

__device__ __forceinline__ uint64_t lane_u64(uint64_t v, int lane) {
    return ((uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
           (unsigned)__builtin_amdgcn_readlane((int)(unsigned)v, lane);
}

// As wave_sum and wave_incl_scan of common.h, for 64 bits.
__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
    v += dpp_u64<0x128>(v);  // row_ror:8, 4, 2, 1
    v += dpp_u64<0x124>(v);
    v += dpp_u64<0x122>(v);
    v += dpp_u64<0x121>(v);
    return lane_u64(v, 0) + lane_u64(v, 16) + lane_u64(v, 32) + lane_u64(v, 48);
}

__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t v) {
    v += dpp_u64<0x111>(v);  // row_shr:1, 2, 4, 8
    v += dpp_u64<0x112>(v);
    v += dpp_u64<0x114>(v);
    v += dpp_u64<0x118>(v);
    const uint64_t r0 = lane_u64(v, 15), r1 = lane_u64(v, 31), r2 = lane_u64(v, 47);
    const int row = (threadIdx.x & 63) >> 4;
    return v + (row > 0 ? r0 : 0) + (row > 1 ? r1 : 0) + (row > 2 ? r2 : 0);
}

// Block of NT threads: the lowest index whose running sum of f(value, i) over
// the row exceeds `want(total)`; -1 if the total is 0.  Each wave owns a
// contiguous part and has 8 loads under way.
template <int NT, bool F32, typename F, typename W>
__device__ int pick(const void *row, int V, F f, W want, uint64_t *sums, int *found, uint64_t *total_out) {
    constexpr int U = 8;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (((V + (NT / 64) - 1) / (NT / 64)) + 63) & ~63;
    const int b = wave * per, e = min(V, b + per);
    auto masses = [&](int i0, uint64_t(&m)[U]) {
        float x[U];
#pragma unroll
        for (int j = 0; j < U; ++j) x[j] = value<F32>(row, min(i0 + 64 * j + lane, V - 1));
        uint64_t all = 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int i = i0 + 64 * j + lane;
            m[j] = i < e ? f(x[j], i) : 0;
            all += m[j];
        }
        return all;
    };
    uint64_t s = 0, m[U];
    for (int i0 = b; i0 < e; i0 += 64 * U) s += masses(i0, m);
    s = wave_sum_u64(s);
    if (lane == 0) sums[wave] = s;
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    uint64_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < (NT / 64); ++w) {
        if (w < wave) before += sums[w];
        total += sums[w];
    }
    *total_out = total;
    if (total) {
        const uint64_t t = want(total);
        if (before <= t && t < before + s) {
            uint64_t run = before;
            for (int i0 = b; i0 < e; i0 += 64 * U) {
                const uint64_t all = wave_sum_u64(masses(i0, m));
                if (run + all <= t) {
                    run += all;
                    continue;
                }
                bool done = false;
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    const uint64_t c = run + wave_scan_u64(m[j]), hit = __ballot(c > t);
                    if (!done && hit) {
                        done = true;
                        if (lane == 0) *found = i0 + 64 * j + __ffsll((unsigned long long)hit) - 1;
                    }
                    run = lane_u64(c, 63);
                }
                break;
            }
        }
    }
    __syncthreads();
    const int r = *found;
    __syncthreads();
    return r;
}

// floor(u * total), below total.
__device__ __forceinline__ uint64_t target(float u, uint64_t total) {
    const double t = u > 0.f ? (double)u * (double)total : 0.0;
    return t < (double)total ? min((uint64_t)t, total - 1) : total - 1;
}

struct Histogram {
    unsigned cnt[2048];
    unsigned long long mass[2048];
    uint64_t wsum[16], wcnt[16];  // a wave each
    // the found bin: what lies above it
    unsigned bin;
    uint64_t above_cnt, above_mass;
};

// Radix descent over the keys from the top: the bin, key after key, in which
// the running count (by_count) or the running weight of the ranking reaches
// `want`.  Leaves the key, and the count and weight strictly above it.  One
// workgroup, six passes or so over the row: tied rows of 32000 tokens take 0.14
// ms in all, of 150001 0.6 (with an atomic a token 0.24 and 1.0).
template <int NT, bool F32>
__device__ void descend(const ExpTable &et, const void *row, int V, float first, double invt, bool by_count, uint64_t want, Histogram &h,
                        unsigned &key, uint64_t &above_cnt, uint64_t &above_mass) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    unsigned prefix = 0;
    above_cnt = above_mass = 0;
#pragma unroll
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        for (int i = tid; i < 2048; i += NT) h.cnt[i] = 0, h.mass[i] = 0;
        __syncthreads();
        // Tied rows have few bins: of a wave's tokens, those of the first one's bin are
        // added together, twice, before the others add their own.
        for (int i0 = 0; i0 < V; i0 += 4 * NT) {
            float x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = value<F32>(row, min(i0 + j * NT + tid, V - 1));
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
                const float v = j == 0 ? x[0] : j == 1 ? x[1] : j == 2 ? x[2] : x[3];
                const unsigned k = key_of(v), b = (k >> shift) & ((1u << bits) - 1);
                bool todo = i0 + j * NT + tid < V && k != 0 && (level == 0 || (k >> (shift + bits)) == prefix);
                if (!__any(todo)) continue;
                const uint64_t m = units(weight(et, v, first, invt));
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const uint64_t left = __ballot(todo);
                    if (!left) break;
                    const int from = __ffsll((unsigned long long)left) - 1;
                    const bool same = todo && b == (unsigned)__builtin_amdgcn_readlane((int)b, from);
                    const uint64_t sum = wave_sum_u64(same ? m : 0);
                    const unsigned n = (unsigned)__popcll(__ballot(same));
                    if (lane == from) {
                        atomicAdd(&h.cnt[b], n);
                        atomicAdd(&h.mass[b], (unsigned long long)sum);
                    }
                    todo = todo && !same;
                }
                if (todo) {
                    atomicAdd(&h.cnt[b], 1u);
                    atomicAdd(&h.mass[b], (unsigned long long)m);
                }
            }
        }
        __syncthreads();
        // thread t owns 4 bins, the first thread the highest
        constexpr int kOwn = 2048 / NT;
        const int b0 = 2047 - kOwn * tid;
        uint64_t cs = 0, ms = 0;
#pragma unroll
        for (int y = 0; y < kOwn; ++y) cs += h.cnt[b0 - y], ms += h.mass[b0 - y];
        uint64_t ca = above_cnt + wave_scan_u64(cs) - cs, ma = above_mass + wave_scan_u64(ms) - ms;
        if (lane == 63) h.wcnt[wave] = ca + cs - above_cnt, h.wsum[wave] = ma + ms - above_mass;
        __syncthreads();
        for (int w = 0; w < wave; ++w) ca += h.wcnt[w], ma += h.wsum[w];
#pragma unroll
        for (int y = 0; y < kOwn; ++y) {
            const uint64_t c = h.cnt[b0 - y], m = h.mass[b0 - y];
            const uint64_t lo = by_count ? ca : ma, hi = lo + (by_count ? c : m);
            if (lo < want && want <= hi) h.bin = b0 - y, h.above_cnt = ca, h.above_mass = ma;
            ca += c;
            ma += m;
        }
        __syncthreads();
        prefix = (prefix << bits) | h.bin;
        above_cnt = h.above_cnt;
        above_mass = h.above_mass;
        __syncthreads();
    }
    key = prefix;
}


// ---------------------------------------------------------------------------
// The row's parameters and the workspace
// ---------------------------------------------------------------------------
struct Filter {
    double invt, minp;
    float topp;
    int topk;
    bool one;  // only the first of the ranking is kept
};

__device__ __forceinline__ Filter filter_of(const SampleArgs &a, int t) {
    const float temp = a.temperature ? a.temperature[t] : 1.f, minp = a.min_p ? a.min_p[t] : 0.f;
    Filter f;
    f.topk = a.top_k ? a.top_k[t] : 0;
    f.topp = a.top_p ? a.top_p[t] : 1.f;
    f.one = !(temp > 0.f) || minp > 1.f || f.topk == 1 || f.topp <= 0.f;
    f.invt = temp > 0.f ? 1.0 / (double)temp : 0.0;
    f.minp = minp > 0.f ? (double)minp : 0.0;
    return f;
}

// Counters of a row: workgroups done, list length.  Zeroed by the first kernel.
struct Header {
    int hist_done, chain_done, listed, pad;
};

// hist_kernel's result: bins below `sure` are kept, tokens up to bin `end`
// with a key of at least `cut` listed.
struct Plan {
    int sure, end, slow;
    unsigned cut;
    uint64_t above_mass, mass;  // of the sure bins, of all
};

// Arrays of one batch of rows, C chunks each.
struct Work {
    RowState *states;  // [T]
    int32_t *drawn;    // [T]
    unsigned *kmax;    // [rows][C] largest key
    int *count;        // [rows][C] tokens with a key
    unsigned *group;   // [rows][C][kGroups] largest keys of 256 tokens each
    uint64_t *sum;     // [rows][C]
    Header *head;      // [rows]
    Plan *plan;        // [rows]
    uint64_t *list;    // [rows][kList] ~key, index
    unsigned *hcnt;    // [rows][H][kBins]
    uint64_t *hmass;   // [rows][H][kBins]
    int row0, C;
    int H;             // histograms of a row
};

template <typename T>
__device__ __forceinline__ void put(T *p, T v) {  // past this XCD's caches, for the row's last workgroup
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get(const T *p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Whether this workgroup is the last of n to come here; everything that the
// others put is complete then (each wave waits for its own stores first).
__device__ __forceinline__ bool last_of(int *done, int n, int *sh) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (threadIdx.x == 0) *sh = __hip_atomic_fetch_add(done, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == n - 1;
    __syncthreads();
    return *sh != 0;
}

// 16 bytes of consecutive tokens a load: 4 float32 or 8 bf16.  Rows begin at
// any element, so the load is unaligned; -inf past the row's end.
template <bool F32>
constexpr int kVec = F32 ? 4 : 8;
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x4 u32x4_any __attribute__((aligned(2)));

template <bool F32>
__device__ __forceinline__ void load_tokens(const void *row, int i, int V, float (&x)[kVec<F32>]) {
    if (i + kVec<F32> <= V) {
        if constexpr (F32) {
            const f32x4 v = *reinterpret_cast<const f32x4_any *>((const float *)row + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = v[e];
        } else {
            const u32x4 v = *reinterpret_cast<const u32x4_any *>((const uint16_t *)row + i);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(e & 1 ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16);
        }
    } else {
#pragma unroll
        for (int e = 0; e < kVec<F32>; ++e)
            x[e] = i + e < V ? (F32 ? ((const float *)row)[i + e] : bf16_to_f32(((const uint16_t *)row)[i + e])) : -INFINITY;
    }
}

template <bool F32>
__device__ __forceinline__ const void *row_of(const SampleArgs &a, int t) {
    return (const char *)a.logits + (size_t)t * a.stride * (F32 ? 4 : 2);
}

// N consecutive tokens by NT threads in rounds of kVec tokens a thread:
// thread tid holds tokens token_at(first, e) .. of round e.
template <int NT, bool F32>
__device__ __forceinline__ int token_at(int first, int e) {
    return first + kVec<F32> * (e * NT + (int)threadIdx.x);
}
template <int NT, bool F32, int N = kChunk>
constexpr int kRounds = N / kVec<F32> / NT;

// All loads of a block are under way together, those of a row's last tokens
// too: one at a time they take most of a kernel's time.
template <int NT, bool F32, int E>
__device__ __forceinline__ void load_block(const SampleArgs &a, int t, int first, float (&x)[E][kVec<F32>]) {
    constexpr int Q = kVec<F32>;
    const void *row = row_of<F32>(a, t);
    if (first + NT * Q * E <= a.V) {
        if constexpr (F32) {
            f32x4 v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = *reinterpret_cast<const f32x4_any *>((const float *)row + token_at<NT, F32>(first, e));
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < Q; ++i) x[e][i] = clean(v[e][i]);
        } else {
            u32x4 v[E];
#pragma unroll
            for (int e = 0; e < E; ++e) v[e] = *reinterpret_cast<const u32x4_any *>((const uint16_t *)row + token_at<NT, F32>(first, e));
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < Q; ++i) x[e][i] = clean(__uint_as_float(i & 1 ? v[e][i >> 1] & 0xffff0000u : v[e][i >> 1] << 16));
        }
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                const int at = min(token_at<NT, F32>(first, e) + i, a.V - 1);
                x[e][i] = F32 ? ((const float *)row)[at] : bf16_to_f32(((const uint16_t *)row)[at]);
            }
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < Q; ++i) x[e][i] = token_at<NT, F32>(first, e) + i < a.V ? clean(x[e][i]) : -INFINITY;
    }
}

__device__ __forceinline__ unsigned wave_max_u32(unsigned v) {
    v = max(v, (unsigned)dpp_ror<8>((int)v));
    v = max(v, (unsigned)dpp_ror<4>((int)v));
    v = max(v, (unsigned)dpp_ror<2>((int)v));
    v = max(v, (unsigned)dpp_ror<1>((int)v));
    const unsigned a = (unsigned)__builtin_amdgcn_readlane((int)v, 0), b = (unsigned)__builtin_amdgcn_readlane((int)v, 16);
    const unsigned c = (unsigned)__builtin_amdgcn_readlane((int)v, 32), d = (unsigned)__builtin_amdgcn_readlane((int)v, 48);
    return max(max(a, b), max(c, d));
}

// Exclusive running sum over a block of NT threads; `total` gets the sum.
// `sh` [NT / 64] is free afterwards.
template <int NT>
__device__ __forceinline__ int block_before(int v, int *sh, int &total) {
    const int incl = wave_incl_scan(v), wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 63) sh[wave] = incl;
    __syncthreads();
    int before = incl - v;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) {
        if (w < wave) before += sh[w];
        total += sh[w];
    }
    __syncthreads();
    return before;
}

// Over a block of NT threads; every thread gets the result, `sh` [NT / 64] is
// free afterwards.
template <int NT>
__device__ __forceinline__ uint64_t block_sum_u64(uint64_t v, uint64_t *sh) {
    v = wave_sum_u64(v);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v += sh[w];
    __syncthreads();
    return v;
}

template <int NT>
__device__ __forceinline__ unsigned block_max_u32(unsigned v, unsigned *sh) {
    v = wave_max_u32(v);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) v = max(v, sh[w]);
    __syncthreads();
    return v;
}

// The first of up to 64 masses, one a lane, whose running sum exceeds `want`,
// which is below their sum; leaves what lies before it in `before`.
__device__ __forceinline__ int lane_of_mass(uint64_t m, uint64_t want, uint64_t &before) {
    const uint64_t incl = wave_scan_u64(m);
    const int l = __ffsll((unsigned long long)__ballot(incl > want)) - 1;
    before = l < 0 ? 0 : (uint64_t)__shfl((unsigned long long)(incl - m), l < 0 ? 0 : l);
    return l;
}

// In chunk c, the lowest token whose running mass f(value, token), in index
// order, exceeds `want`; the last with mass if none does.  A block of NT
// threads, all of which get it.
template <int NT, bool F32, typename F>
__device__ int find_in_chunk(const SampleArgs &a, int t, int c, uint64_t want, F f, uint64_t *sums, int *found) {
    constexpr int E = kRounds<NT, F32>, Q = kVec<F32>, W = NT / 64;
    static_assert(E >= 1 && E * W <= 64, "a part a lane");
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float x[E][Q];
    load_block<NT, F32>(a, t, c * kChunk, x);
    int last = -1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int at = token_at<NT, F32>(c * kChunk, e) + i;
            const uint64_t m = at < a.V ? f(x[e][i], at) : 0;
            if (m) last = at;
            s += m;
        }
        s = wave_sum_u64(s);
        if (lane == 0) sums[e * W + wave] = s;
    }
    if (tid == 0) *found = -1;
    __syncthreads();
    uint64_t run;
    const int part = lane_of_mass(lane < E * W ? sums[lane] : 0, want, run);  // the same in every wave
    if (part < 0) {
        atomicMax(found, last);
    } else if (part % W == wave) {
        float y[Q];
        const int at = token_at<NT, F32>(c * kChunk, part / W);
        load_tokens<F32>(row_of<F32>(a, t), at, a.V, y);
        uint64_t m[Q], s = 0;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            m[i] = at + i < a.V ? f(clean(y[i]), at + i) : 0;
            s += m[i];
        }
        uint64_t b = run + wave_scan_u64(s) - s;
        if (b <= want && want < b + s) {
            int to = -1;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                b += m[i];
                if (to < 0 && want < b) to = at + i;
            }
            *found = to;
        }
    }
    __syncthreads();
    const int r = *found;
    __syncthreads();
    return r;
}

// The probability is computed as probs_kernel does, to the same bits.
__device__ __forceinline__ void finish_row(const ExpTable &et, const RowState &st, RowState *states, int t,
                                           float x, int32_t *token, float *prob) {
    states[t] = st;
    if (token) token[t] = st.token;
    if (prob) prob[t] = st.token < 0 ? 0.f : (float)(kept_weight(et, st, x, st.token) * (kUnit / st.sum));
}

// ---------------------------------------------------------------------------
// Without filters
// ---------------------------------------------------------------------------
// Each chunk's largest value and its sum relative to it.  256 rows of 131072
// float32 logits (134 MB): 34 to 38 us, 3.7 TB/s, of which the exponentials
// are about 20.
template <bool F32>
__global__ __launch_bounds__(kThreads) void part_kernel(SampleArgs a, Work w) {
    constexpr int E = kRounds<kThreads, F32>, Q = kVec<F32>;
    __shared__ ExpTable et;
    __shared__ unsigned sk[kThreads / 64];
    __shared__ uint64_t ss[kThreads / 64];
    const int c = blockIdx.x, t = w.row0 + blockIdx.y;
    float x[E][Q];
    load_block<kThreads, F32>(a, t, c * kChunk, x);
    const Filter f = filter_of(a, t);
    et.fill();
    float v = -INFINITY;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < Q; ++i) v = fmaxf(v, x[e][i]);
    const unsigned k = block_max_u32<kThreads>(key_of(v), sk);
    const float top = of_key(k);
    uint64_t s = 0;
    if (f.one) {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < Q; ++i) s += x[e][i] == top;
    } else {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < Q; ++i) s += raw_units(weight(et, x[e][i], top, f.invt));
        s -= off_units(E * Q);
    }
    s = block_sum_u64<kThreads>(s, ss);
    if (threadIdx.x == 0) {
        w.kmax[blockIdx.y * w.C + c] = k;
        w.sum[blockIdx.y * w.C + c] = s;
        if (c == 0) w.head[blockIdx.y] = Header{0, 0, 0, 0};
    }
}

// The chunks' sums are relative to their own largest values and joined in
// float64 in chunk order, in units of the row's first: off by V 2^-46 of the
// row's sum at most, by what the units drop.  The draw is made inside its chunk
// in those units too; a chunk whose tokens have none of them is passed over, as
// it is with filters.  256 rows: 7.5 us.  (Joining in every workgroup of probs_kernel
// instead takes that from 47 to 71 us: the draw's registers halve its waves.)
template <bool F32>
__global__ __launch_bounds__(kRowThreads) void join_kernel(SampleArgs a, Work w, const float *u, int32_t *token, float *prob) {
    __shared__ ExpTable et;
    __shared__ uint64_t sums[kMaxChunks];
    __shared__ int found;
    const int t = w.row0 + blockIdx.x, lane = threadIdx.x & 63;
    const unsigned kc = lane < w.C ? w.kmax[blockIdx.x * w.C + lane] : 0;
    const uint64_t sc = lane < w.C ? w.sum[blockIdx.x * w.C + lane] : 0;
    const Filter f = filter_of(a, t);
    const float uu = u ? u[t] : 0.f;
    et.fill();
    const unsigned km = wave_max_u32(kc);
    __syncthreads();
    RowState st{f.invt, 0.0, of_key(km), 1u, a.V, -1, 0.0};
    float x = 0.f;
    if (km) {
        // rows that keep one token: only chunks with the largest value count
        const float top = of_key(kc);
        const double wc = weight(et, top, st.first, f.invt);
        const double scale = kc == 0 || (f.one ? kc != km : units(wc) == 0) ? 0.0 : f.one ? 1.0 : wc;
        const double part = (double)sc * scale;
        double incl = part;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        const double total = __shfl(incl, 63);
        const double want = f.one || !(uu > 0.f) ? 0.0 : (double)uu * total;
        uint64_t hit = __ballot(part > 0.0 && incl > want);
        const uint64_t some = __ballot(part > 0.0);
        // a number past the last step takes the last token with weight
        const int c = hit ? __ffsll((unsigned long long)hit) - 1 : 63 - __clzll((long long)some);
        const double inside = want - __shfl(incl - part, c);
        st.token = find_in_chunk<kRowThreads, F32>(
            a, t, c, inside > 0.0 ? (uint64_t)inside : 0,
            [&](float v, int) {
                const uint64_t m = units(weight(et, v, st.first, f.invt));
                return f.one ? (uint64_t)(v == st.first) : m;
            },
            sums, &found);
        st.sum = f.one ? kUnit : total;
        if (f.one) st.key = km, st.last = st.token;
        x = value<F32>(row_of<F32>(a, t), st.token);
    }
    if (threadIdx.x == 0) finish_row(et, st, w.states, t, x, token, prob);
}

// ---------------------------------------------------------------------------
// With filters
// ---------------------------------------------------------------------------
// Largest keys of the chunk and of its groups (16 lanes each), and for rows
// with top_p alone the sum of its weights relative to its largest value.  64
// rows of 150001 bf16 logits (19 MB): 7.7 us.
template <bool F32>
__global__ __launch_bounds__(kThreads) void max_kernel(SampleArgs a, Work w) {
    constexpr int E = kRounds<kThreads, F32>, Q = kVec<F32>;
    static_assert(E * Q * 16 == 256, "a group of 256 tokens");
    __shared__ ExpTable et;
    __shared__ unsigned sk[kThreads / 64];
    __shared__ uint64_t sn[kThreads / 64];
    const int c = blockIdx.x, t = w.row0 + blockIdx.y, tid = threadIdx.x;
    float x[E][Q];
    load_block<kThreads, F32>(a, t, c * kChunk, x);
    const Filter f = filter_of(a, t);
    const bool sums = f.topp < 1.f && !f.one && !(f.topk > 0 && f.topk < a.V);
    if (sums) et.fill();
    float v = -INFINITY;
    int n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            v = fmaxf(v, x[e][i]);
            n += x[e][i] != -INFINITY;
        }
    v = fmaxf(v, dpp_ror<8>(v));
    v = fmaxf(v, dpp_ror<4>(v));
    v = fmaxf(v, dpp_ror<2>(v));
    v = fmaxf(v, dpp_ror<1>(v));
    const int at = blockIdx.y * w.C + c;
    if ((tid & 15) == 0) w.group[at * kGroups + (tid >> 4)] = key_of(v);
    const unsigned k = block_max_u32<kThreads>(key_of(v), sk);
    uint64_t all = block_sum_u64<kThreads>((uint64_t)n, sn);
    if (tid == 0) {
        w.kmax[at] = k;
        w.count[at] = (int)all;
        if (c == 0) w.head[blockIdx.y] = Header{0, 0, 0, 0};
    }
    if (sums) {
        const float top = of_key(k);
        uint64_t s = 0;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < Q; ++i) s += raw_units(weight(et, x[e][i], top, f.invt));
        s -= off_units(E * Q);
        s = block_sum_u64<kThreads>(s, sn);
        if (tid == 0) w.sum[at] = s;
    }
}

// Which thresholds a row has: the first k of the ranking, or a share of the
// sum (of those k, or of the row).
struct Kind {
    unsigned km;
    int k;
    bool by_k, by_p;
};

__device__ __forceinline__ Kind kind_from(const Filter &f, unsigned km, int n, int V) {
    Kind k;
    k.km = km;
    k.k = min(f.topk, n);
    k.by_k = !f.one && f.topk > 0 && f.topk < V && km;
    k.by_p = !f.one && f.topp < 1.f && km;
    return k;
}

__device__ __forceinline__ Kind kind_of(const Filter &f, const Work &w, int row, int V) {
    const int lane = threadIdx.x & 63;
    const unsigned km = lane < w.C ? w.kmax[row * w.C + lane] : 0u;
    const int n = lane < w.C ? w.count[row * w.C + lane] : 0;
    return kind_from(f, wave_max_u32(km), wave_sum_int(n), V);
}

__device__ __forceinline__ float bin_scale(double invt) { return (float)fmin(invt * kBinsPerNat, 1e30); }

// Which tokens can be left out of the search for a threshold.
//   top_p: tokens of weight below (1 - top_p) / V of the row's sum hold less
//   than 1 - top_p of it together, so the threshold lies above them (half of
//   that here, for the roundings).  Returns the distance in nats.
__device__ __forceinline__ double cut_distance(const Filter &f, double mass, int V) {
    return log(2.0 * V * kUnit / ((1.0 - (double)f.topp) * mass));
}

__device__ __forceinline__ unsigned cut_key(float first, double invt, double nats) {
    const double x = (double)first - nats / invt * 1.000001;  // invt = 0: every token weighs the same
    return invt > 0.0 && x > -3.4e38 ? key_of(clean((float)x)) : 1u;
}

//   top_k: the k-th largest of any set of tokens, one of each of some groups,
//   is no larger than the k-th largest of all.  The largest key with at least
//   k of the block's keys (one a thread, NT threads) at or above it, found two
//   bits at a time from the top; the low bits are left 0.  `sh` [2 NT / 64].
template <int NT>
__device__ unsigned key_of_rank(unsigned key, int k, uint64_t *sh) {
    constexpr int W = NT / 64;
    unsigned cut = 0;
#pragma unroll 1
    for (int bit = 30; bit >= 14; bit -= 2) {
        uint64_t n = 0;  // three counts of up to 2^11
#pragma unroll
        for (int y = 3; y >= 1; --y) n = (n << 20) | (unsigned)__popcll(__ballot(key >= (cut | ((unsigned)y << bit))));
        uint64_t *to = sh + ((bit >> 1) & 1) * W;
        if ((threadIdx.x & 63) == 0) to[threadIdx.x >> 6] = n;
        __syncthreads();
        n = 0;
#pragma unroll
        for (int i = 0; i < W; ++i) n += to[i];
        unsigned y = 0;
#pragma unroll
        for (int i = 0; i < 3; ++i) y += (int)((n >> (20 * i)) & 0xFFFFF) >= k;
        cut |= y << bit;
    }
    __syncthreads();
    return max(cut, 1u);
}

// The bins' shared memory; where a row's histogram is searched, 1024 threads
// of a block own two bins each.
struct Bins {
    unsigned cnt[kBins];
    unsigned long long mass[kBins];
    uint64_t wsum[16];
    Plan plan;
};

__device__ __forceinline__ void clear_bins(Bins &h, int nt, bool by_k) {
    for (int b = threadIdx.x; b < kBins; b += nt)
        if (by_k)
            h.cnt[b] = 0;
        else
            h.mass[b] = 0;
}

// Tokens below `cut` are left out, and so is the last bin; a threshold in them
// is seen by its absence.  The weights of the last bin are below 2^-45 / 2 and
// have no units, so a top-p threshold never lies there.
__device__ __forceinline__ void count_token(Bins &h, const Kind &kind, float x, unsigned cut, float first, float scale,
                                            double invt, const ExpTable &et) {
    const int b = bin_of(x, first, scale);
    if (b == kBins - 1 || key_of(x) < cut) return;
    if (kind.by_k)
        atomicAdd(&h.cnt[b], 1u);
    else
        atomicAdd(&h.mass[b], (unsigned long long)units(weight(et, x, first, invt)));
}

// The plan of a whole row's histogram, by 1024 threads; the block gets it in
// h.plan.  `mass`: the row's sum, for top_p alone; `cut`: the least key
// counted; `cap`: of the list.
__device__ void plan_row(Bins &h, const Filter &f, const Kind &kind, uint64_t mass, unsigned cut, int cap) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const uint64_t v0 = kind.by_k ? h.cnt[2 * tid] : h.mass[2 * tid], v1 = kind.by_k ? h.cnt[2 * tid + 1] : h.mass[2 * tid + 1];
    uint64_t run = wave_scan_u64(v0 + v1) - v0 - v1;
    if (lane == 63) h.wsum[wave] = run + v0 + v1;
    if (tid == 0) h.plan = Plan{0, kBins - 1, 1, 1u, 0, mass};  // not among the counted
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < wave) run += h.wsum[i];
    const uint64_t want = kind.by_k ? (uint64_t)kind.k : max((uint64_t)1, (uint64_t)ceil((double)f.topp * (double)mass));
#pragma unroll
    for (int y = 0; y < 2; ++y) {
        const uint64_t v = y ? v1 : v0;
        if (run < want && want <= run + v) {
            Plan p;
            p.sure = kind.by_k ? 0 : 2 * tid + y;  // by_k: the sum of the first top_k comes from the list
            p.end = 2 * tid + y;
            p.slow = kind.by_k && run + v > (uint64_t)cap;
            p.cut = cut;
            p.above_mass = kind.by_k ? 0 : run;
            p.mass = mass;
            h.plan = p;
        }
        run += v;
    }
    __syncthreads();
}

// The row's sum from its chunks' (relative to their own largest values), in
// units of the first's weight; above the sum of all units by V 2^-46 of it at
// most, by what the units drop.
__device__ __forceinline__ double row_mass(const ExpTable &et, const Work &w, int row, const Filter &f, unsigned km) {
    const int lane = threadIdx.x & 63;
    const unsigned kc = lane < w.C ? w.kmax[row * w.C + lane] : 0;
    double v = kc ? (double)w.sum[row * w.C + lane] * weight(et, of_key(kc), of_key(km), f.invt) : 0.0;
#pragma unroll
    for (int d = 32; d; d >>= 1) v += __shfl_xor(v, d);
    return v;
}

// The row's plan.  A top_k that the groups' largest keys settle takes 8 to 10
// us (64 rows; through the histogram 19), the histogram of top_p 15.6 (20 rows of
// 150001 float32 logits: 6 us to this workgroup's histogram, the rest until
// the last one has joined them).
template <bool F32>
__global__ __launch_bounds__(kHistThreads) void hist_kernel(SampleArgs a, Work w) {
    constexpr int E = kRounds<kHistThreads, F32, kHistChunks * kChunk>, Q = kVec<F32>;
    __shared__ ExpTable et;
    __shared__ Bins h;
    __shared__ int sh;
    __shared__ uint64_t ranks[2 * kHistThreads / 64];
    static_assert(kHistThreads == 1024 && kBins == 2048 && kMaxChunks * kGroups <= kHistThreads, "two bins, a group a thread");
    const int hc = blockIdx.x, row = blockIdx.y, t = w.row0 + row, tid = threadIdx.x;
    const unsigned group = hc == 0 && tid < w.C * kGroups ? w.group[row * w.C * kGroups + tid] : 0;
    const Filter f = filter_of(a, t);
    // a small top_k against the groups: no histogram.  At 7 / 8 of the groups
    // about 2 tokens a group lie above the cut.
    const bool ranked = f.topk > 0 && f.topk < a.V && f.topk <= w.C * kGroups * 7 / 8 && f.topk <= kList / 4;
    float x[E][Q];
    if (!ranked) load_block<kHistThreads, F32>(a, t, hc * kHistChunks * kChunk, x);
    const Kind kind = kind_of(f, w, row, a.V);
    if (!kind.by_k && !kind.by_p) return;  // the whole row's workgroups
    if (ranked) {
        if (hc) return;
        const unsigned cut = key_of_rank<kHistThreads>(group, kind.k, ranks);
        if (tid == 0) w.plan[row] = Plan{0, kBins - 1, 0, cut, 0, 0};
        return;
    }
    if (!kind.by_k) et.fill();
    clear_bins(h, kHistThreads, kind.by_k);
    __syncthreads();
    const float first = of_key(kind.km), scale = bin_scale(f.invt);
    const uint64_t mass = kind.by_k ? 0 : (uint64_t)row_mass(et, w, row, f, kind.km);
    const unsigned cut = kind.by_k ? 1u : cut_key(first, f.invt, cut_distance(f, (double)mass, a.V));
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < Q; ++i)
            if (x[e][i] != -INFINITY) count_token(h, kind, x[e][i], cut, first, scale, f.invt, et);
    __syncthreads();
    if (w.H > 1) {
        // bins past that of the least key counted are empty in all of them
        const int bins = cut > 1u ? bin_of(of_key(cut), first, scale) + 1 : kBins;
        const size_t at = (size_t)row * w.H * kBins;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int b = y * kHistThreads + tid;
            if (b >= bins) continue;
            if (kind.by_k)
                put(w.hcnt + at + hc * kBins + b, h.cnt[b]);
            else
                put(w.hmass + at + hc * kBins + b, (uint64_t)h.mass[b]);
        }
        if (!last_of(&w.head[row].hist_done, w.H, &sh)) return;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const int b = y * kHistThreads + tid;
            if (b >= bins) continue;
            if (kind.by_k) {
                unsigned n = 0;
#pragma unroll 8
                for (int i = 0; i < w.H; ++i) n += get(w.hcnt + at + i * kBins + b);
                h.cnt[b] = n;
            } else {
                uint64_t m = 0;
#pragma unroll 8
                for (int i = 0; i < w.H; ++i) m += get(w.hmass + at + i * kBins + b);
                h.mass[b] = m;
            }
        }
        __syncthreads();
    }
    plan_row(h, f, kind, mass, cut, kList);
    if (tid == 0) w.plan[row] = h.plan;
}

// List entries sort as the ranking does.
__device__ __forceinline__ unsigned entry_key(uint64_t e) { return ~(unsigned)(e >> 32); }
__device__ __forceinline__ uint64_t entry_of(float x, int i) { return ((uint64_t)~key_of(x) << 32) | (unsigned)i; }

// The list, and the sums of what is kept for sure.  Reads the logits again,
// from the caches: 64 rows of 150001 bf16 in 9 to 11 us.
template <bool F32>
__global__ __launch_bounds__(kThreads) void gather_kernel(SampleArgs a, Work w) {
    constexpr int E = kRounds<kThreads, F32>, Q = kVec<F32>;
    __shared__ ExpTable et;
    __shared__ uint64_t sums[kThreads / 64];
    __shared__ int sh;
    const int c = blockIdx.x, row = blockIdx.y, t = w.row0 + row, tid = threadIdx.x;
    // all loads before the first wait: none needs another's result
    Plan p = w.plan[row];
    const Filter f = filter_of(a, t);
    float x[E][Q];
    load_block<kThreads, F32>(a, t, c * kChunk, x);
    const Kind kind = kind_of(f, w, row, a.V);
    const bool planned = kind.by_k || kind.by_p;
    if (!planned) p = Plan{kBins, -1, 0, 1u, 0, 0};
    if (p.slow) return;
    et.fill();
    if (tid == 0) sh = f.one ? INT_MAX : 0;
    __syncthreads();
    const float first = of_key(kind.km), scale = bin_scale(f.invt);
    uint64_t sum = 0;
    if (f.one) {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < Q; ++i)
                if (kind.km && key_of(x[e][i]) == kind.km) atomicMin(&sh, token_at<kThreads, F32>(c * kChunk, e) + i);
        __syncthreads();
        sum = (uint64_t)sh;
    } else {
        // tokens below the cut are neither kept nor listed
        const float low = planned && p.cut > 1u ? of_key(p.cut) : -3.402823466e38f;
        float v = -INFINITY;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < Q; ++i) v = fmaxf(v, x[e][i]);
        int mine = 0;
        unsigned in = 0;  // which of the thread's tokens go to the list
        if (v >= low) {
#pragma unroll
            for (int e = 0; e < E; ++e)
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    if (!(x[e][i] >= low)) continue;
                    const int b = planned ? bin_of(x[e][i], first, scale) : 0;
                    if (b < p.sure) {
                        const double wt = weight(et, x[e][i], first, f.invt);
                        if (wt >= f.minp) sum += units(wt);
                    } else if (b <= p.end) {
                        ++mine;
                        in |= 1u << (Q * e + i);
                    }
                }
        }
        if (p.sure) sum = block_sum_u64<kThreads>(sum, sums);
        if (planned) {
            int at = 0;
            if (mine) at = atomicAdd(&sh, mine);
            __syncthreads();
            if (tid == 0 && sh) sh = __hip_atomic_fetch_add(&w.head[row].listed, sh, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (mine) {
                at += sh;
#pragma unroll
                for (int e = 0; e < E; ++e)
#pragma unroll
                    for (int i = 0; i < Q; ++i)
                        if ((in >> (Q * e + i)) & 1 && at < kList)
                            w.list[(size_t)row * kList + at++] =
                                entry_of(x[e][i], token_at<kThreads, F32>(c * kChunk, e) + i);
            }
        }
    }
    if (tid == 0) w.sum[row * w.C + c] = sum;
}

// The row's filter by radix descent, by one workgroup.
template <int NT, bool F32>
__device__ void descend_row(const ExpTable &et, const SampleArgs &a, const void *row, const Filter &f, const Kind &kind,
                            RowState &st, Histogram &h, uint64_t *sums, int *found) {
    uint64_t ca, ma, wk = 0, ties = 0;
    if (kind.by_k) {
        descend<NT, F32>(et, row, a.V, st.first, st.invt, true, (uint64_t)kind.k, h, st.key, ca, ma);
        ties = (uint64_t)kind.k - ca;
        wk = ma + ties * units(weight(et, of_key(st.key), st.first, st.invt));
    } else {
        pick<NT, F32>(
            row, a.V, [&](float x, int) { return x == -INFINITY ? (uint64_t)0 : units(weight(et, x, st.first, st.invt)); },
            [](uint64_t total) { return total; }, sums, found, &wk);
    }
    if (kind.by_p) {
        const uint64_t want = min(max((uint64_t)1, (uint64_t)ceil((double)f.topp * (double)wk)), wk);
        descend<NT, F32>(et, row, a.V, st.first, st.invt, false, want, h, st.key, ca, ma);
        const uint64_t w = units(weight(et, of_key(st.key), st.first, st.invt));
        ties = (want - ma + w - 1) / w;
    }
    uint64_t total;
    st.last = pick<NT, F32>(
        row, a.V, [&](float x, int) { return (uint64_t)(key_of(x) == st.key); },
        [&](uint64_t n) { return min(ties, n) - 1; }, sums, found, &total);
}

typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));

// Bitonic sort of `size` (a power of two >= 64) list entries by NT threads,
// ascending: key descending, index ascending.  Strides up to 64 stay inside
// the 128 entries of a wave and need no barrier of the block.
// Up to 512 entries (all different) are put in the place that the number of
// smaller ones gives, two or four threads counting for each, or two for two
// (250 entries: 2.5 us, where the sort takes 8; a call with 300 of them, 512
// threads: 43.4 against 46.7, with 1000, 1024 threads: 32.6 against 23.6); the
// rest keep ~0.
template <int NT>
__device__ void sort_list(uint64_t *list, int n, int size) {
    if (n <= (NT < 512 ? NT : 512)) {
        const int log = n <= NT / 4 ? 2 : 1;
        const int i0 = threadIdx.x >> log, i1 = i0 + NT / 2, part = threadIdx.x & ((1 << log) - 1);
        const int each = ((n + 7) >> 3) << (3 - log);  // 8 | size
        uint64_t mine0 = 0, mine1 = 0;
        int rank0 = 0, rank1 = 0;
        if (i0 < n) mine0 = list[i0];
        if (i1 < n) mine1 = list[i1];
        const u64x2 *from = reinterpret_cast<const u64x2 *>(list + part * each), *end = from + each / 2;
        if (n <= NT / 2) {
            if (i0 < n)
#pragma unroll 2
                for (; from != end; ++from) {
                    const u64x2 v = *from;
                    rank0 += (v[0] < mine0) + (v[1] < mine0);
                }
        } else {
#pragma unroll 2
            for (; from != end; ++from) {
                const u64x2 v = *from;
                rank0 += (v[0] < mine0) + (v[1] < mine0);
                rank1 += (v[0] < mine1) + (v[1] < mine1);
            }
        }
        auto others = [&](int rank) {
            rank += __builtin_amdgcn_update_dpp(0, rank, 0xB1, 0xF, 0xF, false);  // quad_perm 1, 0, 3, 2
            if (log == 2) rank += __builtin_amdgcn_update_dpp(0, rank, 0x4E, 0xF, 0xF, false);  // quad_perm 2, 3, 0, 1
            return rank;
        };
        rank0 = others(rank0);
        rank1 = others(rank1);
        __syncthreads();
        if (i0 < n && part == 0) list[rank0] = mine0;
        if (i1 < n && part == 0 && log == 1) list[rank1] = mine1;
        __syncthreads();
        return;
    }
    for (int k = 2; k <= size; k <<= 1)
        for (int j = k >> 1; j > 0; j >>= 1) {
            if (j > 64 || (j == 64 && k > 128)) __syncthreads();
            for (int i = threadIdx.x; i < size / 2; i += NT) {
                const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
                const uint64_t x0 = list[lo], x1 = list[hi];
                if ((x0 > x1) == ((lo & k) == 0)) list[lo] = x1, list[hi] = x0;
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
    __syncthreads();
}

template <int CAP>
struct ListShared {
    uint64_t list[CAP];
    unsigned long long sub[1024];
    uint64_t ws[16];
    unsigned klo[16], khi[16];
    int n, kept;
};

// The threshold of a row from its list of n entries (in s.list, unsorted):
// sets st.key and st.last and calls add(index, units) for every kept entry.
// A list for top_p alone is first narrowed to those of 1024 equal parts of its
// key range that the threshold lies in.  False if the threshold is not in the
// list (the sums above it and in it say so).
template <int NT, int CAP, typename Add>
__device__ bool resolve_list(ListShared<CAP> &s, int n, const Filter &f, const Kind &kind, const Plan &p, const ExpTable &et,
                             RowState &st, Add add) {
    constexpr int W = NT / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    auto weight_of = [&](uint64_t e) { return weight(et, of_key(entry_key(e)), st.first, f.invt); };
    auto keep = [&](uint64_t e) {
        const double w = weight_of(e);
        if (w >= st.minp) add((int)(unsigned)e, units(w));
    };
    uint64_t above = p.above_mass;
    const double share = (double)f.topp;
    uint64_t want = max((uint64_t)1, (uint64_t)ceil(share * (double)p.mass));  // by_p alone
    if (!kind.by_k && n > 256) {
        unsigned lo = ~0u, hi = 0;
        for (int i = tid; i < n; i += NT) {
            const unsigned k = entry_key(s.list[i]);
            lo = min(lo, k);
            hi = max(hi, k);
        }
        for (int i = tid; i < 1024; i += NT) s.sub[i] = 0;
        if (tid == 0) s.kept = -1;
        hi = wave_max_u32(hi);
        lo = ~wave_max_u32(~lo);
        if (lane == 0) s.klo[wave] = lo, s.khi[wave] = hi;
        if (tid == 0) s.n = 0;
        __syncthreads();
        for (int i = 0; i < W; ++i) lo = min(lo, s.klo[i]), hi = max(hi, s.khi[i]);
        // parts from the top; a key's part never falls while the key does
        const float part = 1023.f / fmaxf((float)(hi - lo), 1.f);
        auto part_of = [&](uint64_t e) { return min((int)((float)(hi - entry_key(e)) * part), 1023); };
        for (int i = tid; i < n; i += NT) atomicAdd(&s.sub[part_of(s.list[i])], (unsigned long long)units(weight_of(s.list[i])));
        __syncthreads();
        constexpr int B = 1024 / NT;
        uint64_t m = 0;
#pragma unroll
        for (int y = 0; y < B; ++y) m += s.sub[B * tid + y];
        uint64_t run = above + wave_scan_u64(m) - m;
        if (lane == 63) s.ws[wave] = run + m - above;
        __syncthreads();
        for (int i = 0; i < wave; ++i) run += s.ws[i];
#pragma unroll
        for (int y = 0; y < B; ++y) {
            const uint64_t v = s.sub[B * tid + y];
            if (run < want && want <= run + v) s.kept = B * tid + y, s.ws[W - 1] = run;  // the waves before are read
            run += v;
        }
        __syncthreads();
        const int at = s.kept;
        if (at < 0) return false;
        above = s.ws[W - 1];
        // entries above are kept, those of the part go on
        uint64_t mine[CAP / NT];
#pragma unroll
        for (int y = 0; y < CAP / NT; ++y) mine[y] = y * NT + tid < n ? s.list[y * NT + tid] : ~0ull;
        __syncthreads();
#pragma unroll
        for (int y = 0; y < CAP / NT; ++y)
            if (y * NT + tid < n) {
                const int b = part_of(mine[y]);
                if (b < at) keep(mine[y]);
                if (b == at) s.list[atomicAdd(&s.n, 1)] = mine[y];
            }
        __syncthreads();
        n = s.n;
    }
    int size = 64;
    while (size < n) size <<= 1;
    for (int i = n + tid; i < size; i += NT) s.list[i] = ~0ull;
    __syncthreads();
    sort_list<NT>(s.list, n, size);
    // running weights of the list: thread tid holds `per` of them
    const int per = (size + NT - 1) / NT, b = tid * per;
    const int nk = kind.by_k ? min(kind.k, n) : n, e = min(b + per, nk);
    if (tid == 0) s.kept = kind.by_p ? 0 : nk;
    if (kind.by_p) {
        uint64_t mine = 0;
        for (int i = b; i < e; ++i) mine += units(weight_of(s.list[i]));
        uint64_t incl = wave_scan_u64(mine), wk = 0;
        if (lane == 63) s.ws[wave] = incl;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if (i < wave) incl += s.ws[i];
            wk += s.ws[i];
        }
        if (kind.by_k) want = max((uint64_t)1, (uint64_t)ceil(share * (double)wk));
        uint64_t run = above + incl - mine;
        if (run < want && want <= run + mine)
            for (int i = b; i < e; ++i) {
                run += units(weight_of(s.list[i]));
                if (run >= want) {
                    s.kept = i + 1;
                    break;
                }
            }
    }
    __syncthreads();
    const int kept = s.kept;
    if (kept == 0) return false;
    st.key = entry_key(s.list[kept - 1]);
    st.last = (int)(unsigned)s.list[kept - 1];
    for (int i = b; i < e && i < kept; ++i) keep(s.list[i]);
    __syncthreads();
    return true;
}

union DrawShared {
    ListShared<kList> l;
    Histogram h;
};

// Threshold and draw of a row.  64 rows with lists of 250 tokens: 11 us, of
// which the list's order takes 2.5 to 4 and the token in its chunk 3.5.
template <bool F32>
__global__ __launch_bounds__(kRowThreads) void resolve_kernel(SampleArgs a, Work w, const float *u, int32_t *token, float *prob) {
    __shared__ ExpTable et;
    __shared__ DrawShared s;
    __shared__ uint64_t sums[kMaxChunks];
    __shared__ unsigned long long cs[kMaxChunks];
    __shared__ int found;
    const int row = blockIdx.x, t = w.row0 + row, tid = threadIdx.x, lane = tid & 63;
    // everything that does not wait for anything else first
    const uint64_t mine = tid < w.C ? w.sum[row * w.C + tid] : 0;
    const uint64_t head = w.list[(size_t)row * kList + tid];  // most lists end in it; not read past their length
    int n = w.head[row].listed;
    Plan p = w.plan[row];
    const float uu = u ? u[t] : 0.f;
    const Filter f = filter_of(a, t);
    const Kind kind = kind_of(f, w, row, a.V);
    const bool planned = kind.by_k || kind.by_p;
    if (!planned) p = Plan{kBins, -1, 0, 1u, 0, 0};
    if (planned && n > kList) p.slow = 1;  // tied rows: the cut let too many through
    et.fill();
    if (tid < kMaxChunks) cs[tid] = p.slow ? 0 : mine;
    RowState st{f.invt, f.one ? 0.0 : f.minp, of_key(kind.km), 1u, a.V, -1, 0.0};
    float x = 0.f;
    const void *r = row_of<F32>(a, t);
    __syncthreads();
    if (kind.km == 0) {
        // no token
    } else if (f.one) {
        int lo = lane < w.C ? (int)cs[lane] : INT_MAX;
#pragma unroll
        for (int d = 32; d; d >>= 1) lo = min(lo, __shfl_xor(lo, d));
        st.key = kind.km;
        st.last = st.token = lo;
        st.sum = kUnit;
    } else {
        bool slow = p.slow;
        if (planned && !slow) {
            if (tid < n) s.l.list[tid] = head;
            for (int i = kRowThreads + tid; i < n; i += kRowThreads) s.l.list[i] = w.list[(size_t)row * kList + i];
            __syncthreads();
            slow = !resolve_list<kRowThreads>(s.l, n, f, kind, p, et, st,
                                              [&](int i, uint64_t m) { atomicAdd(&cs[i / kChunk], (unsigned long long)m); });
        }
        uint64_t total;
        if (slow) {
            descend_row<kRowThreads, F32>(et, a, r, f, kind, st, s.h, sums, &found);
            st.token = pick<kRowThreads, F32>(
                r, a.V, [&](float x, int i) { return units(kept_weight(et, st, x, i)); },
                [&](uint64_t total) { return target(uu, total); }, sums, &found, &total);
        } else {
            const uint64_t mc = cs[lane];
            total = wave_sum_u64(mc);
            const uint64_t want = target(uu, total);
            uint64_t before;
            const int c = lane_of_mass(mc, want, before);
            st.token = find_in_chunk<kRowThreads, F32>(
                a, t, c, want - before, [&](float v, int i) { return units(kept_weight(et, st, v, i)); }, sums, &found);
        }
        st.sum = (double)total;
    }
    if (st.token >= 0) x = value<F32>(r, st.token);
    if (tid == 0) finish_row(et, st, w.states, t, x, token, prob);
}

// ---------------------------------------------------------------------------
// Rows of up to 32768 tokens: the row in the shared memory of one workgroup,
// all of the above in one launch.  There a launch and a pass over the caches
// cost more than the arithmetic of one compute unit.  A row of 32000 float32
// logits with top_p takes 21 us where few tokens come near the threshold
// (loads 1.5, largest 2, the sum 6, list 4, order and draw 6) and 33 where the
// row is flat (narrowing 7, the sum above the list 9 more); with the kernels
// above, 33 and 39.  The float64 exponentials bound it, 100 cycles of a SIMD
// for 64 of them.  A call of 30 allowed tokens among 32000 with top_k 50 takes 20
// us, of 64 rows whose top_p 0.99 lies in a long tail 35; rows that go through
// the descent take 95 (top_k) to 140 (top_p).
// ---------------------------------------------------------------------------
constexpr int kSmallThreads = 1024;
constexpr int kSmallRound = 4 * kSmallThreads;  // tokens
constexpr int kSmall = 8 * kSmallRound;
constexpr int kSmallList = 2048;

union SmallShared {
    unsigned b[kParts];
    ListShared<kSmallList> l;
    Histogram h;
};

template <bool F32>
__global__ __launch_bounds__(kSmallThreads) void small_kernel(SampleArgs a, RowState *states, Header *head, const float *u,
                                                              int32_t *token, float *prob) {
    constexpr int NT = kSmallThreads, W = NT / 64;
    extern __shared__ __attribute__((aligned(16))) float tokens[];  // whole rounds, -inf past the end
    __shared__ ExpTable et;
    __shared__ SmallShared s;
    __shared__ uint64_t sums[8 * W], masses[W];
    __shared__ unsigned sk[W];
    __shared__ int sn[W], ranks[2], found;
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const void *r = row_of<F32>(a, t);
    const int E = (a.V + kSmallRound - 1) / kSmallRound;  // rounds of 4 tokens a thread
    f32x4 *own = reinterpret_cast<f32x4 *>(tokens) + tid;  // round e at own[e * NT]
    float v = -INFINITY;  // this thread's largest
    int nv = 0;
    const Filter f = filter_of(a, t);
    const float uu = u ? u[t] : 0.f;
    constexpr int Q = kVec<F32>, B = kSmall / Q / NT;
    if (a.V >= Q) {
        // every load is whole and under way at once; the last one, moved into the row,
        // writes some of its neighbour's tokens again
        typedef typename std::conditional<F32, f32x4_any, u32x4_any>::type Raw;
        constexpr int size = F32 ? 4 : 2;
        typename std::conditional<F32, f32x4, u32x4>::type raw[B];
#pragma unroll
        for (int y = 0; y < B; ++y)
            raw[y] = *reinterpret_cast<const Raw *>((const char *)r + size * min(Q * (y * NT + tid), a.V - Q));
        et.fill();
#pragma unroll
        for (int y = 0; y < B; ++y) {
            const int i = Q * (y * NT + tid);
            float x[Q];
#pragma unroll
            for (int e = 0; e < Q; ++e) {
                if constexpr (F32)
                    x[e] = clean(raw[y][e]);
                else
                    x[e] = clean(__uint_as_float(e & 1 ? raw[y][e >> 1] & 0xffff0000u : raw[y][e >> 1] << 16));
            }
            if (i + Q <= a.V) {
#pragma unroll
                for (int e = 0; e < Q; e += 4)
                    *reinterpret_cast<f32x4 *>(tokens + i + e) = f32x4{x[e], x[e + 1], x[e + 2], x[e + 3]};
            } else if (i < E * kSmallRound) {
#pragma unroll
                for (int e = 0; e < Q; ++e) {
                    if (i < a.V) tokens[a.V - Q + e] = x[e];
                    if (i + e >= a.V) tokens[i + e] = -INFINITY;
                }
            }
        }
    } else {
        et.fill();
        for (int i = tid; i < kSmallRound; i += NT) tokens[i] = i < a.V ? value<F32>(r, i) : -INFINITY;
    }
    __syncthreads();
#pragma unroll 1
    for (int e = 0; e < E; ++e) {
        const f32x4 x = own[e * NT];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v = fmaxf(v, x[i]);
            nv += x[i] != -INFINITY;
        }
    }
    nv = wave_sum_int(nv);
    if (lane == 0) sn[wave] = nv;
    const unsigned mykey = key_of(v), km = block_max_u32<NT>(mykey, sk);
    nv = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) nv += sn[i];
    const Kind kind = kind_from(f, km, nv, a.V);
    RowState st{f.invt, f.one ? 0.0 : f.minp, of_key(km), 1u, a.V, -1, 0.0};
    if (km && f.one) {
        if (tid == 0) found = INT_MAX;
        __syncthreads();
        if (mykey == km)
            for (int e = E - 1; e >= 0; --e)
                for (int i = 3; i >= 0; --i)
                    if (own[e * NT][i] == st.first) atomicMin(&found, 4 * (e * NT + tid) + i);
        __syncthreads();
        st.key = km;
        st.last = st.token = found;
        st.sum = kUnit;
    } else if (km) {
        bool summed = false;
        if (kind.by_k || kind.by_p) {
            // tokens above `top` are kept, those from `low` to `top` listed
            Plan p{0, kBins - 1, 0, 1u, 0, 0};
            float low = -3.402823466e38f, top = INFINITY;
            double want = (double)kind.k;
            if (kind.by_k) {
                // Longer lists than a thread an entry take longer to sort than a descent over
                // one round of tokens (3000 tokens, top_k 1500: 29.3 us against 25.0).
                if (kind.k > (E > 1 ? kSmallList : NT)) {
                    low = INFINITY;
                } else {
                    // a thread's tokens are a group: the k-th of their largest, or for a large k the
                    // least of them, which must have the first k above it
                    unsigned cut = kind.k <= NT * 7 / 8 ? key_of_rank<NT>(mykey, kind.k, sums) : ~block_max_u32<NT>(~mykey, sk);
                    if (cut <= 1u) {  // too few groups hold a token: from the row's least on
                        float least = INFINITY;
#pragma unroll 1
                        for (int e = 0; e < E; ++e) {
                            const f32x4 x = own[e * NT];
#pragma unroll
                            for (int i = 0; i < 4; ++i) least = fminf(least, x[i] == -INFINITY ? INFINITY : x[i]);
                        }
                        cut = ~block_max_u32<NT>(~key_of(least), sk);
                    }
                    low = of_key(cut);
                }
            } else {
                uint64_t m = 0;
#pragma unroll 1
                for (int e = 0; e < E; ++e) {
                    const f32x4 x = own[e * NT];
#pragma unroll
                    for (int i = 0; i < 4; ++i) m += raw_units(weight(et, x[i], st.first, f.invt));
                }
                p.mass = block_sum_u64<NT>(m - off_units(4 * E), masses);
                want = (double)f.topp * (double)p.mass;
                const unsigned cut = cut_key(st.first, f.invt, cut_distance(f, (double)p.mass, a.V));
                if (cut > 1u) low = of_key(cut);
            }
            // Narrowing, where too many are left: a histogram of 2048 equal parts of
            // [low, first], by the count or by float32 weights (narrow.h).  The list
            // is widened by those sums' error, and the sum above it taken again in units.
            int n, before = 0;
            auto count = [&]() {  // of the list: this thread's place in it, and its length
                int mine = 0;
                if (v >= low)
#pragma unroll 2
                    for (int e = 0; e < E; ++e) {
                        const f32x4 x = own[e * NT];
#pragma unroll
                        for (int i = 0; i < 4; ++i) mine += x[i] >= low && x[i] <= top;
                    }
                before = block_before<NT>(mine, sn, n);
            };
            count();
            if (n > kSmallList && can_narrow(low, st.first)) {
                const float part = parts_per_unit(low, st.first);
                const float scale = (float)fmin(f.invt * 1.4426950408889634, 1e30);
                const double per_unit = kind.by_k ? 1.0 : kNarrowMass / (double)p.mass;
                const float unit = (float)(per_unit * kUnit);
                for (int i = tid; i < kParts; i += NT) s.b[i] = 0;
                __syncthreads();
                if (v >= low)
#pragma unroll 1
                    for (int e = 0; e < E; ++e) {
                        const f32x4 x = own[e * NT];
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (x[i] >= low)
                                atomicAdd(&s.b[part_at(st.first, x[i], part)],
                                          kind.by_k ? 1u : narrow_mass(unit, __builtin_amdgcn_exp2f((x[i] - st.first) * scale)));
                    }
                __syncthreads();
                // parts from the first down, two a thread
                const unsigned b0 = s.b[2 * tid], b1 = s.b[2 * tid + 1];
                int incl = wave_incl_scan((int)(b0 + b1));
                if (lane == 63) sn[wave] = incl;
                if (tid == 0) ranks[0] = kParts - 1, ranks[1] = -1;  // none above, the end not found
                __syncthreads();
                for (int i = 0; i < wave; ++i) incl += sn[i];
                const unsigned after = (unsigned)incl, mid = after - b1;
                const float goal = (float)(want * per_unit), slack = kind.by_k ? 0.f : narrow_slack(n);
                // the list begins after the last part that surely lies above, and ends with the first that
                // surely holds it; sums do not fall, so one thread finds each (atomics of all to one word take 6 us)
                const float ahead = (float)(after - b0 - b1), lo = goal - slack, hi = goal + slack;
                if (ahead < lo && lo <= (float)after) ranks[1] = 2 * tid - ((float)mid >= lo);
                if (ahead < hi && hi <= (float)after) ranks[0] = 2 * tid + ((float)mid < hi);
                __syncthreads();
                const float width = (st.first - low) / (kParts - 0.1f);
                const int end = ranks[0], begin = ranks[1];
                // a little beyond the parts' edges, which are rounded differently; a token on the rounded
                // `top` itself goes to the list
                if (end < kParts - 1) low = fmaxf(low, st.first - width * ((float)end + 1.01f));
                if (!kind.by_k && begin >= 0) top = st.first - width * ((float)begin + 0.99f);
                __syncthreads();
                count();
            }
            // what is kept above the list: by parts, for the draw, and in whole
            for (int i = tid; i < E * W; i += NT) sums[i] = 0;
            __syncthreads();
            if (top < INFINITY) {
                uint64_t all = 0;
#pragma unroll 1
                for (int e = 0; e < E; ++e) {
                    const f32x4 x = own[e * NT];
                    const bool some = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])) > top;
                    if (!__any(some)) continue;
                    uint64_t m = 0, kept = 0;
                    if (some)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const double w = weight(et, x[i], st.first, f.invt);
                            const uint64_t q = x[i] > top ? units(w) : 0;
                            m += q;
                            kept += w >= st.minp ? q : 0;
                        }
                    all += m;
                    kept = wave_sum_u64(kept);
                    if (lane == 0) sums[e * W + wave] = kept;
                }
                p.above_mass = block_sum_u64<NT>(all, masses);
            }
            if (v >= low && n <= kSmallList)
#pragma unroll 2
                for (int e = 0; e < E; ++e) {
                    const f32x4 x = own[e * NT];
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (x[i] >= low && x[i] <= top) s.l.list[before++] = entry_of(x[i], 4 * (e * NT + tid) + i);
                }
            __syncthreads();
            // Too many equal or close values at the threshold, or a first k beyond the
            // list; and a narrowing that the exact sums do not bear out.
            const uint64_t least = max((uint64_t)1, (uint64_t)ceil((double)f.topp * (double)p.mass));
            bool slow = n > kSmallList || (kind.by_k ? n < kind.k : p.above_mass >= least);
            if (!slow)
                slow = !resolve_list<NT>(s.l, n, f, kind, p, et, st,
                                         [&](int i, uint64_t m) { atomicAdd((unsigned long long *)&sums[i / 256], (unsigned long long)m); });
            if (slow) descend_row<NT, F32>(et, a, r, f, kind, st, s.h, masses, &found);
            summed = !slow;
        }
        // the draw: masses of the kept in index order, a part of 256 tokens a wave and round
        const float keep = st.key > 1u ? of_key(st.key) : -3.402823466e38f;
        if (!summed)
#pragma unroll 1
            for (int e = 0; e < E; ++e) {
                const f32x4 x = own[e * NT];
                uint64_t m = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const double w = weight(et, x[i], st.first, st.invt);
                    const bool kept = w >= st.minp && (x[i] > keep || (x[i] == keep && 4 * (e * NT + tid) + i <= st.last));
                    m += kept ? units(w) : 0;
                }
                m = wave_sum_u64(m);
                if (lane == 0) sums[e * W + wave] = m;
            }
        __syncthreads();
        const uint64_t p0 = 2 * lane < E * W ? sums[2 * lane] : 0, p1 = 2 * lane < E * W ? sums[2 * lane + 1] : 0;
        const uint64_t total = wave_sum_u64(p0 + p1), pick_at = target(uu, total);
        uint64_t run;
        int part = 2 * lane_of_mass(p0 + p1, pick_at, run);
        if (pick_at >= run + sums[part]) run += sums[part++];
        if (part % W == wave) {
            const int e = part / W, at = 4 * (e * NT + tid);
            const f32x4 x = own[e * NT];
            uint64_t m[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m[i] = units(kept_weight(et, st, x[i], at + i));
            const uint64_t ms = m[0] + m[1] + m[2] + m[3], b0 = run + wave_scan_u64(ms) - ms;
            if (b0 <= pick_at && pick_at < b0 + ms) {
                const uint64_t b1 = b0 + m[0], b2 = b1 + m[1], b3 = b2 + m[2];
                found = at + (pick_at < b1 ? 0 : pick_at < b2 ? 1 : pick_at < b3 ? 2 : 3);
            }
        }
        __syncthreads();
        st.token = found;
        st.sum = (double)total;
    }
    if (tid == 0) {
        head[t] = Header{0, 0, 0, 0};
        finish_row(et, st, states, t, st.token >= 0 ? tokens[st.token] : 0.f, token, prob);
    }
}

// ---------------------------------------------------------------------------
// The whole distribution of a row
// ---------------------------------------------------------------------------
// 256 rows of 131072 float32 logits (134 MB in, out of the caches in part, 134
// MB out): 45 to 48 us, 5.7 TB/s: memory.
template <bool F32>
__global__ __launch_bounds__(kThreads) void probs_kernel(SampleArgs a, Work w, float *probs) {
    constexpr int E = kRounds<kThreads, F32>, Q = kVec<F32>;
    __shared__ ExpTable et;
    const int c = blockIdx.x, t = w.row0 + blockIdx.y;
    float x[E][Q];
    load_block<kThreads, F32>(a, t, c * kChunk, x);
    const RowState st = w.states[t];
    et.fill();
    __syncthreads();
    const double k = st.sum > 0.0 ? kUnit / st.sum : 0.0;
    float *out = probs + (size_t)t * a.V;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int at = token_at<kThreads, F32>(c * kChunk, e);
        float v[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) v[i] = (float)(kept_weight(et, st, x[e][i], at + i) * k);
        if (at + Q <= a.V) {
#pragma unroll
            for (int i = 0; i < Q; i += 4) *reinterpret_cast<f32x4_any *>(out + at + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
        } else {
#pragma unroll
            for (int i = 0; i < Q; ++i)
                if (at + i < a.V) out[at + i] = v[i];
        }
    }
}

// ---------------------------------------------------------------------------
// Acceptance
// ---------------------------------------------------------------------------
// Drafts matched against the target's own draws: thread t finds whether row t
// is hit and enters itself with its parent, where the first row wins; then a
// thread a sequence follows the hits.  (Searching the children of each row on
// the way instead takes 4.5 us where this takes 3.1.)
__global__ __launch_bounds__(64) void match_kernel(AcceptArgs c, const int32_t *drawn) {
    __shared__ int32_t drew[kMaxTokens], hit[kMaxTokens];
    const int s = threadIdx.x, T = c.off[c.nseq];
    static_assert(kMaxTokens == 64 && kMaxSegments <= 64, "a thread each");
    int tok = 0, parent = -1;
    if (s < T) tok = c.tokens[s], drew[s] = drawn[s], parent = c.parent[s];
    hit[s] = INT_MAX;
    __syncthreads();
    if (parent >= 0 && tok >= 0 && tok == drew[parent]) atomicMin(&hit[parent], s);
    __syncthreads();
    if (s >= c.nseq) return;
    const int r0 = c.off[s], n = c.off[s + 1] - r0;
    int k = 0;
    for (int cur = n ? r0 : INT_MAX; cur != INT_MAX; cur = hit[cur]) {
        c.path[r0 + k] = cur - r0;
        c.out[r0 + k] = drew[cur];
        ++k;
    }
    c.count[s] = k;
    for (int j = k; j < n; ++j) c.path[r0 + j] = c.out[r0 + j] = -1;
}

// Chains against the drafter's distributions.  Every workgroup of a sequence
// finds the row of the last token (thread j tests draft j + 1), sums its
// chunk of max(p - q, 0) there, or of p, and the last one draws.  4 sequences
// of 5 rows of 150001 float32: 13 us, the latency of tests, row, sums and draw.
template <bool F32>
__global__ __launch_bounds__(kRowThreads) void chain_kernel(SampleArgs a, AcceptArgs c, Work w) {
    constexpr int E = kRounds<kRowThreads, F32>, Q = kVec<F32>;
    __shared__ ExpTable et;
    __shared__ uint64_t sums[kMaxChunks];
    __shared__ int sh, found, row_sh;
    const int ch = blockIdx.x, s = blockIdx.y, r0 = c.off[s], n = c.off[s + 1] - r0, tid = threadIdx.x, lane = tid & 63;
    if (n == 0) {
        if (ch == 0 && tid == 0) c.count[s] = 0;
        return;
    }
    et.fill();
    __syncthreads();
    auto p_of = [&](const RowState &st, double k, float x, int i) { return kept_weight(et, st, x, i) * k; };
    if (tid < 64) {  // n <= 64
        bool stop = true;
        if (tid + 1 < n) {
            const int t = r0 + tid, x = c.tokens[t + 1];
            const RowState st = w.states[t];
            if (x >= 0 && x < a.V && st.sum > 0.0) {
                const double p = p_of(st, kUnit / st.sum, value<F32>(row_of<F32>(a, t), x), x);
                const double qx = (double)c.q[(size_t)t * a.V + x];
                stop = !((double)c.u[t] * (qx < 0.0 ? 0.0 : qx) < p);  // NaN stops
            }
        }
        const uint64_t first = __ballot(stop);  // the last row always stops
        if (tid == 0) row_sh = __ffsll((unsigned long long)first) - 1;
    }
    __syncthreads();
    const int j = row_sh, t = r0 + j;
    const bool rest = j + 1 < n;
    const RowState st = w.states[t];
    const double scale = st.sum > 0.0 ? kUnit / st.sum : 0.0;
    const float *q = c.q + (size_t)t * a.V;
    // q is not below 0, so that the sum is p's at most, whatever q holds
    auto mass = [&](float x, int i) {
        const double v = fmax(p_of(st, scale, x, i) - (rest ? fmax((double)q[i], 0.0) : 0.0), 0.0);
        return (uint64_t)__double_as_longlong(fma(v, kUnitP, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
    };
    float x[E][Q];
    load_block<kRowThreads, F32>(a, t, ch * kChunk, x);
    uint64_t sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < Q; ++i) {
            const int at = token_at<kRowThreads, F32>(ch * kChunk, e) + i;
            if (at < a.V) sum += mass(x[e][i], at);
        }
    sum = block_sum_u64<kRowThreads>(sum, sums);
    if (tid == 0) put(w.sum + r0 * w.C + ch, sum);
    if (!last_of(&w.head[r0].chain_done, w.C, &sh)) return;
    const uint64_t mc = lane < w.C ? get(w.sum + r0 * w.C + lane) : 0, total = wave_sum_u64(mc);
    const float u = c.u_final[s];
    int tok;
    if (total) {
        const uint64_t want = target(u, total);
        uint64_t before;
        const int k = lane_of_mass(mc, want, before);
        tok = find_in_chunk<kRowThreads, F32>(a, t, k, want - before, mass, sums, &found);
    } else {  // nothing of p lies above q
        const void *row = row_of<F32>(a, t);
        uint64_t all;
        tok = pick<kRowThreads, F32>(
            row, a.V, [&](float x, int i) { return units(kept_weight(et, st, x, i)); },
            [&](uint64_t all) { return target(u, all); }, sums, &found, &all);
    }
    for (int i = tid; i < n; i += kRowThreads) {
        c.path[r0 + i] = i <= j ? i : -1;
        c.out[r0 + i] = i < j ? c.tokens[r0 + i + 1] : i == j ? tok : -1;
    }
    if (tid == 0) c.count[s] = j + 1;
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------
size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Layout {
    int C, H, rows;  // as in Work; rows of a batch
    size_t states, drawn, kmax, count, group, sum, head, plan, list, hcnt, hmass, total;
};

Layout layout(int T, int V) {
    const bool small = V <= kSmall;  // one launch for all rows, and only the sums of acceptance
    Layout l{};
    l.C = (V + kChunk - 1) / kChunk;
    l.H = (l.C + kHistChunks - 1) / kHistChunks;
    l.rows = small || T < kBatchChunks / l.C ? T : kBatchChunks / l.C;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    l.states = take((size_t)T * sizeof(RowState));
    l.drawn = take((size_t)T * 4);
    l.sum = take((size_t)l.rows * l.C * 8);
    l.head = take((size_t)l.rows * sizeof(Header));
    const size_t n = small ? 0 : l.rows;
    l.kmax = take(n * l.C * 4);
    l.count = take(n * l.C * 4);
    l.group = take(n * l.C * kGroups * 4);
    l.plan = take(n * sizeof(Plan));
    l.list = take(n * kList * 8);
    l.hcnt = take(n * l.H * kBins * 4);
    l.hmass = take(n * l.H * kBins * 8);
    l.total = off;
    return l;
}

Work work_of(const SampleArgs &a, const Layout &l) {
    char *p = static_cast<char *>(a.ws);
    Work w;
    w.states = reinterpret_cast<RowState *>(p + l.states);
    w.drawn = reinterpret_cast<int32_t *>(p + l.drawn);
    w.kmax = reinterpret_cast<unsigned *>(p + l.kmax);
    w.count = reinterpret_cast<int *>(p + l.count);
    w.group = reinterpret_cast<unsigned *>(p + l.group);
    w.sum = reinterpret_cast<uint64_t *>(p + l.sum);
    w.head = reinterpret_cast<Header *>(p + l.head);
    w.plan = reinterpret_cast<Plan *>(p + l.plan);
    w.list = reinterpret_cast<uint64_t *>(p + l.list);
    w.hcnt = reinterpret_cast<unsigned *>(p + l.hcnt);
    w.hmass = reinterpret_cast<uint64_t *>(p + l.hmass);
    w.row0 = 0;
    w.C = l.C;
    w.H = l.H;
    return w;
}

// States, and draws with u, of all rows.
template <bool F32>
hipError_t rows(const SampleArgs &a, Work w, const Layout &l, const float *u, int32_t *token, float *prob, float *probs,
                hipStream_t s) {
    const dim3 block(kThreads);
    const bool small = a.V <= kSmall;
    if (small) {
        const int lds = (a.V + kSmallRound - 1) / kSmallRound * kSmallRound * 4;
        hipError_t e = allow_lds<small_kernel<F32>>(kSmall * 4);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((small_kernel<F32>), dim3(a.T), dim3(kSmallThreads), lds, s, a, w.states, w.head, u, token, prob);
        if ((e = hipGetLastError()) != hipSuccess) return e;
    }
    for (; w.row0 < a.T; w.row0 += l.rows) {
        const int n = a.T - w.row0 < l.rows ? a.T - w.row0 : l.rows;
        const dim3 grid(l.C, n);
        if (small) {
            // drawn above
        } else if (!a.top_k && !a.top_p && !a.min_p) {
            hipLaunchKernelGGL((part_kernel<F32>), grid, block, 0, s, a, w);
            hipLaunchKernelGGL((join_kernel<F32>), dim3(n), dim3(kRowThreads), 0, s, a, w, u, token, prob);
        } else {
            hipLaunchKernelGGL((max_kernel<F32>), grid, block, 0, s, a, w);
            if (a.top_k || a.top_p) hipLaunchKernelGGL((hist_kernel<F32>), dim3(l.H, n), dim3(kHistThreads), 0, s, a, w);
            hipLaunchKernelGGL((gather_kernel<F32>), grid, block, 0, s, a, w);
            hipLaunchKernelGGL((resolve_kernel<F32>), dim3(n), dim3(kRowThreads), 0, s, a, w, u, token, prob);
        }
        if (probs) hipLaunchKernelGGL((probs_kernel<F32>), grid, block, 0, s, a, w, probs);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <bool F32>
hipError_t accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t s) {
    const Layout l = layout(a.T, a.V);
    const Work w = work_of(a, l);
    hipError_t e = rows<F32>(a, w, l, c.q ? nullptr : c.u, c.q ? nullptr : w.drawn, nullptr, nullptr, s);
    if (e != hipSuccess) return e;
    if (c.q)
        hipLaunchKernelGGL((chain_kernel<F32>), dim3(l.C, c.nseq), dim3(kRowThreads), 0, s, a, c, w);
    else
        hipLaunchKernelGGL(match_kernel, dim3(1), dim3(64), 0, s, c, w.drawn);
    return hipGetLastError();
}

}  // namespace

size_t sample_ws_bytes(int T, int V) { return layout(T > 0 ? T : 1, V).total; }

hipError_t launch_sample(const SampleArgs &a, const float *u, int32_t *token, float *prob, float *probs, hipStream_t s) {
    const Layout l = layout(a.T, a.V);
    const Work w = work_of(a, l);
    return a.f32 ? rows<true>(a, w, l, u, token, prob, probs, s) : rows<false>(a, w, l, u, token, prob, probs, s);
}

hipError_t launch_accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t s) {
    return a.f32 ? accept<true>(a, c, s) : accept<false>(a, c, s);
}

}  // namespace moe
