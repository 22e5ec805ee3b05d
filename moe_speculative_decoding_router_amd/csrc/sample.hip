// Drawing and accepting draft tokens.  The filtered distribution of a row of
// logits is defined in include/moe_verify.h.
//
// Every filter keeps a prefix of the row's ranking (value desc, index asc),
// so a row's filter is one threshold: the last kept value and, among equal
// values, the last kept index.  Weights w = exp(-(first - l) / temperature)
// are computed in float64 and summed as integers in units of 2^-45: a sum
// does not depend on its order, and 2^18 weights of at most 1 fit 63 bits.
//
// A row is cut into chunks of consecutive tokens, a workgroup each.  Without
// filters two launches draw: part_kernel (each chunk's largest value and its
// sum relative to it, one pass over the logits) and join_kernel (a workgroup
// a row: the chunk that holds the draw, then the token).  With filters:
//   max_kernel   the row's largest value
//   hist_kernel  a histogram of the distance from it (1 / 32 nat a bin): the
//                bins above which every token is kept, and the few that the
//                thresholds lie in (top-k, top-p rows only)
//   draw_kernel  sums of the kept, a list of the tokens in those few bins;
//                the row's last workgroup sorts the list, fixes the threshold
//                and draws
// A row whose list would be too long (flat or tied rows, large top-k with
// distant tails) is resolved by a radix descent over the whole row instead.
#include "common.h"
#include "serve.h"

namespace moe {
namespace {

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr int kTile = 4 * kRowThreads;  // tokens that a workgroup loads at once, 4 a thread
constexpr int kMaxChunks = 64;          // of a row (2^18 tokens in tiles)
constexpr int kBins = 1024;             // the last holds all that lies beyond
constexpr int kList = 8192;             // tokens in the bins of the thresholds
constexpr double kUnit = 35184372088832.0;         // 2^45
constexpr double kUnitP = 1152921504606846976.0;   // 2^60, of probabilities (their sum is 1)

// What a row's filter comes to.
struct RowState {
    double invt, minp;
    float first;      // the largest value
    unsigned key;     // last kept value, as an ordered key
    int last;         // last kept index among values of that key
    int token;        // the draw (-1: no token)
    double sum;       // weights kept, in units
};

// Value of a row's token; NaN becomes -inf, +inf the largest float, -0 +0.
__device__ __forceinline__ float clean(float x) {
    x = x != x ? -INFINITY : fminf(x, 3.402823466e38f);
    return x == 0.f ? 0.f : x;
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

// exp for arguments <= 0: 2^(j / 64) from a table of 64 in LDS, e^r of the
// rest |r| <= ln 2 / 128 by its series to r^5 (the next term is 3e-17).
struct ExpTable {
    double t[64];
    __device__ void fill() {  // by the first wave; a barrier follows
        if (threadIdx.x < 64) t[threadIdx.x] = exp2((double)threadIdx.x / 64.0);
    }
    __device__ __forceinline__ double operator()(double d) const {
        const double j = rint(d * (64.0 * 1.4426950408889634074));
        const double r = fma(j, -0.69314718055994530942 / 64.0, d);
        const double e = fma(r, fma(r, fma(r, fma(r, fma(r, 1.0 / 120.0, 1.0 / 24.0), 1.0 / 6.0), 0.5), 1.0), 1.0);
        const int i = (int)j;  // saturates; far arguments give 0
        return ldexp(e * t[i & 63], i >> 6);
    }
};

__device__ __forceinline__ double weight(const ExpTable &et, float x, float first, double invt) {
    return et(((double)x - (double)first) * invt);
}

// w 2^45 rounded to an integer: the low bits of 2^52 + w 2^45.
__device__ __forceinline__ uint64_t units(double w) {
    return (uint64_t)__double_as_longlong(fma(w, kUnit, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;
}

// A kept token's weight, 0 for the others.
__device__ __forceinline__ double kept_weight(const ExpTable &et, const RowState &st, float x, int i) {
    const unsigned k = key_of(x);
    if (k == 0 || k < st.key || (k == st.key && i > st.last)) return 0.0;
    const double w = weight(et, x, st.first, st.invt);
    return w >= st.minp ? w : 0.0;
}

__device__ __forceinline__ uint64_t wave_sum_u64(uint64_t v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v += (uint64_t)__shfl_xor((unsigned long long)v, d);
    return v;
}

__device__ __forceinline__ uint64_t wave_scan_u64(uint64_t v) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const uint64_t o = (uint64_t)__shfl_up((unsigned long long)v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Block of kRowThreads: the lowest index whose running sum of f(i) exceeds
// `want(total)`; -1 if the total is 0.  Each wave owns a contiguous part.
template <typename F, typename W>
__device__ int pick(int V, F f, W want, uint64_t *sums, int *found, uint64_t *total_out) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int per = (((V + kRowWaves - 1) / kRowWaves) + 63) & ~63;
    const int b = wave * per, e = min(V, b + per);
    uint64_t s = 0;
    for (int i = b + lane; i < e; i += 64) s += f(i);
    s = wave_sum_u64(s);
    if (lane == 0) sums[wave] = s;
    if (threadIdx.x == 0) *found = -1;
    __syncthreads();
    uint64_t total = 0, before = 0;
    for (int w = 0; w < kRowWaves; ++w) {
        if (w < wave) before += sums[w];
        total += sums[w];
    }
    *total_out = total;
    if (total) {
        const uint64_t t = want(total);
        if (before <= t && t < before + s) {
            uint64_t run = before;
            for (int i0 = b; i0 < e; i0 += 64) {
                const int i = i0 + lane;
                const uint64_t c = run + wave_scan_u64(i < e ? f(i) : 0);
                const uint64_t hit = __ballot(c > t);
                if (hit) {
                    if (lane == 0) *found = i0 + __ffsll((unsigned long long)hit) - 1;
                    break;
                }
                run = (uint64_t)__shfl((unsigned long long)c, 63);
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
    uint64_t wsum[kRowWaves], wcnt[kRowWaves];
    // the found bin: what lies above it
    unsigned bin;
    uint64_t above_cnt, above_mass;
};

// Radix descent over the keys from the top: the bin, key after key, in which
// the running count (by_count) or the running weight of the ranking reaches
// `want`.  Leaves the key, and the count and weight strictly above it.
template <bool F32>
__device__ void descend(const ExpTable &et, const void *row, int V, float first, double invt, bool by_count, uint64_t want, Histogram &h,
                        unsigned &key, uint64_t &above_cnt, uint64_t &above_mass) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    unsigned prefix = 0;
    above_cnt = above_mass = 0;
#pragma unroll
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        for (int i = tid; i < 2048; i += kRowThreads) h.cnt[i] = 0, h.mass[i] = 0;
        __syncthreads();
        for (int i = tid; i < V; i += kRowThreads) {
            const float x = value<F32>(row, i);
            const unsigned k = key_of(x);
            if (k == 0 || (level && (k >> (shift + bits)) != prefix)) continue;
            const unsigned b = (k >> shift) & ((1u << bits) - 1);
            atomicAdd(&h.cnt[b], 1u);
            atomicAdd(&h.mass[b], (unsigned long long)units(weight(et, x, first, invt)));
        }
        __syncthreads();
        // thread t owns bins 2047 - 2t and 2046 - 2t, from the top
        const int b0 = 2047 - 2 * tid;
        const uint64_t c0 = h.cnt[b0], c1 = h.cnt[b0 - 1], m0 = h.mass[b0], m1 = h.mass[b0 - 1];
        uint64_t ci = wave_scan_u64(c0 + c1), mi = wave_scan_u64(m0 + m1);
        if (lane == 63) h.wcnt[wave] = ci, h.wsum[wave] = mi;
        __syncthreads();
        for (int w = 0; w < wave; ++w) ci += h.wcnt[w], mi += h.wsum[w];
        uint64_t ca = above_cnt + ci - c0 - c1, ma = above_mass + mi - m0 - m1;
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            const uint64_t c = y ? c1 : c0, m = y ? m1 : m0;
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
    int hist_done, draw_done, chain_done, listed;
};

// hist_kernel's result: bins below `sure` are kept, those up to `end` listed.
struct Plan {
    int sure, end, slow, pad;
    uint64_t above_cnt, above_mass, mass;  // of the sure bins, of all
};

// Arrays of one batch of rows, C chunks each.
struct Work {
    RowState *states;  // [T]
    int32_t *drawn;    // [T]
    unsigned *kmax;    // [rows][C] largest key
    int *count;        // [rows][C] tokens with a key
    uint64_t *sum;     // [rows][C]
    Header *head;      // [rows]
    Plan *plan;        // [rows]
    uint64_t *list;    // [rows][kList] ~key, index
    unsigned *hcnt;    // [rows][C][kBins]
    uint64_t *hmass;   // [rows][C][kBins]
    int row0, C;
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

// 4 consecutive values from token i of a row on; -inf past its end.  Rows
// begin at any element, so the load is unaligned.
typedef f32x4 f32x4_any __attribute__((aligned(4)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));

template <bool F32>
__device__ __forceinline__ void load4(const void *row, int i, int V, float (&x)[4]) {
    if (i + 4 <= V) {
        if (F32) {
            const f32x4 v = *reinterpret_cast<const f32x4_any *>((const float *)row + i);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = clean(v[e]);
        } else {
            const u32x2 v = *reinterpret_cast<const u32x2_any *>((const uint16_t *)row + i);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[e] = clean(__uint_as_float(e & 1 ? v[e >> 1] & 0xffff0000u : v[e >> 1] << 16));
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = i + e < V ? value<F32>(row, i + e) : -INFINITY;
    }
}

template <bool F32>
__device__ __forceinline__ const void *row_of(const SampleArgs &a, int t) {
    return (const char *)a.logits + (size_t)t * a.stride * (F32 ? 4 : 2);
}

// The chunk's values; thread tid holds tokens 4 tid .. 4 tid + 3 of each tile.
template <int E, bool F32>
__device__ __forceinline__ void load_chunk(const SampleArgs &a, int t, int c, float (&x)[E][4]) {
    const void *row = row_of<F32>(a, t);
#pragma unroll
    for (int e = 0; e < E; ++e) load4<F32>(row, (c * E + e) * kTile + 4 * threadIdx.x, a.V, x[e]);
}

__device__ __forceinline__ unsigned wave_max_u32(unsigned v) {
#pragma unroll
    for (int d = 32; d; d >>= 1) v = max(v, (unsigned)__shfl_xor((int)v, d));
    return v;
}

// Sum over the block; every thread gets it.  `sh` [kRowWaves] is free afterwards.
__device__ __forceinline__ uint64_t block_sum_u64(uint64_t v, uint64_t *sh) {
    v = wave_sum_u64(v);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) v += sh[w];
    __syncthreads();
    return v;
}

__device__ __forceinline__ unsigned block_max_u32(unsigned v, unsigned *sh) {
    v = wave_max_u32(v);
    if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRowWaves; ++w) v = max(v, sh[w]);
    __syncthreads();
    return v;
}

// Largest key of the row from its chunks' (any thread; C <= 64).
__device__ __forceinline__ unsigned row_key(const unsigned *kmax, int C) {
    const int lane = threadIdx.x & 63;
    return wave_max_u32(lane < C ? kmax[lane] : 0u);
}

// In chunk c, the lowest token whose running mass f(value, token), in index
// order, exceeds `want`; the last with mass if none does.  All threads get it.
template <int E, bool F32, typename F>
__device__ int find_in_chunk(const SampleArgs &a, int t, int c, uint64_t want, F f, uint64_t *sums, int *found) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    float x[E][4];
    load_chunk<E, F32>(a, t, c, x);
    uint64_t m[E][4];
    int last = -1;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        uint64_t s = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (c * E + e) * kTile + 4 * tid + i;
            m[e][i] = at < a.V ? f(x[e][i], at) : 0;
            if (m[e][i]) last = at;
            s += m[e][i];
        }
        s = wave_sum_u64(s);
        if (lane == 0) sums[e * kRowWaves + wave] = s;
    }
    if (tid == 0) *found = -1;
    __syncthreads();
    uint64_t run = 0;
    int part = -1;
    for (int p = 0; p < E * kRowWaves; ++p) {  // the same in every thread
        if (run + sums[p] > want) {
            part = p;
            break;
        }
        run += sums[p];
    }
    if (part < 0) {
        atomicMax(found, last);
    } else if ((part & (kRowWaves - 1)) == wave) {
#pragma unroll
        for (int e = 0; e < E; ++e)
            if (e == part / kRowWaves) {
                const uint64_t s = m[e][0] + m[e][1] + m[e][2] + m[e][3], incl = wave_scan_u64(s);
                uint64_t b = run + incl - s;
                if (b <= want && want < b + s) {
                    int i = 0;
                    while (b + m[e][i] <= want) b += m[e][i++];
                    *found = (c * E + e) * kTile + 4 * tid + i;
                }
            }
    }
    __syncthreads();
    const int r = *found;
    __syncthreads();
    return r;
}

// ---------------------------------------------------------------------------
// Without filters
// ---------------------------------------------------------------------------
template <int E, bool F32>
__global__ __launch_bounds__(kRowThreads) void part_kernel(SampleArgs a, Work w) {
    __shared__ ExpTable et;
    __shared__ unsigned sk[kRowWaves];
    __shared__ uint64_t ss[kRowWaves];
    const int c = blockIdx.x, t = w.row0 + blockIdx.y;
    const Filter f = filter_of(a, t);
    float x[E][4];
    load_chunk<E, F32>(a, t, c, x);
    et.fill();
    unsigned k = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) k = max(k, key_of(x[e][i]));
    k = block_max_u32(k, sk);
    const float top = of_key(k);
    uint64_t s = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (x[e][i] != -INFINITY) s += f.one ? (uint64_t)(x[e][i] == top) : units(weight(et, x[e][i], top, f.invt));
    s = block_sum_u64(s, ss);
    if (threadIdx.x == 0) {
        w.kmax[blockIdx.y * w.C + c] = k;
        w.sum[blockIdx.y * w.C + c] = s;
        if (c == 0) w.head[blockIdx.y] = Header{0, 0, 0, 0};
    }
}

// A workgroup a row.  The chunks' sums are relative to their own largest
// values and joined in float64 in chunk order; the draw is made inside its
// chunk in that chunk's units.
template <int E, bool F32>
__global__ __launch_bounds__(kRowThreads) void join_kernel(SampleArgs a, Work w, const float *u, int32_t *token,
                                                           float *prob) {
    __shared__ ExpTable et;
    __shared__ uint64_t sums[E * kRowWaves];
    __shared__ double part[kMaxChunks];
    __shared__ int found;
    const int t = w.row0 + blockIdx.x, tid = threadIdx.x;
    const Filter f = filter_of(a, t);
    const unsigned *kmax = w.kmax + blockIdx.x * w.C;
    et.fill();
    const unsigned km = row_key(kmax, w.C);
    __syncthreads();
    RowState st{f.invt, 0.0, of_key(km), 1u, a.V, -1, 0.0};
    if (tid < w.C) {
        const unsigned k = kmax[tid];
        // rows that keep one token: only the chunks with the largest value count
        part[tid] = k == 0 || (f.one && k != km) ? 0.0 : (double)w.sum[blockIdx.x * w.C + tid] * weight(et, of_key(k), st.first, f.invt);
    }
    __syncthreads();
    int c = 0, lastc = 0;
    double total = 0.0, before = 0.0;
    for (int i = 0; i < w.C; ++i) total += part[i];
    const float uu = u ? u[t] : 0.f;
    const double want = f.one || !(uu > 0.f) ? 0.0 : (double)uu * total;
    double run = 0.0;
    bool hit = false;
    for (int i = 0; i < w.C; ++i) {
        if (part[i] > 0.0) {
            if (!hit) lastc = i, before = run;
            hit |= run + part[i] > want;
        }
        run += part[i];
    }
    c = lastc;
    if (km) {
        const unsigned kc = kmax[c];
        const float top = of_key(kc);
        // u beyond the last step leaves a want above the chunk's sum: its last token
        const double scale = f.one ? 1.0 : weight(et, top, st.first, f.invt);
        const double inside = fmin((want - before) / scale, 9.0e18);
        st.token = find_in_chunk<E, F32>(
            a, t, c, inside > 0.0 ? (uint64_t)inside : 0,
            [&](float x, int) {
                return x == -INFINITY ? (uint64_t)0 : f.one ? (uint64_t)(x == top) : units(weight(et, x, top, f.invt));
            },
            sums, &found);
        st.sum = f.one ? kUnit : total;
        if (f.one) st.key = km, st.last = st.token;
    }
    if (tid == 0) {
        w.states[t] = st;
        if (token) token[t] = st.token;
        if (prob)
            prob[t] = st.token < 0 ? 0.f
                                   : (float)(kept_weight(et, st, value<F32>(row_of<F32>(a, t), st.token), st.token) * kUnit / st.sum);
    }
}

// ---------------------------------------------------------------------------
// With filters
// ---------------------------------------------------------------------------
template <int E, bool F32>
__global__ __launch_bounds__(kRowThreads) void max_kernel(SampleArgs a, Work w) {
    __shared__ unsigned sk[kRowWaves];
    __shared__ int sn[kRowWaves];
    const int c = blockIdx.x, t = w.row0 + blockIdx.y, tid = threadIdx.x;
    float x[E][4];
    load_chunk<E, F32>(a, t, c, x);
    unsigned k = 0;
    int n = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const unsigned q = key_of(x[e][i]);
            k = max(k, q);
            n += q != 0;
        }
    n = wave_sum_int(n);
    if ((tid & 63) == 0) sn[tid >> 6] = n;
    k = block_max_u32(k, sk);
    if (tid == 0) {
        n = 0;
        for (int i = 0; i < kRowWaves; ++i) n += sn[i];
        w.kmax[blockIdx.y * w.C + c] = k;
        w.count[blockIdx.y * w.C + c] = n;
        if (c == 0) w.head[blockIdx.y] = Header{0, 0, 0, 0};
    }
}

// Which thresholds a row has.
struct Kind {
    unsigned km;
    bool by_k, by_p;
};

__device__ __forceinline__ Kind kind_of(const Filter &f, const Work &w, int row) {
    const int lane = threadIdx.x & 63;
    Kind k;
    k.km = row_key(w.kmax + row * w.C, w.C);
    const int n = wave_sum_int(lane < w.C ? w.count[row * w.C + lane] : 0);
    k.by_k = !f.one && f.topk > 0 && f.topk < n;
    k.by_p = !f.one && f.topp < 1.f && k.km;
    return k;
}

__device__ __forceinline__ int bin_of(float x, float first, double invt) {
    return min((int)(((double)first - (double)x) * invt * 32.0), kBins - 1);
}

// The weights of the last bin are below 2^-45 / 2 and have no units, so a
// top-p threshold never lies in it.
template <int E, bool F32>
__global__ __launch_bounds__(kRowThreads) void hist_kernel(SampleArgs a, Work w) {
    __shared__ ExpTable et;
    __shared__ unsigned cnt[kBins];
    __shared__ unsigned long long mass[kBins];
    __shared__ uint64_t wc[kRowWaves], wm[kRowWaves];
    __shared__ int sh;
    static_assert(kBins == kRowThreads, "a bin a thread");
    const int c = blockIdx.x, row = blockIdx.y, t = w.row0 + row, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Filter f = filter_of(a, t);
    const Kind kind = kind_of(f, w, row);
    if (!kind.by_k && !kind.by_p) return;  // the whole row's workgroups
    float x[E][4];
    load_chunk<E, F32>(a, t, c, x);
    et.fill();
    cnt[tid] = 0;
    mass[tid] = 0;
    __syncthreads();
    const float first = of_key(kind.km);
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (x[e][i] == -INFINITY) continue;
            const int b = bin_of(x[e][i], first, f.invt);
            if (b == kBins - 1) continue;
            atomicAdd(&cnt[b], 1u);
            if (!kind.by_k) atomicAdd(&mass[b], (unsigned long long)units(weight(et, x[e][i], first, f.invt)));
        }
    __syncthreads();
    const size_t at = ((size_t)row * w.C + c) * kBins + tid;
    put(w.hcnt + at, cnt[tid]);
    if (!kind.by_k) put(w.hmass + at, (uint64_t)mass[tid]);
    if (!last_of(&w.head[row].hist_done, w.C, &sh)) return;
    uint64_t n = 0, m = 0;
    for (int i = 0; i < w.C; ++i) {
        const size_t p = ((size_t)row * w.C + i) * kBins + tid;
        n += get(w.hcnt + p);
        if (!kind.by_k) m += get(w.hmass + p);
    }
    uint64_t ni = wave_scan_u64(n), mi = wave_scan_u64(m);
    if (lane == 63) wc[wave] = ni, wm[wave] = mi;
    __syncthreads();
    uint64_t total = 0;
    for (int i = 0; i < kRowWaves; ++i) {
        if (i < wave) ni += wc[i], mi += wm[i];
        total += wm[i];
    }
    const uint64_t want = kind.by_k ? (uint64_t)f.topk : max((uint64_t)1, (uint64_t)ceil((double)f.topp * (double)total));
    const uint64_t hi = kind.by_k ? ni : mi, lo = hi - (kind.by_k ? n : m);
    if (lo < want && want <= hi) {
        Plan p;
        p.sure = kind.by_k ? 0 : tid;  // by_k: the sum of the first top_k comes from the list
        p.end = tid;
        p.slow = (kind.by_k ? ni : n) > (uint64_t)kList;
        p.pad = 0;
        p.above_cnt = kind.by_k ? 0 : ni - n;
        p.above_mass = kind.by_k ? 0 : mi - m;
        p.mass = total;
        w.plan[row] = p;
    }
    // by_k with the threshold in the last bin: no thread above has it
    if (tid == kBins - 1 && kind.by_k && want > ni) w.plan[row] = Plan{0, kBins - 1, 1, 0, 0, 0, 0};
}

// The row's filter by radix descent, by one workgroup.
template <bool F32>
__device__ void descend_row(const ExpTable &et, const SampleArgs &a, const void *row, const Filter &f, const Kind &kind,
                            RowState &st, Histogram &h, uint64_t *sums, int *found) {
    uint64_t ca, ma, wk = 0, ties = 0;
    if (kind.by_k) {
        descend<F32>(et, row, a.V, st.first, st.invt, true, (uint64_t)f.topk, h, st.key, ca, ma);
        ties = (uint64_t)f.topk - ca;
        wk = ma + ties * units(weight(et, of_key(st.key), st.first, st.invt));
    } else {
        pick(
            a.V,
            [&](int i) {
                const float x = value<F32>(row, i);
                return x == -INFINITY ? (uint64_t)0 : units(weight(et, x, st.first, st.invt));
            },
            [](uint64_t total) { return total; }, sums, found, &wk);
    }
    if (kind.by_p) {
        const uint64_t want = min(max((uint64_t)1, (uint64_t)ceil((double)f.topp * (double)wk)), wk);
        descend<F32>(et, row, a.V, st.first, st.invt, false, want, h, st.key, ca, ma);
        const uint64_t w = units(weight(et, of_key(st.key), st.first, st.invt));
        ties = (want - ma + w - 1) / w;
    }
    uint64_t total;
    st.last = pick(
        a.V, [&](int i) { return (uint64_t)(key_of(value<F32>(row, i)) == st.key); },
        [&](uint64_t n) { return min(ties, n) - 1; }, sums, found, &total);
}

union DrawShared {
    uint64_t list[kList];
    Histogram h;
};

template <int E, bool F32>
__global__ __launch_bounds__(kRowThreads) void draw_kernel(SampleArgs a, Work w, const float *u, int32_t *token,
                                                           float *prob) {
    __shared__ ExpTable et;
    __shared__ DrawShared s;
    __shared__ uint64_t sums[(E > 1 ? E : 1) * kRowWaves];
    __shared__ unsigned long long cs[kMaxChunks];
    __shared__ int sh, found;
    __shared__ unsigned lkey;
    __shared__ int lidx;
    const int c = blockIdx.x, row = blockIdx.y, t = w.row0 + row, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const Filter f = filter_of(a, t);
    const Kind kind = kind_of(f, w, row);
    const bool planned = kind.by_k || kind.by_p;
    float x[E][4];
    load_chunk<E, F32>(a, t, c, x);
    et.fill();
    if (tid == 0) sh = 0, found = INT_MAX;
    Plan p{kBins, -1, 0, 0, 0, 0, 0};
    if (planned) p = w.plan[row];
    RowState st{f.invt, f.one ? 0.0 : f.minp, of_key(kind.km), 1u, a.V, -1, 0.0};
    __syncthreads();

    // ---- the chunk: sums of the sure, list of the others ----
    uint64_t sum = 0;
    if (f.one) {
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 3; i >= 0; --i)
                if (kind.km && key_of(x[e][i]) == kind.km) atomicMin(&found, (c * E + e) * kTile + 4 * tid + i);
        __syncthreads();
        sum = (uint64_t)found;
    } else if (!p.slow) {
        int mine = 0;
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (x[e][i] == -INFINITY) continue;
                const int b = planned ? bin_of(x[e][i], st.first, f.invt) : 0;
                if (b < p.sure) {
                    const double wt = weight(et, x[e][i], st.first, f.invt);
                    if (wt >= st.minp) sum += units(wt);
                } else if (b <= p.end) {
                    ++mine;
                }
            }
        sum = block_sum_u64(sum, sums);
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
                    for (int i = 0; i < 4; ++i) {
                        if (x[e][i] == -INFINITY) continue;
                        const int b = bin_of(x[e][i], st.first, f.invt);
                        if (b >= p.sure && b <= p.end && at < kList)
                            put(w.list + (size_t)row * kList + at++,
                                ((uint64_t)~key_of(x[e][i]) << 32) | (unsigned)((c * E + e) * kTile + 4 * tid + i));
                    }
            }
        }
    }
    if (tid == 0) put(w.sum + row * w.C + c, sum);
    if (!last_of(&w.head[row].draw_done, w.C, &sh)) return;

    // ---- the row, by its last workgroup ----
    if (tid < kMaxChunks) cs[tid] = tid < w.C ? get(w.sum + row * w.C + tid) : 0;
    __syncthreads();
    if (kind.km == 0) {
        // no token
    } else if (f.one) {
        uint64_t lo = cs[0];
        for (int i = 1; i < w.C; ++i) lo = min(lo, (uint64_t)cs[i]);
        st.key = kind.km;
        st.last = st.token = (int)lo;
        st.sum = kUnit;
    } else if (p.slow) {
        descend_row<F32>(et, a, row_of<F32>(a, t), f, kind, st, s.h, sums, &found);
        uint64_t total;
        const void *r = row_of<F32>(a, t);
        st.token = pick(
            a.V, [&](int i) { return units(kept_weight(et, st, value<F32>(r, i), i)); },
            [&](uint64_t total) { return target(u ? u[t] : 0.f, total); }, sums, &found, &total);
        st.sum = (double)total;
    } else {
        if (planned) {
            // sort the list: key descending, index ascending
            const int n = min(get(&w.head[row].listed), kList);
            int size = 64;
            while (size < n) size <<= 1;
            for (int i = tid; i < size; i += kRowThreads) s.list[i] = i < n ? get(w.list + (size_t)row * kList + i) : ~0ull;
            __syncthreads();
            for (int k = 2; k <= size; k <<= 1)
                for (int j = k >> 1; j > 0; j >>= 1) {
                    for (int i = tid; i < size / 2; i += kRowThreads) {
                        const int lo = ((i & ~(j - 1)) << 1) | (i & (j - 1)), hi = lo | j;
                        const uint64_t x0 = s.list[lo], x1 = s.list[hi];
                        if ((x0 > x1) == ((lo & k) == 0)) s.list[lo] = x1, s.list[hi] = x0;
                    }
                    __syncthreads();
                }
            // running weights of the list: thread tid holds `per` of them
            const int per = (size + kRowThreads - 1) / kRowThreads, b = tid * per;
            auto unit_at = [&](int i) { return units(weight(et, of_key(~(unsigned)(s.list[i] >> 32)), st.first, f.invt)); };
            const int e = min(b + per, n), nk = kind.by_k ? min(f.topk, n) : n;
            uint64_t mine = 0;
            for (int i = b; i < e && i < nk; ++i) mine += unit_at(i);
            uint64_t incl = wave_scan_u64(mine);
            if (lane == 63) sums[wave] = incl;
            __syncthreads();
            uint64_t wk = 0;
            for (int i = 0; i < kRowWaves; ++i) {
                if (i < wave) incl += sums[i];
                wk += sums[i];
            }
            __syncthreads();
            // how many of the list are kept
            if (tid == 0) found = nk;
            __syncthreads();
            if (kind.by_p) {
                const uint64_t whole = kind.by_k ? wk : p.mass;
                const uint64_t want = max((uint64_t)1, (uint64_t)ceil((double)f.topp * (double)whole));
                uint64_t run = p.above_mass + incl - mine;
                if (run < want && want <= run + mine)
                    for (int i = b; i < e && i < nk; ++i) {
                        run += unit_at(i);
                        if (run >= want) {
                            found = i + 1;
                            break;
                        }
                    }
            }
            __syncthreads();
            const int kept = found;
            if (tid == 0 && kept > 0) {
                lkey = ~(unsigned)(s.list[kept - 1] >> 32);
                lidx = (int)(unsigned)s.list[kept - 1];
            }
            for (int i = b; i < e && i < kept; ++i) {
                const double wt = weight(et, of_key(~(unsigned)(s.list[i] >> 32)), st.first, f.invt);
                if (wt >= st.minp) atomicAdd(&cs[(unsigned)s.list[i] / (E * kTile)], (unsigned long long)units(wt));
            }
            __syncthreads();
            st.key = lkey;
            st.last = lidx;
        }
        uint64_t total = 0;
        for (int i = 0; i < w.C; ++i) total += cs[i];
        uint64_t want = target(u ? u[t] : 0.f, total);
        int ch = 0;
        while (ch + 1 < w.C && want >= cs[ch]) want -= cs[ch++];
        st.token = find_in_chunk<E, F32>(
            a, t, ch, want, [&](float v, int i) { return units(kept_weight(et, st, v, i)); }, sums, &found);
        st.sum = (double)total;
    }
    if (tid == 0) {
        w.states[t] = st;
        if (token) token[t] = st.token;
        if (prob)
            prob[t] = st.token < 0 ? 0.f
                                   : (float)(kept_weight(et, st, value<F32>(row_of<F32>(a, t), st.token), st.token) * kUnit / st.sum);
    }
}

// ---------------------------------------------------------------------------
// The whole distribution of a row
// ---------------------------------------------------------------------------
template <int E, bool F32>
__global__ __launch_bounds__(kRowThreads) void probs_kernel(SampleArgs a, Work w, float *probs) {
    __shared__ ExpTable et;
    const int c = blockIdx.x, t = w.row0 + blockIdx.y;
    float x[E][4];
    load_chunk<E, F32>(a, t, c, x);
    const RowState st = w.states[t];
    et.fill();
    __syncthreads();
    const double k = st.sum > 0.0 ? kUnit / st.sum : 0.0;
    float *out = probs + (size_t)t * a.V;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int at = (c * E + e) * kTile + 4 * threadIdx.x;
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (float)(kept_weight(et, st, x[e][i], at + i) * k);
        if (at + 4 <= a.V) {
            *reinterpret_cast<f32x4_any *>(out + at) = v;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (at + i < a.V) out[at + i] = v[i];
        }
    }
}

// ---------------------------------------------------------------------------
// Acceptance
// ---------------------------------------------------------------------------
// Drafts matched against the target's own draws: one thread a sequence.
__global__ __launch_bounds__(64) void match_kernel(AcceptArgs c, const int32_t *drawn) {
    const int s = threadIdx.x;
    if (s >= c.nseq) return;
    const int r0 = c.off[s], n = c.off[s + 1] - r0;
    int cur = 0, k = 0;
    if (n) {
        while (true) {
            c.path[r0 + k] = cur;
            const int y = drawn[r0 + cur];
            c.out[r0 + k] = y;
            ++k;
            int next = -1;
            if (y >= 0)
                for (int j = cur + 1; j < n && next < 0; ++j)
                    if (c.parent[r0 + j] == cur && c.tokens[r0 + j] == y) next = j;
            if (next < 0) break;
            cur = next;
        }
    }
    c.count[s] = k;
    for (int j = k; j < n; ++j) c.path[r0 + j] = c.out[r0 + j] = -1;
}

// Chains against the drafter's distributions.  Every workgroup of a sequence
// finds the row of the last token (thread j tests draft j + 1), sums its
// chunk of max(p - q, 0) there, or of p, and the last one draws.
template <int E, bool F32>
__global__ __launch_bounds__(kRowThreads) void chain_kernel(SampleArgs a, AcceptArgs c, Work w) {
    __shared__ ExpTable et;
    __shared__ uint64_t sums[(E > 1 ? E : 1) * kRowWaves];
    __shared__ uint64_t cs[kMaxChunks];
    __shared__ int sh, found, row_sh;
    const int ch = blockIdx.x, s = blockIdx.y, r0 = c.off[s], n = c.off[s + 1] - r0, tid = threadIdx.x;
    if (n == 0) {
        if (ch == 0 && tid == 0) c.count[s] = 0;
        return;
    }
    et.fill();
    __syncthreads();
    auto p_of = [&](const RowState &st, float x, int i) {
        return st.sum > 0.0 ? kept_weight(et, st, x, i) * (kUnit / st.sum) : 0.0;
    };
    if (tid < 64) {  // n <= 64
        bool stop = true;
        if (tid + 1 < n) {
            const int t = r0 + tid, x = c.tokens[t + 1];
            if (x >= 0 && x < a.V) {
                const double p = p_of(w.states[t], value<F32>(row_of<F32>(a, t), x), x);
                stop = !((double)c.u[t] * (double)c.q[(size_t)t * a.V + x] < p);
            }
        }
        const uint64_t first = __ballot(stop);  // the last row always stops
        if (tid == 0) row_sh = __ffsll((unsigned long long)first) - 1;
    }
    __syncthreads();
    const int j = row_sh, t = r0 + j;
    const bool rest = j + 1 < n;
    const RowState st = w.states[t];
    const float *q = c.q + (size_t)t * a.V;
    auto mass = [&](float x, int i) {
        const double v = fmax(p_of(st, x, i) - (rest ? (double)q[i] : 0.0), 0.0);
        return (uint64_t)__double_as_longlong(fma(v, 2251799813685248.0, 4503599627370496.0)) & 0xFFFFFFFFFFFFFull;  // 2^51
    };
    float x[E][4];
    load_chunk<E, F32>(a, t, ch, x);
    uint64_t sum = 0;
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (ch * E + e) * kTile + 4 * tid + i;
            if (at < a.V) sum += mass(x[e][i], at);
        }
    sum = block_sum_u64(sum, sums);
    if (tid == 0) put(w.sum + r0 * w.C + ch, sum);
    if (!last_of(&w.head[r0].chain_done, w.C, &sh)) return;
    if (tid < kMaxChunks) cs[tid] = tid < w.C ? get(w.sum + r0 * w.C + tid) : 0;
    __syncthreads();
    uint64_t total = 0;
    for (int i = 0; i < w.C; ++i) total += cs[i];
    const float u = c.u_final[s];
    int tok;
    if (total) {
        uint64_t want = target(u, total);
        int k = 0;
        while (k + 1 < w.C && want >= cs[k]) want -= cs[k++];
        tok = find_in_chunk<E, F32>(a, t, k, want, mass, sums, &found);
    } else {  // nothing of p lies above q
        const void *row = row_of<F32>(a, t);
        tok = pick(
            a.V, [&](int i) { return units(kept_weight(et, st, value<F32>(row, i), i)); },
            [&](uint64_t total) { return target(u, total); }, sums, &found, &total);
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

// Tiles of a chunk: enough workgroups for the chip before longer chunks.
int tiles_of(int T, int V) {
    const int tiles = (V + kTile - 1) / kTile;
    for (int e = 1; e < 4; e *= 2)
        if ((long long)T * ((tiles + e - 1) / e) <= 2048) return e;
    return 4;
}

struct Layout {
    int E, C, rows;  // tiles of a chunk, chunks of a row, rows of a batch
    size_t states, drawn, kmax, count, sum, head, plan, list, hcnt, hmass, total;
};

Layout layout(int T, int V) {
    Layout l{};
    const int tiles = (V + kTile - 1) / kTile;
    l.E = tiles_of(T, V);
    l.C = (tiles + l.E - 1) / l.E;
    l.rows = T < 4096 / l.C ? T : 4096 / l.C;
    if (l.rows < 1) l.rows = 1;
    size_t off = 0;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off = align256(off + bytes);
        return at;
    };
    const size_t rc = (size_t)l.rows * l.C;
    l.states = take((size_t)T * sizeof(RowState));
    l.drawn = take((size_t)T * 4);
    l.kmax = take(rc * 4);
    l.count = take(rc * 4);
    l.sum = take(rc * 8);
    l.head = take((size_t)l.rows * sizeof(Header));
    l.plan = take((size_t)l.rows * sizeof(Plan));
    l.list = take((size_t)l.rows * kList * 8);
    l.hcnt = take(rc * kBins * 4);
    l.hmass = take(rc * kBins * 8);
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
    w.sum = reinterpret_cast<uint64_t *>(p + l.sum);
    w.head = reinterpret_cast<Header *>(p + l.head);
    w.plan = reinterpret_cast<Plan *>(p + l.plan);
    w.list = reinterpret_cast<uint64_t *>(p + l.list);
    w.hcnt = reinterpret_cast<unsigned *>(p + l.hcnt);
    w.hmass = reinterpret_cast<uint64_t *>(p + l.hmass);
    w.row0 = 0;
    w.C = l.C;
    return w;
}

// States, and draws with u, of all rows.
template <int E, bool F32>
hipError_t rows(const SampleArgs &a, Work w, const Layout &l, const float *u, int32_t *token, float *prob, float *probs,
                hipStream_t s) {
    for (; w.row0 < a.T; w.row0 += l.rows) {
        const int n = a.T - w.row0 < l.rows ? a.T - w.row0 : l.rows;
        const dim3 grid(l.C, n), block(kRowThreads);
        if (!a.top_k && !a.top_p && !a.min_p) {
            hipLaunchKernelGGL((part_kernel<E, F32>), grid, block, 0, s, a, w);
            hipLaunchKernelGGL((join_kernel<E, F32>), dim3(n), block, 0, s, a, w, u, token, prob);
        } else {
            hipLaunchKernelGGL((max_kernel<E, F32>), grid, block, 0, s, a, w);
            if (a.top_k || a.top_p) hipLaunchKernelGGL((hist_kernel<E, F32>), grid, block, 0, s, a, w);
            hipLaunchKernelGGL((draw_kernel<E, F32>), grid, block, 0, s, a, w, u, token, prob);
        }
        if (probs) hipLaunchKernelGGL((probs_kernel<E, F32>), grid, block, 0, s, a, w, probs);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

template <int E, bool F32>
hipError_t accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t s) {
    const Layout l = layout(a.T, a.V);
    const Work w = work_of(a, l);
    hipError_t e = rows<E, F32>(a, w, l, c.q ? nullptr : c.u, c.q ? nullptr : w.drawn, nullptr, nullptr, s);
    if (e != hipSuccess) return e;
    if (c.q)
        hipLaunchKernelGGL((chain_kernel<E, F32>), dim3(l.C, c.nseq), dim3(kRowThreads), 0, s, a, c, w);
    else
        hipLaunchKernelGGL(match_kernel, dim3(1), dim3(64), 0, s, c, w.drawn);
    return hipGetLastError();
}

template <typename F>
hipError_t by_type(const SampleArgs &a, F f) {
    switch (layout(a.T, a.V).E) {
        case 1: return a.f32 ? f.template operator()<1, true>() : f.template operator()<1, false>();
        case 2: return a.f32 ? f.template operator()<2, true>() : f.template operator()<2, false>();
        default: return a.f32 ? f.template operator()<4, true>() : f.template operator()<4, false>();
    }
}

struct SampleCall {
    const SampleArgs &a;
    const float *u;
    int32_t *token;
    float *prob, *probs;
    hipStream_t s;
    template <int E, bool F32>
    hipError_t operator()() const {
        const Layout l = layout(a.T, a.V);
        return rows<E, F32>(a, work_of(a, l), l, u, token, prob, probs, s);
    }
};

struct AcceptCall {
    const SampleArgs &a;
    const AcceptArgs &c;
    hipStream_t s;
    template <int E, bool F32>
    hipError_t operator()() const {
        return accept<E, F32>(a, c, s);
    }
};

}  // namespace

size_t sample_ws_bytes(int T, int V) { return layout(T > 0 ? T : 1, V).total; }

hipError_t launch_sample(const SampleArgs &a, const float *u, int32_t *token, float *prob, float *probs, hipStream_t s) {
    return by_type(a, SampleCall{a, u, token, prob, probs, s});
}

hipError_t launch_accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t s) {
    return by_type(a, AcceptCall{a, c, s});
}

}  // namespace moe
