// Drawing and accepting draft tokens.  The filtered distribution of a row of
// logits is defined in include/moe_verify.h.
//
// Every filter keeps a prefix of the row's ranking (value desc, index asc),
// so a row's filter is one threshold: the last kept value and, among equal
// values, the last kept index.  Weights w = exp(-(first - l) / temperature)
// are computed in float64 and summed as integers in units of 2^-45: a sum
// does not depend on its order, and 2^18 weights of at most 1 fit 63 bits.
#include "common.h"
#include "serve.h"

namespace moe {
namespace {

constexpr int kRowThreads = 1024;
constexpr int kRowWaves = kRowThreads / 64;
constexpr double kUnit = 35184372088832.0;         // 2^45
constexpr double kUnitP = 1152921504606846976.0;   // 2^60, of probabilities (their sum is 1)

// What a row's filter comes to.
struct RowState {
    double invt, minp;
    float first;      // the largest value
    unsigned key;     // last kept value, as an ordered key
    int last;         // last kept index among values of that key
    int pad;
    uint64_t sum;     // weights kept
};

struct Logits {
    const void *p;
    int64_t stride;
    int f32;
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

__device__ __forceinline__ double weight(float x, float first, double invt) {
    return exp(((double)x - (double)first) * invt);
}

__device__ __forceinline__ uint64_t units(double w) { return (uint64_t)(w * kUnit + 0.5); }

// A kept token's weight, 0 for the others.
__device__ __forceinline__ double kept_weight(const RowState &st, float x, int i) {
    const unsigned k = key_of(x);
    if (k == 0 || k < st.key || (k == st.key && i > st.last)) return 0.0;
    const double w = weight(x, st.first, st.invt);
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
    uint64_t above_cnt, above_mass, total_cnt;
};

// Radix descent over the keys from the top: the bin, key after key, in which
// the running count (by_count) or the running weight of the ranking reaches
// `want`.  Leaves the key, and the count and weight strictly above it.
template <bool F32>
__device__ void descend(const void *row, int V, float first, double invt, bool by_count, uint64_t want, Histogram &h,
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
            atomicAdd(&h.mass[b], (unsigned long long)units(weight(x, first, invt)));
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

// One workgroup a row: the filter, then (with u) the draw.
template <bool F32>
__global__ __launch_bounds__(kRowThreads) void row_kernel(SampleArgs a, RowState *states, const float *u, int32_t *token,
                                                          float *prob) {
    __shared__ Histogram h;
    __shared__ uint64_t sums[kRowWaves];
    __shared__ int found;
    __shared__ unsigned kmax[kRowWaves];
    __shared__ int nval[kRowWaves];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const void *row = (const char *)a.logits + (size_t)t * a.stride * (F32 ? 4 : 2);
    unsigned km = 0;
    int nv = 0;
    for (int i = tid; i < a.V; i += kRowThreads) {
        const unsigned k = key_of(value<F32>(row, i));
        km = max(km, k);
        nv += k != 0;
    }
#pragma unroll
    for (int d = 32; d; d >>= 1) km = max(km, (unsigned)__shfl_xor((int)km, d));
    nv = wave_sum_int(nv);
    if (lane == 0) kmax[wave] = km, nval[wave] = nv;
    __syncthreads();
    nv = 0;
    for (int w = 0; w < kRowWaves; ++w) km = max(km, kmax[w]), nv += nval[w];

    RowState st{};
    st.first = of_key(km);
    st.key = 1;  // every value
    st.last = a.V;
    const float temp = a.temperature ? a.temperature[t] : 1.f;
    const int topk = a.top_k ? a.top_k[t] : 0;
    const float topp = a.top_p ? a.top_p[t] : 1.f, minp = a.min_p ? a.min_p[t] : 0.f;
    const bool one = !(temp > 0.f) || minp > 1.f || topk == 1 || topp <= 0.f;
    st.invt = temp > 0.f ? 1.0 / (double)temp : 0.0;
    st.minp = !one && minp > 0.f ? (double)minp : 0.0;
    if (nv) {
        uint64_t ties = 0;  // of the values of st.key, how many are kept; 0: all
        if (one) {
            st.key = km;
            ties = 1;
        } else {
            uint64_t ca, ma, wk = 0;
            const bool by_k = topk > 0 && topk < nv, by_p = topp < 1.f;
            if (by_k) {
                descend<F32>(row, a.V, st.first, st.invt, true, (uint64_t)topk, h, st.key, ca, ma);
                ties = (uint64_t)topk - ca;
                wk = ma + ties * units(weight(of_key(st.key), st.first, st.invt));
            } else if (by_p) {
                int none;
                none = pick(
                    a.V,
                    [&](int i) {
                        const float x = value<F32>(row, i);
                        return x == -INFINITY ? (uint64_t)0 : units(weight(x, st.first, st.invt));
                    },
                    [](uint64_t total) { return total; }, sums, &found, &wk);
                (void)none;
            }
            if (by_p) {
                const uint64_t want = max((uint64_t)1, (uint64_t)ceil((double)topp * (double)wk));
                descend<F32>(row, a.V, st.first, st.invt, false, min(want, wk), h, st.key, ca, ma);
                const uint64_t w = units(weight(of_key(st.key), st.first, st.invt));
                ties = (min(want, wk) - ma + w - 1) / w;
            }
        }
        if (ties) {
            uint64_t total;
            const int i = pick(
                a.V, [&](int i) { return (uint64_t)(key_of(value<F32>(row, i)) == st.key); },
                [&](uint64_t total) { return min(ties, total) - 1; }, sums, &found, &total);
            st.last = i;
        }
    }
    uint64_t total;
    const int tok = pick(
        a.V, [&](int i) { return units(kept_weight(st, value<F32>(row, i), i)); },
        [&](uint64_t total) { return target(u ? u[t] : 0.f, total); }, sums, &found, &total);
    st.sum = total;
    if (tid == 0) {
        states[t] = st;
        if (token) token[t] = tok;
        if (prob) prob[t] = tok < 0 ? 0.f : (float)(kept_weight(st, value<F32>(row, tok), tok) * kUnit / (double)total);
    }
}

template <bool F32>
__global__ __launch_bounds__(256) void probs_kernel(SampleArgs a, const RowState *states, float *probs) {
    const int t = blockIdx.x;
    const RowState st = states[t];
    const void *row = (const char *)a.logits + (size_t)t * a.stride * (F32 ? 4 : 2);
    const double k = st.sum ? kUnit / (double)st.sum : 0.0;
    for (int i = blockIdx.y * 256 + threadIdx.x; i < a.V; i += 256 * gridDim.y)
        probs[(size_t)t * a.V + i] = (float)(kept_weight(st, value<F32>(row, i), i) * k);
}

__device__ __forceinline__ int segment_of_thread(const AcceptArgs &c) { return threadIdx.x < (unsigned)c.nseq ? (int)threadIdx.x : -1; }

// Drafts matched against the target's own draws: one thread a sequence.
__global__ __launch_bounds__(64) void match_kernel(AcceptArgs c, const int32_t *drawn) {
    const int s = segment_of_thread(c);
    if (s < 0) return;
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

// Chains against the drafter's distributions: one workgroup a sequence.
template <bool F32>
__global__ __launch_bounds__(kRowThreads) void chain_kernel(SampleArgs a, AcceptArgs c, const RowState *states) {
    __shared__ uint64_t sums[kRowWaves];
    __shared__ int found;
    const int s = blockIdx.x, r0 = c.off[s], n = c.off[s + 1] - r0, tid = threadIdx.x;
    auto row_of = [&](int t) { return (const void *)((const char *)a.logits + (size_t)t * a.stride * (F32 ? 4 : 2)); };
    auto p_of = [&](const RowState &st, const void *row, int i) {
        return st.sum ? kept_weight(st, value<F32>(row, i), i) * kUnit / (double)st.sum : 0.0;
    };
    int j = 0;
    for (; j + 1 < n; ++j) {
        const int t = r0 + j, x = c.tokens[t + 1];
        if (x < 0 || x >= a.V) break;
        const RowState st = states[t];
        if (!((double)c.u[t] * (double)c.q[(size_t)t * a.V + x] < p_of(st, row_of(t), x))) break;
    }
    if (n) {
        const int t = r0 + j;
        const RowState st = states[t];
        const void *row = row_of(t);
        const float *q = c.q + (size_t)t * a.V;
        const float u = c.u_final[s];
        uint64_t total = 0;
        int tok = -1;
        if (j + 1 < n)
            tok = pick(
                a.V, [&](int i) { return (uint64_t)(fmax(p_of(st, row, i) - (double)q[i], 0.0) * kUnitP + 0.5); },
                [&](uint64_t total) { return target(u, total); }, sums, &found, &total);
        if (total == 0)
            tok = pick(
                a.V, [&](int i) { return units(kept_weight(st, value<F32>(row, i), i)); },
                [&](uint64_t total) { return target(u, total); }, sums, &found, &total);
        for (int i = tid; i < n; i += kRowThreads) {
            c.path[r0 + i] = i <= j ? i : -1;
            c.out[r0 + i] = i < j ? c.tokens[r0 + i + 1] : i == j ? tok : -1;
        }
    }
    if (tid == 0) c.count[s] = n ? j + 1 : 0;
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

struct Layout {
    size_t states, drawn, total;
};

Layout layout(int T) {
    Layout l;
    l.states = 0;
    l.drawn = align256((size_t)T * sizeof(RowState));
    l.total = l.drawn + align256((size_t)T * 4);
    return l;
}

template <bool F32>
hipError_t sample(const SampleArgs &a, const float *u, int32_t *token, float *prob, float *probs, hipStream_t s) {
    RowState *st = reinterpret_cast<RowState *>(a.ws);
    hipLaunchKernelGGL(row_kernel<F32>, dim3(a.T), dim3(kRowThreads), 0, s, a, st, u, token, prob);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !probs) return e;
    hipLaunchKernelGGL(probs_kernel<F32>, dim3(a.T, (a.V + 4095) / 4096), dim3(256), 0, s, a, st, probs);
    return hipGetLastError();
}

template <bool F32>
hipError_t accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t s) {
    RowState *st = reinterpret_cast<RowState *>(a.ws);
    int32_t *drawn = reinterpret_cast<int32_t *>((char *)a.ws + layout(a.T).drawn);
    hipLaunchKernelGGL(row_kernel<F32>, dim3(a.T), dim3(kRowThreads), 0, s, a, st, c.q ? nullptr : c.u,
                       c.q ? nullptr : drawn, (float *)nullptr);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (c.q)
        hipLaunchKernelGGL(chain_kernel<F32>, dim3(c.nseq), dim3(kRowThreads), 0, s, a, c, st);
    else
        hipLaunchKernelGGL(match_kernel, dim3(1), dim3(64), 0, s, c, drawn);
    return hipGetLastError();
}

}  // namespace

size_t sample_ws_bytes(int T, int V) {
    (void)V;
    return layout(T).total + 256;
}

hipError_t launch_sample(const SampleArgs &a, const float *u, int32_t *token, float *prob, float *probs, hipStream_t s) {
    return a.f32 ? sample<true>(a, u, token, prob, probs, s) : sample<false>(a, u, token, prob, probs, s);
}

hipError_t launch_accept(const SampleArgs &a, const AcceptArgs &c, hipStream_t s) {
    return a.f32 ? accept<true>(a, c, s) : accept<false>(a, c, s);
}

}  // namespace moe
