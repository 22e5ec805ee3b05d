// The 4-bit K/V cache: quantisation of rows into pages, and the attention of
// the verified tokens over it.  Layout and formulas in include/moe_verify.h.
#include "common.h"
#include "serve.h"

namespace moe {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// 2^(e - 127) of a scale byte.
__device__ __forceinline__ float scale_of(unsigned e) { return __uint_as_float(e << 23); }

// Bytes of a row's 17 D / 16 share: a tile holds 16 rows of K, its scales, V and its scales.
template <int D>
struct Tile {
    static constexpr int kK = 0, kKs = 8 * D, kV = 17 * D / 2, kVs = 33 * D / 2, kBytes = 17 * D;
};

// ---------------------------------------------------------------------------
// Append.  One lane holds 8 consecutive elements of a row, so 4 lanes share a
// block's scale and D / 8 lanes a row; a wave takes 512 / D consecutive rows
// of one head (their V codes lie next to each other, 4 rows in 4 D / 2
// contiguous bytes).  K and V are the grid's z.  Memory bound: a row is read
// once and its codes written once.
// ---------------------------------------------------------------------------
// e2m1 code of a scaled value, round to nearest, ties to the even code.
__device__ __forceinline__ unsigned e2m1(float x) {
    const float a = fabsf(x);
    const unsigned c = (unsigned)(a > 0.25f) + (a >= 0.75f) + (a > 1.25f) + (a >= 1.75f) + (a > 2.5f) + (a >= 3.5f) +
                       (a > 5.0f);
    return c | (x < 0.f && c ? 8u : 0u);
}

__device__ __forceinline__ float e2m1_value(unsigned c) {
    const unsigned m = c & 7;
    // 0, .5, then (1 + frac / 2) * 2^(exp - 1)
    const float v = m < 2 ? 0.5f * m : (m & 1 ? 1.5f : 1.f) * __uint_as_float((126u + (m >> 1)) << 23);
    return c & 8 ? -v : v;
}

template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void append_kernel(KvAppendArgs a) {
    constexpr int LPR = D / 8;         // lanes of a row
    constexpr int RPW = 64 / LPR;      // rows of a wave
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int h = blockIdx.y;
    const bool isv = blockIdx.z != 0;
    const int l = lane % LPR;
    const int t = (blockIdx.x * kWaves + wave) * RPW + lane / LPR;  // call row of the destination
    if (t >= a.T) return;  // whole rows leave together; the shuffles below stay inside a row
    int s = 0;
    while (t >= a.r.off[s + 1]) ++s;
    const int j = t - a.r.off[s], n = a.r.off[s + 1] - a.r.off[s];
    int src = t;
    if (a.path) {
        if (j >= a.count[s]) return;
        const int p = a.path[t];
        if (p < 0 || p >= n) return;
        src = a.r.off[s] + p;
    }
    float x[8];
    const size_t at = (size_t)src * (isv ? a.vs : a.ks) + (size_t)h * D + l * 8;
    if (F32) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>((const float *)(isv ? a.v : a.k) + at);
        const f32x4 u = p[0], w = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = u[i], x[4 + i] = w[i];
    } else {
        const u32x4 u = *reinterpret_cast<const u32x4 *>((const uint16_t *)(isv ? a.v : a.k) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = __uint_as_float(u[i] << 16), x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    // the smallest n with m <= 6 * 2^n = 1.5 * 2^(n + 2)
    const unsigned mb = __float_as_uint(m);
    int e = (int)(mb >> 23) - 127 - 2 + ((mb & 0x7fffffu) > 0x400000u);
    e = min(max(e, -100), 125);
    const float inv = scale_of(127 - e);
    unsigned code[8], word = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        code[i] = e2m1(x[i] * inv);
        word |= code[i] << (4 * i);
    }
    if (a.k_out) {
        const float sc = scale_of(127 + e);
        const size_t o = ((size_t)t * a.r.Hkv + h) * D + l * 8;
        void *dst = isv ? a.v_out : a.k_out;
        if (F32) {
            f32x4 u, w;
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = e2m1_value(code[i]) * sc, w[i] = e2m1_value(code[4 + i]) * sc;
            f32x4 *p = reinterpret_cast<f32x4 *>((float *)dst + o);
            p[0] = u;
            p[1] = w;
        } else {  // 2 significant bits: exact in bf16
            u32x4 u;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = (__float_as_uint(e2m1_value(code[2 * i]) * sc) >> 16) |
                       (__float_as_uint(e2m1_value(code[2 * i + 1]) * sc) & 0xffff0000u);
            *reinterpret_cast<u32x4 *>((uint16_t *)dst + o) = u;
        }
    }
    const int64_t pos = (int64_t)max(a.r.len[s], 0) + j;
    const int64_t slot = pos >> a.r.page_shift;
    if (slot >= a.r.max_pages) return;
    const int pid = a.r.table[(size_t)s * a.r.max_pages + slot];
    if (pid < 0 || pid >= a.r.num_pages) return;
    const int in = (int)pos & ((1 << a.r.page_shift) - 1), i = in & 15;
    uint8_t *tile = a.r.data + ((((size_t)pid * a.r.Hkv + h) << (a.r.page_shift - 4)) + (in >> 4)) * Tile<D>::kBytes;
    if (!isv) {
        *reinterpret_cast<unsigned *>(tile + Tile<D>::kK + i * (D / 2) + l * 4) = word;
    } else {
        uint8_t *v = tile + Tile<D>::kV + (64 * (i >> 2) + (i & 3)) * (D / 32);
        if (D == 64) {  // 4 elements to an operand lane
            *reinterpret_cast<uint16_t *>(v + (2 * l) * 4 * (D / 32)) = (uint16_t)word;
            *reinterpret_cast<uint16_t *>(v + (2 * l + 1) * 4 * (D / 32)) = (uint16_t)(word >> 16);
        } else if (D == 128) {
            *reinterpret_cast<unsigned *>(v + l * 4 * (D / 32)) = word;
        } else {
            *reinterpret_cast<unsigned *>(v + (l >> 1) * 4 * (D / 32) + (l & 1) * 4) = word;
        }
    }
    if ((l & 3) == 0) tile[(isv ? Tile<D>::kVs : Tile<D>::kKs) + 16 * (l >> 2) + i] = (uint8_t)(127 + e);
}

// ---------------------------------------------------------------------------
// Attention.  Work is the flat list of units (sequence, K/V head, block of
// 16 MT query rows), each unit its steps of 32 cache rows; every workgroup
// takes an equal share of consecutive steps, whatever the lengths are, and
// its waves take the steps of a unit in turn.  A unit that more than one
// workgroup worked on is joined by combine_kernel.
//
// A step is two tiles of 16 cache rows.  S^T = K Q^T leaves lane (g, c) = (l / 16, l % 16)
// with the scores of rows 4 g .. 4 g + 3 of both tiles for query c, which is
// just the operand that O^T += V^T P^T needs, so the probabilities never leave
// the lane; the running maximum and sum belong to column c in both products.
// Codes become bf16 by v_cvt_scalef32_pk_bf16_fp4, exactly (2 significant
// bits and a power of two).  The maximum is moved only when a score passes it
// by 2^8, so most steps need no exchange between lanes.
// ---------------------------------------------------------------------------
constexpr float kNone = -3.402823466e38f;  // running maximum before the first score
constexpr float kSlack = 8.f;              // a score may pass the maximum by this (log2) before it moves
constexpr int kMinShare = 8;               // steps of a workgroup at least

__device__ __forceinline__ bf16x8 dequant8(unsigned w, float s) {
    union {
        bf16x2 h[4];
        bf16x8 v;
    } o;
    o.h[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    o.h[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    o.h[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    o.h[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
    return o.v;
}

// The flat list: what sequence `lane` adds to it.
struct Units {
    int len, total, steps, rows, mb;  // rows before the call, all rows, steps, query rows, row blocks
    long long incl;                   // running sum of steps over heads and row blocks
};

__device__ __forceinline__ Units units_of(const KvRows &r, int G, int block_rows, long long &all) {
    const int lane = threadIdx.x & 63;
    Units u{0, 0, 0, 0, 0, 0};
    if (lane < r.nseq) {
        const int n = r.off[lane + 1] - r.off[lane];
        const int cap = r.max_pages << r.page_shift;
        u.len = min(max(r.len[lane], 0), cap);
        u.total = min(u.len + n, cap);
        u.rows = n * G;
        u.mb = (u.rows + block_rows - 1) / block_rows;
        u.steps = (u.total + 31) >> 5;
    }
    u.incl = (long long)u.steps * u.mb * r.Hkv;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const long long v = __shfl_up(u.incl, d);
        if (lane >= d) u.incl += v;
    }
    all = __shfl(u.incl, 63);
    return u;
}

__device__ __forceinline__ long long share_of(long long all, int nwg) {
    const long long s = (all + nwg - 1) / nwg;
    return s > kMinShare ? s : kMinShare;
}

// Values of one step as loaded.
template <int D>
struct Frag {
    static constexpr int W = D / 32;  // words of a lane: D / 4 K elements, or 4 rows of D / 16 V elements
    unsigned k[2][W], v[2][W], vs[2];
    unsigned ks[2];  // one byte, or two for D = 256
    bool ok[2];      // the tile's page is in the pool
};

template <int N>
__device__ __forceinline__ void load_words(unsigned (&w)[N], const uint8_t *p) {
    if (N == 2) {
        const u32x2 a = *reinterpret_cast<const u32x2 *>(p);
        w[0] = a[0], w[1] = a[1];
    } else {
#pragma unroll
        for (int i = 0; i < N / 4; ++i) {
            const u32x4 a = reinterpret_cast<const u32x4 *>(p)[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * i + j] = a[j];
        }
    }
}

template <int MT, int D, bool F32>
constexpr int attend_lds_bytes() {
    const int q = MT * 16 * D * 2 * (F32 ? 3 : 1), m = 2 * MT * 16 * D * 4;
    return q > m ? q : m;
}

// 16-row tiles of a row block: its MT * D / 4 accumulators a lane, with the
// float32 type's three-term operands beside them, have to fit the registers.
constexpr int max_mt(int D, bool f32) { return D == 64 ? 4 : D == 128 ? (f32 ? 2 : 3) : 1; }

template <int MT, int D, bool F32>
__global__ __launch_bounds__(kThreads, MT == 1 && D < 256 ? 2 : 1) void attend_kernel(KvAttendArgs a) {
    constexpr int NS = F32 ? 3 : 1;  // bf16 terms of q and of the probabilities
    constexpr int KS = D / 32;       // k steps of the first product
    constexpr int C = D / 16;        // row tiles of the second
    constexpr int BR = 16 * MT;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float wm[kWaves][BR], wl[kWaves][BR];
    uint16_t *lq = reinterpret_cast<uint16_t *>(lds);  // [MT][NS][KS][64][8]
    float *lo = reinterpret_cast<float *>(lds);        // [2][MT][C][4][64], after the steps
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, c = lane & 15;
    const KvRows &r = a.r;

    long long all;
    const Units un = units_of(r, a.G, BR, all);
    const long long share = share_of(all, a.nwg);
    const long long x0 = (long long)blockIdx.x * share;
    long long x = x0, xe = x0 + share < all ? x0 + share : all;
    const float sl = a.scale * 1.44269504088896341f;

    while (x < xe) {
        const int s = __ffsll((unsigned long long)__ballot(un.incl > x)) - 1;
        const int len = __builtin_amdgcn_readlane(un.len, s), total = __builtin_amdgcn_readlane(un.total, s);
        const int steps = __builtin_amdgcn_readlane(un.steps, s), rows = __builtin_amdgcn_readlane(un.rows, s);
        const int mbs = __builtin_amdgcn_readlane(un.mb, s);
        const long long end_s = __shfl(un.incl, s);
        const long long rel = x - (end_s - (long long)steps * mbs * r.Hkv);
        const int unit = (int)(rel / steps), st0 = (int)(rel - (long long)unit * steps);
        const int h = unit / mbs, mb = unit - h * mbs;
        const int n = (int)(xe - x < steps - st0 ? xe - x : steps - st0);
        const int row0 = mb * BR, t0 = r.off[s], ntok = rows / a.G;

        // ---- the block's queries into LDS as bf16 operand terms ----
        __syncthreads();
        for (int i = threadIdx.x; i < BR * (D / 8); i += kThreads) {
            const int mt = i / (16 * (D / 8)), ks = (i / 64) % KS, ln = i & 63;
            const int row = row0 + mt * 16 + (ln & 15), d = (ln >> 4) * (D / 4) + ks * 8;
            uint16_t *dst = lq + ((size_t)(mt * NS * KS + ks) * 64 + ln) * 8;
            u32x4 z[NS];
#pragma unroll
            for (int p = 0; p < NS; ++p) z[p] = u32x4{0, 0, 0, 0};
            if (row < rows) {
                const size_t at = (size_t)(t0 + row / a.G) * a.qs + (size_t)(h * a.G + row % a.G) * D + d;
                if (F32) {
                    const float *p = (const float *)a.q + at;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float v = p[e];
#pragma unroll
                        for (int y = 0; y < NS; ++y) {
                            const unsigned b = f32_to_bf16_rne(v);
                            v -= bf16_to_f32((uint16_t)b);
                            z[y][e >> 1] |= b << (16 * (e & 1));
                        }
                    }
                } else {
                    z[0] = *reinterpret_cast<const u32x4 *>((const uint16_t *)a.q + at);
                }
            }
#pragma unroll
            for (int p = 0; p < NS; ++p) *reinterpret_cast<u32x4 *>(dst + (size_t)p * KS * 64 * 8) = z[p];
        }
        __syncthreads();

        float m[MT], l[MT];
        f32x4 o[MT][C];
        uint64_t see[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt] = kNone;
            l[mt] = 0.f;
            const int row = row0 + mt * 16 + c;
            see[mt] = row < rows ? a.anc[t0 + row / a.G] : 0;
#pragma unroll
            for (int i = 0; i < C; ++i) o[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // page ids of 64 table entries from slot0 on, one a lane
        int slot0 = -64, pids = -1;
        auto load = [&](int st, Frag<D> &f) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tile = 2 * st + t, slot = tile >> (r.page_shift - 4);
                if (slot >= slot0 + 64 || slot < slot0) {
                    slot0 = slot;
                    pids = slot + lane < r.max_pages ? r.table[(size_t)s * r.max_pages + slot + lane] : -1;
                }
                const int pid = __builtin_amdgcn_readlane(pids, slot - slot0);
                f.ok[t] = pid >= 0 && pid < r.num_pages;
                const int in = tile & ((1 << (r.page_shift - 4)) - 1);
                const uint8_t *b = r.data + ((((size_t)(f.ok[t] ? pid : 0) * r.Hkv + h) << (r.page_shift - 4)) + in) *
                                                Tile<D>::kBytes;
                load_words(f.k[t], b + Tile<D>::kK + c * (D / 2) + g * (D / 8));
                const uint8_t *ks = b + Tile<D>::kKs + c;
                if (D == 256)
                    f.ks[t] = ks[32 * g] | (ks[32 * g + 16] << 8);
                else
                    f.ks[t] = ks[16 * (g * (D / 4) / 32)];
                load_words(f.v[t], b + Tile<D>::kV + lane * (D / 8));
                f.vs[t] = *reinterpret_cast<const unsigned *>(b + Tile<D>::kVs + 16 * (c * (D / 16) / 32) + 4 * g);
            }
        };

        auto compute = [&](int st, Frag<D> &f) {
            f32x4 sc[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) sc[mt][0] = sc[mt][1] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                bf16x8 kf[2];
#pragma unroll
                for (int t = 0; t < 2; ++t) kf[t] = dequant8(f.k[t][ks], scale_of((f.ks[t] >> (8 * (ks / 4))) & 255u));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int y = 0; y < NS; ++y) {
                        const bf16x8 q = *reinterpret_cast<const bf16x8 *>(
                            lq + ((size_t)((mt * NS + NS - 1 - y) * KS + ks) * 64 + lane) * 8);
                        sc[mt][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[0], q, sc[mt][0], 0, 0, 0);
                        sc[mt][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[1], q, sc[mt][1], 0, 0, 0);
                    }
            }
            const bool part = st * 32 + 32 > len || !f.ok[0] || !f.ok[1];  // some rows are hidden or absent
            unsigned there = 0xff;                                         // rows that exist, bit 4 t + i
            bool move = false;
            float mx[MT];
            if (part) {
                there = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (f.ok[e >> 2] && st * 32 + (e >> 2) * 16 + 4 * g + (e & 3) < total) there |= 1u << e;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int e = 0; e < 8; ++e) sc[mt][e >> 2][e & 3] *= sl;
                if (part) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int j = st * 32 + (e >> 2) * 16 + 4 * g + (e & 3) - len;  // row of the call, if >= 0
                        const bool vis = ((there >> e) & 1) && (j < 0 || ((see[mt] >> (j & 63)) & 1));
                        sc[mt][e >> 2][e & 3] = vis ? sc[mt][e >> 2][e & 3] : -INFINITY;
                    }
                }
                mx[mt] = fmaxf(fmaxf(fmaxf(sc[mt][0][0], sc[mt][0][1]), fmaxf(sc[mt][0][2], sc[mt][0][3])),
                               fmaxf(fmaxf(sc[mt][1][0], sc[mt][1][1]), fmaxf(sc[mt][1][2], sc[mt][1][3])));
                move |= mx[mt] > m[mt] + kSlack;
            }
            if (__any(move)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    float v = fmaxf(mx[mt], m[mt]);
                    v = fmaxf(v, __shfl_xor(v, 16));
                    v = fmaxf(v, __shfl_xor(v, 32));
                    const float k = __builtin_amdgcn_exp2f(m[mt] - v);
                    m[mt] = v;
                    l[mt] *= k;
#pragma unroll
                    for (int i = 0; i < C; ++i) o[mt][i] *= k;
                }
            }
            bf16x8 pb[MT][NS];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float p[8], sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    p[e] = __builtin_amdgcn_exp2f(sc[mt][e >> 2][e & 3] - m[mt]);
                    sum += p[e];
                }
                l[mt] += sum;
#pragma unroll
                for (int y = 0; y < NS; ++y)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        pb[mt][y][e] = (__bf16)p[e];
                        if (y + 1 < NS) p[e] -= (float)pb[mt][y][e];
                    }
            }
            float vsc[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    unsigned e = (f.vs[t] >> (8 * b)) & 255u;
                    if (part) e = (there >> (4 * t + b)) & 1 ? e : 127u;  // whatever lies there is finite
                    vsc[t][b] = scale_of(e);
                }
#pragma unroll
            for (int p = 0; p < C / 2; ++p) {
                union {
                    unsigned w[4];
                    bf16x8 v;
                } lo2, hi2;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int b = 0; b < 4; b += 2) {
                        union {
                            bf16x2 h;
                            unsigned w;
                        } x0, x1;
                        const int i0 = b * (D / 32) + p, i1 = (b + 1) * (D / 32) + p;
                        auto cvt = [&](int i, float sv) {
                            switch (i & 3) {
                                case 0: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.v[t][i >> 2], sv, 0);
                                case 1: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.v[t][i >> 2], sv, 1);
                                case 2: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.v[t][i >> 2], sv, 2);
                                default: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(f.v[t][i >> 2], sv, 3);
                            }
                        };
                        x0.h = cvt(i0, vsc[t][b]);
                        x1.h = cvt(i1, vsc[t][b + 1]);
                        lo2.w[2 * t + b / 2] = __builtin_amdgcn_perm(x1.w, x0.w, 0x05040100u);
                        hi2.w[2 * t + b / 2] = __builtin_amdgcn_perm(x1.w, x0.w, 0x07060302u);
                    }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int y = NS - 1; y >= 0; --y) {
                        o[mt][2 * p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo2.v, pb[mt][y], o[mt][2 * p], 0, 0, 0);
                        o[mt][2 * p + 1] =
                            __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi2.v, pb[mt][y], o[mt][2 * p + 1], 0, 0, 0);
                    }
            }
        };

        const int se = st0 + n;
        Frag<D> f0, f1;
        int st = st0 + wave;
        if (st < se) load(st, f0);
        while (st < se) {
            if (st + kWaves < se) load(st + kWaves, f1);
            compute(st, f0);
            st += kWaves;
            if (st >= se) break;
            if (st + kWaves < se) load(st + kWaves, f0);
            compute(st, f1);
            st += kWaves;
        }

        // ---- the waves' results to one ----
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            l[mt] += __shfl_xor(l[mt], 16);
            l[mt] += __shfl_xor(l[mt], 32);
            if (g == 0) wm[wave][mt * 16 + c] = m[mt], wl[wave][mt * 16 + c] = l[mt];
        }
        __syncthreads();
        float mm[MT], ll[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            mm[mt] = kNone;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) mm[mt] = fmaxf(mm[mt], wm[w][mt * 16 + c]);
            ll[mt] = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) ll[mt] += wl[w][mt * 16 + c] * __builtin_amdgcn_exp2f(wm[w][mt * 16 + c] - mm[mt]);
            const float k = __builtin_amdgcn_exp2f(m[mt] - mm[mt]);
#pragma unroll
            for (int i = 0; i < C; ++i) o[mt][i] *= k;
        }
#pragma unroll
        for (int half = kWaves / 2; half >= 1; half >>= 1) {
            if (wave >= half && wave < 2 * half) {
                float *d = lo + (size_t)(wave - half) * MT * C * 256;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < C; ++i) reinterpret_cast<f32x4 *>(d)[(mt * C + i) * 64 + lane] = o[mt][i];
            }
            __syncthreads();
            if (wave < half) {
                const float *d = lo + (size_t)wave * MT * C * 256;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int i = 0; i < C; ++i) o[mt][i] += reinterpret_cast<const f32x4 *>(d)[(mt * C + i) * 64 + lane];
            }
            __syncthreads();
        }
        if (wave == 0) {
            const bool whole = n == steps;
            const size_t slot = (size_t)blockIdx.x * 2 + (st0 > 0 ? 0 : 1);
            float *ml = a.part + slot * BR * 2;
            float *po = a.part + (size_t)a.nwg * 2 * BR * 2 + slot * BR * D;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const int row = row0 + mt * 16 + c;
                if (row >= rows) continue;
                const float inv = ll[mt] > 0.f ? 1.f / ll[mt] : 0.f;
                const size_t at = ((size_t)(t0 + row / a.G) * a.Hq + h * a.G + row % a.G) * D;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int d = (4 * g + i) * C;
                    if (!whole) {
                        float *p = po + (size_t)(mt * 16 + c) * D + d;
#pragma unroll
                        for (int y = 0; y < C; y += 4)
                            *reinterpret_cast<f32x4 *>(p + y) = f32x4{o[mt][y][i], o[mt][y + 1][i], o[mt][y + 2][i], o[mt][y + 3][i]};
                    } else if (F32) {
                        float *p = (float *)a.out + at + d;
#pragma unroll
                        for (int y = 0; y < C; y += 4)
                            *reinterpret_cast<f32x4 *>(p + y) = f32x4{o[mt][y][i] * inv, o[mt][y + 1][i] * inv,
                                                                      o[mt][y + 2][i] * inv, o[mt][y + 3][i] * inv};
                    } else {
                        uint16_t *p = (uint16_t *)a.out + at + d;
#pragma unroll
                        for (int y = 0; y < C; y += 4) {
                            u32x2 z;
                            z[0] = f32_to_bf16_rne(o[mt][y][i] * inv) | ((unsigned)f32_to_bf16_rne(o[mt][y + 1][i] * inv) << 16);
                            z[1] = f32_to_bf16_rne(o[mt][y + 2][i] * inv) | ((unsigned)f32_to_bf16_rne(o[mt][y + 3][i] * inv) << 16);
                            *reinterpret_cast<u32x2 *>(p + y) = z;
                        }
                    }
                }
                if (!whole && g == 0) ml[2 * (mt * 16 + c)] = mm[mt], ml[2 * (mt * 16 + c) + 1] = ll[mt];
            }
        }
        x += n;
    }
}

// Joins the parts of a unit: one workgroup per unit and 16-row tile, 16
// threads a row.  A workgroup's part of a unit that began before it is its
// slot 0, of one that begins in it slot 1.
template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void combine_kernel(KvAttendArgs a) {
    const KvRows &r = a.r;
    const int BR = 16 * a.mt;
    long long all;
    const Units un = units_of(r, a.G, BR, all);
    const long long share = share_of(all, a.nwg);
    // the block's unit: units are counted over sequences in the same order
    const int lane = threadIdx.x & 63;
    int cnt = un.mb * r.Hkv, incl = cnt;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int v = __shfl_up(incl, d);
        if (lane >= d) incl += v;
    }
    const int unit_all = blockIdx.x / a.mt, mt = blockIdx.x % a.mt;
    const uint64_t in = __ballot(incl > unit_all);
    if (in == 0) return;
    const int s = __ffsll((unsigned long long)in) - 1;
    const int steps = __shfl(un.steps, s), rows = __shfl(un.rows, s), mbs = __shfl(un.mb, s);
    const int unit = unit_all - (__shfl(incl, s) - __shfl(cnt, s));
    const long long u0 = __shfl(un.incl, s) - (long long)steps * mbs * r.Hkv + (long long)unit * steps, u1 = u0 + steps;
    const int w0 = (int)(u0 / share), w1 = (int)((u1 - 1) / share);
    if (w0 == w1) return;
    const int h = unit / mbs, rb = mt * 16 + (threadIdx.x >> 4), row = (unit - h * mbs) * BR + rb;
    if (row >= rows) return;
    const float *ml = a.part;
    const float *po = a.part + (size_t)a.nwg * 2 * BR * 2;
    auto slot = [&](int w) { return (size_t)w * 2 + (u0 < (long long)w * share ? 0 : 1); };
    float m = kNone;
    for (int w = w0; w <= w1; ++w) m = fmaxf(m, ml[(slot(w) * BR + rb) * 2]);
    constexpr int E = D / 16;
    const int d = (threadIdx.x & 15) * E;
    float l = 0.f, o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
    for (int w = w0; w <= w1; ++w) {
        const size_t at = slot(w) * BR + rb;
        const float k = __builtin_amdgcn_exp2f(ml[at * 2] - m);
        l += k * ml[at * 2 + 1];
#pragma unroll
        for (int i = 0; i < E; i += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(po + at * D + d + i);
#pragma unroll
            for (int y = 0; y < 4; ++y) o[i + y] += k * v[y];
        }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const size_t at = ((size_t)(r.off[s] + row / a.G) * a.Hq + h * a.G + row % a.G) * D + d;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        if (F32)
            ((float *)a.out)[at + i] = o[i] * inv;
        else
            ((uint16_t *)a.out)[at + i] = f32_to_bf16_rne(o[i] * inv);
    }
}

template <int MT, int D, bool F32>
hipError_t attend_launch(const KvAttendArgs &a, hipStream_t s) {
    constexpr int lds = attend_lds_bytes<MT, D, F32>();
    if (lds > 65536) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(attend_kernel<MT, D, F32>),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, lds);
        if (e != hipSuccess) return e;
    }
    hipLaunchKernelGGL((attend_kernel<MT, D, F32>), dim3(a.nwg), dim3(kThreads), lds, s, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    int units = 0;
    for (int q = 0; q < a.r.nseq; ++q) units += a.r.Hkv * (((a.r.off[q + 1] - a.r.off[q]) * a.G + 16 * MT - 1) / (16 * MT));
    hipLaunchKernelGGL((combine_kernel<D, F32>), dim3(units * MT), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

template <int D, bool F32>
hipError_t attend_mt(const KvAttendArgs &a, hipStream_t s) {
    if (a.mt == 1) return attend_launch<1, D, F32>(a, s);
    if constexpr (max_mt(D, F32) >= 2)
        if (a.mt == 2) return attend_launch<2, D, F32>(a, s);
    if constexpr (max_mt(D, F32) >= 3)
        if (a.mt == 3) return attend_launch<3, D, F32>(a, s);
    if constexpr (max_mt(D, F32) >= 4)
        if (a.mt == 4) return attend_launch<4, D, F32>(a, s);
    return hipErrorInvalidValue;
}

template <int D, bool F32>
hipError_t append_launch(const KvAppendArgs &a, hipStream_t s) {
    const int rows = kWaves * (512 / D);
    hipLaunchKernelGGL((append_kernel<D, F32>), dim3((a.T + rows - 1) / rows, a.r.Hkv, 2), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv4_append(const KvAppendArgs &a, hipStream_t s) {
    switch (a.r.D) {
        case 64: return a.f32 ? append_launch<64, true>(a, s) : append_launch<64, false>(a, s);
        case 128: return a.f32 ? append_launch<128, true>(a, s) : append_launch<128, false>(a, s);
        default: return a.f32 ? append_launch<256, true>(a, s) : append_launch<256, false>(a, s);
    }
}

// Row blocks: as few as max_mt allows, of equal size.
size_t kv4_attend_plan(KvAttendArgs &a, int n_cu) {
    int most = 1;
    for (int s = 0; s < a.r.nseq; ++s) most = max(most, (a.r.off[s + 1] - a.r.off[s]) * a.G);
    const int tiles = (most + 15) / 16, cap = max_mt(a.r.D, a.f32);
    const int blocks = (tiles + cap - 1) / cap;
    a.mt = (tiles + blocks - 1) / blocks;
    a.nwg = n_cu * 2;
    return (size_t)a.nwg * 2 * 16 * a.mt * (a.r.D + 2) * 4;
}

hipError_t launch_kv4_attend(const KvAttendArgs &a, hipStream_t s) {
    switch (a.r.D) {
        case 64: return a.f32 ? attend_mt<64, true>(a, s) : attend_mt<64, false>(a, s);
        case 128: return a.f32 ? attend_mt<128, true>(a, s) : attend_mt<128, false>(a, s);
        default: return a.f32 ? attend_mt<256, true>(a, s) : attend_mt<256, false>(a, s);
    }
}

}  // namespace moe
