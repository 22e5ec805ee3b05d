// The 4-bit K/V cache: quantisation of rows into pages, and the attention of
// the verified tokens over it.  Layout and formulas in include/moe_verify.h.
#include "common.h"
#include "kv4.h"
#include "serve.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

// float32 -> bf16 bits by the hardware's conversion: to nearest, ties to even,
// and NaN stays NaN whatever its payload.
__device__ __forceinline__ unsigned bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// ---------------------------------------------------------------------------
// Append.  One lane holds 8 consecutive elements of a row, so 4 lanes share a
// block's scale and D / 8 lanes a row; a wave takes 512 / D consecutive rows
// of one head (their V codes lie next to each other, 4 rows in 4 D / 2
// contiguous bytes).  K and V are the grid's z.  The hardware's conversion to
// e2m1 does the division by the scale, the rounding and the saturation: with
// compares instead, vector instructions bound it (46.5 us against 36.3 us).
// Now memory does: 16384 bf16 rows of 8 heads of 128 with the stored values
// returned (67 MB read, 67 MB and 17.8 MB written) take 36.3 us, 4.2 TB/s; a
// large copy reaches 4.8.  The 12 rows of a commit take 3.9 us, all latency.
// ---------------------------------------------------------------------------
// A code of 0 has no sign: the signs of the 8 codes of a word stay only where
// the magnitude is not 0.
__device__ __forceinline__ unsigned drop_negative_zeros(unsigned w) {
    const unsigned m = w & 0x77777777u, some = (m | (m >> 1) | (m >> 2)) & 0x11111111u;
    return m | (w & (some << 3));
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
    const size_t at = (size_t)src * (isv ? a.vs : a.ks) + (size_t)h * D + l * 8;
    f32x4 x0, x1;
    u32x4 raw;
    if constexpr (F32) {
        const f32x4 *p = reinterpret_cast<const f32x4 *>((const float *)(isv ? a.v : a.k) + at);
        x0 = p[0];
        x1 = p[1];
    } else {
        raw = *reinterpret_cast<const u32x4 *>((const uint16_t *)(isv ? a.v : a.k) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x0[2 * i] = __uint_as_float(raw[i] << 16), x0[2 * i + 1] = __uint_as_float(raw[i] & 0xffff0000u);
            x1[2 * i] = __uint_as_float(raw[2 + i] << 16), x1[2 * i + 1] = __uint_as_float(raw[2 + i] & 0xffff0000u);
        }
    }
    // NaN counts as 0: e2m1 has none, and the conversion would make a large number of it
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) nan |= x0[i] != x0[i] || x1[i] != x1[i];
    if (nan) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (!F32) {
                const f32x4 &x = i < 2 ? x0 : x1;
                const float lo = x[2 * (i & 1)], hi = x[2 * (i & 1) + 1];
                raw[i] &= (lo == lo ? 0xffffu : 0u) | (hi == hi ? 0xffff0000u : 0u);
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x0[i] = x0[i] == x0[i] ? x0[i] : 0.f;
            x1[i] = x1[i] == x1[i] ? x1[i] : 0.f;
        }
    }
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(x0[i]), fabsf(x1[i])));
    m = fmaxf(m, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(m), 0xB1, 0xF, 0xF, false)));  // of the quad
    m = fmaxf(m, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(m), 0x4E, 0xF, 0xF, false)));
    // the smallest n with m <= 6 * 2^n = 1.5 * 2^(n + 2)
    const unsigned mb = __float_as_uint(m);
    int e = (int)(mb >> 23) - 127 - 2 + ((mb & 0x7fffffu) > 0x400000u);
    e = min(max(e, -100), 125);
    // the conversion divides by the scale, rounds to nearest (ties to the even code) and saturates
    const float sc = scale_of(127 + e);
    unsigned word = 0;
    if constexpr (F32) {
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, x0[0], x0[1], sc, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, x0[2], x0[3], sc, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, x1[0], x1[1], sc, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, x1[2], x1[3], sc, 3);
    } else {
        union {
            u32x4 u;
            bf16x2 h[4];
        } b;
        b.u = raw;
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, b.h[0], sc, 0);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, b.h[1], sc, 1);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, b.h[2], sc, 2);
        word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, b.h[3], sc, 3);
    }
    word = drop_negative_zeros(word);
    if (a.k_out) {  // 2 significant bits and a power of two: exact in either type
        const size_t o = ((size_t)t * a.r.Hkv + h) * D + l * 8;
        void *dst = isv ? a.v_out : a.k_out;
        if constexpr (F32) {
            f32x4 *p = reinterpret_cast<f32x4 *>((float *)dst + o);
            f32x4 y0, y1;
            dequant8_f32(word, sc, y0, y1);
            p[0] = y0;
            p[1] = y1;
        } else {
            *reinterpret_cast<bf16x8 *>((uint16_t *)dst + o) = dequant8(word, sc);
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
// workgroup worked on is joined by combine_kernel.  The lengths are the
// device's, so every workgroup lays the list out for itself.
//
// A step is two tiles of 16 cache rows, which each wave loads straight into a
// ring of its own in LDS, two steps ahead.  S^T = K Q^T leaves lane (g, c) =
// (l / 16, l % 16) with the scores of rows 4 g .. 4 g + 3 of both tiles for
// query c, which is just the operand that O^T += V^T P^T needs, so the
// probabilities never leave the lane; the running maximum and sum belong to
// column c in both products.  Codes become bf16 by
// v_cvt_scalef32_pk_bf16_fp4, exactly (2 significant bits and a power of two).
// The maximum is moved only when a score passes it by 2^8, so most steps need
// no exchange between lanes.
//
// For bf16 queries the probabilities are one bf16 term of the second product:
// each is off by 2^-9 of itself at most, so a result by 2^-9 of sum p |v|, about
// what rounding it to bf16 costs anyway (the sum l and the accumulators are
// float32).  Against 64 bits the results are 0.0018 to 0.0023 of their norm off,
// 0.0017 with a second term, which leaves the result's rounding alone but takes
// 73.5 us instead of 62 for the long tree below and 27.2 instead of 25.7 for 4 x
// 5 tokens.  float32 queries and their probabilities are three terms (24 bits).
//
// What bounds it: 60 query rows a head over 131086 rows of 8 heads of 128 (143
// MB) take 63 us (2.3 TB/s, 510 TFLOP/s); a step is 64 matrix and about 390
// vector instructions (codes to bf16, exponentials, sums), which keep the
// vector unit busy 57% and the matrix unit 30% of the time.  Few query rows
// over many cache rows are bound by memory: eight float32 rows a head over 600000
// rows (660 MB) take 147 us, 4.5 TB/s, where the loads alone take 126.  Short
// calls are latency: 200 rows take 6 us.  D = 256 has one wave a SIMD (its
// accumulators and operands take 288 registers) and one row tile, so that 64
// query rows a head read and convert every tile four times: 4 heads over 100000
// rows (109 MB) take 30.2 us for one row a head, 32.9 for 16 and 74.3 for 64,
// where 8 heads of 128 take 30.1, 31.4 and 53.6.  Matrix instructions on the codes
// themselves would need q in 8-bit terms and the probabilities without the
// rows' own scales, so the codes are converted.
// ---------------------------------------------------------------------------
constexpr float kNone = -3.402823466e38f;  // running maximum before the first score
constexpr float kSlack = 8.f;              // a score may pass the maximum by this (log2) before it moves
// Steps of a workgroup at least: one a wave.  (One sequence of 4000 rows, 4
// heads: 14.8 us, with 2 steps 16.9, with 8 15.3.)
constexpr int kMinShare = 4;
// What a second unit costs a workgroup (queries, first loads, the waves'
// exchange) in its steps.  (Shares that lie in one unit: 4 x 5 tokens over 23000
// rows 26.5 us, 31.3 without.)
constexpr int kSecondUnit = 8;

// The flat list: what sequence `lane` adds to it.
struct Units {
    int len, total, steps, rows, mb;  // rows before the call, all rows, steps, query rows, row blocks
    int span;                         // of a unit in the list: its steps, or those rounded up to whole shares
    long long incl;                   // running sum of spans over heads and row blocks
};

__device__ __forceinline__ long long lane_of(long long v, int lane) {
    return (long long)(((uint64_t)(unsigned)__builtin_amdgcn_readlane((int)(v >> 32), lane) << 32) |
                       (unsigned)__builtin_amdgcn_readlane((int)v, lane));
}

// Quotient of non-negative numbers, short where both are.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
    return a / b;
}

// The list, its length, and the steps of a workgroup: as few as nwg workgroups
// leave.  Where it costs less than kSecondUnit steps, shares are as much
// longer as it takes for each to lie in one unit.
__device__ __forceinline__ Units units_of(const KvRows &r, int G, int block_rows, int nwg, long long &share, long long &all) {
    const int lane = threadIdx.x & 63;
    Units u{0, 0, 0, 0, 0, 0, 0};
    if (lane < r.nseq) {
        const int n = r.off[lane + 1] - r.off[lane];
        const int cap = r.max_pages << r.page_shift;
        u.len = min(max(r.len[lane], 0), cap);
        u.total = min(u.len + n, cap);
        u.rows = n * G;
        u.mb = (u.rows + block_rows - 1) / block_rows;
        u.steps = (u.total + 31) >> 5;
    }
    // below 2^26 steps for each of 2^17 units: sums of 24 low bits and of the rest fit an int
    const int units = u.mb * r.Hkv;
    long long mine = (long long)u.steps * units;
    all = ((long long)wave_sum_int((int)(mine >> 24)) << 24) + wave_sum_int((int)(mine & 0xFFFFFF));
    const long long least = quotient(all + nwg - 1, nwg);
    share = least > kMinShare ? least : kMinShare;
    u.span = u.steps;
    if (share < 1 << 26 && wave_sum_int(units) <= nwg) {
        auto parts_of = [&](unsigned s) { return ((unsigned)u.steps + s - 1) / s; };
        auto count = [&](unsigned parts) { return wave_sum_int((int)parts * units); };  // all / s + units at most
        const unsigned most = (unsigned)share + kSecondUnit;
        unsigned s = (unsigned)share, parts = parts_of(most);
        if (count(parts) <= nwg) {
            while (s < most) {
                const unsigned p = parts_of(s);
                const int sum = count(p);
                if (sum <= nwg) {
                    parts = p;
                    break;
                }
                s = min(max(s + 1, (unsigned)quotient((long long)s * sum, nwg)), most);
            }
            u.span = (int)(parts * s);
            share = s;
        }
    }
    mine = (long long)u.span * units;
    const int lo = wave_incl_scan((int)(mine & 0xFFFFFF)), hi = wave_incl_scan((int)(mine >> 24));
    u.incl = ((long long)hi << 24) + lo;
    all = lane_of(u.incl, 63);
    return u;
}

// row / G for a row of a sequence (row / G < 64, G <= 8192): the quotient of the
// half next to it lies 2^-14 at least from a whole number, and its error is
// below 2^-16.
__device__ __forceinline__ int token_of(int row, float inv_g) { return (int)(((float)row + 0.5f) * inv_g); }

// Values of one step in a lane's registers.
template <int D>
struct Frag {
    static constexpr int W = D / 32;  // words of a lane: D / 4 K elements, or 4 rows of D / 16 V elements
    unsigned k[2][W], v[2][W], vs[2];
    unsigned ks[2];  // one byte, or two for D = 256
};

// From the step's two tiles in LDS at byte `at` into registers.  The loads
// that fill LDS are counted by hand, so the reads are written out: the
// compiler would wait for every one of them that is under way.
template <int D>
__device__ __forceinline__ void read_frag(Frag<D> &f, unsigned at) {
    const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
    const unsigned ka = at + c * (D / 2) + g * (D / 8), va = at + lane * (D / 8);
    const unsigned ksa = at + c + 16 * (g * (D / 4) / 32), vsa = at + 16 * (c * (D / 16) / 32) + 4 * g;
    typedef Tile<D> T;
    if constexpr (D == 64) {
        u32x2 k0, k1, v0, v1;
        asm volatile(
            "ds_read_b64 %0, %8 offset:%12\n\tds_read_b64 %1, %8 offset:%13\n\t"
            "ds_read_u8 %4, %10 offset:%14\n\tds_read_u8 %5, %10 offset:%15\n\t"
            "ds_read_b64 %2, %9 offset:%16\n\tds_read_b64 %3, %9 offset:%17\n\t"
            "ds_read_b32 %6, %11 offset:%18\n\tds_read_b32 %7, %11 offset:%19\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(k0), "=&v"(k1), "=&v"(v0), "=&v"(v1), "=&v"(f.ks[0]), "=&v"(f.ks[1]), "=&v"(f.vs[0]), "=&v"(f.vs[1])
            : "v"(ka), "v"(va), "v"(ksa), "v"(vsa), "i"(T::kK), "i"(T::kBytes + T::kK), "i"(T::kKs), "i"(T::kBytes + T::kKs),
              "i"(T::kV), "i"(T::kBytes + T::kV), "i"(T::kVs), "i"(T::kBytes + T::kVs)
            : "memory");
#pragma unroll
        for (int i = 0; i < 2; ++i) f.k[0][i] = k0[i], f.k[1][i] = k1[i], f.v[0][i] = v0[i], f.v[1][i] = v1[i];
    } else if constexpr (D == 128) {
        u32x4 k0, k1, v0, v1;
        asm volatile(
            "ds_read_b128 %0, %8 offset:%12\n\tds_read_b128 %1, %8 offset:%13\n\t"
            "ds_read_u8 %4, %10 offset:%14\n\tds_read_u8 %5, %10 offset:%15\n\t"
            "ds_read_b128 %2, %9 offset:%16\n\tds_read_b128 %3, %9 offset:%17\n\t"
            "ds_read_b32 %6, %11 offset:%18\n\tds_read_b32 %7, %11 offset:%19\n\ts_waitcnt lgkmcnt(0)"
            : "=&v"(k0), "=&v"(k1), "=&v"(v0), "=&v"(v1), "=&v"(f.ks[0]), "=&v"(f.ks[1]), "=&v"(f.vs[0]), "=&v"(f.vs[1])
            : "v"(ka), "v"(va), "v"(ksa), "v"(vsa), "i"(T::kK), "i"(T::kBytes + T::kK), "i"(T::kKs), "i"(T::kBytes + T::kKs),
              "i"(T::kV), "i"(T::kBytes + T::kV), "i"(T::kVs), "i"(T::kBytes + T::kVs)
            : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) f.k[0][i] = k0[i], f.k[1][i] = k1[i], f.v[0][i] = v0[i], f.v[1][i] = v1[i];
    } else {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            u32x4 k0, k1, v0, v1;
            unsigned s0, s1;
            asm volatile(
                "ds_read_b128 %0, %7 offset:%11\n\tds_read_b128 %1, %7 offset:%12\n\t"
                "ds_read_u8 %4, %9 offset:%13\n\tds_read_u8 %5, %9 offset:%14\n\t"
                "ds_read_b128 %2, %8 offset:%15\n\tds_read_b128 %3, %8 offset:%16\n\t"
                "ds_read_b32 %6, %10 offset:%17\n\ts_waitcnt lgkmcnt(0)"
                : "=&v"(k0), "=&v"(k1), "=&v"(v0), "=&v"(v1), "=&v"(s0), "=&v"(s1), "=&v"(f.vs[t])
                : "v"(ka + t * T::kBytes), "v"(va + t * T::kBytes), "v"(ksa + t * T::kBytes), "v"(vsa + t * T::kBytes), "i"(T::kK),
                  "i"(T::kK + 16), "i"(T::kKs), "i"(T::kKs + 16), "i"(T::kV), "i"(T::kV + 16), "i"(T::kVs)
                : "memory");
            f.ks[t] = s0 | (s1 << 8);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f.k[t][i] = k0[i], f.k[t][4 + i] = k1[i], f.v[t][i] = v0[i], f.v[t][4 + i] = v1[i];
        }
    }
}

// Loads of a tile: 1 KB a wave each, the last one partial.
template <int D>
constexpr int kTileLoads = (Tile<D>::kBytes + 1023) / 1024;

// Waits until at most N loads of this wave are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(N) : "memory");
}

// Bits of the rows j .. j + 3 of the call in `see`; rows before the call
// (j < 0) are seen.
__device__ __forceinline__ unsigned four_seen(uint64_t see, int j) {
    const int n = min(max(-j, 0), 4);
    const unsigned before = (unsigned)(see << n) | ((1u << n) - 1u), from = (unsigned)(see >> min(max(j, 0), 63));
    return (j < 0 ? before : from) & 15u;
}

// Waits here for a loaded value: where it is used, the wait would be for the
// loads into LDS that came after it as well.
template <typename T>
__device__ __forceinline__ void settle(T &v) {
    asm volatile("" : "+v"(v));
}

// Workgroups of a compute unit, by the registers and the LDS they take, and
// the steps of a wave's ring that this leaves room for.  (Three with a ring of
// two steps against two with three, D = 128: the 600000 rows above 146 us
// against 154.  Twice the workgroups that run at once gain nothing anywhere.)
constexpr int groups(int MT, int D) { return D == 256 ? 1 : MT > 1 ? 2 : D == 128 ? 3 : 4; }
constexpr int stages(int MT, int D) { return D == 128 && MT == 1 ? 2 : 3; }

template <int MT, int D, bool F32>
constexpr int ring_offset() {  // the queries' operand terms lie before the rings
    return MT * 16 * D * 2 * (F32 ? 3 : 1);
}

template <int MT, int D, bool F32>
constexpr int attend_lds_bytes() {
    const int q = ring_offset<MT, D, F32>() + kWaves * stages(MT, D) * 2 * Tile<D>::kBytes, m = 2 * MT * 16 * D * 4;
    return q > m ? q : m;
}

// 16-row tiles of a row block: its MT * D / 4 accumulators a lane, with the
// float32 type's three-term operands beside them, have to fit the registers.
constexpr int max_mt(int D, bool f32) { return D == 64 ? 4 : D == 128 ? (f32 ? 2 : 4) : 1; }

// Whether the queries' operand terms stay in registers beside the accumulators
// over all steps of a unit, or come from LDS again in every step, two terms
// ahead of their products.  (All from LDS: the 600000 rows above 148 us instead
// of 146; all in registers with 4 row tiles: spills.)
constexpr int kAhead = 2;
template <int MT, int D, bool F32>
constexpr bool kQueriesStay = D == 256 || MT * (D / 8 * (F32 ? 3 : 1) + D / 4) <= 128;

template <int MT, int D, bool F32>
__global__ __launch_bounds__(kThreads, groups(MT, D)) void attend_kernel(KvAttendArgs a) {
    constexpr int NS = F32 ? 3 : 1;  // bf16 terms of q and of the probabilities
    constexpr int KS = D / 32;       // k steps of the first product
    constexpr int C = D / 16;        // row tiles of the second
    constexpr int BR = 16 * MT;
    constexpr int kStages = stages(MT, D);
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    __shared__ float wm[kWaves][BR], wl[kWaves][BR];
    uint16_t *lq = reinterpret_cast<uint16_t *>(lds);  // [MT][NS][KS][64][8]
    float *lo = reinterpret_cast<float *>(lds);        // [2][MT][C][4][64], after the steps
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int g = lane >> 4, c = lane & 15;
    const KvRows &r = a.r;
    uint8_t *ring = lds + ring_offset<MT, D, F32>() + wave * (kStages * 2 * Tile<D>::kBytes);
    const unsigned ring_at = (unsigned)(uintptr_t)(__attribute__((address_space(3))) uint8_t *)ring;

    long long share, all;
    const Units un = units_of(r, a.G, BR, a.nwg, share, all);
    const long long x0 = (long long)blockIdx.x * share;
    long long x = x0, xe = x0 + share < all ? x0 + share : all;
    // the sign is the queries'; above 0, so that hidden rows' -inf stays what it is, and by no
    // more than a subnormal number, which leaves all finite scores at 0
    const float sl = fmaxf(fabsf(a.scale) * 1.44269504088896341f, 1.4e-45f);
    const unsigned flip = a.scale < 0.f ? 0x8000u : 0u;
    const float inv_g = 1.f / (float)a.G;

    while (x < xe) {
        const int s = __ffsll((unsigned long long)__ballot(un.incl > x)) - 1;
        const int len = __builtin_amdgcn_readlane(un.len, s), total = __builtin_amdgcn_readlane(un.total, s);
        const int steps = __builtin_amdgcn_readlane(un.steps, s), rows = __builtin_amdgcn_readlane(un.rows, s);
        const int mbs = __builtin_amdgcn_readlane(un.mb, s);
        const long long end_s = lane_of(un.incl, s);
        const int span = __builtin_amdgcn_readlane(un.span, s);
        const long long rel = x - (end_s - (long long)span * mbs * r.Hkv);
        const int unit = __builtin_amdgcn_readfirstlane((int)quotient(rel, span));
        const int st0 = __builtin_amdgcn_readfirstlane((int)(rel - (long long)unit * span));
        const int h = unit / mbs, mb = unit - h * mbs;
        const int n = __builtin_amdgcn_readfirstlane((int)(xe - x < steps - st0 ? xe - x : steps - st0));
        const int row0 = mb * BR, t0 = r.off[s], se = st0 + n;

        // ---- loads of a step into stage `at` of the ring; whether its tiles are in the pool (2 bits) ----
        int slot0 = -64, pids = -1;  // page ids of 64 table entries from slot0 on, one a lane
        auto issue = [&](int st, int at) {
            unsigned ok = 0;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int tile = 2 * st + t, slot = tile >> (r.page_shift - 4);
                if (slot >= slot0 + 64 || slot < slot0) {
                    slot0 = slot;
                    pids = slot + lane < r.max_pages ? r.table[(size_t)s * r.max_pages + slot + lane] : -1;
                    settle(pids);
                }
                const int pid = __builtin_amdgcn_readlane(pids, slot - slot0);
                const bool in_pool = pid >= 0 && pid < r.num_pages;
                ok |= (unsigned)in_pool << t;
                const int in = tile & ((1 << (r.page_shift - 4)) - 1);
                const uint8_t *b = r.data + ((((size_t)(in_pool ? pid : 0) * r.Hkv + h) << (r.page_shift - 4)) + in) *
                                                Tile<D>::kBytes + lane * 16;
                uint8_t *d = ring + (at * 2 + t) * Tile<D>::kBytes;
#pragma unroll
                for (int i = 0; i < kTileLoads<D>; ++i)
                    if ((i + 1) * 1024 <= Tile<D>::kBytes || lane * 16 < Tile<D>::kBytes - i * 1024) load_lds16(b + i * 1024, d + i * 1024);
            }
            return ok;
        };

        uint64_t see[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int row = row0 + mt * 16 + c;
            see[mt] = row < rows ? a.anc[t0 + token_of(row, inv_g)] : 0;
            settle(see[mt]);
        }
        __syncthreads();  // the last unit's exchange is over
        unsigned pool = 0;  // 2 bits a step, the newest lowest
        int next = st0 + wave, put = 0;
#pragma unroll
        for (int i = 0; i < kStages - 1; ++i) {
            pool <<= 2;
            if (next < se) pool |= issue(next, put);
            next += kWaves;
            ++put;
        }

        // ---- the block's queries into LDS as bf16 operand terms ----
        for (int i = threadIdx.x; i < BR * (D / 8); i += kThreads) {
            const int mt = i / (16 * (D / 8)), ks = (i / 64) % KS, ln = i & 63;
            const int row = row0 + mt * 16 + (ln & 15), d = (ln >> 4) * (D / 4) + ks * 8;
            uint16_t *dst = lq + ((size_t)(mt * NS * KS + ks) * 64 + ln) * 8;
            u32x4 z[NS];
#pragma unroll
            for (int p = 0; p < NS; ++p) z[p] = u32x4{0, 0, 0, 0};
            if (row < rows) {
                const int tok = token_of(row, inv_g);
                const size_t at = (size_t)(t0 + tok) * a.qs + (size_t)(h * a.G + row - tok * a.G) * D + d;
                if (F32) {
                    const f32x4 *p = reinterpret_cast<const f32x4 *>((const float *)a.q + at);
                    const f32x4 p0 = p[0], p1 = p[1];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float v = e < 4 ? p0[e & 3] : p1[e & 3];
#pragma unroll
                        for (int y = 0; y < NS; ++y) {
                            const unsigned b = bf16_bits(v);
                            v -= bf16_to_f32((uint16_t)b);
                            z[y][e >> 1] |= (b ^ flip) << (16 * (e & 1));
                        }
                    }
                } else {
                    z[0] = *reinterpret_cast<const u32x4 *>((const uint16_t *)a.q + at);
#pragma unroll
                    for (int e = 0; e < 4; ++e) z[0][e] ^= flip | (flip << 16);
                }
            }
#pragma unroll
            for (int p = 0; p < NS; ++p) *reinterpret_cast<u32x4 *>(dst + (size_t)p * KS * 64 * 8) = z[p];
        }

        float m[MT], l[MT];
        f32x4 o[MT][C];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt] = kNone;
            l[mt] = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i) o[mt][i] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        lds_barrier();  // the queries are there; the loads go on
        constexpr bool kStay = kQueriesStay<MT, D, F32>;
        auto query = [&](int mt, int y, int ks) {
            return *reinterpret_cast<const bf16x8 *>(lq + ((size_t)((mt * NS + y) * KS + ks) * 64 + lane) * 8);
        };
        // term i of a step, in the order of the products: the smaller terms first
        constexpr int N = MT * NS * KS, NQ = kStay ? N : kAhead;
        auto term = [&](int i) { return query(i / NS % MT, NS - 1 - i % NS, i / (NS * MT)); };
        bf16x8 q[NQ];
        if constexpr (kStay) {
#pragma unroll
            for (int i = 0; i < NQ; ++i) q[i] = term(i);
        }

        int get = 0;
        for (int st = st0 + wave; st < se; st += kWaves) {
            pool <<= 2;
            if (next < se) {
                pool |= issue(next, put);
                wait_loads<(kStages - 1) * 2 * kTileLoads<D>>();
            } else {
                wait_loads<0>();
            }
            next += kWaves;
            put = put + 1 == kStages ? 0 : put + 1;
            if constexpr (!kStay) {
#pragma unroll
                for (int i = 0; i < NQ; ++i) q[i] = term(i);
            }
            Frag<D> f;
            read_frag<D>(f, ring_at + get * 2 * Tile<D>::kBytes);
            get = get + 1 == kStages ? 0 : get + 1;

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
                        const int i = (ks * MT + mt) * NS + y;
                        bf16x8 &qf = q[i % NQ];
                        sc[mt][0] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[0], qf, sc[mt][0], 0, 0, 0);
                        sc[mt][1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[1], qf, sc[mt][1], 0, 0, 0);
                        if constexpr (!kStay)
                            if (i + NQ < N) {
                                qf = term(i + NQ);
                                __builtin_amdgcn_sched_barrier(6);  // only other ALU work moves across
                            }
                    }
            }
            const unsigned ok = (pool >> (2 * (kStages - 1))) & 3u;
            const bool part = st * 32 + 32 > len || ok != 3u;  // some rows are hidden or absent
            bool move = false;
            float mx[MT];
            if (part) {
                // bit 4 t + i: row 4 g + i of tile t exists
                const int left0 = total - st * 32 - 4 * g, left1 = left0 - 16;
                const unsigned there = ((ok & 1u) ? (1u << min(max(left0, 0), 4)) - 1u : 0u) |
                                       ((ok & 2u) ? ((1u << min(max(left1, 0), 4)) - 1u) << 4 : 0u);
                const int j0 = st * 32 + 4 * g - len, j1 = j0 + 16;  // rows of the call, if >= 0
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const unsigned vis = there & (four_seen(see[mt], j0) | (four_seen(see[mt], j1) << 4));
#pragma unroll
                    for (int e = 0; e < 8; ++e) sc[mt][e >> 2][e & 3] = (vis >> e) & 1u ? sc[mt][e >> 2][e & 3] : -INFINITY;
                }
                // whatever lies in absent rows becomes finite: scale bytes of 127
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    unsigned keep = 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) keep |= (there >> (4 * t + i)) & 1u ? 255u << (8 * i) : 0u;
                    f.vs[t] = (f.vs[t] & keep) | (0x7f7f7f7fu & ~keep);
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const float v = fmaxf(fmaxf(fmaxf(sc[mt][0][0], sc[mt][0][1]), fmaxf(sc[mt][0][2], sc[mt][0][3])),
                                      fmaxf(fmaxf(sc[mt][1][0], sc[mt][1][1]), fmaxf(sc[mt][1][2], sc[mt][1][3])));
                mx[mt] = v == -INFINITY ? kNone : v * sl;
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
                    p[e] = __builtin_amdgcn_exp2f(fmaf(sc[mt][e >> 2][e & 3], sl, -m[mt]));
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
                for (int b = 0; b < 4; ++b) vsc[t][b] = scale_of((f.vs[t] >> (8 * b)) & 255u);
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
            if (half > 1) __syncthreads();
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
                const int tok = token_of(row, inv_g);
                const size_t at = ((size_t)(t0 + tok) * a.Hq + h * a.G + row - tok * a.G) * D;
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
                            z[0] = bf16_bits(o[mt][y][i] * inv) | (bf16_bits(o[mt][y + 1][i] * inv) << 16);
                            z[1] = bf16_bits(o[mt][y + 2][i] * inv) | (bf16_bits(o[mt][y + 3][i] * inv) << 16);
                            *reinterpret_cast<u32x2 *>(p + y) = z;
                        }
                    }
                }
                if (!whole && g == 0) ml[2 * (mt * 16 + c)] = mm[mt], ml[2 * (mt * 16 + c) + 1] = ll[mt];
            }
        }
        x += xe - x < span - st0 ? xe - x : span - st0;
    }
}

// Joins the parts of a unit, one workgroup a query row of it: lane i of every
// wave takes the statistics of part i, the waves take the parts in turn.  A
// workgroup's part of a unit that began before it is its slot 0, of one that
// begins in it slot 1.  64 parts of each of 480 rows take 6.5 us: the latency
// of the list, the statistics and two rounds of parts (9.9 us with one load at
// a time).
template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void combine_kernel(KvAttendArgs a) {
    constexpr int E = D / 64;  // elements of a lane
    __shared__ float sum[kWaves][D];
    const KvRows &r = a.r;
    const int BR = 16 * a.mt, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    long long share, all;
    const Units un = units_of(r, a.G, BR, a.nwg, share, all);
    // the block's row: rows are counted over sequences and heads
    const int cnt = un.rows * r.Hkv, incl = wave_incl_scan(cnt);
    const uint64_t in = __ballot(incl > (int)blockIdx.x);
    if (in == 0) return;
    const int s = __ffsll((unsigned long long)in) - 1;
    const int steps = __builtin_amdgcn_readlane(un.steps, s), rows = __builtin_amdgcn_readlane(un.rows, s);
    const int mbs = __builtin_amdgcn_readlane(un.mb, s);
    const int rel = (int)blockIdx.x - (__builtin_amdgcn_readlane(incl, s) - __builtin_amdgcn_readlane(cnt, s));
    const int h = rel / rows, row = rel - h * rows, unit = h * mbs + row / BR, rb = row % BR;
    const int span = __builtin_amdgcn_readlane(un.span, s);
    const long long u0 = lane_of(un.incl, s) - (long long)span * mbs * r.Hkv + (long long)unit * span, u1 = u0 + steps;
    const int w0 = __builtin_amdgcn_readfirstlane((int)quotient(u0, share)), w1 = __builtin_amdgcn_readfirstlane((int)quotient(u1 - 1, share));
    if (w0 == w1) return;
    const float *ml = a.part;
    const float *po = a.part + (size_t)a.nwg * 2 * BR * 2 + lane * E;
    auto at = [&](int w) { return ((size_t)w * 2 + (w == w0 ? 1 : 0)) * BR + rb; };
    auto stats = [&](int w) { return w <= w1 ? *reinterpret_cast<const f32x2 *>(ml + at(w) * 2) : f32x2{kNone, 0.f}; };
    f32x2 ms = stats(w0 + lane);
    float m = ms[0];
    for (int w = w0 + 64 + lane; w <= w1; w += 64) m = fmaxf(m, ml[at(w) * 2]);
    m = wave_max(m);
    float l = 0.f, o[E];
#pragma unroll
    for (int i = 0; i < E; ++i) o[i] = 0.f;
    for (int b = w0; b <= w1; b += 64) {
        if (b > w0) ms = stats(b + lane);
        const float k = __builtin_amdgcn_exp2f(ms[0] - m);
        l += k * ms[1];
        const int n = min(64, w1 - b + 1);
        constexpr int kTogether = 8;  // loads under way: their latency is what this kernel takes
        for (int i0 = wave; i0 < n; i0 += kTogether * kWaves) {
            float p[kTogether][E];
#pragma unroll
            for (int y = 0; y < kTogether; ++y) {
                const float *from = po + at(b + min(i0 + y * kWaves, n - 1)) * D;
#pragma unroll
                for (int e = 0; e < E; ++e) p[y][e] = from[e];
            }
#pragma unroll
            for (int y = 0; y < kTogether; ++y) {
                const int i = i0 + y * kWaves;
                const float ki = i < n ? __int_as_float(__builtin_amdgcn_readlane(__float_as_int(k), i & 63)) : 0.f;
#pragma unroll
                for (int e = 0; e < E; ++e) o[e] += ki * p[y][e];
            }
        }
    }
    l = wave_sum(l);
#pragma unroll
    for (int e = 0; e < E; ++e) sum[wave][lane * E + e] = o[e];
    __syncthreads();
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const size_t to = ((size_t)(r.off[s] + row / a.G) * a.Hq + h * a.G + row % a.G) * D;
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += sum[w][d];
        if (F32)
            ((float *)a.out)[to + d] = v * inv;
        else
            ((uint16_t *)a.out)[to + d] = (uint16_t)bf16_bits(v * inv);
    }
}

template <int MT, int D, bool F32>
hipError_t attend_launch(const KvAttendArgs &a, hipStream_t s) {
    constexpr int lds = attend_lds_bytes<MT, D, F32>();
    static_assert(lds <= 160 * 1024 - 2 * kWaves * MT * 16 * 4, "one compute unit's LDS");
    hipError_t e = allow_lds<attend_kernel<MT, D, F32>>(lds);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attend_kernel<MT, D, F32>), dim3(a.nwg), dim3(kThreads), lds, s, a);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    hipLaunchKernelGGL((combine_kernel<D, F32>), dim3(a.T * a.Hq), dim3(kThreads), 0, s, a);
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

// Row blocks: as few as max_mt allows, of equal size.  Large ones read the
// cache less often, small ones begin and end a unit sooner: where the tables
// hold no more than 32 steps a workgroup, blocks of two tiles are faster (64
// rows a head, D = 128, 4 sequences: of 2000 rows 25.0 us against 32.1, of 8000
// 31.4 against 37.3; 40 rows a head: of 16000 rows 39.2 against 35.6).  The
// lengths are the device's, so the rule goes by the tables' width: a table much
// wider than its sequences takes the larger blocks (the 4 x 2000 rows in a table
// of 131072: 24.5 against 20.4, calls on one cache).
size_t kv4_attend_plan(KvAttendArgs &a, int n_cu) {
    int most = 1;
    for (int s = 0; s < a.r.nseq; ++s) most = max(most, (a.r.off[s + 1] - a.r.off[s]) * a.G);
    const int tiles = (most + 15) / 16;
    const long long steps = ((((long long)a.r.max_pages << a.r.page_shift) + 31) / 32) * a.r.nseq * a.r.Hkv * ((tiles + 1) / 2);
    int cap = max_mt(a.r.D, a.f32);
    if (steps <= 32ll * n_cu * groups(2, a.r.D)) cap = min(cap, 2);
    const int blocks = (tiles + cap - 1) / cap;
    a.mt = (tiles + blocks - 1) / blocks;
    a.nwg = n_cu * groups(a.mt, a.r.D);  // what runs at once
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
