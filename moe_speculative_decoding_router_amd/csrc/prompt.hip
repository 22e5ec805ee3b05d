// Attention of prompts: many query rows, causal, over dense K and V of packed
// sequences.  Semantics in include/moe_verify.h.
#include "common.h"
#include "dma.h"
#include "plan.h"

namespace moe {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kRows = 32 * kWaves;         // query rows of a workgroup, 32 a wave
static_assert(kRows == plan::kRows, "");
constexpr float kNone = -3.402823466e38f;  // running maximum before the first score
constexpr float kSlack = 8.f;              // a score may pass the maximum by this (log2) before it moves

// Keys of a step, and buffers of K and V tiles, by what LDS holds.
constexpr int tile_keys(int D, int NT) { return NT > 1 || D == 256 ? 32 : 64; }
constexpr int buffers(int D, int NT) { return NT > 1 && D == 256 ? 1 : 2; }
constexpr int groups(int D, int NT) { return NT > 1 ? 1 : 2; }  // workgroups of a compute unit
constexpr int tile_bytes(int D, int NT) { return tile_keys(D, NT) * D * 2; }  // of K or V, one term
constexpr int lds_bytes(int D, int NT) { return 2 * NT * tile_bytes(D, NT) * buffers(D, NT); }

// A tile lies in LDS as rows of D bf16 in 16-byte chunks.  The loads fill LDS in
// lane order, so rows cannot be padded; instead chunk c of row r lies at c ^
// swizzle(r), which spreads the reads of a wave over the banks: K rows are read
// 16 bytes a lane down 16 rows, V by the transposing read, 4 rows of 32 chunks' halves.
template <int D>
__device__ __forceinline__ int swizzle_k(int r) {
    return D == 64 ? ((r >> 1) ^ ((r & 1) << 2)) & 7 : r & 15;
}
template <int D>
__device__ __forceinline__ int swizzle_v(int r) {
    return D == 64 ? ((r & 1) << 2) ^ ((r & 2) ? 6 : 0) : ((r & 1) << 2) ^ ((r & 2) ? 10 : 0);
}

// What a workgroup works on.
struct Unit {
    int s, h, row0;  // sequence, query head, first row
    int n, m;        // rows and keys of the sequence
};

__device__ __forceinline__ Unit unit_of(const PromptArgs &a, int u) {
    Unit r;
    const int block = u / a.Hq, x = u - block * a.Hq;
    // workgroups go to the eight XCDs in turn: each gets neighbouring heads, which share K and V in its L2
    r.h = a.Hq % 8 == 0 ? (x & 7) * (a.Hq >> 3) + (x >> 3) : x;
    int s = 0;
    while (block >= a.blocks[s + 1]) ++s;
    r.s = s;
    r.n = a.q_off[s + 1] - a.q_off[s];
    r.m = a.k_off[s + 1] - a.k_off[s];
    r.row0 = (a.blocks[s + 1] - 1 - block) * kRows;  // the rows with the most keys first
    return r;
}

// float32 -> NT bf16 terms, each the rest's nearest.
template <int NT>
__device__ __forceinline__ void split(float v, __bf16 *t) {
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        t[i] = (__bf16)v;
        v -= (float)t[i];
    }
}

// K and V of the float32 type as three planes of bf16 terms, rows dense.
__global__ __launch_bounds__(kThreads) void split_kernel(const float *k, const float *v, int64_t ks, int64_t vs, int row,
                                                         int64_t rows, __bf16 *out) {
    const int64_t i = ((int64_t)blockIdx.x * kThreads + threadIdx.x) * 4;
    const int64_t r = i / row;
    if (r >= rows) return;
    const bool isv = blockIdx.y != 0;
    const f32x4 x = *reinterpret_cast<const f32x4 *>((isv ? v + r * vs : k + r * ks) + (i - r * row));
    __bf16 t[4][3];
#pragma unroll
    for (int e = 0; e < 4; ++e) split<3>(x[e], t[e]);
    typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int p = 0; p < 3; ++p) {
        const bf16x4 y = {t[0][p], t[1][p], t[2][p], t[3][p]};
        *reinterpret_cast<bf16x4 *>(out + ((int64_t)(isv ? 3 : 0) + p) * rows * row + i) = y;
    }
}

// ---------------------------------------------------------------------------
// One workgroup takes 128 query rows of a head, 32 a wave, and goes over their
// keys in steps of 64 (32 at D = 256 and for float32) with a running maximum
// and sum.  S^T = K Q^T leaves lane (half, c) with the scores of query c, keys
// 8 x + 4 half .. + 3 of each 32; O^T += V^T P^T takes its operand in just that order
// once V's rows are read in it too (ds_read_b64_tr_b16, which transposes 4 rows
// of 16 columns), so probabilities never leave the lane, and the maximum and sum belong
// to column c in both products.  The maximum moves only when a score passes it by
// 2^8, so most steps need no exchange between lanes.  K and V tiles come
// straight into LDS a step ahead; V is read before the softmax and K four products
// ahead, so that their latency is hidden.  Hidden keys are masked in the steps that
// hold some; a wave whose rows see none of a step's keys leaves it out.
//
// Probabilities are rounded to bf16 for the second product, each by at most 2^-8
// of itself, and the sum is taken of the rounded ones (two at a time, v_dot2): the
// results are off by 0.0020 to 0.0023 of their norm, plain float32 ones that are
// rounded to bf16 by 0.0016 to 0.0017.  float32 operands are three bf16 terms each
// (K and V in planes that split_kernel writes), of whose nine products the six
// above 2^-24 are taken: 1e-7 of the norm.
//
// What bounds it: matrix and vector instructions of the two workgroups of a
// compute unit hardly overlap.  12000 rows of six prompts, 64 heads on 4 of 128
// (614 GFLOP) take 620 to 671 us, 915 to 990 TFLOP/s, where a large bf16 product reaches 1352;
// matrix instructions are under way 50% of the cycles and vector instructions
// 46%, and each 32 rows read a step's whole K and V from LDS (61% of its rate).
// 64 rows a wave would halve that, at one wave a SIMD and with the softmax
// placed by hand.  Wave priorities, of the softmax over the products or the other
// way, cost 1% to 3%.  515 rows behind 60001 (508 GFLOP) take 553 to 600 us in three
// shares a unit.  At D = 256 float32 spills 219 registers a lane (4000 rows, 16 heads on 4: 1824 us, with
// D = 128 398, where six products at the large one's rate would take 582 and 291), bf16 three.
// ---------------------------------------------------------------------------
template <int D, int NT>
__global__ __launch_bounds__(kThreads, groups(D, NT)) void prompt_kernel(PromptArgs a) {
    constexpr int BK = tile_keys(D, NT), NB = buffers(D, NT), TB = tile_bytes(D, NT);
    constexpr int KS = D / 16;           // steps of the first product
    constexpr int DT = D / 32;           // row tiles of the second
    constexpr int KT = BK / 32;          // key tiles of a step
    constexpr int CPR = D / 8;           // chunks of a row
    constexpr int RPL = 64 / CPR;        // rows of a load
    constexpr int LPW = TB / 1024 / kWaves;  // loads of a wave, for K or V and a term
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];  // [NB][K: NT, V: NT][TB]
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int half = lane >> 5, c = lane & 31;
    const int part = blockIdx.y;
    const Unit u = unit_of(a, blockIdx.x);
    const int first = u.m - u.n;  // position of the sequence's row 0
    const int last = min(u.row0 + kRows, u.n) - 1 + first;  // of the block's last row: its last key
    const int steps = last < 0 ? 0 : last / BK + 1;
    const int s0 = (int)((int64_t)steps * part / a.parts), s1 = (int)((int64_t)steps * (part + 1) / a.parts);

    // ---- queries: the first product's B operand ----
    const int row = u.row0 + wave * 32 + c;
    const size_t tok = (size_t)a.q_off[u.s] + min(row, u.n - 1);
    const unsigned flip = a.scale < 0.f ? 0x80008000u : 0u;
    // above 0, so that hidden keys' -inf stays what it is, and by no more than a subnormal number,
    // which leaves all finite scores at 0
    const float sl = fmaxf(fabsf(a.scale) * 1.44269504088896341f, 1.4e-45f);
    bf16x8 q[NT][KS];
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        const size_t at = tok * a.qs + (size_t)u.h * D + ks * 16 + half * 8;
        if constexpr (NT == 1) {
            u32x4 x = *reinterpret_cast<const u32x4 *>((const uint16_t *)a.q + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] ^= flip;
            q[0][ks] = __builtin_bit_cast(bf16x8, x);
        } else {
            const f32x4 x0 = *reinterpret_cast<const f32x4 *>((const float *)a.q + at);
            const f32x4 x1 = *reinterpret_cast<const f32x4 *>((const float *)a.q + at + 4);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                __bf16 t[NT];
                const float v = e < 4 ? x0[e & 3] : x1[e & 3];
                split<NT>(flip ? -v : v, t);
#pragma unroll
                for (int p = 0; p < NT; ++p) q[p][ks][e] = t[p];
            }
        }
    }

    // ---- loads of a step's tiles ----
    const int hk = u.h / a.G;
    const uint16_t *kb, *vb;  // the sequence's row 0 of this head, term 0
    size_t kst, vst, plane;   // elements between rows, between terms
    if constexpr (NT == 1) {
        kst = a.ks, vst = a.vs, plane = 0;
        kb = (const uint16_t *)a.k + (size_t)a.k_off[u.s] * kst + (size_t)hk * D;
        vb = (const uint16_t *)a.v + (size_t)a.k_off[u.s] * vst + (size_t)hk * D;
    } else {
        kst = vst = (size_t)a.Hkv * D, plane = (size_t)a.k_off[a.nseq] * kst;
        kb = (const uint16_t *)a.ws + (size_t)a.k_off[u.s] * kst + (size_t)hk * D;
        vb = kb + 3 * plane;
    }
    const unsigned lds0 = lds_address(lds);
    unsigned ko[LPW], vo[LPW];  // byte offsets of a lane's chunks from the step's first row
#pragma unroll
    for (int j = 0; j < LPW; ++j) {
        const int r = (wave * LPW + j) * RPL + lane / CPR, ch = lane % CPR;
        ko[j] = (unsigned)(r * (int)kst + (ch ^ swizzle_k<D>(r)) * 8) * 2u;
        vo[j] = (unsigned)(r * (int)vst + (ch ^ swizzle_v<D>(r)) * 8) * 2u;
    }
    auto issue = [&](int step, int buf) {
        const uint16_t *kt = kb + (size_t)step * BK * kst, *vt = vb + (size_t)step * BK * vst;
        const unsigned at = lds0 + buf * (2 * NT * TB) + wave * LPW * 1024;
        const int over = step * BK + BK - u.m;  // rows behind the last key are copies of it
#pragma unroll
        for (int j = 0; j < LPW; ++j) {
            unsigned kj = ko[j], vj = vo[j];
            if (over > 0) {
                const int r = (wave * LPW + j) * RPL + lane / CPR, back = max(r - (BK - 1 - over), 0);
                kj -= (unsigned)(back * (int)kst) * 2u;
                vj -= (unsigned)(back * (int)vst) * 2u;
            }
#pragma unroll
            for (int p = 0; p < NT; ++p) {
                dma16(kt + p * plane, kj, at + p * TB + j * 1024);
                dma16(vt + p * plane, vj, at + (NT + p) * TB + j * 1024);
            }
        }
    };

    // ---- addresses of the operands inside a buffer ----
    const unsigned ka = c * (D * 2), kx = half ^ swizzle_k<D>(c);
    const int r4 = (lane & 15) >> 2;  // row of the four that a group of 16 lanes transposes
    const unsigned va = (4 * half + r4) * (D * 2) + 8 * (lane & 1);
    const unsigned vx = (2 * ((lane >> 4) & 1) + ((lane & 3) >> 1)) ^ swizzle_v<D>(r4);

    f32x16 o[DT];
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] = 0.f;
    float m = kNone, l = 0.f;
    const int sees = row + first;  // the last key of this lane's row
    const int wave_first = u.row0 + wave * 32 + first;  // of the wave's first row
    const int wave_last = min(u.row0 + wave * 32 + 31, u.n - 1) + first;
    const bool some = u.row0 + wave * 32 < u.n;

    if (s0 < s1) issue(s0, 0);
    int buf = 0;
    for (int st = s0; st < s1; ++st) {
        dma_wait<0>();
        dma_barrier();  // this step's tiles are there, and the last step's were read by all
        if (NB > 1 && st + 1 < s1) issue(st + 1, buf ^ 1);
        const uint8_t *b = lds + buf * (2 * NT * TB);
        if (some && st * BK <= wave_last) {  // some row of the wave sees a key of the step
            f32x16 s[KT];
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) s[t][i] = 0.f;
            auto key = [&](int x, int t, int ks) {
                return *reinterpret_cast<const bf16x8 *>(b + x * TB + t * 32 * D * 2 + ka + ((kx ^ (2 * ks)) << 4));
            };
            if constexpr (NT == 1) {  // keys kAhead products ahead
                constexpr int kAhead = 4;
                bf16x8 kf[kAhead];
#pragma unroll
                for (int i = 0; i < kAhead; ++i) kf[i] = key(0, i % KT, i / KT);
#pragma unroll
                for (int i = 0; i < KS * KT; ++i) {
                    s[i % KT] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i % kAhead], q[0][i / KT], s[i % KT], 0, 0, 0);
                    if (i + kAhead < KS * KT) kf[i % kAhead] = key(0, (i + kAhead) % KT, (i + kAhead) / KT);
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int y = NT - 1; y >= 0; --y)  // the smaller terms first
#pragma unroll
                        for (int x = NT - 1 - y; x >= 0; --x)
#pragma unroll
                            for (int ks = 0; ks < KS; ++ks)
                                s[t] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key(x, t, ks), q[y][ks], s[t], 0, 0, 0);
            }
            auto value = [&](int x, int kk, int d) {
                typedef __attribute__((address_space(3))) s16x4 *lp;
                const uint8_t *at = b + (NT + x) * TB + kk * 16 * D * 2 + va + ((vx ^ (4 * d)) << 4);
                const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(s16x4 *)at);
                const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(s16x4 *)(at + 8 * D * 2));
                const s16x8 vf = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                return __builtin_bit_cast(bf16x8, vf);
            };
            // where registers hold them, the values come while the probabilities are made
            constexpr bool kEarly = NT == 1 && D <= 128;
            bf16x8 vf[kEarly ? 2 * KT : 1][kEarly ? DT : 1];
            if constexpr (kEarly) {
#pragma unroll
                for (int kk = 0; kk < 2 * KT; ++kk)
#pragma unroll
                    for (int d = 0; d < DT; ++d) vf[kk][d] = value(0, kk, d);
                __builtin_amdgcn_sched_barrier(0);
            }
            if (st * BK + BK - 1 > wave_first) {  // some row of the wave does not see all keys
#pragma unroll
                for (int t = 0; t < KT; ++t)
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const int p = st * BK + t * 32 + 8 * (i >> 2) + 4 * half + (i & 3);
                        s[t][i] = p <= sees ? s[t][i] : -__builtin_inff();
                    }
            }
            float top = s[0][0];
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) top = fmaxf(top, s[t][i]);
            top *= sl;
            if (__any(top > m + kSlack)) {
                const auto sw = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
                const float to = fmaxf(m, fmaxf(__uint_as_float(sw[0]), __uint_as_float(sw[1])));
                const float f = __builtin_amdgcn_exp2f(m - to);
                m = to;
                l *= f;
#pragma unroll
                for (int d = 0; d < DT; ++d)
#pragma unroll
                    for (int i = 0; i < 16; ++i) o[d][i] *= f;
            }
            bf16x8 pb[NT][KT * 2];  // the second product's B operand
#pragma unroll
            for (int t = 0; t < KT; ++t)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float p = __builtin_amdgcn_exp2f(fmaf(s[t][i], sl, -m));
                    if (NT > 1) l += p;
                    __bf16 z[NT];
                    split<NT>(p, z);
#pragma unroll
                    for (int y = 0; y < NT; ++y) pb[y][2 * t + (i >> 3)][i & 7] = z[y];
                }
            if constexpr (NT == 1) {  // the sum of what enters the second product, two at a time
                const bf16x2 ones = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
                for (int x = 0; x < KT * 2; ++x)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        l = __builtin_amdgcn_fdot2_f32_bf16(bf16x2{pb[0][x][2 * i], pb[0][x][2 * i + 1]}, ones, l, false);
            }
            // lane slot j of half h in a 16-key product is key 8 (j / 4) + 4 h + j % 4 in both operands
#pragma unroll
            for (int y = NT - 1; y >= 0; --y)
#pragma unroll
                for (int x = NT - 1 - y; x >= 0; --x)
#pragma unroll
                    for (int kk = 0; kk < 2 * KT; ++kk)
#pragma unroll
                        for (int d = 0; d < DT; ++d) {
                            bf16x8 v;
                            if constexpr (kEarly) v = vf[kk][d];
                            else v = value(x, kk, d);
                            o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, pb[y][kk], o[d], 0, 0, 0);
                        }
        }
        if (NB == 1) {
            dma_barrier();
            if (st + 1 < s1) issue(st + 1, 0);
        } else {
            buf ^= 1;
        }
    }

    // ---- the halves' sums, and the result or the share of it ----
    const auto lw = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
    l = __uint_as_float(lw[0]) + __uint_as_float(lw[1]);
    if (row >= u.n) return;
    if (a.parts > 1) {
        float *w = (float *)((uint8_t *)a.ws + a.part_at) + (((size_t)blockIdx.x * a.parts + part) * kRows + wave * 32 + c) * (D + 2);
        if (half == 0) w[D] = m, w[D + 1] = l;
#pragma unroll
        for (int d = 0; d < DT; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f32x2 *p = reinterpret_cast<f32x2 *>(w + d * 32 + 8 * g + 4 * half);
                p[0] = f32x2{o[d][4 * g], o[d][4 * g + 1]};
                p[1] = f32x2{o[d][4 * g + 2], o[d][4 * g + 3]};
            }
        return;
    }
    // Zeros are for rows that see no key; a sum that is NaN, or 0 because every score is -inf, gives NaN.
    const float inv = 1.f / l;
    const size_t at = (tok * a.Hq + u.h) * D + 4 * half;
#pragma unroll
    for (int d = 0; d < DT; ++d)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            f32x4 y;
#pragma unroll
            for (int i = 0; i < 4; ++i) y[i] = sees >= 0 ? o[d][4 * g + i] * inv : 0.f;
            if constexpr (NT > 1) {
                *reinterpret_cast<f32x4 *>((float *)a.out + at + d * 32 + 8 * g) = y;
            } else {
                typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
                const bf16x4 z = {(__bf16)y[0], (__bf16)y[1], (__bf16)y[2], (__bf16)y[3]};
                *reinterpret_cast<bf16x4 *>((uint16_t *)a.out + at + d * 32 + 8 * g) = z;
            }
        }
}

// Joins the shares of a unit's rows: one wave a row, D / 64 elements a lane.
template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void join_kernel(PromptArgs a) {
    constexpr int E = D / 64;
    const int lane = threadIdx.x & 63;
    const int i = blockIdx.y * kWaves + (threadIdx.x >> 6);  // row of the block
    const Unit u = unit_of(a, blockIdx.x);
    if (u.row0 + i >= u.n) return;
    const float *w = (const float *)((const uint8_t *)a.ws + a.part_at) + ((size_t)blockIdx.x * a.parts * kRows + i) * (D + 2);
    const size_t step = (size_t)kRows * (D + 2);
    float m = kNone;
    for (int p = 0; p < a.parts; ++p) m = fmaxf(m, w[p * step + D]);
    float l = 0.f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.f;
    for (int p = 0; p < a.parts; ++p) {
        const float f = __builtin_amdgcn_exp2f(w[p * step + D] - m);
        l += f * w[p * step + D + 1];
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] += f * w[p * step + e * 64 + lane];
    }
    const int sees = u.row0 + i + u.m - u.n;  // the row's last key
    const size_t at = ((size_t)(a.q_off[u.s] + u.row0 + i) * a.Hq + u.h) * D + lane;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const float y = sees >= 0 ? o[e] / l : 0.f;  // as in prompt_kernel
        if constexpr (F32) ((float *)a.out)[at + e * 64] = y;
        else ((__bf16 *)a.out)[at + e * 64] = (__bf16)y;
    }
}

template <int D, int NT>
hipError_t launch(const PromptArgs &a, hipStream_t s) {
    constexpr int lds = lds_bytes(D, NT);
    if (lds > 65536) {
        const hipError_t e = allow_lds<prompt_kernel<D, NT>>(lds);
        if (e != hipSuccess) return e;
    }
    if (NT > 1) {
        const int64_t rows = a.k_off[a.nseq];
        const int64_t n = rows * a.Hkv * D / 4;
        if (n > 0)
            hipLaunchKernelGGL(split_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads), 2), dim3(kThreads), 0, s,
                               (const float *)a.k, (const float *)a.v, a.ks, a.vs, a.Hkv * D, rows, (__bf16 *)a.ws);
    }
    hipLaunchKernelGGL((prompt_kernel<D, NT>), dim3(a.units, a.parts), dim3(kThreads), lds, s, a);
    if (a.parts > 1)
        hipLaunchKernelGGL((join_kernel<D, (NT > 1)>), dim3(a.units, kRows / kWaves), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t prompt_plan(PromptArgs &a, int n_cu) { return plan::prompt(a, n_cu); }

hipError_t launch_prompt(const PromptArgs &a, hipStream_t s) {
    if (a.D == 64) return a.f32 ? launch<64, 3>(a, s) : launch<64, 1>(a, s);
    if (a.D == 128) return a.f32 ? launch<128, 3>(a, s) : launch<128, 1>(a, s);
    return a.f32 ? launch<256, 3>(a, s) : launch<256, 1>(a, s);
}

}  // namespace moe
