// Pages of the 4-bit K/V cache: rows read back as dense K and V, and the page
// tables' bookkeeping (pages taken, shared, let go, moved together, copied).
// Layout and semantics in include/moe_verify.h.
#include "common.h"
#include "kv4.h"
#include "plan.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

// ---------------------------------------------------------------------------
// Read.  The inverse of append: a lane holds 8 consecutive elements of a row
// (4 code bytes in, 16 or 32 bytes out), a wave 512 / D consecutive rows of
// one head, kReadAhead times over so that its loads are under way together.
// Memory bounds it, cold: 100001 bf16 rows of 8 heads of 128 (109 MB read, 409 MB
// written) take 139 us (3.7 TB/s) where the pages come from HBM, 87 (5.9 TB/s)
// where they are still in the last-level cache.  The heads of the same rows run
// side by side, so that what is written lies together (one head after the other
// 148 us), and results are stored past the caches (through them 153; 155 instead of
// 87).  With 8 or 16 in the place of kReadAhead 141 and 149 us.
// ---------------------------------------------------------------------------
constexpr int kReadAhead = 4;

template <int D, bool F32>
__global__ __launch_bounds__(kThreads) void read_kernel(KvReadArgs a) {
    constexpr int LPR = D / 8, RPW = 64 / LPR, W = D / 32;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int h = blockIdx.x % a.r.Hkv;  // the heads of the same rows run side by side
    const bool isv = blockIdx.y != 0;
    const int l = lane % LPR;
    const int t0 = (blockIdx.x / a.r.Hkv * (kThreads / 64) + wave) * RPW * kReadAhead + lane / LPR;
    unsigned word[kReadAhead], sc[kReadAhead];
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
        const int t = t0 + u * RPW;
        word[u] = 0;  // code 0 of any scale: rows without a page are zeros
        sc[u] = 127;
        if (t >= a.T) continue;
        int s = 0;
        while (t >= a.r.off[s + 1]) ++s;
        const int64_t pos = (int64_t)max(a.r.len[s], 0) + (t - a.r.off[s]);
        const int64_t slot = pos >> a.r.page_shift;
        if (slot >= a.r.max_pages) continue;
        const int pid = a.r.table[(size_t)s * a.r.max_pages + slot];
        if (pid < 0 || pid >= a.r.num_pages) continue;
        const int in = (int)pos & ((1 << a.r.page_shift) - 1), i = in & 15;
        const uint8_t *tile =
            a.r.data + ((((size_t)pid * a.r.Hkv + h) << (a.r.page_shift - 4)) + (in >> 4)) * Tile<D>::kBytes;
        if (!isv) {
            word[u] = *reinterpret_cast<const unsigned *>(tile + Tile<D>::kK + i * (D / 2) + l * 4);
        } else {
            const uint8_t *v = tile + Tile<D>::kV + (64 * (i >> 2) + (i & 3)) * W;
            if (D == 64) {
                word[u] = *reinterpret_cast<const uint16_t *>(v + (2 * l) * 4 * W) |
                          (unsigned)*reinterpret_cast<const uint16_t *>(v + (2 * l + 1) * 4 * W) << 16;
            } else if (D == 128) {
                word[u] = *reinterpret_cast<const unsigned *>(v + l * 4 * W);
            } else {
                word[u] = *reinterpret_cast<const unsigned *>(v + (l >> 1) * 4 * W + (l & 1) * 4);
            }
        }
        sc[u] = tile[(isv ? Tile<D>::kVs : Tile<D>::kKs) + 16 * (l >> 2) + i];
    }
#pragma unroll
    for (int u = 0; u < kReadAhead; ++u) {
        const int t = t0 + u * RPW;
        if (t >= a.T) continue;
        const size_t o = ((size_t)t * a.r.Hkv + h) * D + l * 8;
        const float s = scale_of(sc[u]);
        void *dst = isv ? a.v : a.k;
        if constexpr (F32) {
            f32x4 y0, y1;
            dequant8_f32(word[u], s, y0, y1);
            f32x4 *p = reinterpret_cast<f32x4 *>((float *)dst + o);
            __builtin_nontemporal_store(y0, p);
            __builtin_nontemporal_store(y1, p + 1);
        } else {
            __builtin_nontemporal_store(__builtin_bit_cast(u32x4, dequant8(word[u], s)), reinterpret_cast<u32x4 *>((uint16_t *)dst + o));
        }
    }
}

// ---------------------------------------------------------------------------
// Page bookkeeping.  Lists of at most 64 sequences: one workgroup.  Everything is integers and chosen by rank, so
// results do not depend on the order in which atomics arrive.
// ---------------------------------------------------------------------------
constexpr int kBookThreads = 1024;
constexpr int kScan = 8;  // counts of a thread at a time in the search for free pages
constexpr int kAhead = 8;  // table entries of a lane at a time in the search for missing ones

struct Take {  // what the list's entries need, in LDS
    int need[kMaxSegments];      // fresh pages
    int start[kMaxSegments];     // rank of the first of them among the pages taken, -1: not served
    long long at[kMaxSegments];  // table index of the first
    int total;
    int wave[kBookThreads / 64];
};

// Number of free pages before this thread's run of the chunk at `base`, the
// mask of its free ones, and the chunk's number.
__device__ int free_before(const PoolArgs &a, int base, Take &t, unsigned &mask, int &all) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    mask = 0;
    const int p0 = base + threadIdx.x * kScan;
    int v[kScan];
#pragma unroll
    for (int i = 0; i < kScan; ++i)  // past the L1, which may hold older counts
        v[i] = p0 + i < a.num_pages ? __hip_atomic_load(a.refs + p0 + i, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 1;
#pragma unroll
    for (int i = 0; i < kScan; ++i) mask |= (unsigned)(v[i] <= 0) << i;
    const int mine = __popc(mask), incl = wave_incl_scan(mine);
    __syncthreads();  // the last chunk's sums are read
    if (lane == 63) t.wave[wave] = incl;
    __syncthreads();
    const int w = lane < kBookThreads / 64 ? t.wave[lane] : 0, before = wave_incl_scan(w) - w;
    all = wave_sum_int(w);
    return __builtin_amdgcn_readlane(before, __builtin_amdgcn_readfirstlane(wave)) + incl - mine;
}

// Gives entry i of the list its need[i] lowest free pages, the entries in
// order, each whole or not at all; writes them to table[at[i]...] with a count
// of 1 and sets start[i] (-1: not enough pages).
// Latency bounds it, 8192 counts a step: a page for each of 64 sequences takes 57 us in a pool of 8192
// pages, where few threads find all and look up whose they are, and 121 and 156 behind 60000 and 96000
// used pages, which both passes go over from page 0.
__device__ void take_pages(const PoolArgs &a, Take &t) {
    // This workgroup's atomics have arrived in the L2, which is all that its own later accesses need.
    // (A fence would write the whole L2 back as well: the
    // fork of a prompt into 15 then takes 25 us instead of 21.)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int lane = threadIdx.x & 63;
    // every wave for itself: how many pages are needed
    const int mine = lane < a.n ? t.need[lane] : 0;
    const long long sum = ((long long)wave_sum_int(mine >> 12) << 12) + wave_sum_int(mine & 4095);
    const int total = (int)(sum < a.num_pages ? sum : a.num_pages);
    unsigned mask = 0;
    int all = 0, found = 0, end = 0, rank = 0;
    for (int base = 0; base < a.num_pages && found < total; base += kBookThreads * kScan) {
        rank = found + free_before(a, base, t, mask, all);
        found += all;
        end = base + kBookThreads * kScan;
    }
    if (sum <= found) {  // all are served
        const int incl = wave_incl_scan(mine);  // sum <= num_pages
        if (threadIdx.x < a.n) t.start[lane] = incl - mine;
        if (threadIdx.x == 0) t.total = total;
    } else if (threadIdx.x == 0) {
        int used = 0;
        for (int i = 0; i < a.n; ++i) {
            const bool fits = t.need[i] <= found - used;
            t.start[i] = fits ? used : -1;
            if (fits) used += t.need[i];
        }
        t.total = used;
    }
    __syncthreads();
    const bool once = end <= kBookThreads * kScan;  // the last search's ranks are still there
    int before = 0;
    for (int base = 0; base < end && before < t.total; base += kBookThreads * kScan) {
        if (!once) rank = before + free_before(a, base, t, mask, all);
        for (int i = 0; i < kScan; ++i) {
            if (!((mask >> i) & 1)) continue;
            if (rank < t.total) {
                int e = 0;  // the entry whose run holds this rank
                for (int j = 0; j < a.n; ++j)
                    if (t.start[j] >= 0 && t.need[j] > 0 && t.start[j] <= rank) e = j;
                const int p = base + threadIdx.x * kScan + i;
                a.table[t.at[e] + (rank - t.start[e])] = p;
                a.refs[p] = 1;
            }
            ++rank;
        }
        before += all;
        __syncthreads();
    }
    __syncthreads();
}

__global__ __launch_bounds__(kBookThreads) void reserve_kernel(PoolArgs a) {
    __shared__ Take t;
    __shared__ int seq[kMaxSegments], want[kMaxSegments];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave == 0) {
        const int rows = lane < a.n ? a.rows[lane] : 0, s = lane < a.n ? a.dst[lane] : -1;
        const int64_t pages = ((int64_t)max(rows, 0) + (1 << a.page_shift) - 1) >> a.page_shift;
        bool ok = pages <= a.max_pages && s >= 0 && s < a.nseq;
        for (int j = 0; j < a.n; ++j) ok &= j >= lane || __builtin_amdgcn_readlane(s, j) != s;
        if (lane < a.n) seq[lane] = s, want[lane] = ok ? (int)pages : -1;
    }
    __syncthreads();
    for (int i = wave; i < a.n; i += kBookThreads / 64) {
        const int n = want[i];
        const int32_t *row = a.table + (size_t)(n > 0 ? seq[i] : 0) * a.max_pages;
        int run = max(n, 0), held = -1;  // leading entries that name a page, and the last that does
        for (int j0 = lane; j0 < n; j0 += 64 * kAhead) {
            int p[kAhead];
#pragma unroll
            for (int x = 0; x < kAhead; ++x) p[x] = j0 + 64 * x < n ? row[j0 + 64 * x] : -1;
#pragma unroll
            for (int x = 0; x < kAhead; ++x) {
                const int j = j0 + 64 * x;
                if (p[x] >= 0 && p[x] < a.num_pages) held = j;
                else run = min(run, j);
            }
        }
        for (int x = 32; x > 0; x >>= 1) run = min(run, __shfl_xor(run, x)), held = max(held, __shfl_xor(held, x));
        const bool gap = held > run;  // the pages behind it would be lost
        if (lane == 0) {
            if (gap) want[i] = -1;
            t.need[i] = gap ? 0 : max(n, 0) - run;
            t.at[i] = (long long)(n > 0 ? seq[i] : 0) * a.max_pages + run;
        }
    }
    take_pages(a, t);
    if (threadIdx.x < a.n) a.ok[threadIdx.x] = want[threadIdx.x] >= 0 && t.start[threadIdx.x] >= 0;
}

__global__ __launch_bounds__(kBookThreads) void fork_kernel(PoolArgs a) {
    __shared__ Take t;
    __shared__ int src[kMaxSegments], dst[kMaxSegments], full[kMaxSegments], last[kMaxSegments], valid[kMaxSegments];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (wave == 0) {
        const int rows = lane < a.n ? max(a.rows[lane], 0) : 0, page = 1 << a.page_shift;
        const int f = lane < a.n ? a.src[lane] : -1, to = lane < a.n ? a.dst[lane] : -1;
        const int64_t pages = ((int64_t)rows + page - 1) >> a.page_shift;
        bool ok = pages <= a.max_pages && f >= 0 && f < a.nseq && to >= 0 && to < a.nseq;
        for (int j = 0; j < a.n; ++j)
            ok &= __builtin_amdgcn_readlane(f, j) != to && (j >= lane || __builtin_amdgcn_readlane(to, j) != to);
        if (lane < a.n) {
            src[lane] = f, dst[lane] = to, valid[lane] = ok;
            full[lane] = rows >> a.page_shift;
            last[lane] = rows & (page - 1) ? 0 : -1;  // whether a page is filled in part
        }
    }
    __syncthreads();
    // the former pages of the slots that are filled are let go, the shared ones counted
    for (int i = wave; i < a.n; i += kBookThreads / 64) {
        int part = -1;
        bool ok = valid[i];
        const int32_t *from = a.table + (size_t)(ok ? src[i] : 0) * a.max_pages;
        if (ok) {  // whether the source holds all the rows; no entry of the list writes to a source
            const int pages = full[i] + (last[i] == 0);
            bool miss = false;
            for (int j0 = lane; j0 < pages; j0 += 64 * kAhead) {
                int p[kAhead];
#pragma unroll
                for (int x = 0; x < kAhead; ++x) p[x] = j0 + 64 * x < pages ? from[j0 + 64 * x] : 0;
#pragma unroll
                for (int x = 0; x < kAhead; ++x) miss |= p[x] < 0 || p[x] >= a.num_pages;
            }
            ok = !__any(miss);
        }
        if (ok) {
            int32_t *to = a.table + (size_t)dst[i] * a.max_pages;
            for (int j = lane; j < a.max_pages; j += 64) {
                const int old = to[j], p = j < full[i] ? from[j] : -1;
                if (old >= 0 && old < a.num_pages) atomicSub(a.refs + old, 1);
                if (p >= 0 && p < a.num_pages) atomicAdd(a.refs + p, 1);
                to[j] = p;
            }
            if (last[i] == 0) part = from[full[i]];
        }
        if (lane == 0) {
            valid[i] = ok;
            last[i] = part;
            t.need[i] = part >= 0;
            t.at[i] = (long long)(ok ? dst[i] : 0) * a.max_pages + full[i];
        }
    }
    take_pages(a, t);
    for (int i = wave; i < a.n; i += kBookThreads / 64) {
        if (!valid[i] || t.start[i] >= 0) continue;  // no page was left for this one: its slot stays empty
        int32_t *to = a.table + (size_t)dst[i] * a.max_pages;
        for (int j = lane; j < full[i]; j += 64) {
            const int p = to[j];
            if (p >= 0 && p < a.num_pages) atomicSub(a.refs + p, 1);
            to[j] = -1;
        }
    }
    if (tid < a.n) {
        const bool ok = valid[tid] && t.start[tid] >= 0;
        const bool copy = ok && last[tid] >= 0;
        a.pairs[2 * tid] = copy ? last[tid] : -1;
        a.pairs[2 * tid + 1] = copy ? a.table[t.at[tid]] : -1;
        a.ok[tid] = ok;
    }
}

__global__ __launch_bounds__(kThreads) void release_kernel(PoolArgs a) {
    const int i = blockIdx.y, s = a.dst[i];
    if (s < 0 || s >= a.nseq) return;
    const int64_t keep = ((int64_t)max(a.rows[i], 0) + (1 << a.page_shift) - 1) >> a.page_shift;
    int32_t *row = a.table + (size_t)s * a.max_pages;
    for (int64_t j = keep + blockIdx.x * kThreads + threadIdx.x; j < a.max_pages; j += (int64_t)gridDim.x * kThreads) {
        // a sequence listed twice: only one of the two takes the entry
        const int p = atomicExch(row + j, -1);
        if (p >= 0 && p < a.num_pages) atomicSub(a.refs + p, 1);
    }
}

// ---------------------------------------------------------------------------
// Compaction.  The i-th lowest free page takes the i-th highest used one
// while it lies below it: the fewest moves that leave the used pages together
// at the front, and no page is both read and written.  Two launches: ranks, then
// pairs, counts and tables; in a large pool the chunks' used pages before them.
// ---------------------------------------------------------------------------
constexpr int kPerThread = 16;
constexpr int kChunk = kThreads * kPerThread;  // pages of a workgroup
static_assert(kChunk == plan::kCompactChunk, "");
constexpr int kDirect = 16384;  // pages up to which every workgroup counts the used ones of all chunks for itself

__device__ __forceinline__ int block_sum(int v, int *part) {
    v = wave_sum_int(v);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    return part[0] + part[1] + part[2] + part[3];
}

__global__ __launch_bounds__(kThreads) void count_kernel(CompactArgs a) {
    __shared__ int part[kThreads / 64];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int p = blockIdx.x * kChunk + i * kThreads + threadIdx.x;
        n += p < a.num_pages && a.refs[p] > 0;
    }
    n = block_sum(n, part);
    if (threadIdx.x == 0) a.chunk[blockIdx.x] = n;
}

__global__ __launch_bounds__(kThreads) void rank_kernel(CompactArgs a) {
    constexpr int kWaves = kThreads / 64;
    static_assert(kPerThread * kWaves == 64, "one wave scans the counts of all 64 runs of 64 pages");
    __shared__ int part[2][kWaves], run[kPerThread * kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, p0 = blockIdx.x * kChunk + threadIdx.x;
    int v[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) v[i] = p0 + i * kThreads < a.num_pages ? a.refs[p0 + i * kThreads] : 0;
    int below = 0, all = 0;  // used pages of the chunks before this one, and of all
    if (a.num_pages <= kDirect) {
        for (int b = 0; b < a.num_pages; b += kChunk) {
            int x[kPerThread];
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) x[i] = b + i * kThreads + (int)threadIdx.x < a.num_pages ? a.refs[b + i * kThreads + threadIdx.x] : 0;
            int n = 0;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) n += x[i] > 0;
            all += n;
            below += b < (int)blockIdx.x * kChunk ? n : 0;
        }
    } else {
        for (int c = threadIdx.x; c < a.chunks; c += kThreads) {
            const int n = a.chunk[c];
            all += n;
            below += c < (int)blockIdx.x ? n : 0;
        }
    }
    uint64_t used[kPerThread];
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        used[i] = __ballot(v[i] > 0);
        if (lane == 0) run[i * kWaves + wave] = __popcll(used[i]);
    }
    all = block_sum(all, part[0]);
    below = block_sum(below, part[1]);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.chunk[a.chunks] = all;
    const int mine = run[lane], before = below + wave_incl_scan(mine) - mine;  // of run `lane`
#pragma unroll
    for (int i = 0; i < kPerThread; ++i) {
        const int p = p0 + i * kThreads;
        // used pages below p
        const int u = __shfl(before, i * kWaves + wave) + __popcll(used[i] & ((1ull << lane) - 1));
        if (p >= a.num_pages) continue;
        const bool is = (used[i] >> lane) & 1;
        const int rank = is ? all - 1 - u : p - u;  // from the top, or from the bottom
        a.rank[p] = is ? rank : -1;
        if (rank < a.most) (is ? a.high : a.low)[rank] = p;
    }
}

__global__ __launch_bounds__(kThreads) void move_kernel(CompactArgs a) {
    const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int used = a.chunk[a.chunks];
    const int most = min(a.most, min(used, a.num_pages - used));
    if (i < a.max_moves) {
        int from = -1, to = -1;
        if (i < most && a.low[i] < a.high[i]) {
            from = a.high[i];
            to = a.low[i];
            a.refs[to] = a.refs[from];
            a.refs[from] = 0;
        }
        a.pairs[2 * i] = from;
        a.pairs[2 * i + 1] = to;
    }
    if (i < (int64_t)a.nseq * a.max_pages) {
        const int p = a.table[i];
        if (p >= 0 && p < a.num_pages) {
            const int r = a.rank[p];
            if (r >= 0 && r < most && a.low[r] < p) a.table[i] = a.low[r];
        }
    }
}

// ---------------------------------------------------------------------------
// Copy.  A workgroup copies 16 KB of a page, four 16-byte loads a thread
// under way together.
// ---------------------------------------------------------------------------
constexpr int kPiece = 4 * kThreads * 16;

__global__ __launch_bounds__(kThreads) void copy_kernel(CopyArgs a) {
    const int64_t all = (int64_t)a.n * a.pieces;
    for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
        const int i = (int)(w / a.pieces);
        const size_t in = (size_t)(w - (int64_t)i * a.pieces) * kPiece;
        const int from = a.pairs[2 * (size_t)i], to = a.pairs[2 * (size_t)i + 1];
        if (from < 0 || from >= a.num_pages || to < 0 || to >= a.num_pages || from == to) continue;
        const uint8_t *s = a.data + (size_t)from * a.page_bytes;
        uint8_t *d = a.data + (size_t)to * a.page_bytes;
        u32x4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t at = in + (j * kThreads + threadIdx.x) * 16;
            if (at < a.page_bytes) v[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(s + at));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t at = in + (j * kThreads + threadIdx.x) * 16;
            if (at < a.page_bytes) __builtin_nontemporal_store(v[j], reinterpret_cast<u32x4 *>(d + at));
        }
    }
}

}  // namespace

hipError_t launch_kv4_read(const KvReadArgs &a, hipStream_t s) {
    const int rows = kThreads / 64 * (512 / a.r.D) * kReadAhead;
    const dim3 grid((a.T + rows - 1) / rows * a.r.Hkv, 2);
    void (*k)(KvReadArgs) = nullptr;
    if (a.r.D == 64) k = a.f32 ? read_kernel<64, true> : read_kernel<64, false>;
    else if (a.r.D == 128) k = a.f32 ? read_kernel<128, true> : read_kernel<128, false>;
    else k = a.f32 ? read_kernel<256, true> : read_kernel<256, false>;
    hipLaunchKernelGGL(k, grid, dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_reserve(const PoolArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(reserve_kernel, dim3(1), dim3(kBookThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_fork(const PoolArgs &a, hipStream_t s) {
    hipLaunchKernelGGL(fork_kernel, dim3(1), dim3(kBookThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_release(const PoolArgs &a, hipStream_t s) {
    const int x = (a.max_pages + 4 * kThreads - 1) / (4 * kThreads);
    hipLaunchKernelGGL(release_kernel, dim3(x < 256 ? x : 256, a.n), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

size_t compact_ws_bytes(int num_pages, int max_moves) { return plan::compact_bytes(num_pages, max_moves); }

hipError_t launch_compact(CompactArgs a, int32_t *ws, hipStream_t s) {
    a.most = plan::compact_most(a.num_pages, a.max_moves);
    a.chunks = (a.num_pages + kChunk - 1) / kChunk;
    a.chunk = ws;
    a.low = a.chunk + a.chunks + 1;
    a.high = a.low + a.most;
    a.rank = a.high + a.most;
    if (a.num_pages > kDirect) hipLaunchKernelGGL(count_kernel, dim3(a.chunks), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(rank_kernel, dim3(a.chunks), dim3(kThreads), 0, s, a);
    const int64_t n = (int64_t)a.nseq * a.max_pages > a.max_moves ? (int64_t)a.nseq * a.max_pages : a.max_moves;
    hipLaunchKernelGGL(move_kernel, dim3((unsigned)((n + kThreads - 1) / kThreads)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_copy_pages(CopyArgs a, hipStream_t s) {
    a.pieces = (int)((a.page_bytes + kPiece - 1) / kPiece);
    const int64_t all = (int64_t)a.n * a.pieces;
    hipLaunchKernelGGL(copy_kernel, dim3((unsigned)(all < 16384 ? all : 16384)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
