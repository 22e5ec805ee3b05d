// Host side of the operators for prompts: argument validation and launches.
// No allocation, no synchronisation, no per-call state.
#include "prompt.h"

#include <cmath>

#include "checks.h"

namespace {

using namespace moe;

int check_pool(const moe_kv4_pool *p, PoolArgs *a) {
    if (!p) return fail(MOE_EINVAL, "pool is NULL");
    if (!p->refs || !p->table) return fail(MOE_EINVAL, "refs and table must be non-NULL");
    if (p->num_pages < 1 || p->num_pages > (1 << 24)) return fail(MOE_EINVAL, "num_pages=%d outside [1, 2^24]", p->num_pages);
    if (p->page < 16 || p->page > 4096 || (p->page & (p->page - 1)) != 0)
        return fail(MOE_EINVAL, "page=%d must be a power of two, 16 .. 4096", p->page);
    if (p->nseq < 1 || p->nseq > (1 << 16)) return fail(MOE_EINVAL, "nseq=%d outside [1, 2^16]", p->nseq);
    if (p->max_pages < 1 || (int64_t)p->max_pages * p->page > (int64_t)INT32_MAX - (1 << 22))
        return fail(MOE_EINVAL, "max_pages=%d must be positive, and max_pages * page below 2^31 - 2^22", p->max_pages);
    if ((int64_t)p->nseq * p->max_pages > (1 << 30)) return fail(MOE_EINVAL, "nseq * max_pages above 2^30");
    if (misaligned(p->refs, 4) || misaligned(p->table, 4)) return fail(MOE_EINVAL, "refs and table must be 4-byte aligned");
    a->refs = p->refs;
    a->table = p->table;
    a->num_pages = p->num_pages;
    a->page_shift = __builtin_ctz((unsigned)p->page);
    a->nseq = p->nseq;
    a->max_pages = p->max_pages;
    return MOE_OK;
}

// Validates what prompt_attend and its workspace query share and plans the launch.
int plan_prompt(int nseq, const int32_t *q_off, const int32_t *k_off, int Hq, int Hkv, int D, int dtype, PromptArgs *a,
                size_t *need) {
    if (nseq < 1 || nseq > kMaxSegments) return fail(MOE_EINVAL, "nseq=%d outside [1, %d]", nseq, kMaxSegments);
    if (!q_off || !k_off) return fail(MOE_EINVAL, "q_off and k_off must be non-NULL");
    for (int i = 0; i < 2; ++i) {
        const int32_t *off = i ? k_off : q_off;
        const int T = off[nseq];
        if (T < 0 || T > (1 << 22)) return fail(MOE_EINVAL, "%s ends at %d, outside [0, 2^22]", i ? "k_off" : "q_off", T);
        const int rc = check_offsets(T, nseq, off, i ? a->k_off : a->q_off);
        if (rc != MOE_OK) return rc;
    }
    const int rc = check_dtype(dtype);
    if (rc != MOE_OK) return rc;
    if (Hkv < 1 || Hkv > 1024) return fail(MOE_EINVAL, "Hkv=%d outside [1, 1024]", Hkv);
    if (Hq < 1 || Hq > 8192 || Hq % Hkv != 0)
        return fail(MOE_EINVAL, "Hq=%d must be a positive multiple of Hkv=%d, at most 8192", Hq, Hkv);
    if (D != 64 && D != 128 && D != 256) return fail(MOE_ENOTSUP, "D=%d: head sizes 64, 128 and 256 are built", D);
    a->nseq = nseq;
    a->Hq = Hq;
    a->Hkv = Hkv;
    a->G = Hq / Hkv;
    a->D = D;
    a->f32 = dtype == MOE_F32;
    if (a->f32 && (int64_t)a->k_off[nseq] * Hkv * D >= ((int64_t)1 << 33))
        return fail(MOE_ENOTSUP, "float32 K and V of 2^33 elements or more");
    *need = prompt_plan(*a, device_cu_count());
    if (a->units >= 1 << 23) return fail(MOE_ENOTSUP, "rows and heads of one call above 2^23 blocks of 128 rows");
    return MOE_OK;
}

// Validates what moe_experts and its workspace query share.
int check_experts(const moe_layer *L, int T, int dtype, ExpertArgs *a) {
    size_t need = 0;
    int rc = verify_needs(L, 1, nullptr, &need);  // the layer's own checks
    if (rc == MOE_OK) rc = check_dtype(dtype);
    if (rc != MOE_OK) return rc;
    if (L->wdtype == MOE_F32) return fail(MOE_ENOTSUP, "float32 weights: bf16 and fp8 are built");
    if (T < 0 || T > (1 << 20)) return fail(MOE_EINVAL, "T=%d outside [0, 2^20]", T);
    a->T = T;
    a->H = L->H;
    a->I = L->I;
    a->E = L->E;
    a->k = L->k;
    a->fp8 = L->wdtype == MOE_FP8_E4M3;
    a->f32 = dtype == MOE_F32;
    a->shared = L->Wsh_gu != nullptr;
    a->W_gu = L->W_gu;
    a->W_d = L->W_d;
    a->Wsh_gu = L->Wsh_gu;
    a->Wsh_d = L->Wsh_d;
    a->s_gu = L->s_gu;
    a->s_d = L->s_d;
    a->ssh_gu = L->ssh_gu;
    a->ssh_d = L->ssh_d;
    if (!experts_fit(*a)) return fail(MOE_ENOTSUP, "T=%d tokens of this layer are more than one call's grid holds", T);
    return MOE_OK;
}

int check_list(int n) {
    if (n < 0 || n > kMaxSegments) return fail(MOE_EINVAL, "n=%d outside [0, %d]", n, kMaxSegments);
    return MOE_OK;
}

int check_moves(int max_moves) {
    if (max_moves < 1 || max_moves > (1 << 24)) return fail(MOE_EINVAL, "max_moves=%d outside [1, 2^24]", max_moves);
    return MOE_OK;
}

}  // namespace

extern "C" {

int kv4_read(const moe_kv4_cache *cache, const moe_kv4_rows *rows, void *k, void *v, int32_t T, int32_t dtype,
             void *stream) {
    if (T < 0 || T > (1 << 22)) return fail(MOE_EINVAL, "T=%d outside [0, 2^22]", T);
    KvReadArgs a{};
    int rc = check_rows(cache, rows, T, &a.r);
    if (rc == MOE_OK) rc = check_row_pointers(a.r);
    if (rc == MOE_OK) rc = check_dtype(dtype);
    if (rc != MOE_OK) return rc;
    if (T == 0) return MOE_OK;
    if ((int64_t)T * a.r.Hkv > (1 << 28)) return fail(MOE_ENOTSUP, "T * Hkv above 2^28");
    if (!k || !v) return fail(MOE_EINVAL, "k and v must be non-NULL");
    if (misaligned(k, 16) || misaligned(v, 16)) return fail(MOE_EINVAL, "k and v must be 16-byte aligned");
    a.k = k;
    a.v = v;
    a.T = T;
    a.f32 = dtype == MOE_F32;
    return launched(launch_kv4_read(a, static_cast<hipStream_t>(stream)));
}

int kv4_reserve(const moe_kv4_pool *pool, const int32_t *seq, const int32_t *rows, int32_t n, int32_t *ok, void *stream) {
    PoolArgs a{};
    int rc = check_pool(pool, &a);
    if (rc == MOE_OK) rc = check_list(n);
    if (rc != MOE_OK) return rc;
    if (n == 0) return MOE_OK;
    if (!seq || !rows || !ok) return fail(MOE_EINVAL, "seq, rows and ok must be non-NULL");
    a.n = n;
    a.dst = seq;
    a.rows = rows;
    a.ok = ok;
    return launched(launch_reserve(a, static_cast<hipStream_t>(stream)));
}

int kv4_fork(const moe_kv4_pool *pool, const int32_t *src, const int32_t *dst, const int32_t *rows, int32_t n,
             int32_t *pairs, int32_t *ok, void *stream) {
    PoolArgs a{};
    int rc = check_pool(pool, &a);
    if (rc == MOE_OK) rc = check_list(n);
    if (rc != MOE_OK) return rc;
    if (n == 0) return MOE_OK;
    if (!src || !dst || !rows || !pairs || !ok) return fail(MOE_EINVAL, "src, dst, rows, pairs and ok must be non-NULL");
    a.n = n;
    a.src = src;
    a.dst = dst;
    a.rows = rows;
    a.pairs = pairs;
    a.ok = ok;
    return launched(launch_fork(a, static_cast<hipStream_t>(stream)));
}

int kv4_release(const moe_kv4_pool *pool, const int32_t *seq, const int32_t *keep, int32_t n, void *stream) {
    PoolArgs a{};
    int rc = check_pool(pool, &a);
    if (rc == MOE_OK) rc = check_list(n);
    if (rc != MOE_OK) return rc;
    if (n == 0) return MOE_OK;
    if (!seq || !keep) return fail(MOE_EINVAL, "seq and keep must be non-NULL");
    a.n = n;
    a.dst = seq;
    a.rows = keep;
    return launched(launch_release(a, static_cast<hipStream_t>(stream)));
}

size_t kv4_compact_workspace_bytes(const moe_kv4_pool *pool, int32_t max_moves) {
    PoolArgs a{};
    if (check_pool(pool, &a) != MOE_OK || check_moves(max_moves) != MOE_OK) return 0;
    return compact_ws_bytes(a.num_pages, max_moves);
}

int kv4_compact(const moe_kv4_pool *pool, int32_t max_moves, int32_t *pairs, void *ws, size_t ws_bytes, void *stream) {
    PoolArgs a{};
    int rc = check_pool(pool, &a);
    if (rc == MOE_OK) rc = check_moves(max_moves);
    if (rc != MOE_OK) return rc;
    if (!pairs || !ws) return fail(MOE_EINVAL, "pairs and the workspace must be non-NULL");
    if (misaligned(ws, 4)) return fail(MOE_EINVAL, "the workspace must be 4-byte aligned");
    const size_t need = compact_ws_bytes(a.num_pages, max_moves);
    if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    CompactArgs c{};
    c.refs = a.refs;
    c.table = a.table;
    c.num_pages = a.num_pages;
    c.nseq = a.nseq;
    c.max_pages = a.max_pages;
    c.max_moves = max_moves;
    c.pairs = pairs;
    return launched(launch_compact(c, static_cast<int32_t *>(ws), static_cast<hipStream_t>(stream)));
}

int kv4_copy_pages(const moe_kv4_cache *cache, const int32_t *pairs, int32_t n, void *stream) {
    if (!cache) return fail(MOE_EINVAL, "cache is NULL");
    const int rc = check_cache_sizes(cache->num_pages, cache->page, cache->Hkv, cache->D);
    if (rc != MOE_OK) return rc;
    if (n < 0 || n > (1 << 24)) return fail(MOE_EINVAL, "n=%d outside [0, 2^24]", n);
    if (!cache->data) return fail(MOE_EINVAL, "cache data must be non-NULL");
    if (misaligned(cache->data, 16)) return fail(MOE_EINVAL, "cache data must be 16-byte aligned");
    if (n == 0) return MOE_OK;
    if (!pairs) return fail(MOE_EINVAL, "pairs is NULL");
    CopyArgs a{};
    a.data = static_cast<uint8_t *>(cache->data);
    a.page_bytes = (size_t)cache->Hkv * (cache->page / 16) * 17 * cache->D;
    a.pairs = pairs;
    a.num_pages = cache->num_pages;
    a.n = n;
    return launched(launch_copy_pages(a, static_cast<hipStream_t>(stream)));
}

size_t prompt_attend_workspace_bytes(int32_t nseq, const int32_t *q_off, const int32_t *k_off, int32_t Hq, int32_t Hkv,
                                     int32_t D, int32_t dtype) {
    PromptArgs a{};
    size_t need = 0;
    return plan_prompt(nseq, q_off, k_off, Hq, Hkv, D, dtype, &a, &need) == MOE_OK ? need : 0;
}

int prompt_attend(const void *q, const void *k, const void *v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                  int32_t nseq, const int32_t *q_off, const int32_t *k_off, int32_t Hq, int32_t Hkv, int32_t D,
                  int32_t dtype, float scale, void *out, void *ws, size_t ws_bytes, void *stream) {
    PromptArgs a{};
    size_t need = 0;
    int rc = plan_prompt(nseq, q_off, k_off, Hq, Hkv, D, dtype, &a, &need);
    if (rc != MOE_OK) return rc;
    const size_t esz = a.f32 ? 4 : 2;
    if ((rc = check_stride("q_stride", q_stride, (int64_t)Hq * D, esz)) != MOE_OK) return rc;
    if ((rc = check_stride("k_stride", k_stride, (int64_t)Hkv * D, esz)) != MOE_OK) return rc;
    if ((rc = check_stride("v_stride", v_stride, (int64_t)Hkv * D, esz)) != MOE_OK) return rc;
    if (k_stride > (1 << 24) || v_stride > (1 << 24)) return fail(MOE_ENOTSUP, "strides of k and v above 2^24 elements");
    if (!std::isfinite(scale)) return fail(MOE_EINVAL, "scale must be finite");
    if (a.q_off[nseq] == 0) return MOE_OK;
    if (!q || !out) return fail(MOE_EINVAL, "q and out must be non-NULL");
    if ((!k || !v) && a.k_off[nseq] > 0) return fail(MOE_EINVAL, "k and v must be non-NULL");
    if (!ws && need > 0) return fail(MOE_EINVAL, "workspace is NULL");
    if (misaligned(q, 16) || misaligned(k, 16) || misaligned(v, 16) || misaligned(out, 16) || misaligned(ws, 256))
        return fail(MOE_EINVAL, "q, k, v and out must be 16-byte, the workspace 256-byte aligned");
    if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    a.q = q;
    a.k = k;
    a.v = v;
    a.qs = q_stride;
    a.ks = k_stride;
    a.vs = v_stride;
    a.out = out;
    a.ws = ws;
    a.scale = scale;
    return launched(launch_prompt(a, static_cast<hipStream_t>(stream)));
}

int route_tokens(const float *logits, int64_t stride, int32_t T, int32_t E, int32_t k, int32_t *topk_idx, float *topk_w,
                 void *stream) {
    if (T < 0 || T > (1 << 24)) return fail(MOE_EINVAL, "T=%d outside [0, 2^24]", T);
    if (E < 1 || E > MOE_MAX_EXPERTS) return fail(MOE_EINVAL, "E=%d outside [1, %d]", E, MOE_MAX_EXPERTS);
    if (k < 1 || k > E || k > MOE_MAX_TOPK) return fail(MOE_EINVAL, "k=%d outside [1, min(E, %d)]", k, MOE_MAX_TOPK);
    if (stride < E) return fail(MOE_EINVAL, "stride=%lld is below E=%d", (long long)stride, E);
    if (T == 0) return MOE_OK;
    if (!logits || !topk_idx || !topk_w) return fail(MOE_EINVAL, "logits, topk_idx and topk_w must be non-NULL");
    return launched(launch_route_tokens(logits, stride, T, E, k, topk_idx, topk_w, static_cast<hipStream_t>(stream)));
}

size_t moe_experts_workspace_bytes(const moe_layer *layer, int32_t T, int32_t dtype) {
    ExpertArgs a{};
    return check_experts(layer, T, dtype, &a) == MOE_OK ? experts_ws_bytes(a) : 0;
}

int moe_experts(const moe_layer *layer, const void *x, int64_t x_stride, int32_t T, int32_t dtype,
                const int32_t *topk_idx, const float *topk_w, void *y, void *ws, size_t ws_bytes, void *stream) {
    ExpertArgs a{};
    int rc = check_experts(layer, T, dtype, &a);
    if (rc != MOE_OK) return rc;
    if ((rc = check_stride("x_stride", x_stride, a.H, a.f32 ? 4 : 2)) != MOE_OK) return rc;
    if (T == 0) return MOE_OK;
    if (!x || !topk_idx || !topk_w || !y || !ws) return fail(MOE_EINVAL, "x, topk_idx, topk_w, y and the workspace must be non-NULL");
    if (misaligned(x, 16) || misaligned(y, 16) || misaligned(ws, 256))
        return fail(MOE_EINVAL, "x and y must be 16-byte, the workspace 256-byte aligned");
    if (misaligned(a.W_gu, 16) || misaligned(a.W_d, 16) || misaligned(a.Wsh_gu, 16) || misaligned(a.Wsh_d, 16))
        return fail(MOE_EINVAL, "weights must be 16-byte aligned");
    const size_t need = experts_ws_bytes(a);
    if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    a.x = x;
    a.xs = x_stride;
    a.idx = topk_idx;
    a.w = topk_w;
    a.y = y;
    a.ws = ws;
    return launched(launch_experts(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
