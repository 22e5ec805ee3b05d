// Host side of the serving operators: argument validation and launches.  No
// allocation, no synchronisation, no per-call state.
#include "serve.h"

#include <cmath>

#include "checks.h"

namespace {

using namespace moe;

// Parents inside each sequence: -1 for its first row, an earlier row for the others.
int check_parent(int nseq, const int *off, const int32_t *parent) {
    for (int s = 0; s < nseq; ++s)
        for (int j = 0; j < off[s + 1] - off[s]; ++j) {
            const int p = parent[off[s] + j];
            if (j == 0 ? p != -1 : (p < 0 || p >= j))
                return fail(MOE_EINVAL, "parent[%d]=%d: a sequence's row 0 has parent -1, row j one in [0, j)",
                            off[s] + j, p);
        }
    return MOE_OK;
}

// Validates what kv4_attend and its workspace query share and plans the launch.
int plan_attend(const moe_kv4_cache *c, const moe_kv4_rows *r, int T, int Hq, int dtype, moe::KvAttendArgs *a,
                size_t *need) {
    if (T < 1 || T > MOE_MAX_TOKENS) return fail(MOE_EINVAL, "T=%d outside [1, %d]", T, MOE_MAX_TOKENS);
    int rc = check_rows(c, r, T, &a->r);
    if (rc == MOE_OK) rc = check_dtype(dtype);
    if (rc != MOE_OK) return rc;
    if (Hq < 1 || Hq > 8192 || Hq % c->Hkv != 0)
        return fail(MOE_EINVAL, "Hq=%d must be a positive multiple of Hkv=%d, at most 8192", Hq, c->Hkv);
    a->T = T;
    a->Hq = Hq;
    a->G = Hq / c->Hkv;
    a->f32 = dtype == MOE_F32;
    *need = moe::kv4_attend_plan(*a, moe::device_cu_count());
    return MOE_OK;
}

int check_logits(int T, int Tmin, int Tmax, int V, int dtype) {
    if (T < Tmin || T > Tmax) return fail(MOE_EINVAL, "T=%d outside [%d, %d]", T, Tmin, Tmax);
    if (V < 1) return fail(MOE_EINVAL, "V=%d must be positive", V);
    if (V > (1 << 18)) return fail(MOE_ENOTSUP, "V=%d above 2^18", V);
    return check_dtype(dtype);
}

int sampling_args(const void *logits, int64_t stride, int T, int V, int dtype, const moe_sampling *f, void *ws,
                  size_t ws_bytes, moe::SampleArgs *a) {
    if (!logits) return fail(MOE_EINVAL, "logits is NULL");
    if (stride < V) return fail(MOE_EINVAL, "stride=%lld is below V=%d", (long long)stride, V);
    if (misaligned(logits, dtype == MOE_F32 ? 4 : 2)) return fail(MOE_EINVAL, "logits must be aligned to an element");
    if (!ws) return fail(MOE_EINVAL, "workspace is NULL");
    if (misaligned(ws, 256)) return fail(MOE_EINVAL, "workspace must be 256-byte aligned");
    const size_t need = moe::sample_ws_bytes(T, V);
    if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    *a = {logits, stride, T, V, dtype == MOE_F32, f ? f->temperature : nullptr, f ? f->top_p : nullptr,
          f ? f->min_p : nullptr, f ? f->top_k : nullptr, ws};
    return MOE_OK;
}

}  // namespace

extern "C" {

size_t kv4_cache_bytes(int32_t num_pages, int32_t page, int32_t Hkv, int32_t D) {
    if (check_cache_sizes(num_pages, page, Hkv, D) != MOE_OK) return 0;
    return (size_t)num_pages * Hkv * (page / 16) * 17 * D;
}

int kv4_append(const moe_kv4_cache *cache, const moe_kv4_rows *rows, const void *k, const void *v, int64_t k_stride,
               int64_t v_stride, int32_t T, int32_t dtype, const int32_t *path, const int32_t *count, void *k_out,
               void *v_out, void *stream) {
    if (T < 1 || T > (1 << 20)) return fail(MOE_EINVAL, "T=%d outside [1, 2^20]", T);
    moe::KvAppendArgs a{};
    int rc = check_rows(cache, rows, T, &a.r);
    if (rc == MOE_OK) rc = check_row_pointers(a.r);
    if (rc == MOE_OK) rc = check_dtype(dtype);
    if (rc != MOE_OK) return rc;
    const size_t esz = dtype == MOE_F32 ? 4 : 2;
    const int64_t row = (int64_t)a.r.Hkv * a.r.D;
    if (!k || !v) return fail(MOE_EINVAL, "k and v must be non-NULL");
    if ((rc = check_stride("k_stride", k_stride, row, esz)) != MOE_OK) return rc;
    if ((rc = check_stride("v_stride", v_stride, row, esz)) != MOE_OK) return rc;
    if ((path == nullptr) != (count == nullptr)) return fail(MOE_EINVAL, "path and count come together");
    if ((k_out == nullptr) != (v_out == nullptr)) return fail(MOE_EINVAL, "k_out and v_out come together");
    if (path && k_out) return fail(MOE_EINVAL, "k_out and v_out are given for whole calls, without path");
    if (misaligned(k, 16) || misaligned(v, 16) || misaligned(k_out, 16) || misaligned(v_out, 16))
        return fail(MOE_EINVAL, "k, v, k_out and v_out must be 16-byte aligned");
    a.k = k;
    a.v = v;
    a.ks = k_stride;
    a.vs = v_stride;
    a.path = path;
    a.count = count;
    a.k_out = k_out;
    a.v_out = v_out;
    a.T = T;
    a.f32 = dtype == MOE_F32;
    return launched(moe::launch_kv4_append(a, static_cast<hipStream_t>(stream)));
}

size_t kv4_attend_workspace_bytes(const moe_kv4_cache *cache, const moe_kv4_rows *rows, int32_t T, int32_t Hq,
                                  int32_t dtype) {
    moe::KvAttendArgs a{};
    size_t need = 0;
    if (plan_attend(cache, rows, T, Hq, dtype, &a, &need) != MOE_OK) return 0;
    return need;
}

int kv4_attend(const moe_kv4_cache *cache, const moe_kv4_rows *rows, const void *q, int64_t q_stride, int32_t T,
               int32_t Hq, int32_t dtype, float scale, const int32_t *parent, void *out, void *ws, size_t ws_bytes,
               void *stream) {
    moe::KvAttendArgs a{};
    size_t need = 0;
    int rc = plan_attend(cache, rows, T, Hq, dtype, &a, &need);
    if (rc == MOE_OK) rc = check_row_pointers(a.r);
    if (rc != MOE_OK) return rc;
    if (!q || !out) return fail(MOE_EINVAL, "q and out must be non-NULL");
    if ((rc = check_stride("q_stride", q_stride, (int64_t)Hq * a.r.D, a.f32 ? 4 : 2)) != MOE_OK) return rc;
    if (!std::isfinite(scale)) return fail(MOE_EINVAL, "scale must be finite");
    if (!ws) return fail(MOE_EINVAL, "workspace is NULL");
    if (misaligned(q, 16) || misaligned(out, 16) || misaligned(ws, 16))
        return fail(MOE_EINVAL, "q, out and the workspace must be 16-byte aligned");
    if (ws_bytes < need) return fail(MOE_EWORKSPACE, "workspace has %zu bytes, needs %zu", ws_bytes, need);
    if (parent && (rc = check_parent(a.r.nseq, a.r.off, parent)) != MOE_OK) return rc;
    for (int s = 0; s < a.r.nseq; ++s)
        for (int t = a.r.off[s], j = 0; t < a.r.off[s + 1]; ++t, ++j) {
            const int p = parent ? parent[t] : j - 1;
            a.anc[t] = (1ull << j) | (p >= 0 ? a.anc[a.r.off[s] + p] : 0ull);
        }
    a.q = q;
    a.qs = q_stride;
    a.out = out;
    a.part = static_cast<float *>(ws);
    a.scale = scale;
    return launched(moe::launch_kv4_attend(a, static_cast<hipStream_t>(stream)));
}

size_t sample_workspace_bytes(int32_t T, int32_t V) {
    if (check_logits(T, 0, 65535, V, MOE_F32) != MOE_OK) return 0;
    return moe::sample_ws_bytes(T, V);
}

int sample_tokens(const void *logits, int64_t stride, int32_t T, int32_t V, int32_t dtype, const moe_sampling *f,
                  const float *u, int32_t *token, float *prob, float *probs, void *ws, size_t ws_bytes,
                  void *stream) {
    int rc = check_logits(T, 0, 65535, V, dtype);
    if (rc != MOE_OK) return rc;
    if (T == 0) return MOE_OK;
    moe::SampleArgs a{};
    if ((rc = sampling_args(logits, stride, T, V, dtype, f, ws, ws_bytes, &a)) != MOE_OK) return rc;
    if (!u || !token) return fail(MOE_EINVAL, "u and token must be non-NULL");
    return launched(moe::launch_sample(a, u, token, prob, probs, static_cast<hipStream_t>(stream)));
}

int accept_drafts(const void *logits, int64_t stride, int32_t T, int32_t V, int32_t dtype, const moe_sampling *f,
                  const int32_t *tokens, int32_t nseq, const int32_t *seg_off, const int32_t *parent,
                  const float *draft_probs, const float *u, const float *u_final, int32_t *out, int32_t *path,
                  int32_t *count, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_logits(T, 1, MOE_MAX_TOKENS, V, dtype);
    if (rc != MOE_OK) return rc;
    moe::AcceptArgs c{};
    if ((rc = check_offsets(T, nseq, seg_off, c.off)) != MOE_OK) return rc;
    if (parent && (rc = check_parent(nseq, c.off, parent)) != MOE_OK) return rc;
    for (int s = 0; s < nseq; ++s)
        for (int j = 0; j < c.off[s + 1] - c.off[s]; ++j) {
            const int p = parent ? parent[c.off[s] + j] : j - 1;
            if (draft_probs && p != j - 1)
                return fail(MOE_ENOTSUP, "draft_probs are for chains: row %d has parent %d", c.off[s] + j, p);
            c.parent[c.off[s] + j] = (int8_t)(p < 0 ? -1 : c.off[s] + p);
        }
    moe::SampleArgs a{};
    if ((rc = sampling_args(logits, stride, T, V, dtype, f, ws, ws_bytes, &a)) != MOE_OK) return rc;
    if (!tokens || !u || !out || !path || !count)
        return fail(MOE_EINVAL, "tokens, u, out, path and count must be non-NULL");
    if ((draft_probs == nullptr) != (u_final == nullptr))
        return fail(MOE_EINVAL, "u_final comes with draft_probs");
    c.tokens = tokens;
    c.q = draft_probs;
    c.u = u;
    c.u_final = u_final;
    c.out = out;
    c.path = path;
    c.count = count;
    c.nseq = nseq;
    return launched(moe::launch_accept(a, c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
