// Argument checks that the host sides of the serving operators share.
#pragma once

#include <cstdarg>
#include <cstdio>

#include "../../include/moe_verify.h"
#include "serve.h"

namespace moe {

inline int fail(int code, const char *fmt, ...) {
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return moe::set_error(code, msg);
}

inline bool misaligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

inline int launched(hipError_t err) {
    if (err != hipSuccess) return fail(MOE_EHIP, "kernel launch failed: %s", hipGetErrorString(err));
    return MOE_OK;
}

inline int check_offsets(int T, int nseq, const int32_t *off, int *out) {
    if (nseq < 1 || nseq > moe::kMaxSegments)
        return fail(MOE_EINVAL, "nseq=%d outside [1, %d]", nseq, moe::kMaxSegments);
    if (!off) return fail(MOE_EINVAL, "seg_off is NULL");
    if (off[0] != 0 || off[nseq] != T) return fail(MOE_EINVAL, "seg_off must run from 0 to T=%d", T);
    for (int s = 0; s <= nseq; ++s) {
        if (s > 0 && off[s] < off[s - 1]) return fail(MOE_EINVAL, "seg_off must not decrease");
        out[s] = off[s];
    }
    return MOE_OK;
}

inline int check_dtype(int dtype) {
    if (dtype != MOE_F32 && dtype != MOE_BF16) return fail(MOE_ENOTSUP, "dtype %d: float32 and bf16 are built", dtype);
    return MOE_OK;
}

inline int check_cache_sizes(int64_t num_pages, int page, int Hkv, int D) {
    if (num_pages < 1) return fail(MOE_EINVAL, "num_pages=%lld must be positive", (long long)num_pages);
    if (page < 16 || page > 4096 || (page & (page - 1)) != 0)
        return fail(MOE_EINVAL, "page=%d must be a power of two, 16 .. 4096", page);
    if (Hkv < 1 || Hkv > 1024) return fail(MOE_EINVAL, "Hkv=%d outside [1, 1024]", Hkv);
    if (D != 64 && D != 128 && D != 256) return fail(MOE_ENOTSUP, "D=%d: head sizes 64, 128 and 256 are built", D);
    return MOE_OK;
}

inline int check_rows(const moe_kv4_cache *c, const moe_kv4_rows *r, int T, moe::KvRows *o) {
    if (!c || !r) return fail(MOE_EINVAL, "cache and rows must be non-NULL");
    int rc = check_cache_sizes(c->num_pages, c->page, c->Hkv, c->D);
    if (rc != MOE_OK) return rc;
    if (r->max_pages < 1 || (int64_t)r->max_pages * c->page > (int64_t)INT32_MAX - (1 << 22))
        return fail(MOE_EINVAL, "max_pages=%d must be positive, and max_pages * page below 2^31 - 2^22", r->max_pages);
    rc = check_offsets(T, r->nseq, r->seg_off, o->off);
    if (rc != MOE_OK) return rc;
    o->data = static_cast<uint8_t *>(c->data);
    o->table = r->table;
    o->len = r->len;
    o->num_pages = c->num_pages;
    o->page_shift = __builtin_ctz((unsigned)c->page);
    o->Hkv = c->Hkv;
    o->D = c->D;
    o->max_pages = r->max_pages;
    o->nseq = r->nseq;
    return MOE_OK;
}

inline int check_row_pointers(const moe::KvRows &r) {
    if (!r.data || !r.table || !r.len) return fail(MOE_EINVAL, "cache data, table and len must be non-NULL");
    if (misaligned(r.data, 16)) return fail(MOE_EINVAL, "cache data must be 16-byte aligned");
    return MOE_OK;
}

inline int check_stride(const char *name, int64_t stride, int64_t row, size_t esz) {
    if (stride < row) return fail(MOE_EINVAL, "%s=%lld is below a row's %lld elements", name, (long long)stride, (long long)row);
    if ((stride * (int64_t)esz) % 16 != 0) return fail(MOE_EINVAL, "%s must be a multiple of 16 bytes", name);
    return MOE_OK;
}

}  // namespace moe
