// kv_host.h -- argument checks shared by the cache's entry points.
#pragma once

#include <cstdint>
#include <cstdio>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "kv_cache.cuh"

namespace clef {

inline int kv_fail(const char *what) {
    char text[200];
    snprintf(text, sizeof text, "invalid argument: %s", what);
    internal_set_error(text);
    return CLEF_ERR_INVALID_ARG;
}

inline bool kv_misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Checks a pool of `planes` planes and fills p.
inline int kv_pool_args(KvPool &p, int kind, void *codes, int64_t plane_bytes, float *scales, int64_t plane_scales,
                        int64_t planes, int64_t pages, int heads, int page, int dim) {
    if (kind != kKvInt8 && kind != kKvE4m3) return kv_fail("kind must be 0 (int8) or 1 (e4m3)");
    if (pages < 0 || pages > kKvMaxPages) return kv_fail("pages out of range");
    if (heads < 1 || heads > 1024) return kv_fail("heads must be in 1..1024");
    if (page != 16 && page != 32 && page != 64 && page != 128) return kv_fail("page must be 16, 32, 64 or 128 tokens");
    if (dim != 64 && dim != 128 && dim != 256) return kv_fail("dim must be 64, 128 or 256");
    const int64_t tile = (int64_t)heads * page * dim;
    if (planes > 1 && (plane_bytes < pages * tile || plane_bytes % 16 != 0 || plane_scales < pages * heads))
        return kv_fail("plane pitches must hold a plane (codes: a multiple of 16 bytes)");
    if (kv_misaligned(codes, 16) || kv_misaligned(scales, 4))
        return kv_fail("codes must be 16-byte and scales 4-byte aligned");
    p.codes = static_cast<uint8_t *>(codes);
    p.scales = scales;
    p.plane_codes = plane_bytes;
    p.plane_scales = plane_scales;
    p.pages = (int)pages;
    p.heads = heads;
    p.dim = dim;
    p.page = page;
    p.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    return CLEF_OK;
}

inline int kv_table_args(KvTable &t, const int32_t *table, int64_t ldt, int64_t seqs, int64_t width, const int32_t *lens) {
    if (seqs < 0 || seqs > kKvMaxSeqs) return kv_fail("sequences must be in 0..4096");
    if (width < 0 || width > kKvMaxWidth || ldt < width) return kv_fail("table width out of range, or its pitch is smaller");
    if (kv_misaligned(table, 4) || kv_misaligned(lens, 4)) return kv_fail("table and lens must be 4-byte aligned");
    t.table = table;
    t.lens = lens;
    t.ldt = ldt;
    t.seqs = (int)seqs;
    t.width = (int)width;
    return CLEF_OK;
}

}  // namespace clef
