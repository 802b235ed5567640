// kv_cache.cuh -- the paged 8-bit cache as the kernels see it.
//
// A pool holds `pages` pages.  A page of one plane (a layer's keys or its
// values) is `page` tokens of every key/value head, stored [head][token][dim]
// in one byte each, with one fp32 scale for each head: value = code * scale.
// A sequence is a row of the page table and a length; its token i lives in
// page table[i / page] at place i % page.  Page indices, lengths and sequence
// numbers come from device memory, so the kernels check them: what is out of
// range is left out and reported through the status word.
#pragma once

#include <cstdint>

#include "clef_ptx.cuh"

namespace clef {

enum : unsigned int {
    kStatusBadPage = 5u,   // CLEF_ERR_BAD_PAGE
    kStatusNoPages = 6u,   // CLEF_ERR_NO_PAGES
};

enum KvKind : int { kKvInt8 = 0, kKvE4m3 = 1 };

constexpr int kKvMaxSeqs = 4096;
constexpr int kKvMaxWidth = 1 << 20;    // pages of a sequence
constexpr int kKvMaxPages = 1 << 24;

struct KvPool {
    uint8_t *codes;          // plane 0
    float *scales;
    int64_t plane_codes;     // bytes from a plane to the next
    int64_t plane_scales;    // floats from a plane to the next
    int pages, heads, dim, page;
    int page_log2;
};

struct KvTable {
    const int32_t *table;    // [seqs][ldt]
    const int32_t *lens;     // [seqs]
    int64_t ldt;
    int seqs, width;
};

// Length of a sequence, cut to what its row of the table can hold.
__device__ __forceinline__ int kv_length(const KvTable &t, int b, int page_log2, unsigned int *status) {
    const int len = t.lens[b];
    const int64_t top = (int64_t)t.width << page_log2;
    if (len < 0 || len > top) {
        record_status(status, kStatusBadPage);
        return len < 0 ? 0 : (int)(top > 0x7FFFFFFF ? 0x7FFFFFFF : top);
    }
    return len;
}

// fp32 -> code.  INT8: round to nearest even, clamped to -127..127.
template <int KIND>
__device__ __forceinline__ uint32_t kv_encode2(float lo, float hi) {
    if constexpr (KIND == kKvInt8) {
        const int a = (int)fminf(fmaxf(rintf(lo), -127.0f), 127.0f);
        const int b = (int)fminf(fmaxf(rintf(hi), -127.0f), 127.0f);
        return (uint32_t)(a & 0xFF) | ((uint32_t)(b & 0xFF) << 8);
    } else {
        uint16_t r;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
        return r;
    }
}

// two codes (bits 0-15) -> fp32
template <int KIND>
__device__ __forceinline__ float2 kv_decode2(uint32_t c) {
    if constexpr (KIND == kKvInt8) {
        return make_float2((float)(int8_t)(c & 0xFF), (float)(int8_t)((c >> 8) & 0xFF));
    } else {
        uint32_t h;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
        float2 f;
        asm("{\n\t.reg .f16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(f.x), "=f"(f.y) : "r"(h));
        return f;
    }
}

}  // namespace clef
