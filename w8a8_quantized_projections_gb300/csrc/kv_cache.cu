// kv_cache.cu -- writing keys and values into the paged 8-bit cache, and
// reading them back as bf16.
//
// Append.  A page of one head has one scale, but its tokens arrive over many
// calls, so the scale grows with the largest value seen:
//   s = max(s_old, fp32(amax / top))      s_old: 0 for a page without tokens
//   the page's earlier codes, if s > s_old:  encode(value(code) * fp32(s_old / s))
//   the new codes:                           encode(v * min(fp32(1 / s), FLT_MAX))
// with top = 127 (INT8, rounded to nearest even, -127..127) or 448 (e4m3), and
// amax the largest magnitude of the call's tokens in that page and head.  A
// scale of zero (only zeros seen) gives codes of zero.
//
// Bound by the rows read (2 bytes an element) and the codes written (1 byte): 26 us
// for 16 x 1,502 tokens of 8 heads of 128, keys and values (148 MB, 5.6 TB/s).
// One CTA takes one (touched page, head) of the keys or of the values: the
// rows stay in registers between the maximum and the codes, so they are read
// once.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "kv_cache.cuh"
#include "kv_host.h"

namespace clef {

namespace {

constexpr int kThreads = 256;

struct AppendArgs {
    KvPool pool;
    KvTable tab;
    const uint16_t *src[2];    // new keys, new values
    int64_t ld_tok[2], ld_head[2];
    const int32_t *start;      // first row of each sequence, [seqs + 1]; null: per_seq rows each
    int per_seq, slots, rows;  // slots: touched pages a sequence can have (start == null)
    unsigned int *status;
};

// The number of pages that n tokens ending at position len touch.
__device__ __forceinline__ int touched(int len, int n, int log2) {
    return n > 0 ? ((len - 1) >> log2) - ((len - n) >> log2) + 1 : 0;
}

// Rows of sequence b, cut to what is there (start arrays come from the device).
__device__ __forceinline__ void rows_of(const AppendArgs &a, int b, int &row0, int &n) {
    if (!a.start) {
        row0 = b * a.per_seq;
        n = a.per_seq;
        return;
    }
    row0 = a.start[b];
    const int end = a.start[b + 1];
    if (row0 < 0 || end < row0 || end > a.rows) {
        record_status(a.status, kStatusBadPage);
        row0 = 0;
        n = 0;
        return;
    }
    n = end - row0;
}

template <int KIND, int NV>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendArgs a) {
    __shared__ int s_scan[kThreads / 32], s_found[2];
    __shared__ float s_max[kThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, log2 = a.pool.page_log2;
    pdl_wait();
    int b = -1, slot = 0;
    if (!a.start) {
        b = (int)blockIdx.x / a.slots;
        slot = (int)blockIdx.x - b * a.slots;
    } else {
        // the sequence that holds touched page number blockIdx.x
        if (tid == 0) s_found[0] = -1;
        int before = 0;
        for (int b0 = 0; b0 < a.tab.seqs; b0 += kThreads) {
            int cnt = 0;
            if (b0 + tid < a.tab.seqs) {
                int row0, n;
                rows_of(a, b0 + tid, row0, n);
                const int len = kv_length(a.tab, b0 + tid, log2, a.status);
                cnt = touched(len, min(n, len), log2);
            }
            int inc = cnt;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
                if (lane >= o) inc += v;
            }
            __syncthreads();
            if (lane == 31) s_scan[warp] = inc;
            __syncthreads();
            int base = before, all = 0;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) {
                if (w < warp) base += s_scan[w];
                all += s_scan[w];
            }
            const int at = (int)blockIdx.x - (base + inc - cnt);
            if (at >= 0 && at < cnt) {
                s_found[0] = b0 + tid;
                s_found[1] = at;
            }
            before += all;
            if (before > (int)blockIdx.x) break;
        }
        __syncthreads();
        b = s_found[0];
        slot = s_found[1];
    }
    if (b < 0) return;
    int row0, n;
    rows_of(a, b, row0, n);
    const int len = kv_length(a.tab, b, log2, a.status);
    if (n > len) {   // more rows than the sequence has tokens: the last len of them have a place
        if (tid == 0) record_status(a.status, kStatusBadPage);
        row0 += n - len;
        n = len;
    }
    if (slot >= touched(len, n, log2)) return;
    const int first = len - n;                            // position of the first new token
    const int pi = (first >> log2) + slot;                // the page's place in the table
    const int p0 = max(first, pi << log2), p1 = min(len, (pi + 1) << log2);
    const int held = p0 - (pi << log2);                   // tokens that the page holds already
    const int page = a.tab.table[(int64_t)b * a.tab.ldt + pi];
    if (page < 0 || page >= a.pool.pages) {
        if (tid == 0) record_status(a.status, kStatusBadPage);
        return;
    }
    const int head = blockIdx.y, plane = blockIdx.z, D = a.pool.dim, vec_log2 = __ffs(D) - 4;   // vectors of 8 of a row
    const uint16_t *src = a.src[plane] + (int64_t)(row0 + p0 - first) * a.ld_tok[plane] + (int64_t)head * a.ld_head[plane];
    uint8_t *codes = a.pool.codes + plane * a.pool.plane_codes +
                     (((int64_t)page * a.pool.heads + head) << log2) * D;
    float *scale = a.pool.scales + plane * a.pool.plane_scales + (int64_t)page * a.pool.heads + head;
    const int total = (p1 - p0) << vec_log2;

    uint4 v[NV];
    uint32_t top2 = 0;   // the largest magnitudes, as bf16 bits: they order like integers
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = tid + i * kThreads;
        v[i] = make_uint4(0, 0, 0, 0);
        if (u < total) {
            const int tok = u >> vec_log2, c = u & ((1 << vec_log2) - 1);
            v[i] = *reinterpret_cast<const uint4 *>(src + (int64_t)tok * a.ld_tok[plane] + c * 8);
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) top2 = __vmaxu2(top2, w[k] & 0x7FFF7FFFu);
    }
    uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    top = __reduce_max_sync(0xFFFFFFFFu, top);
    if (lane == 0) s_max[warp] = __uint_as_float(top << 16);
    const float s_old = held > 0 ? *scale : 0.0f;
    __syncthreads();
    float amax = 0.0f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
    const float s_new = fmaxf(s_old, __fdiv_rn(amax, KIND == kKvInt8 ? 127.0f : 448.0f));
    const float r = s_new > 0.0f ? fminf(__fdiv_rn(1.0f, s_new), 3.402823466e38f) : 0.0f;
    if (s_new > s_old && held > 0) {
        const float f = __fdiv_rn(s_old, s_new);
        for (int u = tid; u < held * (D >> 4); u += kThreads) {
            uint4 *at = reinterpret_cast<uint4 *>(codes) + u;
            const uint4 q = *at;
            uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 lo = kv_decode2<KIND>(w[k] & 0xFFFFu), hi = kv_decode2<KIND>(w[k] >> 16);
                w[k] = kv_encode2<KIND>(__fmul_rn(lo.x, f), __fmul_rn(lo.y, f)) |
                       (kv_encode2<KIND>(__fmul_rn(hi.x, f), __fmul_rn(hi.y, f)) << 16);
            }
            *at = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    uint2 *dst = reinterpret_cast<uint2 *>(codes + (int64_t)held * D);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int u = tid + i * kThreads;
        if (u < total) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
                o[k] = kv_encode2<KIND>(__fmul_rn(__uint_as_float(w[k] << 16), r),
                                        __fmul_rn(__uint_as_float(w[k] & 0xFFFF0000u), r));
            dst[u] = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
        }
    }
    if (tid == 0) *scale = s_new;   // every thread read the old one before the barrier
    pdl_launch_dependents();
}

struct GatherArgs {
    KvPool pool;
    KvTable tab;
    const int32_t *seq, *pos;
    int64_t rows;
    uint16_t *out[2];
    int64_t ld[2];
    unsigned int *status;
};

// bf16(code * scale) of given tokens: 8 codes in, 16 bytes out per lane and
// vector, four vectors on their way at a time.  2^lanes_log2 lanes, a warp or the
// part of one that a row fills, take a row, so that its page is looked up and its
// places are found once.  Bound by the 3 bytes an element that move: 27 us for 24,032 rows of 8
// heads of 128, keys and values (148 MB, 5.5 TB/s).
template <int KIND>
__global__ void __launch_bounds__(kThreads) kv_gather_kernel(const GatherArgs a, int lanes_log2) {
    const int log2 = a.pool.page_log2, plane = blockIdx.y, vec_log2 = __ffs(a.pool.dim) - 4, per_row = a.pool.heads << vec_log2;
    const int lanes = 1 << lanes_log2, sub = (int)threadIdx.x & (lanes - 1), in_head = (1 << vec_log2) - 1;
    const int head_codes = a.pool.dim << log2;
    const int64_t step = (int64_t)gridDim.x * kThreads >> lanes_log2;
    pdl_wait();
    for (int64_t row = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> lanes_log2; row < a.rows; row += step) {
        const int b = a.seq[row], p = a.pos[row];
        int page = -1;
        if (b >= 0 && b < a.tab.seqs && p >= 0 && (p >> log2) < a.tab.width) page = a.tab.table[(int64_t)b * a.tab.ldt + (p >> log2)];
        const bool there = page >= 0 && page < a.pool.pages;
        if (!there) {
            record_status(a.status, kStatusBadPage);
            page = 0;
        }
        const float *scales = a.pool.scales + plane * a.pool.plane_scales + (int64_t)page * a.pool.heads;
        const uint8_t *codes = a.pool.codes + plane * a.pool.plane_codes + (int64_t)page * a.pool.heads * head_codes +
                               (p & (a.pool.page - 1)) * a.pool.dim;
        uint16_t *out = a.out[plane] + row * a.ld[plane];
        for (int v0 = sub; v0 < per_row; v0 += 4 * lanes) {
            uint2 q[4];
            float s[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int v = v0 + k * lanes, head = v >> vec_log2;
                q[k] = make_uint2(0, 0);
                s[k] = 0.0f;
                if (there && v < per_row) {
                    q[k] = *reinterpret_cast<const uint2 *>(codes + (int64_t)head * head_codes + ((v & in_head) << 3));
                    s[k] = scales[head];
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int v = v0 + k * lanes;
                const uint32_t w[4] = {q[k].x & 0xFFFFu, q[k].x >> 16, q[k].y & 0xFFFFu, q[k].y >> 16};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = kv_decode2<KIND>(w[i]);
                    const __nv_bfloat162 h = __floats2bfloat162_rn(__fmul_rn(f.x, s[k]), __fmul_rn(f.y, s[k]));
                    o[i] = *reinterpret_cast<const uint32_t *>(&h);
                }
                if (v < per_row) *reinterpret_cast<uint4 *>(out + v * 8) = make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
    }
    pdl_launch_dependents();
}

}  // namespace

}  // namespace clef

using namespace clef;

extern "C" int clef_kv_append(const void *k, int64_t ldk, int64_t ldk_head, const void *v, int64_t ldv, int64_t ldv_head,
                              int64_t rows, const int32_t *row_start, int kind, void *codes, int64_t plane_bytes,
                              float *scales, int64_t plane_scales, int64_t pages, int heads, int page, int dim,
                              const int32_t *table, int64_t ldt, int64_t seqs, int64_t width, const int32_t *lens,
                              void *stream) {
    AppendArgs a;
    int rc = kv_pool_args(a.pool, kind, codes, plane_bytes, scales, plane_scales, 2, pages, heads, page, dim);
    if (!rc) rc = kv_table_args(a.tab, table, ldt, seqs, width, lens);
    if (rc) return rc;
    if (rows < 0 || rows > ((int64_t)1 << 30)) return kv_fail("rows out of range");
    if (rows == 0 || seqs == 0) return rows == 0 ? CLEF_OK : kv_fail("rows without a sequence");
    if (!row_start && rows % seqs != 0) return kv_fail("without row_start, rows must be a multiple of the sequences");
    if (!k || !v || !codes || !scales || !table || !lens) return kv_fail("null pointer");
    if (kv_misaligned(k, 16) || kv_misaligned(v, 16) || kv_misaligned(row_start, 4))
        return kv_fail("k and v must be 16-byte, row_start 4-byte aligned");
    if (ldk % 8 || ldv % 8 || ldk_head % 8 || ldv_head % 8 || ldk < 0 || ldv < 0 || ldk_head < 0 || ldv_head < 0)
        return kv_fail("token and head pitches must be multiples of 8");
    int sms = 0;
    if ((rc = internal_device(&sms, &a.status))) return rc;
    a.src[0] = static_cast<const uint16_t *>(k);
    a.src[1] = static_cast<const uint16_t *>(v);
    a.ld_tok[0] = ldk;
    a.ld_tok[1] = ldv;
    a.ld_head[0] = ldk_head;
    a.ld_head[1] = ldv_head;
    a.start = row_start;
    a.rows = (int)rows;
    a.per_seq = (int)(rows / seqs);
    a.slots = (a.per_seq + page - 2) / page + 1;
    // touched pages: with equal rows a fixed number of slots a sequence; else
    // at most one for each token, and two more than the whole pages
    int64_t units = (int64_t)a.slots * seqs;
    if (row_start) units = rows < rows / page + 2 * seqs ? rows : rows / page + 2 * seqs;
    const dim3 grid((unsigned)units, (unsigned)heads, 2);
    const bool big = page * dim > 4 * 8 * kThreads;
    auto kern = kind == kKvInt8 ? (big ? kv_append_kernel<kKvInt8, 16> : kv_append_kernel<kKvInt8, 4>)
                                : (big ? kv_append_kernel<kKvE4m3, 16> : kv_append_kernel<kKvE4m3, 4>);
    const cudaError_t e = launch_kernel(kern, grid, dim3(kThreads), 0, static_cast<cudaStream_t>(stream), 1, true, a);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "cache append launch");
}

extern "C" int clef_kv_gather(int kind, const void *codes, int64_t plane_bytes, const float *scales,
                              int64_t plane_scales, int64_t pages, int heads, int page, int dim, const int32_t *table,
                              int64_t ldt, int64_t seqs, int64_t width, const int32_t *seq, const int32_t *pos,
                              int64_t rows, void *k_out, int64_t ldk, void *v_out, int64_t ldv, void *stream) {
    GatherArgs a;
    int rc = kv_pool_args(a.pool, kind, const_cast<void *>(codes), plane_bytes, const_cast<float *>(scales), plane_scales,
                          2, pages, heads, page, dim);
    if (!rc) rc = kv_table_args(a.tab, table, ldt, seqs, width, nullptr);
    if (rc) return rc;
    if (rows < 0 || rows > ((int64_t)1 << 30)) return kv_fail("rows out of range");
    const int64_t row = (int64_t)heads * dim;
    if (ldk < row || ldv < row || ldk % 8 || ldv % 8) return kv_fail("output pitches must hold a row and be multiples of 8");
    if (rows == 0) return CLEF_OK;
    if (!codes || !scales || !table || !seq || !pos || !k_out || !v_out) return kv_fail("null pointer");
    if (kv_misaligned(k_out, 16) || kv_misaligned(v_out, 16) || kv_misaligned(seq, 4) || kv_misaligned(pos, 4))
        return kv_fail("outputs must be 16-byte, seq and pos 4-byte aligned");
    int sms = 0;
    if ((rc = internal_device(&sms, &a.status))) return rc;
    a.seq = seq;
    a.pos = pos;
    a.rows = rows;
    a.out[0] = static_cast<uint16_t *>(k_out);
    a.out[1] = static_cast<uint16_t *>(v_out);
    a.ld[0] = ldk;
    a.ld[1] = ldv;
    const int per_row = (int)(row / 8), lanes_log2 = per_row >= 32 ? 5 : per_row >= 16 ? 4 : 3;
    const int64_t at_once = kThreads >> lanes_log2;
    int64_t blocks = (rows + at_once - 1) / at_once;
    if (blocks > (int64_t)sms * 8) blocks = (int64_t)sms * 8;
    const cudaError_t e = launch_kernel(kind == kKvInt8 ? kv_gather_kernel<kKvInt8> : kv_gather_kernel<kKvE4m3>,
                                        dim3((unsigned)blocks, 2), dim3(kThreads), 0, static_cast<cudaStream_t>(stream), 1, true,
                                        a, lanes_log2);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "cache gather launch");
}
