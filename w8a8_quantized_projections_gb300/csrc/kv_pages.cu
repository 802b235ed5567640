// kv_pages.cu -- the page pool's bookkeeping and the copies behind it.
//
// refs[p] is how many sequences hold page p (0: free).  Whole pages may be
// shared by sequences; a part-filled last page has one owner, because fork
// copies it.  Allocation takes the lowest free pages in the order of the
// sequences that ask, so the outcome is the same on every run, and a call
// that cannot be served in full changes nothing (CLEF_ERR_NO_PAGES in the
// status word).  Everything stays on the device: a step can reserve, append
// and attend without the host seeing a length.
//
// The bookkeeping reads at most a few hundred KB of integers and each step
// of it needs the one before: it runs as one CTA of 1,024 threads, 16 pages a
// thread and round: trips to memory one after the other, about 6 us a call alone
// and 15 us for a fork, a reserve and a free back to back.  The page copies are
// separate launches over all SMs, bound by memory bandwidth (2 bytes moved for a
// byte copied): 91 us to compact a pool with 270 MB of pages to move, 5.9 TB/s.
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "kv_cache.cuh"
#include "kv_host.h"

namespace clef {

namespace {

constexpr int kBook = 1024;           // threads of a bookkeeping CTA
constexpr int kPer = 16;              // pages a thread looks at in a round
constexpr int kCopyThreads = 256;
constexpr int kPiece = kCopyThreads * 64;   // bytes of a copy piece: four 16-byte words a thread

// Exclusive prefix sum over the CTA; *total gets the sum.  Two barriers.
__device__ __forceinline__ int block_scan(int v, int *warps, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
        if (lane >= o) inc += u;
    }
    __syncthreads();   // warps[] may still be read from the scan before
    if (lane == 31) warps[warp] = inc;
    __syncthreads();
    const int w = warps[lane];   // kBook / 32 = 32 warps, one a lane
    int winc = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, winc, o);
        if (lane >= o) winc += u;
    }
    *total = __shfl_sync(0xFFFFFFFFu, winc, 31);
    return __shfl_sync(0xFFFFFFFFu, winc - w, warp) + inc - v;
}

// Bit i: page p0 + i satisfies what (0: free, 1: held).  Pages past the end
// satisfy nothing.
__device__ __forceinline__ uint32_t page_bits(const int32_t *refs, int p0, int pages, bool held) {
    uint32_t m = 0;
    if (p0 + kPer <= pages && (reinterpret_cast<uintptr_t>(refs + p0) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i < kPer / 4; ++i) {
            const int4 v = *reinterpret_cast<const int4 *>(refs + p0 + 4 * i);
            m |= (uint32_t)((v.x > 0) == held) << (4 * i) | (uint32_t)((v.y > 0) == held) << (4 * i + 1) |
                 (uint32_t)((v.z > 0) == held) << (4 * i + 2) | (uint32_t)((v.w > 0) == held) << (4 * i + 3);
        }
    } else {
        for (int i = 0; i < kPer; ++i)
            if (p0 + i < pages && (refs[p0 + i] > 0) == held) m |= 1u << i;
    }
    return m;
}

// The free pages of the first round (the whole pool, up to 16,384 pages): read
// beside a call's other arguments, they save two trips to memory of the three
// that follow one another.
struct FreePages {
    const int32_t *refs;
    int pages;
    uint32_t first;      // this thread's bits
    int at, all;         // free pages before them, and of the round

    __device__ __forceinline__ FreePages(const int32_t *refs, int pages)
        : refs(refs), pages(pages), first(page_bits(refs, (int)threadIdx.x * kPer, pages, false)) {}

    // Whether there are `need` (need <= pages).
    __device__ __forceinline__ bool have(int need, int *warps) {
        at = block_scan(__popc(first), warps, &all);
        int found = all;
        for (int p = kBook * kPer; p < pages && found < need; p += kBook * kPer) {
            int more;
            block_scan(__popc(page_bits(refs, p + (int)threadIdx.x * kPer, pages, false)), warps, &more);
            found += more;
        }
        return found >= need;
    }

    // After have(): hands the r-th lowest to give(r, page) for every r < need.
    template <typename Give>
    __device__ __forceinline__ void hand_out(int need, int *warps, Give give) {
        int found = 0;
        for (int p = 0; p < pages && found < need; p += kBook * kPer) {
            const int p0 = p + (int)threadIdx.x * kPer;
            uint32_t m = p == 0 ? first : page_bits(refs, p0, pages, false);
            int more = all, r = at;
            if (p > 0) r = found + block_scan(__popc(m), warps, &more);
            for (; m && r < need; m &= m - 1, ++r) give(r, p0 + __ffs(m) - 1);
            found += more;
        }
    }
};

// The asker of allocation r: the last i with off[i] <= r (off is the
// exclusive prefix sum of the needs, so askers of nothing are skipped).
__device__ __forceinline__ int asker(const int *off, int n, int r) {
    int lo = 0, hi = n;   // off[lo] <= r < off[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (off[mid] <= r) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct BookArgs {
    int32_t *table;
    int64_t ldt;
    int seqs, width;
    int32_t *lens, *refs;
    int pages, page_log2;
    unsigned int *status;
};

__device__ __forceinline__ int pages_of(int64_t len, int log2) {
    return (int)((len + ((int64_t)1 << log2) - 1) >> log2);
}

// lens[b] += grow[b], with the pages that takes.  row_start (may be null): the running sum of
// grow, or zeros where nothing is reserved, so that an append of those rows writes nothing: without
// it the rows would land on the last tokens that the sequences have.
__global__ void __launch_bounds__(kBook) kv_reserve_kernel(const BookArgs a, const int32_t *grow, int32_t *row_start) {
    extern __shared__ int off[];     // [seqs + 1]
    __shared__ int warps[32];
    pdl_wait();
    const int tid = threadIdx.x;
    FreePages free_pages(a.refs, a.pages);
    int64_t need = 0;
    int bad = 0;
    for (int b0 = 0; b0 < a.seqs; b0 += kBook) {
        const int b = b0 + tid;
        int want = 0;
        if (b < a.seqs) {
            const int64_t len = a.lens[b], g = grow[b];
            if (len < 0 || g < 0 || len + g > 0x7FFFFFFF || pages_of(len + g, a.page_log2) > a.width) bad = 1;
            else want = pages_of(len + g, a.page_log2) - pages_of(len, a.page_log2);
        }
        int all;
        const int at = block_scan(want, warps, &all);
        if (b < a.seqs) off[b] = (int)min((int64_t)0x7FFFFFFF, need + at);
        need += all;
    }
    if (tid == 0) off[a.seqs] = (int)min((int64_t)0x7FFFFFFF, need);
    bad = __syncthreads_or(bad);
    const bool fits = !bad && need <= a.pages && free_pages.have((int)need, warps);
    if (!fits) {
        if (tid == 0) record_status(a.status, bad ? kStatusBadPage : kStatusNoPages);
    } else {
        if (need > 0)
            free_pages.hand_out((int)need, warps, [&](int r, int p) {
                const int b = asker(off, a.seqs, r);
                a.table[(int64_t)b * a.ldt + pages_of(a.lens[b], a.page_log2) + (r - off[b])] = p;
                a.refs[p] = 1;
            });
        __syncthreads();   // the lengths are read until here
        for (int b = tid; b < a.seqs; b += kBook) a.lens[b] += grow[b];
    }
    if (row_start) {
        uint32_t rows = 0;      // under 2^32: at most a page for each sequence beside the pool's pages
        for (int b0 = 0; b0 < a.seqs; b0 += kBook) {
            const int b = b0 + tid;
            int all;
            const uint32_t at = rows + (uint32_t)block_scan(fits && b < a.seqs ? grow[b] : 0, warps, &all);
            if (b < a.seqs) row_start[b] = (int)min(at, 0x7FFFFFFFu);
            rows += (uint32_t)all;
        }
        if (tid == 0) row_start[a.seqs] = (int)min(rows, 0x7FFFFFFFu);
    }
    pdl_launch_dependents();
}

// Sequence dst[i], empty so far, becomes a copy of src[i] as it was before the call: whole
// pages shared, a part-filled last page given a page of its own, which the copy launch after
// this one fills: moves[i] = (from, to), or (-1, -1).
__global__ void __launch_bounds__(kBook) kv_fork_kernel(const BookArgs a, const int32_t *src, const int32_t *dst, int n,
                                                        int32_t *from, int32_t *to) {
    extern __shared__ int off[];     // [n + 1], then a bit for each sequence
    __shared__ int warps[32];
    uint32_t *seen = reinterpret_cast<uint32_t *>(off + n + 1);
    pdl_wait();
    const int tid = threadIdx.x;
    FreePages free_pages(a.refs, a.pages);
    for (int i = tid; i < (a.seqs + 31) / 32; i += kBook) seen[i] = 0;
    __syncthreads();
    const int in_page = (1 << a.page_log2) - 1;
    int need = 0, bad = 0;
    for (int i0 = 0; i0 < n; i0 += kBook) {
        const int i = i0 + tid;
        int want = 0;
        if (i < n) {
            const int s = src[i], d = dst[i];
            from[i] = to[i] = -1;
            if (s < 0 || s >= a.seqs || d < 0 || d >= a.seqs) {
                bad = 1;
            } else {
                const int len = a.lens[s];
                // the target is empty, asked for once, and the source's pages are there
                if (a.lens[d] != 0 || (atomicOr(&seen[d >> 5], 1u << (d & 31)) >> (d & 31) & 1u)) bad = 1;
                if (len < 0 || pages_of(len, a.page_log2) > a.width) bad = 1;
                else want = (len & in_page) != 0;
            }
        }
        int all;
        const int at = block_scan(want, warps, &all);
        if (i < n) off[i] = need + at;
        need += all;
    }
    if (tid == 0) off[n] = need;
    bad = __syncthreads_or(bad);
    // every page that would be shared or copied is one of the pool
    if (!bad)
        for (int i = tid >> 5; i < n; i += kBook / 32)
            for (int j = tid & 31; j < pages_of(a.lens[src[i]], a.page_log2); j += 32) {
                const int p = a.table[(int64_t)src[i] * a.ldt + j];
                if (p < 0 || p >= a.pages) bad = 1;
            }
    bad = __syncthreads_or(bad);
    const bool fits = !bad && need <= a.pages && free_pages.have(need, warps);
    if (!fits) {
        if (tid == 0) record_status(a.status, bad ? kStatusBadPage : kStatusNoPages);
    } else {
        if (need > 0)
            free_pages.hand_out(need, warps, [&](int r, int p) {
                const int i = asker(off, n, r), last = a.lens[src[i]] >> a.page_log2;
                from[i] = a.table[(int64_t)src[i] * a.ldt + last];
                to[i] = p;
                a.table[(int64_t)dst[i] * a.ldt + last] = p;
                a.refs[p] = 1;
            });
        __syncthreads();
        for (int i = tid >> 5; i < n; i += kBook / 32)
            for (int j = tid & 31; j < a.lens[src[i]] >> a.page_log2; j += 32) {
                const int p = a.table[(int64_t)src[i] * a.ldt + j];
                a.table[(int64_t)dst[i] * a.ldt + j] = p;
                atomicAdd(&a.refs[p], 1);      // whole numbers: the order does not matter
            }
        __syncthreads();
        // a target may be a source too (an empty one): every length is read before any is written
        constexpr int kRounds = kKvMaxSeqs / kBook;
        int len[kRounds];
#pragma unroll
        for (int k = 0; k < kRounds; ++k) len[k] = tid + k * kBook < n ? a.lens[src[tid + k * kBook]] : 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kRounds; ++k)
            if (tid + k * kBook < n) a.lens[dst[tid + k * kBook]] = len[k];
    }
    pdl_launch_dependents();
}

// Sequences seqs[i] give their pages back and become empty.
__global__ void __launch_bounds__(256) kv_free_kernel(const BookArgs a, const int32_t *list, int n) {
    __shared__ int s_len;
    pdl_wait();
    const int b = list[blockIdx.x];
    if (b < 0 || b >= a.seqs) {
        if (threadIdx.x == 0) record_status(a.status, kStatusBadPage);
    } else {
        if (threadIdx.x == 0) s_len = atomicExch(&a.lens[b], 0);   // a sequence listed twice is given back once
        __syncthreads();
        int count = s_len < 0 ? 0 : pages_of(s_len, a.page_log2);
        if (s_len < 0 || count > a.width) {
            if (threadIdx.x == 0) record_status(a.status, kStatusBadPage);
            count = min(count, a.width);
        }
        for (int j = threadIdx.x; j < count; j += 256) {
            const int p = a.table[(int64_t)b * a.ldt + j];
            if (p < 0 || p >= a.pages) {
                record_status(a.status, kStatusBadPage);
            } else if (atomicSub(&a.refs[p], 1) <= 0) {   // nobody held it: put back what was taken
                atomicAdd(&a.refs[p], 1);
                record_status(a.status, kStatusBadPage);
            }
        }
    }
    pdl_launch_dependents();
}

// Compact, first part: with L pages held, the k-th lowest held page at or
// past L goes to the k-th lowest free page below L.  Both lists and every
// page's new place are written to scratch; refs_out to the new order.
//   scratch: [0] moves, [1 .. 1 + pages) new place, then from[], then to[]
__global__ void __launch_bounds__(kBook) kv_compact_kernel(const BookArgs a, int32_t *refs_out, int32_t *scratch,
                                                           int32_t *live_out) {
    __shared__ int warps[32];
    pdl_wait();
    const int tid = threadIdx.x;
    int32_t *place = scratch + 1, *from = place + a.pages, *to = from + a.pages;
    int live = 0;
    for (int p = 0; p < a.pages; p += kBook * kPer) {
        int all;
        block_scan(__popc(page_bits(a.refs, p + tid * kPer, a.pages, true)), warps, &all);
        live += all;
    }
    int slots = 0, moved = 0;
    for (int p = 0; p < a.pages; p += kBook * kPer) {
        const int p0 = p + tid * kPer;
        const uint32_t held = page_bits(a.refs, p0, a.pages, true);
        const int inside = max(0, min(kPer, a.pages - p0)), low = max(0, min(inside, live - p0));
        const uint32_t lows = (1u << low) - 1u, all_bits = (1u << inside) - 1u;
        uint32_t gap = ~held & lows, high = held & ~lows & all_bits;
        int sum;
        const int at = block_scan(__popc(gap) | __popc(high) << 16, warps, &sum);   // at most 16,384 of each
        int r = slots + (at & 0xFFFF), h = moved + (at >> 16);
        for (; gap; gap &= gap - 1) to[r++] = p0 + __ffs(gap) - 1;
        for (; high; high &= high - 1) from[h++] = p0 + __ffs(high) - 1;
        slots += sum & 0xFFFF;
        moved += sum >> 16;
    }
    // as many gaps below L as pages held past it
    __syncthreads();
    for (int p = tid; p < a.pages; p += kBook) {
        place[p] = p;
        if (p < live) refs_out[p] = a.refs[p];        // gaps are filled below
    }
    __syncthreads();
    for (int i = tid; i < moved; i += kBook) {
        place[from[i]] = to[i];
        refs_out[to[i]] = a.refs[from[i]];
    }
    __syncthreads();
    for (int p = live + tid; p < a.pages; p += kBook) refs_out[p] = 0;
    if (tid == 0) {
        scratch[0] = moved;
        if (live_out) *live_out = live;
    }
    pdl_launch_dependents();
}

struct CopyArgs {
    KvPool pool;
    int planes;
    const int32_t *from, *to;
    const int32_t *count;    // number of moves on the device; null: n
    int n;
    // compact: the page tables, rewritten by the first CTAs beside the copies
    const int32_t *place;
    const int32_t *table;
    int32_t *table_out;
    const int32_t *lens;
    int64_t ldt, ldt_out;
    int seqs, width;
    unsigned int *status;
};

// Copies pages (codes and scales) of every plane, a 16 KB piece a round and
// CTA.  Sources and targets are disjoint, so the order does not matter.
__global__ void __launch_bounds__(kCopyThreads) kv_copy_kernel(const CopyArgs a) {
    pdl_wait();
    const int tid = threadIdx.x;
    if (a.table) {
        for (int b = blockIdx.x; b < a.seqs; b += gridDim.x) {
            const int len = a.lens[b];
            int count = len < 0 ? 0 : pages_of(len, a.pool.page_log2);
            if (len < 0 || count > a.width) {
                if (tid == 0) record_status(a.status, kStatusBadPage);
                count = min(count, a.width);
            }
            for (int j = tid; j < count; j += kCopyThreads) {
                const int p = a.table[(int64_t)b * a.ldt + j];
                if (p < 0 || p >= a.pool.pages) record_status(a.status, kStatusBadPage);
                else a.table_out[(int64_t)b * a.ldt_out + j] = a.place[p];
            }
        }
    }
    const int64_t bytes = ((int64_t)a.pool.heads * a.pool.dim) << a.pool.page_log2;
    const int pieces = (int)((bytes + kPiece - 1) / kPiece);
    const int64_t moves = a.count ? *a.count : a.n, units = moves * a.planes * pieces;
    for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
        const int64_t pl = u / pieces;
        const int piece = (int)(u - pl * pieces);
        const int plane = (int)(pl % a.planes);
        const int64_t i = pl / a.planes;
        const int from = a.from[i], to = a.to[i];
        if (from < 0 || to < 0 || from >= a.pool.pages || to >= a.pool.pages) {
            // (-1, -1) is a fork without a part-filled page
            if ((from != -1 || to != -1) && tid == 0) record_status(a.status, kStatusBadPage);
            continue;
        }
        uint8_t *base = a.pool.codes + plane * a.pool.plane_codes + (int64_t)piece * kPiece;
        const uint4 *s = reinterpret_cast<const uint4 *>(base + from * bytes);
        uint4 *d = reinterpret_cast<uint4 *>(base + to * bytes);
        const int words = (int)(min((int64_t)kPiece, bytes - (int64_t)piece * kPiece) >> 4);
        uint4 v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (tid + k * kCopyThreads < words) v[k] = __ldcs(s + tid + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (tid + k * kCopyThreads < words) __stcs(d + tid + k * kCopyThreads, v[k]);
        if (piece == 0) {
            float *sc = a.pool.scales + plane * a.pool.plane_scales;
            for (int h = tid; h < a.pool.heads; h += kCopyThreads)
                sc[(int64_t)to * a.pool.heads + h] = sc[(int64_t)from * a.pool.heads + h];
        }
    }
    pdl_launch_dependents();
}

int book_args(BookArgs &a, void *table, int64_t ldt, int64_t seqs, int64_t width, int32_t *lens, int32_t *refs,
              int64_t pages, int page) {
    KvTable t;
    int rc = kv_table_args(t, static_cast<int32_t *>(table), ldt, seqs, width, lens);
    if (rc) return rc;
    if (pages < 0 || pages > kKvMaxPages) return kv_fail("pages out of range");
    if (page != 16 && page != 32 && page != 64 && page != 128) return kv_fail("page must be 16, 32, 64 or 128 tokens");
    if (kv_misaligned(refs, 4)) return kv_fail("refs must be 4-byte aligned");
    a.table = static_cast<int32_t *>(table);
    a.ldt = ldt;
    a.seqs = (int)seqs;
    a.width = (int)width;
    a.lens = lens;
    a.refs = refs;
    a.pages = (int)pages;
    a.page_log2 = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
    return CLEF_OK;
}

int copy_grid(int64_t units, int sms) {
    const int64_t most = (int64_t)sms * 8;   // 8 CTAs of 256 threads fill an SM
    return (int)(units < 1 ? 1 : units > most ? most : units);
}

}  // namespace

}  // namespace clef

using namespace clef;

extern "C" int clef_kv_reserve(int32_t *table, int64_t ldt, int64_t seqs, int64_t width, int32_t *lens, int32_t *refs,
                               int64_t pages, int page, const int32_t *grow, void *stream) {
    return clef_kv_reserve_rows(table, ldt, seqs, width, lens, refs, pages, page, grow, nullptr, stream);
}

extern "C" int clef_kv_reserve_rows(int32_t *table, int64_t ldt, int64_t seqs, int64_t width, int32_t *lens,
                                    int32_t *refs, int64_t pages, int page, const int32_t *grow, int32_t *row_start,
                                    void *stream) {
    BookArgs a;
    int rc = book_args(a, table, ldt, seqs, width, lens, refs, pages, page);
    if (rc) return rc;
    if (kv_misaligned(grow, 4) || kv_misaligned(row_start, 4)) return kv_fail("grow and row_start must be 4-byte aligned");
    if (seqs == 0) return CLEF_OK;
    if (!table || !lens || !refs || !grow) return kv_fail("null pointer");
    int sms = 0;
    if ((rc = internal_device(&sms, &a.status))) return rc;
    static SmemOptIn opt;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(kv_reserve_kernel), (kKvMaxSeqs + 1) * 4);
    if (e == cudaSuccess)
        e = launch_kernel(kv_reserve_kernel, dim3(1), dim3(kBook), (size_t)(seqs + 1) * 4,
                          static_cast<cudaStream_t>(stream), 1, true, a, grow, row_start);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "page reservation launch");
}

extern "C" int clef_kv_fork(void *codes, int64_t plane_bytes, float *scales, int64_t plane_scales, int64_t planes,
                            int64_t pages, int heads, int page, int dim, int32_t *table, int64_t ldt, int64_t seqs,
                            int64_t width, int32_t *lens, int32_t *refs, const int32_t *src, const int32_t *dst,
                            int64_t n, int32_t *scratch, void *stream) {
    BookArgs a;
    CopyArgs c = {};
    int rc = kv_pool_args(c.pool, kKvInt8, codes, plane_bytes, scales, plane_scales, planes, pages, heads, page, dim);
    if (!rc) rc = book_args(a, table, ldt, seqs, width, lens, refs, pages, page);
    if (rc) return rc;
    if (planes < 1 || planes > 4096) return kv_fail("planes must be in 1..4096");
    if (n < 0 || n > kKvMaxSeqs) return kv_fail("forks must be in 0..4096");
    if (kv_misaligned(src, 4) || kv_misaligned(dst, 4) || kv_misaligned(scratch, 4))
        return kv_fail("src, dst and scratch must be 4-byte aligned");
    if (n == 0) return CLEF_OK;
    if (!codes || !scales || !table || !lens || !refs || !src || !dst || !scratch) return kv_fail("null pointer");
    int sms = 0;
    if ((rc = internal_device(&sms, &a.status))) return rc;
    const size_t smem = (size_t)(n + 1) * 4 + (size_t)((seqs + 31) / 32) * 4;
    static SmemOptIn opt;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(kv_fork_kernel), (kKvMaxSeqs + 1) * 4 + kKvMaxSeqs / 8);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (e == cudaSuccess)
        e = launch_kernel(kv_fork_kernel, dim3(1), dim3(kBook), smem, st, 1, true, a, src, dst, (int)n, scratch,
                          scratch + n);
    if (e != cudaSuccess) return internal_cuda_error(e, "page fork launch");
    c.planes = (int)planes;
    c.from = scratch;
    c.to = scratch + n;
    c.n = (int)n;
    c.status = a.status;
    const int64_t pieces = ((int64_t)heads * page * dim + kPiece - 1) / kPiece;
    e = launch_kernel(kv_copy_kernel, dim3(copy_grid(n * planes * pieces, sms)), dim3(kCopyThreads), 0, st, 1, true, c);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "page copy launch");
}

extern "C" int clef_kv_free(int32_t *table, int64_t ldt, int64_t seqs, int64_t width, int32_t *lens, int32_t *refs,
                            int64_t pages, int page, const int32_t *list, int64_t n, void *stream) {
    BookArgs a;
    int rc = book_args(a, table, ldt, seqs, width, lens, refs, pages, page);
    if (rc) return rc;
    if (n < 0 || n > ((int64_t)1 << 20)) return kv_fail("listed sequences out of range");
    if (kv_misaligned(list, 4)) return kv_fail("the list must be 4-byte aligned");
    if (n == 0) return CLEF_OK;
    if (!table || !lens || !refs || !list) return kv_fail("null pointer");
    int sms = 0;
    if ((rc = internal_device(&sms, &a.status))) return rc;
    const cudaError_t e = launch_kernel(kv_free_kernel, dim3((unsigned)n), dim3(256), 0,
                                        static_cast<cudaStream_t>(stream), 1, true, a, list, (int)n);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "page free launch");
}

extern "C" int clef_kv_compact(void *codes, int64_t plane_bytes, float *scales, int64_t plane_scales, int64_t planes,
                               int64_t pages, int heads, int page, int dim, const int32_t *table, int64_t ldt,
                               int64_t seqs, int64_t width, const int32_t *lens, const int32_t *refs,
                               int32_t *table_out, int64_t ldt_out, int32_t *refs_out, int32_t *live,
                               int32_t *scratch, void *stream) {
    BookArgs a;
    CopyArgs c = {};
    int rc = kv_pool_args(c.pool, kKvInt8, codes, plane_bytes, scales, plane_scales, planes, pages, heads, page, dim);
    if (!rc) rc = book_args(a, const_cast<int32_t *>(table), ldt, seqs, width, const_cast<int32_t *>(lens),
                            const_cast<int32_t *>(refs), pages, page);
    if (rc) return rc;
    if (planes < 1 || planes > 4096) return kv_fail("planes must be in 1..4096");
    if (ldt_out < width) return kv_fail("the output table's pitch is smaller than its width");
    if (table_out == table && ldt_out != ldt) return kv_fail("a table compacted in place keeps its pitch");
    if (kv_misaligned(table_out, 4) || kv_misaligned(refs_out, 4) || kv_misaligned(scratch, 4) || kv_misaligned(live, 4))
        return kv_fail("outputs and scratch must be 4-byte aligned");
    if (pages == 0) return CLEF_OK;
    if (!codes || !scales || !refs || !refs_out || !scratch || (seqs > 0 && width > 0 && (!table || !table_out || !lens)))
        return kv_fail("null pointer");
    int sms = 0;
    if ((rc = internal_device(&sms, &a.status))) return rc;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = launch_kernel(kv_compact_kernel, dim3(1), dim3(kBook), 0, st, 1, true, a, refs_out, scratch, live);
    if (e != cudaSuccess) return internal_cuda_error(e, "page compaction launch");
    c.planes = (int)planes;
    c.count = scratch;
    c.place = scratch + 1;
    c.from = scratch + 1 + pages;
    c.to = scratch + 1 + 2 * pages;
    c.table = seqs > 0 && width > 0 ? table : nullptr;
    c.table_out = table_out;
    c.lens = lens;
    c.ldt = ldt;
    c.ldt_out = ldt_out;
    c.seqs = (int)seqs;
    c.width = (int)width;
    c.status = a.status;
    const int64_t pieces = ((int64_t)heads * page * dim + kPiece - 1) / kPiece;
    const int64_t most = pages / 2 * planes * pieces;   // at most half of the pages move
    e = launch_kernel(kv_copy_kernel, dim3(copy_grid(most > seqs ? most : seqs, sms)), dim3(kCopyThreads), 0, st, 1, true, c);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "page copy launch");
}

extern "C" int clef_kv_copy_pages(void *codes, int64_t plane_bytes, float *scales, int64_t plane_scales, int64_t planes,
                                  int64_t pages, int heads, int page, int dim, const int32_t *src, const int32_t *dst,
                                  int64_t n, void *stream) {
    CopyArgs c = {};
    int rc = kv_pool_args(c.pool, kKvInt8, codes, plane_bytes, scales, plane_scales, planes, pages, heads, page, dim);
    if (rc) return rc;
    if (planes < 1 || planes > 4096) return kv_fail("planes must be in 1..4096");
    if (n < 0 || n > kKvMaxPages) return kv_fail("copies out of range");
    if (kv_misaligned(src, 4) || kv_misaligned(dst, 4)) return kv_fail("src and dst must be 4-byte aligned");
    if (n == 0) return CLEF_OK;
    if (!codes || !scales || !src || !dst) return kv_fail("null pointer");
    int sms = 0;
    if ((rc = internal_device(&sms, &c.status))) return rc;
    c.planes = (int)planes;
    c.from = src;
    c.to = dst;
    c.n = (int)n;
    const int64_t pieces = ((int64_t)heads * page * dim + kPiece - 1) / kPiece;
    const cudaError_t e = launch_kernel(kv_copy_kernel, dim3(copy_grid(n * planes * pieces, sms)), dim3(kCopyThreads), 0,
                                        static_cast<cudaStream_t>(stream), 1, true, c);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "page copy launch");
}
