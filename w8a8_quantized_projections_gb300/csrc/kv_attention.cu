// kv_attention.cu -- attention over the paged 8-bit cache.
//
// For a query row i of sequence b and query head h (key/value head h / G):
//   x_j = scale * sum_d q_d * kcode[j][d] * ks[page(j)]
//   o   = sum_j softmax(x)_j * vcode[j] * vs[page(j)]
// over the tokens j < len (causal: j <= len - n + i, the n queries being the
// sequence's last tokens).  A row that sees no token gives zeros and a
// log-sum-exp of minus infinity.
//
// Few rows a key/value head (up to 16: a token or a few, times the G heads
// that share it) are bound by reading the codes once.  kv_split_kernel cuts a
// sequence into runs of tokens, one CTA each, whose warps stream keys and
// values from memory straight into registers in the layout of the tensor
// core's operands, and a second kernel joins the runs.  The cut follows the
// sequence's own length alone, so the other sequences of a call do not change
// a row's bits.
//
// Many rows are bound by the tensor cores and the exponentials:
// kv_tile_kernel keeps 128 or 256 rows on chip and passes over the sequence's
// tokens 128 at a time with tcgen05 products.
//
// Numbers.  Codes are widened to fp16, exactly (INT8 integers; e4m3 values are
// multiples of 2^-9 up to 448).  A query row is scaled by a power of two to a
// largest magnitude in [2^13, 2^14) and held in fp16: bf16 has fewer bits than
// fp16, so only values under 2^-27 of the row's largest lose anything, less
// than fp32 sums do.  Products are summed in fp32.  The softmax's
// reference is a running maximum m of x + log2 vs: the weights exp2(x + log2 vs
// - m + 15) that multiply values, rounded to fp16 (11 bits against the output's
// 8), are at most 2^15 whatever the pages' scales are, and only those under 2^-29
// of the largest fall below fp16's normal numbers; the softmax's sum takes each
// page's weights times 1 / vs.  A page whose value scale is zero counts with a
// scale of 2^-60, small enough not to set the reference of the others, in the
// sum, and with weights of zero.
// That holds while no scale is further than 2^40 from 1 (neither 1 / vs nor the sum leaves fp32, and a
// weight times its vs is at least 2^-80 of the largest).  From the first page past that on, a row's sum has
// a reference of its own, the running maximum of x alone: two exponentials a weight, and 2 to the power of
// the references' difference comes back as a factor of the output.
#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "kv_cache.cuh"
#include "kv_host.h"

namespace clef {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kFewRows = 16;       // rows a key/value head up to which a sequence is split along its tokens
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLift = 15.0f;     // the largest weight of P is 2^kLift

// Tokens of a split of a sequence of `len` tokens: short enough that one
// sequence spreads over the SMs, long enough that an item's own work (finding
// it, its queries, joining the warps' sums: as much as 90 tokens) and its
// partial results stay a small part.  One sequence of 1,024 tokens takes 7.7,
// 8.7 or 11 us in splits of 128, 256 or 512, of 2,000 tokens 8.9 or 11.2 us in
// splits of 256 or 512; 16 of 1,000 take 17.3, 15.3 or 13.6 us, 128 of 1,000 to
// 1,500 take 96 or 82 us (8 heads of 128, int8).
__host__ __device__ inline int split_tokens(int len) { return len <= 512 ? 512 : len <= 1024 ? 256 : len <= 8192 ? 512 : 1024; }
__host__ __device__ inline int split_count(int len) {
    const int t = split_tokens(len);
    return len / t + (len % t != 0);
}
constexpr int kMaxSplitTokens = 1024;

// Rows that kv_tile_kernel keeps on chip at a time.
__host__ __device__ constexpr int tile_rows(int dim) { return dim <= 128 ? 256 : 128; }

// Splits of a sequence with more than kFewRows rows: while its row tiles leave
// SMs idle (152 on this GPU; a fixed number, so that a row's bits do not follow
// an SM budget), runs of at least 1,024 tokens, at most 16 of them.  A run's
// partial results (128 KB a tile) and the join cost as much as 500 tokens.
constexpr int kTileSlots = 152, kTileMaxSplits = 16;
__host__ __device__ inline int tile_splits(int rows, int len, int heads, int dim) {
    const int tiles = (rows + tile_rows(dim) - 1) / tile_rows(dim) * heads;
    if (tiles < 1 || tiles > kTileSlots / 2) return 1;
    const int steps = (len >> 7) + ((len & 127) != 0);       // of 128 tokens
    int s = kTileSlots / tiles;
    if (s > steps / 8) s = steps / 8;
    if (s > kTileMaxSplits) s = kTileMaxSplits;
    if (s <= 1) return 1;
    const int per = (steps + s - 1) / s;      // equal splits, none of them empty
    return (steps + per - 1) / per;
}
__host__ __device__ inline int tile_split_tokens(int len, int splits) {
    const int steps = (len >> 7) + ((len & 127) != 0);
    return (steps + splits - 1) / splits * 128;
}

// Where the places of a sequence begin: no sequence needs more than per_seq of
// them, nor more than per_row for each of its rows of queries, so that sequence b, whose
// first row is row0, may begin at the smaller of what those before it can have needed.
struct Places {
    int64_t first, per_seq, per_row;
    __device__ __forceinline__ int64_t of(int b, int row0) const {
        const int64_t x = b * per_seq, y = row0 * per_row;
        return first + (x < y ? x : y);
    }
};

struct AttnArgs {
    KvPool pool;
    KvTable tab;
    const uint16_t *q;
    int64_t ldq, ldq_head;
    uint16_t *out;
    int64_t ldo, ldo_head;
    float *lse;                 // [rows][q heads], natural log; may be null
    const int32_t *start;       // [seqs + 1] or null
    int rows, per_seq, group, q_heads, causal;
    float scale_log2;
    // partial results of the sequences that are cut, place (head * rows + row) * splits + split
    // from the sequence's first one on
    float *part;                // [places][dim]
    float *part_lse;            // [places], base 2
    Places few, many;           // of sequences with few and with many rows
    unsigned int *status;
    uint64_t wait_limit_ns;
    int force_timeout;
};

__device__ __forceinline__ void query_rows(const AttnArgs &a, int b, int &row0, int &n) {
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

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A value scale that needs the two references.
__device__ __forceinline__ bool far_scale(float vs) { return vs != 0.0f && !(vs >= 0x1p-40f && vs <= 0x1p40f); }

// 2^(a - b) for running maxima, 0 when a is -inf (b may be -inf then too)
__device__ __forceinline__ float ex2_diff(float a, float b) { return a == -INFINITY ? 0.0f : ex2(a - b); }

// What a query row is multiplied by on its way to fp16, of whose largest magnitude top is the bits:
// 2^e, or NaN for a row that is not finite, so that its result is whatever its tokens are (an infinity
// as it is would make minus infinity of a product, which is a token that is not seen).
__device__ __forceinline__ float row_factor(uint32_t top, int e) {
    return __uint_as_float(top >= 0x7F800000u ? 0x7FC00000u : (uint32_t)(127 + e) << 23);
}

__device__ __forceinline__ void mma_regs(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four codes of a word as two fp16 pairs.  INT8: c ^ 0x80 = c + 128 under the
// exponent of 1024 is 1152 + c; subtracting 1152 is exact.
template <int KIND>
__device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (KIND == kKvInt8) {
        const uint32_t u = w ^ 0x80808080u;
        asm("prmt.b32 %0, %2, %3, 0x4140;\n\tprmt.b32 %1, %2, %3, 0x4342;"
            : "=r"(lo), "=r"(hi) : "r"(u), "r"(0x64646464u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
        asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
    } else {
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
            : "=r"(lo), "=r"(hi) : "r"(w));
    }
}

__device__ __forceinline__ uint4 load_codes(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t *p) {
    uint2 v;
    asm volatile("ld.global.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

// Quotients of small numbers by one divisor (the query heads that share a
// key/value head, or the heads): x / g = umulhi(x, ceil(2^32 / g)), exact while
// x * g < 2^32.
struct GroupDiv {
    int g;
    uint32_t mul;
    __device__ __forceinline__ explicit GroupDiv(int group) : g(group), mul(0xFFFFFFFFu / (uint32_t)group + 1u) {}
    __device__ __forceinline__ int div(int x) const { return g == 1 ? x : (int)__umulhi((uint32_t)x, mul); }
};

// Four codes of the keys as two pairs of fp16 operands.  INT8: c ^ 0x80 = c + 128
// as the halfword it is, (c + 128) 2^-24, below fp16's normal numbers and exact;
// tensor cores take such numbers whole.  That is three instructions for four
// codes instead of five; the 128 leaves with the sum of the query.  (For the
// values the same costs too much: next to one large weight, sums of 128 P leave
// their rounding in dimensions whose codes are small.)
template <int KIND>
__device__ __forceinline__ void expand4(uint32_t w, uint32_t &lo, uint32_t &hi) {
    if constexpr (KIND == kKvInt8) {
        const uint32_t u = w ^ 0x80808080u;
        lo = __byte_perm(u, 0u, 0x4140);
        hi = __byte_perm(u, 0u, 0x4342);
    } else {
        widen4<KIND>(w, lo, hi);
    }
}

// Tokens that a warp takes a step: two 16-token tiles where the registers allow.
template <int D>
__host__ __device__ constexpr int step_tiles() { return D <= 128 ? 2 : 1; }

template <int D, int NT>
__host__ __device__ constexpr int split_smem_floats() { return kWarps * NT * 8 * (D + 6); }

// What a CTA needs of an item before it can stream: made while the item before
// is streamed, so that no item waits for it.
template <int D, int NT>
struct SplitPrep {
    static constexpr int kRows = NT * 8;
    static constexpr int kPitch = D + 4;        // fp16 elements: the lanes' 8-byte reads meet every bank once
    static constexpr int kPages = kMaxSplitTokens / 16;
    uint16_t q[kRows * kPitch];
    float qs[kRows], lift[kRows];               // what S is multiplied by, after lift is taken off it
    int end[kRows];                             // tokens a row sees
    int64_t at[kPages];                         // a page's first code of the head; -1: not there
    float ks[kPages], lv[kPages], inv[kPages];  // key scale; log2 of the value scale; its reciprocal (negative: no weight)
    int far[kPages / 32];                       // whether a page's value scale needs the two references
};

struct SplitItem {
    int b, row0, n, len, rows, head, split, splits, r0, rn, tok0, tok1;
};

// One item: a split of a sequence for one key/value head and NT * 8 of its
// rows (row r = query i * G + head g).
//
// S^T = K Q^T has 16 tokens as the mma's rows and 8 query rows as its columns:
// lane (g, t) loads 16 bytes of the keys of tokens g and g + 8 at 16 t of
// every 64 dimensions, which are its operands of four k-steps (any order of k
// will do that the queries follow).  O^T = V^T P^T has 16 dimensions as rows
// and 16 tokens as k: the lane loads dim / 8 bytes of the values of tokens
// 2 t, 2 t + 1, 2 t + 8, 2 t + 9, interleaved bytewise into token pairs; the
// two bytes 2 j and 2 j + 1 of its run are rows g and g + 8 of tile j.  P
// leaves S^T's layout for that of the right-hand operand by an 8 x 8
// transpose.  No data passes through shared memory but the queries.
//
// A warp's registers hold a step of keys and one of values; each is loaded
// again, for the next step, as soon as its products are done.
//
// Measured: 64 sequences of 512 to 8,192 int8 tokens, 8 heads of 128 read by 48
// query heads: 91.5 us with the join, 4.2 TB/s; three of 32,768 e4m3 tokens at dim
// 256: 46 us, 4.2 TB/s (57 us with two CTAs an SM instead of three, although with
// three a thread spills 140 bytes).  Bound by the latency of a warp's own chain: 45% of
// the issue slots at three warps a scheduler, about 320 instructions a 16-token tile
// and as many as six such tiles an item.  One sequence of 298 tokens: 7.5 us, eight CTAs
// whose warps take three steps one after the other.  The two references of far value
// scales are one branch of a step; as two (at the maximum and at the sum) they cost the
// 298 tokens 0.3 us by their place in the code alone.
template <int D, int NT>
__host__ __device__ constexpr int split_ctas() { return D * NT <= 64 ? 4 : D * NT <= 128 || NT == 1 ? 3 : 2; }     // of an SM, by registers

template <int KIND, int D, int NT>
__global__ void __launch_bounds__(kThreads, split_ctas<D, NT>()) kv_split_kernel(const AttnArgs a) {
    using Prep = SplitPrep<D, NT>;
    constexpr int ROWS = NT * 8, TILES = step_tiles<D>(), STEP = TILES * 16, KB = D / 64, MT = D / 16;
    constexpr int VW = D / 32;               // 32-bit words of values a lane holds of each token
    constexpr int PER = D / 32;              // elements of a query row a lane has
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) Prep s_prep[2];
    __shared__ int s_scan[kWarps], s_total;
    __shared__ float s_ref[2][kWarps * ROWS];      // items with far scales: the references of the sums
    constexpr int OPITCH = D + 4;            // floats: the lanes' writes meet every bank once
    float *s_o = reinterpret_cast<float *>(smem);          // [kWarps][ROWS][OPITCH], then m, l
    float *s_m = s_o + kWarps * ROWS * OPITCH, *s_l = s_m + kWarps * ROWS;
    int *s_items = reinterpret_cast<int *>(smem + split_smem_floats<D, NT>() * 4);   // [seqs + 1] first item of each sequence
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int log2 = a.pool.page_log2, H = a.pool.heads;
    const GroupDiv by_group(a.group), by_heads(H);
    pdl_wait();

    // items of each sequence
    if (tid == 0) s_total = 0;
    __syncthreads();
    for (int b0 = 0; b0 < a.tab.seqs; b0 += kThreads) {
        int cnt = 0;
        if (b0 + tid < a.tab.seqs) {
            int row0, n;
            query_rows(a, b0 + tid, row0, n);
            const int rows = n * a.group;
            // a sequence without tokens still has rows of zeros to write
            if (rows > 0 && rows <= kFewRows)
                cnt = max(1, split_count(kv_length(a.tab, b0 + tid, log2, a.status))) * ((rows + ROWS - 1) / ROWS) * H;
        }
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int base = s_total, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += s_scan[w];
            all += s_scan[w];
        }
        if (b0 + tid < a.tab.seqs) s_items[b0 + tid] = base + inc - cnt;
        __syncthreads();
        if (tid == 0) s_total += all;
        __syncthreads();
    }
    const int items = s_total;
    if ((int)blockIdx.x >= items) return;

    const auto item_at = [&](int item) {
        SplitItem t;
        int b = 0, hi = a.tab.seqs;
        while (hi - b > 1) {
            const int mid = (b + hi) >> 1;
            if (s_items[mid] <= item) b = mid;
            else hi = mid;
        }
        t.b = b;
        query_rows(a, b, t.row0, t.n);
        t.len = kv_length(a.tab, b, log2, a.status);
        t.rows = t.n * a.group;
        const int groups = (t.rows + ROWS - 1) / ROWS;
        int rest = item - s_items[b];
        const int over = rest < (1 << 20) ? by_heads.div(rest) : rest / H;
        t.head = rest - over * H;
        rest = over;
        t.split = groups == 1 ? rest : rest >> 1;      // at most 16 rows: one group or two
        t.r0 = (rest - t.split * groups) * ROWS;
        t.rn = min(ROWS, t.rows - t.r0);
        t.splits = max(1, split_count(t.len));
        t.tok0 = t.split * split_tokens(t.len);
        t.tok1 = min(t.len, t.tok0 + split_tokens(t.len));
        if (a.causal) t.tok1 = min(t.tok1, max(0, t.len - t.n + by_group.div(t.r0 + t.rn - 1) + 1));   // what the last row sees
        return t;
    };

    // the item's preparation in three parts, with a load's latency between them
    uint32_t pq[ROWS / kWarps][PER / 2];
    int p_page = -1;
    float p_ks = 0.0f, p_vs = 0.0f;
    const auto prep_rows = [&](const SplitItem &it) {
#pragma unroll
        for (int k = 0; k < ROWS / kWarps; ++k) {
            const int r = warp + k * kWarps;
#pragma unroll
            for (int w = 0; w < PER / 2; ++w) pq[k][w] = 0u;
            if (r < it.rn) {
                const int i = by_group.div(it.r0 + r), hq = it.head * a.group + (it.r0 + r) - i * a.group;
                const uint32_t *src = reinterpret_cast<const uint32_t *>(a.q + (int64_t)(it.row0 + i) * a.ldq + (int64_t)hq * a.ldq_head);
#pragma unroll
                for (int w = 0; w < PER / 2; ++w) pq[k][w] = src[lane + 32 * w];
            }
        }
        p_page = -1;
        if (tid < Prep::kPages && it.tok0 + (tid << log2) < it.tok1) {
            p_page = a.tab.table[(int64_t)it.b * a.tab.ldt + (it.tok0 >> log2) + tid];
            if (p_page < 0 || p_page >= a.pool.pages) {
                record_status(a.status, kStatusBadPage);
                p_page = -1;
            }
        }
    };
    const auto prep_scales = [&](const SplitItem &it) {
        p_ks = p_vs = 0.0f;
        if (p_page >= 0) {
            const int64_t tile = (int64_t)p_page * H + it.head;
            p_ks = a.pool.scales[tile];
            p_vs = a.pool.scales[a.pool.plane_scales + tile];
        }
    };
    const auto prep_store = [&](const SplitItem &it, Prep &to) {
#pragma unroll
        for (int k = 0; k < ROWS / kWarps; ++k) {
            const int r = warp + k * kWarps;
            // the row's largest magnitude (bf16 bits order like integers) to [2^13, 2^14), in fp16
            uint32_t top = 0;
#pragma unroll
            for (int w = 0; w < PER / 2; ++w) top = __vmaxu2(top, pq[k][w] & 0x7FFF7FFFu);
            top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16)) << 16;
            const int e = top ? min(120, 13 - (int)(top >> 23) + 127) : 0;      // -115 or more
            // a negative scale turns the queries, so that x grows with S
            float up = row_factor(top, e);
            if (a.scale_log2 < 0.0f) up = -up;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < PER / 2; ++w) {
                const uint32_t h = pack_half(__uint_as_float(pq[k][w] << 16) * up, __uint_as_float(pq[k][w] & 0xFFFF0000u) * up);
                *reinterpret_cast<uint32_t *>(&to.q[r * Prep::kPitch + 2 * (lane + 32 * w)]) = h;
                const __half2 h2 = *reinterpret_cast<const __half2 *>(&h);
                sum += __low2float(h2) + __high2float(h2);
            }
            if constexpr (KIND == kKvInt8) {
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
            }
            if (lane == 0) {
                const int i = by_group.div(it.r0 + r);
                to.qs[r] = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 - e) << 23);
                to.lift[r] = KIND == kKvInt8 ? 0x1p-17f * sum : 0.0f;
                to.end[r] = r >= it.rn || !a.causal ? it.len : max(0, it.len - it.n + i + 1);
            }
        }
        if (tid < Prep::kPages) {
            // a page whose value scale is zero counts in the sum with a small scale, and gives no weight
            const float vs = p_vs == 0.0f ? 0x1p-60f : p_vs;
            to.at[tid] = p_page < 0 ? -1 : (((int64_t)p_page * H + it.head) << log2) * D;
            to.ks[tid] = p_ks;
            to.lv[tid] = log2f(vs);
            to.inv[tid] = p_vs == 0.0f ? -0x1p60f : __fdiv_rn(1.0f, vs);      // the sign marks it
            const int far = __any_sync(0xFFFFFFFFu, far_scale(p_vs));
            if (lane == 0) to.far[warp] = far;
        }
    };

    uint4 kc[TILES][2][KB];
    uint32_t vc[TILES][4][VW];
    // (a step whose tokens are all there, the usual one, without a test or a zero at each load)
    const auto page_at = [&](const SplitItem &it, const Prep &pr, int tk) {
        return tk < it.tok1 ? pr.at[(tk - it.tok0) >> log2] : (int64_t)-1;
    };
    const auto load_k = [&](const SplitItem &it, const Prep &pr, int s0) {
        int64_t at[TILES];
        bool there = true;
#pragma unroll
        for (int u = 0; u < TILES; ++u) {
            at[u] = page_at(it, pr, s0 + u * 16);
            there = there && at[u] >= 0;
        }
        const auto load = [&](auto all) {
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                const uint8_t *base = a.pool.codes + at[u] + (((s0 + u * 16) & (a.pool.page - 1)) + g) * D + t * 16;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int k = 0; k < KB; ++k)
                        kc[u][h][k] = decltype(all)::value || at[u] >= 0 ? load_codes(base + h * 8 * D + k * 64) : make_uint4(0, 0, 0, 0);
            }
        };
        if (there) load(std::true_type());
        else load(std::false_type());
    };
    const auto load_v = [&](const SplitItem &it, const Prep &pr, int s0) {
        int64_t at[TILES];
        bool there = s0 + STEP <= it.len;
#pragma unroll
        for (int u = 0; u < TILES; ++u) {
            at[u] = page_at(it, pr, s0 + u * 16);
            there = there && at[u] >= 0;
        }
        const auto load = [&](auto all) {
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                const int tk = s0 + u * 16;
                const uint8_t *base = a.pool.codes + a.pool.plane_codes + at[u] + ((tk & (a.pool.page - 1)) + 2 * t) * D + g * (D >= 128 ? 16 : 8);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int row = (c & 1) + 8 * (c >> 1);
                    // what lies past the sequence's end may be anything, NaN codes included: read as zeros
                    const bool in = decltype(all)::value || (at[u] >= 0 && tk + 2 * t + row < it.len);
                    if constexpr (D == 64) {
                        const uint2 v = in ? load_codes8(base + row * D) : make_uint2(0, 0);
                        vc[u][c][0] = v.x;
                        vc[u][c][1] = v.y;
                    } else {
#pragma unroll
                        for (int k = 0; k < D / 128; ++k) {
                            const uint4 v = in ? load_codes(base + row * D + k * 128) : make_uint4(0, 0, 0, 0);
                            vc[u][c][4 * k] = v.x;
                            vc[u][c][4 * k + 1] = v.y;
                            vc[u][c][4 * k + 2] = v.z;
                            vc[u][c][4 * k + 3] = v.w;
                        }
                    }
                }
            }
        };
        if (there) load(std::true_type());
        else load(std::false_type());
    };

    SplitItem it = item_at(blockIdx.x);
    prep_rows(it);
    prep_scales(it);
    prep_store(it, s_prep[0]);
    __syncthreads();
    int s0 = it.tok0 + warp * STEP;
    if (s0 < it.tok1) {
        load_k(it, s_prep[0], s0);
        load_v(it, s_prep[0], s0);
    }
    int turn = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, turn ^= 1) {
        const Prep &pr = s_prep[turn];
        const bool more = item + (int)gridDim.x < items;
        SplitItem next = it;
        if (more) {
            next = item_at(item + gridDim.x);
            prep_rows(next);
        }
        bool scales_due = more;

        float acc[NT][MT][4], m[NT][2], l[NT][2], qs[NT][2], lift[NT][2];
        int end[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[x][k][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[x][i] = -INFINITY;
                l[x][i] = 0.0f;
                qs[x][i] = pr.qs[x * 8 + 2 * t + i];
                lift[x][i] = pr.lift[x * 8 + 2 * t + i];
                end[x][i] = min(pr.end[x * 8 + 2 * t + i], it.tok1);
            }
        }
        int all_see = min(end[0][0], end[0][1]);
        if (NT == 2) all_see = min(all_see, min(end[NT - 1][0], end[NT - 1][1]));
        all_see = __reduce_min_sync(0xFFFFFFFFu, all_see);
        static_assert(Prep::kPages == 64, "two flags");
        const bool far = (pr.far[0] | pr.far[1]) != 0;
        float *refs = &s_ref[turn][warp * ROWS];
        if (far && lane < ROWS) refs[lane] = -INFINITY;
        __syncwarp();

        // what a sum of products is multiplied by; INT8: the sums are of (c + 128) 2^-24 q, and 2^24
        // comes last because 2^24 times a large row's own factor does not fit in fp32
        const auto factor = [](float q, float k) { return KIND == kKvInt8 ? q * k * 0x1p24f : q * k; };
        for (; s0 < it.tok1; s0 += kWarps * STEP) {
            const int s1 = s0 + kWarps * STEP;
            // S^T
            float s[NT][TILES][4];
#pragma unroll
            for (int x = 0; x < NT; ++x)
#pragma unroll
                for (int u = 0; u < TILES; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[x][u][i] = 0.0f;
#pragma unroll
            for (int k = 0; k < KB; ++k) {
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint2 qf[NT];
#pragma unroll
                    for (int x = 0; x < NT; ++x)
                        qf[x] = *reinterpret_cast<const uint2 *>(&pr.q[(x * 8 + g) * Prep::kPitch + k * 64 + t * 16 + w * 4]);
#pragma unroll
                    for (int u = 0; u < TILES; ++u) {
                        uint32_t f[4];
                        const uint4 &ka = kc[u][0][k], &kb = kc[u][1][k];
                        expand4<KIND>(w == 0 ? ka.x : w == 1 ? ka.y : w == 2 ? ka.z : ka.w, f[0], f[2]);
                        expand4<KIND>(w == 0 ? kb.x : w == 1 ? kb.y : w == 2 ? kb.z : kb.w, f[1], f[3]);
#pragma unroll
                        for (int x = 0; x < NT; ++x) mma_regs(s[x][u], f, qf[x].x, qf[x].y);
                    }
                }
            }
            if (s1 < it.tok1) load_k(it, pr, s1);
            if (scales_due) {
                prep_scales(next);
                scales_due = false;
            }

            // softmax: this lane has rows 2 t, 2 t + 1 and tokens g, g + 8 of each tile
            uint32_t pf[NT][TILES][2];
            float ks[TILES], lv[TILES], inv[TILES];
#pragma unroll
            for (int u = 0; u < TILES; ++u) {
                const int p = (min(s0 + u * 16, it.tok1 - 1) - it.tok0) >> log2;
                ks[u] = pr.ks[p];
                lv[u] = pr.lv[p];
                inv[u] = pr.inv[p];
            }
            const bool whole = s0 + STEP <= all_see;
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                if (!whole) {
#pragma unroll
                    for (int u = 0; u < TILES; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (s0 + u * 16 + g + 8 * (i >> 1) >= end[x][i & 1]) s[x][u][i] = -INFINITY;
                }
                // the largest x + log2 vs
                float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
                for (int u = 0; u < TILES; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float v = fmaxf(s[x][u][i], s[x][u][i + 2]);
                        const float f = factor(qs[x][i], ks[u]);
                        if (whole || v != -INFINITY) top[i] = fmaxf(top[i], fmaf(v, f, fmaf(-lift[x][i], f, lv[u])));
                    }
                if (__builtin_expect(far, 0)) {      // the sum over the step, and top without the pages of zeros
                    float ml[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        top[i] = ml[i] = -INFINITY;
#pragma unroll
                        for (int u = 0; u < TILES; ++u) {
                            const float v = fmaxf(s[x][u][i], s[x][u][i + 2]), f = factor(qs[x][i], ks[u]);
                            if (v == -INFINITY) continue;
                            ml[i] = fmaxf(ml[i], fmaf(v, f, -lift[x][i] * f));
                            if (inv[u] >= 0.0f) top[i] = fmaxf(top[i], fmaf(v, f, fmaf(-lift[x][i], f, lv[u])));
                        }
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) ml[i] = fmaxf(ml[i], __shfl_xor_sync(0xFFFFFFFFu, ml[i], o));
                        const float was = refs[x * 8 + 2 * t + i];
                        ml[i] = fmaxf(ml[i], was);
                        l[x][i] *= ex2_diff(was, ml[i]);
#pragma unroll
                        for (int u = 0; u < TILES; ++u) {
                            const float f = factor(qs[x][i], ks[u]), off = fmaf(-lift[x][i], f, kLift - ml[i]);
#pragma unroll
                            for (int h = 0; h < 4; h += 2)
                                if (s[x][u][i + h] != -INFINITY) l[x][i] += ex2(fmaf(s[x][u][i + h], f, off));
                        }
                    }
                    __syncwarp();
                    if (g == 0) {
                        refs[x * 8 + 2 * t] = ml[0];
                        refs[x * 8 + 2 * t + 1] = ml[1];
                    }
                    __syncwarp();
                }
#pragma unroll
                for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                    for (int i = 0; i < 2; ++i) top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], o));
                float co[2], ref[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float mn = fmaxf(m[x][i], top[i]);
                    co[i] = ex2_diff(m[x][i], mn);
                    m[x][i] = mn;
                    ref[i] = mn == -INFINITY ? 0.0f : mn - kLift;
                    l[x][i] *= far ? 1.0f : co[i];
                }
                if (__any_sync(0xFFFFFFFFu, co[0] != 1.0f || co[1] != 1.0f)) {
#pragma unroll
                    for (int k = 0; k < MT; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) acc[x][k][i] *= co[i & 1];
                }
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    float p[4], f[2], off[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        f[i] = factor(qs[x][i], ks[u]);
                        off[i] = fmaf(-lift[x][i], f[i], lv[u] - ref[i]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = fmaf(s[x][u][i], f[i & 1], off[i & 1]);
                        p[i] = ex2(whole || s[x][u][i] != -INFINITY ? v : -INFINITY);
                    }
                    // (selects, no branch: with far scales the sum has the step's weights already)
                    const float back = far ? 0.0f : fabsf(inv[u]);
                    l[x][0] = fmaf(far ? 0.0f : p[0] + p[2], back, l[x][0]);
                    l[x][1] = fmaf(far ? 0.0f : p[1] + p[3], back, l[x][1]);
                    const uint32_t keep = inv[u] < 0.0f ? 0u : 0xFFFFFFFFu;
                    pf[x][u][0] = transpose8x8(pack_half(p[0], p[1]) & keep);
                    pf[x][u][1] = transpose8x8(pack_half(p[2], p[3]) & keep);
                }
            }
            // O^T
#pragma unroll
            for (int u = 0; u < TILES; ++u)
#pragma unroll
                for (int w = 0; w < VW; ++w) {
                    const uint32_t v0 = vc[u][0][w], v1 = vc[u][1][w], v2 = vc[u][2][w], v3 = vc[u][3][w];
                    uint32_t fa[4], fb[4];   // bytes 0, 1 and bytes 2, 3 of the four tokens
                    widen4<KIND>(__byte_perm(v0, v1, 0x5140), fa[0], fa[1]);
                    widen4<KIND>(__byte_perm(v2, v3, 0x5140), fa[2], fa[3]);
                    widen4<KIND>(__byte_perm(v0, v1, 0x7362), fb[0], fb[1]);
                    widen4<KIND>(__byte_perm(v2, v3, 0x7362), fb[2], fb[3]);
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        mma_regs(acc[x][2 * w], fa, pf[x][u][0], pf[x][u][1]);
                        mma_regs(acc[x][2 * w + 1], fb, pf[x][u][0], pf[x][u][1]);
                    }
                }
            if (s1 < it.tok1) load_v(it, pr, s1);
        }
        if (more) {
            if (scales_due) prep_scales(next);
            prep_store(next, s_prep[turn ^ 1]);
        }

        // the warps' results meet in shared memory
        __syncthreads();      // which the item before is done with
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[x][i] += __shfl_xor_sync(0xFFFFFFFFu, l[x][i], o);
                if (g == 0) {
                    const int row = x * 8 + 2 * t + i;
                    s_m[warp * ROWS + row] = m[x][i];
                    s_l[warp * ROWS + row] = l[x][i];
                }
            }
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // tile k: word k / 2 of the lane's run of values, its bytes 2 (k & 1) and 2 (k & 1) + 1
                    const int byte = 4 * (k / 2) + 2 * (k & 1) + (i >> 1);
                    s_o[(warp * ROWS + x * 8 + 2 * t + (i & 1)) * OPITCH + byte * 8 + g] = acc[x][k][i];
                }
        }
        __syncthreads();
        const SplitItem done = it;
        it = next;
        s0 = it.tok0 + warp * STEP;
        if (more && s0 < it.tok1) {
            load_k(it, s_prep[turn ^ 1], s0);
            load_v(it, s_prep[turn ^ 1], s0);
        }
        for (int r = warp; r < done.rn; r += kWarps) {
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * ROWS + r]);
            float f[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                f[w] = ex2_diff(s_m[w * ROWS + r], mm);
                ll = fmaf(s_l[w * ROWS + r], f[w], ll);
            }
            float ml = mm, back = 1.0f;      // the reference of the sum; the root of 2^(mm - ml)
            if (__builtin_expect(far, 0)) {
                const float *at = &s_ref[turn][r];
                ml = fmaxf(fmaxf(at[0], at[ROWS]), fmaxf(at[2 * ROWS], at[3 * ROWS]));
                ll = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) ll = fmaf(s_l[w * ROWS + r], ex2_diff(at[w * ROWS], ml), ll);
                back = ml == -INFINITY ? 0.0f : ex2(0.5f * (mm - ml));
            }
            const float inv = ll == 0.0f ? 0.0f : __fdiv_rn(1.0f, ll);      // (NaN stays)
            const float lse = ll == 0.0f ? -INFINITY : ml - kLift + log2f(ll);
            const int i = by_group.div(done.r0 + r), hq = done.head * a.group + (done.r0 + r) - i * a.group;
            const int64_t place = a.few.of(done.b, done.row0) + ((int64_t)done.head * done.rows + done.r0 + r) * done.splits + done.split;
            if (done.splits > 1) {
                if (lane == 0) a.part_lse[place] = lse;
            } else if (a.lse && lane == 0) {
                a.lse[(int64_t)(done.row0 + i) * a.q_heads + hq] = lse == -INFINITY ? -INFINITY : lse * (1.0f / kLog2e);
            }
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                // two neighbouring dimensions: bytes of run lane & 7 (its bytes past 16 are 128 dimensions on)
                const int run = lane & 7, byte = 2 * ((lane >> 3) + 4 * k);
                const int d = D == 64 ? run * 8 + byte : (byte / 16) * 128 + run * 16 + byte % 16;
                float o0 = 0.0f, o1 = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float *at = &s_o[(w * ROWS + r) * OPITCH + byte * 8 + run];
                    o0 = fmaf(at[0], f[w], o0);
                    o1 = fmaf(at[8], f[w], o1);
                }
                o0 *= inv;
                o1 *= inv;
                if (__builtin_expect(far, 0)) {
                    o0 = o0 * back * back;
                    o1 = o1 * back * back;
                }
                if (done.splits > 1) {
                    *reinterpret_cast<float2 *>(a.part + place * D + d) = make_float2(o0, o1);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(o0, o1);
                    *reinterpret_cast<__nv_bfloat162 *>(a.out + (int64_t)(done.row0 + i) * a.ldo + (int64_t)hq * a.ldo_head + d) = h;
                }
            }
        }
    }
    pdl_launch_dependents();
}

// ---------------------------------------------------------------- many rows

constexpr float kSlack = 4.0f;        // how far a row's maximum may outgrow its reference (log2)

// Roles, shared memory and tensor memory of kv_tile_kernel.
template <int D>
struct Tile {
    static constexpr int kQ = D <= 128 ? 2 : 1;              // 128-row query tiles on chip
    static constexpr int kStep = D <= 128 ? 128 : 64;        // tokens of a step
    static constexpr int kSub = kStep / 64;                  // blocks of 64 tokens of a step
    static constexpr int kSlots = D <= 128 ? 1 : 2;          // places for S of a row tile
    // Operands: two steps of keys; blocks of values, which the products take one by one: with more than
    // a step's, the next step's first block is there before this step's are done with.
    static constexpr int kKStages = 2, kVBlocks = D == 64 ? 4 : D == 128 ? 3 : 1;
    static constexpr int kRawK = D == 64 ? 4 : 2, kRawV = D == 64 ? 4 : D == 128 ? 3 : 1;   // blocks of codes on their way
    static constexpr int kCols = kStep * kQ / 2;             // columns of S that a softmax thread has
    static constexpr int kOutCols = kQ == 2 ? D : D / 2;     // and of O
    // 20 warps of 96 registers in whole warpgroups: eight of softmax (four for each row tile, or eight
    // for one), four that turn keys into operands and four for values, then one that issues the products
    // for each row tile (one that issued for two waited for one tile's product while the other's could
    // have started: 77 us instead of 69 for 2,270 rows over as many tokens), one that copies the codes of keys and one for values.  Each of the SM's four register files holds two warps of
    // softmax, two of conversion and one of the last group, and setmaxnreg's 2 x 144 + 2 x 56 + 80 =
    // 5 x 96 fit in every one of them.
    static constexpr int kSoftWarps = 8, kConvWarps = 4;     // conversion: for each operand
    static constexpr int kMmaWarp = kSoftWarps + 2 * kConvWarps, kCopyWarp = kMmaWarp + 2;
    static constexpr int kThreadsAll = (kMmaWarp + 4) * 32;
    static constexpr int kChunks = D / 64;                   // 64-element columns of 128-byte rows
    static constexpr int kChunkQ = 128 * 128, kChunkK = kStep * 128;
    static constexpr int kQuery = kChunks * kChunkQ;         // 128 x D in fp16
    static constexpr int kOperand = kChunks * kChunkK;       // kStep x D
    static constexpr int kChunkV = 64 * 128, kBlockV = kChunks * kChunkV;      // a block of values
    static constexpr int kCodes = 64 * D;                    // a block's
    static constexpr int kSmemQ = 0, kSmemK = kQ * kQuery, kSmemV = kSmemK + kKStages * kOperand;
    static constexpr int kSmemRaw = kSmemV + kVBlocks * kBlockV;      // keys' blocks, then values'
    static constexpr int kSmemEnd = kSmemRaw + (kRawK + kRawV) * kCodes;
    static constexpr int kSmem = kSmemEnd + 1024;
    // tensor memory: 256 columns for S (P takes the first half of the columns of its threads), then O.
    // More than half an SM's shared memory is taken, so no two CTAs of an SM wait for one another's
    // tensor memory.
    static constexpr uint32_t kTmemO = 256;
    static constexpr uint32_t kTmemCols = 512;
    static_assert(kSmem > 114 * 1024, "one CTA an SM");
};
constexpr int kRing = 16;             // blocks of page scales
constexpr int kItemStep = 4;          // sequences of an entry of the item table

struct TileItem {
    int b, row0, n, len, rows, head, tile, split, splits, first, rn, tok0, steps;
};

// The item of a CTA's round: rounds go through the CTAs forth and back, so that
// the CTA with the longest item of one round has the shortest of the next.
__device__ __forceinline__ int round_item(int round) {
    return round * (int)gridDim.x + ((round & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x);
}

// Items of sequence b.
template <int D>
__device__ __forceinline__ int tile_items(const AttnArgs &a, int b) {
    int row0, n;
    query_rows(a, b, row0, n);
    const int rows = n * a.group;
    if (rows <= kFewRows) return 0;
    return tile_splits(rows, kv_length(a.tab, b, a.pool.page_log2, a.status), a.pool.heads, D) *
           ((rows + tile_rows(D) - 1) / tile_rows(D)) * a.pool.heads;
}

// What item number `item` is, for a whole warp; s_items has the first item of every kItemStep-th
// sequence.  The row tiles of a sequence come last one first: with a causal mask
// it has the most tokens to see.
template <int D>
__device__ __forceinline__ TileItem tile_item(const AttnArgs &a, const int *s_items, int item) {
    TileItem t;
    int b = 0, hi = (a.tab.seqs + kItemStep - 1) / kItemStep;
    while (hi - b > 1) {
        const int mid = (b + hi) >> 1;
        if (s_items[mid] <= item) b = mid;
        else hi = mid;
    }
    int rest = item - s_items[b];
    b *= kItemStep;
    const int lane = (int)threadIdx.x & 31, own = lane < kItemStep && b + lane < a.tab.seqs ? tile_items<D>(a, b + lane) : 0;
    for (int k = 0; k < kItemStep - 1; ++k) {
        const int cnt = __shfl_sync(0xFFFFFFFFu, own, k);
        if (rest < cnt) break;
        rest -= cnt;
        ++b;
    }
    t.b = b;
    query_rows(a, b, t.row0, t.n);
    t.len = kv_length(a.tab, b, a.pool.page_log2, a.status);
    t.rows = t.n * a.group;
    t.splits = tile_splits(t.rows, t.len, a.pool.heads, D);
    const int tiles = (t.rows + tile_rows(D) - 1) / tile_rows(D);
    t.head = rest % a.pool.heads;
    rest /= a.pool.heads;
    t.split = rest % t.splits;
    t.tile = tiles - 1 - rest / t.splits;
    t.first = t.tile * tile_rows(D);
    t.rn = min(tile_rows(D), t.rows - t.first);
    const int per = tile_split_tokens(t.len, t.splits);
    t.tok0 = t.split * per;
    int end = min(t.len, t.tok0 + per);
    if (a.causal) end = min(end, max(0, t.len - t.n + (t.first + t.rn - 1) / a.group + 1));
    t.steps = end > t.tok0 ? (end - t.tok0 + Tile<D>::kStep - 1) / Tile<D>::kStep : 0;
    return t;
}

// Products and commits issued by one lane of a warp that stays together
// (elect.sync picks the same lane each time): an MMA then costs its warp about 24
// cycles of issue, against 55 to 90 from a branch that one thread runs alone.
__device__ __forceinline__ void mma_f16_warp(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_f16_tmem(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                             uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void commit_warp(uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n"
        ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
          "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Untiled copy to shared memory: 16-byte aligned addresses and size; completion
// is signalled as transaction bytes on `bar`.
__device__ __forceinline__ void bulk_copy(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Descriptor of the values as the right-hand operand of O = P V, "MN-major":
// 64 dimensions of a token are a 128-byte row, eight tokens a 1,024-byte atom
// (the stride between groups of eight k, bits 32-45), the next 64 dimensions a
// chunk further (bits 16-29); 128-byte swizzle.
__device__ __forceinline__ uint64_t sdesc_values(uint32_t smem_addr, uint32_t chunk_bytes) {
    return (uint64_t)((smem_addr & 0x3FFFFu) >> 4) | ((uint64_t)(chunk_bytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ uint64_t pair_of(float x) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(x));
    return r;
}

// mbar_wait for a whole warp: the same answer in every lane, so that the warp
// stays together for the aligned instructions that follow.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, const WaitCtx &w, unsigned int site) {
    return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, w, site));
}

struct TileBars {
    uint64_t q_full[2], k_full[2], k_empty[2], v_full[4], v_empty[4], s_full[2], p_half[2], p_full[2], o_done[2];
    uint64_t raw_full[2][4], raw_empty[2][4];      // of keys and of values
    uint64_t pair[4], never, drain[2], item_full[2], item_empty[2];
};

// Step number i of a pipeline of N stages: its stage, and the parity of the
// barrier phase that its use number completes.
template <int N>
__device__ __forceinline__ int stage_of(uint32_t i) { return (int)(i % N); }
template <int N>
__device__ __forceinline__ uint32_t parity_of(uint32_t i) { return i / N & 1u; }

// Where S number n of row tile q is and, the same way, the product P V number n:
// its place and barriers, and the parity of the phase.  With one row tile the
// next S is under way before the last product is, so two of each may be
// outstanding; they take turns on two places, as a parity tells a phase only
// from the one before it.
template <typename T>
__device__ __forceinline__ int slot_of(int q, uint32_t n) { return T::kSlots == 1 ? q : (int)(n & 1u); }
template <typename T>
__device__ __forceinline__ uint32_t turn_of(uint32_t n) { return T::kSlots == 1 ? n & 1u : n >> 1 & 1u; }

// Scales of the pages of a block of 64 tokens, kRing blocks deep.
struct BlockScales {
    float ks[4], lv[4], inv[4];    // key scale; log2 of the value scale; its reciprocal
    int odd;                       // bit p: page p's value scale is zero; bit 4: this block or one before it in the item has a far one
};

// 128 rows of query i * G + head g at a time (two such tiles up to dim 128),
// against 128 tokens (64 at dim 256) a step.  Per row tile and step:
//   S = Q K^T         tcgen05, both operands fp16 in shared memory
//   softmax           a thread a row (two at dim 256): S from tensor memory, the row's
//                     maximum, the exponentials, P in fp16 back over S
//   O += P V          tcgen05, P from tensor memory, V from shared memory
// Two warps copy the codes of the steps' pages to shared memory, several blocks
// ahead, keys and values each at their own pace; eight turn them into fp16 operands in the 128-byte swizzle.  With two row
// tiles the products of one run while the other's softmax does.  At dim 256,
// whose O leaves room for one row tile only, the next step's S runs while the
// softmax of this one does.
//
// The row's reference m is a running maximum of x_j + log2 vs(page(j)): the
// weights of P are exp2(x_j + log2 vs - m + 11), and the softmax's sum takes each
// page's part times 1 / vs (or, past a far scale, is a sum of its own).  O is rescaled only when the
// maximum has grown by more than 2^4 (the weights are then at most 2^15, within fp16).
//
// Measured: 2,270 rows x 32 heads over as many e4m3 tokens, 8 heads of 128, causal:
// 65 us, 645 TFLOP/s; 8 x 48 rows x 24 heads over 1,550 int8 tokens, 4 heads of 256:
// 50 us, 288 TFLOP/s.  Bound by the chain of a row tile's step, S, softmax, P V
// (4,500 cycles for 128 tokens at dim 128, of which 2,300 softmax; the tensor cores
// work for 2,000 of them with two row tiles), and by what surrounds the steps of an
// item: 12,000 cycles before the first one, 7,000 to write the rows.
template <int KIND, int D>
__global__ void __launch_bounds__(Tile<D>::kThreadsAll, 1) kv_tile_kernel(const AttnArgs a) {
    using T = Tile<D>;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    __shared__ TileBars bar;
    __shared__ BlockScales s_scale[kRing];
    __shared__ int s_there[2][kRing];              // bit p: page p of the block is one of the pool
    __shared__ float s_qs[T::kQ * 128], s_pair[2][2][128];   // rows' query scales; what the threads of a row exchange
    __shared__ float s_ref[T::kSoftWarps * 32];              // past a far scale: the reference of a softmax thread's sum
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort, s_scan[32], s_total;
    __shared__ TileItem s_item[2];
    uint8_t *smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    int *s_items = reinterpret_cast<int *>(smem_raw + T::kSmem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, log2 = a.pool.page_log2, H = a.pool.heads;

    if (tid == 0) {
        s_abort = 0;
        s_total = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.q_full[i], 8 / T::kQ);
            mbar_init(&bar.p_full[i], 8 / T::kQ);
            mbar_init(&bar.p_half[i], 8 / T::kQ);
            mbar_init(&bar.k_full[i], T::kConvWarps);
            mbar_init(&bar.k_empty[i], T::kQ);
            mbar_init(&bar.drain[i], 1);
            mbar_init(&bar.item_full[i], 1);
            mbar_init(&bar.item_empty[i], T::kSoftWarps + 2 * T::kConvWarps + T::kQ + 1);
            mbar_init(&bar.s_full[i], 1);
            mbar_init(&bar.o_done[i], 1);
            for (int k = 0; k < 4; ++k) {
                mbar_init(&bar.raw_full[i][k], 1);
                mbar_init(&bar.raw_empty[i][k], T::kConvWarps);
            }
        }
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.v_full[i], T::kConvWarps);
            mbar_init(&bar.v_empty[i], T::kQ);
            mbar_init(&bar.pair[i], 2);
        }
        mbar_init(&bar.never, 1);
        fence_barrier_init();
    }
    if (warp == T::kMmaWarp) {
        tmem_alloc(&s_tmem, T::kTmemCols);
        tmem_relinquish();
    }
    pdl_wait();
    __syncthreads();
    for (int b0 = 0; b0 < a.tab.seqs; b0 += T::kThreadsAll) {
        const int b = b0 + tid, cnt = b < a.tab.seqs ? tile_items<D>(a, b) : 0;
        int inc = cnt;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
            if (lane >= o) inc += v;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int base = s_total, all = 0;
        for (int w = 0; w < T::kThreadsAll / 32; ++w) {
            if (w < warp) base += s_scan[w];
            all += s_scan[w];
        }
        if (b < a.tab.seqs && b % kItemStep == 0) s_items[b / kItemStep] = base + inc - cnt;
        __syncthreads();
        if (tid == 0) s_total += all;
        __syncthreads();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const int items = s_total;
    const uint32_t tmem = s_tmem;
    const WaitCtx wait = {a.wait_limit_ns, &s_abort, a.status};
    // the item of a round, from the warp that looks it up for all (the one that copies values)
    const auto take_item = [&](int round, TileItem &t) -> bool {
        if (!warp_wait(&bar.item_full[round & 1], (uint32_t)round >> 1 & 1u, wait, kSiteKvLoad)) return false;
        t = s_item[round & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.item_empty[round & 1]);
        return true;
    };

    if (warp < T::kSoftWarps) {
        // ---------------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
        const int q = T::kQ == 2 ? warp >> 2 : 0, half = T::kQ == 2 ? 0 : warp >> 2, quad = warp & 3;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const GroupDiv by(a.group);
        uint32_t ns = 0, npv = 0, step_no = 0, pairs = 0;   // S and O products of this row tile so far; steps of the CTA
        bool ok = true;
        // the warps that share rows meet (a time-limited wait, unlike a named barrier)
        const auto pair_sync = [&]() -> bool {
            __syncwarp();
            if constexpr (T::kQ == 1) {
                if (lane == 0) mbar_arrive(&bar.pair[quad]);
                return warp_wait(&bar.pair[quad], pairs++ & 1u, wait, kSiteKvSoftmax);
            }
            return true;
        };
        for (int round = 0; round * (int)gridDim.x < items && ok; ++round) {
            if (round_item(round) >= items) break;
            TileItem t;
            if (!take_item(round, t)) break;
            const uint32_t step0 = step_no;
            step_no += (uint32_t)t.steps;
            const int mine = min(128, t.rn - q * 128);     // rows of this tile
            if (mine <= 0) continue;
            const int row = quad * 32 + lane;              // this thread's row of the tile
            const int r = t.first + q * 128 + min(row, mine - 1);
            // query and head of row rr of this tile: i0 + (g0 + rr) / G and the rest
            const int i0 = (t.first + q * 128) / a.group, g0 = t.first + q * 128 - i0 * a.group;
            const int i = i0 + by.div(g0 + min(row, mine - 1)), hq = t.head * a.group + r - i * a.group;
            uint8_t *sq = smem + T::kSmemQ + q * T::kQuery;

            // queries of the warp's rows to shared memory, each row scaled by a power of two
            float qs = 0.0f;
            if (t.steps > 0) {
                constexpr int LPR = D / 16, RPI = 32 / LPR;              // lanes of a row, rows at a time
                constexpr int WROWS = 32 * T::kQ / 2, ITER = WROWS / RPI;
                const int lr = lane / LPR, lu = lane % LPR, base = quad * 32 + half * WROWS + lr;
                constexpr int AHEAD = ITER < 8 ? ITER : 8;      // rounds whose loads are on their way at a time
#pragma unroll 1
                for (int k0 = 0; k0 < ITER; k0 += AHEAD) {
                    uint4 v[AHEAD][2];
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k) {
                        const int x = g0 + min(base + (k0 + k) * RPI, mine - 1), qi = by.div(x);
                        const uint16_t *src = a.q + (int64_t)(t.row0 + i0 + qi) * a.ldq +
                                              (int64_t)(t.head * a.group + x - qi * a.group) * a.ldq_head + lu * 8;
                        v[k][0] = *reinterpret_cast<const uint4 *>(src);
                        v[k][1] = *reinterpret_cast<const uint4 *>(src + LPR * 8);
                    }
#pragma unroll
                    for (int k = 0; k < AHEAD; ++k) {
                        const int rr = base + (k0 + k) * RPI;
                        uint32_t w[8] = {v[k][0].x, v[k][0].y, v[k][0].z, v[k][0].w, v[k][1].x, v[k][1].y, v[k][1].z, v[k][1].w};
                        uint32_t top = 0;
#pragma unroll
                        for (int x = 0; x < 8; ++x) {
                            if (rr >= mine) w[x] = 0u;
                            top = __vmaxu2(top, w[x] & 0x7FFF7FFFu);
                        }
#pragma unroll
                        for (int o = 1; o < LPR; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
                        top = max(top & 0xFFFFu, top >> 16) << 16;
                        const int e = top ? min(120, 13 - (int)(top >> 23) + 127) : 0;      // -115 or more
                        // a negative scale turns the queries, so that x grows with S
                        float up = row_factor(top, e);
                        if (a.scale_log2 < 0.0f) up = -up;
#pragma unroll
                        for (int x = 0; x < 8; ++x)
                            w[x] = pack_half(__uint_as_float(w[x] << 16) * up, __uint_as_float(w[x] & 0xFFFF0000u) * up);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const int u = lu + x * LPR;
                            *reinterpret_cast<uint4 *>(sq + (u >> 3) * T::kChunkQ + rr * 128 + (((u & 7) ^ (rr & 7)) << 4)) =
                                make_uint4(w[4 * x], w[4 * x + 1], w[4 * x + 2], w[4 * x + 3]);
                        }
                        if (lu == 0) s_qs[q * 128 + rr] = fabsf(a.scale_log2) * __uint_as_float((uint32_t)(127 - e) << 23);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.q_full[q]);
                if (!pair_sync()) break;
                qs = s_qs[q * 128 + row];
            }

            const int sees = a.causal ? max(0, t.len - t.n + i + 1) : t.len;    // tokens this row sees
            float m = -INFINITY, l = 0.0f;
            bool apart = false;      // the sum's reference is s_ref[tid], not m
            for (int s = 0; s < t.steps; ++s) {
                const int slot = slot_of<T>(q, ns);
                const uint32_t ts = tmem + (uint32_t)(slot * T::kStep + half * T::kCols) + lanes;
                if (!warp_wait(&bar.s_full[slot], turn_of<T>(ns), wait, kSiteKvSoftmax)) {
                    ok = false;
                    break;
                }
                ++ns;
                tc_fence_after();
                const int seen = sees - (t.tok0 + s * T::kStep) - half * T::kCols;   // of this thread's columns, what its row sees
                const int p0 = half * T::kCols;      // first column, for the page of a column
                const auto scales_at = [&](int c) -> const BlockScales & {
                    return s_scale[((step0 + (uint32_t)s) * T::kSub + (uint32_t)((p0 + c) >> 6)) % kRing];
                };
                int odd = scales_at(0).odd;
                if (T::kCols > 64) odd |= scales_at(64).odd;
                const bool far = odd >= 16;
                // whole steps take code without masks (the compiler turns a test in the loops into selects
                // for every column: 1,120 + 2,040 cycles for 128 columns instead of 450 + 1,350)
                const int least = __reduce_min_sync(0xFFFFFFFFu, seen);
                const bool whole = least >= T::kCols && odd == 0;

                const int most = __reduce_max_sync(0xFFFFFFFFu, seen);

                // the largest x + log2 vs
                uint32_t va[32], vb[32];
                float top = -INFINITY, top_x = -INFINITY;
                const auto largest = [&](const uint32_t *v, int c, auto two) {      // of columns c .. c + 15
                    const BlockScales &sc = scales_at(c);
                    const int p = ((p0 + c) & 63) >> log2;
                    float g[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) g[k] = fmaxf(__uint_as_float(v[k]), __uint_as_float(v[8 + k]));
#pragma unroll
                    for (int w = 4; w > 0; w >>= 1)
#pragma unroll
                        for (int k = 0; k < w; ++k) g[k] = fmaxf(g[k], g[k + w]);
                    if constexpr (decltype(two)::value) {
                        top_x = fmaxf(top_x, g[0] * (qs * sc.ks[p]));
                        if (sc.odd >> p & 1) return;
                    }
                    top = fmaxf(top, fmaf(g[0], qs * sc.ks[p], sc.lv[p]));
                };
                if (whole) {
#pragma unroll
                    for (int c = 0; c < T::kCols; c += 64) {
                        tmem_ld32(ts + (uint32_t)c, va);
                        if constexpr (T::kCols >= 64) tmem_ld32(ts + (uint32_t)c + 32u, vb);
                        tmem_ld_wait();
#pragma unroll
                        for (int h = 0; h < (T::kCols < 64 ? T::kCols : 64) / 16; ++h)
                            largest(h < 2 ? va + h * 16 : vb + (h - 2) * 16, c + h * 16, std::false_type());
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < T::kCols && c < most; c += 32) {
                        tmem_ld32(ts + (uint32_t)c, va);
                        tmem_ld_wait();
                        if (c + 32 > least) {
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                if (c + k >= seen) va[k] = 0xFF800000u;
                        }
                        // (keys of a column that is not seen have a place below all others, whatever their page's scale)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            if (!far && c + h * 16 < seen) largest(va + h * 16, c + h * 16, std::false_type());
                        if (__builtin_expect(far, 0)) {
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                if (c + h * 16 < seen) largest(va + h * 16, c + h * 16, std::true_type());
                        }
                    }
                }
                if constexpr (T::kQ == 1) {
                    s_pair[s & 1][half][row] = top;
                    if (!pair_sync()) {
                        ok = false;
                        break;
                    }
                    top = fmaxf(top, s_pair[s & 1][half ^ 1][row]);
                }
                float ml = 0.0f;
                if (__builtin_expect(far, 0)) {
                    if constexpr (T::kQ == 1) {      // (read at the next exchange's place once all have passed this one)
                        if (!pair_sync()) {
                            ok = false;
                            break;
                        }
                        s_pair[s & 1][half][row] = top_x;
                        if (!pair_sync()) {
                            ok = false;
                            break;
                        }
                        top_x = fmaxf(top_x, s_pair[s & 1][half ^ 1][row]);
                    }
                    const float was = apart ? s_ref[tid] : m;
                    apart = true;
                    ml = fmaxf(was, top_x);
                    l *= ex2_diff(was, ml);
                    s_ref[tid] = ml;
                }
                if (__any_sync(0xFFFFFFFFu, top > m + kSlack || (m == -INFINITY && top != -INFINITY))) {
                    const float mn = fmaxf(m, top), f = ex2_diff(m, mn);
                    m = mn;
                    if (!far) l *= f;
                    if (s > 0) {
                        // O is at rest once the product before this step's is done
                        if (!warp_wait(&bar.o_done[slot_of<T>(q, npv - 1)], turn_of<T>(npv - 1), wait, kSiteKvSoftmax)) {
                            ok = false;
                            break;
                        }
                        tc_fence_after();
                        const uint32_t to = tmem + T::kTmemO + (uint32_t)(q * 128 + half * T::kOutCols) + lanes;
#pragma unroll 1
                        for (int c = 0; c < T::kOutCols / 16; ++c) {
                            uint32_t v[16];
                            tmem_ld16(to + (uint32_t)(c * 16), v);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * f);
                            tmem_st16(to + (uint32_t)(c * 16), v);
                        }
                        tmem_st_wait();
                    }
                }
                const float ref = m == -INFINITY ? 0.0f : m - (kLift - kSlack);
                const auto weights = [&](const uint32_t *v, int c) {      // of columns c .. c + 31
                    uint32_t o[16];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const BlockScales &sc = scales_at(c);
                        const int p = ((p0 + c + h * 16) & 63) >> log2;
                        const uint64_t f2 = pair_of(qs * sc.ks[p]), off2 = pair_of(sc.lv[p] - ref);
                        uint64_t g[2] = {0, 0};
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            uint64_t x;
                            float y, z;
                            asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(v[h * 16 + 2 * k]), "r"(v[h * 16 + 2 * k + 1]));
                            asm("fma.rn.f32x2 %0, %0, %1, %2;" : "+l"(x) : "l"(f2), "l"(off2));
                            asm("mov.b64 {%0, %1}, %2;" : "=f"(y), "=f"(z) : "l"(x));
                            y = ex2(y);
                            z = ex2(z);
                            asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "f"(y), "f"(z));
                            asm("add.rn.f32x2 %0, %0, %1;" : "+l"(g[k & 1]) : "l"(x));
                            o[h * 8 + k] = pack_half(y, z);
                        }
                        float y, z;
                        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(g[0]) : "l"(g[1]));
                        asm("mov.b64 {%0, %1}, %2;" : "=f"(y), "=f"(z) : "l"(g[0]));
                        l = fmaf(y + z, sc.inv[p], l);
                    }
                    tmem_st16(ts + (uint32_t)(c / 2), o);
                };
                // the product starts when the first of two blocks is there
                const auto half_done = [&]() {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_half[slot]);
                };
                if (whole) {
#pragma unroll
                    for (int c = 0; c < T::kCols; c += 64) {
                        if constexpr (T::kCols > 64) {
                            tmem_ld32(ts + (uint32_t)c, va);
                            tmem_ld32(ts + (uint32_t)c + 32u, vb);
                            tmem_ld_wait();
                        }
                        weights(va, c);
                        if constexpr (T::kCols >= 64) weights(vb, c + 32);
                        if (T::kCols > 64 && c == 0) half_done();
                    }
                } else {
#pragma unroll 1
                    for (int c = 0; c < T::kCols; c += 32) {
                        if (T::kCols > 64 && c == 64) half_done();
                        if (c + 32 <= least && odd == 0) {      // seen by every row of the warp
                            tmem_ld32(ts + (uint32_t)c, va);
                            tmem_ld_wait();
                            weights(va, c);
                            continue;
                        }
                        uint32_t o[16];
                        if (c >= most) {                      // by none
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = 0u;
                            tmem_st16(ts + (uint32_t)(c / 2), o);
                            continue;
                        }
                        tmem_ld32(ts + (uint32_t)c, va);
                        tmem_ld_wait();
                        const BlockScales &sc = scales_at(c);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int c0 = c + h * 16, p = ((p0 + c0) & 63) >> log2;
                            const float f = qs * sc.ks[p], off = sc.lv[p] - ref;
                            const uint32_t keep = (sc.odd >> p & 1) ? 0u : 0xFFFFFFFFu;
                            float g = 0.0f;
#pragma unroll
                            for (int k = 0; k < 16; k += 2) {
                                const float y = c0 + k < seen ? ex2(fmaf(__uint_as_float(va[h * 16 + k]), f, off)) : 0.0f;
                                const float z = c0 + k + 1 < seen ? ex2(fmaf(__uint_as_float(va[h * 16 + k + 1]), f, off)) : 0.0f;
                                g += y + z;
                                o[h * 8 + k / 2] = pack_half(y, z) & keep;
                            }
                            if (__builtin_expect(far, 0)) {
                                const float off_l = (kLift - kSlack) - ml;
#pragma unroll
                                for (int k = 0; k < 16; ++k)
                                    l += c0 + k < seen ? ex2(fmaf(__uint_as_float(va[h * 16 + k]), f, off_l)) : 0.0f;
                            } else {
                                l = fmaf(g, sc.inv[p], l);
                            }
                        }
                        tmem_st16(ts + (uint32_t)(c / 2), o);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[slot]);
                ++npv;
            }
            if (!ok) break;

            // the rows' results, through shared memory in the place and layout of the warp's
            // queries (whose last product is done), so that whole rows leave at a time
            if (t.steps > 0 && !warp_wait(&bar.o_done[slot_of<T>(q, npv - 1)], turn_of<T>(npv - 1), wait, kSiteKvSoftmax)) break;
            tc_fence_after();
            if constexpr (T::kQ == 1) {
                s_pair[0][half][row] = l;
                if (!pair_sync()) break;
                l += s_pair[0][half ^ 1][row];
            }
            const float inv = l == 0.0f ? 0.0f : __fdiv_rn(1.0f, l);      // (NaN stays)
            const float ml = apart ? s_ref[tid] : m;
            if (row < mine && half == 0) {
                const float lse = l == 0.0f ? -INFINITY : ml - (kLift - kSlack) + log2f(l);
                if (t.splits > 1)
                    a.part_lse[a.many.of(t.b, t.row0) + ((int64_t)t.head * t.rows + r) * t.splits + t.split] = lse;
                else if (a.lse)
                    a.lse[(int64_t)(t.row0 + i) * a.q_heads + hq] = lse == -INFINITY ? -INFINITY : lse * (1.0f / kLog2e);
            }
            constexpr int CHUNKS = T::kOutCols / 64;             // 128-byte chunks of the warp's rows
            const bool part = t.splits > 1, none = l == 0.0f;
            uint8_t *stage = sq + half * CHUNKS * T::kChunkQ + quad * 32 * 128;
            for (int pass = 0; pass < (part ? 2 : 1); ++pass) {          // fp32 takes two
                // 32 columns at a time: four 16-byte units of bf16, or eight of fp32
                const int groups = part ? T::kOutCols / 64 : T::kOutCols / 32;
                const auto put = [&](int u, uint4 o) {
                    *reinterpret_cast<uint4 *>(stage + (u >> 3) * T::kChunkQ + lane * 128 + (((u & 7) ^ (lane & 7)) << 4)) = o;
                };
#pragma unroll 1
                for (int c = 0; c < groups; ++c) {
                    uint32_t v[32];
                    // (rows without a step have nothing there, and `none`)
                    tmem_ld32(tmem + T::kTmemO + (uint32_t)(q * 128 + half * T::kOutCols + (pass * groups + c) * 32) + lanes, v);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = none ? 0u : __float_as_uint(__uint_as_float(v[k]) * inv);
                    if (apart) {
                        const float back = ex2(0.5f * (m - ml));
#pragma unroll
                        for (int k = 0; k < 32; ++k) v[k] = none ? 0u : __float_as_uint(__uint_as_float(v[k]) * back * back);
                    }
                    if (part) {
#pragma unroll
                        for (int u = 0; u < 8; ++u) put(c * 8 + u, make_uint4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]));
                    } else {
                        uint32_t w[16];
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1]));
                            w[k] = *reinterpret_cast<const uint32_t *>(&b2);
                        }
#pragma unroll
                        for (int u = 0; u < 4; ++u) put(c * 4 + u, make_uint4(w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]));
                    }
                }
                __syncwarp();
                constexpr int UNITS = CHUNKS * 8, RPI = 32 / UNITS;      // 16-byte units of a row, rows at a time
                const int u = lane % UNITS, lr = lane / UNITS;
#pragma unroll 4
                for (int k = 0; k < 32; k += RPI) {
                    const int rr = quad * 32 + k + lr;
                    if (rr < mine) {
                        const uint4 o = *reinterpret_cast<const uint4 *>(stage + (u >> 3) * T::kChunkQ + (k + lr) * 128 +
                                                                         (((u & 7) ^ ((k + lr) & 7)) << 4));
                        const int ra = t.first + q * 128 + rr;
                        if (t.splits > 1) {
                            const int64_t place = a.many.of(t.b, t.row0) + ((int64_t)t.head * t.rows + ra) * t.splits + t.split;
                            *reinterpret_cast<uint4 *>(a.part + place * D + half * T::kOutCols + pass * (T::kOutCols / 2) + u * 4) = o;
                        } else {
                            const int x = g0 + rr, qi = by.div(x);
                            *reinterpret_cast<uint4 *>(a.out + (int64_t)(t.row0 + i0 + qi) * a.ldo +
                                                       (int64_t)(t.head * a.group + x - qi * a.group) * a.ldo_head +
                                                       half * T::kOutCols + u * 8) = o;
                        }
                    }
                }
                __syncwarp();
            }
            tc_fence_before();
            // before the next queries are written where the other warp of these rows may still be reading
            if (!pair_sync()) break;
        }
    } else if (warp < T::kMmaWarp) {
        // ---------------------------------------------------------- codes to operands
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        const bool values = warp >= T::kSoftWarps + T::kConvWarps;
        const int ct = (tid - T::kSoftWarps * 32) % (T::kConvWarps * 32);
        constexpr int PIECES = D / 16, N = 64 * PIECES / (T::kConvWarps * 32);   // 16-byte pieces of a row; of a thread and block
        constexpr int AT_ONCE = 2;
        const int crow = ct / PIECES, piece = ct % PIECES;
        // a piece becomes two 16-byte units of a row
        const int chunk = piece >> 2, unit = (piece & 3) * 2, swap = (chunk & 1) * 16;
        uint64_t *full = values ? bar.v_full : bar.k_full, *empty = values ? bar.v_empty : bar.k_empty;
        uint64_t *raw_full = bar.raw_full[values], *raw_empty = bar.raw_empty[values];
        const uint8_t *raw = smem + T::kSmemRaw + (values ? T::kRawK * T::kCodes : 0);
        uint8_t *operands = smem + (values ? T::kSmemV + chunk * T::kChunkV : T::kSmemK + chunk * T::kChunkK);
        uint32_t step_no = 0, block = 0;
        bool ok = true;
        for (int round = 0; round * (int)gridDim.x < items && ok; ++round) {
            if (round_item(round) >= items) break;
            TileItem t;
            if (!take_item(round, t)) break;
            for (int s = 0; s < t.steps && ok; ++s, ++step_no) {
#pragma unroll 1
                for (int sub = 0; sub < T::kSub; ++sub, ++block) {
                    // keys: a step a stage; values: a block
                    const int st = values ? stage_of<T::kVBlocks>(block) : stage_of<T::kKStages>(step_no);
                    const uint32_t turn = values ? parity_of<T::kVBlocks>(block) : parity_of<T::kKStages>(step_no);
                    const int rs = values ? stage_of<T::kRawV>(block) : stage_of<T::kRawK>(block);
                    const uint32_t raw_turn = values ? parity_of<T::kRawV>(block) : parity_of<T::kRawK>(block);
                    const bool last = values || sub == T::kSub - 1;
                    uint8_t *dst = operands + (values ? st * T::kBlockV : st * T::kOperand + sub * 64 * 128);
                    ok = warp_wait(&raw_full[rs], raw_turn, wait, kSiteKvLoad);
                    if (values || sub == 0) ok = ok && warp_wait(&empty[st], turn ^ 1u, wait, kSiteKvLoad);
                    if (!ok) break;
                    const int there = s_there[values][block % kRing], left = t.len - t.tok0 - s * T::kStep - sub * 64;
                    const uint8_t *src = raw + rs * T::kCodes + piece * 16;
                    // lanes of every second chunk take a piece's halves the other way round, so that the
                    // eight lanes of a store meet every bank once
                    const auto convert = [&](auto part) {
#pragma unroll
                        for (int k0 = 0; k0 < N; k0 += AT_ONCE) {
                            uint4 v[AT_ONCE];
#pragma unroll
                            for (int k = 0; k < AT_ONCE; ++k) {
                                const int rr = crow + (k0 + k) * (64 / N);
                                v[k] = *reinterpret_cast<const uint4 *>(src + rr * D);
                                // past the sequence's end anything may lie, NaN codes included
                                if (decltype(part)::value && (rr >= left || !(there >> (rr >> log2) & 1))) v[k] = make_uint4(0, 0, 0, 0);
                            }
#pragma unroll
                            for (int k = 0; k < AT_ONCE; ++k) {
                                const int rr = crow + (k0 + k) * (64 / N);
                                uint8_t *row = dst + rr * 128;
                                uint4 h;
                                const int at = ((unit ^ (rr & 7)) << 4) ^ swap;
                                widen4<KIND>(swap ? v[k].z : v[k].x, h.x, h.y);
                                widen4<KIND>(swap ? v[k].w : v[k].y, h.z, h.w);
                                *reinterpret_cast<uint4 *>(row + at) = h;
                                widen4<KIND>(swap ? v[k].x : v[k].z, h.x, h.y);
                                widen4<KIND>(swap ? v[k].y : v[k].w, h.z, h.w);
                                *reinterpret_cast<uint4 *>(row + (at ^ 16)) = h;
                            }
                        }
                    };
                    if (left >= 64 && there == (int)((2u << (63 >> log2)) - 1u))
                        convert(std::false_type());
                    else
                        convert(std::true_type());
                    if (last) fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&raw_empty[rs]);
                        if (last) mbar_arrive(&full[st]);
                    }
                }
            }
        }
    } else {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
      if (warp == T::kCopyWarp || warp == T::kCopyWarp + 1) {
        // ---------------------------------------------------------- codes to shared memory
        // A lane a page of the block: the page's run of tokens of this head is contiguous, one copy.  The
        // keys' warp also keeps the pages' scales for the softmax.
        const int plane = warp - T::kCopyWarp;
        const int run = min(64, a.pool.page), per = 64 / run;      // tokens of a page in a block; pages of a block
        const uint8_t *codes = a.pool.codes + plane * a.pool.plane_codes;
        uint8_t *raw = smem + T::kSmemRaw + plane * (T::kRawK * T::kCodes);
        uint32_t block = 0;
        bool ok = true;
        for (int round = 0; round * (int)gridDim.x < items && ok; ++round) {
            if (round_item(round) >= items) break;
            TileItem t;
            if (plane == 0) {
                if (!take_item(round, t)) break;
            } else {
                if (!warp_wait(&bar.item_empty[round & 1], ((uint32_t)round >> 1 & 1u) ^ 1u, wait, kSiteKvLoad)) break;
                t = tile_item<D>(a, s_items, round_item(round));
                if (lane == 0) {
                    s_item[round & 1] = t;
                    mbar_arrive(&bar.item_full[round & 1]);
                }
                __syncwarp();
            }
            if (t.steps == 0) continue;
            // 32 pages of the item and the next 32, one of each a lane: their numbers (-1 where there is
            // none) and scales, so that no step waits for a look-up
            struct Page {
                int page;
                float ks, vs;
            };
            const auto look_up = [&](int p) {
                Page x = {-1, 0.0f, 1.0f};
                if (p < (t.len + a.pool.page - 1) >> log2) {
                    x.page = a.tab.table[(int64_t)t.b * a.tab.ldt + p];
                    if (x.page < 0 || x.page >= a.pool.pages) {
                        record_status(a.status, kStatusBadPage);
                        x.page = -1;
                    } else if (plane == 0) {
                        const int64_t tile = (int64_t)x.page * H + t.head;
                        x.ks = a.pool.scales[tile];
                        x.vs = a.pool.scales[a.pool.plane_scales + tile];
                    }
                }
                return x;
            };
            int page0 = t.tok0 >> log2;
            bool far = false;
            Page now = look_up(page0 + lane), next = look_up(page0 + 32 + lane);
            for (int s = 0; s < t.steps * T::kSub; ++s, ++block) {
                const int rs = plane ? stage_of<T::kRawV>(block) : stage_of<T::kRawK>(block);
                const int t0 = t.tok0 + s * 64;
                if ((t0 >> log2) - page0 >= 32) {
                    page0 += 32;
                    now = next;
                    next = look_up(page0 + 32 + lane);
                }
                const int p = (t0 >> log2) - page0 + (lane < per ? lane : 0);      // under 64
                const bool later = p >= 32;
                const int page_a = __shfl_sync(0xFFFFFFFFu, now.page, p & 31), page_b = __shfl_sync(0xFFFFFFFFu, next.page, p & 31);
                const int page = lane < per && t0 + lane * run < t.len ? (later ? page_b : page_a) : -1;
                const unsigned int there = __ballot_sync(0xFFFFFFFFu, page >= 0);
                const uint32_t turn = plane ? parity_of<T::kRawV>(block) : parity_of<T::kRawK>(block);
                if (!warp_wait(&bar.raw_empty[plane][rs], turn ^ 1u, wait, kSiteKvLoad)) {
                    ok = false;
                    break;
                }
                if (plane == 0) {
                    const float ks_a = __shfl_sync(0xFFFFFFFFu, now.ks, p & 31), ks_b = __shfl_sync(0xFFFFFFFFu, next.ks, p & 31);
                    const float vs_a = __shfl_sync(0xFFFFFFFFu, now.vs, p & 31), vs_b = __shfl_sync(0xFFFFFFFFu, next.vs, p & 31);
                    const float ks = page >= 0 ? (later ? ks_b : ks_a) : 0.0f;
                    float vs = page >= 0 ? (later ? vs_b : vs_a) : 1.0f;
                    BlockScales &sc = s_scale[block % kRing];
                    const unsigned int zero = __ballot_sync(0xFFFFFFFFu, vs == 0.0f);
                    far = __any_sync(0xFFFFFFFFu, far || far_scale(vs));
                    if (vs == 0.0f) vs = 0x1p-60f;
                    if (lane < 4) {
                        sc.ks[lane] = ks;
                        sc.lv[lane] = log2f(vs);
                        sc.inv[lane] = __fdiv_rn(1.0f, vs);
                    }
                    if (lane == 0) sc.odd = (int)zero | (far ? 16 : 0);
                }
                if (lane == 0) s_there[plane][block % kRing] = (int)there;
                const int64_t at = ((((int64_t)page * H + t.head) << log2) + (t0 & (a.pool.page - 1))) * D;
                __syncwarp();
                if (lane == 0) mbar_arrive_expect_tx(&bar.raw_full[plane][rs], (uint32_t)(__popc(there) * run * D));
                __syncwarp();
                if (page >= 0) bulk_copy(raw + rs * T::kCodes + lane * run * D, codes + at, (uint32_t)(run * D), &bar.raw_full[plane][rs]);
            }
        }
        // no copy is in flight when the CTA ends
        const uint32_t depth = plane ? T::kRawV : T::kRawK;
        for (uint32_t k = block > depth ? block - depth : 0; k < block; ++k)
            warp_wait(&bar.raw_full[plane][plane ? stage_of<T::kRawV>(k) : stage_of<T::kRawK>(k)],
                      plane ? parity_of<T::kRawV>(k) : parity_of<T::kRawK>(k), wait, kSiteDrain);
      } else if (warp < T::kMmaWarp + T::kQ) {
        // ---------------------------------------------------------- products of row tile q
        const int q = warp - T::kMmaWarp;
        const uint32_t is = idesc_f32acc(0, 0, 128, T::kStep);
        const uint32_t io = idesc_f32acc(0, 0, 128, D) | (1u << 16);    // bit 16: the right-hand operand is MN-major
        const uint64_t dq = sdesc_sw128(smem_u32(smem + T::kSmemQ + q * T::kQuery)), dk = sdesc_sw128(smem_u32(smem + T::kSmemK));
        const uint64_t dv = sdesc_values(smem_u32(smem + T::kSmemV), T::kChunkV);      // offsets add to the address field
        const uint32_t to = tmem + T::kTmemO + (uint32_t)(q * 128);
        uint32_t nk = 0, nv = 0, nq = 0, ns = 0, npv = 0;
        bool ok = !a.force_timeout || warp_wait(&bar.never, 0, wait, kSiteKvMma);
        for (int round = 0; round * (int)gridDim.x < items && ok; ++round) {
            if (round_item(round) >= items) break;
            TileItem t;
            if (!take_item(round, t)) break;
            const bool here = q * 128 < t.rn;       // a tile without rows only gives its operands back
            const auto issue_s = [&](int s) -> bool {      // S of step s
                const int st = stage_of<T::kKStages>(nk);
                if (!warp_wait(&bar.k_full[st], parity_of<T::kKStages>(nk), wait, kSiteKvMma)) return false;
                if (here) {
                    if (s == 0 && !warp_wait(&bar.q_full[q], nq++ & 1u, wait, kSiteKvMma)) return false;
                    // its place is free once the product that read P from there is done
                    if (npv > 0 && !warp_wait(&bar.o_done[slot_of<T>(q, npv - 1)], turn_of<T>(npv - 1), wait, kSiteKvMma))
                        return false;
                    tc_fence_after();
                    const int slot = slot_of<T>(q, ns);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        mma_f16_warp(tmem + (uint32_t)(slot * T::kStep), dq + (uint32_t)(((k >> 2) * T::kChunkQ + (k & 3) * 32) >> 4),
                                     dk + (uint32_t)((st * T::kOperand + (k >> 2) * T::kChunkK + (k & 3) * 32) >> 4), is, k > 0);
                    commit_warp(&bar.s_full[slot]);
                    ++ns;
                }
                commit_warp(&bar.k_empty[st]);
                ++nk;
                return true;
            };
            const auto issue_o = [&](int s) -> bool {      // O += P V of step s
                const int slot = slot_of<T>(q, npv);
#pragma unroll
                for (int h = 0; h < T::kSub; ++h, ++nv) {
                    if (here && !warp_wait(h < T::kSub - 1 ? &bar.p_half[slot] : &bar.p_full[slot], turn_of<T>(npv), wait, kSiteKvMma))
                        return false;
                    const int st = stage_of<T::kVBlocks>(nv);
                    if (!warp_wait(&bar.v_full[st], parity_of<T::kVBlocks>(nv), wait, kSiteKvMma)) return false;
                    tc_fence_after();
                    if (here) {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int k = h * 4 + j;
                            mma_f16_tmem(to, tmem + (uint32_t)(slot * T::kStep + k * 16 / T::kCols * T::kCols + k * 16 % T::kCols / 2),
                                         dv + (uint32_t)((st * T::kBlockV + j * 2048) >> 4), io, s > 0 || k > 0);
                        }
                    }
                    commit_warp(&bar.v_empty[st]);
                }
                if (here) {
                    commit_warp(&bar.o_done[slot]);
                    ++npv;
                }
                return true;
            };
            for (int s = 0; s <= t.steps && t.steps > 0 && ok; ++s) {
                const bool has_s = s < t.steps, has_o = s > 0;
                // with two places the step's S goes ahead of the last step's O
                if (T::kSlots == 2 && has_s) ok = issue_s(s);
                if (has_o) ok = ok && issue_o(s - 1);
                if (T::kSlots == 1 && has_s) ok = ok && issue_s(s);
            }
        }
        // nothing is in flight when tensor memory is given back
        commit_warp(&bar.drain[q]);
        warp_wait(&bar.drain[q], 0, wait, kSiteDrain);
      }
      __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == T::kMmaWarp) tmem_dealloc(tmem, T::kTmemCols);
    pdl_launch_dependents();
}

// Joins the splits of each row: a CTA a row, its warps taking turns on the
// splits; the warps' sums are added in their order.  Bound by latency: 5 us for the
// rows of one sequence, 12 us for 2,496 rows of up to 16 splits.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(const AttnArgs a) {
    __shared__ float s_max[kWarps], s_sum[kWarps], s_o[kWarps][D];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, b = blockIdx.y, H = a.pool.heads;
    pdl_wait();
    int row0, n;
    query_rows(a, b, row0, n);
    const int rows = n * a.group, len = kv_length(a.tab, b, a.pool.page_log2, a.status);
    const int splits = rows <= kFewRows ? split_count(len) : tile_splits(rows, len, H, D);
    const int64_t first = (rows <= kFewRows ? a.few : a.many).of(b, row0);
    if (splits > 1)
        for (int64_t slot = blockIdx.x; slot < (int64_t)rows * H; slot += gridDim.x) {
            const int head = (int)(slot / rows), r = (int)(slot - (int64_t)head * rows);
            const float *pl = a.part_lse + first + slot * splits, *po = a.part + (first + slot * splits) * D;
            float mm = -INFINITY;
            for (int s = tid; s < splits; s += kThreads) mm = fmaxf(mm, pl[s]);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
            __syncthreads();      // the row before is done with shared memory
            if (lane == 0) s_max[warp] = mm;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_max[w]);
            float o[D / 32], sum = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) o[k] = 0.0f;
#pragma unroll 4
            for (int s = warp; s < splits; s += kWarps) {
                const float w = ex2_diff(pl[s], mm);
                const float2 *p = reinterpret_cast<const float2 *>(po + (int64_t)s * D);
                sum += w;
#pragma unroll
                for (int k = 0; k < D / 64; ++k) {
                    const float2 v = p[lane + 32 * k];
                    o[2 * k] = fmaf(w, v.x, o[2 * k]);
                    o[2 * k + 1] = fmaf(w, v.y, o[2 * k + 1]);
                }
            }
            if (lane == 0) s_sum[warp] = sum;
#pragma unroll
            for (int k = 0; k < D / 64; ++k)
                *reinterpret_cast<float2 *>(&s_o[warp][64 * k + 2 * lane]) = make_float2(o[2 * k], o[2 * k + 1]);
            __syncthreads();
            sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
            const float inv = sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);      // (NaN stays)
            const int i = r / a.group, hq = head * a.group + r - i * a.group;
            uint16_t *dst = a.out + (int64_t)(row0 + i) * a.ldo + (int64_t)hq * a.ldo_head;
            for (int d = tid * 2; d < D; d += 2 * kThreads) {
                const float x = (s_o[0][d] + s_o[1][d]) + (s_o[2][d] + s_o[3][d]);
                const float y = (s_o[0][d + 1] + s_o[1][d + 1]) + (s_o[2][d + 1] + s_o[3][d + 1]);
                *reinterpret_cast<__nv_bfloat162 *>(dst + d) = __floats2bfloat162_rn(x * inv, y * inv);
            }
            if (a.lse && tid == 0)
                a.lse[(int64_t)(row0 + i) * a.q_heads + hq] = sum == 0.0f ? -INFINITY : (mm + log2f(sum)) * (1.0f / kLog2e);
        }
    pdl_launch_dependents();
}

template <int KIND, int D, int NT>
cudaError_t launch_split(const AttnArgs &a, int64_t items, int sms, cudaStream_t st) {
    const size_t smem = (size_t)split_smem_floats<D, NT>() * 4 + (size_t)(a.tab.seqs + 1) * 4;
    static SmemOptIn opt;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(kv_split_kernel<KIND, D, NT>),
                            (size_t)split_smem_floats<D, NT>() * 4 + (kKvMaxSeqs + 1) * 4);
    if (e != cudaSuccess) return e;
    const int64_t most = (int64_t)sms * split_ctas<D, NT>();
    return launch_kernel(kv_split_kernel<KIND, D, NT>, dim3((unsigned)(items < most ? items : most)), dim3(kThreads), smem,
                         st, 1, true, a);
}

template <int KIND, int D>
cudaError_t launch_tile(const AttnArgs &a, int64_t items, int sms, cudaStream_t st) {
    using T = Tile<D>;
    const size_t smem = (size_t)T::kSmem + (size_t)((a.tab.seqs + kItemStep - 1) / kItemStep + 1) * 4;
    static SmemOptIn opt;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(kv_tile_kernel<KIND, D>), (size_t)T::kSmem + (kKvMaxSeqs / kItemStep + 1) * 4);
    if (e != cudaSuccess) return e;
    return launch_kernel(kv_tile_kernel<KIND, D>, dim3((unsigned)(items < sms ? items : sms)), dim3(T::kThreadsAll), smem,
                         st, 1, true, a);
}

// What the host knows of a call's rows: which kernels it needs, how many items
// each may have, and the places for partial results of a sequence.
struct Plan {
    bool few, tile;
    int row_max;                     // most rows a key/value head of a sequence with few
    int64_t few_items, tile_items;   // at most
    Places few_at, many_at;
    int64_t places;                  // 0: nothing is split
    int64_t join_rows;               // rows of a sequence that may be split, over its heads, at most
};

Plan make_plan(int64_t rows, bool ragged, int64_t seqs, int group, int heads, int dim, int64_t max_len) {
    Plan p = {};
    if (rows == 0 || seqs == 0) return p;
    // a shorter sequence may be cut into more runs than the longest: the cut grows in steps
    int few_splits = 1;
    for (int64_t len : {max_len, (int64_t)1024, (int64_t)8192})
        if (len <= max_len && split_count((int)len) > few_splits) few_splits = split_count((int)len);
    const int64_t per = ragged ? rows * group : rows / seqs * group;   // rows of one sequence, at most
    const auto reserve = [&](Places &at, int64_t per_seq, int64_t per_row) {
        at = {p.places, per_seq, per_row};
        p.places += per_seq * seqs < per_row * rows ? per_seq * seqs : per_row * rows;
    };
    p.few = ragged || per <= kFewRows;
    p.tile = per > kFewRows;
    if (p.few) {
        p.row_max = (int)(per < kFewRows ? per : kFewRows);
        p.few_items = seqs * heads * ((p.row_max + 7) / 8) * few_splits;
        if (few_splits > 1) {
            p.join_rows = (int64_t)heads * p.row_max;
            reserve(p.few_at, p.join_rows * few_splits, (int64_t)heads * group * few_splits);
        }
    }
    if (p.tile) {
        const int tr = tile_rows(dim);
        // a split sequence has at most kTileSlots items
        p.tile_items = ragged ? (rows * group / tr + seqs) * heads + seqs * kTileSlots
                              : seqs * (((per + tr - 1) / tr) * heads * tile_splits((int)per, (int)max_len, heads, dim));
        // the most splits of a sequence of up to max_len tokens: of 1,024 and more, over the SMs that its
        // heads leave (one row tile)
        int64_t splits = ((max_len >> 7) + ((max_len & 127) != 0)) / 8;
        if (splits > kTileMaxSplits) splits = kTileMaxSplits;
        if (splits > kTileSlots / heads) splits = kTileSlots / heads;
        const bool cut = ragged ? splits > 1 : tile_splits((int)per, (int)max_len, heads, dim) > 1;
        if (cut) {
            const int64_t units = (int64_t)kTileSlots * tr, most = per * heads;      // a split sequence has at most kTileSlots items
            const int64_t join = units / 2 < most ? units / 2 : most;
            reserve(p.many_at, units < most * splits ? units : most * splits, (int64_t)heads * group * splits);
            if (p.join_rows < join) p.join_rows = join;
        }
    }
    return p;
}

template <int D>
cudaError_t launch_attention(const AttnArgs &a, int kind, const Plan &p, int sms, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (p.tile)
        e = kind == kKvInt8 ? launch_tile<kKvInt8, D>(a, p.tile_items, sms, st) : launch_tile<kKvE4m3, D>(a, p.tile_items, sms, st);
    if (e == cudaSuccess && p.few) {
        if (p.row_max <= 8)
            e = kind == kKvInt8 ? launch_split<kKvInt8, D, 1>(a, p.few_items, sms, st)
                                : launch_split<kKvE4m3, D, 1>(a, p.few_items, sms, st);
        else
            e = kind == kKvInt8 ? launch_split<kKvInt8, D, 2>(a, p.few_items, sms, st)
                                : launch_split<kKvE4m3, D, 2>(a, p.few_items, sms, st);
    }
    if (e != cudaSuccess || p.places == 0) return e;
    // a CTA a row, up to 64 CTAs an SM over all sequences
    int64_t x = p.join_rows;
    const int64_t most = (int64_t)sms * 64 / a.tab.seqs + 1;
    if (x > most) x = most;
    return launch_kernel(kv_join_kernel<D>, dim3((unsigned)x, (unsigned)a.tab.seqs), dim3(kThreads), 0, st, 1, true, a);
}

}  // namespace

}  // namespace clef

using namespace clef;

extern "C" int clef_kv_attention_workspace(int64_t rows, int ragged, int64_t seqs, int q_heads, int heads, int dim,
                                           int64_t max_len, int64_t *bytes) {
    if (!bytes) return kv_fail("null pointer");
    if (rows < 0 || rows > ((int64_t)1 << 30) || seqs < 0 || seqs > kKvMaxSeqs) return kv_fail("rows or sequences out of range");
    if (heads < 1 || q_heads < heads || q_heads % heads != 0) return kv_fail("q_heads must be a multiple of heads");
    if (dim != 64 && dim != 128 && dim != 256) return kv_fail("dim must be 64, 128 or 256");
    if (max_len < 0 || max_len > 0x7FFFFFFF) return kv_fail("max_len out of range");
    *bytes = make_plan(rows, ragged != 0, seqs, q_heads / heads, heads, dim, max_len).places * (dim + 1) * 4;
    return CLEF_OK;
}

extern "C" int clef_kv_attention(const void *q, int64_t ldq, int64_t ldq_head, int64_t rows, const int32_t *row_start,
                                 int q_heads, int kind, const void *codes, int64_t plane_bytes, const float *scales,
                                 int64_t plane_scales, int64_t pages, int heads, int page, int dim, const int32_t *table,
                                 int64_t ldt, int64_t seqs, int64_t width, const int32_t *lens, float scale, int causal,
                                 void *out, int64_t ldo, int64_t ldo_head, float *lse, void *workspace,
                                 int64_t workspace_bytes, void *stream) {
    AttnArgs a = {};
    int rc = kv_pool_args(a.pool, kind, const_cast<void *>(codes), plane_bytes, const_cast<float *>(scales), plane_scales,
                          2, pages, heads, page, dim);
    if (!rc) rc = kv_table_args(a.tab, table, ldt, seqs, width, lens);
    if (rc) return rc;
    if (q_heads < heads || q_heads % heads != 0) return kv_fail("q_heads must be a multiple of heads");
    if (rows < 0 || rows * q_heads > ((int64_t)1 << 30)) return kv_fail("rows out of range");
    if (rows == 0) return CLEF_OK;
    if (seqs == 0) return kv_fail("rows without a sequence");
    if (!row_start && rows % seqs != 0) return kv_fail("without row_start, rows must be a multiple of the sequences");
    if (!(fabsf(scale * kLog2e) <= 3.402823466e38f)) return kv_fail("scale must be finite, in units of log2 too");
    if (ldq < 0 || ldq_head < 0 || ldq % 8 || ldq_head % 8) return kv_fail("query pitches must be multiples of 8");
    if (ldo < dim || ldo_head < dim || ldo % 8 || ldo_head % 8) return kv_fail("output pitches must be multiples of 8 that hold a head");
    if (!q || !codes || !scales || !table || !lens || !out) return kv_fail("null pointer");
    if (kv_misaligned(q, 16) || kv_misaligned(out, 16) || kv_misaligned(workspace, 16) || kv_misaligned(lse, 4) ||
        kv_misaligned(row_start, 4))
        return kv_fail("q, out and workspace must be 16-byte, lse and row_start 4-byte aligned");
    const int64_t top = width * page < 0x7FFFFFFF ? width * page : 0x7FFFFFFF;
    const Plan plan = make_plan(rows, row_start != nullptr, seqs, q_heads / heads, heads, dim, top);
    const int64_t need = plan.places * (dim + 1) * 4;
    if (need > 0 && (!workspace || workspace_bytes < need)) return kv_fail("workspace smaller than clef_kv_attention_workspace says");
    int sms = 0;
    if ((rc = internal_device(&sms, &a.status))) return rc;
    a.q = static_cast<const uint16_t *>(q);
    a.ldq = ldq;
    a.ldq_head = ldq_head;
    a.out = static_cast<uint16_t *>(out);
    a.ldo = ldo;
    a.ldo_head = ldo_head;
    a.lse = lse;
    a.start = row_start;
    a.rows = (int)rows;
    a.per_seq = (int)(rows / seqs);
    a.group = q_heads / heads;
    a.q_heads = q_heads;
    a.causal = causal != 0;
    a.scale_log2 = scale * kLog2e;
    a.few = plan.few_at;
    a.many = plan.many_at;
    a.part = static_cast<float *>(workspace);
    a.part_lse = a.part + plan.places * dim;
    a.wait_limit_ns = internal_wait_limit(&a.force_timeout);
    sms = internal_launch_sms(sms);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dim == 64    ? launch_attention<64>(a, kind, plan, sms, st)
                          : dim == 128 ? launch_attention<128>(a, kind, plan, sms, st)
                                       : launch_attention<256>(a, kind, plan, sms, st);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "cache attention launch");
}
