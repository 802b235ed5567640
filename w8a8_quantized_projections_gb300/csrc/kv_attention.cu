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
// Numbers.  Codes are widened to fp16, exactly (INT8 integers; e4m3 values are
// multiples of 2^-9 up to 448).  A query row is scaled by a power of two to a
// largest magnitude in [2^13, 2^14) and held in fp16: bf16 has fewer bits than
// fp16, so only values under 2^-27 of the row's largest lose anything, less
// than fp32 sums do.  Products are summed in fp32.  The softmax keeps two
// running maxima: m of x for the sum of weights, and m2 of x + log2 vs for
// the weights that multiply values, so the weights p * vs rounded to fp16 (11
// bits against the output's 8) are at most 1 whatever the pages' scales are.
#include <cstdint>

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
constexpr int kMaxSplits = 64;
constexpr float kLog2e = 1.4426950408889634f;

// Tokens of a split of a sequence of `len` tokens: short enough that one
// sequence spreads over the SMs, long enough that the partial results (16 B
// a value and split against 1 B a code) stay a small part of the traffic.
__host__ __device__ inline int split_tokens(int len) {
    if (len <= 2048) return 128;
    if (len <= 8192) return 256;
    if (len <= 32768) return 512;
    const int t = (int)(((int64_t)len + kMaxSplits - 1) / kMaxSplits);
    return (t + 511) / 512 * 512;
}
__host__ __device__ inline int split_count(int len) {
    const int t = split_tokens(len);
    return (int)(((int64_t)len + t - 1) / t);
}

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
    float *part;                // [seqs * heads * row_cap][split_cap][dim] partial outputs
    float *part_lse;            // [seqs * heads * row_cap][split_cap], base 2
    int row_cap, split_cap;
    unsigned int *status;
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

// 2^(a - b) for running maxima, 0 when a is -inf (b may be -inf then too)
__device__ __forceinline__ float ex2_diff(float a, float b) { return a == -INFINITY ? 0.0f : ex2(a - b); }

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

// Tokens that a warp takes a step: two 16-token tiles where the registers allow.
template <int D>
__host__ __device__ constexpr int step_tiles() { return D <= 128 ? 2 : 1; }

template <int D, int NT>
__host__ __device__ constexpr int split_smem_floats() { return kWarps * NT * 8 * (D + 3); }

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
template <int KIND, int D, int NT>
__global__ void __launch_bounds__(kThreads) kv_split_kernel(const AttnArgs a) {
    constexpr int ROWS = NT * 8, TILES = step_tiles<D>(), STEP = TILES * 16, KB = D / 64, MT = D / 16;
    constexpr int VW = D / 32;               // 32-bit words of values a lane holds of each token
    constexpr int QPITCH = D + 4;            // fp16 elements: the lanes' 8-byte reads meet every bank once
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) uint16_t s_q[ROWS * QPITCH];
    __shared__ float s_qs[ROWS];
    __shared__ int s_end[ROWS];              // tokens a row sees
    __shared__ int s_page[64];               // pages of the split (at most 1,024 tokens at a time)
    __shared__ float s_ks[64], s_lv[64];
    float *s_o = reinterpret_cast<float *>(smem);          // [kWarps][ROWS][D], then m, l, m2
    float *s_m = s_o + kWarps * ROWS * D, *s_l = s_m + kWarps * ROWS, *s_m2 = s_l + kWarps * ROWS;
    int *s_items = reinterpret_cast<int *>(smem + split_smem_floats<D, NT>() * 4);   // [seqs + 1] first item of each sequence
    __shared__ int s_scan[kWarps], s_total;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int log2 = a.pool.page_log2, H = a.pool.heads;
    pdl_wait();

    // items of each sequence
    if (tid == 0) s_total = 0;
    __syncthreads();
    for (int b0 = 0; b0 < a.tab.seqs; b0 += kThreads) {
        int cnt = 0;
        if (b0 + tid < a.tab.seqs) {
            int row0, n;
            query_rows(a, b0 + tid, row0, n);
            if (n > 0) {
                const int len = kv_length(a.tab, b0 + tid, log2, a.status);
                const int rows = n * a.group;
                // a sequence without tokens still has rows of zeros to write
                const int sp = rows <= kFewRows ? max(1, split_count(len)) : 1;
                cnt = sp * ((rows + ROWS - 1) / ROWS) * H;
            }
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
    if (tid == 0) s_items[a.tab.seqs] = s_total;
    __syncthreads();
    const int items = s_total;

    for (int item = blockIdx.x; item < items; item += gridDim.x) {
        // the item's sequence, split, head and rows
        int b = 0;
        {
            int hi = a.tab.seqs;
            while (hi - b > 1) {
                const int mid = (b + hi) >> 1;
                if (s_items[mid] <= item) b = mid;
                else hi = mid;
            }
        }
        int row0, n;
        query_rows(a, b, row0, n);
        const int len = kv_length(a.tab, b, log2, a.status);
        const int rows = n * a.group, groups = (rows + ROWS - 1) / ROWS;
        int rest = item - s_items[b];
        const int head = rest % H;
        rest /= H;
        const int rg = rest % groups, split = rest / groups;
        const bool few = rows <= kFewRows;
        const int splits = few ? max(1, split_count(len)) : 1;
        const int tok0 = few ? split * split_tokens(len) : 0;
        int tok1 = few ? min(len, tok0 + split_tokens(len)) : len;
        const int r0 = rg * ROWS, rn = min(ROWS, rows - r0);
        if (a.causal) tok1 = min(tok1, max(0, len - n + (r0 + rn - 1) / a.group + 1));   // what the last row sees

        __syncthreads();   // the item before is done with shared memory
        // queries: row's largest magnitude to [2^13, 2^14), fp16
        for (int r = warp; r < ROWS; r += kWarps) {
            const int i = (r0 + r) / a.group, hq = head * a.group + (r0 + r) - i * a.group;
            const uint16_t *src = a.q + (int64_t)(row0 + i) * a.ldq + (int64_t)hq * a.ldq_head;
            float v[D / 32], top = 0.0f;
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                v[k] = r < rn ? __uint_as_float((uint32_t)*(src + lane + 32 * k) << 16) : 0.0f;
                top = fmaxf(top, fabsf(v[k]));
            }
            top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
            const int e = top > 0.0f ? max(-100, min(120, 13 - (int)((__float_as_uint(top) >> 23) & 0xFF) + 127)) : 0;
            const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const __half h = __float2half_rn(v[k] * up);
                s_q[r * QPITCH + lane + 32 * k] = *reinterpret_cast<const uint16_t *>(&h);
            }
            if (lane == 0) {
                s_qs[r] = a.scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
                s_end[r] = r >= rn ? 0 : a.causal ? max(0, len - n + i + 1) : len;
            }
        }

        float acc[NT][MT][4];
        float m[NT][2], m2[NT][2], l[NT][2];
#pragma unroll
        for (int x = 0; x < NT; ++x) {
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[x][k][i] = 0.0f;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[x][i] = m2[x][i] = -INFINITY;
                l[x][i] = 0.0f;
            }
        }

        // at most 1,024 tokens at a time, whose pages fit the arrays in shared memory
        for (int c0 = tok0; c0 < tok1; c0 += 1024) {
            const int c1 = min(tok1, c0 + 1024);
            if (c0 > tok0) __syncthreads();
            for (int p = tid; p <= ((c1 - 1) >> log2) - (c0 >> log2); p += kThreads) {
                int page = a.tab.table[(int64_t)b * a.tab.ldt + (c0 >> log2) + p];
                float ks = 0.0f, lv = -INFINITY;
                if (page < 0 || page >= a.pool.pages) {
                    record_status(a.status, kStatusBadPage);
                    page = -1;
                } else {
                    const int64_t tile = (int64_t)page * H + head;
                    ks = a.pool.scales[tile];
                    lv = log2f(a.pool.scales[a.pool.plane_scales + tile]);
                }
                s_page[p] = page;
                s_ks[p] = ks;
                s_lv[p] = lv;
            }
            __syncthreads();

            uint4 kc[TILES][2][KB];
            uint32_t vc[TILES][4][VW];
            const auto load_k = [&](int s0) {
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    const int tk = s0 + u * 16, page = tk < c1 ? s_page[(tk - c0) >> log2] : -1;
                    const uint8_t *base = a.pool.codes + ((((int64_t)page * H + head) << log2) + (tk & (a.pool.page - 1)) + g) * D + t * 16;
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < KB; ++k)
                            kc[u][h][k] = page >= 0 ? load_codes(base + h * 8 * D + k * 64) : make_uint4(0, 0, 0, 0);
                }
            };
            const auto load_v = [&](int s0) {
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    const int tk = s0 + u * 16, page = tk < c1 ? s_page[(tk - c0) >> log2] : -1;
                    const uint8_t *base = a.pool.codes + a.pool.plane_codes +
                                          ((((int64_t)page * H + head) << log2) + (tk & (a.pool.page - 1)) + 2 * t) * D + g * (D >= 128 ? 16 : 8);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        const int row = (c & 1) + 8 * (c >> 1);
                        // what lies past the sequence's end may be anything, NaN codes included: read as zeros
                        const bool in = page >= 0 && tk + 2 * t + row < len;
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

            int s0 = c0 + warp * STEP;
            if (s0 < c1) {
                load_k(s0);
                load_v(s0);
            }
            for (; s0 < c1; s0 += kWarps * STEP) {
                const int next = s0 + kWarps * STEP;
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
                            qf[x] = *reinterpret_cast<const uint2 *>(&s_q[(x * 8 + g) * QPITCH + k * 64 + t * 16 + w * 4]);
#pragma unroll
                        for (int u = 0; u < TILES; ++u) {
                            uint32_t f[4];
                            const uint4 &ka = kc[u][0][k], &kb = kc[u][1][k];
                            widen4<KIND>(w == 0 ? ka.x : w == 1 ? ka.y : w == 2 ? ka.z : ka.w, f[0], f[2]);
                            widen4<KIND>(w == 0 ? kb.x : w == 1 ? kb.y : w == 2 ? kb.z : kb.w, f[1], f[3]);
#pragma unroll
                            for (int x = 0; x < NT; ++x) mma_f16(s[x][u], f, qf[x].x, qf[x].y);
                        }
                    }
                }
                if (next < c1) load_k(next);

                // softmax: this lane has rows 2 t, 2 t + 1 and tokens g, g + 8 of each tile
                uint32_t pf[NT][TILES][2];
                float lv[TILES], ks[TILES];
#pragma unroll
                for (int u = 0; u < TILES; ++u) {
                    const int p = min(s0 + u * 16, c1 - 1) - c0;
                    lv[u] = s_lv[p >> log2];
                    ks[u] = s_ks[p >> log2];
                }
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    float top[2] = {-INFINITY, -INFINITY}, top2[2] = {-INFINITY, -INFINITY};
#pragma unroll
                    for (int u = 0; u < TILES; ++u)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = x * 8 + 2 * t + (i & 1), tk = s0 + u * 16 + g + 8 * (i >> 1);
                            float v = s[x][u][i] * (s_qs[row] * ks[u]);
                            if (tk >= min(s_end[row], c1)) v = -INFINITY;
                            s[x][u][i] = v;
                            top[i & 1] = fmaxf(top[i & 1], v);
                            top2[i & 1] = fmaxf(top2[i & 1], v + lv[u]);
                        }
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            top[i] = fmaxf(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], o));
                            top2[i] = fmaxf(top2[i], __shfl_xor_sync(0xFFFFFFFFu, top2[i], o));
                        }
                    float cl[2], co[2], base[2], lift[2][TILES];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mn = fmaxf(m[x][i], top[i]), mn2 = fmaxf(m2[x][i], top2[i]);
                        cl[i] = ex2_diff(m[x][i], mn);
                        co[i] = ex2_diff(m2[x][i], mn2);
                        m[x][i] = mn;
                        m2[x][i] = mn2;
                        base[i] = mn == -INFINITY ? 0.0f : mn;
                        l[x][i] *= cl[i];
#pragma unroll
                        for (int u = 0; u < TILES; ++u)
                            lift[i][u] = (mn2 == -INFINITY || lv[u] == -INFINITY) ? 0.0f : ex2(fminf(base[i] - mn2 + lv[u], 126.0f));
                    }
                    if (__any_sync(0xFFFFFFFFu, co[0] != 1.0f || co[1] != 1.0f)) {
#pragma unroll
                        for (int k = 0; k < MT; ++k)
#pragma unroll
                            for (int i = 0; i < 4; ++i) acc[x][k][i] *= co[i & 1];
                    }
#pragma unroll
                    for (int u = 0; u < TILES; ++u) {
                        float p[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p[i] = ex2(s[x][u][i] - base[i & 1]);
                            l[x][i & 1] += p[i];
                        }
                        pf[x][u][0] = transpose8x8(pack_half(p[0] * lift[0][u], p[1] * lift[1][u]));
                        pf[x][u][1] = transpose8x8(pack_half(p[2] * lift[0][u], p[3] * lift[1][u]));
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
                            mma_f16(acc[x][2 * w], fa, pf[x][u][0], pf[x][u][1]);
                            mma_f16(acc[x][2 * w + 1], fb, pf[x][u][0], pf[x][u][1]);
                        }
                    }
                if (next < c1) load_v(next);
            }
        }

        // the warps' results meet in shared memory
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
                    s_m2[warp * ROWS + row] = m2[x][i];
                }
            }
#pragma unroll
            for (int k = 0; k < MT; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    // tile k: word k / 2 of the lane's run of values, its bytes 2 (k & 1) and 2 (k & 1) + 1
                    const int byte = 4 * (k / 2) + 2 * (k & 1) + (i >> 1);
                    const int d = D == 64 ? g * 8 + byte : (byte / 16) * 128 + g * 16 + byte % 16;
                    s_o[(warp * ROWS + x * 8 + 2 * t + (i & 1)) * D + d] = acc[x][k][i];
                }
        }
        __syncthreads();
        for (int r = warp; r < rn; r += kWarps) {
            float mm = -INFINITY, ll = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * ROWS + r]);
            float f[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ll += s_l[w * ROWS + r] * ex2_diff(s_m[w * ROWS + r], mm);
                f[w] = mm == -INFINITY ? 0.0f : ex2_diff(s_m2[w * ROWS + r], mm);
            }
            const float inv = ll > 0.0f ? __fdiv_rn(1.0f, ll) : 0.0f;
            const float lse = ll > 0.0f ? mm + log2f(ll) : -INFINITY;
            const int i = (r0 + r) / a.group, hq = head * a.group + (r0 + r) - i * a.group;
            const int64_t slot = ((int64_t)b * H + head) * a.row_cap + r0 + r;
            if (splits > 1) {
                if (lane == 0) a.part_lse[slot * a.split_cap + split] = lse;
            } else if (a.lse && lane == 0) {
                a.lse[(int64_t)(row0 + i) * a.q_heads + hq] = lse == -INFINITY ? -INFINITY : lse * (1.0f / kLog2e);
            }
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                const int d = k * 64 + lane * 2;
                float o0 = 0.0f, o1 = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float2 v = *reinterpret_cast<const float2 *>(&s_o[(w * ROWS + r) * D + d]);
                    o0 += v.x * f[w];
                    o1 += v.y * f[w];
                }
                o0 *= inv;
                o1 *= inv;
                if (splits > 1) {
                    *reinterpret_cast<float2 *>(a.part + (slot * a.split_cap + split) * D + d) = make_float2(o0, o1);
                } else {
                    const __nv_bfloat162 h = __floats2bfloat162_rn(o0, o1);
                    *reinterpret_cast<__nv_bfloat162 *>(a.out + (int64_t)(row0 + i) * a.ldo + (int64_t)hq * a.ldo_head + d) = h;
                }
            }
        }
    }
    pdl_launch_dependents();
}

// Joins the splits of each row: a warp a row, the splits in order.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(const AttnArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    const int64_t slots = (int64_t)a.tab.seqs * a.pool.heads * a.row_cap;
    for (int64_t slot = (int64_t)blockIdx.x * kWarps + warp; slot < slots; slot += (int64_t)gridDim.x * kWarps) {
        const int64_t bh = slot / a.row_cap;
        const int r = (int)(slot - bh * a.row_cap), b = (int)(bh / a.pool.heads), head = (int)(bh - (int64_t)b * a.pool.heads);
        int row0, n;
        query_rows(a, b, row0, n);
        const int rows = n * a.group;
        if (r >= rows || rows > kFewRows) continue;
        const int splits = split_count(kv_length(a.tab, b, a.pool.page_log2, a.status));
        if (splits <= 1) continue;
        const float *pl = a.part_lse + slot * a.split_cap, *po = a.part + slot * a.split_cap * D;
        float w0 = lane < splits ? pl[lane] : -INFINITY, w1 = lane + 32 < splits ? pl[lane + 32] : -INFINITY;
        float mm = fmaxf(w0, w1);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, o));
        w0 = ex2_diff(w0, mm);
        w1 = ex2_diff(w1, mm);
        float sum = w0 + w1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
        float o[D / 32];
#pragma unroll
        for (int k = 0; k < D / 32; ++k) o[k] = 0.0f;
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            const float w = __shfl_sync(0xFFFFFFFFu, s < 32 ? w0 : w1, s & 31);
            const float2 *p = reinterpret_cast<const float2 *>(po + (int64_t)s * D);
#pragma unroll
            for (int k = 0; k < D / 64; ++k) {
                const float2 v = p[lane + 32 * k];
                o[2 * k] += w * v.x;
                o[2 * k + 1] += w * v.y;
            }
        }
        const int i = r / a.group, hq = head * a.group + r - i * a.group;
        uint16_t *dst = a.out + (int64_t)(row0 + i) * a.ldo + (int64_t)hq * a.ldo_head;
#pragma unroll
        for (int k = 0; k < D / 64; ++k)
            *reinterpret_cast<__nv_bfloat162 *>(dst + 64 * k + 2 * lane) =
                __floats2bfloat162_rn(o[2 * k] * inv, o[2 * k + 1] * inv);
        if (a.lse && lane == 0)
            a.lse[(int64_t)(row0 + i) * a.q_heads + hq] = sum > 0.0f ? (mm + log2f(sum)) * (1.0f / kLog2e) : -INFINITY;
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
    const int64_t most = (int64_t)sms * 4;
    return launch_kernel(kv_split_kernel<KIND, D, NT>, dim3((unsigned)(items < most ? items : most)), dim3(kThreads), smem,
                         st, 1, true, a);
}

template <int D>
cudaError_t launch_attention(const AttnArgs &a, int kind, int row_max, int64_t items, int64_t slots, bool join, int sms,
                             cudaStream_t st) {
    cudaError_t e;
    if (row_max <= 8)
        e = kind == kKvInt8 ? launch_split<kKvInt8, D, 1>(a, items, sms, st) : launch_split<kKvE4m3, D, 1>(a, items, sms, st);
    else
        e = kind == kKvInt8 ? launch_split<kKvInt8, D, 2>(a, items, sms, st) : launch_split<kKvE4m3, D, 2>(a, items, sms, st);
    if (e != cudaSuccess || !join) return e;
    const int64_t blocks = (slots + kWarps - 1) / kWarps, most = (int64_t)sms * 16;
    return launch_kernel(kv_join_kernel<D>, dim3((unsigned)(blocks < most ? blocks : most)), dim3(kThreads), 0, st, 1, true, a);
}

// Rows of a key/value head that may be split, for the workspace: exact when
// every sequence has the same number of queries.
int row_capacity(int64_t rows, int64_t seqs, bool ragged, int group) {
    const int64_t r = ragged ? kFewRows : seqs > 0 ? rows / seqs * group : 0;
    return (int)(r <= kFewRows ? r : 0);
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
    const int cap = row_capacity(rows, seqs, ragged != 0, q_heads / heads);
    // a shorter sequence may have more splits than the longest: the cut grows in steps
    int splits = 0;
    for (int64_t len : {max_len, (int64_t)2048, (int64_t)8192, (int64_t)32768})
        if (len <= max_len) {
            const int s = split_count((int)len);
            if (s > splits) splits = s;
        }
    *bytes = splits <= 1 ? 0 : (int64_t)seqs * heads * cap * splits * (dim + 1) * 4;
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
    if (!(scale == scale) || scale > 3.0e38f || scale < -3.0e38f) return kv_fail("scale must be finite");
    if (ldq < 0 || ldq_head < 0 || ldq % 8 || ldq_head % 8) return kv_fail("query pitches must be multiples of 8");
    if (ldo < dim || ldo_head < dim || ldo % 8 || ldo_head % 8) return kv_fail("output pitches must be multiples of 8 that hold a head");
    if (!q || !codes || !scales || !table || !lens || !out) return kv_fail("null pointer");
    if (kv_misaligned(q, 16) || kv_misaligned(out, 16) || kv_misaligned(workspace, 16) || kv_misaligned(lse, 4) ||
        kv_misaligned(row_start, 4))
        return kv_fail("q, out and workspace must be 16-byte, lse and row_start 4-byte aligned");
    int64_t need = 0;
    const int64_t top = width * page < 0x7FFFFFFF ? width * page : 0x7FFFFFFF;
    if ((rc = clef_kv_attention_workspace(rows, row_start != nullptr, seqs, q_heads, heads, dim, top, &need))) return rc;
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
    a.row_cap = row_capacity(rows, seqs, row_start != nullptr, a.group);
    const int64_t slots = seqs * heads * a.row_cap;
    if (need > 0) {
        a.split_cap = (int)(need / (slots * (dim + 1) * 4));
        a.part = static_cast<float *>(workspace);
        a.part_lse = a.part + slots * a.split_cap * dim;
    }
    // rows of a key/value head, as far as the host knows
    const int64_t row_max = row_start ? kFewRows : (int64_t)a.per_seq * a.group;
    const int64_t items = row_start ? (int64_t)1 << 30 : seqs * heads * ((row_max + 7) / 8) * (need > 0 ? a.split_cap : 1);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rm = (int)(row_max < 64 ? row_max : 64);
    const cudaError_t e = dim == 64    ? launch_attention<64>(a, kind, rm, items, slots, need > 0, sms, st)
                          : dim == 128 ? launch_attention<128>(a, kind, rm, items, slots, need > 0, sms, st)
                                       : launch_attention<256>(a, kind, rm, items, slots, need > 0, sms, st);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "cache attention launch");
}
