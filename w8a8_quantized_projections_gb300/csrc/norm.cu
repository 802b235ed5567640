// norm.cu -- what comes before a linear: the root-mean-square norm with the
// residual's addition, its result as bf16 or as the 8-bit codes and scales of
// the linear that follows, and the quantizer of blocks of 128.
//
//   h = x + r (fp32);  r_out = bf16(h);  g = 1 / sqrt(mean(h^2) + eps)
//   y = h w g;  bf16(y), and codes of y (or of its rotation) by their absmax
//
// Bound by HBM: 2 bytes an element in for x, 2 in and 2 out for the residual, 1
// out for a code (2 for a bf16 result), so the row is read once and stays in
// registers (or, many rows at a time, in shared memory until it is coded).  24,032 x
// 5,120 with a residual: codes in blocks 143 us (89% of the copy rate), e4m3 with a scale a row 141 (90%), rotated INT8
// 128 us (99%), rotated e4m3 129, bf16 150 us (97%); a row of 5,120: 2 us, its launch.  g is a factor of the whole row, and the rotation is linear: the
// absmax of v = h w (rotated) is found beside the sum of squares, in one
// reduction over the row; the codes are rne(v * top / absmax(v)), in which g
// cancels, and the scale is absmax(v) g / top.  Scales of blocks of 128 need no
// more than the eight lanes that hold a block.
//
// Sums and values are fp32, rounded once: the sum to bf16 for the residual
// stream, the result to bf16 or to its code.  The norm takes the sum as it was
// before its rounding.  Squares that pass fp32 (|h| of 2^60 and more) are found
// out by the sum, which is then infinite; the row is read again and summed in
// units of 2^80.
#include <algorithm>
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "clef_pair.cuh"
#include "clef_ptx.cuh"
#include "kv_host.h"

namespace clef {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kE = 16;             // consecutive elements of a piece: two 16-byte loads, one 16-byte store of codes
constexpr int kLanes = 128 / kE;   // lanes that hold a block of 128 at a piece a lane
constexpr float kFltMax = 3.4028234663852886e38f;

enum NormMode : int { kNormBf16 = -1, kNormI8H = kActInt8H128, kNormF8 = kActFp8, kNormF8H = kActFp8H128, kNormF8B = 3 };

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// Pairs of fp32 values in one register pair: one instruction rounds both as the scalar one would.
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unf2(uint64_t p, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ void load16(const uint16_t *p, uint32_t (&w)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p), b = *(reinterpret_cast<const uint4 *>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// Sixteen bf16 values; whole: p is 32-byte aligned (half a sector written at a time costs twice the passes).
__device__ __forceinline__ void store16(uint16_t *p, const uint32_t (&w)[8], bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]) : "memory");
        return;
    }
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    *(reinterpret_cast<uint4 *>(p) + 1) = make_uint4(w[4], w[5], w[6], w[7]);
}

__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// Sixteen codes of v * r; all bits zero where r is (a negative zero has a sign in e4m3).
template <bool kInt8>
__device__ __forceinline__ uint4 codes16(const uint64_t *v, float r) {
    if (!kInt8 && r == 0.0f) return make_uint4(0u, 0u, 0u, 0u);
    const uint64_t rr = f2(r, r);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float u[4];
        unf2(mul2(v[2 * i], rr), u[0], u[1]);
        unf2(mul2(v[2 * i + 1], rr), u[2], u[3]);
        if (kInt8) {
            uint32_t h;
            asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(h) : "r"(__float2int_rn(u[3])), "r"(__float2int_rn(u[2])), "r"(0));
            asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w[i]) : "r"(__float2int_rn(u[1])), "r"(__float2int_rn(u[0])), "r"(h));
        } else {
            w[i] = e4m3x2(u[0], u[1]) | (e4m3x2(u[2], u[3]) << 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Codes of two neighbouring pieces; whole: in one store (the address is a multiple of 32, and both are there).
__device__ __forceinline__ void leave32(uint8_t *q, const uint4 &x, const uint4 &y, bool whole, bool second) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                     :: "l"(q), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w) : "memory");
    } else {
        *reinterpret_cast<uint4 *>(q) = x;
        if (second) *reinterpret_cast<uint4 *>(q + kE) = y;
    }
}

// The multiplier of codes whose largest value is top: 0 for zeros, and finite for the smallest values.
__device__ __forceinline__ float code_factor(float amax, float top) {
    return amax == 0.0f ? 0.0f : fminf(__fdiv_rn(top, amax), kFltMax);
}

__device__ __forceinline__ float absmax16(const uint64_t *v, float amax) {
#pragma unroll
    for (int k = 0; k < kE / 2; ++k) {
        float a, b;
        unf2(v[k], a, b);
        amax = fmaxf(amax, fmaxf(fabsf(a), fabsf(b)));
    }
    return amax;
}

// The orthonormal Walsh-Hadamard transform of a block of 128 held by neighbouring lanes, C pieces of sixteen each:
// strides below 16 C in the thread, the others between lanes, the order of clef_quant_act.
template <int C>
__device__ __forceinline__ void rotate(uint64_t (&v)[8 * C], int lane) {
#pragma unroll
    for (int k = 0; k < 8 * C; ++k) {
        float a, b;
        unf2(v[k], a, b);
        v[k] = f2(a + b, a - b);
    }
#pragma unroll
    for (int h = 1; h < 8 * C; h <<= 1)
#pragma unroll
        for (int k = 0; k < 8 * C; ++k)
            if ((k & h) == 0) {
                const uint64_t a = v[k], b = v[k + h];
                v[k] = add2(a, b);
                v[k + h] = sub2(a, b);
            }
#pragma unroll
    for (int s = 1; s < kLanes / C; s <<= 1) {
        const float sign = (lane & s) ? -1.0f : 1.0f;      // (a product with it is exact)
        const uint64_t ss = f2(sign, sign);
#pragma unroll
        for (int k = 0; k < 8 * C; ++k) {
            float a, b;
            unf2(v[k], a, b);
            v[k] = fma2(ss, v[k], f2(__shfl_xor_sync(kAll, a, s), __shfl_xor_sync(kAll, b, s)));
        }
    }
    const float c = __uint_as_float(0x3DB504F3u);          // fp32(1 / sqrt(128))
#pragma unroll
    for (int k = 0; k < 8 * C; ++k) v[k] = mul2(v[k], f2(c, c));
}

struct NormArgs {
    const uint16_t *x, *r, *w;
    uint16_t *r_out, *y;
    uint8_t *q;
    float *scale;
    int64_t ldx, ldr, ldro, ldy, M;
    int K, blocks;
    float eps;
    bool y32, r32, q32;       // rows of y, r_out and q start on 32 bytes
};

// Sixteen values h of x and the residual (has_r: whether there is one), their sum as bf16, the squares of h in units
// of 1 / unit summed, and v = h w in those units.
__device__ __forceinline__ void take16(const uint32_t (&x)[8], const uint32_t (&r)[8], const uint32_t (&w)[8], bool has_r,
                                       float unit, uint64_t *v, uint32_t (&sum)[8], float &total) {
    const uint64_t uu = f2(unit, unit);
    uint64_t ss = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint64_t h = f2(lo(x[i]), hi(x[i]));
        if (has_r) {
            h = add2(h, f2(lo(r[i]), hi(r[i])));
            float a, b;
            unf2(h, a, b);
            sum[i] = pack2(a, b);
        }
        h = mul2(h, uu);
        ss = fma2(h, h, ss);
        v[i] = mul2(h, f2(lo(w[i]), hi(w[i])));
    }
    float even, odd;
    unf2(ss, even, odd);
    total = even + odd;
}

// Sum and maximum over a row held by `lanes` lanes (a power of two).  Pieces are added as a balanced tree over their
// places in the row, neighbours first, so that the sum is the same however many a thread holds.
template <bool kMax>
__device__ __forceinline__ void lanes_sum(float &ss, float &amax, int lanes) {
#pragma unroll
    for (int s = 1; s < 32; s <<= 1)
        if (s < lanes) {
            ss += __shfl_xor_sync(kAll, ss, s);
            if (kMax) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
        }
}

// The same over a CTA's warps; one barrier.
template <bool kMax>
__device__ __forceinline__ void cta_sum(float &ss, float &amax, float2 *part) {
    const int lane = threadIdx.x & 31;
    lanes_sum<kMax>(ss, amax, 32);
    if (lane == 0) part[threadIdx.x >> 5] = make_float2(ss, amax);
    __syncthreads();
    const float2 o = lane < (int)(blockDim.x >> 5) ? part[lane] : make_float2(0.0f, 0.0f);
    ss = o.x;
    amax = o.y;
    lanes_sum<kMax>(ss, amax, blockDim.x <= 128 ? 4 : blockDim.x <= 256 ? 8 : 32);
    if (blockDim.x <= 256) {      // (from the lanes that hold partial sums to all)
        ss = __shfl_sync(kAll, ss, 0);
        if (kMax) amax = __shfl_sync(kAll, amax, 0);
    }
}

__device__ __forceinline__ float root(float ss, int K, float eps, float unit) {
    return __frsqrt_rn(__fdiv_rn(ss, (float)K) + eps * (unit * unit));
}

__device__ __forceinline__ void leave_y(const NormArgs &a, int64_t m, int e, const uint64_t *v, float g) {
    uint32_t p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float b, c;
        unf2(mul2(v[i], f2(g, g)), b, c);
        p[i] = pack2(b, c);
    }
    store16(a.y + m * a.ldy + e, p, a.y32);
}

// Codes and scales of C pieces from e on; amax: of the row, where it has one scale.
template <int MODE, int C>
__device__ __forceinline__ void leave_codes(const NormArgs &a, int64_t m, int e, bool row, const uint64_t (&v)[8 * C], float g, float amax) {
    constexpr float kTop = MODE == kNormI8H ? 127.0f : 448.0f;
    if (MODE == kNormF8B) {
        amax = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) amax = absmax16(v + 8 * c, amax);
#pragma unroll
        for (int s = 1; s < kLanes / C; s <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
    }
    const float r = code_factor(amax, kTop);
#pragma unroll
    for (int c = 0; c < C; c += 2) {
        uint8_t *q = a.q + m * a.K + e + c * kE;
        if (!row || e + c * kE >= a.K) continue;
        const uint4 x = codes16<MODE == kNormI8H>(v + 8 * c, r);
        if (C == 1) {
            *reinterpret_cast<uint4 *>(q) = x;
        } else {
            const uint4 y = codes16<MODE == kNormI8H>(v + 8 * (c + 1 < C ? c + 1 : c), r);
            leave32(q, x, y, a.q32, e + (c + 1) * kE < a.K);     // (K is a multiple of 32 where q32 says so)
        }
    }
    if (row && e < a.K && (MODE == kNormF8B ? e % 128 == 0 : e == 0))
        a.scale[MODE == kNormF8B ? m * a.blocks + e / 128 : m] = __fdiv_rn(amax * g, kTop);
}

// G lanes a row (K up to 16 G), four rows or more a CTA; G = 0: a CTA a row, C neighbouring pieces a thread.
template <int MODE, int C, int G>
__global__ void __launch_bounds__(G ? 128 : 512) norm_kernel(const NormArgs a) {
    constexpr bool kRotate = MODE == kNormI8H || MODE == kNormF8H;
    constexpr bool kRowMax = MODE != kNormBf16 && MODE != kNormF8B;
    __shared__ float2 part[2][16];

    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t m = G ? blockIdx.x * (int64_t)(128 / (G ? G : 1)) + tid / (G ? G : 1) : (int64_t)blockIdx.x;
    const bool row = !G || m < a.M;
    const int e = (G ? tid % (G ? G : 1) : tid) * C * kE;
    pdl_wait();

    const uint16_t *x = a.x + m * a.ldx;
    const uint16_t *r = a.r + m * a.ldr;
    uint64_t v[8 * C], u[kRotate ? 8 * C : 1];
    uint32_t sum[C][8];
    float g = 0.0f, amax = 0.0f, unit = 1.0f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        float piece[C];
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int at = e + c * kE;
            piece[c] = 0.0f;
            if (row && at < a.K) {
                uint32_t xp[8], rp[8], wp[8];
                load16(x + at, xp);
                if (a.r) load16(r + at, rp);
                load16(a.w + at, wp);
                take16(xp, rp, wp, a.r != nullptr, unit, v + 8 * c, sum[c], piece[c]);
            } else {
#pragma unroll
                for (int k = 0; k < 8; ++k) v[8 * c + k] = 0;
            }
        }
        if constexpr (kRotate) {
            // (blocks lie in whole rows: their lanes are in or out together)
#pragma unroll
            for (int k = 0; k < 8 * C; ++k) u[k] = v[k];
            rotate<C>(u, lane);
        }
        amax = 0.0f;
        if (kRowMax)
#pragma unroll
            for (int c = 0; c < C; ++c) amax = absmax16((kRotate ? u : v) + 8 * c, amax);
        float ss = piece[0];
        if (C == 2) ss += piece[C - 1];
        if (C == 4) ss = (ss + piece[1 % C]) + (piece[2 % C] + piece[3 % C]);
        if (G) lanes_sum<kRowMax>(ss, amax, G);
        else cta_sum<kRowMax>(ss, amax, part[pass]);
        g = root(ss, a.K, a.eps, unit);
        // squares past fp32: once more, in other units (a warp's other rows find the same again)
        const bool over = !(ss <= kFltMax);
        if (over) unit = 0x1p-80f;
        if (G ? !__any_sync(kAll, over) : !over) break;
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
        if (row && e + c * kE < a.K) {
            if (a.r) store16(a.r_out + m * a.ldro + e + c * kE, sum[c], a.r32);
            if (MODE == kNormBf16 || a.y) leave_y(a, m, e + c * kE, v + 8 * c, g);
        }
    if constexpr (kRotate) leave_codes<MODE, C>(a, m, e, row, u, g, amax);
    else if constexpr (MODE != kNormBf16) leave_codes<MODE, C>(a, m, e, row, v, g, amax);
    pdl_launch_dependents();
}

// Many rows: CTAs that stay, each with a ring of rows of x and the residual in shared memory, filled by copies several
// rows ahead, so that HBM is read while earlier rows are reduced and written.  A row is lines of 128 bytes with
// the 128-byte swizzle: unit u of 16 bytes of line l lies at unit u ^ (l & 7).  (Rows of other lengths are copied as
// they are; their reads meet in the banks.)  A thread owns half a line (C = 2), or a line (C = 4); the operations
// and their order are norm_kernel's.
constexpr int kMaxRing = 8;

__device__ __forceinline__ void tma_lines(void *dst, const CUtensorMap *m, int line, int64_t row, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
                 ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(0), "r"(line), "r"((int32_t)row), "r"(smem_u32(bar))
                 : "memory");
}

// A row of up to 256 lines in one copy, of more (a multiple of sixteen) in two.
__device__ __forceinline__ void tma_row(uint8_t *dst, const CUtensorMap *m, int lines, int64_t row, uint64_t *bar) {
    tma_lines(dst, m, 0, row, bar);
    if (lines > 256) tma_lines(dst + lines / 2 * 128, m, lines / 2, row, bar);
}

__device__ __forceinline__ void bulk_row(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)) : "memory");
}

template <int MODE, int C>
__global__ void __launch_bounds__(512) norm_staged_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmr,
                                                          const __grid_constant__ CUtensorMap tmw, const NormArgs a, bool lines, int ring, uint32_t slot_bytes, unsigned int *status,
                                                          uint64_t limit_ns, int force_timeout) {
    constexpr bool kRotate = MODE == kNormI8H || MODE == kNormF8H;
    constexpr bool kRowMax = MODE != kNormBf16 && MODE != kNormF8B;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[kMaxRing], w_full;
    __shared__ float2 part[2][16];
    __shared__ int abort_flag;

    const uint32_t base = smem_u32(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31;
    const uint32_t row_bytes = (uint32_t)a.K * 2u, r_at = (row_bytes + 1023u) & ~1023u;
    uint8_t *weights = smem_raw + (((base + 1023u) & ~1023u) - base), *rows = weights + r_at;
    const int e = tid * C * kE;
    if (tid == 0) {
        for (int s = 0; s < ring; ++s) mbar_init(&full[s], 1);
        mbar_init(&w_full, 1);
        abort_flag = 0;
        fence_barrier_init();
        if (lines) {      // (the maps that are made)
            tma_prefetch_desc(&tmx);
            tma_prefetch_desc(&tmw);
            if (a.r) tma_prefetch_desc(&tmr);
        }
    }
    __syncthreads();
    pdl_wait();
    const WaitCtx w{limit_ns, &abort_flag, status};

    const auto fill = [&](int slot, int64_t m) {
        uint8_t *dst = rows + (uint32_t)slot * slot_bytes;
        mbar_arrive_expect_tx(&full[slot], a.r ? 2u * row_bytes : row_bytes);
        if (lines) {
            tma_row(dst, &tmx, a.K / 64, m, &full[slot]);
            if (a.r) tma_row(dst + r_at, &tmr, a.K / 64, m, &full[slot]);
        } else {
            bulk_row(dst, a.x + m * a.ldx, row_bytes, &full[slot]);
            if (a.r) bulk_row(dst + r_at, a.r + m * a.ldr, row_bytes, &full[slot]);
        }
    };
    const int64_t first = blockIdx.x, step = gridDim.x;
    if (tid == 0) {
        mbar_arrive_expect_tx(&w_full, row_bytes);
        if (lines) tma_row(weights, &tmw, a.K / 64, 0, &w_full);
        else bulk_row(weights, a.w, row_bytes, &w_full);
    }
    if (tid == 0)
        for (int s = 0; s < ring && first + s * step < a.M; ++s) fill(s, first + s * step);
    const uint32_t line = (uint32_t)tid / (4 / C), unit = (uint32_t)tid % (4 / C) * 4u;
    uint32_t off[2 * C];
#pragma unroll
    for (int j = 0; j < 2 * C; ++j) off[j] = line * 128u + (((unit + j) ^ (lines ? line & 7u : 0u)) << 4);
    const auto piece = [&](const uint8_t *p, int c, uint32_t(&o)[8]) {
        const uint4 x = *reinterpret_cast<const uint4 *>(p + off[2 * c]), y = *reinterpret_cast<const uint4 *>(p + off[2 * c + 1]);
        o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
        o[4] = y.x; o[5] = y.y; o[6] = y.z; o[7] = y.w;
    };

    int slot = 0;
    uint32_t phase = 0, which = 0;
    int64_t m = first;
    mbar_wait(&w_full, 0, w, kSiteQuantFull);
    // test knob: a wait for what nothing signals
    if (force_timeout == 1 || force_timeout - 2 == (int)blockIdx.x) mbar_wait(&w_full, 1, w, kSiteQuantFull);
    for (; m < a.M; m += step) {
        mbar_wait(&full[slot], phase, w, kSiteQuantFull);
        const uint8_t *at = rows + (uint32_t)slot * slot_bytes;
        uint64_t v[8 * C];
        float g = 0.0f, amax = 0.0f, unit = 1.0f;
        const auto take = [&](bool leave) {
            float total[C];
#pragma unroll
            for (int c = 0; c < C; ++c) {
                total[c] = 0.0f;
                if (e + c * kE < a.K) {
                    uint32_t xp[8], rp[8], wp[8], sum[8];
                    piece(at, c, xp);
                    if (a.r) piece(at + r_at, c, rp);
                    piece(weights, c, wp);
                    take16(xp, rp, wp, a.r != nullptr, unit, v + 8 * c, sum, total[c]);
                    if (a.r && leave) store16(a.r_out + m * a.ldro + e + c * kE, sum, a.r32);
                } else {
#pragma unroll
                    for (int k = 0; k < 8; ++k) v[8 * c + k] = 0;
                }
            }
            float ss = total[0] + total[1];
            if (C == 4) ss += total[2 % C] + total[3 % C];
            return ss;
        };
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            float ss = take(pass == 0);
            if (kRotate) rotate<C>(v, lane);
            amax = 0.0f;
            if (kRowMax)
#pragma unroll
                for (int c = 0; c < C; ++c) amax = absmax16(v + 8 * c, amax);
            cta_sum<kRowMax>(ss, amax, part[which]);
            which ^= 1u;
            g = root(ss, a.K, a.eps, unit);
            if (ss <= kFltMax) break;
            unit = 0x1p-80f;
        }
        if (__any_sync(kAll, abort_flag)) break;     // (another warp may be setting it: a warp's lanes leave together)
        if constexpr (MODE != kNormBf16) leave_codes<MODE, C>(a, m, e, true, v, g, amax);
        if (MODE == kNormBf16 || a.y) {
            if constexpr (kRotate) take(false);      // the values before their rotation once more: the row is still there
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (e + c * kE < a.K) leave_y(a, m, e + c * kE, v + 8 * c, g);
        }
        if (kRotate && a.y) __syncthreads();
        // past the last barrier every thread has read the row
        if (tid == 0 && m + ring * step < a.M) {
            fence_proxy_async_smem();
            fill(slot, m + ring * step);
        }
        if (++slot == ring) {
            slot = 0;
            phase ^= 1u;
        }
    }
    pdl_launch_dependents();
    if (abort_flag && tid == 0) {
        // copies already issued land before the CTA ends: the weights, this row's slot and those after it
        mbar_wait_drain(&w_full, 0, 200000000ull, status);
        for (int k = 0; k < ring && m + k * step < a.M; ++k) {
            const int s = slot + k < ring ? slot + k : slot + k - ring;
            mbar_wait_drain(&full[s], slot + k < ring ? phase : phase ^ 1u, 200000000ull, status);
        }
    }
}

// ------------------------------------------------------------ blocks of 128

// Codes of x in blocks of one row by 128: four lanes a block, two pieces each.  24,032 x 5,120: 61 us, 89% of the copy
// rate (eight lanes of a piece: 65 us); 1,502 x 17,408: 15 us.
__global__ void __launch_bounds__(256) quant_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, int K, int blocks,
                                                         int64_t total, bool q32, uint8_t *__restrict__ q,
                                                         float *__restrict__ scale) {
    pdl_wait();
    for (int64_t i0 = blockIdx.x * (int64_t)64; i0 < total; i0 += (int64_t)gridDim.x * 64) {
        const int64_t i = i0 + threadIdx.x / 4;      // block of the matrix
        const int64_t m = i / blocks;
        const int b = (int)(i - m * blocks), e = b * 128 + (int)(threadIdx.x % 4) * 2 * kE;
        uint64_t v[2][8] = {};
        float amax = 0.0f;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            if (i < total && e + c * kE < K) {
                uint32_t p[8];
                load16(x + m * ldx + e + c * kE, p);
#pragma unroll
                for (int k = 0; k < 8; ++k) v[c][k] = f2(lo(p[k]), hi(p[k]));
                amax = absmax16(v[c], amax);
            }
        }
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
        if (i < total && e < K) {
            const float r = code_factor(amax, 448.0f);
            leave32(q + m * K + e, codes16<false>(v[0], r), codes16<false>(v[1], r), q32, e + kE < K);
            if (e % 128 == 0) scale[i] = __fdiv_rn(amax, 448.0f);
        }
    }
    pdl_launch_dependents();
}

// Codes of w in blocks of 128 rows by 128: a CTA a block, two pieces of a row a thread, kept as bf16.  5,120 x 17,408: 44 us, 90% of the
// copy rate (256 threads of four pieces: 48.8 us where this took 45.7).
__global__ void __launch_bounds__(512, 3) quant_tiles_kernel(const uint16_t *__restrict__ w, int64_t ldw, int64_t M, int K,
                                                             int blocks, bool q32, uint8_t *__restrict__ q, float *__restrict__ scale) {
    __shared__ float part[16];
    const int64_t mb = blockIdx.x / blocks, m = mb * 128 + threadIdx.x / 4;
    const int b = (int)(blockIdx.x - mb * blocks), e = b * 128 + (int)(threadIdx.x % 4) * 2 * kE;
    pdl_wait();
    uint32_t p[2][8];
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (e + c * kE < K && m < M) {
            load16(w + m * ldw + e + c * kE, p[c]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) p[c][k] = 0u;
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(lo(p[c][k])), fabsf(hi(p[c][k]))));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
    amax = part[threadIdx.x & 15];
#pragma unroll
    for (int s = 8; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
    if (e < K && m < M) {
        const float r = code_factor(amax, 448.0f);
        uint4 o[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            uint64_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = f2(lo(p[c][k]), hi(p[c][k]));
            o[c] = codes16<false>(v, r);
        }
        leave32(q + m * K + e, o[0], o[1], q32, e + kE < K);
    }
    if (threadIdx.x == 0) scale[blockIdx.x] = __fdiv_rn(amax, 448.0f);
    pdl_launch_dependents();
}

// ------------------------------------------------------------ launches

struct NormEnv {
    int sms;
    unsigned int *status;
    uint64_t limit_ns;
    int force_timeout;
};

// The staged kernel's launch: CTAs an SM for 1,024 threads, with the rows that 220 KB hold.
template <int MODE, int C>
int launch_staged(const NormArgs &a, const NormEnv &env, int threads, cudaStream_t st) {
    static SmemOptIn opt;
    constexpr int kMost = 224 * 1024;
    auto kern = norm_staged_kernel<MODE, C>;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(kern), kMost);
    if (e != cudaSuccess) return internal_cuda_error(e, "norm smem attribute");
    // rows of whole lines, up to 256 of them, or twice a multiple of eight
    const bool lines = a.K % 64 == 0 && (a.K <= 256 * 64 || a.K % 1024 == 0);
    CUtensorMap tx = {}, tr = {}, tw = {};
    if (lines) {
        const uint64_t dims[3] = {64, (uint64_t)(a.K / 64), (uint64_t)a.M}, one[3] = {64, (uint64_t)(a.K / 64), 1};
        const uint32_t box[3] = {64, (uint32_t)(a.K / 64 > 256 ? a.K / 128 : a.K / 64), 1};
        const auto map = [&](CUtensorMap &m, const void *at, const uint64_t *d, int64_t ld) {
            const uint64_t strides[2] = {128, (uint64_t)ld * 2};
            return internal_make_tmap_nd(&m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, at, d, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
        };
        int rc = map(tx, a.x, dims, a.ldx);
        if (!rc) rc = map(tw, a.w, one, a.K);
        if (!rc && a.r) rc = map(tr, a.r, dims, a.ldr);
        if (rc) return rc;
    }
    // CTAs that registers and threads let an SM hold, for each number of warps
    static AskedOnce<17> known;
    int most = 0;
    e = known.get(threads / 32, &most, [&](int *n) { return cudaOccupancyMaxActiveBlocksPerMultiprocessor(n, kern, threads, 0); });
    if (e != cudaSuccess) return internal_cuda_error(e, "norm occupancy");
    const int row = (a.K * 2 + 1023) / 1024 * 1024, slot = row * (a.r ? 2 : 1);
    int per_sm = std::min(most, 16), ring = 0;
    for (;  per_sm > 1; --per_sm)
        if ((ring = (kMost / per_sm - 2048 - row) / slot) >= 2) break;
    ring = std::min((kMost / per_sm - 2048 - row) / slot, kMaxRing);
    const int64_t ctas = (int64_t)per_sm * env.sms;
    e = launch_kernel(kern, dim3((unsigned)(a.M < ctas ? a.M : ctas)), dim3((unsigned)threads), (size_t)(row + ring * slot + 1024), st, 1, true,
                      tx, tr, tw, a, lines, ring, (uint32_t)slot, env.status, env.limit_ns, env.force_timeout);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "norm launch");
}

template <int MODE>
int launch_norm(const NormArgs &a, const NormEnv &env, cudaStream_t st) {
    const int chunks = a.K / kE;
    cudaError_t e;
    const auto lanes = [&](auto kern, int g) {
        const int64_t rows = 128 / g;
        return launch_kernel(kern, dim3((unsigned)((a.M + rows - 1) / rows)), dim3(128), 0, st, 1, true, a);
    };
    const auto cta = [&](auto kern, int c) {
        const unsigned threads = (unsigned)((chunks + 32 * c - 1) / (32 * c) * 32);
        return launch_kernel(kern, dim3((unsigned)a.M), dim3(threads), 0, st, 1, true, a);
    };
    if (chunks <= 8) e = lanes(norm_kernel<MODE, 1, 8>, 8);
    else if (chunks <= 16) e = lanes(norm_kernel<MODE, 1, 16>, 16);
    else if (chunks <= 32) e = lanes(norm_kernel<MODE, 1, 32>, 32);
    // (a warp a row up to 1,024: 100,000 rows to fp8 114 us, 129 staged; rotated rows 150 and 110, rows of 2,048 worse)
    else if (chunks <= 64 && MODE != kNormI8H && MODE != kNormF8H) e = lanes(norm_kernel<MODE, 2, 32>, 32);
    else {
        // Rows enough that CTAs pay which keep some ahead.  (Beside a residual, bf16 results of rows up to 5,120 leave faster
        // where a CTA a row comes and goes: its 64 registers a thread let an SM hold 32 warps, three CTAs of the ten that
        // 5,120 takes, two of eleven.  24,032 rows of 2,048: 57 us, 66 staged; 4,608: 139 and 142; 5,120: 150 and 157; 5,136: 200 and
        // 152; 6,144: 208 and 191; 8,192: 258 and 253; 16,384: 633 and 507.)
        const bool many = a.M >= 8 * (int64_t)env.sms && !(MODE == kNormBf16 && a.r && a.K <= 5120 && a.M >= 32 * (int64_t)env.sms);
        if (many && chunks <= 1024) return launch_staged<MODE, 2>(a, env, (chunks + 63) / 64 * 32, st);
        if (many) return launch_staged<MODE, 4>(a, env, (chunks + 127) / 128 * 32, st);
        e = chunks <= 512 ? cta(norm_kernel<MODE, 1, 0>, 1) : chunks <= 1024 ? cta(norm_kernel<MODE, 2, 0>, 2) : cta(norm_kernel<MODE, 4, 0>, 4);
    }
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "norm launch");
}

constexpr int64_t kMaxNormK = 32768;

int norm_call(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *w, int64_t M, int64_t K,
              float eps, int mode, void *residual_out, int64_t ldro, void *y, int64_t ldy, void *q, float *scale,
              void *stream) {
    if (M < 0 || M > 0x7FFFFFFF) return kv_fail("M out of range");
    const bool rotated = mode == kNormI8H || mode == kNormF8H;
    if (K <= 0 || K > kMaxNormK || K % (rotated ? 128 : kE) != 0)
        return kv_fail("K must be in (0, 32768] and a multiple of 128 (rotated) or 16");
    if (!(eps >= 1e-20f) || eps > 1e20f) return kv_fail("eps must be in 1e-20 .. 1e20");
    if (ldx < K || ldx % 8 != 0) return kv_fail("ldx must be >= K and a multiple of 8");
    if (residual_out && !residual) return kv_fail("residual_out without a residual");
    if (residual && (ldr < K || ldr % 8 != 0 || ldro < K || ldro % 8 != 0))
        return kv_fail("the residuals' pitches must be >= K and multiples of 8");
    if (y && (ldy < K || ldy % 8 != 0)) return kv_fail("ldy must be >= K and a multiple of 8");
    if (M == 0) return CLEF_OK;
    if (!x || !w || (mode == kNormBf16 ? !y : (!q || !scale)) || (residual && !residual_out)) return kv_fail("null pointer");
    if (kv_misaligned(x, 16) || kv_misaligned(w, 16) || kv_misaligned(residual, 16) || kv_misaligned(residual_out, 16) ||
        kv_misaligned(y, 16) || kv_misaligned(q, 16))
        return kv_fail("tensors must be 16-byte aligned");
    if (kv_misaligned(scale, 4)) return kv_fail("scale not 4-byte aligned");
    // (with another pitch a row's result would land on rows not read yet)
    if (M > 1 && ((y == x && ldy != ldx) || (residual && residual_out == residual && ldro != ldr)))
        return kv_fail("in place, the pitches must agree");
    int sms = 0;
    unsigned int *status = nullptr;
    const int rc = internal_device(&sms, &status);
    if (rc) return rc;
    NormEnv env;
    env.sms = internal_launch_sms(sms);
    env.status = status;
    env.limit_ns = internal_wait_limit(&env.force_timeout);
    NormArgs a;
    a.x = static_cast<const uint16_t *>(x);
    a.r = static_cast<const uint16_t *>(residual);
    a.w = static_cast<const uint16_t *>(w);
    a.r_out = static_cast<uint16_t *>(residual_out);
    a.y = static_cast<uint16_t *>(y);
    a.q = static_cast<uint8_t *>(q);
    a.scale = scale;
    a.ldx = ldx;
    a.ldr = ldr;
    a.ldro = ldro;
    a.ldy = ldy;
    a.M = M;
    a.K = (int)K;
    a.blocks = (int)((K + 127) / 128);
    a.eps = eps;
    a.y32 = !kv_misaligned(y, 32) && ldy % 16 == 0;
    // (Residuals of rotated modes are written in halves of sectors up to 8,192, where an SM holds two of the CTAs that keep
    // rows ahead or more -- 16 warps of 104 registers a thread --, and in whole ones beyond, where it holds one.  24,032 rows, INT8,
    // halves and whole: 2,048 55 and 57 us, 4,096 106 and 116, 5,120 128 and 151, 8,192 203 and 216, 9,216 326 and 313,
    // 12,288 355 and 327, 16,384 433 and 410.  The other modes take whole ones: codes in blocks of 5,120 145 us, 156 in halves.)
    a.r32 = !kv_misaligned(residual_out, 32) && ldro % 16 == 0 &&
            !((mode == kNormI8H || mode == kNormF8H) && K <= 8192);
    a.q32 = !kv_misaligned(q, 32) && K % 32 == 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (mode) {
        case kNormBf16: return launch_norm<kNormBf16>(a, env, st);
        case kNormI8H: return launch_norm<kNormI8H>(a, env, st);
        case kNormF8: return launch_norm<kNormF8>(a, env, st);
        case kNormF8H: return launch_norm<kNormF8H>(a, env, st);
        default: return launch_norm<kNormF8B>(a, env, st);
    }
}

}  // namespace

}  // namespace clef

using namespace clef;

extern "C" int clef_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *w, int64_t M,
                             int64_t K, float eps, void *residual_out, int64_t ldro, void *y, int64_t ldy, void *stream) {
    return norm_call(x, ldx, residual, ldr, w, M, K, eps, kNormBf16, residual_out, ldro, y, ldy, nullptr, nullptr, stream);
}

extern "C" int clef_rms_norm_quant(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *w, int64_t M,
                                   int64_t K, float eps, int mode, void *residual_out, int64_t ldro, void *y, int64_t ldy,
                                   void *q, float *scale, void *stream) {
    if (mode != CLEF_ACT_INT8_H128 && mode != CLEF_ACT_FP8_E4M3 && mode != CLEF_ACT_FP8_E4M3_H128 && mode != CLEF_ACT_FP8_E4M3_B128)
        return kv_fail("unknown quantizer mode");
    return norm_call(x, ldx, residual, ldr, w, M, K, eps, mode, residual_out, ldro, y, ldy, q, scale, stream);
}

extern "C" int clef_quant_fp8_block(const void *x, int64_t M, int64_t K, int64_t ldx, int rows, void *q, float *scale,
                                    void *stream) {
    if (rows != 1 && rows != 128) return kv_fail("rows must be 1 or 128");
    if (M < 0 || M > 0x7FFFFFFF) return kv_fail("M out of range");
    if (K <= 0 || K > 65536 || K % kE != 0) return kv_fail("K must be in (0, 65536] and a multiple of 16");
    if (ldx < K || ldx % 8 != 0) return kv_fail("ldx must be >= K and a multiple of 8");
    if (M == 0) return CLEF_OK;
    if (!x || !q || !scale) return kv_fail("null pointer");
    if (kv_misaligned(x, 16) || kv_misaligned(q, 16)) return kv_fail("x and q must be 16-byte aligned");
    if (kv_misaligned(scale, 4)) return kv_fail("scale not 4-byte aligned");
    int sms = 0;
    unsigned int *status = nullptr;
    const int rc = internal_device(&sms, &status);
    if (rc) return rc;
    const int blocks = (int)((K + 127) / 128);
    const bool q32 = !kv_misaligned(q, 32) && K % 32 == 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (rows == 1) {
        const int64_t total = M * blocks, most = (int64_t)internal_launch_sms(sms) * 64;
        const int64_t grid = (total + 63) / 64;
        e = launch_kernel(quant_rows_kernel, dim3((unsigned)(grid < most ? grid : most)), dim3(256), 0, st, 1, true,
                          static_cast<const uint16_t *>(x), ldx, (int)K, blocks, total, q32, static_cast<uint8_t *>(q), scale);
    } else {
        const int64_t grid = (M + 127) / 128 * blocks;   // (under 2^31 / 128 * 512)
        if (grid > 0x7FFFFFFF) return kv_fail("too many blocks");
        e = launch_kernel(quant_tiles_kernel, dim3((unsigned)grid), dim3(512), 0, st, 1, true,
                          static_cast<const uint16_t *>(x), ldx, M, (int)K, blocks, q32, static_cast<uint8_t *>(q), scale);
    }
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "block quantizer launch");
}
