// norm.cu -- what comes before a linear: the root-mean-square norm with the
// residual's addition, its result as bf16 or as the 8-bit codes and scales of
// the linear that follows, and the quantizer of blocks of 128.
//
//   h = x + r (fp32);  r_out = bf16(h);  g = 1 / sqrt(mean(h^2) + eps)
//   y = h w g;  bf16(y), and codes of y (or of its rotation) by their absmax
//
// Bound by HBM: 2 bytes an element in for x, 2 in and 2 out for the residual, 1
// out for a code (2 for a bf16 result), so the row is read once and stays in
// registers.  g is a factor of the whole row, and the rotation is linear: the
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
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "clef_ptx.cuh"
#include "kv_host.h"

namespace clef {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kE = 16;             // consecutive elements of a thread: two 16-byte loads, one 16-byte store of codes
constexpr int kLanes = 128 / kE;   // lanes that hold a block of 128
constexpr float kFltMax = 3.4028234663852886e38f;

enum NormMode : int { kNormBf16 = -1, kNormI8H = kActInt8H128, kNormF8 = kActFp8, kNormF8H = kActFp8H128, kNormF8B = 3 };

__device__ __forceinline__ float lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&p);
}

__device__ __forceinline__ void load16(const uint16_t *p, uint32_t (&w)[8]) {
    const uint4 a = *reinterpret_cast<const uint4 *>(p), b = *(reinterpret_cast<const uint4 *>(p) + 1);
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

__device__ __forceinline__ void store16(uint16_t *p, const uint32_t (&w)[8]) {
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
__device__ __forceinline__ uint4 codes16(const float (&v)[kE], float r) {
    if (!kInt8 && r == 0.0f) return make_uint4(0u, 0u, 0u, 0u);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float *u = v + 4 * i;
        if (kInt8) {
            uint32_t h;
            asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;"
                : "=r"(h) : "r"(__float2int_rn(__fmul_rn(u[3], r))), "r"(__float2int_rn(__fmul_rn(u[2], r))), "r"(0));
            asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;"
                : "=r"(w[i]) : "r"(__float2int_rn(__fmul_rn(u[1], r))), "r"(__float2int_rn(__fmul_rn(u[0], r))), "r"(h));
        } else {
            w[i] = e4m3x2(__fmul_rn(u[0], r), __fmul_rn(u[1], r)) |
                   (e4m3x2(__fmul_rn(u[2], r), __fmul_rn(u[3], r)) << 16);
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// The multiplier of codes whose largest value is top: 0 for zeros, and finite for the smallest values.
__device__ __forceinline__ float code_factor(float amax, float top) {
    return amax == 0.0f ? 0.0f : fminf(__fdiv_rn(top, amax), kFltMax);
}

// The orthonormal Walsh-Hadamard transform of a block of 128 held by eight neighbouring lanes, sixteen
// values each: strides 1 .. 8 in the thread, 16 .. 64 between lanes, the order of clef_quant_act.
__device__ __forceinline__ void rotate16(float (&v)[kE], int lane) {
#pragma unroll
    for (int h = 1; h < kE; h <<= 1)
#pragma unroll
        for (int k = 0; k < kE; ++k)
            if ((k & h) == 0) {
                const float a = v[k], b = v[k + h];
                v[k] = a + b;
                v[k + h] = a - b;
            }
#pragma unroll
    for (int s = 1; s < kLanes; s <<= 1) {
        const float sign = (lane & s) ? -1.0f : 1.0f;
#pragma unroll
        for (int k = 0; k < kE; ++k) v[k] = fmaf(sign, v[k], __shfl_xor_sync(kAll, v[k], s));
    }
#pragma unroll
    for (int k = 0; k < kE; ++k) v[k] *= __uint_as_float(0x3DB504F3u);   // fp32(1 / sqrt(128))
}

struct NormArgs {
    const uint16_t *x, *r, *w;
    uint16_t *r_out, *y;
    uint8_t *q;
    float *scale;
    int64_t ldx, ldr, ldro, ldy, M;
    int K, blocks;
    float eps;
};

// G lanes a row (K up to 16 G), four rows or more a CTA; G = 0: a CTA a row, C chunks of sixteen a thread.
template <int MODE, int C, int G>
__global__ void __launch_bounds__(G ? 128 : (C == 1 ? 1024 : 512)) norm_kernel(const NormArgs a) {
    constexpr bool kRotate = MODE == kNormI8H || MODE == kNormF8H;
    constexpr bool kRowMax = MODE != kNormBf16 && MODE != kNormF8B;
    constexpr bool kInt8 = MODE == kNormI8H;
    constexpr float kTop = kInt8 ? 127.0f : 448.0f;
    __shared__ float2 part[2][32];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t m = G ? blockIdx.x * (int64_t)(128 / (G ? G : 1)) + tid / (G ? G : 1) : (int64_t)blockIdx.x;
    const bool row = !G || m < a.M;
    const int first = G ? tid % (G ? G : 1) : tid, step = G ? 0 : (int)blockDim.x;
    pdl_wait();

    const uint16_t *x = a.x + m * a.ldx;
    const uint16_t *r = a.r + m * a.ldr;
    float v[C][kE];
    float u[kRotate ? C : 1][kE];
    uint32_t sum[C][8];
    float g = 0.0f, amax = 0.0f, unit = 1.0f;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        float ss = 0.0f;
        amax = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = (first + c * step) * kE;
            if (row && e < a.K) {
                uint32_t p[8], w[8];
                load16(x + e, p);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    v[c][2 * i] = lo(p[i]);
                    v[c][2 * i + 1] = hi(p[i]);
                }
                if (a.r) {
                    load16(r + e, p);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        v[c][2 * i] += lo(p[i]);
                        v[c][2 * i + 1] += hi(p[i]);
                        sum[c][i] = pack2(v[c][2 * i], v[c][2 * i + 1]);
                    }
                }
                load16(a.w + e, w);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p0 = v[c][2 * i] * unit, p1 = v[c][2 * i + 1] * unit;
                    ss = fmaf(p0, p0, ss);
                    ss = fmaf(p1, p1, ss);
                    v[c][2 * i] = p0 * lo(w[i]);
                    v[c][2 * i + 1] = p1 * hi(w[i]);
                }
            } else {
#pragma unroll
                for (int k = 0; k < kE; ++k) v[c][k] = 0.0f;
            }
            if (kRotate) {
                // (blocks lie in whole rows: their eight lanes are in or out together)
#pragma unroll
                for (int k = 0; k < kE; ++k) u[c][k] = v[c][k];
                rotate16(u[c], lane);
            }
            if (kRowMax) {
                const float(&t)[kE] = kRotate ? u[c] : v[c];
#pragma unroll
                for (int k = 0; k < kE; ++k) amax = fmaxf(amax, fabsf(t[k]));
            }
        }
#pragma unroll
        for (int s = G ? G / 2 : 16; s > 0; s >>= 1) {
            ss += __shfl_xor_sync(kAll, ss, s);
            if (kRowMax) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
        }
        if (!G) {
            if (lane == 0) part[pass][warp] = make_float2(ss, amax);
            __syncthreads();
            const float2 o = lane < (int)(blockDim.x >> 5) ? part[pass][lane] : make_float2(0.0f, 0.0f);
            ss = o.x;
            amax = o.y;
#pragma unroll
            for (int s = 16; s > 0; s >>= 1) {
                ss += __shfl_xor_sync(kAll, ss, s);
                if (kRowMax) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
            }
        }
        g = __frsqrt_rn(__fdiv_rn(ss, (float)a.K) + a.eps * (unit * unit));
        // squares past fp32: once more, in other units (a warp's other rows find the same again)
        const bool over = !(ss <= kFltMax);
        if (over) unit = 0x1p-80f;
        if (G ? !__any_sync(kAll, over) : !over) break;
    }

#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e = (first + c * step) * kE;
        const bool in = row && e < a.K;
        if (in && a.r) store16(a.r_out + m * a.ldro + e, sum[c]);
        if (in && (MODE == kNormBf16 || a.y)) {
            uint32_t p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) p[i] = pack2(v[c][2 * i] * g, v[c][2 * i + 1] * g);
            store16(a.y + m * a.ldy + e, p);
        }
        if (MODE == kNormF8B) {
            amax = 0.0f;
#pragma unroll
            for (int k = 0; k < kE; ++k) amax = fmaxf(amax, fabsf(v[c][k]));
#pragma unroll
            for (int s = 1; s < kLanes; s <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
        }
        if (MODE != kNormBf16 && in) {
            const float(&t)[kE] = kRotate ? u[kRotate ? c : 0] : v[c];
            *reinterpret_cast<uint4 *>(a.q + m * a.K + e) = codes16<kInt8>(t, code_factor(amax, kTop));
            const float s = __fdiv_rn(amax * g, kTop);
            if (MODE == kNormF8B) {
                if (e % 128 == 0) a.scale[m * a.blocks + e / 128] = s;
            } else if (e == 0) {
                a.scale[m] = s;
            }
        }
    }
    pdl_launch_dependents();
}

// ------------------------------------------------------------ blocks of 128

// Codes of x in blocks of one row by 128: eight lanes a block.
__global__ void __launch_bounds__(256) quant_rows_kernel(const uint16_t *__restrict__ x, int64_t ldx, int K, int blocks,
                                                         int64_t total, uint8_t *__restrict__ q, float *__restrict__ scale) {
    pdl_wait();
    for (int64_t i0 = blockIdx.x * (int64_t)32; i0 < total; i0 += (int64_t)gridDim.x * 32) {
        const int64_t i = i0 + threadIdx.x / kLanes;      // block of the matrix
        const int64_t m = i / blocks;
        const int b = (int)(i - m * blocks), e = b * 128 + (int)(threadIdx.x % kLanes) * kE;
        const bool in = i < total && e < K;
        float v[kE], amax = 0.0f;
        if (in) {
            uint32_t p[8];
            load16(x + m * ldx + e, p);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[2 * k] = lo(p[k]);
                v[2 * k + 1] = hi(p[k]);
                amax = fmaxf(amax, fmaxf(fabsf(v[2 * k]), fabsf(v[2 * k + 1])));
            }
        }
#pragma unroll
        for (int s = 1; s < kLanes; s <<= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
        if (in) {
            *reinterpret_cast<uint4 *>(q + m * K + e) = codes16<false>(v, code_factor(amax, 448.0f));
            if (e % 128 == 0) scale[i] = __fdiv_rn(amax, 448.0f);
        }
    }
    pdl_launch_dependents();
}

// Codes of w in blocks of 128 rows by 128: a CTA a block, 64 values a thread, kept as bf16.
__global__ void __launch_bounds__(256) quant_tiles_kernel(const uint16_t *__restrict__ w, int64_t ldw, int64_t M, int K,
                                                          int blocks, uint8_t *__restrict__ q, float *__restrict__ scale) {
    __shared__ float part[8];
    const int64_t mb = blockIdx.x / blocks;
    const int b = (int)(blockIdx.x - mb * blocks), e = b * 128 + (int)(threadIdx.x % kLanes) * kE;
    const int64_t m0 = mb * 128 + threadIdx.x / kLanes;
    pdl_wait();
    uint32_t p[4][8];
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (e < K && m0 + 32 * j < M) {
            load16(w + (m0 + 32 * j) * ldw + e, p[j]);
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) p[j][k] = 0u;
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) amax = fmaxf(amax, fmaxf(fabsf(lo(p[j][k])), fabsf(hi(p[j][k]))));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, s));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = fmaxf(amax, part[i]);
    const float r = code_factor(amax, 448.0f);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (e < K && m0 + 32 * j < M) {
            float v[kE];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                v[2 * k] = lo(p[j][k]);
                v[2 * k + 1] = hi(p[j][k]);
            }
            *reinterpret_cast<uint4 *>(q + (m0 + 32 * j) * K + e) = codes16<false>(v, r);
        }
    }
    if (threadIdx.x == 0) scale[blockIdx.x] = __fdiv_rn(amax, 448.0f);
    pdl_launch_dependents();
}

// ------------------------------------------------------------ launches

template <int MODE>
cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
    const int chunks = a.K / kE;
    const auto lanes = [&](auto kern, int g) {
        const int64_t rows = 128 / g;
        return launch_kernel(kern, dim3((unsigned)((a.M + rows - 1) / rows)), dim3(128), 0, st, 1, true, a);
    };
    if (chunks <= 8) return lanes(norm_kernel<MODE, 1, 8>, 8);
    if (chunks <= 16) return lanes(norm_kernel<MODE, 1, 16>, 16);
    if (chunks <= 32) return lanes(norm_kernel<MODE, 1, 32>, 32);
    const auto cta = [&](auto kern, int c) {
        const unsigned threads = (unsigned)((chunks + 32 * c - 1) / (32 * c) * 32);
        return launch_kernel(kern, dim3((unsigned)a.M), dim3(threads), 0, st, 1, true, a);
    };
    if (chunks <= 1024) return cta(norm_kernel<MODE, 1, 0>, 1);
    return cta(norm_kernel<MODE, 4, 0>, 4);
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
    int sms = 0;
    unsigned int *status = nullptr;
    const int rc = internal_device(&sms, &status);
    if (rc) return rc;
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
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    switch (mode) {
        case kNormBf16: e = launch_norm<kNormBf16>(a, st); break;
        case kNormI8H: e = launch_norm<kNormI8H>(a, st); break;
        case kNormF8: e = launch_norm<kNormF8>(a, st); break;
        case kNormF8H: e = launch_norm<kNormF8H>(a, st); break;
        default: e = launch_norm<kNormF8B>(a, st); break;
    }
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "norm launch");
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
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e;
    if (rows == 1) {
        const int64_t total = M * blocks, most = (int64_t)internal_launch_sms(sms) * 64;
        const int64_t grid = (total + 31) / 32;
        e = launch_kernel(quant_rows_kernel, dim3((unsigned)(grid < most ? grid : most)), dim3(256), 0, st, 1, true,
                          static_cast<const uint16_t *>(x), ldx, (int)K, blocks, total, static_cast<uint8_t *>(q), scale);
    } else {
        const int64_t grid = (M + 127) / 128 * blocks;   // (under 2^31 / 128 * 512)
        if (grid > 0x7FFFFFFF) return kv_fail("too many blocks");
        e = launch_kernel(quant_tiles_kernel, dim3((unsigned)grid), dim3(256), 0, st, 1, true,
                          static_cast<const uint16_t *>(x), ldx, M, (int)K, blocks, static_cast<uint8_t *>(q), scale);
    }
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "block quantizer launch");
}
