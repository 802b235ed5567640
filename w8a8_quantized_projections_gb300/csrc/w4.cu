// w4.cu -- linears over 4-bit weights with group scales, for calls of few
// rows (a token per sequence), and the quantizer that packs such weights.
//
//   y[m][n] = bf16( sum_g s[n][g] * ( sum_{k in group g} c[n][k] x[m][k] ) + bias[n] )
//
// with c in -8..7 and s a bf16 scale for each run of 32, 64 or 128 weights.
// With one to sixteen rows the call is a read of the weights (half a byte
// each): the work is to keep enough loads in flight and to widen the codes in
// few instructions.
//
// Layout.  A row is cut into blocks of 128 weights (64 bytes), a short last
// block filled with the code of zero.  Byte 16 t + 4 j of a block starts the
// 32-bit word with weights 32 j + 8 t .. + 7 (t, j in 0..3): lane t of a
// four-lane group then reads 16 contiguous bytes and holds, for each of the
// block's four 32-weight runs, the eight weights that it feeds to the tensor
// core, so that every mma stays inside one scale group whatever its length.
// Nibble i < 4 of a word holds weight 2 i, nibble i + 4 weight 2 i + 1, so
// that (w >> 4 i) & 0x000F000F is a pair of neighbours in two halfwords.  A
// nibble holds c + 8.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "clef_ptx.cuh"

namespace clef {

namespace {

constexpr int kBlockK = 128;      // weights of a packed block
constexpr int kWarps = 8;
constexpr int kParts = 8;         // runs of K that are summed apart, then added in order
constexpr int kDepth = 4;         // blocks of weights a warp has in flight

// Two codes (nibbles in bits 0-3 and 16-19 of w) as bf16: 0x4300 | u is
// 128 + u, and 128 + u - 136 = u - 8 without rounding.
__device__ __forceinline__ uint32_t widen(uint32_t w) {
    uint32_t v;
    asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(v) : "r"(w));   // (w & mask) | 0x4300
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(v) : "r"(v), "r"(0x43084308u));
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load_stream(const uint8_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// The scales of one block of a row: 128 / GROUP bf16 values.
template <int GROUP>
struct Scales {
    uint32_t w[GROUP == 32 ? 2 : 1];
    __device__ __forceinline__ void load(const uint16_t *p) {
        if constexpr (GROUP == 32) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p);
            w[0] = v.x;
            w[1] = v.y;
        } else if constexpr (GROUP == 64) {
            w[0] = *reinterpret_cast<const uint32_t *>(p);
        } else {
            w[0] = *p;
        }
    }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t v = w[i / 2];
        return __uint_as_float((i & 1) ? (v & 0xFFFF0000u) : (v << 16));
    }
};

struct W4Args {
    const uint16_t *x;
    int64_t ldx;
    const uint8_t *qw;
    const uint16_t *sw;
    const uint16_t *bias;
    uint16_t *y;
    int64_t ldy;
    int M, N, K;
    int kb, part;      // blocks of a weight row, and of one of its kParts parts
    int tiles;         // of 16 * cluster rows
};

// A cluster of S CTAs takes tiles of 16 S weight rows in turn.  K is cut into
// eight parts whatever S is; CTA r of the cluster has 8 / S of them, and its
// eight warps are 8 / S parts times S groups of 16 rows.  A tile's eight
// partial sums meet in shared memory (of the cluster) and are added in the order
// of K, so a row of y has the same bits whatever M, S and the grid are.
//
// A warp streams its part of 16 rows into registers, kDepth blocks ahead, across
// the tiles: the loads never wait for a sum.  x's columns of the CTA's parts are
// read once into shared memory; S is as large as it takes to fit them.
template <int NT, int GROUP>
__global__ void __launch_bounds__(kWarps * 32, 2) w4_linear_kernel(const W4Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    uint32_t rank, csize;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(csize));
    const int S = (int)csize, own = kParts / S;                  // parts of this CTA
    const int rows = 16 * S, m0 = (int)blockIdx.y * NT * 8, mn = min(NT * 8, a.M - m0);
    const int kb_own = (int)rank * own * a.part;                 // first block of this CTA
    const int slice = own * a.part;                              // its blocks
    const int pitch = slice * kBlockK * 2 + 64;                  // bytes of a row of x: 64 past a multiple of 128
    float *part_sums = reinterpret_cast<float *>(smem + mn * pitch);      // [2][own][NT * 8][rows]
    const int wp = warp % own, wr = warp / own;                  // this warp's part and rows
    const int b0 = kb_own + wp * a.part;
    const int first = (int)blockIdx.x / S, stride = (int)gridDim.x / S;
    constexpr int kPer = kBlockK / GROUP;

    pdl_wait();

    uint4 wa[kDepth], wb[kDepth];
    Scales<GROUP> sa[kDepth], sb[kDepth];
    // where the next load is: tile and block of the part
    int lt = first, lb = 0;
    const auto load = [&](uint4 &va, uint4 &vb, Scales<GROUP> &ua, Scales<GROUP> &ub) {
        if (lt < a.tiles && b0 + lb < a.kb) {
            // rows past N read the last one and are dropped
            const int n = lt * rows + wr * 16 + g, r0 = min(n, a.N - 1), r1 = min(n + 8, a.N - 1);
            const int64_t i0 = (int64_t)r0 * a.kb + b0 + lb, i1 = (int64_t)r1 * a.kb + b0 + lb;
            va = load_stream(a.qw + i0 * 64 + t * 16);
            vb = load_stream(a.qw + i1 * 64 + t * 16);
            ua.load(a.sw + i0 * kPer);
            ub.load(a.sw + i1 * kPer);
        }
        if (++lb == a.part) {
            lb = 0;
            lt += stride;
        }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(wa[d], wb[d], sa[d], sb[d]);

    // x's columns of this CTA, zeros past K
    {
        const int words = slice * (kBlockK / 8);
        for (int m = 0; m < mn; ++m)
            for (int o = tid; o < words; o += kWarps * 32) {
                const int k = kb_own * kBlockK + o * 8;
                uint4 v = make_uint4(0, 0, 0, 0);
                if (k < a.K) v = *reinterpret_cast<const uint4 *>(a.x + (int64_t)(m0 + m) * a.ldx + k);
                *reinterpret_cast<uint4 *>(smem + m * pitch + o * 16) = v;
            }
    }
    __syncthreads();

    const uint8_t *xs = smem + wp * a.part * 256 + t * 16;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    int tile = first, b = 0, turn = 0;
    while (tile < a.tiles) {
#pragma unroll
        for (int d = 0; d < kDepth; ++d) {
            if (tile >= a.tiles) break;
            if (b0 + b < a.kb) {
                const uint32_t ra[4] = {wa[d].x, wa[d].y, wa[d].z, wa[d].w};
                const uint32_t rb[4] = {wb[d].x, wb[d].y, wb[d].z, wb[d].w};
                const Scales<GROUP> ua = sa[d], ub = sb[d];
                load(wa[d], wb[d], sa[d], sb[d]);
                float gr[NT][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (j % (GROUP / 32) == 0) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int i = 0; i < 4; ++i) gr[nt][i] = 0.0f;
                    }
                    uint32_t pa[4], pb[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        pa[i] = widen(ra[j] >> (4 * i));
                        pb[i] = widen(rb[j] >> (4 * i));
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        uint4 xv = make_uint4(0, 0, 0, 0);
                        if (nt * 8 + g < mn)
                            xv = *reinterpret_cast<const uint4 *>(xs + (nt * 8 + g) * pitch + b * 256 + j * 64);
                        mma_bf16(gr[nt], pa[0], pb[0], pa[1], pb[1], xv.x, xv.y);
                        mma_bf16(gr[nt], pa[2], pb[2], pa[3], pb[3], xv.z, xv.w);
                    }
                    if ((j + 1) % (GROUP / 32) == 0) {
                        const float fa = ua.get(j / (GROUP / 32)), fb = ub.get(j / (GROUP / 32));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            acc[nt][0] = fmaf(fa, gr[nt][0], acc[nt][0]);
                            acc[nt][1] = fmaf(fa, gr[nt][1], acc[nt][1]);
                            acc[nt][2] = fmaf(fb, gr[nt][2], acc[nt][2]);
                            acc[nt][3] = fmaf(fb, gr[nt][3], acc[nt][3]);
                        }
                    }
                }
            } else {
                load(wa[d], wb[d], sa[d], sb[d]);
            }
            if (++b < a.part) continue;
            // the tile's partial sums, [part][row of x][weight row]; two buffers in turns, so that one
            // meeting of the warps a tile is enough
            float *sums = part_sums + turn * own * NT * 8 * rows;
            float *mine = sums + wp * NT * 8 * rows + wr * 16;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int m = nt * 8 + 2 * t + (i & 1);
                    if (m < mn) mine[m * rows + g + 8 * (i >> 1)] = acc[nt][i];
                    acc[nt][i] = 0.0f;
                }
            if (S == 1)
                __syncthreads();
            else
                asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
            // each CTA finishes 16 of the rows
            for (int i = tid; i < mn * 16; i += kWarps * 32) {
                const int m = i >> 4, r = (int)rank * 16 + (i & 15), n = tile * rows + r;
                if (n < a.N) {
                    float v = 0.0f;
                    for (int p = 0; p < kParts; ++p) {
                        const float *at = sums + ((p % own) * NT * 8 + m) * rows + r;
                        if (S == 1) {
                            v += *at;
                        } else {
                            uint32_t addr;
                            float q;
                            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(at)), "r"((uint32_t)(p / own)));
                            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q) : "r"(addr) : "memory");
                            v += q;
                        }
                    }
                    if (a.bias) v += __uint_as_float((uint32_t)a.bias[n] << 16);
                    const __nv_bfloat16 o = __float2bfloat16_rn(v);
                    a.y[(int64_t)(m0 + m) * a.ldy + n] = *reinterpret_cast<const uint16_t *>(&o);
                }
            }
            b = 0;
            turn ^= 1;
            tile += stride;
        }
    }
    pdl_launch_dependents();
    // no CTA of a cluster ends while another reads its sums
    if (S > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Packs bf16 weight rows: s = bf16(amax / 7) of each group, codes
// clamp(rne(w / s), -8, 7) with one IEEE division each (a scale of zero gives
// codes of zero).  A thread owns one word of eight weights; the lanes of a
// group meet by shuffles.  Weight set-up, run once per weight.
template <int GROUP>
__global__ void __launch_bounds__(256) quant_w4_kernel(const uint16_t *w, int64_t ldw, int K, int kb,
                                                       int64_t words, uint32_t *qw,
                                                       uint16_t *sw) {
    pdl_wait();
    const int64_t stride = (int64_t)gridDim.x * blockDim.x;
    // every lane of a warp runs the same number of rounds (words is a multiple of 16; the loop bound is rounded up)
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < (words + 31) / 32 * 32; i += stride) {
        const bool in = i < words;
        const int64_t row = i / (kb * 16), rest = in ? i - row * (kb * 16) : 0;
        const int blk = (int)(rest >> 4), j = (int)(rest >> 2) & 3, t = (int)rest & 3;
        const int k = blk * kBlockK + 32 * j + 8 * t;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (in && k < K) v = *reinterpret_cast<const uint4 *>(w + row * ldw + k);
        const uint32_t r[4] = {v.x, v.y, v.z, v.w};
        float f[8], amax = 0.0f;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            f[2 * p] = __uint_as_float(r[p] << 16);
            f[2 * p + 1] = __uint_as_float(r[p] & 0xFFFF0000u);
            amax = fmaxf(amax, fmaxf(fabsf(f[2 * p]), fabsf(f[2 * p + 1])));
        }
#pragma unroll
        for (int o = 1; o < GROUP / 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
        const __nv_bfloat16 sb = __float2bfloat16_rn(__fdiv_rn(amax, 7.0f));
        const float s = __bfloat162float(sb);
        uint32_t word = 0;
#pragma unroll
        for (int o = 0; o < 8; ++o) {
            float c = s > 0.0f ? rintf(__fdiv_rn(f[o], s)) : 0.0f;
            c = fminf(fmaxf(c, -8.0f), 7.0f);
            word |= (uint32_t)((int)c + 8) << (4 * (o / 2 + 4 * (o & 1)));
        }
        if (in) {
            qw[(row * kb + blk) * 16 + t * 4 + j] = word;
            if ((k & (GROUP - 1)) == 0)
                sw[(row * kb + blk) * (kBlockK / GROUP) + (k & (kBlockK - 1)) / GROUP] =
                    *reinterpret_cast<const uint16_t *>(&sb);
        }
    }
    pdl_launch_dependents();
}

int fail(const char *msg) {
    internal_set_error(msg);
    return CLEF_ERR_INVALID_ARG;
}

bool misaligned(const void *p, unsigned to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

constexpr int64_t kMaxW4 = (int64_t)1 << 24, kMaxK = 65536;

template <int NT, int GROUP>
cudaError_t launch_w4(const W4Args &a, int split, int blocks_m, int sms, cudaStream_t st) {
    const int own = kParts / split, rows = 16 * split, m = a.M < NT * 8 ? a.M : NT * 8;
    const size_t smem = (size_t)m * (own * a.part * kBlockK * 2 + 64) + (size_t)2 * own * NT * 8 * rows * 4;
    static SmemOptIn opt;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(w4_linear_kernel<NT, GROUP>), 220 * 1024);
    if (e != cudaSuccess) return e;
    const int per_sm = smem <= 110 * 1024 ? 2 : 1;
    int clusters = sms * per_sm / split;
    if (clusters < 1) clusters = 1;
    if (clusters > a.tiles) clusters = a.tiles;
    return launch_kernel(w4_linear_kernel<NT, GROUP>, dim3((unsigned)(clusters * split), (unsigned)blocks_m), dim3(kWarps * 32),
                         smem, st, split, true, a);
}

template <int NT>
cudaError_t launch_w4_group(const W4Args &a, int group, int split, int blocks_m, int sms, cudaStream_t st) {
    switch (group) {
        case 32: return launch_w4<NT, 32>(a, split, blocks_m, sms, st);
        case 64: return launch_w4<NT, 64>(a, split, blocks_m, sms, st);
        default: return launch_w4<NT, 128>(a, split, blocks_m, sms, st);
    }
}

}  // namespace

}  // namespace clef

using namespace clef;

extern "C" int clef_quant_w4(const void *w, int64_t N, int64_t K, int64_t ldw, int group, void *qw, void *sw,
                             void *stream) {
    if (N < 0 || N > kMaxW4) return fail("invalid argument: N out of range");
    if (K <= 0 || K > kMaxK || K % 8 != 0) return fail("invalid argument: K must be in (0, 65536] and a multiple of 8");
    if (ldw < K || ldw % 8 != 0) return fail("invalid argument: ldw must be >= K and a multiple of 8");
    if (group != 32 && group != 64 && group != 128) return fail("invalid argument: group must be 32, 64 or 128");
    if (N == 0) return CLEF_OK;
    if (!w || !qw || !sw) return fail("invalid argument: null pointer");
    if (misaligned(w, 16) || misaligned(qw, 16) || misaligned(sw, 16))
        return fail("invalid argument: w, qw and sw must be 16-byte aligned");
    int sms = 0;
    unsigned int *status = nullptr;
    int rc = internal_device(&sms, &status);
    if (rc) return rc;
    const int kb = (int)((K + kBlockK - 1) / kBlockK);
    const int64_t words = N * kb * 16;
    int64_t grid = (words + 255) / 256;
    if (grid > (int64_t)sms * 8) grid = (int64_t)sms * 8;
    auto kern = group == 32 ? quant_w4_kernel<32> : group == 64 ? quant_w4_kernel<64> : quant_w4_kernel<128>;
    cudaError_t e = launch_kernel(kern, dim3((unsigned)grid), dim3(256), 0, static_cast<cudaStream_t>(stream), 1, true,
                                  static_cast<const uint16_t *>(w), ldw, (int)K, kb, words,
                                  static_cast<uint32_t *>(qw), static_cast<uint16_t *>(sw));
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "4-bit weight quantizer launch");
}

extern "C" int clef_w4_linear(const void *x, int64_t ldx, const void *qw, const void *sw, int group, const void *bias,
                              int64_t M, int64_t N, int64_t K, void *y, int64_t ldy, void *stream) {
    if (M < 0 || M > kMaxW4 / 32) return fail("invalid argument: M out of range");
    if (N <= 0 || N > kMaxW4) return fail("invalid argument: N out of range");
    if (K <= 0 || K > kMaxK || K % 8 != 0) return fail("invalid argument: K must be in (0, 65536] and a multiple of 8");
    if (group != 32 && group != 64 && group != 128) return fail("invalid argument: group must be 32, 64 or 128");
    if (ldx < K || ldx % 8 != 0) return fail("invalid argument: ldx must be >= K and a multiple of 8");
    if (ldy < N) return fail("invalid argument: ldy must be >= N");
    if (M == 0) return CLEF_OK;
    if (!x || !qw || !sw || !y) return fail("invalid argument: null pointer");
    if (misaligned(x, 16) || misaligned(qw, 16) || misaligned(sw, 16))
        return fail("invalid argument: x, qw and sw must be 16-byte aligned");
    if (misaligned(y, 2) || misaligned(bias, 2)) return fail("invalid argument: y and bias must be 2-byte aligned");
    int sms = 0;
    unsigned int *status = nullptr;
    int rc = internal_device(&sms, &status);
    if (rc) return rc;
    const int kb = (int)((K + kBlockK - 1) / kBlockK);
    const int part = (kb + kParts - 1) / kParts;
    // CTAs of a cluster: so many that a CTA's columns of x leave room for two CTAs an SM
    const auto x_bytes = [&](int64_t m, int split) { return m * (kParts / split * part * kBlockK * 2 + 64); };
    const int64_t block_m = M > 8 && x_bytes(M < 16 ? M : 16, kParts) <= 200 * 1024 ? 16 : 8;
    int split = 1;
    while (split < kParts && x_bytes(M < block_m ? M : block_m, split) > 80 * 1024) split *= 2;
    W4Args a;
    a.x = static_cast<const uint16_t *>(x);
    a.ldx = ldx;
    a.qw = static_cast<const uint8_t *>(qw);
    a.sw = static_cast<const uint16_t *>(sw);
    a.bias = static_cast<const uint16_t *>(bias);
    a.y = static_cast<uint16_t *>(y);
    a.ldy = ldy;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.kb = kb;
    a.part = part;
    a.tiles = (int)((N + 16 * split - 1) / (16 * split));
    sms = internal_launch_sms(sms);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int blocks_m = (int)((M + block_m - 1) / block_m);
    const cudaError_t e = block_m == 8 ? launch_w4_group<1>(a, group, split, blocks_m, sms, st)
                                       : launch_w4_group<2>(a, group, split, blocks_m, sms, st);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "4-bit linear launch");
}
