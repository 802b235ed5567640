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
// nibble holds u = c + 8.
//
// Widening.  The halfword u is an fp16 number as it is: u 2^-24, below the
// normal numbers and exact, and tensor cores take such numbers whole.  With
// w & 0x00F000F0 it is u 2^-20, whose x is stored 2^-4 as large.  So a word's
// eight codes become operands in five instructions: w and w >> 8 under two masks.
// The 8 in u leaves by the sum's start value, -8 2^-24 sum x over the group.
// x is held in fp16, each run of K that is summed apart scaled by a power of
// two to a largest magnitude in [2^13, 2^14): bf16 has fewer bits than fp16,
// so only values under 2^-23 of the run's largest lose any, and none more than 2^-38
// of it.  As the sums are of (c + 8) x, their rounding goes by (|c| + 8) |x|: a value of x some 2^20 times as
// large as the others hides theirs in its group, whatever its own code is.
#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/clef.h"
#include "clef_kernels.h"
#include "clef_ptx.cuh"

namespace clef {

namespace {

constexpr int kBlockK = 128;      // weights of a packed block
constexpr int kParts = 8;         // runs of K that are summed apart, then added in order
constexpr int kDepth = 2;         // stages of two blocks that a warp has on their way; one more is in use
constexpr int kStage = 2048 + 256;    // bytes of a stage: 16 rows of 128, and their scales

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The scales of one block of a row: 128 / GROUP bf16 values.
template <int GROUP>
struct Scales {
    uint32_t w[GROUP == 32 ? 2 : 1];
    // block b (0 or 1) of a stage; GROUP 128: `odd`, which of the first word's two the first block has
    __device__ __forceinline__ void load(const uint8_t *p, uint32_t odd, int b) {
        if constexpr (GROUP == 32) {
            const uint2 v = *reinterpret_cast<const uint2 *>(p + 8 * b);
            w[0] = v.x;
            w[1] = v.y;
        } else if constexpr (GROUP == 64) {
            w[0] = *reinterpret_cast<const uint32_t *>(p + 4 * b);
        } else {
            w[0] = *reinterpret_cast<const uint16_t *>(p + 2 * (odd + b));
        }
    }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t v = w[i / 2];
        return __uint_as_float((i & 1) ? (v & 0xFFFF0000u) : (v << 16));
    }
};

// 16 bytes, of which the last 16 - there are zeros
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int there = 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there) : "memory");
}
template <int BYTES>
__device__ __forceinline__ void copy_some(uint32_t dst, const void *src, int there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(BYTES), "r"(there) : "memory");
}

template <int N>
struct Count {
    static constexpr int value = N;
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
    int tiles;         // of 2 * warps * cluster rows
    int split_log2;    // CTAs of a cluster
};

// A cluster of S CTAs takes tiles of 16 S weight rows (24 S with twelve warps) in
// turn.  K is cut into eight parts whatever S is; CTA r of the cluster has 8 / S of
// them, and its eight warps are 8 / S parts times S groups of 16 rows.  A tile's eight
// partial sums meet in shared memory (of the cluster) and are added in the order
// of K, so a row of y has the same bits whatever M, S and the grid are.
//
// A warp streams its part of 16 rows through a ring of its own in shared memory,
// kDepth stages ahead, across the tiles: the copies never wait for a sum.  x's columns of the CTA's parts
// are read once into shared memory; S is as large as it takes to fit them.
//
// Measured (K x N, us a call back to back, weights from memory): one row 5120 x
// 34816 in groups of 64, 19.8 us, 4.8 TB/s; 6144 x 5120 in groups of 128, 6.8 us.
// The same over 16 weight rows alone, which leaves the launch, x to fp16 and one
// tile, takes 3.5 and 3.8 us (2.0 us of them without x: K = 128).  13 rows
// of 17408 x 5120 in groups of 32, 29.6 us; over 16 weight rows 15.6 us, most of it x to fp16 and the
// length of a part.  They take two rounds of tiles (1.5 would do), in which three warps a scheduler wait
// for products and for x from shared memory.
template <int NT, int GROUP, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, NT == 1 ? 2 : 1) w4_linear_kernel(const W4Args a) {
    extern __shared__ __align__(16) uint8_t smem[];
    // what a part's sum of a row of x is multiplied by, but for 2^12 (up to 2^138 does not fit) that
    // the finished sum is
    __shared__ float s_unit[NT * 8][kParts];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    uint32_t rank;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    const int S = 1 << a.split_log2, own_log2 = 3 - a.split_log2, own = 1 << own_log2;      // own: parts of this CTA
    const int rows = 16 * (WARPS >> own_log2), m0 = (int)blockIdx.y * NT * 8, mn = min(NT * 8, a.M - m0);
    const int kb_own = (int)rank * own * a.part;                 // first block of this CTA
    const int slice = own * a.part;                              // its blocks
    const int pitch = slice * kBlockK * 2 + 64;                  // bytes of a row of x: 64 past a multiple of 128
    constexpr int kPer = kBlockK / GROUP;
    const int groups = slice * kPer;
    float *x_sums = reinterpret_cast<float *>(smem + mn * pitch);         // [groups][NT * 8]: where the sums start
    float *part_sums = x_sums + groups * NT * 8;                          // [2][own][NT * 8][rows]
    const int wp = warp & (own - 1), wr = warp >> own_log2;                  // this warp's part and rows
    const int b0 = kb_own + wp * a.part, nb = max(0, min(a.part, a.kb - b0));     // its blocks (a last part may have fewer)
    const int first = (int)blockIdx.x >> a.split_log2, stride = (int)gridDim.x >> a.split_log2;
    uint8_t *ring = reinterpret_cast<uint8_t *>(part_sums + 2 * own * NT * 8 * rows) + warp * (kDepth + 1) * kStage;

    pdl_wait();

    // where the next copy is: its tile, block and addresses (rows past N read the last one and are
    // dropped).  A lane copies 16 bytes of rows lane / 8 + 4 i, so that eight lanes take a whole 128-byte
    // line, and the scales of a block of row lane % 16; in the stage the halves of every second row are
    // swapped, so that the lanes' reads meet every bank once.
    int lt = first, lb = 0, put = 0;
    const uint8_t *wsrc = nullptr;
    int woff[4];
    const uint16_t *sc = nullptr;
    const uint16_t *sc_end = a.sw + (int64_t)a.N * a.kb * kPer;
    const auto to_tile = [&]() {
        const int n = lt * rows + wr * 16, n0 = min(n + (lane >> 3), a.N - 1);
        wsrc = a.qw + ((int64_t)n0 * a.kb + b0) * 64 + (lane & 7) * 16;
#pragma unroll
        for (int i = 0; i < 4; ++i) woff[i] = (min(n + (lane >> 3) + 4 * i, a.N - 1) - n0) * a.kb * 64;
        sc = a.sw + ((int64_t)min(n + (lane & 15), a.N - 1) * a.kb + b0) * kPer;
        if constexpr (GROUP == 128)      // the aligned word that holds the row's first scale, or the next one
            sc = reinterpret_cast<const uint16_t *>(reinterpret_cast<uintptr_t>(sc) & ~(uintptr_t)3) + 2 * (lane >> 4);
        else
            sc += (lane >> 4) * kPer;
    };
    const uint32_t ring_at = smem_u32(ring), lane_at = ring_at + (lane >> 3) * 128 + (((lane & 7) ^ ((lane >> 3 & 1) << 2)) << 4);
    const auto fetch = [&]() {
        if (nb > 0 && lt < a.tiles) {
            const uint32_t dst = (uint32_t)(put * kStage);
            // a part's odd last block is copied twice, the second time for nothing
            const bool both = lb + 1 < nb;
            const uint8_t *src = both || (lane & 4) == 0 ? wsrc : wsrc - 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) copy16(lane_at + dst + i * 512, src + woff[i]);
            wsrc += 128;
            const uint32_t at = ring_at + dst + 2048 + (lane & 15) * 16 + (lane >> 4) * (GROUP == 32 ? 8 : 4);
            if constexpr (GROUP == 128) {      // past the array's end nothing is read
                const int64_t left = sc_end - sc;
                copy_some<4>(at, left > 0 ? sc : a.sw, left >= 2 ? 4 : left == 1 ? 2 : 0);
            } else {
                copy_some<2 * kPer>(at, both || lane < 16 ? sc : sc - kPer, 2 * kPer);
            }
            sc += 2 * kPer;
            lb += 2;
            if (lb >= nb) {
                lb = 0;
                lt += stride;
                to_tile();
            }
        }
        put = put == kDepth ? 0 : put + 1;
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    // x's columns of this CTA, zeros past K: a warp a (row, part)
    for (int i = warp; i < mn * own; i += WARPS) {
        const int m = i >> own_log2, p = i & (own - 1), words = a.part * (kBlockK / 8), k0 = (kb_own + p * a.part) * kBlockK;
        const uint16_t *src = a.x + (int64_t)(m0 + m) * a.ldx;
        const uint32_t dst = smem_u32(smem + m * pitch + p * a.part * 256);
        for (int o = lane; o < words; o += 32) {
            const int k = k0 + o * 8;
            copy16(dst + o * 16, src + (k < a.K ? k : 0), k < a.K ? 16 : 0);
        }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    if (nb > 0) to_tile();
    for (int d = 0; d < kDepth; ++d) fetch();
    asm volatile("cp.async.wait_group %0;" ::"n"(kDepth) : "memory");      // x is there
    __syncwarp();

    // to fp16
    for (int i = warp; i < mn * own; i += WARPS) {
        const int m = i >> own_log2, p = i & (own - 1), words = a.part * (kBlockK / 8);
        uint4 *at = reinterpret_cast<uint4 *>(smem + m * pitch + p * a.part * 256);
        uint32_t top = 0;
#pragma unroll 4
        for (int o = lane; o < words; o += 32) {
            const uint4 v = at[o];
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu), __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
        }
        top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16)) << 16;      // bf16 bits order like integers
        const int e = top ? min(120, 13 - (int)(top >> 23) + 127) : 0;      // -115 or more
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll 2
        for (int o = lane; o < (words + 31) / 32 * 32; o += 32) {
            float sum = 0.0f;
            if (o < words) {
                const uint4 v = at[o];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    // the second and fourth pair meet codes 2^4 as large
                    const float f = (k & 1) ? up * 0.0625f : up, back = (k & 1) ? 16.0f : 1.0f;
                    h[k] = pack_half(__uint_as_float(w[k] << 16) * f, __uint_as_float(w[k] & 0xFFFF0000u) * f);
                    const __half2 r = *reinterpret_cast<const __half2 *>(&h[k]);
                    sum = fmaf(back, __low2float(r) + __high2float(r), sum);
                }
                at[o] = make_uint4(h[0], h[1], h[2], h[3]);
            }
            // the lanes of a group: 8 weights each (words is a multiple of 16)
#pragma unroll
            for (int s = 1; s < GROUP / 8; s <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
            if (o < words && (o & (GROUP / 8 - 1)) == 0) x_sums[(p * a.part * kPer + o / (GROUP / 8)) * NT * 8 + m] = -0x1p-21f * sum;
        }
        if (lane == 0) s_unit[m][p] = __uint_as_float((uint32_t)(127 + 12 - e) << 23);
    }
    __syncthreads();

    // x's rows of this lane's columns (columns that are not there read the last row and are dropped)
    const uint8_t *xs[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) xs[nt] = smem + min(nt * 8 + g, mn - 1) * pitch + wp * a.part * 256 + t * 16;
    const float2 *starts = reinterpret_cast<const float2 *>(x_sums + wp * a.part * kPer * NT * 8) + t;
    float unit[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) unit[nt][i] = nt * 8 + 2 * t + i < mn ? s_unit[nt * 8 + 2 * t + i][wp] : 0.0f;
    float acc[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[nt][i] = 0.0f;
    int turn = 0, get = 0;
    const uint8_t *st = ring;
    for (int tile = first; tile < a.tiles; tile += stride, turn ^= 1) {
        // which half of its four bytes a row's first scale of the part is in
        uint32_t odd_a = 0, odd_b = 0;
        if constexpr (GROUP == 128) {
            const int n = tile * rows + wr * 16 + g;
            odd_a = (uint32_t)(((int64_t)min(n, a.N - 1) * a.kb + b0) & 1);
            odd_b = (uint32_t)(((int64_t)min(n + 8, a.N - 1) * a.kb + b0) & 1);
        }
        // COUNT blocks of the stage, from the part's block b on
        const auto multiply = [&](auto count, int b) {
            constexpr int COUNT = decltype(count)::value, kRuns = GROUP / 32;
            // the sums of each group; a single one in two chains, as a chain of products is as long as the
            // tensor core is deep
            constexpr int kChains = kPer == 1 ? 2 : 1;
            float gr[COUNT * kPer * kChains][NT][4];
            Scales<GROUP> ua[COUNT], ub[COUNT];
            uint32_t ra[COUNT][4], rb[COUNT][4];
#pragma unroll
            for (int k = 0; k < COUNT; ++k) {
                const int odd = (b + k) & 1;
                const uint8_t *at = st + g * 128 + (((odd ^ (g & 1)) << 6) | (t << 4));
                const uint4 va = *reinterpret_cast<const uint4 *>(at), vb = *reinterpret_cast<const uint4 *>(at + 1024);
                ra[k][0] = va.x, ra[k][1] = va.y, ra[k][2] = va.z, ra[k][3] = va.w;
                rb[k][0] = vb.x, rb[k][1] = vb.y, rb[k][2] = vb.z, rb[k][3] = vb.w;
                ua[k].load(st + 2048 + g * 16, odd_a, odd);
                ub[k].load(st + 2048 + (g + 8) * 16, odd_b, odd);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int k = 0; k < COUNT; ++k) {
                    const uint32_t la = ra[k][j], lb = rb[k][j], ha = la >> 8, hb = lb >> 8;
                    const int group = k * kPer + j / kRuns;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 xv = *reinterpret_cast<const uint4 *>(xs[nt] + (b + k) * 256 + j * 64);
                        float(&lo)[4] = gr[group * kChains][nt], (&hi)[4] = gr[group * kChains + kChains - 1][nt];
                        float c[4], z[4];
                        if (j % kRuns == 0) {
                            const float2 v = starts[(b * kPer + group) * (NT * 4) + nt * 4];
                            c[0] = c[2] = v.x;
                            c[1] = c[3] = v.y;
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) c[i] = lo[i];
                        }
                        mma_f16(lo, la & 0x000F000Fu, lb & 0x000F000Fu, la & 0x00F000F0u, lb & 0x00F000F0u, xv.x, xv.y, c[0], c[1],
                                c[2], c[3]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) z[i] = kChains == 2 && j == 0 ? 0.0f : hi[i];
                        mma_f16(hi, ha & 0x000F000Fu, hb & 0x000F000Fu, ha & 0x00F000F0u, hb & 0x00F000F0u, xv.z, xv.w, z[0], z[1],
                                z[2], z[3]);
                    }
                }
#pragma unroll
            for (int p = 0; p < COUNT * kPer; ++p) {
                const float fa = ua[p / kPer].get(p % kPer), fb = ub[p / kPer].get(p % kPer);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = kChains == 2 ? gr[p * kChains][nt][i] + gr[p * kChains + kChains - 1][nt][i] : gr[p][nt][i];
                        acc[nt][i] = fmaf(i < 2 ? fa : fb, v, acc[nt][i]);
                    }
            }
        };
        for (int b = 0; b < nb; b += 2) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            __syncwarp();      // every lane's copies are there, and the stage that is filled next is read
            st = ring + get * kStage;
            get = get == kDepth ? 0 : get + 1;
            fetch();
            if (NT == 2 && b + 1 < nb) {      // both at once: two warps a scheduler leave gaps to fill
                multiply(Count<2>(), b);
            } else {
                multiply(Count<1>(), b);
                if (b + 1 < nb) multiply(Count<1>(), b + 1);
            }
        }
        // the tile's partial sums, [part][row of x][weight row]; two buffers in turns, so that one
        // meeting of the warps a tile is enough
        float *sums = part_sums + turn * own * NT * 8 * rows;
        float *mine = sums + wp * NT * 8 * rows + wr * 16;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = nt * 8 + 2 * t + (i & 1);
                if (m < mn) mine[m * rows + g + 8 * (i >> 1)] = acc[nt][i] * unit[nt][i & 1];
                acc[nt][i] = 0.0f;
            }
        if (S == 1)
            __syncthreads();
        else
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        // each CTA finishes its share of the rows
        constexpr int SHARE = 2 * WARPS;      // 16 S (WARPS / 8) rows over S CTAs
        for (int i = tid; i < mn * SHARE; i += WARPS * 32) {
            const int m = i / SHARE, r = (int)rank * SHARE + i - m * SHARE, n = tile * rows + r;
            if (n < a.N) {
                float q[kParts];
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const float *at = sums + ((p & (own - 1)) * NT * 8 + m) * rows + r;
                    if (S == 1) {
                        q[p] = *at;
                    } else {
                        uint32_t addr;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(addr) : "r"(smem_u32(at)), "r"((uint32_t)(p >> own_log2)));
                        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(q[p]) : "r"(addr) : "memory");
                    }
                }
                float v = q[0];
#pragma unroll
                for (int p = 1; p < kParts; ++p) v += q[p];
                v *= 0x1p12f;
                if (a.bias) v += __uint_as_float((uint32_t)a.bias[n] << 16);
                const __nv_bfloat16 o = __float2bfloat16_rn(v);
                a.y[(int64_t)(m0 + m) * a.ldy + n] = *reinterpret_cast<const uint16_t *>(&o);
            }
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

constexpr size_t kMaxSmem = 226 * 1024, kPairSmem = 110 * 1024;      // of a CTA alone on an SM, and of one of two

// Shared memory of a CTA: x's columns, the sums' starts, two tiles' partial sums and the rings.
size_t w4_smem(int nt, int64_t m, int part, int group, int split, int warps) {
    const int own = kParts / split, rows = 2 * warps * split;
    return (size_t)m * (own * part * kBlockK * 2 + 64) + (size_t)own * part * (kBlockK / group) * nt * 8 * 4 +
           (size_t)2 * own * nt * 8 * rows * 4 + (size_t)warps * (kDepth + 1) * kStage;
}

// How many clusters run at once: they do not fill every group of SMs (of 152
// CTAs, 15 clusters of eight do).
template <int NT, int GROUP, int WARPS>
cudaError_t resident_clusters(int split, size_t smem, int sms, int *clusters) {
    static SmemOptIn opt;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(w4_linear_kernel<NT, GROUP, WARPS>), kMaxSmem);
    if (e != cudaSuccess) return e;
    const int per_sm = NT == 1 && smem <= kPairSmem ? 2 : 1;
    *clusters = sms * per_sm / split;
    if (split > 1) {
        static std::atomic<int> known[64][4][2];   // asked once for each device
        int dev = 0;
        e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        std::atomic<int> &slot = known[dev & 63][split == 2 ? 1 : split == 4 ? 2 : 3][per_sm - 1];
        int most = slot.load(std::memory_order_relaxed);
        if (most == 0) {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr;
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = (unsigned)split;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.gridDim = dim3((unsigned)split);
            cfg.blockDim = dim3(WARPS * 32);
            cfg.dynamicSmemBytes = smem;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&most, w4_linear_kernel<NT, GROUP, WARPS>, &cfg);
            if (e != cudaSuccess) return e;
            if (most > 0 && dev < 64) slot.store(most, std::memory_order_relaxed);
        }
        if (most > 0 && *clusters > most) *clusters = most;
    }
    if (*clusters < 1) *clusters = 1;
    return cudaSuccess;
}

template <int NT, int GROUP, int WARPS>
cudaError_t launch_w4(W4Args a, int split, int clusters, int blocks_m, size_t smem, cudaStream_t st) {
    a.tiles = (a.N + 2 * WARPS * split - 1) / (2 * WARPS * split);
    if (clusters > a.tiles) clusters = a.tiles;
    return launch_kernel(w4_linear_kernel<NT, GROUP, WARPS>, dim3((unsigned)(clusters * split), (unsigned)blocks_m), dim3(WARPS * 32),
                         smem, st, split, true, a);
}

template <int NT, int GROUP>
cudaError_t launch_w4_warps(const W4Args &a, int split, int blocks_m, int sms, cudaStream_t st) {
    const int m = a.M < NT * 8 ? a.M : NT * 8;
    const size_t smem = w4_smem(NT, m, a.part, GROUP, split, 8);
    int clusters = 0;
    cudaError_t e = resident_clusters<NT, GROUP, 8>(split, smem, sms, &clusters);
    if (e != cudaSuccess) return e;
    if constexpr (NT == 2) {
        // With a CTA an SM the warps wait more than they issue: a tile of twelve warps takes less than 4 / 3
        // of the time of one of eight.  Twelve where that saves more rounds than it lengthens: 13 x 17408 x
        // 5120, three rounds of eight take 32.1 us, two of twelve 29.7.
        const size_t smem12 = w4_smem(NT, m, a.part, GROUP, split, 12);
        if (split > 1 && smem12 <= kMaxSmem) {
            int clusters12 = 0;
            e = resident_clusters<NT, GROUP, 12>(split, smem12, sms, &clusters12);
            if (e != cudaSuccess) return e;
            const auto rounds = [&](int warps, int at_once) {
                const int tiles = (a.N + 2 * warps * split - 1) / (2 * warps * split);
                return (tiles + at_once - 1) / at_once;
            };
            if (rounds(12, clusters12) * 4 < rounds(8, clusters) * 3 + 1)
                return launch_w4<NT, GROUP, 12>(a, split, clusters12, blocks_m, smem12, st);
        }
    }
    return launch_w4<NT, GROUP, 8>(a, split, clusters, blocks_m, smem, st);
}

template <int NT>
cudaError_t launch_w4_group(const W4Args &a, int group, int split, int blocks_m, int sms, cudaStream_t st) {
    switch (group) {
        case 32: return launch_w4_warps<NT, 32>(a, split, blocks_m, sms, st);
        case 64: return launch_w4_warps<NT, 64>(a, split, blocks_m, sms, st);
        default: return launch_w4_warps<NT, 128>(a, split, blocks_m, sms, st);
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
    // CTAs of a cluster: up to eight rows of x, so many that two CTAs fit into an SM with their columns of x
    // and the sums' starts (laid out for eight rows: half of one row's columns in groups of 32; 1 x 17408 x
    // 5120 takes 17.2 us so, 17.6 where the columns alone decide), and that the columns stay under 40 KB
    // (8 x 5120 x 14336: 14.5 us, 15.8 by the fit alone);
    // past that as few as it takes to fit, as larger clusters leave more SMs without work
    const auto x_bytes = [&](int64_t m, int split) { return m * (kParts / split * part * kBlockK * 2 + 64); };
    const auto too_large = [&](int64_t m, int split) {
        return x_bytes(m, split) > 40 * 1024 || w4_smem(1, m, part, group, split, 8) > kPairSmem;
    };
    const int64_t block_m = M > 8 && x_bytes(M < 16 ? M : 16, kParts) <= 120 * 1024 ? 16 : 8;
    const int64_t m = M < block_m ? M : block_m;
    int split = 1;
    while (split < kParts && (block_m == 8 ? too_large(m, split) : w4_smem(2, m, part, group, split, 8) > kMaxSmem)) split *= 2;
    W4Args a;
    a.x = static_cast<const uint16_t *>(x);
    a.ldx = ldx;
    a.qw = static_cast<const uint8_t *>(qw);
    a.sw = static_cast<const uint16_t *>(sw);
    a.bias = static_cast<const uint16_t *>(bias);
    a.y = static_cast<uint16_t *>(y);
    a.ldy = ldy;
    a.N = (int)N;
    a.K = (int)K;
    a.kb = kb;
    a.part = part;
    a.split_log2 = split == 1 ? 0 : split == 2 ? 1 : split == 4 ? 2 : 3;
    a.tiles = 0;      // by the number of warps
    sms = internal_launch_sms(sms);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // (a grid has up to 65,535 blocks of rows)
    cudaError_t e = cudaSuccess;
    for (int64_t left = M; left > 0 && e == cudaSuccess; left -= a.M) {
        a.M = (int)(left < 65535 * block_m ? left : 65535 * block_m);
        const int blocks_m = (int)((a.M + block_m - 1) / block_m);
        e = block_m == 8 ? launch_w4_group<1>(a, group, split, blocks_m, sms, st)
                         : launch_w4_group<2>(a, group, split, blocks_m, sms, st);
        a.x += a.M * ldx;
        a.y += a.M * ldy;
    }
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "4-bit linear launch");
}
