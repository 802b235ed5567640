// fp8_block.cu -- linears over e4m3 codes with a scale for each block of 128
// of K (activations) or 128 x 128 (weights):
//
//   y[m][n] = sum_b sx[m][b] sw[n / 128][b] * (sum_{k in block b} qx[m][k] qw[n][k])
//
// The tensor cores (tcgen05 kind::f8f6f4, fp32 accumulators in TMEM) sum one
// block of 128 of K at a time, which is one k-block of 128 bytes in the 128-byte
// swizzle; the scales differ from block to block, so each block's sums are read
// back (tcgen05.ld) and added, scaled, to fp32 totals in registers while the
// tensor core sums the next block into another TMEM buffer.
//
// Two kernels:
//  wide  many rows.  A cluster of two CTAs (cta_group::2) owns a tile of 256
//        rows by 256 columns (128 gate and the 128 matching up columns); each CTA
//        stages its 128 rows and half of the weight rows of a k-block (32 KB) in
//        a ring.  A TMEM lane is a row of x, so a thread's scale is its row's times
//        one of the weight's, the same for its 128 columns.  Persistent over tiles, in
//        bands of rows that stay in L2; a tile leaves through shared memory and TMA.
//        24,032 x 5,120 x 6,144: 496 us, 3,050 TFLOP/s, ten calls in a row (557 for a second, under
//        the power cap); 1,502 x 5,120 x 17,408 gate/up 200 us (215).  MMAs that are not read back take
//        406 and 154 us (462 and 173; operands' shared-memory traffic: 64 KB a k-block and SM), the
//        per-row linears of gemm.cu 430 and 170 (486 and 185); the rest is a tile's end
//        (about 3,000 clocks of 30,000, two k-blocks of which are hidden) and the way from
//        an MMA's end over both CTAs' reading back to the MMA that reuses the buffer
//        (about 1,300 clocks, 1,000 of them hidden).  What was tried: sixteen warps
//        that read back (8% slower: the fixed part of a k-block, some 80 instructions, counts
//        for each), halves of a buffer with MMAs of 128 columns (45% slower: A is
//        read twice from shared memory), scales by 16-byte loads (no gain).
//        Where tiles are few, two or four pairs share one, each with a part of K; each takes
//        a part of its columns to the end with the sums that the others write into its shared
//        memory (1,502 x 5,120 x 1,024: 20.5 to 16.5 us, 1,024 x 17,408 x 2,048: 54 to 35; sums that
//        each leaves in its own memory for the others to read: 1 us slower).
//  few   few rows, bound by the weight's bytes; operands change places.  A CTA
//        owns 128 rows of the weight (TMEM lanes) and 16 to 128 rows of x
//        (columns), so that the weight streams through rings of about 200 KB a SM; K
//        is cut among the CTAs of a cluster where the weight's tiles alone leave SMs
//        without work, and their sums meet through distributed shared memory, always
//        in the same order.  1 x 5,120 x 17,408 gate/up: 28.9 us (178 MB, 6.2 TB/s); 13 x
//        17,408 x 5,120: 19.1 us (89 MB; 2.5 us are a launch's, the bytes alone take 14 at
//        the 6.4 TB/s of a long call).  Copies of later k-blocks into L2 ahead of the
//        ring: 20% slower; MMAs of two k-blocks side by side: no gain.
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

struct BlockArgs {
    int M, N, nkb;            // rows, columns of the output, k-blocks
    const float *sx, *sw;     // [M][nkb], [weight rows / 128][nkb]
    const uint16_t *bias;     // of the weight's rows, or null
    uint16_t *out;
    int64_t ldo;
    int band;                 // wide: tiles of rows a band
    int split;                // few: CTAs that share a tile's K
    bool whole;               // wide: the output's rows start on 32 bytes
    int tiles_m;              // few: tiles of rows
    unsigned int *status;
    uint64_t limit_ns;
    int force_timeout;
};

__device__ __forceinline__ uint64_t pack_f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t pack_u2(uint32_t a, uint32_t b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ void unpack_f2(uint64_t p, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p));
}
__device__ __forceinline__ uint64_t fma_f2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

__device__ __forceinline__ uint64_t mul_f2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add_f2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// g / (1 + e^-g) u of two values, as (g / 4) u / (1/4 + 2^(-g log2 e - 2)): the divisor is below 2^126, where the
// reciprocal underflows, for every e^-g that fp32 holds, so that none has to be looked at and scaled
// (1,502 x 5,120 x 17,408, ten calls in a row: 4 us of 200; 8 more without a silu, whose exponentials and reciprocals are what a tile
// waits for).
__device__ __forceinline__ uint64_t silu_mul2(uint64_t g, uint64_t u) {
    constexpr float kLog2E = 1.44269504088896341f;
    float a, b;
    unpack_f2(fma_f2(g, pack_f2(-kLog2E, -kLog2E), pack_f2(-2.0f, -2.0f)), a, b);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
    unpack_f2(add_f2(pack_f2(a, b), pack_f2(0.25f, 0.25f)), a, b);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
    return mul_f2(mul_f2(mul_f2(g, pack_f2(0.25f, 0.25f)), pack_f2(a, b)), u);
}

constexpr unsigned kWarp = 0xFFFFFFFFu;

// Waits of a whole warp.  Each lane polls for itself, so that where a wait runs out some lanes may see the phase complete
// and others give up; the instructions around (elect.sync, TMEM loads, cluster barriers) want them together.  So no lane
// leaves a loop on its own answer: it keeps it (`ok`, false from then on), the elected lane issues while its own holds,
// sums of the others go on and are not used, and a tile's end votes.  (24,032 x 5,120 x 6,144 and 1,502 x 5,120 x 17,408
// gate/up within 0.5% of lanes that leave, few rows 0.1 us slower; a vote beside each wait costs 2-3% of both.)

// mbar_wait for lanes that stay: once a wait of this CTA has run out no further one is sat through.
__device__ __forceinline__ bool stay_wait(uint64_t *bar, uint32_t parity, const WaitCtx &w, unsigned int site) {
    return mbar_try_wait(smem_u32(bar), parity) || (!*w.abort && mbar_wait(bar, parity, w, site));
}

// One lane of a whole warp.  The warps that issue copies and MMAs run with all lanes and elect one for each k-block:
// what they count then stays in uniform registers, which those instructions take their operands from.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Whether the phase has completed, without waiting for it.  The MMA issuers ask for the next k-block's barriers before
// they issue a k-block's MMAs: a wait takes some 60 clocks even where there is nothing to wait for.
__device__ __forceinline__ bool mbar_done(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// Waits for this thread's TMEM loads; the registers are operands, so that no use of them moves before it.
__device__ __forceinline__ void tmem_ready(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                   "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
                 :: "memory");
}
__device__ __forceinline__ void tmem_ready(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
                 :: "memory");
}

__device__ __forceinline__ float bf16_at(const uint16_t *p) { return __uint_as_float((uint32_t)__ldg(p) << 16); }

// Copies of tiles from shared memory, and the waits for them.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap *m, const void *src, int32_t c0, int32_t c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(src)), "r"(c0), "r"(c1) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read_all() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

// An address in the same shared memory of another CTA of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t local, int rank) {
    uint32_t at;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(local), "r"(rank));
    return at;
}
__device__ __forceinline__ float ld_cluster(uint32_t at) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void st_cluster(uint32_t at, uint64_t a, uint64_t b) {
    asm volatile("st.shared::cluster.v2.b64 [%0], {%1, %2};" ::"r"(at), "l"(a), "l"(b) : "memory");
}

// ------------------------------------------------------------ many rows

constexpr int kBoxBytes = 128 * 128;         // 128 rows of a k-block
constexpr int kWideStage = 2 * kBoxBytes;    // rows of x, then of the weight
constexpr int kMaxWideStages = 6;
constexpr int kWideEpi = 8;                  // warps that read TMEM back
constexpr int kParts = kWideEpi / 4, kSums = 256 / kParts;    // of a row, and columns that each holds
constexpr int kWideThreads = 128 + 32 * kWideEpi;
constexpr int kOutBox = 32 * 128;            // 32 rows of 64 columns of the output, bf16
template <bool GU, int S>
struct Wide {
    static constexpr int kBoxes = GU ? 1 : 2;                    // of 64 columns of the output a warp
    static constexpr int kMine = kSums / S;                      // sums of a thread that it brings to their end
    // what leaves through shared memory, or the other pairs' sums
    static constexpr int kOut = S == 1 ? kWideEpi * kBoxes * kOutBox : (S - 1) * kWideEpi * 32 * kMine * 4;
    static constexpr int kStages = S == 1 ? (GU ? 6 : 5) : S == 2 ? 5 : 4;
    static constexpr int kSmem = kStages * kWideStage + kOut + 1024 + 512;
    static_assert(kSmem <= 232448, "shared memory");
};

struct WideBars {
    uint64_t full[kMaxWideStages];
    uint64_t done[kMaxWideStages];      // a k-block's MMAs: its stage is free, its sums are complete
    uint64_t acc_empty[2];
    uint64_t drain, never;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(WideBars) <= 512, "barrier block");

struct WideTile {
    int mb, nb;
};

// Tile t in bands of `band` tiles of rows: all columns of a band, its rows fastest.
__device__ __forceinline__ WideTile wide_tile(int t, int num_m, int num_n, int band) {
    const int b = t / (band * num_n), m0 = b * band, rows = min(band, num_m - m0), i = t - b * band * num_n;
    return {m0 + i % rows, i / rows};
}

// As mma2_commit_both, for the pair of CTAs from rank `first` on of a larger cluster.
__device__ __forceinline__ void commit_pair(uint64_t *bar, uint32_t first) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(smem_u32(bar)), "h"((uint16_t)(3u << first)) : "memory");
}

// S > 1: a cluster is S pairs that share a tile, each with a part of K.  A pair takes a part of the columns to their end: the
// others leave their sums of these in its shared memory, and it adds them to its own, always in the same order.
template <bool GU, int S>
__global__ void __launch_bounds__(kWideThreads, 1)
wide_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmw,
            const __grid_constant__ CUtensorMap tmo, const BlockArgs a) {
    using W = Wide<GU, S>;
    constexpr bool SPLIT = S > 1;
    constexpr int kWideStages = W::kStages;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((base + 1023u) & ~1023u) - base);
    WideBars *bar = reinterpret_cast<WideBars *>(smem + kWideStages * kWideStage + W::kOut);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t place = cluster_rank(), rank = SPLIT ? place & 1u : place, first = SPLIT ? place & ~1u : 0u;
    const auto leader = [&](const void *p) { return SPLIT ? cluster_addr(smem_u32(p), (int)first) : leader_addr(p); };
    constexpr int kCols = GU ? 128 : 256;     // columns of the output a tile

    if (threadIdx.x == 0) {
        for (int s = 0; s < kWideStages; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->done[s], 1);
        }
        for (int s = 0; s < 2; ++s) mbar_init(&bar->acc_empty[s], 2 * kWideEpi);
        mbar_init(&bar->drain, 1);
        mbar_init(&bar->never, 1);
        bar->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmx);
        tma_prefetch_desc(&tmw);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&bar->tmem)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    pdl_wait();

    const uint32_t own_tmem = bar->tmem;
    uint32_t tmem;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(tmem) : "r"(leader(&bar->tmem)));
    const int slot = (int)blockIdx.x / (2 * S), slots = (int)gridDim.x / (2 * S);
    const int num_m = (a.M + 255) / 256, num_n = (a.N + kCols - 1) / kCols, tiles = num_m * num_n, nkb = a.nkb;
    const int share = (int)(place >> 1), k0 = SPLIT ? share * nkb / S : 0, k1 = SPLIT ? (share + 1) * nkb / S : nkb;
    // Where a tile's sums meet: all warps come by twice, before they are read and, where another tile's follow, after.
    const auto meet = [&](int t) {
        __syncwarp();
        cluster_sync();
        if (t + slots < tiles) cluster_sync();
    };
    const WaitCtx w{a.limit_ns, &bar->abort, a.status};

    // 4 x 32 x 56 + 8 x 32 x 224 registers of the 384 x 168 launched
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == 0) {
            uint32_t s = 0, ph = 0, filled = 0, last = 0;
            bool ok = true;
            for (int t = slot; t < tiles && (SPLIT || ok); t += slots) {
                const WideTile o = wide_tile(t, num_m, num_n, a.band);
                const int row = o.mb * 256 + (int)rank * 128;
                const int wrow = GU ? (rank ? a.N : 0) + o.nb * 128 : o.nb * 256 + (int)rank * 128;
                for (int kb = k0; kb < k1; ++kb) {
                    ok = ok && mbar_wait(&bar->done[s], ph ^ 1u, w, kSiteTmaEmpty);
                    uint8_t *st = smem + s * kWideStage;
                    const uint32_t full = leader(&bar->full[s]);
                    if (elect_one() && ok) {
                        if (rank == 0) mbar_arrive_expect_tx(&bar->full[s], 2 * kWideStage);
                        tma_load_2d_pair(st, &tmx, kb * 128, row, full);
                        tma_load_2d_pair(st + kBoxBytes, &tmw, kb * 128, wrow, full);
                    }
                    __syncwarp();
                    if (ok) {
                        filled |= 1u << s;
                        last = (last & ~(1u << s)) | ph << s;
                    }
                    if (++s == kWideStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                }
                if (SPLIT) meet(t);
                else ok = __all_sync(kWarp, ok);
            }
            // every copy of the pair has landed (they are counted on the leader's barriers) before a CTA ends
            if (rank == 0)
                for (int i = 0; i < kWideStages; ++i)
                    if (filled >> i & 1u) mbar_wait_drain(&bar->full[i], last >> i & 1u, 200000000ull, a.status);
        } else if (warp == 1 && rank == 0) {
            constexpr uint32_t idesc = idesc_f32acc(0, 0, 256, 256);
            const bool forced = a.force_timeout == 1 || (a.force_timeout >= 2 && a.force_timeout - 2 == slot);
            if (forced) warp_wait(&bar->never, 0, w, kSiteMmaFull);
            if (SPLIT || !forced) {
                uint32_t s = 0, ph = 0, acc = 0, aph = 0;
                const int64_t steps = SPLIT ? k1 - k0 : (int64_t)((tiles - 1 - slot) / slots + 1) * nkb;
                bool ready = false, ok = !forced;
                for (int t = slot; t < (SPLIT ? tiles : slot + 1); t += SPLIT ? slots : 1) {
                    for (int64_t i = 0; i < steps; ++i) {
                        // (the buffer comes back last)
                        ok = ok && (ready || (mbar_wait(&bar->full[s], ph, w, kSiteMmaFull) &&
                                              mbar_wait(&bar->acc_empty[acc], aph ^ 1u, w, kSiteMmaAccEmpty)));
                        tc_fence_after();
                        const uint32_t sa = smem_u32(smem + s * kWideStage), d = tmem + acc * 256, s0 = s;
                        const uint64_t da = sdesc_sw128(sa), db = sdesc_sw128(sa + kBoxBytes);
                        if (++s == kWideStages) {
                            s = 0;
                            ph ^= 1u;
                        }
                        acc ^= 1u;
                        if (!acc) aph ^= 1u;
                        const bool e0 = mbar_done(&bar->acc_empty[acc], aph ^ 1u), e1 = mbar_done(&bar->full[s], ph);
                        if (elect_one() && ok) {
#pragma unroll
                            for (int k = 0; k < 4; ++k) mma2_f8(d, da + 2 * k, db + 2 * k, idesc, k > 0);
                            if (SPLIT) commit_pair(&bar->done[s0], first);
                            else mma2_commit_both(&bar->done[s0]);
                        }
                        __syncwarp();
                        ready = e0 && e1;
                    }
                    if (SPLIT) meet(t);
                }
            }
            if (elect_one()) mma2_commit_local(&bar->drain);
            __syncwarp();
            mbar_wait_drain(&bar->drain, 0, 200000000ull, a.status);
        } else if (SPLIT) {
            for (int t = slot; t < tiles; t += slots) meet(t);
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        const int quad = warp & 3, part = (warp - 4) >> 2;
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        // TMEM column of this warp's piece j of 32: consecutive ones of the tile, or first gate's, then up's
        constexpr int kPieces = kSums / 32;
        const auto piece = [&](int j) {
            return GU ? (j / (kPieces / 2)) * 128 + part * (kSums / 2) + (j % (kPieces / 2)) * 32 : part * kSums + 32 * j;
        };
        uint8_t *box0 = smem + kWideStages * kWideStage, *box = box0 + (warp - 4) * W::kBoxes * kOutBox;
        uint32_t acc = 0, s = 0, ph = 0;
        bool ok = true;
        int row = 0, n0 = 0;
        const float *sx, *sw0, *sw1;
        float x, w0, w1;
        // where a tile's rows, columns and scales are, and its first scales
        const auto enter = [&](int t) {
            const WideTile o = wide_tile(t, num_m, num_n, a.band);
            row = o.mb * 256 + (int)rank * 128 + quad * 32;
            n0 = o.nb * kCols + part * (kCols / kParts);
            sx = a.sx + (int64_t)min(row + lane, a.M - 1) * nkb;
            sw0 = a.sw + (int64_t)(GU ? o.nb : min(n0 / 128, (a.N - 1) / 128)) * nkb;
            sw1 = GU ? sw0 + (int64_t)(a.N / 128) * nkb : sw0;
            x = __ldg(sx + k0);
            w0 = __ldg(sw0 + k0);
            w1 = GU ? __ldg(sw1 + k0) : 0.0f;
        };
        if (slot < tiles) enter(slot);
        for (int t = slot; t < tiles && (SPLIT || ok); t += slots) {
            uint64_t sum[kSums / 2];
#pragma unroll
            for (int i = 0; i < kSums / 2; ++i) sum[i] = 0;
            for (int kb = k0; kb < k1; ++kb) {
                const float f0 = x * w0, f1 = GU ? x * w1 : f0;
                const int next = min(kb + 1, k1 - 1);      // its scales are on their way meanwhile
                x = __ldg(sx + next);
                w0 = __ldg(sw0 + next);
                if (GU) w1 = __ldg(sw1 + next);
                if (!stay_wait(&bar->done[s], ph, w, kSiteEpiAccFull)) ok = false;
                tc_fence_after();
                const uint32_t at = tmem + acc * 256 + lanes;
                constexpr int kAtOnce = kPieces / 2;
                uint32_t r[kAtOnce][32];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int q = 0; q < kAtOnce; ++q) tmem_ld32(at + piece(kAtOnce * h + q), r[q]);
#pragma unroll
                    for (int q = 0; q < kAtOnce; ++q) tmem_ready(r[q]);
                    if (h == 1) {
                        // the last pieces are in registers: the buffer goes back.  (Relaxed: the values read
                        // are held, nothing else passes between the two.)
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0 && ok) arrive_cluster_relaxed(leader(&bar->acc_empty[acc]));
                    }
                    const float f = (GU && h) ? f1 : f0;
                    const uint64_t ff = pack_f2(f, f);
#pragma unroll
                    for (int q = 0; q < kAtOnce; ++q)
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            uint64_t &o2 = sum[16 * (kAtOnce * h + q) + i];
                            o2 = fma_f2(ff, pack_u2(r[q][2 * i], r[q][2 * i + 1]), o2);
                        }
                }
                acc ^= 1u;
                if (++s == kWideStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
            if constexpr (SPLIT) {
                constexpr int kMine = W::kMine, kUnits = kMine / 4, kCount = GU ? kMine / 2 : kMine;
                // unit u of four columns of pair j's: consecutive ones, or first gate's, then up's
                const auto unit = [&](int j, int u) {
                    return GU ? (u / (kUnits / 2)) * (kSums / 2) + j * (kMine / 2) + u % (kUnits / 2) * 4 : j * kMine + 4 * u;
                };
                const int share = (int)(cluster_rank() >> 1), rank = (int)(cluster_rank() & 1u);   // (read again: no registers to spare)
                const uint32_t in = smem_u32(box0) + (uint32_t)((warp - 4) * kUnits * 512 + lane * 16);
#pragma unroll
                for (int j = 0; j < S; ++j)
                    if (j != share && ok) {
                        const uint32_t to = cluster_addr(in + (uint32_t)((share - (share > j)) * kWideEpi * kUnits * 512), 2 * j + (int)rank);
#pragma unroll
                        for (int u = 0; u < kUnits; ++u) st_cluster(to + u * 512, sum[unit(j, u) / 2], sum[unit(j, u) / 2 + 1]);
                    }
                __syncwarp();
                cluster_sync();
                // (the sums stay in their registers: a copy of this for each pair)
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    if (j != share || bar->abort) continue;
#pragma unroll
                    for (int q = 0; q < S - 1; ++q)
#pragma unroll
                        for (int u = 0; u < kUnits; ++u) {
                            uint64_t v0, v1;
                            asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v0), "=l"(v1) : "r"(in + (q * kWideEpi * kUnits + u) * 512) : "memory");
                            uint64_t &o0 = sum[unit(j, u) / 2], &o1 = sum[unit(j, u) / 2 + 1];
                            o0 = add_f2(o0, v0);
                            o1 = add_f2(o1, v1);
                        }
                    const int m = row + lane, n = n0 + j * kCount;
                    // the sums of two columns from c on: consecutive ones, or of the gate and, kSums / 2 on, of up
                    const auto at = [&](int c) -> uint64_t & { return sum[(j * kCount + c) / 2]; };
                    if (a.bias) {
#pragma unroll
                        for (int c = 0; c < kCount; c += 2)
                            if (n + c < a.N) {
                                const uint32_t *b = reinterpret_cast<const uint32_t *>(a.bias + n + c);
                                uint32_t bb = __ldg(b);
                                at(c) = add_f2(at(c), pack_f2(__uint_as_float(bb << 16), __uint_as_float(bb & 0xFFFF0000u)));
                                if (GU) {
                                    bb = __ldg(b + a.N / 2);
                                    at(c + kSums / 2) = add_f2(at(c + kSums / 2), pack_f2(__uint_as_float(bb << 16), __uint_as_float(bb & 0xFFFF0000u)));
                                }
                            }
                    }
                    if (m < a.M) {
                        uint16_t *y = a.out + (int64_t)m * a.ldo + n;
#pragma unroll
                        for (int c = 0; c < kCount; c += 16) {
                            uint32_t p[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                float v0, v1;
                                unpack_f2(GU ? silu_mul2(at(c + 2 * i), at((GU ? kSums / 2 : 0) + c + 2 * i)) : at(c + 2 * i), v0, v1);
                                p[i] = pack_bf16x2(v0, v1);
                            }
                            if (a.whole && n + c + 16 <= a.N) {
                                asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                                             ::"l"(y + c), "r"(p[0]), "r"(p[1]), "r"(p[2]), "r"(p[3]), "r"(p[4]), "r"(p[5]), "r"(p[6]), "r"(p[7])
                                             : "memory");
                            } else {
                                if (n + c < a.N) *reinterpret_cast<uint4 *>(y + c) = make_uint4(p[0], p[1], p[2], p[3]);
                                if (n + c + 8 < a.N) *reinterpret_cast<uint4 *>(y + c + 8) = make_uint4(p[4], p[5], p[6], p[7]);
                            }
                        }
                    }
                }
                if (t + slots < tiles) {
                    enter(t + slots);
                    __syncwarp();
                    cluster_sync();
                }
                continue;
            }
            if (!(ok = __all_sync(kWarp, ok))) break;
            const int trow = row, tn = n0;
            if (t + slots < tiles) enter(t + slots);
            if (a.bias) {
#pragma unroll
                for (int c = 0; c < kSums; c += 2) {
                    const int n = tn + (GU ? c % (kSums / 2) : c);
                    if (n < a.N) {
                        const uint32_t bb = __ldg(reinterpret_cast<const uint32_t *>(a.bias + (GU && c >= kSums / 2 ? a.N : 0) + n));
                        float v0, v1;
                        unpack_f2(sum[c / 2], v0, v1);
                        sum[c / 2] = pack_f2(v0 + __uint_as_float(bb << 16), v1 + __uint_as_float(bb & 0xFFFF0000u));
                    }
                }
            }
            // through shared memory, 64 columns a box: 16-byte units swizzled as the copy expects them
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
#pragma unroll
            for (int b = 0; b < W::kBoxes; ++b)
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    uint32_t p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float v0, v1;
                        const int c = 64 * b + 8 * q + 2 * i;
                        unpack_f2(GU ? silu_mul2(sum[c / 2], sum[(GU ? kSums / 4 : 0) + c / 2]) : sum[c / 2], v0, v1);
                        p[i] = pack_bf16x2(v0, v1);
                    }
                    *reinterpret_cast<uint4 *>(box + b * kOutBox + lane * 128 + ((q ^ (lane & 7)) << 4)) =
                        make_uint4(p[0], p[1], p[2], p[3]);
                }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0 && trow < a.M) {
#pragma unroll
                for (int b = 0; b < W::kBoxes; ++b)
                    if (tn + 64 * b < a.N) tma_store_2d(&tmo, box + b * kOutBox, tn + 64 * b, trow);
                bulk_commit();
            }
        }
        if (lane == 0) bulk_wait_all();     // the copies have read the boxes before the CTA ends
    }
    __syncwarp();
    pdl_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (bar->abort) {   // copies that still signal the other CTA land first
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 2000000ull) {
        }
    }
    cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(own_tmem), "r"(512) : "memory");
    }
}

// ------------------------------------------------------------ few rows

constexpr int kMaxStages = 12, kMaxSplit = 8, kMaxBufs = 8;

template <int T, bool GU>
struct Few {
    // The warps that read TMEM back: a k-block takes four (of 32 weight rows each), or eight that share the rows
    // of x where one thread cannot hold them all.  For fewer rows a k-block's copy arrives in less time than
    // one group of warps takes for it, so that `kSets` groups take k-blocks in turn.
    static constexpr int kHalves = T == 128 ? 2 : 1;
    static constexpr int kSets = T <= 32 || (T == 64 && !GU) ? 2 : 1;
    static constexpr int kPerSm = T <= 32 && !GU ? 2 : 1;      // CTAs an SM
    static constexpr int kEpi = 4 * kHalves * kSets;
    static constexpr int kCols = T / kHalves;                  // rows of x a warp holds
    static constexpr int kTiles = GU ? 2 : 1;                  // weight tiles: gate, up
    static constexpr int kStage = kTiles * kBoxBytes + T * 128;
    static constexpr int kAcc = kTiles * T;                    // TMEM columns of a buffer
    static constexpr int kBufs = 512 / kPerSm / kAcc >= kMaxBufs ? kMaxBufs : 512 / kPerSm / kAcc;
    static constexpr int kTmem = kBufs * kAcc;
    static constexpr int kScales = kEpi * 2 * kTiles * kCols;  // floats
    static constexpr int kRest = 1024 + 512 + kScales * 4;
    static constexpr int kFit = ((kPerSm == 2 ? 115712 : 232448) - kRest) / kStage;
    static constexpr int kStages = kFit > kMaxStages ? kMaxStages : kFit;
    static constexpr int kSmem = kStages * kStage + kRest;
    static constexpr int kThreads = 64 + 32 * kEpi;
    static_assert(kTmem >= 32 && kTmem <= 512 && (kTmem & (kTmem - 1)) == 0, "TMEM columns");
    static_assert(kStages >= 3 && kBufs >= 2 && kBufs % kSets == 0, "stages, buffers");
    static_assert(kSets * kTiles * T * 512 <= kStages * kStage, "the sums of the groups fit in the ring");
};

struct FewBars {
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[kMaxBufs], acc_empty[kMaxBufs];
    uint64_t drain, never;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(FewBars) <= 512, "barrier block");

template <int T, bool GU>
__global__ void __launch_bounds__(Few<T, GU>::kThreads, Few<T, GU>::kPerSm)
few_kernel(const __grid_constant__ CUtensorMap tmx, const __grid_constant__ CUtensorMap tmw, const BlockArgs a) {
    using F = Few<T, GU>;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t base = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + (((base + 1023u) & ~1023u) - base);
    FewBars *bar = reinterpret_cast<FewBars *>(smem + F::kStages * F::kStage);
    float *scales = reinterpret_cast<float *>(smem + F::kStages * F::kStage + 512);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < F::kStages; ++s) {
            mbar_init(&bar->full[s], 1);
            mbar_init(&bar->empty[s], 1);
        }
        for (int s = 0; s < F::kBufs; ++s) {
            mbar_init(&bar->acc_full[s], 1);
            mbar_init(&bar->acc_empty[s], 4 * F::kHalves);
        }
        mbar_init(&bar->drain, 1);
        mbar_init(&bar->never, 1);
        bar->abort = 0;
        fence_barrier_init();
        tma_prefetch_desc(&tmx);
        tma_prefetch_desc(&tmw);
    }
    if (warp == 1) {
        tmem_alloc(&bar->tmem, F::kTmem);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();

    const uint32_t tmem = bar->tmem;
    const int split = a.split, rank = split > 1 ? (int)cluster_rank() : 0;
    const int k0 = rank * a.nkb / split, k1 = (rank + 1) * a.nkb / split;      // (at most 8 times 512)
    const int tiles = (a.N + 127) / 128 * a.tiles_m, clusters = (int)gridDim.x / split;
    const WaitCtx w{a.limit_ns, &bar->abort, a.status};
    // Under a budget of SMs a cluster takes one tile after another; otherwise there is a cluster for each.  The
    // rings go on where they are: s, ph of the stages, and `done` k-blocks of the TMEM buffers before this tile.
    uint32_t s = 0, ph = 0, done = 0, filled = 0, last = 0;
    bool ok = true;

    for (int both = (int)blockIdx.x / split; both < tiles; both += clusters, done += (uint32_t)(k1 - k0)) {
        // tiles of one part of the weight side by side, so that it is read from memory once
        const int tile = both / a.tiles_m, n0 = tile * 128, m0 = (both - tile * a.tiles_m) * T;
        if (warp == 0) {
            for (int kb = k0; kb < k1; ++kb) {
                ok = ok && mbar_wait(&bar->empty[s], ph ^ 1u, w, kSiteTmaEmpty);
                uint8_t *st = smem + s * F::kStage;
                if (elect_one() && ok) {
                    mbar_arrive_expect_tx(&bar->full[s], F::kStage);
                    tma_load_2d(st, &tmw, kb * 128, n0, &bar->full[s]);
                    if (GU) tma_load_2d(st + kBoxBytes, &tmw, kb * 128, a.N + n0, &bar->full[s]);
                    tma_load_2d(st + F::kTiles * kBoxBytes, &tmx, kb * 128, m0, &bar->full[s]);
                }
                __syncwarp();
                if (ok) {
                    filled |= 1u << s;
                    last = (last & ~(1u << s)) | ph << s;
                }
                if (++s == F::kStages) {
                    s = 0;
                    ph ^= 1u;
                }
            }
        } else if (warp == 1) {
            constexpr uint32_t idesc = idesc_f32acc(0, 0, 128, T);
            if (a.force_timeout == 1 || (a.force_timeout >= 2 && a.force_timeout - 2 == (int)blockIdx.x)) {
                warp_wait(&bar->never, 0, w, kSiteMmaFull);
            } else {
                bool ready = false;
                for (uint32_t g = done; g != done + (uint32_t)(k1 - k0); ++g) {
                    const uint32_t acc = g % F::kBufs, s0 = s;
                    ok = ok && (ready || (mbar_wait(&bar->full[s], ph, w, kSiteMmaFull) &&
                                          mbar_wait(&bar->acc_empty[acc], (g / F::kBufs & 1u) ^ 1u, w, kSiteMmaAccEmpty)));
                    tc_fence_after();
                    const uint32_t sa = smem_u32(smem + s * F::kStage), d = tmem + acc * F::kAcc;
                    const uint64_t da = sdesc_sw128(sa), db = sdesc_sw128(sa + F::kTiles * kBoxBytes);
                    if (++s == F::kStages) {
                        s = 0;
                        ph ^= 1u;
                    }
                    const bool e0 = mbar_done(&bar->acc_empty[(g + 1) % F::kBufs], ((g + 1) / F::kBufs & 1u) ^ 1u);
                    const bool e1 = mbar_done(&bar->full[s], ph);
                    if (elect_one() && ok) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
#pragma unroll
                            for (int h = 0; h < F::kTiles; ++h)
                                mma_f8(d + h * T, da + 2 * k + h * (kBoxBytes >> 4), db + 2 * k, idesc, k > 0);
                        mma_commit(&bar->acc_full[acc]);
                        mma_commit(&bar->empty[s0]);
                    }
                    __syncwarp();
                    ready = e0 && e1;
                }
            }
        } else {
            const int quad = warp & 3, e = warp - 2, set = (e >> 2) / F::kHalves, c0 = (e >> 2) % F::kHalves * F::kCols;
            const uint32_t lanes = (uint32_t)(quad * 32) << 16;
            float *mine = scales + e * 2 * F::kTiles * F::kCols;     // two buffers of this warp's products of scales
            constexpr int kPer = (F::kCols + 31) / 32;               // of them a lane
            const float *sx[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int c = 32 * i + lane, m = m0 + c0 + c;
                sx[i] = (c < F::kCols && m < a.M) ? a.sx + (int64_t)m * a.nkb : nullptr;
            }
            const float *sw0 = a.sw + (int64_t)tile * a.nkb, *sw1 = GU ? sw0 + (int64_t)(a.N / 128) * a.nkb : sw0;
            uint64_t sum[F::kTiles][F::kCols / 2];
#pragma unroll
            for (int h = 0; h < F::kTiles; ++h)
#pragma unroll
                for (int i = 0; i < F::kCols / 2; ++i) sum[h][i] = 0;
            float x[kPer], w0 = 0.0f, w1 = 0.0f;
            const auto fetch = [&](int kb) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) x[i] = sx[i] ? __ldg(sx[i] + kb) : 0.0f;
                w0 = __ldg(sw0 + kb);
                if (GU) w1 = __ldg(sw1 + kb);
            };
            if (k0 + set < k1) fetch(k0 + set);
            uint32_t flip = 0;
            for (int kb = k0 + set; kb < k1; kb += F::kSets) {
                const uint32_t g = done + (uint32_t)(kb - k0), acc = g % F::kBufs;
                float *f = mine + flip * F::kTiles * F::kCols;
                flip ^= 1u;
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (32 * i + lane < F::kCols) {
                        f[32 * i + lane] = x[i] * w0;
                        if (GU) f[F::kCols + 32 * i + lane] = x[i] * w1;
                    }
                }
                __syncwarp();
                if (kb + F::kSets < k1) fetch(kb + F::kSets);
                if (!stay_wait(&bar->acc_full[acc], g / F::kBufs & 1u, w, kSiteEpiAccFull)) ok = false;
                tc_fence_after();
                const uint32_t at = tmem + acc * F::kAcc + lanes + c0;
                constexpr int kPiece = F::kCols < 32 ? 16 : 32, kPieces = F::kTiles * F::kCols / kPiece;
                const auto load = [&](int j, uint32_t(&r)[kPiece]) {
                    const uint32_t from = at + j * kPiece / F::kCols * T + j * kPiece % F::kCols;
                    if constexpr (kPiece == 16) tmem_ld16(from, r);
                    else tmem_ld32(from, r);
                };
                uint32_t r[2][kPiece];
                load(0, r[0]);
                tmem_ready(r[0]);
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    if (j + 1 < kPieces) {
                        load(j + 1, r[(j + 1) & 1]);
                    } else {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0 && ok) mbar_arrive(&bar->acc_empty[acc]);
                    }
                    const int h = j * kPiece / F::kCols, c = j * kPiece % F::kCols;
#pragma unroll
                    for (int i = 0; i < kPiece / 4; ++i) {
                        const ulonglong2 p = *reinterpret_cast<const ulonglong2 *>(f + h * F::kCols + c + 4 * i);
                        const uint32_t *d = r[j & 1] + 4 * i;
                        uint64_t *o = &sum[h][(c + 4 * i) / 2];
                        o[0] = fma_f2(p.x, pack_u2(d[0], d[1]), o[0]);
                        o[1] = fma_f2(p.y, pack_u2(d[2], d[3]), o[1]);
                    }
                    if (j + 1 < kPieces) tmem_ready(r[(j + 1) & 1]);
                }
            }
            // The ring is free once every group has seen its last k-block complete; then each leaves its sums
            // there, [group][gate, up][row of x][weight row].
            asm volatile("bar.sync 1, %0;" ::"n"(32 * F::kEpi) : "memory");
            if (ok) {
                float *part = reinterpret_cast<float *>(smem) + set * F::kTiles * T * 128 + quad * 32 + lane;
#pragma unroll
                for (int h = 0; h < F::kTiles; ++h)
#pragma unroll
                    for (int i = 0; i < F::kCols; ++i) {
                        if (m0 + c0 + i >= a.M) break;
                        float v[2];
                        unpack_f2(sum[h][i / 2], v[0], v[1]);
                        part[(h * T + c0 + i) * 128] = v[i & 1];
                    }
            }
        }
        tc_fence_before();
        __syncthreads();
        if (split > 1) cluster_sync();
        const bool failed = bar->abort != 0;
        if (warp >= 2 && !failed) {
            // this CTA's share of the rows of x: the sums of the cluster's CTAs and their groups, always in this order
            const int i = threadIdx.x - 64, n = n0 + (i & 127);
            const float b0 = a.bias && n < a.N ? bf16_at(a.bias + n) : 0.0f;
            const float b1 = GU && a.bias && n < a.N ? bf16_at(a.bias + a.N + n) : 0.0f;
            for (int c = rank + split * (i >> 7); c < T && m0 + c < a.M; c += split * (F::kEpi / 4)) {
                float v = 0.0f, u = 0.0f;
                const uint32_t local = base + (uint32_t)(smem - smem_raw) + (uint32_t)((c * 128 + (i & 127)) * 4);
                for (int q = 0; q < split; ++q) {
                    const uint32_t at = split > 1 ? cluster_addr(local, q) : local;
#pragma unroll
                    for (int g = 0; g < F::kSets; ++g) {
                        v += ld_cluster(at + g * F::kTiles * T * 512);
                        if (GU) u += ld_cluster(at + (g * F::kTiles + 1) * T * 512);
                    }
                }
                v += b0;
                if (GU) v = silu_mul_fast(v, u + b1);
                if (n < a.N) a.out[(int64_t)(m0 + c) * a.ldo + n] = __bfloat16_as_ushort(__float2bfloat16_rn(v));
            }
        }
        __syncwarp();
        if (both + clusters < tiles) fence_proxy_async_smem();     // the sums, before the next tile's copies over them
        if (split > 1) cluster_sync();
        else if (both + clusters < tiles) __syncthreads();
        tc_fence_after();
    }
    // Copies and MMAs have ended before the CTA does: each has been waited for, but where a wait ran out.
    if (bar->abort) {
        if (warp == 0) {
            for (int i = 0; i < F::kStages; ++i)
                if (filled >> i & 1u) mbar_wait_drain(&bar->full[i], last >> i & 1u, 200000000ull, a.status);
        } else if (warp == 1) {
            if (elect_one()) mma_commit(&bar->drain);
            __syncwarp();
            mbar_wait_drain(&bar->drain, 0, 200000000ull, a.status);
        }
        __syncwarp();
        tc_fence_before();
        __syncthreads();
    }
    pdl_launch_dependents();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, F::kTmem);
    }
}

// ------------------------------------------------------------ launches

int maps(CUtensorMap &tx, CUtensorMap &tw, const void *qx, const void *qw, int64_t M, int64_t wrows, int64_t K, uint32_t xrows) {
    const int rc = internal_make_tmap(&tx, CU_TENSOR_MAP_DATA_TYPE_UINT8, qx, (uint64_t)K, (uint64_t)M, (uint64_t)K, 128, xrows,
                                      CU_TENSOR_MAP_SWIZZLE_128B);
    return rc ? rc : internal_make_tmap(&tw, CU_TENSOR_MAP_DATA_TYPE_UINT8, qw, (uint64_t)K, (uint64_t)wrows, (uint64_t)K, 128, 128,
                                        CU_TENSOR_MAP_SWIZZLE_128B);
}

// Clusters of `split` CTAs that a device of `all_sms` SMs holds at once where an SM holds one CTA: how many fit into its
// groups of SMs.  (Where it cannot be asked: as if any SMs could form one.)
int clusters_at_once(int split, int all_sms) {
    using F = Few<64, false>;
    static SmemOptIn opt;
    static AskedOnce<kMaxSplit + 1> known;
    int n = 0;
    const cudaError_t e = known.get(split, &n, [&](int *most) {
        auto kern = few_kernel<64, false>;
        const cudaError_t set = opt.set(reinterpret_cast<const void *>(kern), F::kSmem);
        if (set != cudaSuccess) return set;
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)split;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.gridDim = dim3((unsigned)(split * 1024), 1, 1);
        cfg.blockDim = dim3(F::kThreads, 1, 1);
        cfg.dynamicSmemBytes = F::kSmem;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        return cudaOccupancyMaxActiveClusters(most, kern, &cfg);
    });
    return e == cudaSuccess ? n : std::max(1, all_sms / split);
}

template <bool GU, int S>
int launch_wide(const void *qx, const void *qw, int64_t K, BlockArgs a, int sms, int all_sms, cudaStream_t st) {
    constexpr int kWideSmem = Wide<GU, S>::kSmem;
    static SmemOptIn opt;
    auto kern = wide_kernel<GU, S>;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(kern), kWideSmem);
    if (e != cudaSuccess) return internal_cuda_error(e, "block linear smem attribute");
    // clusters that the device holds at once, or this call's SM budget
    const int clusters = std::max(1, std::min(clusters_at_once(2 * S, all_sms), sms / (2 * S)));
    const int num_m = (a.M + 255) / 256, num_n = GU ? a.N / 128 : (a.N + 255) / 256;
    // bands whose rows of x take up to 24 MB, so that they stay in L2 while the weight passes; of even size
    const int64_t per = 256 * K, fit = std::max<int64_t>(1, ((int64_t)24 << 20) / per);
    const int bands = (int)((num_m + fit - 1) / fit);
    a.band = (num_m + bands - 1) / bands;
    a.whole = !kv_misaligned(a.out, 32) && a.ldo % 16 == 0;
    CUtensorMap tx, tw;
    const int rc = maps(tx, tw, qx, qw, a.M, (GU ? 2 : 1) * (int64_t)a.N, K, 128);
    if (rc) return rc;
    CUtensorMap to;
    const int rco = internal_make_tmap(&to, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.out, (uint64_t)a.N, (uint64_t)a.M, (uint64_t)a.ldo * 2,
                                       64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rco) return rco;
    const int tiles = num_m * num_n;
    e = launch_kernel(kern, dim3((unsigned)(2 * S * std::min(tiles, clusters))), dim3(kWideThreads), kWideSmem, st, 2 * S, true,
                      tx, tw, to, a);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "block linear launch");
}

struct FewPlan {
    int rows, split;      // rows of x a tile, CTAs that share a tile
    double us;            // what the call is expected to take
};

// A call with tiles of T rows.  CTAs that share a tile's K: as many as run at once, each with four k-blocks or more.
// Expected time: 4 us for launch, first copies and end, which grow with the sums that meet at the end; then
// k-blocks at what one takes a CTA while the weight comes out of L2, or the weight's bytes at 6 TB/s.
template <int T, bool GU>
FewPlan plan_few(const BlockArgs &a, int sms) {
    using F = Few<T, GU>;
    const int64_t tiles = (int64_t)((a.N + 127) / 128) * ((a.M + T - 1) / T), slots = (int64_t)F::kPerSm * sms;
    FewPlan p{T, 1, 0.0};
    for (int n = 2; n <= kMaxSplit && 4 * n <= a.nkb; ++n)
        if (tiles * n <= slots && tiles <= (int64_t)F::kPerSm * clusters_at_once(n, sms)) p.split = n;
    const double step = GU ? (T == 16 ? 0.30 : T == 32 ? 0.40 : 0.60) : (T == 16 ? 0.24 : T == 32 ? 0.31 : T == 64 ? 0.29 : 0.44);
    const double steps = (double)((tiles * p.split + slots - 1) / slots) * ((a.nkb + p.split - 1) / p.split);
    const double bytes = (double)F::kTiles * ((a.N + 127) / 128) * a.nkb * kBoxBytes;
    p.us = 4.0 + 0.04 * F::kTiles * std::min(T, a.M) + std::max(steps * step, bytes / 6.0e6);
    return p;
}

template <int T, bool GU>
int launch_few(const void *qx, const void *qw, int64_t K, BlockArgs a, int split, int sms, int all_sms, cudaStream_t st) {
    using F = Few<T, GU>;
    static SmemOptIn opt;
    auto kern = few_kernel<T, GU>;
    cudaError_t e = opt.set(reinterpret_cast<const void *>(kern), F::kSmem);
    if (e != cudaSuccess) return internal_cuda_error(e, "block linear smem attribute");
    CUtensorMap tx, tw;
    const int rc = maps(tx, tw, qx, qw, a.M, (GU ? 2 : 1) * (int64_t)a.N, K, T);
    if (rc) return rc;
    a.split = split;
    a.tiles_m = (a.M + T - 1) / T;
    int64_t clusters = (int64_t)((a.N + 127) / 128) * a.tiles_m;             // (N is under 2^29, and tiles_m at most 256)
    if (sms < all_sms) clusters = std::min<int64_t>(clusters, std::max(1, sms / split));   // a budget of SMs
    const int64_t grid = clusters * split;
    e = launch_kernel(kern, dim3((unsigned)grid), dim3(F::kThreads), F::kSmem, st, split, true, tx, tw, a);
    return e == cudaSuccess ? CLEF_OK : internal_cuda_error(e, "block linear launch");
}

// The kernel for a call: the one expected to take least on the whole device, so that a budget of SMs changes no
// sum's order.  (Every kernel measured at 2048 x 2048, 1024 x 5120, 6144 x 5120,
// 5120 x 17408 and 34816 x 5120, and at 2048 and 17408 gate/up columns, and narrow ones, for 1 .. 4,096 rows, weights out of
// memory: in 149 of 162 calls the one taken is the fastest or within 6% of it.  The others: 17 to 64 rows by 6144, 34816 or
// 2 x 17408 columns, 8-19%, where tiles of 16 rows are taken and 32, or pairs, are faster; 100 rows by 34816 x 5120, 37%,
// pairs again; 200 and 256 rows by 2048 x 2048 and 1,502 and 2,048 by 256 x 2048, 12-18%, 32 rows a tile taken, 16 faster.)
template <bool GU>
int launch_block(const void *qx, const void *qw, int64_t K, const BlockArgs &a, int sms, int all_sms, cudaStream_t st) {
    // many rows: rounds of tiles, each k-block 0.38 us, or the weight's bytes at 4.5 TB/s
    const int64_t pairs = std::max(1, all_sms / 2), tiles = (int64_t)((a.M + 255) / 256) * (GU ? a.N / 128 : (a.N + 255) / 256);
    const double weight = (GU ? 2.0 : 1.0) * a.N * (double)K;
    FewPlan best{0, 1, 4.0 + std::max((double)((tiles + pairs - 1) / pairs) * a.nkb * 0.38, weight / 4.5e6)};
    // pairs that share a tile's K: clusters that run at once, each pair with four k-blocks or more.  (768 x 5,120 x 1,024
    // 18.4 us by one pair, 13.7 by two, 12.6 by four; 1,024 x 2,048 x 1,024 10.0, 9.4 and 10.1; 768 x 1,536 x 768 8.5
    // and 8.7.)
    for (int n = 2; n <= 4 && 4 * n <= a.nkb && tiles * n <= pairs && tiles <= clusters_at_once(2 * n, all_sms); n *= 2) {
        const double us = (n == 2 ? 6.7 : 9.5) + std::max((a.nkb + n - 1) / n * 0.38, weight / 4.5e6);
        if (us < best.us) best = {0, n, us};
    }
    if (a.M <= 4096) {
        for (const FewPlan &p : {plan_few<16, GU>(a, all_sms), plan_few<32, GU>(a, all_sms), plan_few<64, GU>(a, all_sms)})
            if (p.us < best.us) best = p;
        if constexpr (!GU) {
            const FewPlan p = plan_few<128, GU>(a, all_sms);
            if (p.us < best.us) best = p;
        }
    }
    switch (best.rows) {
        case 16: return launch_few<16, GU>(qx, qw, K, a, best.split, sms, all_sms, st);
        case 32: return launch_few<32, GU>(qx, qw, K, a, best.split, sms, all_sms, st);
        case 64: return launch_few<64, GU>(qx, qw, K, a, best.split, sms, all_sms, st);
        case 128:
            if constexpr (!GU) return launch_few<128, GU>(qx, qw, K, a, best.split, sms, all_sms, st);
            [[fallthrough]];
        default:
            return best.split == 4 ? launch_wide<GU, 4>(qx, qw, K, a, sms, all_sms, st)
                 : best.split == 2 ? launch_wide<GU, 2>(qx, qw, K, a, sms, all_sms, st)
                                   : launch_wide<GU, 1>(qx, qw, K, a, sms, all_sms, st);
    }
}

int block_call(bool gu, const void *qx, const float *sx, const void *qw, const float *sw, const void *bias, int64_t M,
               int64_t N, int64_t K, void *out, int64_t ldo, void *stream) {
    constexpr int64_t kMax = (int64_t)1 << 30;
    if (M < 0 || M > kMax) return kv_fail("M out of range");
    if (N <= 0 || N > kMax / 2 || N % (gu ? 128 : 8) != 0)
        return kv_fail(gu ? "N must be positive and a multiple of 128" : "N must be positive and a multiple of 8");
    if (K <= 0 || K > 65536 || K % 16 != 0) return kv_fail("K must be in (0, 65536] and a multiple of 16");
    if (ldo < N || ldo % 8 != 0) return kv_fail("output row pitch must be >= N and a multiple of 8");
    if (M == 0) return CLEF_OK;
    if (!qx || !qw || !out || !sx || !sw) return kv_fail("null pointer");
    if (kv_misaligned(qx, 16) || kv_misaligned(qw, 16) || kv_misaligned(out, 16) || kv_misaligned(bias, 16))
        return kv_fail("operands, bias and output must be 16-byte aligned");
    if (kv_misaligned(sx, 4) || kv_misaligned(sw, 4)) return kv_fail("scales must be 4-byte aligned");
    const int64_t tiles_n = (N + 127) / 128;
    if ((M + 255) / 256 * (gu ? tiles_n : (N + 255) / 256) > 0x7FFFFFFF) return kv_fail("output too large");
    int sms = 0;
    unsigned int *status = nullptr;
    const int rc = internal_device(&sms, &status);
    if (rc) return rc;
    const int all_sms = sms;
    sms = internal_launch_sms(sms);
    BlockArgs a;
    a.M = (int)M;
    a.N = (int)N;
    a.nkb = (int)((K + 127) / 128);
    a.sx = sx;
    a.sw = sw;
    a.bias = static_cast<const uint16_t *>(bias);
    a.out = static_cast<uint16_t *>(out);
    a.ldo = ldo;
    a.band = a.split = a.tiles_m = 1;
    a.whole = false;
    a.status = status;
    a.limit_ns = internal_wait_limit(&a.force_timeout);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return gu ? launch_block<true>(qx, qw, K, a, sms, all_sms, st) : launch_block<false>(qx, qw, K, a, sms, all_sms, st);
}

}  // namespace

}  // namespace clef

using namespace clef;

extern "C" int clef_fp8_block_linear(const void *qx, const float *sx, const void *qw, const float *sw, const void *bias,
                                     int64_t M, int64_t N, int64_t K, void *y, int64_t ldy, void *stream) {
    return block_call(false, qx, sx, qw, sw, bias, M, N, K, y, ldy, stream);
}

extern "C" int clef_fp8_block_gateup_swiglu(const void *qx, const float *sx, const void *qw_gu, const float *sw_gu,
                                            const void *bias_gu, int64_t M, int64_t N, int64_t K, void *h, int64_t ldh,
                                            void *stream) {
    return block_call(true, qx, sx, qw_gu, sw_gu, bias_gu, M, N, K, h, ldh, stream);
}
