// clef_pair.cuh -- what the tensor-core GEMMs share beyond clef_ptx.cuh: CTA
// pairs (tcgen05 cta_group::2, cluster barriers, copies counted in the peer CTA),
// the wait of a kernel that winds down, and pieces of their epilogues.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "clef_ptx.cuh"

namespace clef {

// Time-limited wait that ignores the abort flag (used only while winding
// down, to let copies and MMAs already in flight finish).
__device__ __forceinline__ bool mbar_wait_drain(uint64_t *bar, uint32_t parity, uint64_t limit_ns,
                                                unsigned int *status) {
    const uint32_t a = smem_u32(bar);
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 0;; ++it) {
        if (mbar_try_wait(a, parity)) return true;
        if ((it & 63u) == 63u && globaltimer_ns() - t0 > limit_ns) {
            record_status(status, kStatusTimeout | (kSiteDrain << 8));
            return false;
        }
    }
}

// ---------------------------------------------------------------- CTA pairs

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

// Shared::cluster address of the same shared variable in the pair's leader (rank 0).
__device__ __forceinline__ uint32_t leader_addr(const void *local) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(local)));
    return r;
}

__device__ __forceinline__ void arrive_cluster(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}

// Relaxed cluster-scope arrive: no release fence.  Used only to forward a
// readiness signal whose data ordering was already established locally (see
// Gemm::forwarder); a release at cluster scope costs about a microsecond.
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t cluster_bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_bar)
                 : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
                 ::: "memory");
}

__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar_addr, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar_addr), "r"(parity)
        : "memory");
    return ok != 0;
}

// Time-limited wait with cluster-scope acquire (barriers that receive arrivals
// from the peer CTA or multicast commits); otherwise as mbar_wait.
__device__ __forceinline__ bool mbar_wait_cl(uint64_t *bar, uint32_t parity, const WaitCtx &w,
                                             unsigned int site) {
    const uint32_t a = smem_u32(bar);
    if (mbar_try_wait_cluster(a, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait_cluster(a, parity)) return true;
        if ((it & 63u) == 0u) {
            if (*w.abort) return false;
            if (globaltimer_ns() - t0 > w.limit_ns) {
                record_status(w.status, kStatusTimeout | (site << 8));
                *w.abort = 1;
                return false;
            }
        }
    }
}

__device__ __forceinline__ void mma2_f16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                         uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void mma2_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                        uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n"
        ::"r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Arrive on the barrier at this shared offset in both CTAs of the pair once
// the pair's MMAs issued so far by this thread have completed.
__device__ __forceinline__ void mma2_commit_both(uint64_t *bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

__device__ __forceinline__ void mma2_commit_local(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_u32(bar)) : "memory");
}

// TMA tile load into this CTA's shared memory whose completion is counted on
// a barrier that may live in the peer CTA (shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void *smem_dst, const CUtensorMap *m, int32_t c0,
                                                 int32_t c1, uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];"
        ::"r"(smem_u32(smem_dst)), "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1),
          "r"(cluster_bar)
        : "memory");
}

// silu(g) * u = g / (1 + exp(-g)) * u in fp32, with CUDA expf and a correctly
// rounded division: the bf16 result stays within one ulp of the correctly rounded value.
__device__ __forceinline__ float silu_mul_ieee(float g, float u) {
    const float d = __fadd_rn(1.0f, expf(-g));
    return __fmul_rn(__fdiv_rn(g, d), u);
}

// The same with the hardware exp2 and reciprocal approximations (a few fp32 ulps; beside
// silu_mul_ieee's, the bf16 results of both stay within one ulp of the correctly rounded value).
// Denominators above 2^126 (g below about -87) are scaled by 2^-64 with the
// numerator, exactly, to keep the fast quotient in its accurate range.
__device__ __forceinline__ float silu_mul_fast(float g, float u) {
    const float d = __fadd_rn(1.0f, __expf(-g));
    const float sc = d > 0x1p126f ? 0x1p-64f : 1.0f;
    return __fmul_rn(__fdividef(g * sc, d * sc), u);
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&p);
}

}  // namespace clef
