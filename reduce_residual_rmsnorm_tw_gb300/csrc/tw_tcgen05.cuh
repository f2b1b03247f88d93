// tw_tcgen05.cuh -- device helpers for the 5th-generation tensor cores: TMEM,
// tcgen05.mma/ld/st/commit, tiled TMA loads, and barriers shared by a CTA pair.
// Everything here is written from the public PTX ISA description.
#pragma once

#include <cuda.h>

#include "tw_device.cuh"

namespace tw {

// ------------------------------------------------------------ clusters ---
__device__ __forceinline__ uint32_t cluster_cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_id_x() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%clusterid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_count_x() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%nclusterid.x;" : "=r"(r));
    return r;
}
// All threads of all CTAs: release this CTA's shared-memory writes, acquire
// the peers'.
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address of `local` (this CTA's shared memory) in CTA `rank`.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t local, uint32_t rank) {
    uint32_t remote;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(rank));
    return remote;
}
// Arrive on a barrier of a CTA of the pair for work that stays in this CTA:
// its own shared-memory writes (already ordered for the async proxy by
// fence_async_shared) and TMEM accesses (complete, behind
// tcgen05.fence::before_thread_sync), which this SM's half of the pair's next
// MMA uses.  No generic access of the other CTA depends on it, so the arrive
// keeps CTA scope: at cluster scope the release first waits for every earlier
// access of the thread to be visible there, about 1000 clocks for each slice
// of a product (the int8 kernel ran at half the speed).
__device__ __forceinline__ void mbar_arrive_pair(uint32_t remote_bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote_bar) : "memory");
}
__device__ __forceinline__ bool mbar_try_wait_cluster(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    return done != 0;
}
// As mbar_wait, for the waits of a product's slices: the abort flag and the
// clock are looked at once in 64 tries.  CLUSTER: see what the cluster's other
// CTAs released (their writes into this CTA's shared memory); without it the
// acquire stays within the CTA, which is all that work signalled with
// mbar_arrive_pair, a TMA or a commit needs, and costs no invalidation.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_slice(uint32_t bar, uint32_t parity,
                                                const volatile int* abort) {
    uint64_t start = 0;
    for (uint32_t tries = 1;; ++tries) {
        if (CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if (tries % 64 == 0) {
            if (abort && *abort) return false;
            const uint64_t now = global_timer_ns();
            if (start == 0) start = now;
            if (now - start > kWaitLimitNs) return false;
        }
    }
}
// `bytes` (a multiple of 16) of this CTA's shared memory to another's, counted
// on that CTA's barrier `bar` when they have landed (remote, bar:
// shared::cluster addresses).
__device__ __forceinline__ void bulk_push(uint32_t remote, uint32_t local, uint32_t bytes,
                                          uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes "
        "[%0], [%1], %2, [%3];" ::"r"(remote),
        "r"(local), "r"(bytes), "r"(bar)
        : "memory");
}
// Order this thread's shared-memory writes before later async-proxy reads
// (the tensor cores').
__device__ __forceinline__ void fence_async_shared() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// 1 in one lane of a whole warp (always the same one), 0 in the others.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one;
}

// ----------------------------------------------------------------- TMA ---
__device__ __forceinline__ void tensormap_prefetch(const CUtensorMap* m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
// One box of a 2-D tensor to this CTA's shared memory, issued by the lane whose
// `one` is not zero (see the MMAs below).  CG 2: `bar` may be a barrier of
// either CTA of the pair (a shared::cluster address).
template <int CG>
__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y,
                                            uint32_t bar, uint32_t one) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile"
            ".mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
            "l"(map), "r"(x), "r"(y), "r"(bar), "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t"
            "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile"
            ".mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(
                dst),
            "l"(map), "r"(x), "r"(y), "r"(bar), "r"(one)
            : "memory");
}
// The same box into L2 only.
__device__ __forceinline__ void tma_warm_2d(const CUtensorMap* map, int x, int y, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
        "@q cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n\t}" ::"l"(map),
        "r"(x), "r"(y), "r"(one)
        : "memory");
}
// As mbar_arrive_expect_tx, by that lane.
__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes, uint32_t one) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
        "r"(bytes), "r"(one)
        : "memory");
}

// One box from this CTA's shared memory to a 2-D tensor (parts outside it are
// not written), in this thread's current bulk group.
__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src) {
    asm volatile(
        "cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
        "r"(x), "r"(y), "r"(src)
        : "memory");
}
__device__ __forceinline__ void bulk_commit() {
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// All but the newest N of this thread's bulk groups have read their source.
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- TMEM ---
// Whole warp.  Writes the base address to *slot (shared memory).
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t columns) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         slot),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         slot),
                     "r"(columns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t columns) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base),
                     "r"(columns));
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base),
                     "r"(columns));
}
__device__ __forceinline__ void tcgen05_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tcgen05_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_loads() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_wait_stores() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 16 columns of this warp's 32 lanes (a register per column); not complete
// before tmem_wait_loads.
__device__ __forceinline__ void tmem_load16(uint32_t (&r)[16], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_load8(uint32_t (&r)[8], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr)
        : "memory");
}
// 16 columns of 16 lanes as 8x8 fragments: registers 4 i, 4 i + 1 of thread t
// hold columns 8 i + 2 (t % 4) and the next of lane t / 4, registers 4 i + 2
// and 4 i + 3 those of lane t / 4 + 8.
__device__ __forceinline__ void tmem_load_fragments(uint32_t (&r)[8], uint32_t addr) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(addr)
        : "memory");
}
// Four 8x8 matrices of 16-bit values, transposed: column i of matrix m to the
// 16 bytes at the address that lane 8 m + i gives.
__device__ __forceinline__ void store_matrices_transposed(uint32_t addr, uint32_t m0, uint32_t m1,
                                                          uint32_t m2, uint32_t m3) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(
                     addr),
                 "r"(m0), "r"(m1), "r"(m2), "r"(m3)
                 : "memory");
}
__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(
            addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

// ----------------------------------------------------------------- MMA ---
// Shared-memory operand, K-major rows of 128 bytes in the 128-byte swizzle
// (what a TMA box 128 bytes wide writes): eight rows are 1024 bytes apart from
// the next eight.  A step of 32 bytes along K adds 2.
// Only the low word depends on the address; it travels alone, so that a step
// costs one 32-bit addition (64-bit ones made the int8 product 3 to 5 % slower:
// beside the widening warps its MMA warp is short of issue slots).
constexpr uint32_t kOperandHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t smem_operand(uint32_t addr) {
    return ((addr & 0x3ffffu) >> 4) | (1u << 16);
}
// Both operands K-major, fp32 accumulator, and operand format 0 for both: f16
// under kind::f16, e4m3 under kind::f8f6f4.
__device__ __forceinline__ uint32_t mma_shape(uint32_t m, uint32_t n) {
    return (1u << 4) | ((n >> 3) << 17) | ((m >> 4) << 24);
}
// The whole warp calls what follows; the lane whose `one` is not zero (exactly
// one: elect_one) issues.  As a predicate rather than a branch, so that the
// operands stay in the warp's uniform registers.
//
// D (TMEM) = A (TMEM, f16) * B (shared memory, f16) + D where `add`.
template <int CG>
__device__ __forceinline__ void mma_f16_tmem(uint32_t d, uint32_t a, uint32_t b, uint32_t shape,
                                             bool add, uint32_t one) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
            "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\tmov.b64 b, {%2, %3};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(kOperandHigh), "r"(shape), "r"(static_cast<uint32_t>(add)),
            "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 b;\n\t"
            "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\tmov.b64 b, {%2, %3};\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(kOperandHigh), "r"(shape), "r"(static_cast<uint32_t>(add)),
            "r"(one)
            : "memory");
}
// D (TMEM) = A * B (both shared memory, e4m3) + D where `add`.
template <int CG>
__device__ __forceinline__ void mma_e4m3(uint32_t d, uint32_t a, uint32_t b, uint32_t shape,
                                         bool add, uint32_t one) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
            "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
            "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(kOperandHigh), "r"(shape), "r"(static_cast<uint32_t>(add)),
            "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
            "setp.ne.u32 p, %5, 0;\n\tsetp.ne.u32 q, %6, 0;\n\t"
            "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
            "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %4, p;\n\t}" ::"r"(d),
            "r"(a), "r"(b), "r"(kOperandHigh), "r"(shape), "r"(static_cast<uint32_t>(add)),
            "r"(one)
            : "memory");
}
// Arrive on `bar` (CG 2: on the barrier at that offset in both CTAs of the
// pair, the bits of `pair` being their ranks) once the issuing lane's MMAs so
// far are complete.
template <int CG>
__device__ __forceinline__ void mma_commit(uint32_t bar, uint16_t pair, uint32_t one) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
            "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::
                "r"(bar),
            "r"(one)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %2, 0;\n\t"
            "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster"
            ".multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
            "h"(pair), "r"(one)
            : "memory");
}

}  // namespace tw
