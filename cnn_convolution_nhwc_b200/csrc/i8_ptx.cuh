// Wrappers that only the 8-bit kernels use, beside those of ptx.cuh: tensor copies and stores issued
// from converged warps, requests to L2, and tcgen05.mma on 8-bit integers.
#pragma once
#include "ptx.cuh"

namespace convb200 {

// Places of the 8-bit kernels' bounds checks (BoundsSite in ptx.cuh has the other kernels').
enum I8BoundsSite : unsigned {
    kSiteI8RowsX = 64, kSiteI8RowsQ, kSiteI8RowsScale, kSiteI8FilterF, kSiteI8FilterQ, kSiteI8FilterScale, kSiteI8Dequant,
    kSiteI8GemmScale, kSiteI8GemmY
};

// The two halves of cluster_sync_all, for work between them.
__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}

__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Asynchronous 16-byte copy by the calling thread: the first `bytes` (0 to 16) of src, zeros after.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Tensor copies issued by a whole converged warp: only the lane whose `leader` is non-zero arms the
// barrier and issues them. As with the MMAs, a producer loop that the whole warp runs, with its
// copies predicated instead of placed under a one-lane branch, issues them faster: measured on
// B200, 0.14 us instead of 0.25 us for a wait, an expect and two copies.
__device__ __forceinline__ void mbar_arrive_expect_tx_if(uint32_t bar, uint32_t bytes, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t"
        "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_if(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y,
                                               uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}"
        :
        : "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(leader)
        : "memory");
}

// Asks for a box to be brought into L2, without waiting for it or reading it: allowed before
// grid_dependency_wait, since L2 is where a predecessor's writes arrive.
__device__ __forceinline__ void tma_prefetch_2d_if(const CUtensorMap *m, int x, int y, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\t"
        "@q cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];\n\t}"
        :
        : "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tma_prefetch_3d_if(const CUtensorMap *m, int x, int y, int z, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];\n\t}"
        :
        : "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tma_load_3d_if(uint32_t dst, const CUtensorMap *m, uint32_t bar, int x, int y, int z,
                                               uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}"
        :
        : "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair_if(uint32_t dst, const CUtensorMap *m, uint32_t bar_cluster, int x,
                                                    int y, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}"
        :
        : "r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(bar_cluster), "r"(x), "r"(y), "r"(leader)
        : "memory");
}

// A tensor store and its bulk group by the lane whose `leader` is non-zero, in a converged warp.
__device__ __forceinline__ void tma_store_2d_commit_if(const CUtensorMap *m, uint32_t src, int x, int y, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];\n\t"
        "@q cp.async.bulk.commit_group;\n\t}"
        :
        : "l"(reinterpret_cast<uint64_t>(m)), "r"(src), "r"(x), "r"(y), "r"(leader)
        : "memory");
}

// mbar_arrive_cluster by the lane whose `leader` is non-zero, in a converged warp.
__device__ __forceinline__ void mbar_arrive_cluster_if(uint32_t addr, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n\t}" ::"r"(addr), "r"(leader)
        : "memory");
}

// D[tmem] (+)= A[smem] * B[smem], kind::i8 (8-bit integers, 32-bit integer accumulator), in a
// converged warp as above.
__device__ __forceinline__ void umma_i8_ss_if(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                              uint32_t accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        :
        : "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

__device__ __forceinline__ void umma_i8_ss_pair_if(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                   uint32_t accumulate, uint32_t leader) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::2.kind::i8 [%0], %1, %2, %3, p;\n\t}"
        :
        : "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(leader)
        : "memory");
}

// Instruction descriptor for kind::i8 with signed 8-bit A and B, both K-major, and 32-bit integer D
// (2 in the D format field, no saturation).
__host__ __device__ constexpr uint32_t idesc_i8_s32(int M, int N) {
    return (2u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace convb200
