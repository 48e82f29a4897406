// tc.cuh — sm_100a building blocks of the dense tensor-core products: tensor
// maps and TMA loads of 64 x 64 BF16 boxes, shared-memory and instruction
// descriptors, tcgen05 issue / commit / TMEM reads, cluster barriers.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {
namespace tc {

// Every operand tile is built from boxes of 64 x 64 BF16 (64 elements = 128
// bytes along the contiguous dimension, 64 lines), loaded by TMA with the
// 128-byte swizzle: 8 KB each, 1024-byte aligned.
constexpr uint32_t kBox = 8192;

// Shared-memory descriptor of a tile of such boxes, 128-byte swizzle (layout
// 2 at bit 61, version 1 at bit 46).
// K-major (lines = rows of M or N, 64 K per line): 8-line groups 1024 bytes
// apart (stride byte offset), the next 64 rows in the next box; one MMA step
// (K = 16) is 32 bytes further along the line.
// MN-major (lines = K, 64 rows of M or N per line): 8-line groups of K 1024
// bytes apart (stride byte offset), the next 64 rows one box on (leading
// byte offset); one MMA step is 16 lines = 2048 bytes further.
template <bool MN>
__device__ __forceinline__ uint64_t desc(uint32_t addr) {
    const uint64_t lbo = MN ? kBox : 16u;
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16) | ((uint64_t)(1024u >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
template <bool MN>
__device__ __forceinline__ constexpr uint32_t kstep() {
    return MN ? 2048u : 32u;
}

// Instruction descriptor of kind::f16: BF16 x BF16 -> FP32, majorness of A
// and B (bits 15, 16), N / 8 (bit 17), M / 16 (bit 24).
__device__ __forceinline__ constexpr uint32_t idesc(int m, int n, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t id, bool acc) {
    if (CG == 1)
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b),
            "r"(id), "r"(acc ? 1u : 0u)
            : "memory");
    else
        asm volatile(
            "{ .reg .pred p; setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a), "l"(b),
            "r"(id), "r"(acc ? 1u : 0u)
            : "memory");
}

// Arrive on *bar (CG 2: on the barrier at this offset in both CTAs of the
// pair) once the tcgen05 work issued so far by this thread has completed.
template <int CG>
__device__ __forceinline__ void commit(uint64_t *bar) {
    if (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                         smem_u32(bar))
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
            "[%0], %1;" ::"r"(smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}

__device__ __forceinline__ void fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_async() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t cols) {
    if (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)),
                     "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
    if (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// 16 columns of TMEM, one row (lane) per thread of the warp; complete only
// after tmem_wait().
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
          "=r"(r[15])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_wait() {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// True in one lane of a converged warp.  The warps that issue copies and MMAs
// run their loops whole, with the issue under this predicate: loop counters,
// addresses and descriptors stay in uniform registers (with the loop inside
// one lane a K block of 4 MMAs took 745 clocks of issue, whatever its data).
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{ .reg .pred q; elect.sync _|q, 0xffffffff; selp.u32 %0, 1, 0, q; }" : "=r"(p));
    return p != 0;
}

// Position in a ring of `n` slots: the slot, and the parity of its passes.
struct Ring {
    uint32_t slot = 0, pass = 0;
    __device__ __forceinline__ void next(uint32_t n) {
        if (++slot == n) {
            slot = 0;
            ++pass;
        }
    }
    __device__ __forceinline__ void prev(uint32_t n) {
        if (slot-- == 0) {
            slot = n - 1;
            --pass;
        }
    }
};

// ---------------------------------------------------------------- cluster --

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// The address of this CTA's shared-memory address `a` in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t a, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ int ld_cluster(uint32_t a) {
    int v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float4 ld_cluster16(uint32_t a) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(a));
    return v;
}
// Arrivals on a barrier given by its cluster address.  arrive_tx announces a
// copy's bytes and orders nothing (relaxed: a release at cluster scope would
// wait for the thread's own copies in flight; measured, it held the producer
// to one K block per memory latency, 1.0 us instead of 0.3).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void arrive_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cta.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void arrive_tx_cluster(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar),
                 "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2; "
        "selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// Bounded wait on phase `parity` of *bar; gives up after `polls` polls (1.5 us
// each when nothing comes) or once *abort is set, which it sets when it runs
// out.
// CLUSTER: acquire what the other CTA's threads wrote (costs about 0.1 us
// more per wait; copies and tensor-core work need none of it).
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, volatile int *abort, int polls) {
#pragma unroll 1
    for (int i = 0; i < polls; ++i) {
        if (CLUSTER ? try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)) return true;
        if (*abort) return false;
    }
    *abort = 1;
    return false;
}

// TMA load of one box; `bar` is a cluster address (CG 2: may lie in the
// pair's other CTA).  x is a multiple of 64 elements (128 bytes).
template <int CG>
__device__ __forceinline__ void load2(uint32_t dst, const CUtensorMap *m, int x, int y, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
            "%3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3}], [%4];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void load3(uint32_t dst, const CUtensorMap *m, int x, int y, int z, uint32_t bar) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
            "%3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
            "[%1, {%2, %3, %4}], [%5];" ::"r"(dst),
            "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *m) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(m)) : "memory");
}

// ------------------------------------------------------------------- host --

inline PFN_cuTensorMapEncodeTiled map_encoder() {
    static const PFN_cuTensorMapEncodeTiled fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            return reinterpret_cast<PFN_cuTensorMapEncodeTiled>(p);
        return PFN_cuTensorMapEncodeTiled(nullptr);
    }();
    return fn;
}

inline cudaError_t make_map(CUtensorMap *m, const void *base, int rank, const cuuint64_t *dims,
                            const cuuint64_t *strides, const cuuint32_t *box) {
    const PFN_cuTensorMapEncodeTiled fn = map_encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint32_t one[3] = {1, 1, 1};
    const CUresult r =
        fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, one,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// [n][rows][cols], boxes of 64 columns x `lines` rows of one matrix.
inline cudaError_t map_stack(CUtensorMap *m, const uint16_t *base, int64_t n, int64_t rows, int64_t cols,
                             int lines) {
    const cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)n};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)(rows * cols) * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)lines, 1};
    return make_map(m, base, 3, dims, strides, box);
}
// A row-major [rows][cols] BF16 matrix, boxes of 64 columns x `lines` rows;
// elements outside the matrix read as zero.
inline cudaError_t map_matrix(CUtensorMap *m, const uint16_t *base, int64_t rows, int64_t cols, int lines = 64) {
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)cols * 2};
    const cuuint32_t box[2] = {64, (cuuint32_t)lines};
    return make_map(m, base, 2, dims, strides, box);
}
// [rows][2][cols]: the two halves of a row kept apart, so that a box past
// the end of one half reads zeros and not the other half.
inline cudaError_t map_halves(CUtensorMap *m, const uint16_t *base, int64_t rows, int64_t cols, int lines = 64) {
    const cuuint64_t dims[3] = {(cuuint64_t)cols, 2, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)cols * 2, (cuuint64_t)cols * 4};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)lines};
    return make_map(m, base, 3, dims, strides, box);
}

}  // namespace tc
}  // namespace moe
