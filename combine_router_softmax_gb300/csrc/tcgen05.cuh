// tcgen05.cuh -- PTX wrappers of the tensor-core path: tiled TMA loads, TMEM,
// tcgen05.mma on bf16 operands in shared memory, and waits with a time limit.
#pragma once

#include "ep_internal.cuh"

#include <cuda.h>  // CUtensorMap (types only; the encoder is looked up at run time)

#include <mutex>

namespace ep {

// A dense matrix [y][x], or [z][y][x], of bf16 (bytes = 2) or bytes (1), to be read in boxes of bx by
// by elements, 128 bytes wide and swizzled over 128 bytes. What lies outside reads as zero.
bool make_map(CUtensorMap *m, const void *base, int bytes, int64_t x, int64_t y, int64_t z, int bx, int by);
// A dense [z][y][x] of 16-bit values, to be read and written in boxes of 32 by 32, swizzled over their 64 bytes.
bool make_piece_map(CUtensorMap *m, const void *base, int64_t x, int64_t y, int64_t z);

// The dynamic shared memory that one kernel may have on each device. The limit is the kernel's and not the call's:
// set by every call for itself, one thread's call could lower it between another's setting and launch. So it
// only grows. It is not set to the most that 1024 experts need at once: with that the streamed kernel's
// 4-bit layer of 5000 to 4321, 3 rows, took 11.0 us instead of 9.4.
class SharedMemoryLimit {
  public:
    template <typename Kernel>
    cudaError_t allow(Kernel kernel, size_t bytes) {
        int dev = 0;
        cudaError_t e = current_device(&dev);
        if (e != cudaSuccess || bytes <= allowed_[dev].load(std::memory_order_acquire)) return e;
        const std::lock_guard<std::mutex> lock(mutex_);
        if (bytes <= allowed_[dev].load(std::memory_order_relaxed)) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
        if (e == cudaSuccess) allowed_[dev].store(bytes, std::memory_order_release);
        return e;
    }

  private:
    std::mutex mutex_;
    std::atomic<size_t> allowed_[kMaxDevices_] = {};
};

// A wait gives up after about two seconds; no wait of a kernel that works comes near that, the
// longest one spans a single tile's main loop. mbarrier.try_wait puts the thread to sleep until the
// phase completes, for kWaitSliceNs at most: for waits that are long. One thread waits for its warp.
constexpr uint32_t kWaitSliceNs = 2000000;
constexpr int kWaitSlices = 1000;
constexpr int64_t kPollLimitCycles = 4000000000ll;  // the same for a thread that polls

// CLUSTER: what another CTA of the cluster wrote before it arrived is seen as well.
template <bool CLUSTER>
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(kWaitSliceNs)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity), "r"(kWaitSliceNs)
            : "memory");
    return ok != 0;
}

// Waits for the phase of `parity` to complete; false when it did not in time, or once another warp
// of the CTA has given up (*failed).
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_limited(uint64_t *bar, uint32_t parity, volatile int *failed) {
    for (int i = 0; i < kWaitSlices; ++i) {
        if (mbar_sleep_wait<CLUSTER>(bar, parity)) return true;
        if (*failed) return false;
    }
    *failed = 1;
    return false;
}

// Whether the phase of `parity` is complete by now. A loop over stages asks for the next one before it
// works on the present one, so that the answer's latency is behind that work.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    if constexpr (CLUSTER)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
    return ok != 0;
}

// mbar_wait_limited for one thread whose waits are short and on the path of every stage: it polls, as a
// thread that sleeps is woken late.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_poll_limited(uint64_t *bar, uint32_t parity, volatile int *failed) {
    int64_t begin = 0;
    for (;;) {
        for (int i = 0; i < 1024; ++i)
            if (mbar_test<CLUSTER>(bar, parity)) return true;
        const int64_t now = clock64();
        if (begin == 0) begin = now;
        if (*failed || now - begin > kPollLimitCycles) {
            *failed = 1;
            return false;
        }
    }
}

// mbar_wait_limited by every lane of a warp, each of which is to see what the phase brings: true in
// all of them or in none. A warp's lanes read `failed` at different times, and another warp may set it in
// between: lanes that went by their own readings could part, and the next instruction that needs all of
// them would wait without a limit.
template <bool CLUSTER = false>
__device__ __forceinline__ bool mbar_wait_warp(uint64_t *bar, uint32_t parity, volatile int *failed) {
    return __all_sync(0xFFFFFFFFu, mbar_wait_limited<CLUSTER>(bar, parity, failed)) != 0;
}

// Waits until the copies of a producer have landed: of the fills first, first + step, ... below `it`, the last
// one of each of the `stages` stages, whose barriers are `full`. One time limit for all of them. By one thread,
// after a failure, once nobody else uses the barriers.
__device__ __forceinline__ bool wait_for_fills(uint64_t *full, uint32_t it, uint32_t first, uint32_t step, uint32_t stages) {
    int gave_up = 0;
    for (uint32_t i = first; i < stages; i += step)
        if (it > i) mbar_wait_limited(&full[i], (it - 1 - i) / stages & 1, &gave_up);
    return gave_up == 0;
}

// True in one lane of the warp, all of which are active. The compiler knows of this predicate that
// one lane alone passes: the instructions below take uniform operands, and behind an ordinary
// `lane == 0` each of them becomes a loop over the active lanes.
__device__ __forceinline__ bool elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xFFFFFFFF;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok));
    return ok != 0;
}

// The address of `p`, a shared-memory address of this CTA, in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_smem_u32(const void *p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// Sets the int at `addr`, a shared::cluster address.
__device__ __forceinline__ void st_cluster(uint32_t addr, int v) {
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t cluster_cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Arrives on a barrier named by its shared::cluster address (any CTA of the cluster).
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Tiled TMA loads; x, the innermost coordinate, lies on a 16-byte boundary. CG = 2: the
// barrier may be the one of the CTA pair's other CTA (a shared::cluster address).
template <int CG>
__device__ __forceinline__ void tma_load_2d(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::
                "r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%2, %3}], [%4];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
            "[%5];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, "
            "{%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// TMEM. Allocation and release are done by one whole warp (of each CTA of a pair).
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst_smem, uint32_t columns) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                     "r"(columns)
                     : "memory");
    else
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst_smem)),
                     "r"(columns)
                     : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    } else {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns));
    }
}
__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 consecutive columns of this thread's TMEM lane (a warp reads 32 lanes).
__device__ __forceinline__ void tmem_load_32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}

// The values of this thread's loads so far are there. They pass through as operands, so no use
// of them moves ahead of the wait.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
                 :: "memory");
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// The 64-bit shared-memory descriptor of an operand whose rows are 128 bytes, swizzled over
// 128 bytes as TMA wrote them. K-major: a row is one m (or n), 8 rows every 1024 bytes.
// MN-major: a row is one k and holds 64 consecutive m; 8 rows every 1024 bytes, the next
// 64 m after mn_stride bytes.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t mn_stride) {
    return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)((mn_stride >> 4) & 0x3FFFu) << 16 | (uint64_t)(1024u >> 4) << 32 |
           1ull << 46 | 2ull << 61;
}

// The instruction descriptor: bf16 operands, fp32 accumulators.
constexpr uint32_t mma_idesc(int m, int n, bool a_mn_major, bool b_mn_major) {
    return 1u << 4 | 1u << 7 | 1u << 10 | (a_mn_major ? 1u : 0u) << 15 | (b_mn_major ? 1u : 0u) << 16 | (uint32_t)(n >> 3) << 17 |
           (uint32_t)(m >> 4) << 24;
}

// D[tmem] (+)= A[smem] B[smem], K = 16; issued by one thread.
template <int CG>
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
            : "memory");
}
// The barrier gets one arrival when this thread's MMAs so far are done (CG = 2: the barrier
// at the same offset in both CTAs of the pair).
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                     : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}

}  // namespace ep
