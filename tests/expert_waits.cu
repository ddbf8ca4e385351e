// What the expert kernels' bounded waits rest on, run alone: warps whose lanes have to agree on a failure, and
// a barrier that nothing arrives at, waited for until the limit. Built and called by test_expert_waits.py.
#include "tcgen05.cuh"

namespace {

// Warp 0 waits for a phase, lane by lane; warp 1 says that it has failed, and completes the phase, at about
// the time that the waits look at either: whatever comes first, the lanes have one answer. results[0] rounds on
// which they differ, [1] rounds that succeed, [2] rounds that fail.
__global__ void agreement_kernel(int rounds, int *results) {
    __shared__ uint64_t bar;
    __shared__ volatile int failed;
    int differ = 0, good = 0, bad = 0;
    for (int i = 0; i < rounds; ++i) {
        if (threadIdx.x == 0) {
            ep::mbar_init(&bar, 1);
            failed = 0;
            ep::fence_mbar_init();
        }
        __syncthreads();
        if (threadIdx.x / 32 == 0) {
            const unsigned votes = __ballot_sync(0xFFFFFFFFu, ep::mbar_wait_warp(&bar, 0, &failed));
            differ += votes != 0 && votes != 0xFFFFFFFFu;
            good += votes == 0xFFFFFFFFu;
            bad += votes == 0;
        } else if (threadIdx.x == 32) {
            if (i & 1) failed = 1;
            __nanosleep(i % 64 * 50);
            if (i % 4 != 1) ep::mbar_arrive(&bar);
        }
        __syncthreads();
        if (threadIdx.x == 0) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(ep::smem_u32(&bar)) : "memory");
    }
    if (threadIdx.x == 0) results[0] = differ, results[1] = good, results[2] = bad;
}

// results: [0] lanes whose wait succeeded, [1] the flag after it, [2] whether a poll that starts after the
// failure succeeds, [3] lanes that succeed on a phase that is complete.
__global__ void give_up_kernel(int *results, int *error) {
    __shared__ uint64_t never, done;
    __shared__ volatile int failed;
    if (threadIdx.x == 0) {
        ep::mbar_init(&never, 1);
        ep::mbar_init(&done, 1);
        failed = 0;
        ep::fence_mbar_init();
        ep::mbar_arrive(&done);
    }
    __syncwarp();
    const bool complete = ep::mbar_wait_warp(&done, 0, &failed);
    const unsigned d = __ballot_sync(0xFFFFFFFFu, complete);
    const bool ok = ep::mbar_wait_warp(&never, 0, &failed);
    const unsigned v = __ballot_sync(0xFFFFFFFFu, ok);
    if (threadIdx.x == 0) {
        results[0] = __popc(v);
        results[1] = failed;
        results[2] = ep::mbar_poll_limited(&never, 0, &failed);
        results[3] = __popc(d);
        if (failed) atomicOr(error, ep::kErrExpertWait);
    }
}

// A ring of four stages after `fills` fills, all of which have landed, or all but the last one:
// results[late] = whether the wait says that all of them have.
__global__ void fills_kernel(int fills, int *results) {
    __shared__ uint64_t full[4];
    for (int late = 0; late < 2; ++late) {
        for (int i = 0; i < 4; ++i) ep::mbar_init(&full[i], 1);
        ep::fence_mbar_init();
        for (int i = 0; i < fills - late; ++i) ep::mbar_arrive(&full[i % 4]);
        results[late] = ep::wait_for_fills(full, fills, 0, 2, 4) + 2 * ep::wait_for_fills(full, fills, 1, 2, 4);
        for (int i = 0; i < 4; ++i) asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(ep::smem_u32(&full[i])) : "memory");
    }
}

}  // namespace

extern "C" int run_fills(int fills, int *results) {
    fills_kernel<<<1, 1>>>(fills, results);
    return (int)cudaDeviceSynchronize();
}
extern "C" int run_agreement(int rounds, int *results) {
    agreement_kernel<<<1, 64>>>(rounds, results);
    return (int)cudaDeviceSynchronize();
}
extern "C" int run_give_up(int *results, int *error) {
    give_up_kernel<<<1, 32>>>(results, error);
    return (int)cudaDeviceSynchronize();
}
