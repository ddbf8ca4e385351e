// The cache of occupancies (device_info.cu) on a device that is not there: the runtime's answers are made up here, and its
// questions counted. Built and called by test_occupancy_cache.py.
#include <cuda_runtime.h>

#include <atomic>

namespace {
std::atomic<int> asked, device, fails;
cudaError_t fake_device(int *d) {
    *d = device;
    return cudaSuccess;
}
cudaError_t fake_occupancy(int *blocks, const void *, int threads, size_t smem) {
    ++asked;
    if (fails) return cudaErrorUnknown;
    *blocks = 1 + (threads + (int)smem + 7 * device) % 31;
    return cudaSuccess;
}
}  // namespace

#define cudaGetDevice fake_device
#define cudaOccupancyMaxActiveBlocksPerMultiprocessor(b, f, t, s) fake_occupancy(b, f, t, s)
#include "device_info.cu"

extern "C" int occupancy_of(int kernel, int threads, size_t smem) {
    return ep::max_blocks_per_sm(reinterpret_cast<const void *>((intptr_t)(1 + kernel)), threads, smem);
}
extern "C" int occupancy_questions() { return asked; }
extern "C" void use_device(int d) { device = d; }
extern "C" void fail(int f) { fails = f; }
