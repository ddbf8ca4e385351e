// device_info.cu -- what the host asks a device about once: its number of SMs, and how many CTAs of a kernel an SM holds.
#include <mutex>
#include <unordered_map>

#include "ep_internal.cuh"

namespace ep {

namespace {
constexpr int kMaxDevices = kMaxDevices_;
std::atomic<int> g_sm_count[kMaxDevices];  // zero-initialised: not yet queried

// What an occupancy depends on. A process may come to use many: the norms have some for every width, form and type.
struct Shape {
    const void *fn;
    int dev, threads;
    size_t smem;
    bool operator==(const Shape &o) const { return fn == o.fn && dev == o.dev && threads == o.threads && smem == o.smem; }
};
struct ShapeHash {
    size_t operator()(const Shape &s) const {
        size_t h = reinterpret_cast<uintptr_t>(s.fn);
        for (const size_t v : {(size_t)s.dev, (size_t)s.threads, s.smem}) h = (h ^ v) * 0x9E3779B97F4A7C15ull;
        return h ^ h >> 32;
    }
};
std::mutex g_occ_mu;
std::unordered_map<Shape, int, ShapeHash> &occupancies() {
    static auto *map = new std::unordered_map<Shape, int, ShapeHash>;  // lives as long as the process, whatever ends first
    return *map;
}
}  // namespace

int sm_count(int device) {
    if (device < 0 || device >= kMaxDevices) return 0;
    int v = g_sm_count[device].load(std::memory_order_relaxed);
    if (v == 0) {
        if (cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, device) != cudaSuccess) return 0;
        g_sm_count[device].store(v, std::memory_order_relaxed);
    }
    return v;
}

int current_device_sm_count() {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return sm_count(dev);
}

int max_blocks_per_sm(const void *fn, int threads, size_t smem) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 1;
    const Shape shape{fn, dev, threads, smem};
    int b = 0;
    try {
        const std::lock_guard<std::mutex> lock(g_occ_mu);
        const auto known = occupancies().find(shape);
        if (known != occupancies().end()) return known->second;
        if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, fn, threads, smem) == cudaSuccess && b > 0) {
            occupancies().emplace(shape, b);
            return b;
        }
    } catch (...) {  // no memory for what would be kept
        return b > 0 ? b : 1;
    }
    cudaGetLastError();
    return 1;
}

}  // namespace ep
