// grad_clip.cu -- the global norm of many gradient tensors, and clipping by it.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kClipThreads = 512;
constexpr int kClipTensors = 768;  // tensors of one launch: their table is a kernel argument
// The largest grid of either kernel: four CTAs of 512 threads fill an SM, on 152 of them.
constexpr int kClipGrid = 4 * 152;

// The tensors of a launch. Work is dealt out in chunks of `chunk` values of one tensor.
struct ClipTable {
    const void *data[kClipTensors];
    void *out[kClipTensors];
    int64_t numel[kClipTensors];
    int32_t first[kClipTensors + 1];  // chunks before each tensor
    uint8_t dtype[kClipTensors];
    int32_t n, chunk;
};
static_assert(sizeof(ClipTable) + 64 <= 32764, "kernel arguments");

template <typename V>
struct Io;
template <>
struct Io<float> {
    static constexpr int kVec = 4;
    static __device__ float load(const float *p) { return *p; }
    static __device__ void store(float *p, float v) { *p = v; }
    static __device__ void unpack(const uint4 &q, float (&v)[4]) {
        v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y), v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
    }
    static __device__ uint4 pack(const float (&v)[4]) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <>
struct Io<__nv_bfloat16> {
    static constexpr int kVec = 8;
    static __device__ float load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
    static __device__ void store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
    static __device__ void unpack(const uint4 &q, float (&v)[8]) {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(u[i] << 16), v[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    }
    static __device__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <>
struct Io<__half> {
    static constexpr int kVec = 8;
    static __device__ float load(const __half *p) { return __half2float(*p); }
    static __device__ void store(__half *p, float v) { *p = __float2half_rn(v); }
    static __device__ void unpack(const uint4 &q, float (&v)[8]) {
        const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
            v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
    }
    static __device__ uint4 pack(const float (&v)[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(u[0], u[1], u[2], u[3]);
    }
};

// Values before the first 16-byte boundary at or after p.
template <typename V>
__device__ __forceinline__ int64_t values_to_boundary(const V *p) {
    return (int64_t)((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(V);
}

// The sum of the squares of n values, this thread's part. Four independent sums of fp32; a chunk
// leaves at most chunk / kClipThreads values to a thread, so no sum grows long before it is added
// up in 64 bits.
template <typename V>
__device__ double square_sum(const V *p, int64_t n) {
    constexpr int kVec = Io<V>::kVec;
    float acc[4] = {0, 0, 0, 0};
    const int64_t head = min(values_to_boundary(p), n);
    if (threadIdx.x < head) {
        const float v = Io<V>::load(p + threadIdx.x);
        acc[0] = v * v;
    }
    const uint4 *q = reinterpret_cast<const uint4 *>(p + head);
    const int64_t vecs = (n - head) / kVec;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < vecs; i += kClipThreads) {
        float v[kVec];
        Io<V>::unpack(q[i], v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) acc[j % 4] = fmaf(v[j], v[j], acc[j % 4]);
    }
    const int64_t tail = head + vecs * kVec + threadIdx.x;
    if (tail < n) {
        const float v = Io<V>::load(p + tail);
        acc[1] = fmaf(v, v, acc[1]);
    }
    return ((double)acc[0] + acc[1]) + ((double)acc[2] + acc[3]);
}

template <typename V>
__device__ void scale_values(const V *p, V *out, int64_t n, float coef) {
    constexpr int kVec = Io<V>::kVec;
    // where input and output lie differently to the boundary, value by value
    const bool same = ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(out)) & 15) == 0;
    const int64_t head = same ? min(values_to_boundary(p), n) : n;
    for (int64_t i = threadIdx.x; i < head; i += kClipThreads) Io<V>::store(out + i, Io<V>::load(p + i) * coef);
    const uint4 *q = reinterpret_cast<const uint4 *>(p + head);
    uint4 *o = reinterpret_cast<uint4 *>(out + head);
    const int64_t vecs = (n - head) / kVec;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < vecs; i += kClipThreads) {
        float v[kVec];
        Io<V>::unpack(q[i], v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] *= coef;
        o[i] = Io<V>::pack(v);
    }
    const int64_t tail = head + vecs * kVec + threadIdx.x;
    if (tail < n) Io<V>::store(out + tail, Io<V>::load(p + tail) * coef);
}

// The tensor of chunk c.
__device__ __forceinline__ int tensor_of(const ClipTable &tab, int c) {
    int a = 0, b = tab.n;  // first[a] <= c < first[b]
    while (b - a > 1) {
        const int m = (a + b) / 2;
        if (tab.first[m] <= c)
            a = m;
        else
            b = m;
    }
    return a;
}

// The sum of `v` over the CTA, in a fixed order; in every thread.
__device__ double cta_sum(double v) {
    __shared__ double part[kClipThreads / 32];
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    __syncthreads();
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    double sum = 0;
    for (int i = 0; i < kClipThreads / 32; ++i) sum += part[i];
    return sum;
}

// partial[blockIdx.x] = the sum of the squares of this CTA's chunks.
__global__ void __launch_bounds__(kClipThreads) grad_square_kernel(const __grid_constant__ ClipTable tab, double *partial) {
    grid_dependency_wait();
    grid_launch_dependents();
    double sum = 0;
    for (int64_t c = blockIdx.x; c < tab.first[tab.n]; c += gridDim.x) {
        const int i = tensor_of(tab, (int)c);
        const int64_t begin = (c - tab.first[i]) * tab.chunk;
        const int64_t n = min((int64_t)tab.chunk, tab.numel[i] - begin);
        if (tab.dtype[i] == EP_F32)
            sum += square_sum(static_cast<const float *>(tab.data[i]) + begin, n);
        else if (tab.dtype[i] == EP_BF16)
            sum += square_sum(static_cast<const __nv_bfloat16 *>(tab.data[i]) + begin, n);
        else
            sum += square_sum(static_cast<const __half *>(tab.data[i]) + begin, n);
    }
    sum = cta_sum(sum);
    if (threadIdx.x == 0) partial[blockIdx.x] = sum;
}

// norm = sqrt of the partials' sum; out = data * min(1, max_norm / (norm + 1e-6)). Every CTA adds
// the partials up for itself, all in the same order. Chunks are taken from the last to the first:
// the last ones are what the sum of squares read last, and so what the L2 cache still holds.
__global__ void __launch_bounds__(kClipThreads) grad_scale_kernel(const __grid_constant__ ClipTable tab,
                                                                  const double *partial, int partials, float max_norm,
                                                                  float *norm) {
    grid_dependency_wait();
    grid_launch_dependents();
    double v = 0;
    for (int i = threadIdx.x; i < partials; i += kClipThreads) v += partial[i];
    const float total = (float)sqrt(cta_sum(v));
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    if (tab.n == 0) return;
    float coef = max_norm / (total + 1e-6f);
    if (coef > 1.0f) coef = 1.0f;  // a NaN stays one
    for (int64_t c = (int64_t)tab.first[tab.n] - 1 - blockIdx.x; c >= 0; c -= gridDim.x) {
        const int i = tensor_of(tab, (int)c);
        if (coef == 1.0f && tab.out[i] == tab.data[i]) continue;  // in place, and nothing to change
        const int64_t begin = (c - tab.first[i]) * tab.chunk;
        const int64_t n = min((int64_t)tab.chunk, tab.numel[i] - begin);
        if (tab.dtype[i] == EP_F32)
            scale_values(static_cast<const float *>(tab.data[i]) + begin, static_cast<float *>(tab.out[i]) + begin, n, coef);
        else if (tab.dtype[i] == EP_BF16)
            scale_values(static_cast<const __nv_bfloat16 *>(tab.data[i]) + begin,
                         static_cast<__nv_bfloat16 *>(tab.out[i]) + begin, n, coef);
        else
            scale_values(static_cast<const __half *>(tab.data[i]) + begin, static_cast<__half *>(tab.out[i]) + begin, n, coef);
    }
}

// Fills `tab` with the tensors from `from` on that are not empty; returns the index after the last.
int32_t fill_table(ClipTable &tab, const ep_grad_tensor *t, int32_t n, int32_t from) {
    int64_t values = 0;
    int32_t i = from;
    tab.n = 0;
    for (; i < n && tab.n < kClipTensors; ++i) {
        if (t[i].numel == 0) continue;
        tab.data[tab.n] = t[i].data;
        tab.out[tab.n] = t[i].out;
        tab.numel[tab.n] = t[i].numel;
        tab.dtype[tab.n++] = (uint8_t)t[i].dtype;
        values += t[i].numel;
    }
    // at most about 16 chunks for every CTA, so that the last ones leave little of the GPU idle;
    // a chunk stays below 2^20 values unless their number would not fit an int
    int64_t chunk = 4096;
    while (chunk < (1 << 20) && values / chunk > (int64_t)kClipGrid * 16) chunk *= 2;
    while (values / chunk + tab.n > INT32_MAX) chunk *= 2;
    int64_t first = 0;
    for (int32_t j = 0; j < tab.n; ++j) {
        tab.first[j] = (int32_t)first;
        first += (tab.numel[j] + chunk - 1) / chunk;
    }
    tab.first[tab.n] = (int32_t)first;
    tab.chunk = (int32_t)chunk;
    return i;
}

}  // namespace

size_t grad_workspace_bytes(int32_t n) {
    const size_t launches = n > 0 ? ((size_t)n + kClipTensors - 1) / kClipTensors : 1;
    return launches * (size_t)kClipGrid * sizeof(double);
}

cudaError_t launch_grad_clip(const ep_grad_tensor *t, int32_t n, bool scale, float max_norm, float *norm, double *partial,
                             cudaStream_t s) {
    ClipTable tab;
    int partials = 0;
    for (int32_t i = 0; i < n;) {
        i = fill_table(tab, t, n, i);
        if (tab.n == 0) break;
        const int grid = tab.first[tab.n] < kClipGrid ? tab.first[tab.n] : kClipGrid;
        const cudaError_t e = launch_dependent(grad_square_kernel, dim3(grid), dim3(kClipThreads), 0, s, tab, partial + partials);
        if (e != cudaSuccess) return e;
        partials += grid;
    }
    // with nothing to scale one CTA still writes the norm
    int32_t i = 0;
    do {
        tab.n = 0;
        tab.first[0] = 0;
        if (scale && n > 0) i = fill_table(tab, t, n, i);
        const int grid = tab.n == 0 ? 1 : tab.first[tab.n] < kClipGrid ? tab.first[tab.n] : kClipGrid;
        const cudaError_t e = launch_dependent(grad_scale_kernel, dim3(grid), dim3(kClipThreads), 0, s, tab,
                                               const_cast<const double *>(partial), partials, max_norm, norm);
        if (e != cudaSuccess) return e;
    } while (scale && i < n);
    return cudaSuccess;
}

}  // namespace ep
