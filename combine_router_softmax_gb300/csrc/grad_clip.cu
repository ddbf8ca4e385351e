// grad_clip.cu -- the global norm of many gradient tensors, and clipping by it.
//
// norm = sqrt(sum g^2) needs every value before the first can be scaled: two kernels, the values read
// twice and written once (the second alone where the norm is given). HBM bounds them where the tensors are large (0.8 GB in and out: 378 us, of
// which the three crossings need 358 at the measured copy rate), the two launches where they are
// small (300 tensors, 14 MB: 14 us).
#include "values.cuh"

namespace ep {

namespace {

constexpr int kClipThreads = 512;
constexpr int kClipTensors = 768;  // tensors of one launch: their table is a kernel argument
// The largest grid of either kernel: four CTAs of 512 threads fill an SM, on 152 of them.
constexpr int kClipGrid = 4 * 152;

// The tensors of a launch. Work is dealt out in chunks of `chunk` values of one tensor; a CTA takes
// consecutive ones, from chunk `at` of tensor `tensor` on, up to where the next CTA begins.
struct ClipTable {
    const void *data[kClipTensors];
    void *out[kClipTensors];
    int64_t numel[kClipTensors];
    int32_t at[kClipGrid + 1];
    uint16_t tensor[kClipGrid + 1];
    uint8_t dtype[kClipTensors];
    int32_t n, chunk, grid;
};
static_assert(sizeof(ClipTable) + 64 <= 32764, "kernel arguments");

// The sum of the squares of n values (SCALED: times `scale`), this thread's part: four independent sums of
// fp32, of at most chunk / kClipThreads / 4 values each. `bits` gets those of all values' magnitudes.
template <bool SCALED, typename V>
__device__ __forceinline__ float square_sum(const V *p, int n, float scale, uint32_t &bits) {
    constexpr int kVec = Io<V>::kVec;
    float acc[4] = {0, 0, 0, 0};
    const int head = min((int)values_to_boundary(p), n);
    if (threadIdx.x < head) {
        const float v = Io<V>::load(p + threadIdx.x) * (SCALED ? scale : 1.0f);
        acc[0] = v * v;
        bits |= __float_as_uint(v) << 1;
    }
    const uint4 *q = reinterpret_cast<const uint4 *>(p + head);
    const int vecs = (n - head) / kVec;
    uint32_t words = 0;
#pragma unroll(SCALED ? 1 : 4)
    for (int i = threadIdx.x; i < vecs; i += kClipThreads) {
        const uint4 w = q[i];
        float v[kVec];
        Io<V>::unpack(w, v);
        words |= w.x | w.y | w.z | w.w;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            if (SCALED) v[j] *= scale;
            acc[j % 4] = fmaf(v[j], v[j], acc[j % 4]);
        }
    }
    const int tail = head + vecs * kVec + threadIdx.x;
    if (tail < n) {
        const float v = Io<V>::load(p + tail) * (SCALED ? scale : 1.0f);
        acc[1] = fmaf(v, v, acc[1]);
        bits |= __float_as_uint(v) << 1;
    }
    bits |= words & (sizeof(V) == 2 ? 0x7FFF7FFFu : 0x7FFFFFFFu);  // without the signs
    return (acc[0] + acc[1]) + (acc[2] + acc[3]);
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

// A tensor as the kernels hold it.
struct ClipTensor {
    const void *data;
    void *out;
    int64_t numel;
    int32_t chunks;
    uint8_t dtype;
    __device__ ClipTensor(const ClipTable &tab, int i)
        : data(tab.data[i]), out(tab.out[i]), numel(tab.numel[i]),
          chunks((int32_t)((tab.numel[i] + tab.chunk - 1) / tab.chunk)), dtype(tab.dtype[i]) {}
};

// The sum of `v` over the CTA as a tree; in thread 0.
__device__ float cta_sum(float v) {
    __shared__ float part[kClipThreads / 32];
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
    __syncthreads();
    if (threadIdx.x >= 32) return 0;
    v = threadIdx.x < kClipThreads / 32 ? part[threadIdx.x] : 0.0f;
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}

// This thread's part of the sum of the squares of the CTA's chunks.
template <bool SCALED>
__device__ __forceinline__ float share_sum(const ClipTable &tab, float scale, uint32_t &bits) {
    float sum = 0;
    const int end_tensor = tab.tensor[blockIdx.x + 1], end_at = tab.at[blockIdx.x + 1];
    int i = tab.tensor[blockIdx.x], c = tab.at[blockIdx.x];
    while (i < end_tensor || (i == end_tensor && c < end_at)) {
        const ClipTensor t(tab, i);
        const int stop = i < end_tensor ? t.chunks : end_at;
        const int64_t begin = (int64_t)c * tab.chunk, end = min((int64_t)stop * tab.chunk, t.numel);
        // chunk by chunk, so that no fp32 sum grows long
        for (int64_t v = begin; v < end; v += tab.chunk) {
            const int n = (int)min((int64_t)tab.chunk, end - v);
            if (t.dtype == EP_F32)
                sum += square_sum<SCALED>(static_cast<const float *>(t.data) + v, n, scale, bits);
            else if (t.dtype == EP_BF16)
                sum += square_sum<SCALED>(static_cast<const __nv_bfloat16 *>(t.data) + v, n, scale, bits);
            else
                sum += square_sum<SCALED>(static_cast<const __half *>(t.data) + v, n, scale, bits);
        }
        ++i;
        c = 0;
    }
    return sum;
}
__device__ __noinline__ float scaled_share_sum(const ClipTable &tab, float scale) {
    uint32_t bits = 0;
    return share_sum<true>(tab, scale, bits);
}

// partial[blockIdx.x] = the sum of the squares of this CTA's chunks. fp32 up to the CTA's sum: the chains are
// short (some hundred steps in a thread, ten in the tree), and the 64-bit units are few: with the
// tree in 64 bits it took longer than the values (300 tensors, 14 MB, both kernels: 36 us).
// Where the squares leave fp32's range the CTA reads its values again, times 2^90 or 2^-90. Below kLeast the
// squares lost, each by half of fp32's smallest step, 2^-150, of up to 2^40 values could be 2^-20 of the sum;
// above kMost some may have overflowed. Zeros are told from values that are lost by their bits.
// Four CTAs an SM, as many as the grid has, leave 32 registers a thread; with three, 0.8 GB take 5% longer.
constexpr float kLeast = 0x1p-90f, kMost = 0x1p126f;

__global__ void __launch_bounds__(kClipThreads, 4) grad_square_kernel(const __grid_constant__ ClipTable tab, double *partial) {
    __shared__ int scale_by;
    grid_dependency_wait();
    grid_launch_dependents();
    uint32_t bits = 0;
    const float mine = share_sum<false>(tab, 1.0f, bits);
    const bool values = __syncthreads_or(bits != 0);
    const float sum = cta_sum(mine);
    if (threadIdx.x == 0) {
        partial[blockIdx.x] = sum;
        scale_by = sum < kLeast ? values ? 1 : 0 : sum <= kMost ? 0 : -1;  // -1: also infinities and NaN
    }
    __syncthreads();
    if (scale_by != 0) {
        const float scaled = cta_sum(scaled_share_sum(tab, scale_by > 0 ? 0x1p90f : 0x1p-90f));
        if (threadIdx.x == 0) partial[blockIdx.x] = scaled * (scale_by > 0 ? 0x1p-180 : 0x1p180);
    }
}

// norm = sqrt of the partials' sum, or the one that is given; out = data * min(1, max_norm / (norm + 1e-6)). Every
// CTA adds the partials up for itself, all in the same order. A CTA takes its chunks from the last to the
// first: the last ones are what the sum of squares read last, and so what the L2 cache still holds.
__global__ void __launch_bounds__(kClipThreads) grad_scale_kernel(const __grid_constant__ ClipTable tab,
                                                                  const double *partial, int partials, float max_norm,
                                                                  float *norm, const float *given) {
    grid_dependency_wait();
    grid_launch_dependents();
    __shared__ float total_shared;
    if (given) {
        if (threadIdx.x == 0) total_shared = *given;
    } else if (threadIdx.x < 32) {  // one warp, in 64 bits: the CTAs' sums may be many
        double v = 0;
        for (int i = threadIdx.x; i < partials; i += 32) v += partial[i];
        for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
        if (threadIdx.x == 0) total_shared = (float)sqrt(v);
    }
    __syncthreads();
    const float total = total_shared;
    if (!given && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
    if (tab.n == 0) return;
    float coef = max_norm / (total + 1e-6f);
    if (coef > 1.0f) coef = 1.0f;  // a NaN stays one
    const int first_tensor = tab.tensor[blockIdx.x], first_at = tab.at[blockIdx.x];
    int i = tab.tensor[blockIdx.x + 1], c = tab.at[blockIdx.x + 1];  // c: one past the chunk to take next
    while (i > first_tensor || (i == first_tensor && c > first_at)) {
        if (c == 0) {
            --i;
            c = (int)((tab.numel[i] + tab.chunk - 1) / tab.chunk);
            continue;
        }
        const ClipTensor t(tab, i);
        const int stop = i > first_tensor ? 0 : first_at;
        if (coef != 1.0f || t.out != t.data)  // else in place, and nothing to change
            for (int k = c - 1; k >= stop; --k) {
                const int64_t v = (int64_t)k * tab.chunk;
                const int64_t n = min((int64_t)tab.chunk, t.numel - v);
                if (t.dtype == EP_F32)
                    scale_values(static_cast<const float *>(t.data) + v, static_cast<float *>(t.out) + v, n, coef);
                else if (t.dtype == EP_BF16)
                    scale_values(static_cast<const __nv_bfloat16 *>(t.data) + v, static_cast<__nv_bfloat16 *>(t.out) + v, n, coef);
                else
                    scale_values(static_cast<const __half *>(t.data) + v, static_cast<__half *>(t.out) + v, n, coef);
            }
        c = stop;
        if (i == first_tensor) break;
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
    // at most about 16 chunks for every CTA, so that their shares differ little; a chunk stays at
    // most 2^20 values unless their number would not fit an int
    int64_t chunk = 4096;
    while (chunk < (1 << 20) && values / chunk > (int64_t)kClipGrid * 16) chunk *= 2;
    while (values / chunk + tab.n > INT32_MAX) chunk *= 2;
    int64_t total = 0;
    for (int32_t j = 0; j < tab.n; ++j) total += (tab.numel[j] + chunk - 1) / chunk;
    tab.chunk = (int32_t)chunk;
    tab.grid = (int32_t)(total < kClipGrid ? total : kClipGrid);
    int64_t before = 0;  // chunks before tensor j
    int32_t j = 0;
    for (int32_t b = 0; b <= tab.grid; ++b) {
        const int64_t c = tab.grid > 0 ? total * b / tab.grid : 0;
        while (j < tab.n && before + (tab.numel[j] + chunk - 1) / chunk <= c) before += (tab.numel[j++] + chunk - 1) / chunk;
        tab.tensor[b] = (uint16_t)j;
        tab.at[b] = (int32_t)(c - before);
    }
    return i;
}

}  // namespace

size_t grad_workspace_bytes(int32_t n) {
    const size_t launches = n > 0 ? ((size_t)n + kClipTensors - 1) / kClipTensors : 1;
    return launches * (size_t)kClipGrid * sizeof(double);
}

namespace {

// One launch with the table passed by address: it is large, and copied once, by the runtime.
cudaError_t launch_clip(const void *kernel, int grid, void **args, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kClipThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

}  // namespace

cudaError_t launch_grad_clip(const ep_grad_tensor *t, int32_t n, bool scale, float max_norm, float *norm, double *partial,
                             cudaStream_t s) {
    ClipTable tab;
    tab.n = 0;
    int partials = 0;
    int32_t filled_from = -1;  // the first tensor of what `tab` holds
    for (int32_t i = 0; i < n;) {
        filled_from = i;
        i = fill_table(tab, t, n, i);
        if (tab.n == 0) break;
        double *to = partial + partials;
        void *args[] = {&tab, &to};
        const cudaError_t e = launch_clip((const void *)grad_square_kernel, tab.grid, args, s);
        if (e != cudaSuccess) return e;
        partials += tab.grid;
    }
    // with nothing to scale one CTA still writes the norm
    int32_t i = 0;
    do {
        if (!scale)
            tab.n = 0;
        else if (n > 0 && i == 0 && filled_from == 0)  // the only launch's: still there
            i = n;
        else if (n > 0)
            i = fill_table(tab, t, n, i);
        const double *sums = partial;
        const float *given = nullptr;
        void *args[] = {&tab, &sums, &partials, &max_norm, &norm, &given};
        const cudaError_t e = launch_clip((const void *)grad_scale_kernel, tab.n == 0 ? 1 : tab.grid, args, s);
        if (e != cudaSuccess) return e;
    } while (scale && i < n);
    return cudaSuccess;
}

cudaError_t launch_grad_scale(const ep_grad_tensor *t, int32_t n, float max_norm, const float *norm, cudaStream_t s) {
    ClipTable tab;
    for (int32_t i = 0; i < n;) {
        i = fill_table(tab, t, n, i);
        if (tab.n == 0) break;
        const double *sums = nullptr;
        int partials = 0;
        float *out = nullptr;
        void *args[] = {&tab, &sums, &partials, &max_norm, &out, &norm};
        const cudaError_t e = launch_clip((const void *)grad_scale_kernel, tab.grid, args, s);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace ep
