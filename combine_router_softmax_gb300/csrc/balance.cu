// balance.cu -- the router's balance loss, the squared log-sum-exp loss, per-expert counts, and their gradient.
//
// Every row's softmax is a warp's: the logits are read once, a lane holds every 32nd. The sums over a
// sequence's rows are formed in registers, joined in shared memory, and left as one row of partial sums for
// every pair of a tile of rows and a sequence that meet; a second kernel adds those up. Tile i and sequence s
// write row i + s: as both only grow along the rows, no two pairs share one.
#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kBalWarps = 8;
constexpr int kBalThreads = 32 * kBalWarps;
constexpr int kFinishThreads = 1024;

struct Sequences {
    const int32_t *first, *len;
    int32_t n, T;
    __device__ __forceinline__ int begin(int s) const { return first ? min(max(first[s], 0), T) : 0; }
    __device__ __forceinline__ int end(int s) const {
        if (!first) return T;
        const int b = begin(s);
        const int e = max(min(max(first[s + 1], 0), T), b);
        return len ? (int)min((int64_t)e, (int64_t)b + max(len[s], 0)) : e;
    }
    // The last sequence that begins at or before `row`; -1: none.
    __device__ __forceinline__ int find(int row) const {
        if (!first) return 0;
        int lo = 0, hi = n;  // the first that begins after it lies in [lo, hi]
        while (lo < hi) {
            const int mid = lo + (hi - lo) / 2;
            if (begin(mid) <= row)
                lo = mid + 1;
            else
                hi = mid;
        }
        return lo - 1;
    }
};

struct Partials {
    float *prob, *z;  // [rows][E], [rows]
    int32_t *count;   // [rows][E]
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
}

template <int VPL>
__device__ __forceinline__ void load_row(const float *l, int E, int lane, float (&p)[VPL]) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = i * 32 + lane < E ? l[i * 32 + lane] : -INFINITY;
}
// The softmax of a row in place; the log of the sum of exponentials. All zero where nothing is above -infinity.
template <int VPL>
__device__ __forceinline__ float softmax_row(float (&p)[VPL]) {
    float top = p[0], sum = 0.0f;
#pragma unroll
    for (int i = 1; i < VPL; ++i) top = fmaxf(top, p[i]);
    top = warp_max(top);
    const float base = top == -INFINITY ? 0.0f : top;  // exp(-inf - 0) = 0
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        p[i] = __expf(p[i] - base);
        sum += p[i];
    }
    sum = warp_sum(sum);
    if (sum == 0.0f) return 0.0f;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] *= inv;
    return base + logf(sum);
}

template <int VPL>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(Sequences seq, int E, int k, int tile_rows, const float *logits,
                                                              const int32_t *idx, Partials part) {
    extern __shared__ unsigned char smem[];
    float *sums = reinterpret_cast<float *>(smem);                  // [warp][E]
    int32_t *count = reinterpret_cast<int32_t *>(sums + kBalWarps * E);  // [E]
    __shared__ float z_sums[kBalWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t begin64 = (int64_t)blockIdx.x * tile_rows;
    const int begin = (int)begin64, end = (int)min(begin64 + tile_rows, (int64_t)seq.T);
    for (int s = max(seq.find(begin), 0); s < seq.n; ++s) {
        if (seq.begin(s) >= end) break;
        const int lo = max(seq.begin(s), begin), hi = min(seq.end(s), end);
        if (lo >= hi) continue;
        for (int e = threadIdx.x; e < E; e += kBalThreads) count[e] = 0;
        __syncthreads();
        for (int64_t i = (int64_t)lo * k + threadIdx.x; i < (int64_t)hi * k; i += kBalThreads) {
            const int e = idx[i];
            if (e >= 0 && e < E) atomicAdd(&count[e], 1);
        }
        float acc[VPL], z = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) acc[i] = 0.0f;
        for (int64_t t = lo + warp; t < hi; t += kBalWarps) {
            float p[VPL];
            load_row(logits + (size_t)t * E, E, lane, p);
            const float lse = softmax_row(p);
            z = fmaf(lse, lse, z);
#pragma unroll
            for (int i = 0; i < VPL; ++i) acc[i] += p[i];
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i * 32 + lane < E) sums[warp * E + i * 32 + lane] = acc[i];
        if (lane == 0) z_sums[warp] = z;
        __syncthreads();
        const size_t row = (size_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < E; e += kBalThreads) {
            float v = 0.0f;
            for (int w = 0; w < kBalWarps; ++w) v += sums[w * E + e];
            part.prob[row * E + e] = v;
            part.count[row * E + e] = count[e];
        }
        if (threadIdx.x == 0) {
            float v = 0.0f;
            for (int w = 0; w < kBalWarps; ++w) v += z_sums[w];
            part.z[row] = v;
        }
        __syncthreads();
    }
}

// One CTA a sequence.
__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(Sequences seq, int E, int k, int tile_rows, Partials part,
                                                                        int32_t *count, float *load, float *prob, float *loss) {
    __shared__ float sums[kFinishThreads], inner[32];
    __shared__ int32_t counts[kFinishThreads];
    grid_dependency_wait();
    grid_launch_dependents();
    const int s = blockIdx.x;
    const int begin = seq.begin(s), end = seq.end(s), rows = end - begin;
    const int first = begin / tile_rows, last = rows > 0 ? (end - 1) / tile_rows : first - 1;
    const float inv = rows > 0 ? 1.0f / (float)rows : 0.0f;
    // threads: a power of two of columns, the rest of them takes the partial rows in turns
    int columns = 32;
    while (columns < E) columns *= 2;
    const int turns = kFinishThreads / columns, e = threadIdx.x % columns, turn = threadIdx.x / columns;
    float v = 0.0f;
    int32_t c = 0;
    if (e < E)
        for (int i = first + turn; i <= last; i += turns) {
            const size_t at = ((size_t)i + s) * E + e;
            v += part.prob[at];
            c += part.count[at];
        }
    sums[threadIdx.x] = v;
    counts[threadIdx.x] = c;
    __syncthreads();
    float product = 0.0f;
    if (turn == 0 && e < E) {
        for (int i = 1; i < turns; ++i) v += sums[i * columns + e], c += counts[i * columns + e];
        const float p = v * inv, f = rows > 0 ? (float)c / ((float)k * (float)rows) : 0.0f;
        count[(size_t)s * E + e] = c;
        load[(size_t)s * E + e] = f;
        prob[(size_t)s * E + e] = p;
        product = f * p;
    }
    product = warp_sum(product);
    if (threadIdx.x % 32 == 0) inner[threadIdx.x / 32] = product;
    __syncthreads();
    if (threadIdx.x < 32) {
        product = warp_sum(inner[threadIdx.x]);
        float z = 0.0f;
        for (int i = first + threadIdx.x; i <= last; i += 32) z += part.z[(size_t)i + s];
        z = warp_sum(z);
        if (threadIdx.x == 0) {
            loss[2 * (size_t)s] = (float)E * product;
            loss[2 * (size_t)s + 1] = z * inv;
        }
    }
}

// A warp takes `rows` consecutive rows.
template <int VPL>
__global__ void __launch_bounds__(kBalThreads) balance_backward_kernel(Sequences seq, int E, int rows, const float *logits,
                                                                       const float *load, const float *d_loss,
                                                                       const float *d_in, float *d_logits) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32;
    const int64_t first = ((int64_t)blockIdx.x * kBalWarps + threadIdx.x / 32) * rows;
    const int64_t stop = min(first + rows, (int64_t)seq.T);
    int begin = 0, end = 0;  // of the sequence that f, c0 and c1 are of
    float f[VPL], c0 = 0.0f, c1 = 0.0f;
    for (int64_t t64 = first; t64 < stop; ++t64) {
        const int t = (int)t64;
        float p[VPL], d[VPL];
        load_row(logits + (size_t)t * E, E, lane, p);
#pragma unroll
        for (int i = 0; i < VPL; ++i) d[i] = d_in && i * 32 + lane < E ? d_in[(size_t)t * E + i * 32 + lane] : 0.0f;
        if (t < begin || t >= end) {
            const int s = seq.find(t);
            begin = end = 0;
            if (s >= 0 && t < seq.end(s)) {
                begin = seq.begin(s), end = seq.end(s);
                const float inv = 1.0f / (float)(end - begin);
                c0 = d_loss[2 * (size_t)s] * (float)E * inv;
                c1 = 2.0f * d_loss[2 * (size_t)s + 1] * inv;
#pragma unroll
                for (int i = 0; i < VPL; ++i) f[i] = i * 32 + lane < E ? load[(size_t)s * E + i * 32 + lane] : 0.0f;
            }
        }
        if (end > begin) {
            const float lse = softmax_row(p);
            float mean = 0.0f;
#pragma unroll
            for (int i = 0; i < VPL; ++i) mean = fmaf(f[i], p[i], mean);
            mean = warp_sum(mean);
#pragma unroll
            for (int i = 0; i < VPL; ++i) d[i] = fmaf(p[i], fmaf(c0, f[i] - mean, c1 * lse), d[i]);
        }
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (i * 32 + lane < E) d_logits[(size_t)t * E + i * 32 + lane] = d[i];
    }
}

// Rows of a tile: two tiles for every SM where there are enough rows, and no fewer than two rows a warp.
int tile_rows(const ep_config &c) {
    const int64_t sms = 152;
    const int64_t rows = (c.T + 2 * sms - 1) / (2 * sms);
    return (int)(rows < 2 * kBalWarps ? 2 * kBalWarps : rows);
}
int tiles(const ep_config &c) { return (c.T + tile_rows(c) - 1) / tile_rows(c); }

template <int VPL>
cudaError_t run_balance(const ep_config &c, const Sequences &seq, const float *logits, const int32_t *idx, const Partials &part,
                        cudaStream_t s) {
    const size_t smem = (size_t)(kBalWarps + 1) * c.E * sizeof(float);
    return launch_dependent(balance_kernel<VPL>, dim3((unsigned)tiles(c)), dim3(kBalThreads), smem, s, seq, c.E, c.k, tile_rows(c),
                            logits, idx, part);
}
template <int VPL>
cudaError_t run_backward(const ep_config &c, const Sequences &seq, const float *logits, const float *load, const float *d_loss,
                         const float *d_in, float *d_logits, cudaStream_t s) {
    const int rows = c.T >= 16384 ? 4 : 1;
    const int64_t warps = ((int64_t)c.T + rows - 1) / rows;
    return launch_dependent(balance_backward_kernel<VPL>, dim3((unsigned)((warps + kBalWarps - 1) / kBalWarps)), dim3(kBalThreads),
                            0, s, seq, c.E, rows, logits, load, d_loss, d_in, d_logits);
}

}  // namespace

size_t balance_workspace_bytes(const ep_config &c, int32_t n_seq) {
    return ((size_t)tiles(c) + (size_t)n_seq) * (2 * (size_t)c.E + 1) * sizeof(float);
}

cudaError_t launch_balance(const ep_config &c, int32_t n_seq, const float *logits, const int32_t *idx, const int32_t *seq_first,
                           const int32_t *seq_len, int32_t *count, float *load, float *prob, float *loss, void *workspace,
                           cudaStream_t s) {
    const Sequences seq{seq_first, seq_len, n_seq, c.T};
    const size_t rows = (size_t)tiles(c) + (size_t)n_seq;
    Partials part;
    part.prob = static_cast<float *>(workspace);
    part.count = reinterpret_cast<int32_t *>(part.prob + rows * c.E);
    part.z = reinterpret_cast<float *>(part.count + rows * c.E);
    if (c.T > 0) {
        const cudaError_t e = c.E <= 32    ? run_balance<1>(c, seq, logits, idx, part, s)
                              : c.E <= 128 ? run_balance<4>(c, seq, logits, idx, part, s)
                              : c.E <= 256 ? run_balance<8>(c, seq, logits, idx, part, s)
                                           : run_balance<kMaxE / 32>(c, seq, logits, idx, part, s);
        if (e != cudaSuccess) return e;
    }
    return launch_dependent(balance_finish_kernel, dim3((unsigned)n_seq), dim3(kFinishThreads), 0, s, seq, c.E, c.k, tile_rows(c),
                            part, count, load, prob, loss);
}

cudaError_t launch_balance_backward(const ep_config &c, int32_t n_seq, const float *logits, const int32_t *seq_first,
                                    const int32_t *seq_len, const float *load, const float *d_loss, const float *d_in,
                                    float *d_logits, cudaStream_t s) {
    const Sequences seq{seq_first, seq_len, n_seq, c.T};
    if (c.E <= 32) return run_backward<1>(c, seq, logits, load, d_loss, d_in, d_logits, s);
    if (c.E <= 128) return run_backward<4>(c, seq, logits, load, d_loss, d_in, d_logits, s);
    if (c.E <= 256) return run_backward<8>(c, seq, logits, load, d_loss, d_in, d_logits, s);
    return run_backward<kMaxE / 32>(c, seq, logits, load, d_loss, d_in, d_logits, s);
}

}  // namespace ep
