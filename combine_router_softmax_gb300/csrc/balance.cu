// balance.cu -- the router's balance loss, the squared log-sum-exp loss, per-expert counts, and their gradient.
//
// Every row's softmax is 2 to 32 lanes': the logits are read once, each lane holding some. The sums over a
// sequence's rows are formed in registers, joined in shared memory, and left as one row of partial sums for
// every pair of a tile of rows and a sequence that meet; a second kernel adds those up. Tile i and sequence s
// write row i + s: as both only grow along the rows, no two pairs share one. The gradient computes the softmax again.
//
// HBM bounds both at many rows, the launches and a chain of dependent loads at few: forward 128 rows 3.4 us, 32768 x
// 256 15.4 (of which joining the partial sums 5; 5.1 for its bytes at the copy rate), 131072 x 128 in 64 sequences 24.1
// (10.5); backward 1.9, 18.1 (14.8), 25.2 (19.8).
#include "pairs.cuh"
#include "tcgen05.cuh"  // clusters

namespace ep {

namespace {

constexpr int kBalWarps = 8;  // of a CTA of the backward pass
constexpr int kBalThreads = 32 * kBalWarps;
constexpr int kSumThreads = 384;      // of a large CTA of the forward pass: two an SM with 80 registers
constexpr int kShortThreads = 256;
constexpr int kFinishThreads = 1024;  // at most

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
    // The last sequence that begins at or before `row`, if it is one's (its bounds are asked then); -1: none. By a warp: every lane looks at one of 32 places
    // at a time, as a search by halves is a chain of twice to five times as many loads.
    __device__ __forceinline__ int find(int row) const {
        if (!first || n == 1) return 0;  // its bounds say the rest
        int lo = 0, hi = n;  // the first that begins after it lies in [lo, hi]
        while (lo < hi) {
            const int step = (hi - lo + 31) / 32;
            const int64_t at = lo + (int64_t)(threadIdx.x % 32) * step;
            const int c = __popc(__ballot_sync(0xFFFFFFFFu, at < hi && begin((int)at) <= row));
            if (c == 0) break;
            const int next = lo + (c - 1) * step + 1;
            hi = (int)min((int64_t)hi, lo + (int64_t)c * step);
            lo = next;
        }
        return lo - 1;
    }
    // The same by each lane for itself.
    __device__ __forceinline__ int find_alone(int row) const {
        if (!first || n == 1) return 0;
        int lo = 0, hi = n;
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

// What stands in v stays there unless `in`. By a predicate: behind a branch for each of them the loads of a row would not go
// out together, and with clamped addresses and selections each has an address of its own (50000 rows of 150, forward and
// backward, 35 and 49 us instead of 19 and 22).
__device__ __forceinline__ void load_if(float &v, const float *p, bool in) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q ld.global.f32 %0, [%1];\n\t}" : "+f"(v) : "l"(p), "r"((int)in) : "memory");
}
__device__ __forceinline__ void load_if(uint64_t &v, uint64_t &w, const float *p, bool in) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %3, 0;\n\t@q ld.global.v2.b64 {%0, %1}, [%2];\n\t}" : "+l"(v), "+l"(w) : "l"(p), "r"((int)in) : "memory");
}

// A row of logits over L lanes, NQ times four to a lane, so that a warp takes 32 / L rows together: what the
// instructions are that a row takes whatever its length (shuffles, a logarithm, a quotient) is shared by them
// (131072 rows of 128: 34 us by whole warps, which issue 120 instructions a row, 20 by 8 lanes). WIDE: rows begin on
// 16-byte boundaries, and the four are neighbours; else they lie L apart, so that lanes read neighbours.
template <int L, int NQ, bool WIDE>
struct Row {
    static constexpr int kRows = 32 / L;
    uint64_t v[2 * NQ];  // pairs
    static __device__ __forceinline__ int element(int i, int j) {
        const int lane = threadIdx.x % L;
        return WIDE ? (i * L + lane) * 4 + j : (i * 4 + j) * L + lane;
    }
    // The row at p; `none` where it has no element, and throughout unless `in`.
    __device__ __forceinline__ void load(const float *p, int E, bool in, float none) {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if constexpr (WIDE) {
                const int e = element(i, 0);
                v[2 * i] = v[2 * i + 1] = pair(none, none);
                load_if(v[2 * i], v[2 * i + 1], p + e, in && e < E);
            } else {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = none;
                    load_if(x[j], p + element(i, j), in && element(i, j) < E);
                }
                v[2 * i] = pair(x[0], x[1]), v[2 * i + 1] = pair(x[2], x[3]);
            }
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 2 * NQ; ++i) v[i] = 0;
    }
    __device__ __forceinline__ void store(float *p, int E) const {
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            if constexpr (WIDE) {
                if (element(i, 0) < E) *reinterpret_cast<ulonglong2 *>(p + element(i, 0)) = make_ulonglong2(v[2 * i], v[2 * i + 1]);
            } else {
                const float x[4] = {low(v[2 * i]), high(v[2 * i]), low(v[2 * i + 1]), high(v[2 * i + 1])};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (element(i, j) < E) p[element(i, j)] = x[j];
            }
        }
    }
};
// exp2 of what is at most 0; results below fp32's normal range count as 0. Of a probability's 2^-21 that this and the quotient
// leave, the mean over a sequence keeps less: the losses of 32768 x 256 are 1.5e-7 off, 1.2e-7 with 64-bit sums of exact
// exponentials rounded to fp32. So sums are fp32 too: a lane's are of some hundred rows at most at any usual size, the rest a tree.
__device__ __forceinline__ float exp2_flushed(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// exp(l - top) in place, top the row's largest value, and their sum, this lane's part.
template <int L, int NQ, bool WIDE>
__device__ __forceinline__ float exponentials(Row<L, NQ, WIDE> &r, float &top) {
    top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2 * NQ; ++i) top = fmaxf(top, fmaxf(low(r.v[i]), high(r.v[i])));
#pragma unroll
    for (int d = L / 2; d > 0; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
    top = top == -INFINITY ? 0.0f : top;  // exp(-inf - 0) = 0
    const uint64_t base = pair(-top, -top), log2e = pair(1.44269504f, 1.44269504f);
    uint64_t sum = 0;
#pragma unroll
    for (int i = 0; i < 2 * NQ; ++i) {
        // the difference first: it is exact near the top, where the large terms are
        const uint64_t x = mul2(add2(r.v[i], base), log2e);
        r.v[i] = pair(exp2_flushed(low(x)), exp2_flushed(high(x)));
        sum = add2(sum, r.v[i]);
    }
    return total(sum);
}

// The sums of a CTA over rows first + i step, i = 0, 1, ..., below hi (`first` is this lane's) and over the ids
// [id, id_end) in steps of `id_step`: probabilities to sums[0][E], counts to count[E], the squared log-sum-exps returned in
// thread 0. sums: [warp][E] of shared memory.
template <int L, int NQ, bool WIDE>
__device__ __forceinline__ float sum_rows(const float *logits, const int32_t *idx, int E, int64_t t, int64_t step, int hi, int64_t id,
                                          int64_t id_step, int64_t id_end, float *sums, int32_t *count, float *z_sums) {
    using R = Row<L, NQ, WIDE>;
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, threads = blockDim.x, warps = threads / 32;
    R next;  // asked for ahead
    const auto ask = [&](int64_t t) { next.load(logits + (size_t)min(t, (int64_t)hi - 1) * E, E, t < hi, -INFINITY); };
    ask(t);
    for (int e = threadIdx.x; e < E; e += threads) count[e] = 0;
    __syncthreads();
    for (; id < id_end; id += 8 * id_step) {
        int e[8];  // asked for together
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = id + j * id_step < id_end ? idx[id + j * id_step] : -1;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (e[j] >= 0 && e[j] < E) atomicAdd(&count[e[j]], 1);
    }
    R acc;
    float z = 0.0f;
    acc.clear();
    for (; t - lane / L < hi; t += step) {  // all lanes alike
        R r = next;
        ask(t + step);
        float top, sum = exponentials(r, top);
#pragma unroll
        for (int d = L / 2; d > 0; d /= 2) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        const float inv = sum == 0.0f ? 0.0f : __fdividef(1.0f, sum);  // 0: no row
        const float lse = sum == 0.0f ? 0.0f : top + __logf(sum);
        z = fmaf(lse, lse, z);
        const uint64_t inv2 = pair(inv, inv);
#pragma unroll
        for (int i = 0; i < 2 * NQ; ++i) acc.v[i] = fma2(r.v[i], inv2, acc.v[i]);
    }
    // over the warp's rows, then over the warps
    z = lane % L == 0 ? z : 0.0f;
#pragma unroll
    for (int d = 16; d >= L; d /= 2) {
        z += __shfl_xor_sync(0xFFFFFFFFu, z, d);
#pragma unroll
        for (int i = 0; i < 2 * NQ; ++i) acc.v[i] = add2(acc.v[i], __shfl_xor_sync(0xFFFFFFFFu, acc.v[i], d));
    }
    if (lane < L) acc.store(sums + warp * E, E);
    if (lane == 0) z_sums[warp] = z;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += threads) {
        float v = 0.0f;
#pragma unroll 8
        for (int w = 0; w < warps; ++w) v += sums[w * E + e];
        sums[e] = v;
    }
    z = 0.0f;
    if (threadIdx.x == 0)
        for (int w = 0; w < warps; ++w) z += z_sums[w];
    return z;
}

template <int L, int NQ, bool WIDE>
__global__ void __launch_bounds__(kSumThreads, NQ <= 4 ? 2 : 1) balance_kernel(Sequences seq, int E, int k, int tile_rows, const float *logits,
                                                                              const int32_t *idx, Partials part) {
    using R = Row<L, NQ, WIDE>;
    extern __shared__ __align__(16) float smem[];  // rows are stored 16 bytes at a time
    const int threads = blockDim.x, warps = threads / 32;
    float *sums = smem;                                                // [warp][E]
    int32_t *count = reinterpret_cast<int32_t *>(sums + warps * E);  // [E]
    __shared__ float z_sums[32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int64_t begin64 = (int64_t)blockIdx.x * tile_rows;
    const int begin = (int)begin64, end = (int)min(begin64 + tile_rows, (int64_t)seq.T);
    for (int s = max(seq.find(begin), 0); s < seq.n; ++s) {
        if (seq.begin(s) >= end) break;
        const int lo = max(seq.begin(s), begin), hi = min(seq.end(s), end);
        if (lo >= hi) continue;
        const float z = sum_rows<L, NQ, WIDE>(logits, idx, E, (int64_t)lo + warp * R::kRows + lane / L, warps * R::kRows, hi,
                                              (int64_t)lo * k + threadIdx.x, threads, (int64_t)hi * k, sums, count, z_sums);
        __syncthreads();
        const size_t row = (size_t)blockIdx.x + s;
        for (int e = threadIdx.x; e < E; e += threads) {
            part.prob[row * E + e] = sums[e];
            part.count[row * E + e] = count[e];
        }
        if (threadIdx.x == 0) part.z[row] = z;
        __syncthreads();
    }
}

// Sequences of some hundred rows: a cluster takes one, and nothing is left to a second kernel. The CTAs share its rows,
// then each adds up a part of the columns of all.
template <int L, int NQ, bool WIDE>
__global__ void __launch_bounds__(kShortThreads, NQ <= 4 ? 3 : 1) balance_short_kernel(Sequences seq, int E, int k, int ctas, const float *logits,
                                                                                      const int32_t *idx, int32_t *count_out, float *load,
                                                                                      float *prob, float *loss) {
    using R = Row<L, NQ, WIDE>;
    extern __shared__ __align__(16) float smem[];  // rows are stored 16 bytes at a time
    constexpr int kWarps = kShortThreads / 32;
    float *sums = smem;                                                 // [warp][E]
    int32_t *count = reinterpret_cast<int32_t *>(sums + kWarps * E);  // [E]
    __shared__ float z_sums[32], z_mine, products[8], inner[kWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const int s = blockIdx.x / ctas, rank = blockIdx.x % ctas;
    const int lo = seq.begin(s), hi = seq.end(s), rows = hi - lo;
    float z = 0.0f;
    if (rows > 0) {  // in all CTAs of the cluster alike
        z = sum_rows<L, NQ, WIDE>(logits, idx, E, lo + (int64_t)(rank * kWarps + warp) * R::kRows + lane / L,
                                  (int64_t)ctas * kWarps * R::kRows, hi, (int64_t)lo * k + rank * kShortThreads + threadIdx.x,
                                  (int64_t)ctas * kShortThreads, (int64_t)hi * k, sums, count, z_sums);
    } else {
        for (int e = threadIdx.x; e < E; e += kShortThreads) sums[e] = 0.0f, count[e] = 0;
    }
    if (threadIdx.x == 0) z_mine = z;
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    const float inv = rows > 0 ? 1.0f / (float)rows : 0.0f;
    const int mine = (E + ctas - 1) / ctas;
    float product = 0.0f;
    for (int e = rank * mine + threadIdx.x; e < min((rank + 1) * mine, E); e += kShortThreads) {
        float v = 0.0f;
        int32_t c = 0;
        for (int q = 0; q < ctas; ++q) {
            float f;
            int32_t n;
            asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(cluster_smem_u32(sums + e, q)));
            asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(cluster_smem_u32(count + e, q)));
            v += f, c += n;
        }
        const float p = v * inv, f = rows > 0 ? (float)c / ((float)k * (float)rows) : 0.0f;
        count_out[(size_t)s * E + e] = c;
        load[(size_t)s * E + e] = f;
        prob[(size_t)s * E + e] = p;
        product = fmaf(f, p, product);
    }
    product = warp_sum(product);
    if (lane == 0) inner[warp] = product;
    __syncthreads();
    if (threadIdx.x == 0) {
        product = 0.0f;
        for (int w = 0; w < kWarps; ++w) product += inner[w];
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_smem_u32(&products[rank], 0)), "f"(product) : "memory");
        if (rank == 0) {
            z = 0.0f;
            for (int q = 0; q < ctas; ++q) {
                float f;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(f) : "r"(cluster_smem_u32(&z_mine, q)));
                z += f;
            }
        }
    }
    if (ctas > 1) cluster_sync();  // the products are there; no CTA ends while another one reads its memory
    if (rank == 0 && threadIdx.x == 0) {
        product = 0.0f;
        for (int q = 0; q < ctas; ++q) product += products[q];
        loss[2 * (size_t)s] = (float)E * product;
        loss[2 * (size_t)s + 1] = z * inv;
    }
}

// A cluster of CTAs a sequence, each of which adds up a part of the columns; the first one joins the losses.
// (One CTA for 256 columns of 304 partial rows took 28 us.)
__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(Sequences seq, int E, int k, int tile_rows, int ctas, Partials part,
                                                                        int32_t *count, float *load, float *prob, float *loss) {
    __shared__ float sums[kFinishThreads], inner[32], z_sums[32], products[8];
    __shared__ int32_t counts[kFinishThreads];
    cluster_arrive();  // the others' memory is there from the wait below on: a CTA that starts late may still get it
    grid_dependency_wait();
    grid_launch_dependents();
    const int s = blockIdx.x / ctas, rank = blockIdx.x % ctas;
    const int begin = seq.begin(s), end = seq.end(s), rows = end - begin;
    const int first = begin / tile_rows, last = rows > 0 ? (end - 1) / tile_rows : first - 1;
    const float inv = rows > 0 ? 1.0f / (float)rows : 0.0f;
    // threads: a power of two of columns, the rest of them takes the partial rows in turns
    const int mine = (E + ctas - 1) / ctas;
    int columns = 32;
    while (columns < mine) columns *= 2;
    const int turns = blockDim.x / columns, c0 = threadIdx.x % columns, turn = threadIdx.x / columns;
    const int e = rank * mine + c0;
    const bool in = c0 < mine && e < E;
    float v = 0.0f;
    int32_t c = 0;
    if (in)
#pragma unroll 8
        for (int i = first + turn; i <= last; i += turns) {
            const size_t at = ((size_t)i + s) * E + e;
            v += part.prob[at];
            c += part.count[at];
        }
    float z = 0.0f;
    if (rank == 0)
        for (int i = first + threadIdx.x; i <= last; i += blockDim.x) z += part.z[(size_t)i + s];
    sums[threadIdx.x] = v;
    counts[threadIdx.x] = c;
    z = warp_sum(z);
    if (threadIdx.x % 32 == 0) z_sums[threadIdx.x / 32] = z;
    __syncthreads();
    float product = 0.0f;
    if (turn == 0 && in) {
#pragma unroll 4
        for (int i = 1; i < turns; ++i) v += sums[i * columns + c0], c += counts[i * columns + c0];
        const float p = v * inv, f = rows > 0 ? (float)c / ((float)k * (float)rows) : 0.0f;
        count[(size_t)s * E + e] = c;
        load[(size_t)s * E + e] = f;
        prob[(size_t)s * E + e] = p;
        product = f * p;
    }
    product = warp_sum(product);
    if (threadIdx.x % 32 == 0) inner[threadIdx.x / 32] = product;
    __syncthreads();
    cluster_wait();
    if (threadIdx.x < 32) {
        product = warp_sum(threadIdx.x < blockDim.x / 32 ? inner[threadIdx.x] : 0.0f);
        if (threadIdx.x == 0)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_smem_u32(&products[rank], 0)), "f"(product) : "memory");
    }
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        product = 0.0f;
        for (int i = 0; i < ctas; ++i) product += products[i];
        z = 0.0f;
        for (int i = 0; i < blockDim.x / 32; ++i) z += z_sums[i];
        loss[2 * (size_t)s] = (float)E * product;
        loss[2 * (size_t)s + 1] = z * inv;
    }
}

// A warp takes `mine` consecutive rows.
template <int L, int NQ, bool WIDE>
__global__ void __launch_bounds__(kBalThreads, NQ <= 4 ? 2 : 1) balance_backward_kernel(Sequences seq, int E, int mine, const float *logits,
                                                                                       const float *load, const float *d_loss,
                                                                                       const float *d_in, float *d_logits) {
    using R = Row<L, NQ, WIDE>;
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32;
    const int64_t first = ((int64_t)blockIdx.x * kBalWarps + threadIdx.x / 32) * mine;
    const int64_t stop = min(first + mine, (int64_t)seq.T);
    int64_t t = first + lane / L;
    R next, next_d;
    const auto ask = [&](int64_t t) {
        const size_t at = (size_t)min(t, (int64_t)seq.T - 1) * E;
        next.load(logits + at, E, t < stop, -INFINITY);
        if (d_in)
            next_d.load(d_in + at, E, true, 0.0f);
        else
            next_d.clear();
    };
    ask(t);
    int begin = 0, end = 0;  // of the sequence that f, c0 and c1 are of
    R f;
    float c0 = 0.0f, c1 = 0.0f;
    for (; t - lane / L < stop; t += R::kRows) {
        if (t < stop && (t < begin || t >= end)) {
            const int s = L == 32 ? seq.find((int)t) : seq.find_alone((int)t);
            begin = end = 0;
            if (s >= 0 && t < seq.end(s)) {
                begin = seq.begin(s), end = seq.end(s);
                const float inv = 1.0f / (float)(end - begin);
                c0 = d_loss[2 * (size_t)s] * (float)E * inv;
                c1 = 2.0f * d_loss[2 * (size_t)s + 1] * inv;
                f.load(load + (size_t)s * E, E, true, 0.0f);
            }
        }
        if (L < 32) __syncwarp();
        R r = next, d = next_d;
        ask(t + R::kRows);
        float top, sum = exponentials(r, top), dot = 0.0f;
        const bool owned = t >= begin && t < end;
        if (owned) {
            uint64_t dots = 0;
#pragma unroll
            for (int i = 0; i < 2 * NQ; ++i) dots = fma2(f.v[i], r.v[i], dots);
            dot = total(dots);
        }
        if (L < 32) __syncwarp();
#pragma unroll
        for (int k = L / 2; k > 0; k /= 2) {
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, k);
            dot += __shfl_xor_sync(0xFFFFFFFFu, dot, k);
        }
        if (owned && sum != 0.0f) {
            // p (c0 (f - mean) + c1 lse) = e (g f + h)
            const float inv = __fdividef(1.0f, sum), g = c0 * inv, h = inv * fmaf(c1, top + __logf(sum), -g * dot);
            const uint64_t g2 = pair(g, g), h2 = pair(h, h);
#pragma unroll
            for (int i = 0; i < 2 * NQ; ++i) d.v[i] = fma2(r.v[i], fma2(g2, f.v[i], h2), d.v[i]);
        }
        if (t < stop) d.store(d_logits + (size_t)t * E, E);
    }
}

// Lanes of a row: as many as hold it with 16 values each, all 32 beyond 256 experts.
constexpr int lanes_of(int E) { return E <= 32 ? 2 : E <= 64 ? 4 : E <= 128 ? 8 : E <= 256 ? 16 : 32; }

// Whether a cluster takes each sequence: up to as many rows, in the mean, as its eight CTAs' warps take in eight
// turns, if the clusters find an SM for every CTA, else in one turn. One sequence by a cluster and by tiles: 8
// experts, 4096 rows 5.6 and 8.1 us, 8192 7.8 and 8.9; 128 experts, 512 rows 4.7 and 7.0, 2048 7.1 and 7.9, 4096 12.5 and
// 8.9; 256 experts, 1024 rows 7.5 and 7.3. 64 sequences of 2048 rows, 128 experts: 35 and 24. A sequence that has
// most of the rows among many short ones is slow here, not wrong (1024 of 131072 rows in all, 128 experts: 27 us, with three
// quarters of the rows in one of them 694).
bool short_sequences(const ep_config &c, int32_t n_seq) {
    const int rows = c.T / n_seq, turn = 8 * (kShortThreads / 32) * (32 / lanes_of(c.E));
    return rows <= turn || (rows <= 8 * turn && 8 * (int64_t)n_seq <= 152);
}

// The tiles of the forward pass otherwise: two for every SM, by CTAs of as many warps as fit, so that few partial sums
// are left (607 rows of them, from four CTAs an SM, took longer to join than to make).
struct Tiles {
    int rows, n;
    size_t partials;  // rows of partial sums, at most
};
Tiles tiles(const ep_config &c, int32_t n_seq) {
    Tiles t;
    const int64_t n = 152 * 2;
    const int64_t rows = (c.T + n - 1) / n;
    t.rows = (int)(rows < 16 ? 16 : rows);
    t.n = (int)(((int64_t)c.T + t.rows - 1) / t.rows);
    t.partials = (size_t)t.n + (size_t)n_seq;
    return t;
}

// A launch by clusters along the grid's first dimension.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), int64_t grid, int threads, size_t smem, int ctas, cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

bool on16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

struct ForwardCall {
    const ep_config &c;
    const Sequences &seq;
    const float *logits;
    const int32_t *idx;
    const Partials &part;
    cudaStream_t s;
    bool wide() const { return c.E % 4 == 0 && on16(logits); }
    template <int L, int NQ, bool WIDE>
    cudaError_t run() const {
        const Tiles t = tiles(c, seq.n);
        const size_t smem = (size_t)(kSumThreads / 32 + 1) * c.E * sizeof(float);
        static SharedMemoryLimit limit;
        const cudaError_t e = limit.allow(balance_kernel<L, NQ, WIDE>, smem);
        if (e != cudaSuccess) return e;
        return launch_dependent(balance_kernel<L, NQ, WIDE>, dim3((unsigned)t.n), dim3(kSumThreads), smem, s, seq, c.E, c.k,
                                t.rows, logits, idx, part);
    }
};
struct ShortCall {
    const ep_config &c;
    const Sequences &seq;
    const float *logits;
    const int32_t *idx;
    int32_t *count;
    float *load, *prob, *loss;
    cudaStream_t s;
    bool wide() const { return c.E % 4 == 0 && on16(logits); }
    template <int L, int NQ, bool WIDE>
    cudaError_t run() const {
        // as many CTAs as leave each warp two turns of rows in the mean
        int ctas = 1;
        while (ctas < 8 && (int64_t)ctas * (kShortThreads / 32) * (32 / L) * 2 * seq.n < c.T) ctas *= 2;
        const size_t smem = (size_t)(kShortThreads / 32 + 1) * c.E * sizeof(float);
        return launch_clusters(balance_short_kernel<L, NQ, WIDE>, (int64_t)ctas * seq.n, kShortThreads, smem, ctas, s, seq, c.E, c.k,
                               ctas, logits, idx, count, load, prob, loss);
    }
};
struct BackwardCall {
    const ep_config &c;
    const Sequences &seq;
    const float *logits, *load, *d_loss, *d_in;
    float *d_logits;
    cudaStream_t s;
    bool wide() const { return c.E % 4 == 0 && on16(logits) && on16(load) && on16(d_in) && on16(d_logits); }
    template <int L, int NQ, bool WIDE>
    cudaError_t run() const {
        // as many warps as fill the SMs, with equal numbers of rows
        const int64_t warps = (NQ <= 4 ? 2 : 1) * (int64_t)current_device_sm_count() * kBalWarps;
        const int64_t rows = ((c.T + warps - 1) / warps + 32 / L - 1) / (32 / L) * (32 / L);
        const int64_t used = ((int64_t)c.T + rows - 1) / rows;
        return launch_dependent(balance_backward_kernel<L, NQ, WIDE>, dim3((unsigned)((used + kBalWarps - 1) / kBalWarps)),
                                dim3(kBalThreads), 0, s, seq, c.E, (int)rows, logits, load, d_loss, d_in, d_logits);
    }
};
template <bool WIDE, typename Call>
cudaError_t by_experts(const Call &call) {
    if (call.c.E <= 32) return call.template run<2, 4, WIDE>();
    if (call.c.E <= 64) return call.template run<4, 4, WIDE>();
    if (call.c.E <= 128) return call.template run<8, 4, WIDE>();
    if (call.c.E <= 256) return call.template run<16, 4, WIDE>();
    if (call.c.E <= 512) return call.template run<32, 4, WIDE>();
    return call.template run<32, kMaxE / 128, WIDE>();
}
template <typename Call>
cudaError_t run_call(const Call &call) {
    return call.wide() ? by_experts<true>(call) : by_experts<false>(call);
}

cudaError_t run_finish(const ep_config &c, const Sequences &seq, const Partials &part, int32_t *count, float *load, float *prob,
                       float *loss, cudaStream_t s) {
    // CTAs of 32 columns each, up to the eight of a cluster, with as many turns of rows as a sequence has rows of
    // partial sums, about
    const Tiles t = tiles(c, seq.n);
    const int ctas = c.E >= 256 ? 8 : (c.E + 31) / 32, share = t.n / seq.n + 1, columns = (c.E + ctas - 1) / ctas;
    int threads = 32;
    while (threads < columns) threads *= 2;
    for (int turns = 1; turns < share && threads < kFinishThreads; turns *= 2) threads *= 2;
    return launch_clusters(balance_finish_kernel, (int64_t)ctas * seq.n, threads, 0, ctas, s, seq, c.E, c.k, t.rows, ctas, part, count,
                           load, prob, loss);
}

}  // namespace

size_t balance_workspace_bytes(const ep_config &c, int32_t n_seq) {
    return short_sequences(c, n_seq) ? 256 : tiles(c, n_seq).partials * (2 * (size_t)c.E + 1) * sizeof(float);
}

cudaError_t launch_balance(const ep_config &c, int32_t n_seq, const float *logits, const int32_t *idx, const int32_t *seq_first,
                           const int32_t *seq_len, int32_t *count, float *load, float *prob, float *loss, void *workspace,
                           cudaStream_t s) {
    const Sequences seq{seq_first, seq_len, n_seq, c.T};
    if (short_sequences(c, n_seq)) return run_call(ShortCall{c, seq, logits, idx, count, load, prob, loss, s});
    const size_t rows = tiles(c, n_seq).partials;
    Partials part;
    part.prob = static_cast<float *>(workspace);
    part.count = reinterpret_cast<int32_t *>(part.prob + rows * c.E);
    part.z = reinterpret_cast<float *>(part.count + rows * c.E);
    const cudaError_t e = run_call(ForwardCall{c, seq, logits, idx, part, s});
    if (e != cudaSuccess) return e;
    return run_finish(c, seq, part, count, load, prob, loss, s);
}

cudaError_t launch_balance_backward(const ep_config &c, int32_t n_seq, const float *logits, const int32_t *seq_first,
                                    const int32_t *seq_len, const float *load, const float *d_loss, const float *d_in,
                                    float *d_logits, cudaStream_t s) {
    const Sequences seq{seq_first, seq_len, n_seq, c.T};
    return run_call(BackwardCall{c, seq, logits, load, d_loss, d_in, d_logits, s});
}

}  // namespace ep
