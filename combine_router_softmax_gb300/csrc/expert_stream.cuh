// expert_stream.cuh -- products of few rows with the experts' weights: the weights are streamed once.
//
// y[s, n] = sum_k x[s, k] w[e, n, k], e the expert that owns row s, and the gated block's first half
// silu(g) u from two such products. For single tokens the weights are the traffic (N K values of
// every expert that has rows, against 2 rows N K operations), so what counts is to keep enough of
// them on their way: a producer warp fetches stages of 64 weight rows x 256 bytes by TMA into a ring of
// four, on across work items. Eight warps consume a stage: each takes 32 weight rows and a quarter of
// the stage's k. Two CTAs share an SM (128 KB of stages, 19 MB on the GPU; HBM needs about 10 MB under
// way; a fifth stage took L1 from the activations and cost 5%): all warps of one wait for the same stage,
// and what each then does before its products is latency, which the other CTA's products fill.
//
// bf16 weights run at HBM's rate (8 rows over 32 experts of 4096 / 1024 in 33 us, 5.4 TB/s with both
// launches). 4-bit weights need more of L1: a load of activations by a warp touches eight rows, eight
// lines for 512 bytes, and with 16 weight rows and half the k a warp they kept L1 81% busy. With twice the
// rows they are loaded half as often: 8 rows over 64 experts of 7168 / 2048 took 5 us less (52 now), 512 rows
// of 4096 / 1024 30 us less (136 now), of which 23 are one fragment at a time for more than 8 rows (both at
// once need 48 registers more than the 96 a thread can have, with 18 warps on four quarters of an SM).
//
// The product is the matrix instruction m16n8k16 with the weights as its 16 rows and 8 rows of x as
// its columns. Which k a lane's register stands for is free as long as both operands agree, so a
// lane takes 8 consecutive k of a row of x, 16 bytes, and the same 8 k of its two weight rows.
//
// Weights are bf16, or 4 bits with one bf16 scale for G consecutive k. There a nibble v becomes the
// bf16 value 128 + v by setting the bits 0x4300 over it (bf16 has 7 bits of fraction, so at 128 its
// step is 1): one logic operation for two nibbles. What is over, 136, is taken off the values, exactly. Taken
// off the sums, sum (128 + v) x - 136 sum x, it would save the subtraction (shifts, logic and subtraction take
// two cycles a quarter of an SM each: 22 for a word of 8 nibbles, 14 without it; the 52 us would be 50) but
// leave the rounding of 136 x behind, which an activation some hundred times the others' size makes larger than bf16's, and NaN of
// an infinite one. Products with bf16 activations are exact in fp32; a group is summed in fp32 and
// scaled as a whole.
#pragma once

#include <cuda_bf16.h>

#include <type_traits>

#include "tcgen05.cuh"

namespace ep {

constexpr int kStreamWarps = 8;                        // consumers
constexpr int kStreamThreads = (kStreamWarps + 1) * 32;
constexpr int kStreamCtas = 2;                         // on an SM
constexpr int kStreamRows = 64;                        // weight rows of a work item (gated: 32 of either projection)
constexpr int kStreamBox = kStreamRows * 128;          // bytes of 128 bytes of every row: a stage has two
constexpr int kStreamStageBytes = 2 * kStreamBox;
constexpr int kStreamStages = 4;
constexpr int kStreamTokens = 16;                      // rows of x that one pass over the weights serves
constexpr int kStreamParts = 4;                        // of a stage's k, one to a warp
constexpr int kStreamRedRow = kStreamRows + 4;         // floats of a token's sums: the four tokens of a store meet different banks
constexpr int kStreamRed = kStreamParts * kStreamTokens * kStreamRedRow;  // of a pass's

struct StreamParams {
    CUtensorMap w[2];         // [E][N][bytes of a row], boxes of 128 bytes x 32 or 64 rows, swizzled
    const ep_bf16 *scale[2];  // 4-bit weights: [E][N][Kp / G]
    const ep_bf16 *x;
    const int32_t *expert_offset;
    ep_bf16 *y;
    int32_t S, N, K, E;
    int32_t *error;
};

// Nibbles i and i + 4 of a word as the bf16 values v - 8.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i) {
    uint32_t v;
    // 128 + v: (word >> 4 i) & 0x000F000F | 0x43004300
    asm("lop3.b32 %0, %1, 0x000F000F, 0x43004300, 0xEA;" : "=r"(v) : "r"(word >> (4 * i)));
    const __nv_bfloat162 m = __float2bfloat162_rn(136.0f);
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), m);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t word_of(const uint4 &v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

// G = 0: bf16 weights, 128 k a stage; else 4-bit weights, 512 k a stage. A part is 64 bytes of every
// weight row of the stage.
template <int G>
struct StreamShape {
    static constexpr int kStageK = G == 0 ? 128 : 512;
    static constexpr int kPartK = kStageK / kStreamParts;
    static constexpr int kVecs = kPartK / 32;  // 16-byte words of a row of x for it
};

// The scales of 128 k of a row: one bf16 (G = 128), two or four of them.
template <int G>
__device__ __forceinline__ uint2 load_scales(const ep_bf16 *row) {
    if constexpr (G == 128)
        return make_uint2(*row, 0);
    else if constexpr (G == 64)
        return make_uint2(*reinterpret_cast<const uint32_t *>(row), 0);
    else if constexpr (G == 32)
        return *reinterpret_cast<const uint2 *>(row);
    else
        return make_uint2(0, 0);
}

// An expert that has rows.
struct StreamExpert {
    int e, first, rows;
};
// The work items of one CTA, item blockIdx.x + i gridDim.x for i = 0, 1, ...: each a block of output
// columns of an expert. Stepped through without a division, which every warp would wait for.
struct StreamItems {
    const StreamExpert *experts;  // those that have rows, in shared memory
    int count, blocks;
    int index, block;
    __device__ StreamItems(const StreamExpert *x, int n, int b)
        : experts(x), count(n), blocks(b), index((int)(blockIdx.x / (unsigned)b)), block((int)(blockIdx.x % (unsigned)b)) {}
    __device__ bool any() const { return index < count; }
    __device__ void next() {
        block += gridDim.x;
        while (block >= blocks && index < count) block -= blocks, ++index;
    }
};

// What one consumer warp does with the work items' stages.
struct StreamWarp {
    unsigned char *stages;
    uint64_t *full, *empty;
    volatile int *failed;
    uint32_t it;
    bool ready;  // stage `it` has been seen to be there
    int lane, pair, part;  // 32 weight rows, a quarter of a stage's k
};

__device__ __forceinline__ void consumers_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(kStreamWarps * 32) : "memory");
}

// One pass over an item's stages for up to NT * 8 rows of x (`tokens` of them exist); red[part]
// [token][row] gets the warp's sums.
template <bool GATED, int G, int NT>
__device__ __forceinline__ void stream_pass(const StreamParams &p, StreamWarp &w, int e, int n0, int64_t x0, int tokens,
                                            float *red) {
    using Sh = StreamShape<G>;
    const int g = w.lane / 4, t = w.lane % 4;
    // weight rows of the first fragment's rows g and g + 8 (the second's are 16 more): with g's order
    // changed so that the eight lanes of one shared-memory phase, two rows, meet different banks of the
    // swizzled stage
    const int r0 = w.pair * 32 + (g >> 1) + 4 * (g & 1);
    const uint4 *at = reinterpret_cast<const uint4 *>(w.stages + w.part / 2 * kStreamBox + r0 * 128) +
                      ((w.part % 2 * 4 + t) ^ (r0 & 7));
    // scales of the four rows, activations of this lane's row: at the warp's part of the present stage
    const ep_bf16 *sc = nullptr;
    int sc_row[4] = {};
    if constexpr (G > 0) {
        const size_t row_groups = (size_t)((p.K + 127) / 128) * (128 / G);
        const int n = min(n0 + (GATED ? r0 % (kStreamRows / 2) : r0), p.N - 1);  // past the last: that one, not stored
        sc = p.scale[GATED && w.pair] + ((size_t)e * p.N + n) * row_groups + w.part * (Sh::kPartK / G);
#pragma unroll
        for (int h = 1; h < 4; ++h) sc_row[h] = min(8 * h, p.N - 1 - n) * (int)row_groups;
    }
    const ep_bf16 *x[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)  // past the last row: the first again; its sums are not stored
        x[i] = p.x + (size_t)(x0 + (i * 8 + g < tokens ? i * 8 + g : 0)) * p.K + w.part * Sh::kPartK + 8 * t;
    const int kb = (p.K + Sh::kStageK - 1) / Sh::kStageK;

    float acc[2][NT][4] = {};
    // A stage, without a branch from the wait on. CHECK: it goes past K.
    const auto stage = [&](auto check, int b) {
        const uint32_t s = w.it % kStreamStages;
        uint4 v[NT][Sh::kVecs];
        uint2 scale[4];
        const int left = p.K - b * Sh::kStageK - w.part * Sh::kPartK;  // k from the part's first on
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < Sh::kVecs; ++j)
                v[i][j] = !check || 32 * j + 8 * t < left ? *reinterpret_cast<const uint4 *>(x[i] + 32 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int h = 0; h < 4; ++h) scale[h] = check && left <= 0 ? make_uint2(0, 0) : load_scales<G>(sc + sc_row[h]);
        if (!w.ready) {
            if (w.lane == 0 && !*w.failed) mbar_poll_limited(&w.full[s], (w.it / kStreamStages) & 1, w.failed);
            __syncwarp();  // the barrier's completion was seen by one lane; the others' reads are ordered behind it
        }
        const uint4 *from = at + s * (kStreamStageBytes / 16);
        const uint4 q[2][2] = {{from[0], from[64]}, {from[128], from[192]}};
        __syncwarp();
        if (w.lane == 0) mbar_arrive(&w.empty[s]);
        ++w.it;
        // every lane asks whether the next stage is there: the answer's latency is behind the products
        const bool there = mbar_test(&w.full[w.it % kStreamStages], (w.it / kStreamStages) & 1);
        if constexpr (G == 0) {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    mma_16816(acc[m][i], q[m][0].x, q[m][1].x, q[m][0].y, q[m][1].y, v[i][0].x, v[i][0].y);
                    mma_16816(acc[m][i], q[m][0].z, q[m][1].z, q[m][0].w, q[m][1].w, v[i][0].z, v[i][0].w);
                }
        } else {
            constexpr int M = NT > 1 ? 1 : 2;  // fragments at a time: two chains of dependent products either way
#pragma unroll
            for (int m0 = 0; m0 < 2; m0 += M) {
                float sum[M][NT][4] = {};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
#pragma unroll
                    for (int m = 0; m < M; ++m) {
                        const uint32_t w0 = word_of(q[m0 + m][0], j), w1 = word_of(q[m0 + m][1], j);
#pragma unroll
                        for (int step = 0; step < 2; ++step) {
                            const uint32_t a0 = w4_pair(w0, 2 * step), a1 = w4_pair(w1, 2 * step);
                            const uint32_t a2 = w4_pair(w0, 2 * step + 1), a3 = w4_pair(w1, 2 * step + 1);
#pragma unroll
                            for (int i = 0; i < NT; ++i)
                                mma_16816(sum[m][i], a0, a1, a2, a3, step ? v[i][j].z : v[i][j].x, step ? v[i][j].w : v[i][j].y);
                        }
                    }
                    if ((32 * (j + 1)) % G == 0) {
                        const int part = 32 * j / G;
#pragma unroll
                        for (int m = 0; m < M; ++m)
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const uint2 of = scale[2 * (m0 + m) + r / 2];
                                const float f = __uint_as_float(((part / 2 ? of.y : of.x) >> (16 * (part % 2))) << 16);
#pragma unroll
                                for (int i = 0; i < NT; ++i) {
                                    acc[m0 + m][i][r] = fmaf(f, sum[m][i][r], acc[m0 + m][i][r]);
                                    sum[m][i][r] = 0.0f;
                                }
                            }
                    }
                }
            }
        }
        w.ready = __all_sync(0xFFFFFFFFu, there);
#pragma unroll
        for (int i = 0; i < NT; ++i) x[i] += Sh::kStageK;
        if constexpr (G > 0) sc += Sh::kStageK / G;
    };
    const int whole = p.K / Sh::kStageK;
#pragma unroll 1
    for (int b = 0; b < whole; ++b) stage(std::false_type{}, b);
    if (whole < kb) stage(std::true_type{}, whole);
    float *mine = red + (size_t)w.part * kStreamTokens * kStreamRedRow;
    consumers_sync();  // the sums before these have been read
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r) mine[(i * 8 + 2 * t + r % 2) * kStreamRedRow + m * 16 + r0 + r / 2 * 8] = acc[m][i][r];
}

// The line of `p` into L1.
__device__ __forceinline__ void ask_for_line(const void *p) { asm volatile("prefetch.global.L1 [%0];" ::"l"(p)); }

template <bool GATED, int G>
__global__ void __launch_bounds__(kStreamThreads, kStreamCtas) expert_stream_kernel(const __grid_constant__ StreamParams p) {
    using Sh = StreamShape<G>;
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t full[kStreamStages], empty[kStreamStages];
    __shared__ int hits;
    __shared__ volatile int failed;
    unsigned char *stages = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    // [part][token][row]
    float *red = reinterpret_cast<float *>(stages + kStreamStages * kStreamStageBytes);
    StreamExpert *hit = reinterpret_cast<StreamExpert *>(red + kStreamRed);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kStreamStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], kStreamWarps);
        failed = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.w[0]);
        if (GATED) tma_prefetch_map(&p.w[1]);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    if (warp == 0) {
        int n = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            int first = 0, rows = 0;
            if (e < p.E) {
                first = min(max(p.expert_offset[e], 0), p.S);
                rows = min(p.expert_offset[e + 1], p.S) - first;
            }
            const unsigned m = __ballot_sync(0xFFFFFFFFu, rows > 0);
            if (rows > 0) hit[n + __popc(m & ((1u << lane) - 1))] = StreamExpert{e, first, rows};
            n += __popc(m);
        }
        if (lane == 0) hits = n;
    }
    __syncthreads();
    constexpr int kOut = GATED ? kStreamRows / 2 : kStreamRows;  // output columns of a work item
    const int blocks = (p.N + kOut - 1) / kOut;
    StreamItems items(hit, hits, blocks);
    const int kb = (p.K + Sh::kStageK - 1) / Sh::kStageK;
    uint32_t it = 0;  // the producer's next stage

    if (warp == kStreamWarps) {
        // ---- producer. Besides the weights it asks for the lines of x and of the scales that the stage's
        // consumers will read, three stages ahead of them: fetched by each warp for itself they cost an L2
        // latency a stage.
        bool ok = true;
        for (; ok && items.any(); items.next()) {
            const auto [e, first, rows] = hit[items.index];
            const int n0 = items.block * kOut;
            for (int done = 0; ok && done < rows; done += kStreamTokens)
                for (int b = 0; b < kb; ++b, ++it) {
                    const int s = it % kStreamStages;
                    if (it >= kStreamStages) {
                        if (lane == 0) ok = mbar_poll_limited(&empty[s], (it / kStreamStages - 1) & 1, &failed);
                        ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
                        if (!ok) break;
                    }
                    if (elect_one()) {
                        mbar_arrive_expect_tx(&full[s], kStreamStageBytes);
                        unsigned char *to = stages + s * kStreamStageBytes;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int at = (2 * b + h) * (G == 0 ? 64 : 128);  // the map's elements: bf16, or bytes of nibbles
                            tma_load_3d<1>(to + h * kStreamBox, &p.w[0], at, n0, e, smem_u32(&full[s]));
                            if (GATED)
                                tma_load_3d<1>(to + h * kStreamBox + kStreamBox / 2, &p.w[1], at, n0, e, smem_u32(&full[s]));
                        }
                    }
                    __syncwarp();
                    constexpr int kLines = Sh::kStageK / 64;
                    for (int i = lane; i < min(rows - done, kStreamTokens) * kLines; i += 32) {
                        const int k = b * Sh::kStageK + i % kLines * 64;
                        if (k < p.K) ask_for_line(p.x + (size_t)(first + done + i / kLines) * p.K + k);
                    }
                    if (G > 0 && b == 0) {
                        const size_t row_bytes = (size_t)((p.K + 127) / 128) * (256 / (G > 0 ? G : 1));
                        for (int i = lane; i < kStreamRows; i += 32) {
                            const int n = min(n0 + (GATED ? i % kOut : i), p.N - 1);
                            const char *row = reinterpret_cast<const char *>(p.scale[GATED && i >= kOut]) + ((size_t)e * p.N + n) * row_bytes;
                            for (size_t off = 0; off < row_bytes; off += 128) ask_for_line(row + off);
                        }
                    }
                }
        }
        __syncwarp();
    } else {
        // ---- consumers. After a failure they go on without waiting: every warp reaches the barriers.
        StreamWarp w{stages, full, empty, &failed, 0, false, lane, warp / kStreamParts, warp % kStreamParts};
        for (; items.any(); items.next()) {
            const auto [e, first, rows] = hit[items.index];
            const int n0 = items.block * kOut;
            for (int done = 0; done < rows; done += kStreamTokens) {
                const int tokens = min(rows - done, kStreamTokens);
                const int64_t x0 = (int64_t)first + done;
                if (tokens <= 8)
                    stream_pass<GATED, G, 1>(p, w, e, n0, x0, tokens, red);
                else
                    stream_pass<GATED, G, 2>(p, w, e, n0, x0, tokens, red);
                consumers_sync();
                for (int i = threadIdx.x; i < tokens * kOut; i += kStreamWarps * 32) {
                    const int token = i / kOut, n = i % kOut;
                    const auto sum = [&](int n) {
                        float v = 0.0f;
#pragma unroll
                        for (int part = 0; part < kStreamParts; ++part) v += red[(part * kStreamTokens + token) * kStreamRedRow + n];
                        return v;
                    };
                    float v = sum(n);
                    if constexpr (GATED) v = __fdividef(v, 1.0f + __expf(-v)) * sum(kOut + n);
                    if (n0 + n < p.N)
                        reinterpret_cast<__nv_bfloat16 *>(p.y)[(size_t)(x0 + token) * p.N + n0 + n] = __float2bfloat16_rn(v);
                }
            }
        }
    }
    __syncthreads();
    // No copy may be under way when the CTA ends. A consumer may have given up after the producer had
    // finished; from here on nobody sets `failed`.
    if (failed && threadIdx.x == kStreamWarps * 32) {
        wait_for_fills(full, it, 0, 1, kStreamStages);
        atomicOr(p.error, kErrExpertWait);
    }
}

template <bool GATED, int G>
cudaError_t launch_stream(StreamParams &p, const void *w0, const void *w1, cudaStream_t s) {
    using Sh = StreamShape<G>;
    auto kernel = expert_stream_kernel<GATED, G>;
    cudaError_t e = expert_error_word(&p.error);
    if (e != cudaSuccess) return e;
    const int64_t row = G == 0 ? p.K : (int64_t)(p.K + 127) / 128 * 64;
    constexpr int kBoxRows = GATED ? kStreamRows / 2 : kStreamRows;
    constexpr int kBytes = G == 0 ? 2 : 1;
    if (!make_map(&p.w[0], w0, kBytes, row, p.N, p.E, 128 / kBytes, kBoxRows)) return cudaErrorInvalidValue;
    if (GATED && !make_map(&p.w[1], w1, kBytes, row, p.N, p.E, 128 / kBytes, kBoxRows)) return cudaErrorInvalidValue;
    const size_t smem = 1024 + (size_t)kStreamStages * kStreamStageBytes + kStreamRed * sizeof(float) +
                        (size_t)p.E * sizeof(StreamExpert);
    static SharedMemoryLimit limit;
    e = limit.allow(kernel, smem);
    if (e != cudaSuccess) return e;
    constexpr int kOut = GATED ? kStreamRows / 2 : kStreamRows;
    const int64_t most = (int64_t)(p.E < p.S ? p.E : p.S) * ((p.N + kOut - 1) / kOut);
    const int sms = current_device_sm_count();
    if (sms <= 0) return cudaErrorInvalidDevice;
    return launch_dependent(kernel, dim3((unsigned)(most < kStreamCtas * sms ? most : kStreamCtas * sms)), dim3(kStreamThreads), smem, s, p);
}

}  // namespace ep
