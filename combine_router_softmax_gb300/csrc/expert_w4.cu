// expert_w4.cu -- products of few rows with 4-bit weights and group scales, by expert.
//
// y[s, n] = sum_k x[s, k] scale[e, n, k / G] (q[e, n, k] - 8), e the expert that owns row s. For
// single tokens the weights are the traffic: N K / 2 bytes and the scales of every expert that has
// rows, against 2 rows N K operations, so the kernel is built to stream them: each is read once,
// unpacked in registers and multiplied at once.
//
// Unpacking. A nibble v becomes the bf16 value 128 + v by setting the bits 0x4300 over it (bf16 has
// 7 bits of fraction, so at 128 its step is 1): one logic operation for two nibbles; minus 136 gives
// v - 8, exactly. Products of these with bf16 activations are exact in fp32; a group is summed in
// fp32 by the matrix instruction m16n8k16 (16 weight rows x 8 tokens) and scaled once as a whole.
// A lane's two pairs of k per instruction are whatever its word holds, as long as the activations
// are taken at the same k: the packed order (ep_w4_pack) is made so that activations are read in
// their own order, 16 bytes at a time.
#include <cuda_bf16.h>

#include "ep_internal.cuh"

namespace ep {

namespace {

constexpr int kW4Warps = 8;
constexpr int kW4Threads = kW4Warps * 32;
constexpr int kW4Rows = 64;   // weight rows of a work item (gated: 32 of each projection)
constexpr int kW4Chunk = 128;  // k of one step of a warp: 64 bytes of a weight row
constexpr int kW4Tokens = 16;  // rows of x that one pass over the weights serves

struct W4Params {
    const uint8_t *q[2];
    const uint16_t *scale[2];
    const ep_bf16 *x;
    const int32_t *expert_offset;
    ep_bf16 *y;
    int32_t S, N, K, E;
};

__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i) {
    uint32_t v;
    // (word >> 4 i) & 0x000F000F | 0x43004300
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

// One pass over a work item's weights for NT * 8 rows of x from x0 on (`tokens` of them exist):
// warp w takes the chunks w, w + 8, ...; red[warp][token][row] gets its sums.
template <bool GATED, int G, int NT>
__device__ void w4_pass(const W4Params &p, int e, int n0, int64_t x0, int tokens, float *red) {
    constexpr int kMt = kW4Rows / 16;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int chunks = (p.K + kW4Chunk - 1) / kW4Chunk;
    const size_t row_bytes = (size_t)chunks * 64, row_groups = (size_t)chunks * (kW4Chunk / G);
    const uint8_t *q[kMt][2];
    const uint16_t *sc[kMt][2];
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int half = GATED ? m / (kMt / 2) : 0;
            const int n = n0 + (GATED ? m % (kMt / 2) : m) * 16 + h * 8 + g;
            const size_t row = (size_t)e * p.N + min(n, p.N - 1);  // past the last row: that one again, not stored
            q[m][h] = p.q[half] + row * row_bytes + t * 16;
            sc[m][h] = p.scale[half] + row * row_groups;
        }
    const ep_bf16 *x[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) x[i] = i * 8 + g < tokens ? p.x + (size_t)(x0 + i * 8 + g) * p.K : nullptr;

    float acc[kMt][NT][4] = {};
    for (int c = warp; c < chunks; c += kW4Warps) {
        uint4 w[kMt][2];
#pragma unroll
        for (int m = 0; m < kMt; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) w[m][h] = ld_stream_v4(reinterpret_cast<const uint4 *>(q[m][h] + (size_t)c * 64));
        uint4 b[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int k = c * kW4Chunk + 32 * j + 8 * t;
                b[i][j] = x[i] && k < p.K ? *reinterpret_cast<const uint4 *>(x[i] + k) : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
        for (int m = 0; m < kMt; ++m) {
            float s[2][kW4Chunk / G];
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < kW4Chunk / G; ++i)
                    s[h][i] = __uint_as_float((uint32_t)sc[m][h][(size_t)c * (kW4Chunk / G) + i] << 16);
            float part[NT][4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t w0 = word_of(w[m][0], j), w1 = word_of(w[m][1], j);
#pragma unroll
                for (int step = 0; step < 2; ++step) {
                    const uint32_t a0 = w4_pair(w0, 2 * step), a1 = w4_pair(w1, 2 * step);
                    const uint32_t a2 = w4_pair(w0, 2 * step + 1), a3 = w4_pair(w1, 2 * step + 1);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        mma_16816(part[i], a0, a1, a2, a3, step ? b[i][j].z : b[i][j].x, step ? b[i][j].w : b[i][j].y);
                }
                if ((32 * (j + 1)) % G == 0) {
                    const int group = 32 * j / G;
#pragma unroll
                    for (int i = 0; i < NT; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            acc[m][i][r] = fmaf(s[r / 2][group], part[i][r], acc[m][i][r]);
                            part[i][r] = 0.0f;
                        }
                }
            }
        }
    }
    float *mine = red + warp * kW4Rows * kW4Tokens;
#pragma unroll
    for (int m = 0; m < kMt; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                mine[(i * 8 + 2 * t + r % 2) * kW4Rows + m * 16 + r / 2 * 8 + g] = acc[m][i][r];
}

template <bool GATED, int G>
__global__ void __launch_bounds__(kW4Threads, 2) w4_kernel(const __grid_constant__ W4Params p) {
    extern __shared__ float red[];  // [warp][token][row], then the list of experts that have rows
    int *hit = reinterpret_cast<int *>(red + kW4Warps * kW4Rows * kW4Tokens);
    __shared__ int hits;
    grid_dependency_wait();
    grid_launch_dependents();
    if (threadIdx.x < 32) {
        int n = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + threadIdx.x;
            bool has = false;
            if (e < p.E) {
                const int first = min(max(p.expert_offset[e], 0), p.S);
                has = min(p.expert_offset[e + 1], p.S) > first;
            }
            const unsigned m = __ballot_sync(0xFFFFFFFFu, has);
            if (has) hit[n + __popc(m & ((1u << threadIdx.x) - 1))] = e;
            n += __popc(m);
        }
        if (threadIdx.x == 0) hits = n;
    }
    __syncthreads();
    constexpr int kOut = GATED ? kW4Rows / 2 : kW4Rows;  // output columns of a work item
    const int blocks = (p.N + kOut - 1) / kOut;
    for (int64_t item = blockIdx.x; item < (int64_t)hits * blocks; item += gridDim.x) {
        const int e = hit[item / blocks], n0 = (int)(item % blocks) * kOut;
        const int first = min(max(p.expert_offset[e], 0), p.S);
        const int rows = min(p.expert_offset[e + 1], p.S) - first;
        for (int done = 0; done < rows; done += kW4Tokens) {
            const int tokens = min(rows - done, kW4Tokens);
            const int64_t x0 = (int64_t)first + done;
            if (tokens <= 8)
                w4_pass<GATED, G, 1>(p, e, n0, x0, tokens, red);
            else
                w4_pass<GATED, G, 2>(p, e, n0, x0, tokens, red);
            __syncthreads();
            for (int i = threadIdx.x; i < tokens * kOut; i += kW4Threads) {
                const int token = i / kOut, n = i % kOut;
                float v = 0, u = 0;
                for (int w = 0; w < kW4Warps; ++w) {
                    const float *r = red + (w * kW4Tokens + token) * kW4Rows + n;
                    v += r[0];
                    if constexpr (GATED) u += r[kOut];
                }
                if constexpr (GATED) v = __fdividef(v, 1.0f + __expf(-v)) * u;
                if (n0 + n < p.N)
                    reinterpret_cast<__nv_bfloat16 *>(p.y)[(size_t)(x0 + token) * p.N + n0 + n] = __float2bfloat16_rn(v);
            }
            __syncthreads();
        }
    }
}

template <bool GATED, int G>
cudaError_t launch_g(const W4Params &p, cudaStream_t s) {
    auto kernel = w4_kernel<GATED, G>;
    const size_t smem = (size_t)kW4Warps * kW4Rows * kW4Tokens * sizeof(float) + (size_t)p.E * sizeof(int);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    constexpr int kOut = GATED ? kW4Rows / 2 : kW4Rows;
    const int64_t most = (int64_t)(p.E < p.S ? p.E : p.S) * ((p.N + kOut - 1) / kOut);
    const int64_t resident = (int64_t)current_device_sm_count() * max_blocks_per_sm((const void *)kernel, kW4Threads, smem);
    if (resident <= 0) return cudaErrorInvalidDevice;
    return launch_dependent(kernel, dim3((unsigned)(most < resident ? most : resident)), dim3(kW4Threads), smem, s, p);
}

template <bool GATED>
cudaError_t launch_w4(const W4Params &p, int group, cudaStream_t s) {
    switch (group) {
        case 32: return launch_g<GATED, 32>(p, s);
        case 64: return launch_g<GATED, 64>(p, s);
        default: return launch_g<GATED, 128>(p, s);
    }
}

// One warp packs one chunk of 128 k of one weight row; lane l holds k = 4 l .. 4 l + 3.
__global__ void __launch_bounds__(256) w4_pack_kernel(int64_t rows, int K, int G, const __nv_bfloat16 *w, uint32_t *q,
                                                      __nv_bfloat16 *scale) {
    const int lane = threadIdx.x % 32;
    const int chunks = (K + kW4Chunk - 1) / kW4Chunk;
    const int64_t total = rows * chunks;
    for (int64_t i = (int64_t)blockIdx.x * 8 + threadIdx.x / 32; i < total; i += (int64_t)gridDim.x * 8) {
        const int64_t row = i / chunks;
        const int c = (int)(i % chunks), k = c * kW4Chunk + 4 * lane;
        float v[4] = {0, 0, 0, 0};
        if (k < K)  // K is a multiple of 8
            for (int j = 0; j < 4; ++j) v[j] = __bfloat162float(w[row * K + k + j]);
        float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
        for (int d = 1; d < G / 4; d *= 2) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
        const __nv_bfloat16 s = __float2bfloat16_rn(__fdiv_rn(top, 7.0f));
        const float sf = __bfloat162float(s);
        uint32_t n[4];
        for (int j = 0; j < 4; ++j) {
            const float r = sf > 0 ? rintf(__fdiv_rn(v[j], sf)) : 0.0f;
            n[j] = (uint32_t)((int)fminf(fmaxf(r, -8.0f), 7.0f) + 8);
        }
        // nibble i of a word is offset 2 (i mod 4) + i / 4 of its 8 k: this lane's four are offsets
        // 0..3 (even lane) or 4..7 (odd lane) -> nibbles 0, 4, 1, 5 or 2, 6, 3, 7
        uint32_t word = n[0] | n[1] << 16 | n[2] << 4 | n[3] << 20;
        if (lane & 1) word <<= 8;
        word |= __shfl_xor_sync(0xFFFFFFFFu, word, 1);
        const int eight = lane / 2, j = eight / 4, t = eight % 4;  // k = 32 j + 8 t
        if (!(lane & 1)) q[i * 16 + t * 4 + j] = word;
        if (lane % (G / 4) == 0) scale[i * (kW4Chunk / G) + lane / (G / 4)] = s;
    }
}

}  // namespace

cudaError_t launch_w4_pack(const ep_w4_config &c, const ep_bf16 *w, uint8_t *q, ep_bf16 *scale, cudaStream_t s) {
    const int64_t rows = (int64_t)c.E * c.N;
    const int64_t warps = rows * ((c.K + kW4Chunk - 1) / kW4Chunk);
    const int64_t most = (int64_t)current_device_sm_count() * 8, want = (warps + 7) / 8;
    if (most <= 0) return cudaErrorInvalidDevice;
    w4_pack_kernel<<<(unsigned)(want < most ? want : most), 256, 0, s>>>(
        rows, c.K, c.group, reinterpret_cast<const __nv_bfloat16 *>(w), reinterpret_cast<uint32_t *>(q),
        reinterpret_cast<__nv_bfloat16 *>(scale));
    return cudaGetLastError();
}

cudaError_t launch_w4_linear(const ep_w4_config &c, const ep_bf16 *x, const int32_t *expert_offset, const uint8_t *q,
                             const ep_bf16 *scale, ep_bf16 *y, cudaStream_t s) {
    const W4Params p{{q, q}, {scale, scale}, x, expert_offset, y, c.rows, c.N, c.K, c.E};
    return launch_w4<false>(p, c.group, s);
}

cudaError_t launch_expert_ffn_w4(const ep_ffn_config &c, int group, const ep_bf16 *rows, const int32_t *expert_offset,
                                 const uint8_t *q_gate, const ep_bf16 *s_gate, const uint8_t *q_up, const ep_bf16 *s_up,
                                 const uint8_t *q_down, const ep_bf16 *s_down, ep_bf16 *h, ep_bf16 *y, cudaStream_t s) {
    const W4Params first{{q_gate, q_up}, {s_gate, s_up}, rows, expert_offset, h, c.rows, c.I, c.H, c.E};
    const cudaError_t e = launch_w4<true>(first, group, s);
    if (e != cudaSuccess) return e;
    const W4Params second{{q_down, q_down}, {s_down, s_down}, h, expert_offset, y, c.rows, c.H, c.I, c.E};
    return launch_w4<false>(second, group, s);
}

}  // namespace ep
