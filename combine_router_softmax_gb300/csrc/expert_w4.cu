// expert_w4.cu -- the experts' weights in 4 bits: packing, and the products with few rows
// (expert_stream.cuh).
#include "expert_stream.cuh"

namespace ep {

namespace {

constexpr int kW4Chunk = 128;  // k of 16 words of the packed form, its unit

template <bool GATED>
cudaError_t launch_w4(StreamParams p, const uint8_t *q0, const uint8_t *q1, int group, cudaStream_t s) {
    switch (group) {
        case 32: return launch_stream<GATED, 32>(p, q0, q1, s);
        case 64: return launch_stream<GATED, 64>(p, q0, q1, s);
        default: return launch_stream<GATED, 128>(p, q0, q1, s);
    }
}

StreamParams stream_params(const ep_bf16 *s0, const ep_bf16 *s1, const ep_bf16 *x, const int32_t *expert_offset, ep_bf16 *y,
                           int32_t S, int32_t N, int32_t K, int32_t E) {
    StreamParams p = {};
    p.scale[0] = s0;
    p.scale[1] = s1;
    p.x = x;
    p.expert_offset = expert_offset;
    p.y = y;
    p.S = S;
    p.N = N;
    p.K = K;
    p.E = E;
    return p;
}

// One warp packs one chunk of 128 k of one weight row; lane l holds k = 4 l .. 4 l + 3. Loads of two bytes
// bound it: 64 x 2048 x 7168 weights, 2.4 GB in and out, in 2.1 ms = 1.1 TB/s; a model is packed once.
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
    return launch_w4<false>(stream_params(scale, nullptr, x, expert_offset, y, c.rows, c.N, c.K, c.E), q, nullptr, c.group, s);
}

cudaError_t launch_expert_ffn_w4(const ep_ffn_config &c, int group, const ep_bf16 *rows, const int32_t *expert_offset,
                                 const uint8_t *q_gate, const ep_bf16 *s_gate, const uint8_t *q_up, const ep_bf16 *s_up,
                                 const uint8_t *q_down, const ep_bf16 *s_down, ep_bf16 *h, ep_bf16 *y, cudaStream_t s) {
    const cudaError_t e =
        launch_w4<true>(stream_params(s_gate, s_up, rows, expert_offset, h, c.rows, c.I, c.H, c.E), q_gate, q_up, group, s);
    if (e != cudaSuccess) return e;
    return launch_w4<false>(stream_params(s_down, nullptr, h, expert_offset, y, c.rows, c.H, c.I, c.E), q_down, nullptr, group, s);
}

}  // namespace ep
