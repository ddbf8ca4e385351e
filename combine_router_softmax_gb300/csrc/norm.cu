// norm.cu -- the norms before and after a block, fused with its gate and the residual scale: the launches, and
// what joins the sums over rows.
#include "norm_rows.cuh"

namespace ep {

namespace {

struct FinishArgs {
    const float *partial;
    int32_t partials, H, next_at, y_at;
    const uint16_t *w_post, *gate;       // gate: of channels, else null
    float *d_w_next, *d_w_post, *d_gate;
    float offset;
    int32_t sigmoid;
};

constexpr int kFinishRows = 32;  // a CTA takes 32 columns, each warp every 32nd partial row

__global__ void __launch_bounds__(32 * kFinishRows) block_norm_finish_kernel(const FinishArgs p) {
    __shared__ float part[2][kFinishRows][33];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, w = threadIdx.x / 32, h = blockIdx.x * 32 + lane;
    const int sums = (p.next_at >= 0) + (p.y_at >= 0);
    float a = 0.0f, b = 0.0f;
    if (h < p.H)
#pragma unroll 4
        for (int i = w; i < p.partials; i += kFinishRows) {
            const float *row = p.partial + (size_t)i * sums * p.H + h;
            if (p.next_at >= 0) a += row[(size_t)p.next_at * p.H];
            if (p.y_at >= 0) b += row[(size_t)p.y_at * p.H];
        }
    part[0][w][lane] = a, part[1][w][lane] = b;
    __syncthreads();
    if (w >= 2) return;  // warp 0: d_w_next, warp 1: the others
    float s = 0.0f;
    for (int i = 0; i < kFinishRows; ++i) s += part[w][i][lane];
    if (h >= p.H) return;
    if (w == 0) {
        if (p.next_at >= 0) p.d_w_next[h] = s;
        return;
    }
    if (p.y_at < 0) return;
    float slope = 1.0f, f = 1.0f, wj = 1.0f;
    if (p.gate) f = gate_act(__uint_as_float((uint32_t)p.gate[h] << 16), p.sigmoid, slope);
    if (p.w_post) wj = p.offset + __uint_as_float((uint32_t)p.w_post[h] << 16);
    if (p.d_w_post) p.d_w_post[h] = f * s;
    if (p.gate && p.d_gate) p.d_gate[h] = s * (wj * slope);
}

NormArgs norm_args(const ep_norm_config &c, const void *x, const ep_bf16 *y, const ep_bf16 *w_post, const void *gate,
                   const ep_bf16 *w_next) {
    NormArgs p = {};
    p.x = x;
    p.y = reinterpret_cast<const uint4 *>(y);
    p.w_post = reinterpret_cast<const uint4 *>(w_post);
    p.w_next = reinterpret_cast<const uint4 *>(w_next);
    p.gate = gate;
    p.T = c.T;
    p.vecs = c.H / 8;
    p.kind = c.gate;
    p.sigmoid = c.gate_sigmoid;
    p.eps = c.eps;
    p.scale = c.scale;
    p.offset = c.weight_offset;
    p.inv_h = 1.0f / (float)c.H;
    p.next_at = p.y_at = -1;
    return p;
}

}  // namespace

size_t block_norm_workspace_bytes(const ep_norm_config &c) {
    return (size_t)norm_partials(c) * 2 * (size_t)c.H * sizeof(float);
}

cudaError_t launch_block_norm(const ep_norm_config &c, const void *x, const ep_bf16 *y, const ep_bf16 *w_post, const void *gate,
                              const ep_bf16 *w_next, void *out, ep_bf16 *n, float *rstd_post, float *rstd_next,
                              cudaStream_t s) {
    NormArgs p = norm_args(c, x, y, w_post, gate, w_next);
    p.out = out;
    p.n = reinterpret_cast<uint4 *>(n);
    p.rstd_post = rstd_post;
    p.rstd_next = rstd_next;
    return launch_norm_forward(p, c.residual_f32 != 0, s);
}

cudaError_t launch_block_norm_backward(const ep_norm_config &c, const void *x, const ep_bf16 *y, const ep_bf16 *w_post,
                                       const void *gate, const ep_bf16 *w_next, const float *rstd_post,
                                       const float *rstd_next, const void *d_out, const ep_bf16 *d_n, void *d_x, ep_bf16 *d_y,
                                       float *d_w_post, void *d_gate, float *d_w_next, float *partial, cudaStream_t s) {
    NormArgs p = norm_args(c, x, y, w_post, gate, w_next);
    p.rstd_post = const_cast<float *>(rstd_post);
    p.rstd_next = const_cast<float *>(rstd_next);
    p.d_out = d_out;
    p.d_n = reinterpret_cast<const uint4 *>(d_n);
    p.d_x = d_x;
    p.d_y = reinterpret_cast<uint4 *>(d_y);
    p.d_gate = d_gate;
    p.partial = partial;
    const bool channel = c.gate == EP_GATE_CHANNEL;
    int sums = 0;
    if (d_w_next) p.next_at = sums++;
    if (d_w_post || (channel && d_gate)) p.y_at = sums++;
    int partials = 0;
    const cudaError_t e = launch_norm_backward(p, c.residual_f32 != 0, norm_partials(c), &partials, s);
    if (e != cudaSuccess || sums == 0) return e;
    FinishArgs f = {};
    f.partial = partial;
    f.partials = partials;
    f.H = c.H;
    f.next_at = p.next_at;
    f.y_at = p.y_at;
    f.w_post = w_post;
    f.gate = channel ? static_cast<const uint16_t *>(gate) : nullptr;
    f.d_w_next = d_w_next;
    f.d_w_post = d_w_post;
    f.d_gate = channel ? static_cast<float *>(d_gate) : nullptr;
    f.offset = c.weight_offset;
    f.sigmoid = c.gate_sigmoid;
    return launch_dependent(block_norm_finish_kernel, dim3((unsigned)((c.H + 31) / 32)), dim3(32 * kFinishRows), 0, s, f);
}

}  // namespace ep
