// experts_api.cu -- the extern "C" entry points declared in include/ep_experts.h.
//
// As in ep_api.cu every argument is checked on the host, and a status is
// returned before anything is enqueued; nothing here allocates device memory or
// synchronises.
#include "ep_internal.cuh"

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Given and 16-byte aligned.
bool usable(const void *p) { return p && aligned16(p); }

ep_status from_cuda(cudaError_t e) { return e == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

ep_status check_ffn(const ep_ffn_config *c) {
    if (!c) return EP_ERR_INVALID_ARG;
    if (c->rows < 0 || c->H <= 0 || c->I <= 0 || c->E <= 0) return EP_ERR_INVALID_ARG;
    if (c->H % 8 != 0 || c->I % 8 != 0 || c->E > ep::kMaxE) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status ep_expert_ffn(const ep_ffn_config *cfg, const ep_bf16 *rows, const int32_t *expert_offset,
                        const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, ep_bf16 *g, ep_bf16 *u,
                        ep_bf16 *h, ep_bf16 *y, cudaStream_t stream) {
    const ep_status st = check_ffn(cfg);
    if (st != EP_OK) return st;
    if (cfg->rows == 0) return EP_OK;
    if (!usable(rows) || !expert_offset || !usable(w_gate) || !usable(w_up) || !usable(w_down) || !usable(h) || !usable(y))
        return EP_ERR_INVALID_ARG;
    if ((g == nullptr) != (u == nullptr) || !aligned16(g) || !aligned16(u)) return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_expert_ffn(*cfg, rows, expert_offset, w_gate, w_up, w_down, g, u, h, y, stream));
}

ep_status ep_expert_ffn_backward(const ep_ffn_config *cfg, const ep_bf16 *rows, const int32_t *expert_offset,
                                 const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, const ep_bf16 *g,
                                 const ep_bf16 *u, const ep_bf16 *h, const ep_bf16 *d_y, ep_bf16 *d_g, ep_bf16 *d_u,
                                 ep_bf16 *d_rows, ep_bf16 *d_w_gate, ep_bf16 *d_w_up, ep_bf16 *d_w_down,
                                 cudaStream_t stream) {
    const ep_status st = check_ffn(cfg);
    if (st != EP_OK) return st;
    if (!aligned16(d_rows) || !aligned16(d_w_gate) || !aligned16(d_w_up) || !aligned16(d_w_down)) return EP_ERR_INVALID_ARG;
    if (cfg->rows == 0) {
        const size_t bytes = (size_t)cfg->E * (size_t)cfg->H * (size_t)cfg->I * 2;
        for (ep_bf16 *w : {d_w_gate, d_w_up, d_w_down})
            if (w && cudaMemsetAsync(w, 0, bytes, stream) != cudaSuccess) return EP_ERR_CUDA;
        return EP_OK;
    }
    if (!usable(rows) || !expert_offset || !usable(w_gate) || !usable(w_up) || !usable(w_down) || !usable(g) || !usable(u) ||
        !usable(h) || !usable(d_y) || !usable(d_g) || !usable(d_u))
        return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_expert_ffn_backward(*cfg, rows, expert_offset, w_gate, w_up, w_down, g, u, h, d_y, d_g, d_u,
                                                    d_rows, d_w_gate, d_w_up, d_w_down, stream));
}

}  // extern "C"
