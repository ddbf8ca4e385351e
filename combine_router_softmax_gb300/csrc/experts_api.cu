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
    if (c->saved_bf16 != 0 && c->saved_bf16 != 1) return EP_ERR_INVALID_ARG;
    if (c->H % 8 != 0 || c->I % 8 != 0 || c->E > ep::kMaxE) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

ep_status check_w4(const ep_w4_config *c) {
    if (!c) return EP_ERR_INVALID_ARG;
    if (c->rows < 0 || c->N <= 0 || c->K <= 0 || c->E <= 0) return EP_ERR_INVALID_ARG;
    if (c->group != 32 && c->group != 64 && c->group != 128) return EP_ERR_UNSUPPORTED;
    if (c->K % 8 != 0 || c->E > ep::kMaxE) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

// What combine and router check of a layer's shape.
ep_status check_layer(const ep_config *c, bool needs_rows) {
    if (!c) return EP_ERR_INVALID_ARG;
    if (c->T < 0 || c->E <= 0 || c->k <= 0 || c->k > c->E || (int64_t)c->T * c->k > INT32_MAX) return EP_ERR_INVALID_ARG;
    if (c->renormalize != 0 && c->renormalize != 1) return EP_ERR_INVALID_ARG;
    if (c->E > ep::kMaxE || c->k > ep::kMaxK) return EP_ERR_UNSUPPORTED;
    if (needs_rows && c->H <= 0) return EP_ERR_INVALID_ARG;
    if (needs_rows && c->H % 8 != 0) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

ep_status check_grad_list(const ep_grad_tensor *t, int32_t n, const float *norm, bool clip) {
    if (n < 0 || (n > 0 && !t) || !norm || (reinterpret_cast<uintptr_t>(norm) & 3u) != 0) return EP_ERR_INVALID_ARG;
    for (int32_t i = 0; i < n; ++i) {
        if (t[i].dtype != EP_F32 && t[i].dtype != EP_BF16 && t[i].dtype != EP_F16) return EP_ERR_INVALID_ARG;
        const uintptr_t size = t[i].dtype == EP_F32 ? 4 : 2;
        if (t[i].numel < 0 || t[i].reserved != 0) return EP_ERR_INVALID_ARG;
        if (t[i].numel == 0) continue;
        if (!t[i].data || reinterpret_cast<uintptr_t>(t[i].data) % size != 0) return EP_ERR_INVALID_ARG;
        if (clip && (!t[i].out || reinterpret_cast<uintptr_t>(t[i].out) % size != 0)) return EP_ERR_INVALID_ARG;
    }
    return EP_OK;
}

ep_status check_grads(const ep_grad_tensor *t, int32_t n, const float *norm, const void *ws, size_t bytes, bool clip) {
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & 7u) != 0) return EP_ERR_INVALID_ARG;
    const ep_status st = check_grad_list(t, n, norm, clip);
    if (st != EP_OK) return st;
    return bytes < ep::grad_workspace_bytes(n) ? EP_ERR_CAPACITY : EP_OK;
}

}  // namespace

extern "C" {

ep_status ep_expert_ffn(const ep_ffn_config *cfg, const ep_bf16 *rows, const int32_t *expert_offset,
                        const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, uint16_t *g, uint16_t *u,
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
                                 const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, const uint16_t *g,
                                 const uint16_t *u, const ep_bf16 *h, const ep_bf16 *d_y, ep_bf16 *d_g, ep_bf16 *d_u,
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

ep_status ep_w4_sizes(const ep_w4_config *cfg, size_t *q_bytes, size_t *scale_bytes) {
    const ep_status st = check_w4(cfg);
    if (st != EP_OK) return st;
    if (!q_bytes || !scale_bytes) return EP_ERR_INVALID_ARG;
    const size_t rows = (size_t)cfg->E * (size_t)cfg->N, kp = ((size_t)cfg->K + 127) / 128 * 128;
    *q_bytes = rows * kp / 2;
    *scale_bytes = rows * (kp / (size_t)cfg->group) * 2;
    return EP_OK;
}

ep_status ep_w4_pack(const ep_w4_config *cfg, const ep_bf16 *w, uint8_t *q, ep_bf16 *scale, cudaStream_t stream) {
    const ep_status st = check_w4(cfg);
    if (st != EP_OK) return st;
    if (!usable(w) || !usable(q) || !usable(scale)) return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_w4_pack(*cfg, w, q, scale, stream));
}

ep_status ep_w4_linear(const ep_w4_config *cfg, const ep_bf16 *x, const int32_t *expert_offset, const uint8_t *q,
                       const ep_bf16 *scale, ep_bf16 *y, cudaStream_t stream) {
    const ep_status st = check_w4(cfg);
    if (st != EP_OK) return st;
    if (cfg->rows == 0) return EP_OK;
    if (!usable(x) || !expert_offset || !usable(q) || !usable(scale) || !usable(y)) return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_w4_linear(*cfg, x, expert_offset, q, scale, y, stream));
}

ep_status ep_expert_ffn_w4(const ep_ffn_config *cfg, int32_t group, const ep_bf16 *rows, const int32_t *expert_offset,
                           const uint8_t *q_gate, const ep_bf16 *s_gate, const uint8_t *q_up, const ep_bf16 *s_up,
                           const uint8_t *q_down, const ep_bf16 *s_down, ep_bf16 *h, ep_bf16 *y, cudaStream_t stream) {
    const ep_status st = check_ffn(cfg);
    if (st != EP_OK) return st;
    if (group != 32 && group != 64 && group != 128) return EP_ERR_UNSUPPORTED;
    if (cfg->rows == 0) return EP_OK;
    if (!usable(rows) || !expert_offset || !usable(q_gate) || !usable(s_gate) || !usable(q_up) || !usable(s_up) ||
        !usable(q_down) || !usable(s_down) || !usable(h) || !usable(y))
        return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_expert_ffn_w4(*cfg, group, rows, expert_offset, q_gate, s_gate, q_up, s_up, q_down, s_down, h,
                                              y, stream));
}

ep_status ep_combine_backward(const ep_config *cfg, const ep_bf16 *d_out, const ep_bf16 *y, const int32_t *slot,
                              const float *topk_w, ep_bf16 *d_y, float *d_topk_w, cudaStream_t stream) {
    const ep_status st = check_layer(cfg, true);
    if (st != EP_OK) return st;
    if (cfg->T == 0) return EP_OK;
    if (!usable(d_out) || !usable(y) || !slot || !topk_w || !usable(d_y) || !d_topk_w) return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_combine_backward(*cfg, d_out, y, slot, topk_w, d_y, d_topk_w, stream));
}

ep_status ep_route_backward(const ep_config *cfg, const float *logits, const int32_t *topk_idx, const float *topk_w,
                            const float *d_topk_w, float *d_logits, cudaStream_t stream) {
    const ep_status st = check_layer(cfg, false);
    if (st != EP_OK) return st;
    if (cfg->T == 0) return EP_OK;
    if (!topk_idx || !topk_w || !d_topk_w || !d_logits || (!cfg->renormalize && !logits)) return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_route_backward(*cfg, logits, topk_idx, topk_w, d_topk_w, d_logits, stream));
}

ep_status ep_grad_workspace_size(int32_t n, size_t *bytes) {
    if (n < 0 || !bytes) return EP_ERR_INVALID_ARG;
    *bytes = ep::grad_workspace_bytes(n);
    return EP_OK;
}

ep_status ep_grad_norm(const ep_grad_tensor *tensors, int32_t n, float *norm, void *workspace, size_t workspace_bytes,
                       cudaStream_t stream) {
    const ep_status st = check_grads(tensors, n, norm, workspace, workspace_bytes, false);
    if (st != EP_OK) return st;
    return from_cuda(ep::launch_grad_clip(tensors, n, false, 0.0f, norm, static_cast<double *>(workspace), stream));
}

ep_status ep_grad_clip(const ep_grad_tensor *tensors, int32_t n, float max_norm, float *norm, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
    if (!(max_norm >= 0.0f)) return EP_ERR_INVALID_ARG;
    const ep_status st = check_grads(tensors, n, norm, workspace, workspace_bytes, true);
    if (st != EP_OK) return st;
    return from_cuda(ep::launch_grad_clip(tensors, n, true, max_norm, norm, static_cast<double *>(workspace), stream));
}

ep_status ep_grad_clip_with_norm(const ep_grad_tensor *tensors, int32_t n, float max_norm, const float *norm,
                                 cudaStream_t stream) {
    if (!(max_norm >= 0.0f)) return EP_ERR_INVALID_ARG;
    const ep_status st = check_grad_list(tensors, n, norm, true);
    if (st != EP_OK) return st;
    return from_cuda(ep::launch_grad_scale(tensors, n, max_norm, norm, stream));
}

}  // extern "C"
