// layer_api.cu -- the extern "C" entry points declared in include/ep_layer.h.
//
// As in ep_api.cu every argument is checked on the host, and a status is
// returned before anything is enqueued; nothing here allocates device memory or
// synchronises.
#include "ep_internal.cuh"

namespace {

bool aligned(const void *p, uintptr_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }
bool aligned16(const void *p) { return aligned(p, 16); }
// Given and 16-byte aligned.
bool usable(const void *p) { return p && aligned16(p); }

ep_status from_cuda(cudaError_t e) { return e == cudaSuccess ? EP_OK : EP_ERR_CUDA; }

constexpr int kMaxNormH = 16384;

ep_status check_norm(const ep_norm_config *c) {
    if (!c) return EP_ERR_INVALID_ARG;
    if (c->T < 0 || c->H <= 0 || c->gate < EP_GATE_NONE || c->gate > EP_GATE_ELEMENT) return EP_ERR_INVALID_ARG;
    if ((c->gate_sigmoid != 0 && c->gate_sigmoid != 1) || (c->residual_f32 != 0 && c->residual_f32 != 1)) return EP_ERR_INVALID_ARG;
    // NaN and infinities fail these too
    if (!(c->eps >= 0.0f && c->eps <= 3.4e38f) || !(c->scale >= -3.4e38f && c->scale <= 3.4e38f) ||
        !(c->weight_offset >= -3.4e38f && c->weight_offset <= 3.4e38f))
        return EP_ERR_INVALID_ARG;
    if (c->H % 8 != 0 || c->H > kMaxNormH) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

// What both directions check of a block's inputs; `next`: whether the stream is normed.
ep_status check_block(const ep_norm_config &c, const void *x, const ep_bf16 *y, const ep_bf16 *w_post, const void *gate,
                      const ep_bf16 *w_next, bool next) {
    if (!usable(x) || !aligned16(y) || !aligned16(w_post) || !aligned16(w_next)) return EP_ERR_INVALID_ARG;
    if (!y && (w_post || gate || c.gate != EP_GATE_NONE)) return EP_ERR_INVALID_ARG;
    if ((gate != nullptr) != (c.gate != EP_GATE_NONE) || next != (w_next != nullptr)) return EP_ERR_INVALID_ARG;
    if (!aligned(gate, c.gate == EP_GATE_TOKEN ? 4 : 16)) return EP_ERR_INVALID_ARG;
    return EP_OK;
}

// What the balance loss uses of a layer's shape, and the sequences.
ep_status check_balance(const ep_config *c, int32_t n_seq, const int32_t *seq_first, const int32_t *seq_len) {
    if (!c || n_seq < 1) return EP_ERR_INVALID_ARG;
    if (c->T < 0 || c->E <= 0 || c->k <= 0 || c->k > c->E || (int64_t)c->T * c->k > INT32_MAX) return EP_ERR_INVALID_ARG;
    if (c->E > ep::kMaxE || c->k > ep::kMaxK) return EP_ERR_UNSUPPORTED;
    if (!seq_first && (n_seq != 1 || seq_len)) return EP_ERR_INVALID_ARG;
    return aligned(seq_first, 4) && aligned(seq_len, 4) ? EP_OK : EP_ERR_INVALID_ARG;
}

constexpr int kMaxOrthoSide = 65536, kMaxOrthoSteps = 64;
// A quintic that lifts small singular values quickly and keeps the others near one, for every step: K. Jordan's published
// coefficients (2024) for orthogonalising momentum by Newton-Schulz steps.
constexpr float kOrthoDefault[3] = {3.4445f, -4.7750f, 2.0315f};

ep_status check_ortho(const ep_ortho_config *c) {
    if (!c) return EP_ERR_INVALID_ARG;
    if (c->B < 0 || c->N <= 0 || c->K <= 0 || c->steps <= 0 || !(c->eps >= 0.0f && c->eps <= 3.4e38f)) return EP_ERR_INVALID_ARG;
    if (c->dtype != EP_F32 && c->dtype != EP_BF16 && c->dtype != EP_F16) return EP_ERR_INVALID_ARG;
    if (c->N > kMaxOrthoSide || c->K > kMaxOrthoSide || c->B > kMaxOrthoSide || c->steps > kMaxOrthoSteps) return EP_ERR_UNSUPPORTED;
    return EP_OK;
}

}  // namespace

extern "C" {

ep_status ep_block_norm(const ep_norm_config *cfg, const void *x, const ep_bf16 *y, const ep_bf16 *w_post, const void *gate,
                        const ep_bf16 *w_next, void *out, ep_bf16 *n, float *rstd_post, float *rstd_next,
                        cudaStream_t stream) {
    ep_status st = check_norm(cfg);
    if (st != EP_OK) return st;
    if (cfg->T == 0) return EP_OK;
    st = check_block(*cfg, x, y, w_post, gate, w_next, n != nullptr);
    if (st != EP_OK) return st;
    if ((out != nullptr) != (y != nullptr) || (!y && !n) || !aligned16(out) || !aligned16(n)) return EP_ERR_INVALID_ARG;
    if ((rstd_post && !w_post) || (rstd_next && !n) || !aligned(rstd_post, 4) || !aligned(rstd_next, 4)) return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_block_norm(*cfg, x, y, w_post, gate, w_next, out, n, rstd_post, rstd_next, stream));
}

ep_status ep_block_norm_workspace_size(const ep_norm_config *cfg, size_t *bytes) {
    const ep_status st = check_norm(cfg);
    if (st != EP_OK) return st;
    if (!bytes) return EP_ERR_INVALID_ARG;
    *bytes = ep::block_norm_workspace_bytes(*cfg);
    return EP_OK;
}

ep_status ep_block_norm_backward(const ep_norm_config *cfg, const void *x, const ep_bf16 *y, const ep_bf16 *w_post,
                                 const void *gate, const ep_bf16 *w_next, const float *rstd_post, const float *rstd_next,
                                 const void *d_out, const ep_bf16 *d_n, void *d_x, ep_bf16 *d_y, float *d_w_post,
                                 void *d_gate, float *d_w_next, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream) {
    ep_status st = check_norm(cfg);
    if (st != EP_OK) return st;
    const ep_norm_config &c = *cfg;
    const bool channel = c.gate == EP_GATE_CHANNEL;
    if (!aligned16(d_w_post) || !aligned16(d_w_next) || !aligned(d_gate, c.gate == EP_GATE_TOKEN ? 4 : 16)) return EP_ERR_INVALID_ARG;
    if (c.T == 0) {
        for (void *w : {static_cast<void *>(d_w_post), static_cast<void *>(d_w_next), channel ? d_gate : nullptr})
            if (w && cudaMemsetAsync(w, 0, (size_t)c.H * sizeof(float), stream) != cudaSuccess) return EP_ERR_CUDA;
        return EP_OK;
    }
    st = check_block(c, x, y, w_post, gate, w_next, d_n != nullptr);
    if (st != EP_OK) return st;
    if ((!d_out && !d_n) || !aligned16(d_out) || !aligned16(d_n) || !usable(d_x)) return EP_ERR_INVALID_ARG;
    if ((y != nullptr) != (d_y != nullptr) || !aligned16(d_y)) return EP_ERR_INVALID_ARG;
    if ((rstd_post != nullptr) != (w_post != nullptr) || (rstd_next != nullptr) != (d_n != nullptr)) return EP_ERR_INVALID_ARG;
    if (!aligned(rstd_post, 4) || !aligned(rstd_next, 4)) return EP_ERR_INVALID_ARG;
    if ((d_w_post && !w_post) || (d_w_next && !w_next) || (d_gate && !gate)) return EP_ERR_INVALID_ARG;
    if (d_w_post || d_w_next || (channel && d_gate)) {
        if (!usable(workspace)) return EP_ERR_INVALID_ARG;
        if (workspace_bytes < ep::block_norm_workspace_bytes(c)) return EP_ERR_CAPACITY;
    }
    return from_cuda(ep::launch_block_norm_backward(c, x, y, w_post, gate, w_next, rstd_post, rstd_next, d_out, d_n, d_x, d_y,
                                                    d_w_post, d_gate, d_w_next, static_cast<float *>(workspace), stream));
}

ep_status ep_balance_workspace_size(const ep_config *cfg, int32_t n_seq, size_t *bytes) {
    const int32_t any = 0;
    const ep_status st = check_balance(cfg, n_seq, &any, nullptr);
    if (st != EP_OK) return st;
    if (!bytes) return EP_ERR_INVALID_ARG;
    *bytes = ep::balance_workspace_bytes(*cfg, n_seq);
    return EP_OK;
}

ep_status ep_balance(const ep_config *cfg, int32_t n_seq, const float *logits, const int32_t *topk_idx,
                     const int32_t *seq_first, const int32_t *seq_len, int32_t *count, float *load, float *prob, float *loss,
                     void *workspace, size_t workspace_bytes, cudaStream_t stream) {
    const ep_status st = check_balance(cfg, n_seq, seq_first, seq_len);
    if (st != EP_OK) return st;
    if (cfg->T > 0 && (!logits || !topk_idx)) return EP_ERR_INVALID_ARG;
    if (!count || !load || !prob || !loss || !usable(workspace)) return EP_ERR_INVALID_ARG;
    for (const void *p : {(const void *)logits, (const void *)topk_idx, (const void *)count, (const void *)load, (const void *)prob, (const void *)loss})
        if (!aligned(p, 4)) return EP_ERR_INVALID_ARG;
    if (workspace_bytes < ep::balance_workspace_bytes(*cfg, n_seq)) return EP_ERR_CAPACITY;
    return from_cuda(ep::launch_balance(*cfg, n_seq, logits, topk_idx, seq_first, seq_len, count, load, prob, loss, workspace, stream));
}

ep_status ep_balance_backward(const ep_config *cfg, int32_t n_seq, const float *logits, const int32_t *seq_first,
                              const int32_t *seq_len, const float *load, const float *d_loss, const float *d_in,
                              float *d_logits, cudaStream_t stream) {
    const ep_status st = check_balance(cfg, n_seq, seq_first, seq_len);
    if (st != EP_OK) return st;
    if (cfg->T == 0) return EP_OK;
    if (!logits || !load || !d_loss || !d_logits) return EP_ERR_INVALID_ARG;
    for (const void *p : {(const void *)logits, (const void *)load, (const void *)d_loss, (const void *)d_in, (const void *)d_logits})
        if (!aligned(p, 4)) return EP_ERR_INVALID_ARG;
    return from_cuda(ep::launch_balance_backward(*cfg, n_seq, logits, seq_first, seq_len, load, d_loss, d_in, d_logits, stream));
}

ep_status ep_orthogonalize_workspace_size(const ep_ortho_config *cfg, size_t *bytes) {
    const ep_status st = check_ortho(cfg);
    if (st != EP_OK) return st;
    if (!bytes) return EP_ERR_INVALID_ARG;
    *bytes = ep::ortho_workspace_bytes(*cfg);
    return EP_OK;
}

ep_status ep_orthogonalize(const ep_ortho_config *cfg, const float *coefficients, const void *m, ep_bf16 *out, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream) {
    const ep_status st = check_ortho(cfg);
    if (st != EP_OK) return st;
    float k[3 * kMaxOrthoSteps];
    for (int i = 0; i < 3 * cfg->steps; ++i) k[i] = coefficients ? coefficients[i] : kOrthoDefault[i % 3];
    if (!ep::ortho_fits(k, cfg->steps)) return EP_ERR_UNSUPPORTED;
    if (cfg->B == 0) return EP_OK;
    if (!m || !aligned(m, cfg->dtype == EP_F32 ? 4 : 2) || !usable(out)) return EP_ERR_INVALID_ARG;
    // floats: one matrix's result would lie where another one is still to be read
    if (m == out && cfg->dtype == EP_F32) return EP_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return EP_ERR_INVALID_ARG;
    if (workspace_bytes < ep::ortho_workspace_bytes(*cfg)) return EP_ERR_CAPACITY;
    return from_cuda(ep::launch_orthogonalize(*cfg, k, m, out, workspace, stream));
}

}  // extern "C"
