/*
 * ep_experts.h -- C ABI of what stands between dispatch and combine, and of
 * the way back: the experts' gated feed-forward block (forward and backward),
 * the same block with 4-bit weights for decoding, the backward pass of combine
 * and router, and the global gradient norm with clipping.
 *
 * The conventions are those of ep.h: device pointers the caller owns, dense and
 * row-major, nothing allocated, arguments checked on the host before anything
 * is enqueued, status codes, work asynchronous on `stream`.
 *
 * Rows lie grouped by expert, as ep_layout and ep_dispatch leave them: expert e
 * owns rows [expert_offset[e], expert_offset[e + 1]) of the row buffers, with
 * expert_offset (int32 [E + 1], device) non-decreasing and within [0, rows].
 * Bounds outside that are clamped into the buffer. expert_offset[0] need not
 * be 0: passing `expert_offset + e0`, weights from expert e0 on and a smaller E
 * runs part of the experts, one rank's for instance. Rows that no expert owns
 * are neither read nor written.
 */
#ifndef EP_GB300_EXPERTS_H
#define EP_GB300_EXPERTS_H

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The shape of one layer's experts. */
typedef struct ep_ffn_config {
    int32_t rows; /* rows of the row buffers (>= 0)                                       */
    int32_t H;    /* hidden size (> 0, a multiple of 8)                                    */
    int32_t I;    /* width of the block between its projections (> 0, a multiple of 8)     */
    int32_t E;    /* experts (1 .. 1024)                                                   */
} ep_ffn_config;

/*
 * ep_expert_ffn -- every expert's gated feed-forward block over its rows:
 *   g = x Wg^T, u = x Wu^T, h = silu(g) u, y = h Wd^T,    silu(g) = g / (1 + exp(-g))
 * with x a row and Wg, Wu, Wd the weights of the expert that owns it. Sums are
 * fp32; h is rounded to bf16 (it is the operand of the second product), y once
 * at the end.
 *
 * Two kernels: both first projections, the activation and the product in one,
 * the last projection in the other.
 *
 * rows   : const bf16 [rows, H]
 * w_gate : const bf16 [E, I, H]     w_up : const bf16 [E, I, H]
 * w_down : const bf16 [E, H, I]
 * g, u   : bf16 [rows, I] outputs for ep_expert_ffn_backward, both or neither
 *          (NULL); rounded from the same fp32 sums that h is made of
 * h      : bf16 [rows, I] output
 * y      : bf16 [rows, H] output
 * All 16-byte aligned. rows = 0 enqueues nothing. Outputs must not overlap
 * inputs. A CTA that gives up a bounded wait sets ep_device_error bit 4 (16).
 */
ep_status ep_expert_ffn(const ep_ffn_config *cfg, const ep_bf16 *rows, const int32_t *expert_offset,
                        const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, ep_bf16 *g, ep_bf16 *u,
                        ep_bf16 *h, ep_bf16 *y, cudaStream_t stream);

/*
 * ep_expert_ffn_backward -- the gradients of ep_expert_ffn for d_y, the gradient
 * of y, from the g, u and h that it wrote:
 *   dh = d_y Wd, s = 1 / (1 + exp(-g))
 *   d_u = dh g s, d_g = dh u s (1 + g (1 - s))
 *   d_rows = d_g Wg + d_u Wu
 *   d_w_down[e] = sum d_y^T h, d_w_gate[e] = sum d_g^T x, d_w_up[e] = sum d_u^T x
 * the sums over the rows of expert e; the gradients of an expert without rows
 * are zero. Sums are fp32; d_g and d_u are rounded to bf16, the results once at
 * the end.
 *
 * d_y                     : const bf16 [rows, H]
 * d_g, d_u                : bf16 [rows, I] outputs
 * d_rows                  : bf16 [rows, H] output, or NULL where it is not wanted
 * d_w_gate, d_w_up        : bf16 [E, I, H] outputs, overwritten, or NULL
 * d_w_down                : bf16 [E, H, I] output, overwritten, or NULL
 * The other arguments are ep_expert_ffn's. rows = 0 sets the weights'
 * gradients to zero.
 */
ep_status ep_expert_ffn_backward(const ep_ffn_config *cfg, const ep_bf16 *rows, const int32_t *expert_offset,
                                 const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, const ep_bf16 *g,
                                 const ep_bf16 *u, const ep_bf16 *h, const ep_bf16 *d_y, ep_bf16 *d_g, ep_bf16 *d_u,
                                 ep_bf16 *d_rows, ep_bf16 *d_w_gate, ep_bf16 *d_w_up, ep_bf16 *d_w_down,
                                 cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_GB300_EXPERTS_H */
