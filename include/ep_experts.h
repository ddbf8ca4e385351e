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
 * The kernels here are launched as programmatic dependents, as ep_combine is
 * (ep.h): each waits for the kernel before it on the stream before it touches
 * memory.
 *
 * Rows lie grouped by expert, as ep_layout and ep_dispatch leave them: expert e
 * owns rows [expert_offset[e], expert_offset[e + 1]) of the row buffers, with
 * expert_offset (int32 [E + 1], device) non-decreasing and within [0, rows].
 * Bounds outside that are clamped into the buffer. expert_offset[0] need not
 * be 0: passing `expert_offset + e0`, weights from expert e0 on and a smaller E
 * runs part of the experts, one rank's for instance. Rows that no expert owns
 * are not written, and no result depends on what they hold (they may be fetched
 * along with the rows beside them).
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
    int32_t saved_bf16; /* g and u, kept for the backward pass: 0 IEEE halves, 1 bf16
                           (not there before ep_version 200)                             */
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
 * g, u   : 16-bit [rows, I] outputs for ep_expert_ffn_backward, both or neither
 *          (NULL): the fp32 sums that h is made of, in the type that cfg->saved_bf16
 *          names, whatever the caller's memory is declared as. Halves round eight
 *          times finer than bf16 from 6.1e-5 to 65504; finite sums beyond that are
 *          kept as 65504 with their sign (h and y are not limited), and below it a
 *          half's step is 6e-8, whatever the value. bf16 holds the whole range of
 *          the sums
 * h      : bf16 [rows, I] output
 * y      : bf16 [rows, H] output
 * With and without g and u, and with few or many rows, other kernels may run,
 * whose sums go in another order; the same call repeats bit by bit.
 * All 16-byte aligned. rows = 0 enqueues nothing. Outputs must not overlap
 * inputs. A CTA that gives up a bounded wait sets ep_device_error bit 4 (16).
 */
ep_status ep_expert_ffn(const ep_ffn_config *cfg, const ep_bf16 *rows, const int32_t *expert_offset,
                        const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, uint16_t *g, uint16_t *u,
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
 * The gradients are those of the g and u that were kept (cfg->saved_bf16 as in
 * the forward call). With halves: beyond 65504 d_u is that of g = 65504 with its
 * sign, d_g that of u = 65504; where g and u are all small, d_u and d_g are off by
 * what a half's step of 6e-8 is of g and u, 0.2% at 1e-5, 2% at 1e-6, 20% at 1e-7.
 * With bf16 each is within 2^-8 at any size; over values between 6.1e-5 and 65504
 * the weights' gradients are then 0.0031 off in norm, 0.0024 with halves.
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
                                 const ep_bf16 *w_gate, const ep_bf16 *w_up, const ep_bf16 *w_down, const uint16_t *g,
                                 const uint16_t *u, const ep_bf16 *h, const ep_bf16 *d_y, ep_bf16 *d_g, ep_bf16 *d_u,
                                 ep_bf16 *d_rows, ep_bf16 *d_w_gate, ep_bf16 *d_w_up, ep_bf16 *d_w_down,
                                 cudaStream_t stream);

/*
 * Products with 4-bit weights, for few rows (decoding): each weight is
 * scale (q - 8) with q in 0 .. 15 and one bf16 scale for `group` consecutive k.
 *
 * Packed form of a weight [E, N, K]: K is filled up to Kp, a multiple of 128,
 * with q = 8.
 *   q     : uint8 [E, N, Kp / 2]. A row is 32-bit little-endian words; word
 *           16 c + 4 t + j (t, j = 0 .. 3) holds k = k0 .. k0 + 7 with
 *           k0 = 128 c + 32 j + 8 t, and its nibble i (bits 4 i .. 4 i + 3) the
 *           one at k0 + 2 (i mod 4) + i / 4.
 *   scale : bf16 [E, N, Kp / group], scale[e, n, k / group]
 */
typedef struct ep_w4_config {
    int32_t rows;  /* rows of x and y (>= 0)                    */
    int32_t N;     /* outputs (> 0)                              */
    int32_t K;     /* inputs (> 0, a multiple of 8)              */
    int32_t E;     /* experts (1 .. 1024); 1: an ordinary layer  */
    int32_t group; /* k of one scale: 32, 64 or 128              */
} ep_w4_config;

/* Bytes of the packed form's q and scale (rows is not looked at). */
ep_status ep_w4_sizes(const ep_w4_config *cfg, size_t *q_bytes, size_t *scale_bytes);

/*
 * ep_w4_pack -- rounds bf16 weights to 4 bits: per group
 *   scale = bf16(max |w| / 7), q = clamp(rint(w / scale), -8, 7) + 8
 * (q = 8 where scale is 0). Weights must be finite.
 *
 * w : const bf16 [E, N, K], 16-byte aligned; q and scale 16-byte aligned.
 */
ep_status ep_w4_pack(const ep_w4_config *cfg, const ep_bf16 *w, uint8_t *q, ep_bf16 *scale, cudaStream_t stream);

/*
 * ep_w4_linear -- y[s, n] = sum_k x[s, k] w[e, n, k], e the expert that owns
 * row s, w the packed weight's values. The products x (q - 8) are exact; they are
 * summed in fp32 over a group, times its scale, then over the groups; y is rounded
 * to bf16 once. An infinite x times a weight has the weight's sign, and is NaN
 * where q = 8. Right for any number of rows; made for few: the weights are read
 * once for every 16 rows of an expert.
 *
 * x : const bf16 [rows, K], 16-byte aligned
 * y : bf16 [rows, N] output, 16-byte aligned
 */
ep_status ep_w4_linear(const ep_w4_config *cfg, const ep_bf16 *x, const int32_t *expert_offset, const uint8_t *q,
                       const ep_bf16 *scale, ep_bf16 *y, cudaStream_t stream);

/*
 * ep_expert_ffn_w4 -- ep_expert_ffn's forward pass with 4-bit weights: q_gate,
 * q_up packed [E, I, H], q_down packed [E, H, I], all with the same group. Two
 * kernels, as there; h is rounded to bf16 between them.
 */
ep_status ep_expert_ffn_w4(const ep_ffn_config *cfg, int32_t group, const ep_bf16 *rows, const int32_t *expert_offset,
                           const uint8_t *q_gate, const ep_bf16 *s_gate, const uint8_t *q_up, const ep_bf16 *s_up,
                           const uint8_t *q_down, const ep_bf16 *s_down, ep_bf16 *h, ep_bf16 *y, cudaStream_t stream);

/*
 * ep_combine_backward -- the gradients of ep_combine for d_out, the gradient of
 * its out:
 *   d_y[slot[t, j], :] = bf16(topk_w[t, j] d_out[t, :])
 *   d_topk_w[t, j]     = sum_h d_out[t, h] y[slot[t, j], h]
 * Sums in fp32. A slot outside [0, T k) writes no row, and 0 to d_topk_w. The
 * gradient of ep_dispatch is ep_combine itself with weights of one: it sums the
 * k rows of every token's gradient.
 *
 * d_out    : const bf16 [T, H]           y   : const bf16 [T k, H]
 * slot     : const int32 [T, k]          topk_w : const float [T, k]
 * d_y      : bf16 [T k, H] output        d_topk_w : float [T, k] output
 * d_out, y, d_y 16-byte aligned; d_y may not overlap y.
 */
ep_status ep_combine_backward(const ep_config *cfg, const ep_bf16 *d_out, const ep_bf16 *y, const int32_t *slot,
                              const float *topk_w, ep_bf16 *d_y, float *d_topk_w, cudaStream_t stream);

/*
 * ep_route_backward -- the gradient of ep_route's weights with respect to the
 * logits (the choice itself has none). With inner = sum_i topk_w_i d_topk_w_i:
 *   renormalize: d_logits[t, idx_j] = topk_w_j (d_topk_w_j - inner), 0 elsewhere
 *   else       : d_logits[t, e] = p_e (d_e - inner), p the softmax over all E
 *                logits, d_e = d_topk_w_j for e = idx_j and 0 for the others
 *
 * logits   : const float [T, E]; read only without renormalize (else may be NULL)
 * topk_idx : const int32 [T, k], distinct in a row; ids outside [0, E) count
 *            for inner only
 * topk_w, d_topk_w : const float [T, k]
 * d_logits : float [T, E] output
 */
ep_status ep_route_backward(const ep_config *cfg, const float *logits, const int32_t *topk_idx, const float *topk_w,
                            const float *d_topk_w, float *d_logits, cudaStream_t stream);

/* One gradient tensor of a list: numel values at `data` (device), dense. */
typedef enum ep_dtype { EP_F32 = 0, EP_BF16 = 1, EP_F16 = 2 } ep_dtype;

typedef struct ep_grad_tensor {
    const void *data; /* aligned to its values                                     */
    void *out;        /* ep_grad_clip: where the clipped values go; data itself, or
                         memory that overlaps no tensor of the list                */
    int64_t numel;    /* >= 0                                                      */
    int32_t dtype;    /* ep_dtype                                                  */
    int32_t reserved; /* 0                                                         */
} ep_grad_tensor;

/* Bytes of device scratch that the two calls below need for n tensors. */
ep_status ep_grad_workspace_size(int32_t n, size_t *bytes);

/*
 * ep_grad_norm -- norm[0] = sqrt(sum of the squares of all values of all
 * tensors), fp32. Values are squared and added up in fp32, in short chains whose
 * sums are joined in 64 bits, in an order that depends on the sizes and on the
 * tensors' alignment only. Values whose squares leave fp32's range are scaled by
 * 2^90 or 2^-90 first. The result repeats bit by bit and is within 2e-5 of
 * exact at any size of the values, infinite where the norm itself is beyond fp32.
 *
 * tensors   : HOST array of n records (n >= 0), read during the call
 * workspace : device, 8-byte aligned, >= ep_grad_workspace_size bytes
 */
ep_status ep_grad_norm(const ep_grad_tensor *tensors, int32_t n, float *norm, void *workspace, size_t workspace_bytes,
                       cudaStream_t stream);

/*
 * ep_grad_clip -- ep_grad_norm, then for every value
 *   out = data min(1, max_norm / (norm + 1e-6))
 * in fp32, rounded to the tensor's type. No host synchronisation. A NaN in the
 * norm passes to every value; an infinite norm gives a factor of 0.
 * max_norm >= 0. The norm is that of this list: where it is to span the
 * gradients of several processes, use ep_grad_norm, join the processes' norms
 * and call ep_grad_clip_with_norm.
 */
ep_status ep_grad_clip(const ep_grad_tensor *tensors, int32_t n, float max_norm, float *norm, void *workspace,
                       size_t workspace_bytes, cudaStream_t stream);

/*
 * ep_grad_clip_with_norm -- ep_grad_clip's second half: the same for a norm that
 * is given, norm[0] (const float, device, 4-byte aligned), read when the stream
 * gets there. It may not be part of an output. No host synchronisation.
 */
ep_status ep_grad_clip_with_norm(const ep_grad_tensor *tensors, int32_t n, float max_norm, const float *norm,
                                 cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_GB300_EXPERTS_H */
