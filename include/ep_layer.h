/*
 * ep_layer.h -- C ABI of what surrounds an MoE layer in a model and its
 * training: the norms before and after a block with the block's gate and the
 * residual scale, the router's balance loss, and orthogonalised weight updates.
 *
 * The conventions are those of ep.h: device pointers the caller owns, dense and
 * row-major, nothing allocated, arguments checked on the host before anything is
 * enqueued, status codes, work asynchronous on `stream`. Like those of
 * ep_experts.h the kernels are launched as programmatic dependents: each waits
 * for the kernel before it on the stream before it touches memory.
 *
 * Workspaces need no initialisation and keep nothing between calls. Two calls
 * that may run at the same time (on two streams, or in two graphs that are
 * replayed side by side) need one each.
 */
#ifndef EP_GB300_LAYER_H
#define EP_GB300_LAYER_H

#include "ep_experts.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * The norms around a block
 * ------------------------------------------------------------------------ */

/* What a block's result is multiplied by before it joins the residual stream. */
typedef enum ep_gate {
    EP_GATE_NONE = 0,
    EP_GATE_CHANNEL = 1, /* gate: const bf16 [H], d_gate: float [H]                   */
    EP_GATE_TOKEN = 2,   /* gate: const float [T], d_gate: float [T]                  */
    EP_GATE_ELEMENT = 3  /* gate: const bf16 [T, H], d_gate: bf16 [T, H]              */
} ep_gate;

typedef struct ep_norm_config {
    int32_t T;            /* rows (>= 0)                                              */
    int32_t H;            /* hidden size (> 0, a multiple of 8, at most 16384)        */
    int32_t gate;         /* ep_gate                                                  */
    int32_t gate_sigmoid; /* 1: the gate goes through a sigmoid first                 */
    int32_t residual_f32; /* x, out, d_out, d_x: 0 bf16, 1 float                      */
    float eps;            /* added to the mean square (>= 0)                          */
    float scale;          /* residual scale: of what joins the stream                 */
    float weight_offset;  /* the norms multiply by weight_offset + weight             */
} ep_norm_config;

/*
 * ep_block_norm -- a block's result joins the residual stream, and the stream is
 * normed for the next block. For every row, with r(v) = 1 / sqrt(mean(v^2) + eps):
 *   z   = (weight_offset + w_post) y r(y)       (w_post NULL: z = y)
 *   out = x + scale act(gate) z                 (gate none: out = x + scale z)
 *   n   = (weight_offset + w_next) out r(out)   (n NULL: not wanted)
 * y NULL: there is no block yet, out = x, only n is computed (w_post, gate and out
 * are NULL then, and cfg->gate EP_GATE_NONE). Everything is fp32 and rounded once on
 * storing: n comes from out before that is rounded. The squares of a row are to stay
 * within fp32's range (beyond it r is 0).
 *
 * x, out    : const / bf16 or float [T, H]; out may be x
 * y, n      : const bf16 / bf16 [T, H]; n may be y, and x where x is bf16 and y NULL
 * w_post, w_next : const bf16 [H]; w_next exactly where n is given
 * rstd_post, rstd_next : optional float [T], r(y) and r(out), for the backward pass
 * T = 0 enqueues nothing. 16-byte aligned, but for the [T] ones (4 bytes).
 */
ep_status ep_block_norm(const ep_norm_config *cfg, const void *x, const ep_bf16 *y, const ep_bf16 *w_post,
                        const void *gate, const ep_bf16 *w_next, void *out, ep_bf16 *n, float *rstd_post,
                        float *rstd_next, cudaStream_t stream);

/* Bytes of device scratch that ep_block_norm_backward needs where it writes d_w_post,
 * d_w_next or a channel gate's d_gate. */
ep_status ep_block_norm_workspace_size(const ep_norm_config *cfg, size_t *bytes);

/*
 * ep_block_norm_backward -- gradients of ep_block_norm for d_out and d_n, those of
 * out and n. With gn = (weight_offset + w_next) d_n, r = r(out), and out computed
 * again from x and y, in fp32:
 *   D    = d_out + r gn - out r^3 mean(gn out)
 *   d_x  = D,   ez = scale act(gate) D,   ew = (weight_offset + w_post) ez
 *   d_y  = r(y) ew - y r(y)^3 mean(ew y)   (w_post NULL: d_y = ez)
 *   d_w_next = sum_t d_n out r;  d_w_post = sum_t ez y r(y)
 *   d_gate   = scale D z act'(gate), summed over what the gate is broadcast over
 * Sums over rows are fp32 in an order that depends on the configuration, on which
 * arguments are given and on the device only: results repeat bit by bit.
 *
 * x, y, w_post, gate, w_next, rstd_* : as for / from ep_block_norm (rstd_post with
 *             w_post, rstd_next with d_n)
 * d_out     : const bf16 or float [T, H], NULL for zeros; d_n : const bf16 [T, H],
 *             exactly where w_next is given; one of the two at least
 * d_x       : bf16 or float [T, H], may be d_out; d_y : bf16 [T, H], exactly where y
 *             is, may be d_n, which then is no input any more
 * d_w_post, d_w_next : optional float [H], overwritten; d_gate : optional
 * workspace : 16-byte aligned, may be NULL where ep_block_norm_workspace_size says so
 * T = 0 writes zeros to the sums over rows.
 */
ep_status ep_block_norm_backward(const ep_norm_config *cfg, const void *x, const ep_bf16 *y, const ep_bf16 *w_post,
                                 const void *gate, const ep_bf16 *w_next, const float *rstd_post,
                                 const float *rstd_next, const void *d_out, const ep_bf16 *d_n, void *d_x,
                                 ep_bf16 *d_y, float *d_w_post, void *d_gate, float *d_w_next, void *workspace,
                                 size_t workspace_bytes, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * The router's balance loss
 * ------------------------------------------------------------------------ */

/*
 * ep_balance -- per-expert counts of every sequence, and the two losses that a
 * router is trained with: that of balance (how often the experts of a sequence
 * were chosen, times the mean probability they were given) and that of the
 * logits' size (the squared log-sum-exp, "z").
 *
 * Sequence s owns rows [seq_first[s], seq_end(s)) of the T tokens, seq_end(s) being
 * seq_first[s + 1] or, with seq_len, seq_first[s] + seq_len[s] where that comes first
 * (padded batches). seq_first is non-decreasing; bounds outside [0, T] count as the
 * nearest one within, a negative seq_len as 0. Rows of no sequence are not read.
 * With N rows, p the softmax over all E logits of a row:
 *   count[s, e] = #{(t, j) : topk_idx[t, j] = e};   load[s, e] = count[s, e] / (k N)
 *   prob[s, e]  = sum_t p[t, e] / N
 *   loss[s, 0]  = E sum_e load[s, e] prob[s, e]     (1 for an even choice)
 *   loss[s, 1]  = sum_t logsumexp(logits[t, :])^2 / N
 * all zero for N = 0. The loss of a batch is the caller's weighted sum of them: the
 * weights are ep_balance_backward's d_loss.
 *
 * Logits are finite or -infinity (an expert that is masked: p = 0, no gradient). A row
 * of -infinities alone has p = 0 throughout and counts 0 in loss[s, 1]; a square
 * beyond fp32 makes that loss infinite and leaves the gradient finite. Ids outside
 * [0, E) are not counted. A NaN stays in its sequence.
 * Sums are fp32, exponentials within 2^-21 and with what is below fp32's normal range as 0. Their order depends on the sizes,
 * the bounds and the alignment of logits (16 bytes or less) only: results repeat bit by bit. counts are exact.
 * Which kernels run goes by T / n_seq: one sequence with most of the rows among many short ones is slow (131072 rows of 128
 * experts in 1024 sequences 27 us; with three quarters of the rows in one of them 0.7 ms).
 *
 * cfg       : T, E, k are used; n_seq sequences (>= 1)
 * logits    : const float [T, E];   topk_idx : const int32 [T, k]
 * seq_first : const int32 [n_seq + 1], or NULL with n_seq = 1: all T rows
 * seq_len   : optional const int32 [n_seq], with seq_first
 * count     : int32 [n_seq, E];  load, prob : float [n_seq, E];  loss : float [n_seq, 2]
 * workspace : 16-byte aligned, >= ep_balance_workspace_size bytes
 */
ep_status ep_balance_workspace_size(const ep_config *cfg, int32_t n_seq, size_t *bytes);

ep_status ep_balance(const ep_config *cfg, int32_t n_seq, const float *logits, const int32_t *topk_idx,
                     const int32_t *seq_first, const int32_t *seq_len, int32_t *count, float *load, float *prob,
                     float *loss, void *workspace, size_t workspace_bytes, cudaStream_t stream);

/*
 * ep_balance_backward -- the losses' gradient, added to another one of the logits
 * (ep_route_backward's): with s the row's sequence of N rows,
 *   d_logits[t, e] = d_in[t, e] + p[t, e] (c0 (load[s, e] - sum_i load[s, i] p[t, i]) + c1 lse)
 *   c0 = d_loss[s, 0] E / N,  c1 = 2 d_loss[s, 1] / N,  lse = logsumexp(logits[t, :])
 * Choosing experts has no gradient: load is a constant. It may be another one than
 * ep_balance's, for instance its mean over the processes that share a batch. A row of
 * no sequence gets d_in alone. The order of a row's sums depends on E and on the alignment of logits, load, d_in and d_logits.
 *
 * load   : const float [n_seq, E];  d_loss : const float [n_seq, 2], device
 * d_in   : const float [T, E], NULL for zeros;  d_logits : float [T, E], may be d_in
 */
ep_status ep_balance_backward(const ep_config *cfg, int32_t n_seq, const float *logits, const int32_t *seq_first,
                              const int32_t *seq_len, const float *load, const float *d_loss, const float *d_in,
                              float *d_logits, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Orthogonalised updates
 * ------------------------------------------------------------------------ */

typedef struct ep_ortho_config {
    int32_t B;     /* matrices (0 .. 65536)                                            */
    int32_t N, K;  /* rows and columns of each (1 .. 65536)                            */
    int32_t dtype; /* of m: ep_dtype                                                   */
    int32_t steps; /* Newton-Schulz steps (1 .. 64)                                    */
    float eps;     /* added to the norm (>= 0)                                         */
} ep_ortho_config;

/*
 * ep_orthogonalize -- every matrix of a batch, the update of an expert's weight for
 * instance, with its singular values drawn towards one and its singular vectors kept,
 * by Newton-Schulz products. For each matrix M:
 *   X = M / (|M| + eps), |M| the root of the sum of its squares
 *   step i: A = X X^T, X = a_i X + (b_i A + c_i A A) X     (with X^T X where N > K: the
 *   same result)
 *   out = X
 * The products take operands of fp16, whatever the type of m, with the known bounds of X, A and B as their
 * scale, the parts that matter most apart in higher precision, and are summed in fp32. Before
 * it is rounded to bf16 once (0.17% in norm) the result is, with the default coefficients,
 *   0.02 to 0.12% off in norm after five steps, up to 0.2% after ten, for matrices of 64 rows and columns or more, of
 *   whatever rank; 0.2 and 0.5% for 16 or more. Of fewer rows single roundings show (8 x 8, five steps: 0.12% in
 *   the mean, 0.4% at most of 3000).
 * Where M has fewer singular vectors than rows and columns, X gets some 2^-24 to 2^-22 of its norm in the directions that
 * M does not have, as in any fp32 arithmetic, and every step multiplies that by its a, on top of the above: of rank r
 * about 2^-22 3.44^steps / sqrt(r) (rank 1 of 1024 x 1024: 0.5% after eight steps, 5% after ten; in fp32 throughout 0.7 and 8),
 * until after some 13 steps those directions are as large as the others.
 * |M| is right at any size of the values. A matrix of zeros gives
 * zeros (eps > 0), a NaN or infinity makes its own matrix NaN. Results repeat bit by bit.
 *
 * coefficients : HOST float [steps][3] = (a, b, c) of each step, read during the call;
 *                NULL: (3.4445, -4.7750, 2.0315) for all. EP_ERR_UNSUPPORTED where a
 *                singular value of at most 1 could reach 4, or b u + c u^2 (u its square) 31
 * m         : const [B, N, K] of cfg->dtype, aligned to its values
 * out       : bf16 [B, N, K], 16-byte aligned; may be m where that is of 16 bits
 * workspace : 256-byte aligned, >= ep_orthogonalize_workspace_size bytes: about 8 bytes a
 *             value and 4 min(N, K)^2 a matrix, 256 for min(N, K) <= 128 and
 *             max(N, K) <= 2048, where every device keeps a matrix on the chip (up to 4096 where it has the place)
 * A CTA that gives up a bounded wait sets ep_device_error bit 5 (32).
 */
ep_status ep_orthogonalize_workspace_size(const ep_ortho_config *cfg, size_t *bytes);

ep_status ep_orthogonalize(const ep_ortho_config *cfg, const float *coefficients, const void *m, ep_bf16 *out,
                           void *workspace, size_t workspace_bytes, cudaStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* EP_GB300_LAYER_H */
