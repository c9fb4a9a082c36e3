/*
 * msign_train.h - C ABI of the training-block operators of libmsign (gfx950):
 * the gated feed-forward block whose weights a Muon step updates, the
 * root-mean-square norm with the residual's addition in front of it, and the
 * distillation loss on a teacher's top logits, each with its gradient.
 *
 * Conventions (as in msign.h): pointers are device pointers; the caller owns
 * every buffer; nothing is allocated and no call synchronises the host; all
 * work is queued on `stream`.  Arguments are checked on the host before
 * anything is launched, and a status other than MSIGN_OK means that nothing
 * was launched (MSIGN_ERR_HIP: that a launch failed);
 * msign_train_last_error() then says why.  Results do not depend on timing:
 * every sum has a fixed order and no atomics are used.
 *
 * Matrices are row-major with unit stride along a row; a pitch is the
 * distance of two rows in elements, at least the row's length and, where
 * nothing else is said, at most 2^36.  dtype is one
 * of msign_dtype_t.  No output may overlap an input, another output or the
 * workspace, except where stated; a matrix counts from its first to its last
 * element, with what lies between its rows.
 */
#ifndef MSIGN_TRAIN_H_
#define MSIGN_TRAIN_H_

#include "msign.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FFN_SILU = 0, /* a(g) = g / (1 + exp(-g))                                   */
  FFN_GELU = 1  /* a(g) = g/2 (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3)))       */
} ffn_activation_t;

/*
 * A gated feed-forward block:
 *     g = x Wg^T,  u = x Wu^T,  h = a(g) * u,  y = h Wd^T
 * x [tokens, dim], w_gate and w_up [hidden, dim], w_down [dim, hidden], all
 * of `dtype`; ld_* are their pitches.  dim and hidden are at most 2^20,
 * tokens at most 2^24, pitches (those of the calls' other matrices too) at
 * most 2^21.
 */
typedef struct {
  int64_t tokens, dim, hidden;
  int32_t dtype, activation;
  const void *x, *w_gate, *w_up, *w_down;
  int64_t ldx, ld_gate, ld_up, ld_down;
} ffn_block_t;

/*
 * Bytes of workspace (256-byte aligned) of ffn_forward and ffn_backward for
 * this block.  Operands whose address or pitch is not a multiple of 16 bytes
 * or whose rows do not end on 16 bytes are copied there first: the struct's
 * addresses and pitches, and dy and ld_dy, count for that reason.
 * (size_t)-1: sizes or dtype are invalid.
 */
size_t ffn_forward_workspace_bytes(const ffn_block_t* b);
size_t ffn_backward_workspace_bytes(const ffn_block_t* b, const void* dy, int64_t ld_dy);

/*
 * y [tokens, dim] with pitch ldy.  gate and up, both null or both given: g
 * and u [tokens, hidden] with pitch ld_act, kept for ffn_backward.
 * g and u are summed in fp32; h is rounded once to dtype, as the matrix
 * instructions take it (with FP16, |h| above 65504 becomes infinite).
 */
msign_status_t ffn_forward(const ffn_block_t* b, void* y, int64_t ldy, void* gate, void* up, int64_t ld_act,
                           void* workspace, size_t workspace_bytes, hipStream_t stream);

/*
 * Gradients of sum(dy * y) from dy [tokens, dim] and ffn_forward's gate and up:
 *     dh = dy Wd,  du = dh a(g),  dg = dh u a'(g)
 *     dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x,  dWd = dy^T h
 * dx [tokens, dim], dw_gate, dw_up [hidden, dim] and dw_down [dim, hidden]
 * are contiguous.  dg, du and h are rounded once to dtype.
 */
msign_status_t ffn_backward(const ffn_block_t* b, const void* dy, int64_t ld_dy, const void* gate, const void* up,
                            int64_t ld_act, void* dx, void* dw_gate, void* dw_up, void* dw_down, void* workspace,
                            size_t workspace_bytes, hipStream_t stream);

/*
 * h = x + residual (residual null: h = x, and h_out is not written);
 * rstd = (mean(h^2) + eps)^(-1/2) over the `dim` values of a row;
 * y = h rstd weight.  Sums and products are in fp32 from the unrounded h.
 * x, residual, y and h_out are [tokens, dim] of dtype with pitches ldx, ldr
 * and, for the outputs, dim; weight [dim] is of w_dtype; rstd [tokens] is
 * fp32.  h_out may be x or residual themselves, if they are contiguous.
 * eps > 0.
 */
msign_status_t add_rms_norm(const void* x, int64_t ldx, const void* residual, int64_t ldr, const void* weight,
                            void* y, void* h_out, float* rstd, int64_t tokens, int64_t dim, int32_t dtype,
                            int32_t w_dtype, float eps, hipStream_t stream);

/*
 * From dy (the gradient of y), h, rstd and optionally dh (the gradient that
 * reaches h by the residual path; null: none):
 *     a = dy weight,  n = h rstd
 *     dx = rstd (a - n mean(a n)) + dh      (of x and of the residual alike)
 *     dweight = sum over tokens of dy n     (of w_dtype)
 * dy, h and dh have pitches; dx is contiguous and may be dy or dh themselves,
 * if they are contiguous.
 */
size_t add_rms_norm_backward_workspace_bytes(int64_t tokens, int64_t dim);
msign_status_t add_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ldh, const float* rstd,
                                     const void* weight, const void* dh, int64_t ld_dh, void* dx, void* dweight,
                                     int64_t tokens, int64_t dim, int32_t dtype, int32_t w_dtype, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream);

/*
 * Distillation on a teacher's top logits, per row of logits z [rows, vocab]:
 *     p = softmax(teacher / tau) over the row's valid entries
 *     q = softmax(z / tau) over the vocabulary
 *     loss = tau^2 sum_k p_k (log p_k - log q_{i_k})
 * indices [rows, top] (int32, or int64 where indices_64) and teacher
 * [rows, top] of teacher_dtype are contiguous; an entry is valid where
 * 0 <= index < vocab, and a row without valid entries has loss 0.  An index
 * may come more than once.  A logit of minus infinity has q = 0; a teacher's
 * logit of minus infinity has p = 0 and adds nothing.
 * If dlogits is given, it gets grad[row] tau (q - p) (p summed over equal
 * indices), in dtype, contiguous; rows without valid entries and rows whose
 * grad is 0 get zeros, whatever their logits are.  grad [rows] is fp32 with
 * stride grad_stride (0: one value for all rows).  dlogits may be the logits
 * themselves if they are contiguous.  loss [rows] is fp32.
 * tau is positive and finite; top is at most DISTILL_MAX_TOP.
 */
#define DISTILL_MAX_TOP 1024
msign_status_t distill_topk(const void* logits, int64_t ld_logits, const void* indices, int32_t indices_64,
                            const void* teacher, int32_t teacher_dtype, const float* grad, int64_t grad_stride,
                            float* loss, void* dlogits, int64_t rows, int64_t vocab, int64_t top, float tau,
                            int32_t dtype, hipStream_t stream);

/* Detail of the last non-OK status of these calls on the calling thread. */
const char* msign_train_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MSIGN_TRAIN_H_ */
