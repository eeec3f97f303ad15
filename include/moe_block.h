/*
 * moe_block.h -- C ABI of the operators a model needs directly around the
 * expert layer of moe_ffn.h, in training and in scoring, on one GB300:
 *
 *   moe_embedding_forward / _backward     token embedding and its gradient
 *   moe_block_norm_forward / _backward    RMS norms before and after a block,
 *                                         fused with its gate and residual
 *   moe_linear_ce_forward / _backward     softmax cross entropy of a linear
 *                                         layer, the logits never kept whole
 *   moe_clip_grad_norm                    global gradient norm and clipping
 *
 * The conventions are those of moe_ffn.h: device pointers owned by the
 * caller, nothing allocated, everything enqueued on `stream`, arguments
 * checked on the host before any launch, statuses of moe_status, a
 * caller-provided 256-byte aligned workspace whose first word is the status
 * word of moe_get_device_status.  Beyond them:
 *   - token ids and labels are int32; a negative one marks a masked token.  One
 *     at or above the vocabulary is treated as masked and recorded as
 *     MOE_ERR_DEVICE_INDEX in the workspace's status word.
 *   - pointers need their element's alignment only, unless the entry point
 *     says otherwise; 16-byte aligned rows (base, width and row stride) take
 *     the wide-load kernels.
 *   - results are bitwise reproducible on one device (no floating-point
 *     atomics): sums over tokens are split by a rule on the sizes and the
 *     number of SMs and joined in a fixed order.
 *   - values are computed in fp32 and rounded once to an output's type.
 *   - infinities and NaN of the inputs reach the outputs that their formula
 *     takes them to.
 */
#ifndef MOE_BLOCK_H_
#define MOE_BLOCK_H_

#include "moe_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F32 = 1 } moe_dtype;

/* ---- Block norms ----------------------------------------------------------
 * With y the block's output (branch), r the residual stream, w' = w +
 * weight_offset and rms(x) = sqrt(mean(x^2) + eps) over the row:
 *   v            = y / rms(y)            (v = y when w_post is NULL)
 *   residual_out = residual_scale * r + branch_scale * gate * v * w_post'
 *   normed       = residual_out / rms(residual_out) * w_pre'
 * that is, the norm after one block and the norm before the next.  `normed`
 * is computed from the unrounded residual_out. */
typedef enum {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1, /* gate [H], shared by the tokens */
  MOE_GATE_TOKEN = 2,   /* gate [T], shared by the channels */
  MOE_GATE_ELEMENT = 3  /* gate [T, H] dense */
} moe_gate_kind;

#define MOE_MAX_NORM_WIDTH 16384

typedef struct moe_norm_problem {
  int32_t T, H;           /* rows; width, 1 .. MOE_MAX_NORM_WIDTH */
  int32_t branch_dtype;   /* moe_dtype of branch, normed and their gradients */
  int32_t residual_dtype; /* of residual, residual_out and their gradients */
  int32_t weight_dtype;   /* of w_post, w_pre, gate and their gradients */
  int32_t gate_kind;      /* moe_gate_kind */
  float eps, weight_offset, residual_scale, branch_scale;
  /* Row strides in elements, >= H (0 = H): branch and d_branch; residual and
     d_residual; residual_out and d_residual_out; normed and d_normed. */
  int64_t ld_branch, ld_residual, ld_residual_out, ld_normed;
} moe_norm_problem;

/* Forward.  branch NULL: residual_out = r (residual_out must be NULL; w_post
 * and gate must be NULL and the scales do not apply), only the norm before
 * the block runs.  w_pre NULL: normed must be NULL, only the residual update
 * runs.  residual_out may be the same tensor as residual (equal row strides). */
MOE_API int moe_block_norm_forward(const moe_norm_problem* p, const void* branch,
                                   const void* w_post, const void* gate, const void* residual,
                                   const void* w_pre, void* residual_out, void* normed,
                                   void* stream);

/* Bytes of workspace of the backward (0 if the problem is invalid). */
MOE_API size_t moe_block_norm_workspace_size(const moe_norm_problem* p);

/* Backward, from the forward's inputs and its residual_out as stored (without
 * a branch: the residual itself); the norms' statistics are recomputed.
 *   d_normed        gradient of normed; NULL iff w_pre is
 *   d_residual_out  gradient of residual_out from later layers, NULL = zero
 *   d_residual      out; may be the same tensor as d_residual_out
 *   d_branch        out; NULL iff branch is
 *   d_w_post, d_gate, d_w_pre  out, shaped like their weight and written
 *                   exactly where the weight is given
 * The gradient of a shared gate is its sum over what it is shared by. */
MOE_API int moe_block_norm_backward(const moe_norm_problem* p, const void* branch,
                                    const void* w_post, const void* gate,
                                    const void* residual_out, const void* w_pre,
                                    const void* d_residual_out, const void* d_normed,
                                    void* d_residual, void* d_branch, void* d_w_post,
                                    void* d_gate, void* d_w_pre, void* ws, size_t ws_bytes,
                                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H_ */
