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
 *     says otherwise; rows of a width that is a multiple of 8 whose base and
 *     row stride are multiples of 16 bytes (bf16) or 32 (fp32) take the
 *     kernels of wide accesses.
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

/* ---- Gradient clipping by the global norm ---------------------------------
 *   norm = |grad_scale| * sqrt(sum over all tensors and elements of grad^2)
 *   coef = min(1, max_norm / (norm + eps))
 *   out  = grad * (grad_scale * coef)
 * grad_scale undoes a loss scale in the same pass.  Squares are summed in
 * fp32 over at most 65 elements of one thread, those sums in fp64; a thread's
 * sum that overflows fp32 or falls below 2^-80 (or to 0, of elements that are
 * not) is taken again in fp64, so the norm leaves the fp32 range only where it
 * is outside it itself. */
typedef struct moe_grad_tensor {
  const void* grad; /* device, numel elements, dense; any element alignment */
  void* out;        /* device, same type; may be grad; NULL: counted, not written */
  int64_t numel;
  int32_t dtype; /* moe_dtype */
  int32_t reserved;
} moe_grad_tensor;

#define MOE_MAX_GRAD_TENSORS (1 << 16)

/* Bytes of workspace for n tensors (0 if n is out of range). */
MOE_API size_t moe_clip_workspace_size(int32_t n);

/*   tensors   [n] in HOST memory, read before the call returns
 *   max_norm  >= 0; +infinity: only grad_scale is applied (coef 1, whatever the
 *             norm: an element that is not finite stays the only one)
 *   norm_out  [2] fp32 device out: norm and coef
 * Under a finite max_norm, a norm that is not finite gives the coef its formula
 * has (0 for infinity, NaN for NaN); the caller can read it from norm_out.  In
 * place, a factor of exactly 1 writes nothing. */
MOE_API int moe_clip_grad_norm(int32_t n, const moe_grad_tensor* tensors, float grad_scale,
                               float max_norm, float eps, float* norm_out, void* ws,
                               size_t ws_bytes, void* stream);

/* ---- Embedding ------------------------------------------------------------ */
typedef struct moe_embed_problem {
  int32_t T, V, H;      /* tokens, vocabulary, width */
  int32_t table_dtype;  /* moe_dtype of table and d_table */
  int32_t out_dtype;    /* of out and d_out */
  float scale;
} moe_embed_problem;

/* out[t] = scale * table[ids[t]]; a zero row for a masked token.
 *   ids [T] int32, table [V, H], out [T, H], dense
 *   ws  optional (NULL): any workspace whose status word gets the report of
 *       an id at or above V */
MOE_API int moe_embedding_forward(const moe_embed_problem* p, const int32_t* ids,
                                  const void* table, void* out, void* ws, void* stream);

/* Bytes of workspace of the backward (0 if the problem is invalid). */
MOE_API size_t moe_embedding_workspace_size(const moe_embed_problem* p);

/* d_table[v] = scale * sum of d_out[t] over the tokens with ids[t] = v, for
 * every v (zero rows where there is none; masked tokens count nowhere).  The
 * tokens are sorted by id (stable), so the order of the sums is fixed. */
MOE_API int moe_embedding_backward(const moe_embed_problem* p, const int32_t* ids,
                                   const void* d_out, void* d_table, void* ws, size_t ws_bytes,
                                   void* stream);

/* ---- Linear cross entropy --------------------------------------------------
 * With the logits z_tv = logit_scale * <x_t, w_v> of token t, which are
 * computed tile by tile on the tensor cores (fp32 accumulation) and never
 * kept whole:
 *   lse[t]  = log sum_v exp(z_tv)
 *   loss[t] = lse[t] - z_t,labels[t]   (0 for a masked token)
 * and, given the gradients d_loss [T] of loss and (optionally) d_lse [T] of
 * lse, with d_loss[t] taken as 0 for a masked token:
 *   d z_tv = (d_loss[t] + d_lse[t]) exp(z_tv - lse[t]) - d_loss[t] [v = labels[t]]
 *   dx[t]  = logit_scale * sum_v d z_tv w_v
 *   dw[v]  = logit_scale * sum_t d z_tv x_t
 * A masked token has a loss of 0 and an lse, and its weight in dw is
 * d_lse[t] exp(z - lse) or 0; as the formula has it, 0 times NaN is NaN, so the x
 * of a masked token has to be finite where dw is wanted.
 * x [T, H] and w [V, H] bf16, dense, 16-byte aligned; H a multiple of 8;
 * loss, lse, d_loss, d_lse fp32.  The backward recomputes the logits in pieces
 * of the vocabulary and rounds d z / max |d_loss| to bf16 for its two products,
 * as the layer's backward does its intermediate gradients; sums are fp32. */
typedef struct moe_ce_problem {
  int32_t T, H, V;
  float logit_scale;
} moe_ce_problem;

/* Bytes of workspace of the forward, and of both directions (0 if the problem
 * is invalid). */
MOE_API size_t moe_linear_ce_workspace_size(const moe_ce_problem* p);
MOE_API size_t moe_linear_ce_backward_workspace_size(const moe_ce_problem* p);

MOE_API int moe_linear_ce_forward(const moe_ce_problem* p, const void* x, const void* w,
                                  const int32_t* labels, float* loss, float* lse, void* ws,
                                  size_t ws_bytes, void* stream);

/* lse as the forward wrote it; d_lse may be NULL (zero). */
MOE_API int moe_linear_ce_backward(const moe_ce_problem* p, const void* x, const void* w,
                                   const int32_t* labels, const float* lse, const float* d_loss,
                                   const float* d_lse, void* dx, void* dw, void* ws,
                                   size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H_ */
