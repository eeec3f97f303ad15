/*
 * moe_experts.h -- C ABI of the operators a layer of many experts needs around
 * its products when its weights are held in 8 bits, on one GB300:
 *
 *   moe_router_forward / _backward    softmax or sigmoid scores, a balance bias,
 *                                     groups of experts, top-k, their weights
 *   moe_fp8_quantize_rows             rows, or SwiGLU of their halves, to E4M3
 *                                     with a scale per 128 values
 *   moe_fp8_quantize_weights          weights to E4M3 with a scale per 128 x 128
 *   moe_fp8_matmul                    the product of the two, grouped by expert
 *                                     or dense
 *
 * As a layer: moe_router_forward gives the topk_idx and topk_w that
 * moe_forward_routed, moe_backward_routed and moe_permute take (and
 * moe_router_backward takes moe_backward_routed's d_topk_w); in 8 bits the rows
 * that moe_fp8_quantize_rows writes are permuted by moe_permute_rows, go through
 * moe_fp8_matmul with W1, moe_fp8_quantize_rows with SwiGLU and moe_fp8_matmul
 * with W2, and moe_unpermute_combine adds them up.
 *
 * The conventions are those of moe_ffn.h and moe_block.h: device pointers owned
 * by the caller, nothing allocated, everything enqueued on `stream`, arguments
 * checked on the host before any launch, statuses of moe_status; results are
 * bitwise reproducible; values are computed in fp32 and rounded once to an
 * output's type; infinities and NaN of the inputs reach the outputs that their
 * formula takes them to.  E4M3 is the 8-bit format with 3 bits of mantissa, no
 * infinities and a largest value of 448.
 */
#ifndef MOE_EXPERTS_H_
#define MOE_EXPERTS_H_

#include "moe_block.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- Router ----------------------------------------------------------------
 * For every token, with l its logits over the E experts:
 *   s     = softmax(l) or sigmoid(l)
 *   c     = s + bias                      (bias moves the choice, not the weights)
 * The experts lie in `groups` equal groups of consecutive ids.  A group's score is
 * the sum of its group_top highest c; the topk_groups groups of the highest scores
 * stay, and of their experts the k of the highest c are chosen, highest first.
 * Equal c (equal scores) go to the lowest id.  Without a bias the experts, and
 * groups by one expert, are ordered by their logits; otherwise c and the groups'
 * scores are compared as 64 bits have them: fp32 values that are too near to tell are
 * computed again, in pairs of fp32 and in fp64 where those do not tell.
 *   w_j   = scale * s_j / (renormalize ? sum over the chosen of s : 1)
 * An expert whose logit is -infinity is out of the token's choice: it counts in
 * no group, and slots for which no expert is left get the id -1, which masks a
 * route elsewhere, and the weight 0.  A NaN c ranks below every number. */
typedef enum { MOE_SCORE_SOFTMAX = 0, MOE_SCORE_SIGMOID = 1 } moe_score_kind;

#define MOE_MAX_EXPERT_GROUPS 32

typedef struct moe_router_problem {
  int32_t T, E, k;       /* tokens; experts, up to MOE_MAX_EXPERTS; chosen, up to MOE_MAX_TOPK */
  int32_t logits_dtype;  /* moe_dtype of logits and d_logits */
  int32_t score;         /* moe_score_kind */
  int32_t groups;        /* divides E; 1 .. MOE_MAX_EXPERT_GROUPS */
  int32_t topk_groups;   /* 1 .. groups, with k experts in them */
  int32_t group_top;     /* 1 or 2 (2: at least two experts in a group) */
  int32_t renormalize;
  float scale;
  int64_t ld_logits;     /* row stride in elements of logits and d_logits, >= E (0 = E) */
} moe_router_problem;

/*   logits   [T, E]
 *   bias     [E] fp32 or NULL (zero)
 *   topk_idx [T, k] int32 out, topk_w [T, k] fp32 out */
MOE_API int moe_router_forward(const moe_router_problem* p, const void* logits, const float* bias,
                               int32_t* topk_idx, float* topk_w, void* stream);

/* Gradient of the logits from the gradients of the weights; the choice passes
 * none.  Sigmoids' and renormalised weights go by the chosen experts' logits alone,
 * and so does their gradient: the others get 0, whatever their logits are.  Every
 * element of d_logits [T, E] is written (not what lies between its rows).
 *   topk_idx  [T, k] as the forward wrote it; an id outside [0, E) is a masked slot
 *   d_topk_w  [T, k] fp32 (masked slots' values are not used) */
MOE_API int moe_router_backward(const moe_router_problem* p, const void* logits,
                                const int32_t* topk_idx, const float* d_topk_w, void* d_logits,
                                void* stream);

/* ---- Quantisation ----------------------------------------------------------
 * For every block: scale = max |v| / 448 (1 where every v is 0, and 2^-126 at
 * least), code = E4M3(v / scale), rounded to nearest, ties to even; both quotients
 * are those of fp32.  A block with a NaN, or an infinity, has that as its scale;
 * its codes are what v / scale has then (NaN, and 0 for the finite values next to
 * an infinity). */

/* Rows: a block is 128 consecutive values of a row (the last one may be
 * shorter).  With swiglu a row of src holds 2H pre-activations and
 *   v = silu(min(g, c)) * clamp(u, -c, c)
 * of its gate and up values g and u, which lie as moe_problem.glu_interleave has
 * them (0: halves; I: alternating blocks of I); c as moe_problem.swiglu_clamp. */
typedef struct moe_quant_problem {
  int32_t T, H;            /* rows; width of the codes, a multiple of 16 */
  int32_t src_dtype;       /* moe_dtype */
  int32_t swiglu;
  int32_t glu_interleave;  /* 0, or a multiple of 16 that divides H */
  float swiglu_clamp;
  int64_t ld_src;          /* row stride of src in elements, a multiple of 8, >= its width (0 =) */
} moe_quant_problem;

/*   src    [T, H] or [T, 2H], 16-byte aligned
 *   codes  [T, H] out, dense, 16-byte aligned
 *   scales [T, ceil(H / 128)] fp32 out */
MOE_API int moe_fp8_quantize_rows(const moe_quant_problem* p, const void* src, void* codes,
                                  float* scales, void* stream);

/* Weights: a block is 128 x 128 values of one expert's [N, K] (fewer at its
 * edges). */
typedef struct moe_quant_weights_problem {
  int32_t E, N, K;    /* experts; rows; width, a multiple of 16 */
  int32_t src_dtype;  /* moe_dtype */
} moe_quant_weights_problem;

/*   src      [E, N, K] dense, 16-byte aligned
 *   codes    [E, N, K] out, 16-byte aligned
 *   scales   [E, ceil(N / 128), ceil(K / 128)] fp32 out
 *   codes_t  [E, K, N] out, 16-byte aligned, and scales_t [E, ceil(K / 128), ceil(N / 128)]
 *            out: the same blocks transposed, for the gradient of the product's
 *            rows (N then has to be a multiple of 16); both or neither */
MOE_API int moe_fp8_quantize_weights(const moe_quant_weights_problem* p, const void* src,
                                     void* codes, float* scales, void* codes_t, float* scales_t,
                                     void* stream);

/* ---- Product ---------------------------------------------------------------
 *   out[r, n] = sum over blocks b of 128 along K of
 *     x_scale[r, b] * w_scale[e, n / 128, b] * <x[r, b], w[e, n, b]>
 * for the rows r of every expert e.  A block's products are summed by the tensor
 * cores, the blocks in fp32; the two scales are multiplied first, so that their
 * product has to be a number of fp32 (it loses bits below 2^-126).  The gradient of the rows is the same product with
 * the transposed codes: d_x[r] = d_out[r] W_e, rows of d_out quantised as x. */
typedef struct moe_fp8_problem {
  int32_t M, N, K;    /* rows of all experts; width of out; length of the sums, a multiple of 16 */
  int32_t E;          /* experts, up to MOE_MAX_EXPERTS */
  int32_t out_dtype;  /* moe_dtype */
} moe_fp8_problem;

/* Bytes of workspace (0 if the problem is invalid). */
MOE_API size_t moe_fp8_matmul_workspace_size(const moe_fp8_problem* p);

/*   x        [M, K] E4M3 codes, x_scale [M, ceil(K / 128)] fp32
 *   w        [E, N, K] E4M3 codes, w_scale [E, ceil(N / 128), ceil(K / 128)] fp32
 *   expert_offsets [E + 1] int32: expert e has the rows offsets[e] .. offsets[e + 1];
 *            NULL: every row is expert 0's (E = 1).  Offsets that decrease or leave
 *            [0, M] are recorded as MOE_ERR_DEVICE_INDEX, and no row is written.
 *   out      [M, N], dense; rows outside the experts' are left as they were
 * x, w and out are 16-byte aligned. */
MOE_API int moe_fp8_matmul(const moe_fp8_problem* p, const void* x, const float* x_scale,
                           const void* w, const float* w_scale, const int32_t* expert_offsets,
                           void* out, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EXPERTS_H_ */
