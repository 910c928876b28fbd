/*
 * ep_router.h -- token router, balance losses and their gradient.
 *
 * Part of the C ABI of libep_b200.so, beside ep.h, whose notation, status
 * codes, error word and stream rules hold here too: all tensors are dense
 * row-major device memory of the caller, on the device of the stream; nothing is
 * allocated, nothing synchronises, and every call may be captured.
 */
#ifndef EP_B200_ROUTER_H_
#define EP_B200_ROUTER_H_

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Router: the step before the layout.  One row of E logits per token becomes
 * the token's K experts and their gate weights (the topk_idx / topk_weights
 * that ep_get_layout, ep_dispatch and ep_combine take); for training, the
 * losses that keep the experts evenly used, and the gradient of the logits.
 *
 * Logits: bf16 or fp32 [T, E].  -inf (or NaN) closes an expert for the token:
 * it takes no part in anything and its gradient is 0; values above the
 * largest finite fp32 count as that value.  token_mask is uint8 [T] (0 = the
 * token is padding: it is routed nowhere, counts nowhere and its gradient is
 * 0), or NULL: every token takes part.
 *
 * For a token with open logits l, and its open experts e:
 *   s[e] = softmax(l)[e]  or  sigmoid(l[e])            (score)
 *   c[e] = s[e] + bias[e]  (fp32 [E], or NULL: 0)      the value chosen by;
 *          -inf or NaN in bias closes the expert for the choice alone.
 * With num_groups > 1 the experts are num_groups runs of E / num_groups; a
 * group's value is the sum of its group_top (1 or 2) largest c (of the one it
 * has, if only one is open), and only the topk_groups groups of the largest
 * values stay in the choice.
 * The K experts of the largest c are chosen in descending order; equal values
 * go to the lower id, for groups too.  The order is that of the values in
 * real arithmetic as far as fp64 tells them apart (without bias and groups,
 * that of the logits themselves), not that of fp32 roundings.
 * Weights: scale * s[e], or with normalize scale * s[e] / (sum of the chosen
 * experts' s); the bias is not part of them.  Where fewer than K experts can
 * be chosen, the slots left over get id -1 and weight 0.
 *
 * Limits: 0 <= T <= 2^30, T * E and T * K below 2^31; 1 <= E <= 1024; 1 <= K <= 32,
 * K <= E; num_groups a power of two up to 32 that divides E; 1 <= topk_groups
 * <= num_groups; group_top 1 or 2; scale finite.  logits aligned to their
 * element size.
 * ---------------------------------------------------------------------- */
typedef enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 } ep_score_t;

typedef struct {
    ep_score_t score;
    ep_dtype_t logits_dtype; /* EP_BF16 or EP_FP32 */
    int32_t num_tokens;
    int32_t num_experts;
    int32_t num_topk;
    int32_t num_groups; /* 1: no groups */
    int32_t topk_groups;
    int32_t group_top;
    int32_t normalize; /* 0 or 1 */
    float scale;
} ep_router_desc_t;

/* Logits -> topk_idx int64 [T, K] and topk_weights fp32 [T, K], as above. */
EP_API ep_status_t ep_router_topk(const ep_router_desc_t* router, const void* logits, const float* bias,
                                  const uint8_t* token_mask, int64_t* topk_idx, float* topk_weights,
                                  ep_stream_t stream);

/* Workspace of ep_balance_loss for this router and number of sequences (a
 * multiple of 256; 0 for a bad description).  Pure host function. */
EP_API size_t ep_balance_workspace_bytes(const ep_router_desc_t* router, int32_t num_seqs);

/* Balance loss, z loss and expert counts of each of S = num_seqs sequences.
 *   seq_offsets  int32 [S+1], not decreasing: sequence s is tokens
 *                [seq_offsets[s], seq_offsets[s+1]); NULL (with S = 1): all
 *                tokens.  Tokens of no sequence contribute nothing.  S at most
 *                2^24.  (Offsets that decrease leave the results undefined;
 *                nothing else is touched.)
 * Over the N tokens of sequence s that are not masked and have an open logit:
 *   counts      int32 [S, E]  entries of topk_idx [T, K] equal to e; ids
 *                             outside [0, E) are not counted
 *   mean_scores fp32 [S, E]   optional: P[e] = mean of q[e], q = s / sum(s)
 *                             (the softmax itself for EP_SCORE_SOFTMAX)
 *   losses      fp32 [S, 2]   [s, 0] = E / (K * N) * sum over e of counts[e] *
 *                             P[e];  [s, 1] = mean of logsumexp(l)^2
 *   seq_tokens  int32 [S]     N (0: losses, counts and mean_scores are 0)
 * Sums are fp32 in a fixed order: the same inputs give the same bytes.
 * workspace: ep_balance_workspace_bytes() bytes, 256-byte aligned; its contents
 * need no initialisation.  One workspace per stream: calls that share one must
 * not overlap on the GPU. */
EP_API ep_status_t ep_balance_loss(const ep_router_desc_t* router, const void* logits, const int64_t* topk_idx,
                                   const uint8_t* token_mask, const int32_t* seq_offsets, int32_t num_seqs,
                                   float* losses, int32_t* counts, int32_t* seq_tokens, float* mean_scores,
                                   void* workspace, size_t workspace_bytes, ep_stream_t stream);

/* Gradient of the logits, d_logits [T, E] (the logits' type), the sum of
 *   - that of the gate weights from d_topk_weights fp32 [T, K] (NULL: none),
 *     with the chosen ids held fixed; an id outside [0, E), or of a closed
 *     logit, has no weight;
 *   - that of the losses from d_losses fp32 [S, 2] (NULL: none), with the
 *     counts held fixed; needs counts and seq_tokens as ep_balance_loss wrote
 *     them for the same router, logits, token_mask, seq_offsets and num_seqs.
 * Masked tokens, closed logits and tokens without either gradient get 0.
 * d_logits must not overlap logits. */
EP_API ep_status_t ep_router_backward(const ep_router_desc_t* router, const void* logits, const int64_t* topk_idx,
                                      const uint8_t* token_mask, const float* d_topk_weights,
                                      const int32_t* seq_offsets, int32_t num_seqs, const int32_t* counts,
                                      const int32_t* seq_tokens, const float* d_losses, void* d_logits,
                                      ep_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* EP_B200_ROUTER_H_ */
