/*
 * ep_lora.h -- low-rank adapters on the rows of a layout, and their gradients.
 *
 * Part of the C ABI of libep_b200.so, beside ep.h, whose notation, status
 * codes, error word and stream rules hold here too: all tensors are dense
 * row-major device memory of the caller, on the device of the stream; nothing is
 * allocated, nothing synchronises, and every call may be captured.
 */
#ifndef EP_B200_LORA_H_
#define EP_B200_LORA_H_

#include "ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Low-rank adapters beside a shared projection (token-choice routing).  The
 * routing names the adapter of every row, the layout groups the rows by
 * adapter, and the call adds each row's low-rank product to what the shared
 * projection gave:
 *   h[row]   = scales[e] * A[e] x[row]          fp32 [num_rows, rank]
 *   out[row] = base[row] + B[e] h[row]          rounded once to bf16
 * for every row of every adapter e.  Rows are those of ep_dispatch (COMPACT:
 * expert_offsets[e] + slot; PADDED: e * max_tokens_per_expert + slot).
 *
 * Where x, base and out are found depends on row_token:
 *   NULL       x bf16 [num_rows, hidden_in], base and out bf16 [num_rows,
 *              hidden_out] are dispatched rows (recv_x of ep_dispatch, the
 *              y that ep_combine takes): the low-rank part of the experts.
 *              Rows that no pair names are left as they are.
 *   int32      [num_rows], the source token of every row, as ep_row_tokens or
 *              ep_dispatch (recv_src) writes it: x, base and out are [T, ...]
 *              in token order and nothing is copied into groups; each token
 *              uses one adapter, so this form needs num_topk = 1 (the requests'
 *              adapter ids as topk_idx [T, 1], -1 = no adapter).  A token with
 *              no adapter gets out = base.  An entry outside [0, T) is skipped
 *              and flagged EP_DEVERR_BAD_INDEX.  (With num_rows 0 nothing is
 *              read, but the pointer still tells the two forms apart.)
 * h is always in row order.  One layout and one row_token serve every
 * projection of a step.
 *   a       bf16 [E, rank, hidden_in]    b  bf16 [E, hidden_out, rank]
 *   scales  fp32 [E], or NULL: 1
 *   base    NULL: zeros.  out may be the same buffer as base; otherwise no
 *           output may overlap an input.
 * The products run on the tensor cores with fp32 sums; fp32 operands (h, dh)
 * enter them as three bf16 terms, which keep all of their bits, and no more than
 * 24 products in a row are summed there before fp32 arithmetic adds them up.
 * Sums are taken in a fixed order: the same call gives the same bytes.
 * Limits: num_rows <= 2^31 - 1024; rank a multiple of 8, 8 <= rank <= 128;
 * hidden_in and hidden_out positive multiples of 8 up to 2^20; E <= 1024; T * K
 * <= 2^24; x, a, b, base, out, h and the gradients 16-byte aligned.  Rows at or
 * past num_rows are skipped with EP_DEVERR_OVERFLOW.  The layout is the routing's own: with one that has rows of
 * more pairs than the routing (of which the routing is a part) all rows are
 * skipped and flagged so.
 * ---------------------------------------------------------------------- */
typedef struct {
    int32_t rank;
    int32_t hidden_in;
    int32_t hidden_out;
    const void* a;
    const void* b;
    const float* scales;
} ep_lora_desc_t;

/* row_token[row] = t for the row of every routed pair (t, k), -1 for the
 * other rows of [0, num_rows): recv_src of ep_dispatch, without a dispatch.
 * A row at or past num_rows is skipped with EP_DEVERR_OVERFLOW. */
EP_API ep_status_t ep_row_tokens(const ep_routing_desc_t* routing, const ep_layout_t* layout, ep_buffer_mode_t mode,
                                 int32_t max_tokens_per_expert, int64_t num_rows, int32_t* row_token,
                                 ep_stream_t stream);

/* out and h as above.  h may be kept for ep_lora_backward. */
EP_API ep_status_t ep_lora(const void* x, const void* base, const ep_routing_desc_t* routing,
                           const ep_layout_t* layout, ep_buffer_mode_t mode, int32_t max_tokens_per_expert,
                           int64_t num_rows, const int32_t* row_token, const ep_lora_desc_t* lora, void* out,
                           float* h, ep_stream_t stream);

/* Gradients of ep_lora for dy bf16 (laid out as out), x and the h that the
 * forward call wrote:
 *   dh[row] = scales[e] * B[e]^T dy[row]     fp32 [num_rows, rank]
 *   dx[row] = dx_base[row] + A[e]^T dh[row]  bf16, laid out as x; dx_base may
 *             be NULL (zeros) or dx itself: the shared projection's gradient
 *   da[e]   = sum over e's rows of dh[row] x[row]^T   bf16 [E, rank, hidden_in]
 *   db[e]   = sum over e's rows of dy[row] h[row]^T   bf16 [E, hidden_out, rank]
 * (base's gradient is dy.)  dx may be NULL; da and db both or neither.  Every
 * element of da and db is written, zeros for an adapter without rows; rows of
 * no pair, and with row_token tokens without an adapter, are treated in dx as
 * in out.  dh is scratch the size of h.  x and h are read only for da and db. */
EP_API ep_status_t ep_lora_backward(const void* dy, const void* x, const float* h, const void* dx_base,
                                    const ep_routing_desc_t* routing, const ep_layout_t* layout,
                                    ep_buffer_mode_t mode, int32_t max_tokens_per_expert, int64_t num_rows,
                                    const int32_t* row_token, const ep_lora_desc_t* lora, float* dh, void* dx,
                                    void* da, void* db, ep_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* EP_B200_LORA_H_ */
