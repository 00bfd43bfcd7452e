/*
 * sbp_step.h -- operators around the streamed backward of sbp.h: scaled token embedding with its
 * gradient by sorted tokens, the per-head RMS norm of queries and keys with RoPE in the same
 * pass (alone and inside the decoder layer), and the global gradient norm with clipping.
 *
 * Conventions are those of sbp.h (caller-owned buffers, no allocation, no host synchronisation,
 * everything queued on `stream`, statuses returned before anything is queued, fp32 gradients).
 * A call reads its host arrays and structs before it returns.  A workspace belongs to one call at
 * a time: calls (or replays of captured graphs) that may run at the same time need one each.
 * Results do not depend on timing: repeated calls on the same inputs give the same bits.
 */
#ifndef SBP_STEP_H_
#define SBP_STEP_H_

#include "sbp.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------------------------
 * Scaled token embedding:  y[r] = scale * table[ids[r]]   (fp32 product, rounded once to dt)
 *   ids    device int32 [rows]; a row whose id is outside [0, vocab) (padding) becomes zero
 *   table  device [vocab, cols], dt;   y  device [rows, cols], dt
 * Here and below rows < 2^30, cols <= 2^20 and vocab <= 2^22 (else SBP_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------------------------ */
sbp_status sbp_embedding_scaled_forward(int64_t rows, int64_t cols, int64_t vocab, sbp_dtype dt,
                                        float scale, const int32_t* ids, const void* table,
                                        void* y, void* stream);

/*
 * Its gradient by sorted tokens:  d_table[v] = (accumulate ? d_table[v] : 0)
 *                                              + scale * sum over rows r with ids[r] == v of dy[r]
 * The rows are sorted by id (stable); the rows of an id are added in ascending order inside
 * fixed blocks of the sorted list, the block sums in order.  Without `accumulate` the whole
 * table is written (ids that do not occur get zeros): no clearing pass is needed.  Rows whose id
 * is outside [0, vocab) are skipped; their dy is not read.  dy fp32 [rows, cols], d_table fp32
 * [vocab, cols].
 */
size_t sbp_embedding_scaled_backward_workspace_size(int64_t rows, int64_t cols, int64_t vocab);
sbp_status sbp_embedding_scaled_backward(int64_t rows, int64_t cols, int64_t vocab, float scale,
                                         const int32_t* ids, const float* dy, float* d_table,
                                         int accumulate, void* workspace, size_t workspace_bytes,
                                         void* stream);

/* ------------------------------------------------------------------------------------------
 * Norm and rotation of queries and keys, per head x of head_dim elements at position p:
 *   n = x / sqrt(mean(x^2) + eps) * g      (g: one gain vector for the queries, one for the keys)
 *   y_j = n_j cos[p, j] - n_{j+h} sin[p, j],   y_{j+h} = n_{j+h} cos[p, j] + n_j sin[p, j]
 * with h = head_dim / 2 (the rotate-half RoPE of the decoder layer).  The position of row r is
 * positions[r] where positions is given, else r % seq_len.  A row whose position lies outside
 * [0, table_len) gets zeros (and, in the backward, zero gradients and no share in the gains').
 *
 * Rows are tokens; the heads of a row are contiguous and rows are ld elements apart, so that q
 * and k may lie inside one fused projection.  Pointers need their element's alignment only;
 * 16-byte aligned pointers, ld a multiple of 16 bytes and head_dim a multiple of 16 take the
 * vector path.  Inputs and outputs may be the same buffer (with the same ld); they must not
 * overlap in any other way.  n_kv_heads = 0 leaves the keys out (their pointers are not read).
 * rows < 2^30, heads <= 65536, rows x heads < 2^31 (else SBP_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------------------------ */
typedef struct {
  int64_t rows, n_heads, n_kv_heads, head_dim; /* head_dim even, <= 256                        */
  int64_t seq_len;   /* without positions: 1 <= seq_len <= table_len                           */
  int64_t table_len; /* rows of the cos / sin tables [table_len, head_dim / 2] (16-byte aligned) */
  float eps;
  int dtype;         /* sbp_dtype of q, k, the gains and the forward's outputs                 */
} sbp_qk_cfg;

/* cos / sin tables [positions, head_dim / 2] fp32 of the angles p * theta^(-2j / head_dim),
 * formed in 64 bits (the decoder layer's own tables). */
sbp_status sbp_rope_table(int64_t positions, int64_t head_dim, double theta, float* cos_table,
                          float* sin_table, void* stream);

sbp_status sbp_qk_norm_rope_forward(const sbp_qk_cfg* cfg, const void* q, int64_t ldq,
                                    const void* k, int64_t ldk, const void* q_g, const void* k_g,
                                    const int32_t* positions, const float* cos_table,
                                    const float* sin_table, void* q_out, int64_t ldqo,
                                    void* k_out, int64_t ldko, void* stream);

/* The forward's backward, from its inputs q, k (nothing is saved by the forward): with u the
 * inverse rotation of the upstream gradient and xhat = x / sqrt(mean(x^2) + eps),
 *   dg += sum over rows and heads of u * xhat       (accumulated)
 *   dx  = (g u - xhat * mean(xhat * g u)) / sqrt(mean(x^2) + eps)      (overwritten)
 * dq_out / dk_out (upstream), dq / dk and the gain gradients dq_g / dk_g are fp32.  dq_g and dk_g
 * may be one vector (a gain that queries and keys share), which then receives both sums; they
 * must not overlap in part. */
size_t sbp_qk_norm_rope_backward_workspace_size(const sbp_qk_cfg* cfg);
sbp_status sbp_qk_norm_rope_backward(const sbp_qk_cfg* cfg, const void* q, int64_t ldq,
                                     const void* k, int64_t ldk, const void* q_g, const void* k_g,
                                     const int32_t* positions, const float* cos_table,
                                     const float* sin_table, const float* dq_out, int64_t lddqo,
                                     const float* dk_out, int64_t lddko, float* dq, int64_t lddq,
                                     float* dk, int64_t lddk, float* dq_g, float* dk_g,
                                     void* workspace, size_t workspace_bytes, void* stream);

/*
 * The decoder layer of sbp.h with these norms between its projections and the attention (eps =
 * cfg->rms_eps; biases, where given, come before the norm):
 *   q = rope(norm(n1 W_q^T + b_q; q_g)),  k = rope(norm(n1 W_k^T + b_k; k_g))   per head
 * Arguments, layouts, accumulation and errors are those of sbp_decoder_layer_forward_stream and
 * sbp_decoder_layer_backward_stream (or, with `reverse`, its _reverse form).  The projections
 * are rounded to cfg->dtype before the norm; only one chunk of them is kept, the backward forms
 * the keys' again.  dq_g, dk_g: device fp32 [head_dim], accumulated.  For a chunk's rows (batch x
 * the longest chunk) and heads the limits of sbp_qk_norm_rope_forward hold.
 */
typedef struct { /* device [head_dim], cfg.dtype, 16-byte aligned */
  const void *q_g, *k_g;
} sbp_qk_gains;

size_t sbp_decoder_layer_qk_norm_workspace_size(const sbp_layer_cfg* cfg);
sbp_status sbp_decoder_layer_qk_norm_forward_stream(const sbp_layer_cfg* cfg,
                                                    const sbp_layer_weights* w,
                                                    const sbp_qk_gains* gains, const void* x,
                                                    void* y, void* workspace,
                                                    size_t workspace_bytes, void* stream);
sbp_status sbp_decoder_layer_qk_norm_backward_stream(const sbp_layer_cfg* cfg,
                                                     const sbp_layer_weights* w,
                                                     const sbp_qk_gains* gains, const void* x,
                                                     const float* dy, float* dx,
                                                     const sbp_layer_grads* grads, float* dq_g,
                                                     float* dk_g, int reverse, void* workspace,
                                                     size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------------
 * Global gradient norm over many tensors, and clipping:
 *   norm = sqrt(sum over all tensors and elements of g^2)          (products and sums in 64 bits)
 *   coef = min(1, max_norm / (norm + 1e-6)),   out = g * coef
 * grads / outs are HOST arrays of n_tensors device pointers (fp32, 16-byte aligned), numel a
 * HOST array of their element counts (0 allowed; such a tensor's pointer is not read).  outs
 * may be NULL (in place), or name other buffers; an out may equal its grad and must not overlap
 * any other tensor.  In place and with coef = 1 nothing is written.  Where the norm is not
 * finite there is no right coefficient: out = g, unscaled, and norm_out tells the caller.
 *
 * sbp_grad_sqsum gives sum g^2 of one rank's tensors as a device double, so that the ranks of a
 * partitioned gradient add theirs before sbp_grad_clip; sbp_grad_clip_norm is both in one call.
 *   sqsum device double [1];   norm_out device fp32 [1], may be NULL in sbp_grad_clip
 * ------------------------------------------------------------------------------------------ */
size_t sbp_grad_norm_workspace_size(int64_t n_tensors);
sbp_status sbp_grad_sqsum(int64_t n_tensors, const float* const* grads, const int64_t* numel,
                          double* sqsum, void* workspace, size_t workspace_bytes, void* stream);
sbp_status sbp_grad_clip(int64_t n_tensors, const float* const* grads, float* const* outs,
                         const int64_t* numel, const double* sqsum, float max_norm,
                         float* norm_out, void* stream);
sbp_status sbp_grad_clip_norm(int64_t n_tensors, const float* const* grads, float* const* outs,
                              const int64_t* numel, float max_norm, float* norm_out,
                              void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* SBP_STEP_H_ */
