// C ABI of the operators around the streamed step (include/sbp_step.h): argument checks and
// workspace layout; the kernels are in embedding.cu, qk_norm.cu and grad_norm.cu.
#include "api_checks.cuh"
#include "sbp_step.h"

using namespace sbp;

namespace {

// whether two ranges of n bytes have bytes in common
inline bool overlap(const void* p, const void* q, size_t n) {
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + n && b < a + n;
}

// ------------------------------------------------------------------------ embedding
constexpr int64_t kMaxRows = (int64_t)1 << 30, kMaxCols = (int64_t)1 << 20;

sbp_status check_embed(int64_t rows, int64_t cols, int64_t vocab, int dt, const void* ids,
                       const void* a, const void* b) {
  if (rows <= 0 || cols <= 0 || vocab <= 0)
    return fail(SBP_ERR_INVALID_ARG, "rows, cols and vocab must be positive");
  if (dt != SBP_F32 && dt != SBP_BF16) return fail(SBP_ERR_INVALID_ARG, "unknown dtype %d", dt);
  if (rows >= kMaxRows || cols > kMaxCols)
    return fail(SBP_ERR_UNSUPPORTED, "rows must be below 2^30 and cols at most 2^20");
  if (vocab > kEmbedMaxVocab) return fail(SBP_ERR_UNSUPPORTED, "vocab must be at most 2^22");
  const void* ptrs[] = {ids, a, b};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 16))
      return fail(SBP_ERR_INVALID_ARG, "a pointer is NULL or not 16-byte aligned");
  return SBP_OK;
}

// ------------------------------------------------------------------------ queries and keys
sbp_status check_qk(const sbp_qk_cfg* c) {
  if (!c) return fail(SBP_ERR_INVALID_ARG, "cfg is NULL");
  if (c->rows <= 0 || c->n_heads <= 0 || c->n_kv_heads < 0 || c->head_dim <= 0 ||
      c->table_len <= 0)
    return fail(SBP_ERR_INVALID_ARG, "rows, n_heads, head_dim and table_len must be positive");
  if (c->head_dim % 2 != 0 || c->head_dim > 256)
    return fail(SBP_ERR_UNSUPPORTED, "head_dim must be even and <= 256");
  const int64_t heads = imax(c->n_heads, c->n_kv_heads);
  if (c->rows >= kQkMaxRows || heads > kQkMaxHeads || c->rows * heads >= 2 * kQkMaxRows)
    return fail(SBP_ERR_UNSUPPORTED,
                "rows must be below 2^30, heads at most 65536 and rows x heads below 2^31");
  if (c->dtype != SBP_F32 && c->dtype != SBP_BF16)
    return fail(SBP_ERR_INVALID_ARG, "unknown dtype %d", c->dtype);
  if (!(c->eps >= 0.f)) return fail(SBP_ERR_INVALID_ARG, "eps must be >= 0");
  return SBP_OK;
}

// the arguments that both directions share, into a
sbp_status set_qk(const sbp_qk_cfg* c, const void* q, int64_t ldq, const void* k, int64_t ldk,
                  const void* q_g, const void* k_g, const int32_t* positions, const float* cosb,
                  const float* sinb, QkNorm& a) {
  if (sbp_status s = check_qk(c)) return s;
  const size_t es = dt_size(c->dtype);
  const bool has_k = c->n_kv_heads > 0;
  if (!q || !q_g || !cosb || !sinb || (has_k && (!k || !k_g)))
    return fail(SBP_ERR_INVALID_ARG, "a required pointer is NULL");
  if (!aligned(cosb, 16) || !aligned(sinb, 16))
    return fail(SBP_ERR_INVALID_ARG, "cos / sin table not 16-byte aligned");
  if (!aligned(q, es) || !aligned(q_g, es) ||
      (has_k && (!aligned(k, es) || !aligned(k_g, es))) || (positions && !aligned(positions, 4)))
    return fail(SBP_ERR_INVALID_ARG, "a pointer is not aligned to its elements");
  if (!positions && (c->seq_len < 1 || c->seq_len > c->table_len))
    return fail(SBP_ERR_INVALID_ARG, "need 1 <= seq_len <= table_len (got %lld, %lld)",
                (long long)c->seq_len, (long long)c->table_len);
  if (ldq < c->n_heads * c->head_dim || (has_k && ldk < c->n_kv_heads * c->head_dim))
    return fail(SBP_ERR_INVALID_ARG, "a row stride is smaller than the row's heads");
  a.rows = c->rows;
  a.hd = c->head_dim;
  a.dt = c->dtype;
  a.eps = c->eps;
  a.q.n = c->n_heads;
  a.q.x = q;
  a.q.ldx = ldq;
  a.q.g = q_g;
  a.k.n = c->n_kv_heads;
  a.k.x = k;
  a.k.ldx = ldk;
  a.k.g = k_g;
  a.positions = positions;
  a.seq_len = positions ? 1 : c->seq_len;
  a.table_len = c->table_len;
  a.cosb = cosb;
  a.sinb = sinb;
  return SBP_OK;
}

sbp_status check_out(const QkNormHeads& h, int64_t hd, const void* p, int64_t ld, size_t es) {
  if (h.n == 0) return SBP_OK;
  if (!p || !aligned(p, es))
    return fail(SBP_ERR_INVALID_ARG, "an output or gradient pointer is NULL or misaligned");
  if (ld < h.n * hd)
    return fail(SBP_ERR_INVALID_ARG, "a row stride is smaller than the row's heads");
  return SBP_OK;
}

// ------------------------------------------------------------------------ gradients
sbp_status check_grads(int64_t n, const float* const* grads, float* const* outs,
                       const int64_t* numel) {
  if (n < 0) return fail(SBP_ERR_INVALID_ARG, "n_tensors is negative");
  if (n > 0 && (!grads || !numel)) return fail(SBP_ERR_INVALID_ARG, "grads or numel is NULL");
  for (int64_t i = 0; i < n; ++i) {
    if (numel[i] < 0 || numel[i] > ((int64_t)1 << 40))
      return fail(SBP_ERR_INVALID_ARG, "tensor %lld: bad element count", (long long)i);
    if (numel[i] == 0) continue;
    if (!grads[i] || !aligned(grads[i], 16) || (outs && (!outs[i] || !aligned(outs[i], 16))))
      return fail(SBP_ERR_INVALID_ARG, "tensor %lld: pointer NULL or not 16-byte aligned",
                  (long long)i);
  }
  return SBP_OK;
}

GradTensors tensors_of(int64_t n, const float* const* grads, float* const* outs,
                       const int64_t* numel) {
  GradTensors g;
  g.n = n;
  g.src = grads;
  g.dst = outs;
  g.numel = numel;
  return g;
}

sbp_status check_max_norm(float max_norm) {
  if (!(max_norm >= 0.f)) return fail(SBP_ERR_INVALID_ARG, "max_norm must be >= 0");
  return SBP_OK;
}

}  // namespace

extern "C" {

sbp_status sbp_embedding_scaled_forward(int64_t rows, int64_t cols, int64_t vocab, sbp_dtype dt,
                                        float scale, const int32_t* ids, const void* table,
                                        void* y, void* stream) {
  if (sbp_status s = check_embed(rows, cols, vocab, dt, ids, table, y)) return s;
  SBP_CK(embed_scaled_fwd(rows, cols, vocab, dt, scale, ids, table, y,
                           static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

size_t sbp_embedding_scaled_backward_workspace_size(int64_t rows, int64_t cols, int64_t vocab) {
  if (rows <= 0 || cols <= 0 || vocab <= 0 || rows >= kMaxRows || cols > kMaxCols ||
      vocab > kEmbedMaxVocab)
    return 0;
  return embed_scaled_bwd_ws_bytes(rows, cols, vocab);
}

sbp_status sbp_embedding_scaled_backward(int64_t rows, int64_t cols, int64_t vocab, float scale,
                                         const int32_t* ids, const float* dy, float* d_table,
                                         int accumulate, void* workspace, size_t workspace_bytes,
                                         void* stream) {
  if (sbp_status s = check_embed(rows, cols, vocab, SBP_F32, ids, dy, d_table)) return s;
  if (sbp_status s = check_ws(workspace, workspace_bytes,
                              embed_scaled_bwd_ws_bytes(rows, cols, vocab)))
    return s;
  SBP_CK(embed_scaled_bwd(rows, cols, vocab, scale, ids, dy, d_table, accumulate, workspace,
                           static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

sbp_status sbp_rope_table(int64_t positions, int64_t head_dim, double theta, float* cos_table,
                          float* sin_table, void* stream) {
  if (positions <= 0 || head_dim <= 0)
    return fail(SBP_ERR_INVALID_ARG, "positions and head_dim must be positive");
  if (head_dim % 2 != 0 || head_dim > 256 || positions >= kMaxRows)
    return fail(SBP_ERR_UNSUPPORTED, "head_dim must be even and <= 256, positions below 2^30");
  if (!(theta > 0.0)) return fail(SBP_ERR_INVALID_ARG, "theta must be > 0");
  if (!cos_table || !sin_table || !aligned(cos_table, 16) || !aligned(sin_table, 16))
    return fail(SBP_ERR_INVALID_ARG, "a table pointer is NULL or not 16-byte aligned");
  SBP_CK(rope_table(positions, head_dim, theta, cos_table, sin_table,
                     static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

sbp_status sbp_qk_norm_rope_forward(const sbp_qk_cfg* cfg, const void* q, int64_t ldq,
                                    const void* k, int64_t ldk, const void* q_g, const void* k_g,
                                    const int32_t* positions, const float* cos_table,
                                    const float* sin_table, void* q_out, int64_t ldqo,
                                    void* k_out, int64_t ldko, void* stream) {
  QkNorm a;
  if (sbp_status s = set_qk(cfg, q, ldq, k, ldk, q_g, k_g, positions, cos_table, sin_table, a))
    return s;
  const size_t es = dt_size(a.dt);
  if (sbp_status s = check_out(a.q, a.hd, q_out, ldqo, es)) return s;
  if (sbp_status s = check_out(a.k, a.hd, k_out, ldko, es)) return s;
  a.q.y = q_out;
  a.q.ldy = ldqo;
  a.k.y = k_out;
  a.k.ldy = ldko;
  SBP_CK(qk_norm_rope_fwd(a, static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

size_t sbp_qk_norm_rope_backward_workspace_size(const sbp_qk_cfg* cfg) {
  if (check_qk(cfg) != SBP_OK) return 0;
  return sizeof(float) * qk_norm_bwd_partial_floats(cfg->head_dim);
}

sbp_status sbp_qk_norm_rope_backward(const sbp_qk_cfg* cfg, const void* q, int64_t ldq,
                                     const void* k, int64_t ldk, const void* q_g, const void* k_g,
                                     const int32_t* positions, const float* cos_table,
                                     const float* sin_table, const float* dq_out, int64_t lddqo,
                                     const float* dk_out, int64_t lddko, float* dq, int64_t lddq,
                                     float* dk, int64_t lddk, float* dq_g, float* dk_g,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  QkNorm a;
  if (sbp_status s = set_qk(cfg, q, ldq, k, ldk, q_g, k_g, positions, cos_table, sin_table, a))
    return s;
  if (sbp_status s = check_out(a.q, a.hd, dq_out, lddqo, 4)) return s;
  if (sbp_status s = check_out(a.q, a.hd, dq, lddq, 4)) return s;
  if (sbp_status s = check_out(a.k, a.hd, dk_out, lddko, 4)) return s;
  if (sbp_status s = check_out(a.k, a.hd, dk, lddk, 4)) return s;
  if (!dq_g || !aligned(dq_g, 4) || (a.k.n && (!dk_g || !aligned(dk_g, 4))))
    return fail(SBP_ERR_INVALID_ARG, "a gain gradient is NULL or misaligned");
  if (a.k.n && dq_g != dk_g && overlap(dq_g, dk_g, sizeof(float) * a.hd))
    return fail(SBP_ERR_INVALID_ARG, "dq_g and dk_g overlap in part");
  if (sbp_status s = check_ws(workspace, workspace_bytes,
                              sbp_qk_norm_rope_backward_workspace_size(cfg)))
    return s;
  a.q.dy = dq_out;
  a.q.lddy = lddqo;
  a.q.dx = dq;
  a.q.lddx = lddq;
  a.k.dy = dk_out;
  a.k.lddy = lddko;
  a.k.dx = dk;
  a.k.lddx = lddk;
  SBP_CK(qk_norm_rope_bwd(a, dq_g, dk_g, static_cast<float*>(workspace),
                           static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

size_t sbp_grad_norm_workspace_size(int64_t n_tensors) {
  return n_tensors < 0 ? 0 : grad_norm_ws_bytes(n_tensors);
}

sbp_status sbp_grad_sqsum(int64_t n, const float* const* grads, const int64_t* numel,
                          double* sqsum, void* workspace, size_t workspace_bytes, void* stream) {
  if (sbp_status s = check_grads(n, grads, nullptr, numel)) return s;
  if (!sqsum || !aligned(sqsum, 8)) return fail(SBP_ERR_INVALID_ARG, "sqsum NULL or misaligned");
  if (sbp_status s = check_ws(workspace, workspace_bytes, grad_norm_ws_bytes(n))) return s;
  SBP_CK(grad_sqsum(tensors_of(n, grads, nullptr, numel), sqsum, workspace,
                     static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

sbp_status sbp_grad_clip(int64_t n, const float* const* grads, float* const* outs,
                         const int64_t* numel, const double* sqsum, float max_norm,
                         float* norm_out, void* stream) {
  if (sbp_status s = check_grads(n, grads, outs, numel)) return s;
  if (!sqsum || !aligned(sqsum, 8)) return fail(SBP_ERR_INVALID_ARG, "sqsum NULL or misaligned");
  if (sbp_status s = check_max_norm(max_norm)) return s;
  if (!aligned(norm_out, 4)) return fail(SBP_ERR_INVALID_ARG, "norm_out is misaligned");
  SBP_CK(grad_clip(tensors_of(n, grads, outs, numel), sqsum, max_norm, norm_out,
                    static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

sbp_status sbp_grad_clip_norm(int64_t n, const float* const* grads, float* const* outs,
                              const int64_t* numel, float max_norm, float* norm_out,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (sbp_status s = check_grads(n, grads, outs, numel)) return s;
  if (sbp_status s = check_max_norm(max_norm)) return s;
  if (!norm_out || !aligned(norm_out, 4))
    return fail(SBP_ERR_INVALID_ARG, "norm_out is NULL or misaligned");
  if (sbp_status s = check_ws(workspace, workspace_bytes, grad_norm_ws_bytes(n))) return s;
  SBP_CK(grad_clip_norm(tensors_of(n, grads, outs, numel), max_norm, norm_out, workspace,
                         static_cast<cudaStream_t>(stream)));
  return SBP_OK;
}

}  // extern "C"
