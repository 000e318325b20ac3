// C ABI of the operators around the projections (declared in
// include/poetx.h): argument checks and workspace sizes.
#include <cmath>

#include "internal.h"
#include "poetx.h"

using namespace poetx;

namespace {

constexpr int64_t kMaxTokens = 1ll << 22;
constexpr int kMaxFeatures = 1 << 20;
constexpr int64_t kMaxElements = 1ll << 42;  // of one tensor list

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

poetx_status to_status(cudaError_t e) { return e == cudaSuccess ? POETX_OK : POETX_ERR_CUDA; }

bool dtype_ok(poetx_dtype t) { return t == POETX_F32 || t == POETX_BF16; }

bool linear_dims_ok(int d_in, int d_out, int64_t tokens, poetx_dtype dtype) {
  return dtype_ok(dtype) && d_in > 0 && d_out > 0 && d_in <= kMaxFeatures &&
         d_out <= kMaxFeatures && tokens >= 0 && tokens <= kMaxTokens;
}

bool act_ok(poetx_activation a) { return a >= POETX_ACT_NONE && a <= POETX_ACT_GELU_TANH; }

poetx_status check_workspace(size_t need, const void* workspace, size_t bytes) {
  if (need == 0) return POETX_OK;
  return workspace == nullptr || bytes < need || !aligned(workspace, 16) ? POETX_ERR_WORKSPACE
                                                                         : POETX_OK;
}

// One tensor of q / k: rows of heads * head_dim elements, ld apart.
bool rows_ok(const void* p, int64_t ld, int heads, int head_dim, int64_t tokens, size_t es) {
  if (heads == 0) return true;
  return p != nullptr && aligned(p, es) &&
         (tokens <= 1 || ld >= static_cast<int64_t>(heads) * head_dim) && ld >= 0 &&
         ld <= (1ll << 32);
}

poetx_status check_qk(int hq, int hk, int D, int rot, int64_t table_rows, float eps,
                      int64_t tokens, poetx_dtype dtype) {
  if (!dtype_ok(dtype) || tokens < 0 || tokens > kMaxTokens || hq <= 0 || hk < 0 || hq > 65536 ||
      hk > 65536 || D <= 0 || rot < 0 || rot > D || rot % 2 != 0 || table_rows < 0 ||
      !(eps > 0.f) || std::isinf(eps))
    return POETX_ERR_INVALID_ARG;
  return D > 512 ? POETX_ERR_UNSUPPORTED : POETX_OK;
}

// An output may be an input of its own side with the same rows, never the other
// side's: warps read and write the heads of both at their own pace.
bool in_place_ok(const void* in, int64_t ld_in, const void* other_in, const void* out,
                 int64_t ld_out, int64_t tokens) {
  return out != other_in && (out != in || ld_in == ld_out || tokens <= 1);
}

// Counts, pointers and types of a tensor list.
poetx_status check_list(int n, const int64_t* counts, const int32_t* dtypes) {
  if (n < 0 || (n > 0 && counts == nullptr)) return POETX_ERR_INVALID_ARG;
  int64_t total = 0;
  for (int i = 0; i < n; ++i) {
    if (counts[i] < 0 || counts[i] > kMaxElements) return POETX_ERR_INVALID_ARG;
    total += counts[i];
    if (total > kMaxElements) return POETX_ERR_INVALID_ARG;
    if (dtypes != nullptr && dtypes[i] != POETX_F32 && dtypes[i] != POETX_BF16)
      return POETX_ERR_INVALID_ARG;
  }
  return POETX_OK;
}

bool pointers_ok(int n, const void* const* p, const int64_t* counts, const int32_t* dtypes) {
  if (n > 0 && p == nullptr) return false;
  for (int i = 0; i < n; ++i) {
    const uintptr_t es = dtypes != nullptr && dtypes[i] == POETX_BF16 ? 2 : 4;
    if (counts[i] > 0 && (p[i] == nullptr || !aligned(p[i], es))) return false;
  }
  return true;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ linear

size_t poetx_linear_forward_workspace_size(int d_in, int d_out, int64_t tokens,
                                           poetx_dtype dtype) {
  if (!linear_dims_ok(d_in, d_out, tokens, dtype) || tokens == 0) return 0;
  return linear_forward_scratch(d_in, d_out, tokens, dtype == POETX_BF16, true);
}

poetx_status poetx_linear_forward(const void* x, const void* W, const float* bias,
                                  const void* residual, void* y, void* z_saved, int d_in,
                                  int d_out, int64_t tokens, poetx_activation act,
                                  poetx_dtype dtype, void* workspace, size_t workspace_bytes,
                                  poetx_stream stream) {
  if (!linear_dims_ok(d_in, d_out, tokens, dtype) || !act_ok(act)) return POETX_ERR_INVALID_ARG;
  if (tokens == 0) return POETX_OK;
  if (x == nullptr || W == nullptr || y == nullptr || y == x || z_saved == x || z_saved == y ||
      (z_saved != nullptr && z_saved == residual))
    return POETX_ERR_INVALID_ARG;
  for (const void* p : {x, W, static_cast<const void*>(bias), residual,
                        static_cast<const void*>(y), static_cast<const void*>(z_saved)})
    if (!aligned(p, 16)) return POETX_ERR_INVALID_ARG;
  const bool is_bf16 = dtype == POETX_BF16;
  const poetx_status st =
      check_workspace(linear_forward_scratch(d_in, d_out, tokens, is_bf16, false), workspace,
                      workspace_bytes);
  if (st != POETX_OK) return st;
  return to_status(linear_forward(x, W, bias, residual, y, z_saved, d_in, d_out, tokens, act,
                                  is_bf16, workspace, static_cast<cudaStream_t>(stream)));
}

size_t poetx_linear_backward_workspace_size(int d_in, int d_out, int64_t tokens,
                                            poetx_activation act, poetx_dtype dtype,
                                            int with_dbias) {
  if (!linear_dims_ok(d_in, d_out, tokens, dtype) || !act_ok(act) || tokens == 0) return 0;
  return linear_backward_scratch(d_in, d_out, tokens, act, dtype == POETX_BF16, with_dbias != 0,
                                 true);
}

poetx_status poetx_linear_backward(const void* dy, const void* z_saved, const void* W, void* dx,
                                   float* dbias, int d_in, int d_out, int64_t tokens,
                                   poetx_activation act, poetx_dtype dtype, void* workspace,
                                   size_t workspace_bytes, poetx_stream stream) {
  if (!linear_dims_ok(d_in, d_out, tokens, dtype) || !act_ok(act)) return POETX_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!aligned(dbias, 16)) return POETX_ERR_INVALID_ARG;
  if (tokens == 0)
    return dbias == nullptr ? POETX_OK
                            : to_status(cudaMemsetAsync(dbias, 0, sizeof(float) * d_out, s));
  if (dx == nullptr && dbias == nullptr) return POETX_OK;
  if (dy == nullptr || (dx != nullptr && W == nullptr) || dx == dy ||
      (act != POETX_ACT_NONE && (z_saved == nullptr || dx == z_saved)))
    return POETX_ERR_INVALID_ARG;
  for (const void* p : {dy, z_saved, W, static_cast<const void*>(dx)})
    if (!aligned(p, 16)) return POETX_ERR_INVALID_ARG;
  const bool is_bf16 = dtype == POETX_BF16;
  const poetx_status st = check_workspace(
      linear_backward_scratch(d_in, d_out, tokens, act, is_bf16, dbias != nullptr, false),
      workspace, workspace_bytes);
  if (st != POETX_OK) return st;
  return to_status(linear_backward(dy, z_saved, W, dx, dbias, d_in, d_out, tokens, act, is_bf16,
                                   workspace, s));
}

// ------------------------------------------------- query / key norm + rotary

poetx_status poetx_qk_norm_rope_forward(const void* q, const void* k, const float* gamma_q,
                                        const float* gamma_k, const float* cos_table,
                                        const float* sin_table, const int32_t* positions,
                                        void* q_out, void* k_out, int64_t ld_q, int64_t ld_k,
                                        int64_t ld_q_out, int64_t ld_k_out, int n_q_heads,
                                        int n_k_heads, int head_dim, int rot_dim,
                                        int64_t table_rows, int interleaved, float eps,
                                        int64_t tokens, poetx_dtype dtype, poetx_stream stream) {
  poetx_status st =
      check_qk(n_q_heads, n_k_heads, head_dim, rot_dim, table_rows, eps, tokens, dtype);
  if (st != POETX_OK) return st;
  if (tokens == 0) return POETX_OK;
  const size_t es = dtype == POETX_BF16 ? 2 : 4;
  if (!rows_ok(q, ld_q, n_q_heads, head_dim, tokens, es) ||
      !rows_ok(k, ld_k, n_k_heads, head_dim, tokens, es) ||
      !rows_ok(q_out, ld_q_out, n_q_heads, head_dim, tokens, es) ||
      !rows_ok(k_out, ld_k_out, n_k_heads, head_dim, tokens, es))
    return POETX_ERR_INVALID_ARG;
  if (!aligned(gamma_q, 4) || !aligned(gamma_k, 4) || !aligned(positions, 4) ||
      (rot_dim > 0 && (cos_table == nullptr || sin_table == nullptr || !aligned(cos_table, 4) ||
                       !aligned(sin_table, 4))))
    return POETX_ERR_INVALID_ARG;
  if (!in_place_ok(q, ld_q, n_k_heads > 0 ? k : nullptr, q_out, ld_q_out, tokens) ||
      (n_k_heads > 0 && !in_place_ok(k, ld_k, q, k_out, ld_k_out, tokens)))
    return POETX_ERR_INVALID_ARG;
  QkNormRopeArgs a;
  a.q = q, a.k = k, a.ld_q = ld_q, a.ld_k = ld_k;
  a.gamma_q = gamma_q, a.gamma_k = gamma_k;
  a.cos_table = cos_table, a.sin_table = sin_table, a.positions = positions;
  a.table_rows = table_rows, a.T = tokens;
  a.hq = n_q_heads, a.hk = n_k_heads, a.D = head_dim, a.rot = rot_dim;
  a.interleaved = interleaved != 0, a.eps = eps;
  a.out_q = q_out, a.out_k = k_out, a.ld_out_q = ld_q_out, a.ld_out_k = ld_k_out;
  a.status = device_status_ptr();
  if (a.status == nullptr) return POETX_ERR_CUDA;
  return to_status(
      qk_norm_rope_forward(a, dtype == POETX_BF16, static_cast<cudaStream_t>(stream)));
}

size_t poetx_qk_norm_rope_backward_workspace_size(int n_q_heads, int n_k_heads, int head_dim,
                                                  int64_t tokens, poetx_dtype dtype) {
  if (check_qk(n_q_heads, n_k_heads, head_dim, 0, 0, 1.f, tokens, dtype) != POETX_OK) return 0;
  return qk_norm_rope_scratch(n_q_heads, n_k_heads, head_dim, tokens);
}

poetx_status poetx_qk_norm_rope_backward(
    const void* dq_out, const void* dk_out, const void* q, const void* k, const float* gamma_q,
    const float* gamma_k, const float* cos_table, const float* sin_table, const int32_t* positions,
    void* dq, void* dk, float* dgamma_q, float* dgamma_k, int64_t ld_dq_out, int64_t ld_dk_out,
    int64_t ld_q, int64_t ld_k, int64_t ld_dq, int64_t ld_dk, int n_q_heads, int n_k_heads,
    int head_dim, int rot_dim, int64_t table_rows, int interleaved, float eps, int64_t tokens,
    poetx_dtype dtype, void* workspace, size_t workspace_bytes, poetx_stream stream) {
  poetx_status st =
      check_qk(n_q_heads, n_k_heads, head_dim, rot_dim, table_rows, eps, tokens, dtype);
  if (st != POETX_OK) return st;
  const size_t es = dtype == POETX_BF16 ? 2 : 4;
  if (tokens > 0 && (!rows_ok(q, ld_q, n_q_heads, head_dim, tokens, es) ||
                     !rows_ok(k, ld_k, n_k_heads, head_dim, tokens, es) ||
                     !rows_ok(dq_out, ld_dq_out, n_q_heads, head_dim, tokens, es) ||
                     !rows_ok(dk_out, ld_dk_out, n_k_heads, head_dim, tokens, es) ||
                     !rows_ok(dq, ld_dq, n_q_heads, head_dim, tokens, es) ||
                     !rows_ok(dk, ld_dk, n_k_heads, head_dim, tokens, es)))
    return POETX_ERR_INVALID_ARG;
  if (!aligned(gamma_q, 4) || !aligned(gamma_k, 4) || !aligned(positions, 4) ||
      !aligned(dgamma_q, 4) || !aligned(dgamma_k, 4) ||
      (rot_dim > 0 && tokens > 0 &&
       (cos_table == nullptr || sin_table == nullptr || !aligned(cos_table, 4) ||
        !aligned(sin_table, 4))))
    return POETX_ERR_INVALID_ARG;
  st = check_workspace(qk_norm_rope_scratch(n_q_heads, n_k_heads, head_dim, tokens), workspace,
                       workspace_bytes);
  if (st != POETX_OK) return st;
  if (tokens > 0) {
    const bool has_k = n_k_heads > 0;
    if (!in_place_ok(q, ld_q, has_k ? k : nullptr, dq, ld_dq, tokens) ||
        !in_place_ok(dq_out, ld_dq_out, has_k ? dk_out : nullptr, dq, ld_dq, tokens) ||
        (has_k && (!in_place_ok(k, ld_k, q, dk, ld_dk, tokens) ||
                   !in_place_ok(dk_out, ld_dk_out, dq_out, dk, ld_dk, tokens))))
      return POETX_ERR_INVALID_ARG;
  }
  QkNormRopeArgs a;
  a.q = q, a.k = k, a.ld_q = ld_q, a.ld_k = ld_k;
  a.gamma_q = gamma_q, a.gamma_k = gamma_k;
  a.cos_table = cos_table, a.sin_table = sin_table, a.positions = positions;
  a.table_rows = table_rows, a.T = tokens;
  a.hq = n_q_heads, a.hk = n_k_heads, a.D = head_dim, a.rot = rot_dim;
  a.interleaved = interleaved != 0, a.eps = eps;
  a.gq = dq_out, a.gk = dk_out, a.ld_gq = ld_dq_out, a.ld_gk = ld_dk_out;
  a.out_q = dq, a.out_k = dk, a.ld_out_q = ld_dq, a.ld_out_k = ld_dk;
  a.dgamma_q = dgamma_q, a.dgamma_k = dgamma_k;
  a.part = static_cast<float*>(workspace);
  a.status = device_status_ptr();
  if (a.status == nullptr) return POETX_ERR_CUDA;
  return to_status(
      qk_norm_rope_backward(a, dtype == POETX_BF16, static_cast<cudaStream_t>(stream)));
}

// --------------------------------------------- gradient norm, clip and Adam

size_t poetx_grad_norm_workspace_size(int n_tensors) {
  return n_tensors < 0 ? 0 : grad_norm_scratch(n_tensors);
}

poetx_status poetx_grad_norm(int n_tensors, const void* const* grads, const int64_t* counts,
                             const int32_t* dtypes, float* norm, void* workspace,
                             size_t workspace_bytes, poetx_stream stream) {
  poetx_status st = check_list(n_tensors, counts, dtypes);
  if (st != POETX_OK) return st;
  if (!pointers_ok(n_tensors, grads, counts, dtypes) || norm == nullptr || !aligned(norm, 4))
    return POETX_ERR_INVALID_ARG;
  st = check_workspace(grad_norm_scratch(n_tensors), workspace, workspace_bytes);
  if (st != POETX_OK) return st;
  return to_status(grad_norm(n_tensors, grads, counts, dtypes, norm, workspace,
                             static_cast<cudaStream_t>(stream)));
}

poetx_status poetx_clip_grads(int n_tensors, const void* const* grads, void* const* outs,
                              const int64_t* counts, const int32_t* dtypes, float max_norm,
                              float* norm, void* workspace, size_t workspace_bytes,
                              poetx_stream stream) {
  poetx_status st = check_list(n_tensors, counts, dtypes);
  if (st != POETX_OK) return st;
  if (!(max_norm >= 0.f) || !pointers_ok(n_tensors, grads, counts, dtypes) ||
      !pointers_ok(n_tensors, outs, counts, dtypes) || norm == nullptr || !aligned(norm, 4))
    return POETX_ERR_INVALID_ARG;
  st = check_workspace(grad_norm_scratch(n_tensors), workspace, workspace_bytes);
  if (st != POETX_OK) return st;
  return to_status(clip_grads(n_tensors, grads, outs, counts, dtypes, max_norm, norm, workspace,
                              static_cast<cudaStream_t>(stream)));
}

poetx_status poetx_adam_update_many(int n_tensors, float* const* theta, const float* const* grads,
                                    float* const* m, float* const* v, const int64_t* counts,
                                    int step, float lr, float beta1, float beta2, float eps,
                                    float weight_decay, float max_norm, float* norm,
                                    void* workspace, size_t workspace_bytes,
                                    poetx_stream stream) {
  if (step < 1 || !(beta1 >= 0.f && beta1 < 1.f) || !(beta2 >= 0.f && beta2 < 1.f) ||
      !(eps > 0.f) || std::isnan(max_norm))
    return POETX_ERR_INVALID_ARG;
  poetx_status st = check_list(n_tensors, counts, nullptr);
  if (st != POETX_OK) return st;
  for (const void* const* p :
       {reinterpret_cast<const void* const*>(theta), reinterpret_cast<const void* const*>(grads),
        reinterpret_cast<const void* const*>(m), reinterpret_cast<const void* const*>(v)})
    if (!pointers_ok(n_tensors, p, counts, nullptr)) return POETX_ERR_INVALID_ARG;
  const bool clips = max_norm >= 0.f;
  if (clips) {
    if (norm == nullptr || !aligned(norm, 4)) return POETX_ERR_INVALID_ARG;
    st = check_workspace(grad_norm_scratch(n_tensors), workspace, workspace_bytes);
    if (st != POETX_OK) return st;
  }
  AdamHyper h;
  h.lr = lr, h.beta1 = beta1, h.beta2 = beta2, h.eps = eps, h.wd = weight_decay;
  h.bc1 = static_cast<float>(1.0 - std::pow(static_cast<double>(beta1), step));
  h.bc2 = static_cast<float>(1.0 - std::pow(static_cast<double>(beta2), step));
  return to_status(adam_update_many(n_tensors, theta, grads, m, v, counts, h,
                                    clips ? max_norm : -1.f, norm, workspace,
                                    static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
