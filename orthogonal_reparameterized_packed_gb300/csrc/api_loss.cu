// C ABI of the losses at the output head (declared in include/poetx.h):
// argument checks and workspace sizes.
#include <cmath>

#include "internal.h"
#include "loss.h"
#include "poetx.h"

using namespace poetx;

namespace {

constexpr int64_t kMaxTokens = 1ll << 22;
constexpr int kMaxFeatures = 1 << 20;
constexpr int kMaxTop = 1024;

bool aligned(const void* p, uintptr_t to) {
  return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0;
}

poetx_status to_status(cudaError_t e) { return e == cudaSuccess ? POETX_OK : POETX_ERR_CUDA; }

bool dtype_ok(poetx_dtype t) { return t == POETX_F32 || t == POETX_BF16; }

// A tensor's bytes, none where it is null.
struct Span {
  uintptr_t from, to;
  Span(const void* p, size_t bytes)
      : from(reinterpret_cast<uintptr_t>(p)), to(p != nullptr ? from + bytes : from) {}
  bool meets(const Span& o) const { return from < o.to && o.from < to; }
};

// Whether an output or the workspace lies over another of them or over an input.
bool overlaps(const LossArgs& a, const void* workspace, size_t workspace_bytes) {
  const size_t T = static_cast<size_t>(a.T), d = static_cast<size_t>(a.d), es = a.is_bf16 ? 2 : 4;
  const size_t head = static_cast<size_t>(a.V) * d * es, entries = T * a.top;
  const Span written[] = {{a.loss, 4 * T}, {a.total, 4}, {a.dx, T * d * es}, {a.dW, head},
                          {workspace, workspace_bytes}};
  const Span read[] = {{a.x, T * d * es}, {a.W, head}, {a.weights, 4 * T},
                       {a.indices, entries * a.index_bytes},
                       {a.top_logits, entries * (a.top_bf16 ? 2 : 4)}};
  for (const Span& w : written) {
    for (const Span& r : read)
      if (w.meets(r)) return true;
    for (const Span& o : written)
      if (&o != &w && w.meets(o)) return true;
  }
  return false;
}

bool sizes_ok(int d, int vocab, int64_t tokens, int top, poetx_dtype dtype, int64_t block) {
  return dtype_ok(dtype) && d > 0 && vocab > 0 && d <= kMaxFeatures && vocab <= kMaxFeatures &&
         tokens >= 0 && tokens <= kMaxTokens && top > 0 && top <= kMaxTop && block >= 0 &&
         block <= kMaxTokens;
}

size_t workspace_size(int d, int vocab, int64_t tokens, int top, poetx_dtype dtype, int gradients,
                      int64_t block) {
  if (!sizes_ok(d, vocab, tokens, top, dtype, block) || gradients < 0 || gradients > 3 ||
      tokens == 0)
    return 0;
  LossArgs a;
  a.d = d, a.V = vocab, a.T = tokens, a.top = top, a.block = block;
  a.is_bf16 = dtype == POETX_BF16;
  return head_loss_scratch(a, (gradients & POETX_GRAD_X) != 0, (gradients & POETX_GRAD_W) != 0);
}

poetx_status run(LossArgs& a, poetx_dtype dtype, void* workspace, size_t workspace_bytes,
                 poetx_stream stream) {
  if (!sizes_ok(a.d, a.V, a.T, a.top, dtype, a.block) ||
      (a.index_bytes != 4 && a.index_bytes != 8))
    return POETX_ERR_INVALID_ARG;
  if (a.total == nullptr || !aligned(a.total, 4) || !aligned(a.dW, 16))
    return POETX_ERR_INVALID_ARG;
  a.is_bf16 = dtype == POETX_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a.T == 0) {
    cudaError_t e = cudaMemsetAsync(a.total, 0, sizeof(float), s);
    if (e == cudaSuccess && a.dW != nullptr)
      e = cudaMemsetAsync(a.dW, 0, static_cast<size_t>(a.V) * a.d * (a.is_bf16 ? 2 : 4), s);
    return to_status(e);
  }
  if (a.x == nullptr || a.W == nullptr || a.indices == nullptr || a.loss == nullptr ||
      overlaps(a, nullptr, 0))
    return POETX_ERR_INVALID_ARG;
  for (const void* p : {a.x, a.W, static_cast<const void*>(a.dx)})
    if (!aligned(p, 16)) return POETX_ERR_INVALID_ARG;
  if (!aligned(a.indices, a.index_bytes) || !aligned(a.weights, 4) || !aligned(a.loss, 4) ||
      !aligned(a.top_logits, a.top_bf16 ? 2 : 4))
    return POETX_ERR_INVALID_ARG;
  const size_t need = head_loss_scratch(a, a.dx != nullptr, a.dW != nullptr);
  if (workspace == nullptr || !aligned(workspace, 16) || workspace_bytes < need)
    return POETX_ERR_WORKSPACE;
  if (overlaps(a, workspace, need)) return POETX_ERR_INVALID_ARG;
  return to_status(head_loss(a, workspace, s));
}

}  // namespace

extern "C" {

size_t poetx_cross_entropy_workspace_size(int d, int vocab, int64_t tokens, poetx_dtype dtype,
                                          int gradients, int64_t block_tokens) {
  return workspace_size(d, vocab, tokens, 1, dtype, gradients, block_tokens);
}

poetx_status poetx_cross_entropy(const void* x, const void* W, const void* targets,
                                 int index_bytes, const float* weights, float* loss, float* total,
                                 void* dx, void* dW, int d, int vocab, int64_t tokens,
                                 poetx_dtype dtype, int64_t block_tokens, void* workspace,
                                 size_t workspace_bytes, poetx_stream stream) {
  LossArgs a;
  a.x = x, a.W = W, a.indices = targets, a.index_bytes = index_bytes, a.weights = weights;
  a.loss = loss, a.total = total, a.dx = dx, a.dW = dW;
  a.d = d, a.V = vocab, a.T = tokens, a.block = block_tokens;
  return run(a, dtype, workspace, workspace_bytes, stream);
}

size_t poetx_distill_workspace_size(int d, int vocab, int64_t tokens, int top, poetx_dtype dtype,
                                    int gradients, int64_t block_tokens) {
  return workspace_size(d, vocab, tokens, top, dtype, gradients, block_tokens);
}

poetx_status poetx_distill(const void* x, const void* W, const void* top_indices, int index_bytes,
                           const void* top_logits, poetx_dtype logits_dtype, const float* weights,
                           float* loss, float* total, void* dx, void* dW, int d, int vocab,
                           int64_t tokens, int top, float temperature, poetx_dtype dtype,
                           int64_t block_tokens, void* workspace, size_t workspace_bytes,
                           poetx_stream stream) {
  if (!dtype_ok(logits_dtype) || !(temperature >= 1.f / 64.f && temperature <= 64.f) ||
      (tokens > 0 && top_logits == nullptr))
    return POETX_ERR_INVALID_ARG;
  LossArgs a;
  a.x = x, a.W = W, a.indices = top_indices, a.index_bytes = index_bytes, a.weights = weights;
  a.top_logits = top_logits, a.top_bf16 = logits_dtype == POETX_BF16;
  a.loss = loss, a.total = total, a.dx = dx, a.dW = dW;
  a.d = d, a.V = vocab, a.T = tokens, a.top = top, a.tau = temperature, a.block = block_tokens;
  return run(a, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
