// The losses at the output head, shared by their translation units.
#pragma once

#include <cuda_runtime.h>

#include <cstddef>

namespace poetx {

// One call.  x [T][d], W [V][d], dx, dW in the working type; a token's entries
// (index, weight): cross entropy has one, its target, of weight 1; distillation
// `top`, from the teacher's logits.
struct LossArgs {
  const void* x = nullptr;
  const void* W = nullptr;
  const void* indices = nullptr;  // [T][top], index_bytes each
  int index_bytes = 8;
  const void* top_logits = nullptr;  // [T][top]; null: cross entropy
  bool top_bf16 = false;
  const float* weights = nullptr;  // [T]; null: 1 / counted tokens
  float* loss = nullptr;           // [T]
  float* total = nullptr;
  void* dx = nullptr;  // may be null
  void* dW = nullptr;  // may be null
  int d = 0, V = 0, top = 1;
  long long T = 0, block = 0;  // block: tokens whose logits are held at a time, 0: by size
  float tau = 1.f;
  bool is_bf16 = false;
};

// Bytes of workspace for LossArgs' sizes and the presence of dx and dW.
size_t head_loss_scratch(const LossArgs& a, bool want_dx, bool want_dw);
cudaError_t head_loss(const LossArgs& a, void* scratch, cudaStream_t s);

}  // namespace poetx
