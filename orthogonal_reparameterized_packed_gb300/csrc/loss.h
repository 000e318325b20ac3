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

// What the kernels share in the workspace.  "Row": a token that counts, in the
// tokens' order; a block is `block` rows from `first` on.
struct LossRows {
  int* count;    // rows
  float* most;   // the largest |weight| of a row (1 if that is 0 or none is given)
  int* done;     // CTAs of the last kernel that writes losses
  int* again;    // per block: a row's reference did not fit
  int* pos;      // [T]: a token's row, -1 where it does not count
  int* token;    // [T]: a row's token
  int* index;    // [T][top] by token, ascending and different, -1: no entry
  float* p;      // [T][top]
  float* ent;    // [T] by token: sum_k p log p
  int* lead;     // [T] by token: the index of its largest p
  double* totals;  // [T]: w loss, summed over the rows of a CTA
  float* z;      // [T][top] by token: the entries' logits
  float* ref;    // [T] by row: reference of the exponentials, in units of log 2
  float2* scale;  // [T] by row: tau / (sum of its exponentials), weight
};

// The three products of bf16 on CTA pairs (loss_pair.cu), of the rows of a block:
//   logits  z = x W^T; per row and 64 columns the largest z and the sum of
//           e = 2^(z unit - ref), e itself where E is not null (its rows behind the
//           last up to a multiple of 64: 0); without E, e relative to the 64
//           columns' own largest; the logits of the rows' entries.
//   dx      dx[token] = (E W) scale
//   dw      dW = E^T x most, summed over the blocks
struct LossProducts {
  const void* x;  // [x_rows][ldx], from the block's first row on
  long long ldx, x_rows;
  const void* W;  // [V][ldw]
  long long ldw;
  void* E;        // [block][lde]
  long long lde;
  float2* part;   // [parts][ldp]
  long long ldp;
  float unit;     // log2(e) / tau
  long long first, block;
  int d, V, top;
  void* dx;       // [T][d]
  void* dW;       // [V][d]
  float* acc;     // [V][d] fp32, or null: there is one block
  float* parts;   // loss_cut_bytes, needed where loss_cuts(V) for dx, loss_cuts(block) for dw
  void* schedule;  // 64 bytes
  LossRows rows;
};

int loss_parts(int V);
bool loss_cuts(long long K);
size_t loss_cut_bytes();
// only_again: does nothing unless the block's flag is set
cudaError_t loss_logits(const LossProducts& g, bool only_again, cudaStream_t s);
cudaError_t loss_dx(const LossProducts& g, cudaStream_t s);
cudaError_t loss_dw(const LossProducts& g, cudaStream_t s);

}  // namespace poetx
