// One matrix product of poetx_linear_* on the tensor cores, bf16 in and out:
//   z = A B^T + bias,  y = act(z) + residual
// A [M][K], rows lda apart; B [N][K], or [K][N] when b_mn, rows ldb apart
// (lda, ldb multiples of 8; pointers 16-byte aligned); y, z, residual [M][N],
// rows ld apart (any ld).  bias fp32; bias, z and residual may be null.
#pragma once

#include <cuda_runtime.h>

namespace poetx {

struct LinearProduct {
  const void* A = nullptr;
  const void* B = nullptr;
  long long lda = 0, ldb = 0, ld = 0;
  bool b_mn = false;
  const float* bias = nullptr;
  const void* residual = nullptr;
  void* y = nullptr;
  void* z = nullptr;
  long long M = 0;
  int N = 0, K = 0;
  int act = 0;
  // linear_simt: where flags[0] is 0, only rows with one of flags[1 + row * segs ..
  // + segs) not 0 are computed
  const int* flags = nullptr;
  int segs = 0;
  const char* tag = "linear";
};

// On CTA pairs, tiles of 256 x 128 to 256 (linear_pair.cu).
cudaError_t linear_pair(const LinearProduct& g, cudaStream_t s);

// For few tokens: the weight streamed once, K split over a cluster (linear_stream.cu).
cudaError_t linear_stream(const LinearProduct& g, cudaStream_t s);

// In fp32 on the CUDA cores (linear_simt.cu): A, y, z, residual contiguous, B
// [N][K] or, b_mn, [K][N] contiguous; lda, ldb and ld are not used.
cudaError_t linear_simt(const LinearProduct& g, cudaStream_t s);

// In fp32 on the tensor cores, as six bf16 products (linear_split.cu); layouts
// as for linear_simt, scratch of linear_split_scratch(g) bytes.
bool linear_split_pays(long long M, int N, int K);
size_t linear_split_scratch(const LinearProduct& g);
size_t linear_split_scratch_up_to(const LinearProduct& g);  // of any product of at most g.M rows
cudaError_t linear_split(const LinearProduct& g, void* scratch, cudaStream_t s);

}  // namespace poetx
