// One matrix product of poetx_linear_* on the tensor cores, bf16 in and out:
//   z = A B^T + bias,  y = act(z) + residual
// A [M][K], rows lda apart; B [N][K], or [K][N] when b_mn, rows ldb apart
// (lda, ldb multiples of 8; pointers 16-byte aligned); y, z, residual [M][N],
// rows ld apart (any ld).  bias fp32; bias, z and residual may be null.
#pragma once

#include <cuda_runtime.h>

namespace poetx {

// What linear_stream leaves instead of y and z for the head's losses (loss.h), 128
// outputs (vocabulary entries) at a time: part[n / 128][token] = (their largest z,
// the sum of 2^((z - largest) unit)), and the z at a token's `top` ascending indices
// or, where targets are given, at its target.  *done = 0 for the kernel behind.
struct LossColumns {
  float2* part = nullptr;
  long long ldp = 0;
  float unit = 0.f;
  const int* index = nullptr;
  const void* targets = nullptr;  // target_bytes each
  int target_bytes = 8;
  float* z = nullptr;
  int top = 0;
  int* done = nullptr;
};

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
  // linear_simt: where *all_rows is 0, only rows with one of row_flags[row * segs ..
  // + segs) not 0 are computed
  const int* all_rows = nullptr;
  const int* row_flags = nullptr;
  int segs = 0;
  bool a_mn = false;  // linear_simt: A is [K][M], with b_mn
  // fp32: elements between A's rows and between y's (z's, residual's), 0: none lie between.  Up
  // to three of y's elements behind a row's last are written.
  long long pitch_a = 0, pitch_y = 0;
  // linear_fp32: K in `slices` pieces whose products are apart, piece i's in y + i M pitch_y
  // (no bias, residual or activation); linear_split_slices says how many pay
  int slices = 1;
  // linear_split: the last product on this scratch had the same array B
  bool b_ready = false;
  // linear_split: linear_planes_bytes(M, K) for A's planes, null: they are in the scratch
  void* a_planes = nullptr;
  bool a_ready = false;  // they are there, made by the caller
  const LossColumns* loss = nullptr;  // linear_stream with B [N][K]
  const char* tag = "linear";
};

// On CTA pairs, tiles of 256 x 128 to 256 (linear_pair.cu).
cudaError_t linear_pair(const LinearProduct& g, cudaStream_t s);

// For few tokens: the weight streamed once, K split over a cluster (linear_stream.cu).
cudaError_t linear_stream(const LinearProduct& g, cudaStream_t s);

// In fp32 on the CUDA cores (linear_simt.cu): A ([M][K], or a_mn), y, z, residual
// contiguous unless pitch_a, pitch_y say otherwise, B [N][K] or, b_mn, [K][N]
// contiguous; lda, ldb and ld are not used.
cudaError_t linear_simt(const LinearProduct& g, cudaStream_t s);

// In fp32 on the tensor cores, as six bf16 products (linear_split.cu); layouts
// as for linear_simt, scratch of linear_split_scratch(g) bytes.
bool linear_split_pays(long long M, int N, int K);
size_t linear_split_scratch(const LinearProduct& g);
size_t linear_split_b_scratch(const LinearProduct& g);  // with a_planes
size_t linear_split_scratch_up_to(const LinearProduct& g);  // of any product of at most g.M rows
cudaError_t linear_split(const LinearProduct& g, void* scratch, cudaStream_t s);
// Whether linear_split left *scratch not 0: values of B are for the CUDA cores, which
// computed everything (with slices, the first slice).

// The planes of an fp32 array [rows][cols] that are kept.  A caller that makes them itself:
// planes [3][plane_rows][pitch] bf16 as linear_planes.cuh has it, rows behind the last 0,
// and a flag per row, whether a value of it is outside.
struct Fp32Planes {
  void* planes;
  int* flags;
  long long plane_rows, pitch;
};
size_t linear_planes_bytes(long long rows, int cols);
Fp32Planes linear_planes_at(void* at, long long rows, int cols);
cudaError_t linear_split_planes(const float* in, long long rows, int cols, long long ld, void* at,
                                cudaStream_t s);
// With a_mn and b_mn, from the kept planes of A, of the caller's making, and of B.
cudaError_t linear_split_turned(const LinearProduct& g, void* a_planes, void* b_planes,
                                cudaStream_t s);

// In fp32 in the form that takes less time, with linear_split_scratch_up_to(g) bytes
// of scratch or more (linear.cu); in slices always linear_split.
cudaError_t linear_fp32(const LinearProduct& g, void* scratch, cudaStream_t s);

// Pieces of K, 2 to kMaxFp32Slices with outputs of at most most_bytes, where these
// are faster than linear_fp32 on the whole of K: a product of few tiles and a long K.
// Else 1.
constexpr int kMaxFp32Slices = 32;
int linear_split_slices(long long M, int N, int K, size_t most_bytes);

}  // namespace poetx
