// The matrix product with bias, activation and residual, and its gradients:
//   z = x W^T + bias,  y = act(z) + residual
//   dz = dy act'(z),   dx = dz W,   dbias = sum_t dz
#include <algorithm>
#include <cstdint>

#include "activation.cuh"
#include "internal.h"
#include "linear.h"
#include "poetx.h"
#include "ptx.cuh"

namespace poetx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;

// Elements between rows of `cols` bf16 features as TMA operands: as they are
// where that is a multiple of 16 bytes, else copied onto whole 128-byte lines.
long long tma_pitch(int cols) {
  return cols % 8 == 0 ? cols : (static_cast<long long>(cols) + 63) / 64 * 64;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& o, float x) { o = x; }
__device__ __forceinline__ void from_f(bf16& o, float x) { o = __float2bfloat16_rn(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

// dz = dy act'(z) (stored where dz is not null) and, where part is not null,
// its column sums over this CTA's rows: part[blockIdx.y][N].  dz is rounded to the
// working type, which the product takes (in bf16 dx is then 2.3e-3 of its norm from
// the exact one, where one rounding alone leaves 1.7e-3; a second plane of dz would
// halve the product's rate); the sums are of the unrounded values.  32 column
// threads of V columns each, 8 row threads, kDzRows rows per CTA.  Bound by its
// three passes over [T][N]: 8192 x 5632 with silu 47 us, 5.9 TB/s.  It is the
// number of resident warps that hides the loads (32 per SM here): four rows in
// flight per thread at 16 warps took 101 us.
constexpr int kDzRows = 128;

template <typename T, int ACT, int V>
__global__ void __launch_bounds__(kThreads, 4)
    linear_dz_kernel(const T* __restrict__ dy, const T* __restrict__ z, T* __restrict__ dz,
                     long long ld_dz, float* __restrict__ part, long long T_rows, int N) {
  pdl_wait();
  pdl_trigger();
  constexpr bool FAST = sizeof(T) == 2;
  __shared__ float sums[8][32 * V];
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const long long col = (static_cast<long long>(blockIdx.x) * 32 + tx) * V;
  const long long r0 = static_cast<long long>(blockIdx.y) * kDzRows;
  const int rows = static_cast<int>(min(static_cast<long long>(kDzRows), T_rows - r0));
  float sum[V] = {};
  if (col < N) {
    const T* gp = dy + r0 * N + col;
    const T* zp = ACT != POETX_ACT_NONE ? z + r0 * N + col : nullptr;
    T* op = dz != nullptr ? dz + r0 * ld_dz + col : nullptr;
    for (int r = ty; r < rows; r += 8) {
      const long long at = static_cast<long long>(r) * N;
      Pack<T, V> g = *reinterpret_cast<const Pack<T, V>*>(gp + at), zz = g;
      if (ACT != POETX_ACT_NONE) zz = *reinterpret_cast<const Pack<T, V>*>(zp + at);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float d = act_grad<ACT, FAST>(to_f(g.x[j]), to_f(zz.x[j]));
        sum[j] += d;
        from_f(g.x[j], d);
      }
      if (op != nullptr)
        *reinterpret_cast<Pack<T, V>*>(op + static_cast<long long>(r) * ld_dz) = g;
    }
  }
  if (part == nullptr) return;
#pragma unroll
  for (int j = 0; j < V; ++j) sums[ty][tx * V + j] = sum[j];
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * V; i += kThreads) {
    const long long c = static_cast<long long>(blockIdx.x) * 32 * V + i;
    if (c >= N) continue;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) v += sums[w][i];
    part[static_cast<long long>(blockIdx.y) * N + c] = v;
  }
}

// hi + lo += x, the rounding error of hi + x kept in lo (two-sum).
__device__ __forceinline__ void add_to(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}

// dbias[c] = sum over the row blocks' partial sums, in order, as pairs of fp32
// (fp64 runs at 1/64 of the rate); kDbiasFlight loads in flight per thread.
// It waits like every kernel, though the sums were complete before the product
// began: what a grid two launches back wrote is visible only after the wait.  Its
// CTAs get there while the product's last round runs; what follows begins behind
// them.  The backward of 2048 -> 5632, T = 8192, in a graph: 157.5 us with this
// kernel behind the product, 158.5 if it triggers early, 162 before the product.
constexpr int kDbiasFlight = 8;

__global__ void __launch_bounds__(kThreads)
    linear_dbias_kernel(const float* __restrict__ part, int blocks, int N,
                        float* __restrict__ dbias) {
  pdl_wait();
  __shared__ float2 sums[8][32];
  const int tx = threadIdx.x % 32, ty = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + tx;
  float hi = 0.f, lo = 0.f;
  if (c < N)
    for (int b0 = ty; b0 < blocks; b0 += 8 * kDbiasFlight) {
      float p[kDbiasFlight];
#pragma unroll
      for (int i = 0; i < kDbiasFlight; ++i) {
        const int b = b0 + 8 * i;
        p[i] = b < blocks ? part[static_cast<long long>(b) * N + c] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < kDbiasFlight; ++i) add_to(hi, lo, p[i]);
    }
  sums[ty][tx] = make_float2(hi, lo);
  __syncthreads();
  if (ty == 0 && c < N) {
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      add_to(hi, lo, sums[w][tx].x);
      lo = __fadd_rn(lo, sums[w][tx].y);
    }
    // an infinite hi has a lo that is NaN
    dbias[c] = fabsf(hi) < INFINITY ? hi + lo : hi;
  }
}

// The kernel of a function template over the activation, by its runtime value.
#define LINEAR_BY_ACT(act, call)        \
  switch (act) {                        \
    case POETX_ACT_RELU: call(1); break; \
    case POETX_ACT_SILU: call(2); break; \
    case POETX_ACT_GELU: call(3); break; \
    case POETX_ACT_GELU_TANH: call(4); break; \
    default: call(0);                   \
  }

// out[r][0..cols) = in[r][0..cols), rows in_ld and out_ld apart: rows of an odd
// number of bf16 features onto a 16-byte pitch, which TMA needs.  One warp
// per row piece of 256 columns.
__global__ void __launch_bounds__(kThreads)
    pad_rows_kernel(const bf16* __restrict__ in, long long in_ld, bf16* __restrict__ out,
                    long long out_ld, long long rows, int cols) {
  pdl_wait();
  pdl_trigger();
  const int pieces = (cols + 255) / 256;
  const long long items = rows * pieces;
  const int lane = threadIdx.x % 32;
  for (long long it = blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32;
       it < items; it += static_cast<long long>(gridDim.x) * (kThreads / 32)) {
    const long long r = it / pieces;
    const int c0 = static_cast<int>(it - r * pieces) * 256;
    bf16 v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + lane + 32 * j;
      if (c < cols) v[j] = in[r * in_ld + c];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = c0 + lane + 32 * j;
      if (c < cols) out[r * out_ld + c] = v[j];
    }
  }
}

cudaError_t pad_rows(const void* in, void* out, long long rows, int cols, cudaStream_t s) {
  const long long items = rows * ((cols + 255) / 256);
  const int grid = static_cast<int>(
      std::min<long long>((items + kThreads / 32 - 1) / (kThreads / 32), 16ll * sm_count()));
  prof_begin("linear_pad", s);
  const cudaError_t e =
      launch_pdl(pad_rows_kernel, dim3(grid), dim3(kThreads), 0, s, static_cast<const bf16*>(in),
                 static_cast<long long>(cols), static_cast<bf16*>(out), tma_pitch(cols), rows,
                 cols);
  prof_end("linear_pad", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, int V>
cudaError_t run_dz(const void* dy, const void* z, void* dz, long long ld_dz, float* part,
                   long long T_rows, int N, int act, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const dim3 grid(static_cast<unsigned>((N + 32 * V - 1) / (32 * V)),
                  static_cast<unsigned>((T_rows + kDzRows - 1) / kDzRows));
  prof_begin("linear_dz", s);
#define RUN(A)                                                                       \
  e = launch_pdl(linear_dz_kernel<T, A, V>, grid, dim3(kThreads), 0, s,              \
                 static_cast<const T*>(dy), static_cast<const T*>(z), static_cast<T*>(dz), \
                 ld_dz, part, T_rows, N)
  LINEAR_BY_ACT(act, RUN)
#undef RUN
  prof_end("linear_dz", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

// Bytes of a padded copy of [rows][cols] bf16, 0 where the rows are aligned already.
size_t pad_bytes(long long rows, int cols) {
  return cols % 8 == 0 ? 0 : round256(static_cast<size_t>(rows) * tma_pitch(cols) * 2);
}

}  // namespace

namespace {

// Where linear_stream is ahead of linear_pair: up to 64 tokens always (4096 ->
// 4096, one token: 8.5 against 14.8 us), and where its tiles are too few to give
// every cluster of the pairs one while K is long enough to be split.  Up to 128
// tokens: 64 tiles, K / 64 of them (8192 -> 8192, 64 tiles: 28.2 against 30.6 us;
// 2048 -> 4096, 32: 8.7 against 10.3; 2048 -> 5632, 44: 11.4 against 10.7).
// Beyond, with one CTA per SM: 32 tiles, K / 128 of them (256 tokens, 4096 ->
// 4096, 32 tiles: 14.5 against 15.8; 6144 -> 6144, 48: 25.8 against 22.2; 2048 ->
// 4096, 32: 11.3 against 10.4; 1024 tokens, 8192 -> 1024, 32: 18.6 against 25.9).
bool stream_form(long long M, int N, int K) {
  if (M <= 64) return true;
  const long long tiles = (N + 127) / 128 * ((M + 255) / 256);
  return K >= 2048 && tiles <= (M <= 128 ? std::min(64, K / 64) : std::min(32, K / 128));
}

cudaError_t run_product(const LinearProduct& g, cudaStream_t s) {
  return stream_form(g.M, g.N, g.K) ? linear_stream(g, s) : linear_pair(g, s);
}

}  // namespace

namespace {

// fp32: the scratch and the run of a product [M][K] x [K][N] (b_mn as in
// LinearProduct); fewer: the scratch that every product of up to M rows fits.
size_t fp32_scratch(long long M, int N, int K, bool b_mn, bool fewer) {
  LinearProduct g;
  g.M = M;
  g.N = N;
  g.K = K;
  g.b_mn = b_mn;
  if (fewer) return linear_split_scratch_up_to(g);
  return linear_split_pays(M, N, K) ? linear_split_scratch(g) : 0;
}

cudaError_t run_fp32(const LinearProduct& g, void* scratch, cudaStream_t s) {
  return linear_split_pays(g.M, g.N, g.K) ? linear_split(g, scratch, s) : linear_simt(g, s);
}

}  // namespace

// bf16: padded copies of x and W where d_in is no multiple of 8; fp32: the
// planes of x and W where the product runs on the tensor cores.
size_t linear_forward_scratch(int d_in, int d_out, long long T, bool is_bf16, bool fewer) {
  return is_bf16 ? pad_bytes(T, d_in) + pad_bytes(d_out, d_in)
                 : fp32_scratch(T, d_out, d_in, false, fewer);
}

cudaError_t linear_forward(const void* x, const void* W, const float* bias, const void* residual,
                           void* y, void* z, int d_in, int d_out, long long T, int act,
                           bool is_bf16, void* scratch, cudaStream_t s) {
  cudaError_t e;
  LinearProduct g;
  g.A = x;
  g.B = W;
  g.lda = g.ldb = tma_pitch(d_in);
  if (is_bf16 && d_in % 8 != 0) {
    char* xp = static_cast<char*>(scratch);
    char* wp = xp + pad_bytes(T, d_in);
    if ((e = pad_rows(x, xp, T, d_in, s)) != cudaSuccess) return e;
    if ((e = pad_rows(W, wp, d_out, d_in, s)) != cudaSuccess) return e;
    g.A = xp;
    g.B = wp;
  }
  g.ld = d_out;
  g.bias = bias;
  g.residual = residual;
  g.y = y;
  g.z = z;
  g.M = T;
  g.N = d_out;
  g.K = d_in;
  g.act = act;
  return is_bf16 ? run_product(g, s) : run_fp32(g, scratch, s);
}

// Scratch of the backward: dz (unless it is dy itself, aligned), the row
// blocks' sums of dbias, and in bf16 the padded W, in fp32 the planes.
namespace {

struct BackwardPlan {
  size_t dz = 0, part = 0, w = 0;
  int blocks;
  BackwardPlan(int d_in, int d_out, long long T, int act, bool is_bf16, bool with_dbias,
               bool fewer) {
    blocks = static_cast<int>((T + kDzRows - 1) / kDzRows);
    if (is_bf16) {
      if (act != POETX_ACT_NONE || d_out % 8 != 0)
        dz = round256(static_cast<size_t>(T) * tma_pitch(d_out) * 2);
      w = pad_bytes(d_out, d_in);
    } else {
      if (act != POETX_ACT_NONE) dz = round256(static_cast<size_t>(T) * d_out * 4);
      w = fp32_scratch(T, d_in, d_out, true, fewer);
    }
    if (with_dbias) part = round256(static_cast<size_t>(blocks) * d_out * 4);
  }
  size_t bytes() const { return dz + part + w; }
};

}  // namespace

size_t linear_backward_scratch(int d_in, int d_out, long long T, int act, bool is_bf16,
                               bool with_dbias, bool fewer) {
  return BackwardPlan(d_in, d_out, T, act, is_bf16, with_dbias, fewer).bytes();
}

cudaError_t linear_backward(const void* dy, const void* z, const void* W, void* dx, float* dbias,
                            int d_in, int d_out, long long T, int act, bool is_bf16,
                            void* scratch, cudaStream_t s) {
  const BackwardPlan plan(d_in, d_out, T, act, is_bf16, dbias != nullptr, false);
  char* at = static_cast<char*>(scratch);
  void* dz = plan.dz > 0 && dx != nullptr ? at : nullptr;  // null: not stored
  float* part = plan.part > 0 ? reinterpret_cast<float*>(at + plan.dz) : nullptr;
  void* wp = at + plan.dz + plan.part;
  const long long ld_dz = is_bf16 ? tma_pitch(d_out) : d_out;
  cudaError_t e;
  if (dz != nullptr || part != nullptr) {
    if (is_bf16)
      e = d_out % 8 == 0 ? run_dz<bf16, 8>(dy, z, dz, ld_dz, part, T, d_out, act, s)
                         : run_dz<bf16, 1>(dy, z, dz, ld_dz, part, T, d_out, act, s);
    else
      e = d_out % 4 == 0 ? run_dz<float, 4>(dy, z, dz, ld_dz, part, T, d_out, act, s)
                         : run_dz<float, 1>(dy, z, dz, ld_dz, part, T, d_out, act, s);
    if (e != cudaSuccess) return e;
  }
  const auto sum_dbias = [&]() {
    if (part == nullptr) return cudaSuccess;
    prof_begin("linear_dbias", s);
    e = launch_pdl(linear_dbias_kernel, dim3((d_out + 31) / 32), dim3(kThreads), 0, s,
                   static_cast<const float*>(part), plan.blocks, d_out, dbias);
    prof_end("linear_dbias", s);
    return e != cudaSuccess ? e : cudaGetLastError();
  };
  if (dx == nullptr) return sum_dbias();
  const void* grad = dz != nullptr ? dz : dy;
  LinearProduct g;
  g.A = grad;
  g.lda = ld_dz;
  g.B = W;
  g.ldb = tma_pitch(d_in);
  g.b_mn = true;
  if (is_bf16 && plan.w > 0) {
    if ((e = pad_rows(W, wp, d_out, d_in, s)) != cudaSuccess) return e;
    g.B = wp;
  }
  g.ld = d_in;
  g.y = dx;
  g.M = T;
  g.N = d_in;
  g.K = d_out;
  g.tag = "linear_dgrad";
  e = is_bf16 ? run_product(g, s) : run_fp32(g, wp, s);
  return e != cudaSuccess ? e : sum_dbias();
}

}  // namespace poetx
