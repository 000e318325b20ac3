// The losses at the output head, from the last hidden states x and the head's
// weight W:
//   u_tv = x_t . W_v / tau,   lse_t = log sum_v exp(u_tv)
//   loss_t = tau^2 sum_k p_tk (log p_tk - u_t,i_tk + lse_t)
// over a token's entries (index i_tk, weight p_tk): cross entropy is one entry of
// weight 1 at tau = 1, distillation the teacher's top logits s, p = softmax(s / tau).
// With the token weights w, total = sum_t w_t loss_t and its gradients are
//   dz_tv = w_t tau (exp(u_tv - lse_t) - sum_{k: i_tk = v} p_tk)
//   dx = dz W,   dW = dz^T x
// Tokens without an entry do not count: no loss, no gradient, and nothing that x
// holds there reaches another token (0 times NaN would, in dW's sum over tokens).
// So the tokens that count are gathered first, in order, and everything runs on
// the gathered rows; they are taken in blocks whose logits fit the workspace.
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "loss.h"
#include "poetx.h"
#include "ptx.cuh"

namespace poetx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kOrderThreads = 1024;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& o, float x) { o = x; }
__device__ __forceinline__ void from_f(bf16& o, float x) { o = __float2bfloat16_rn(x); }

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ long long index_at(const void* p, int bytes, long long i) {
  return bytes == 8 ? static_cast<const long long*>(p)[i] : static_cast<const int*>(p)[i];
}

// What the kernels share in the workspace.
struct Lists {
  int* count;   // [0]: tokens that count
  int* pos;     // [T]: a token's gathered row, -1 where it does not count
  int* rows;    // [T]: a gathered row's token
  int* index;   // [T][top] of the token, -1: no entry
  float* p;     // [T][top]
  float* ent;   // [T]: sum_k p log p
};

// The entries of a token, a warp each: p = softmax of the teacher's logits at tau
// over the entries that are there (for the cross entropy 1).  Differences are
// divided by tau, not the logits: the type's lowest value stays finite.
__global__ void __launch_bounds__(kThreads)
    loss_entries_kernel(const void* indices, int index_bytes, const void* logits, bool logits_bf16,
                        long long T, int top, int V, float inv_tau, Lists l, int* status) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32;
  const long long t = blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32;
  if (t >= T) return;
  const long long base = t * top;
  bool outside = false, any = false;
  float m = -INFINITY;
  const auto logit = [&](int k) {
    if (logits == nullptr) return 0.f;
    return logits_bf16 ? to_f(static_cast<const bf16*>(logits)[base + k])
                       : static_cast<const float*>(logits)[base + k];
  };
  for (int k = lane; k < top; k += 32) {
    const long long i = index_at(indices, index_bytes, base + k);
    outside |= i >= V;
    const bool there = i >= 0 && i < V && !(logit(k) == -INFINITY);
    l.index[base + k] = there ? static_cast<int>(i) : -1;
    if (there) m = fmaxf(m, logit(k));
    any |= there;
  }
  m = warp_max(m);
  any = __any_sync(0xffffffffu, any);
  outside = __any_sync(0xffffffffu, outside);
  float sum = 0.f;
  for (int k = lane; k < top; k += 32)
    if (l.index[base + k] >= 0) sum += expf((logit(k) - m) * inv_tau);
  const float log_sum = logf(warp_sum(sum));
  float ent = 0.f;
  for (int k = lane; k < top; k += 32) {
    float p = 0.f;
    if (l.index[base + k] >= 0) {
      const float log_p = (logit(k) - m) * inv_tau - log_sum;
      p = expf(log_p);
      if (p > 0.f) ent += p * log_p;
      if (isnan(log_p)) ent = log_p;
    }
    l.p[base + k] = p;
  }
  ent = warp_sum(ent);
  if (lane == 0) {
    l.pos[t] = any ? 0 : -1;
    l.ent[t] = ent;
    if (outside) atomicCAS(status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
  }
}

// pos[t] (0 or -1) -> the number of tokens before t that count, or -1; rows its
// inverse.  One CTA, kOrderThreads tokens at a time.
__global__ void __launch_bounds__(kOrderThreads) loss_order_kernel(Lists l, long long T) {
  __shared__ int sums[32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int before = 0;
  for (long long t0 = 0; t0 < T; t0 += kOrderThreads) {
    const long long t = t0 + threadIdx.x;
    const bool on = t < T && l.pos[t] >= 0;
    const unsigned mask = __ballot_sync(0xffffffffu, on);
    if (lane == 0) sums[warp] = __popc(mask);
    __syncthreads();
    int mine = before, all = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) mine += sums[w];
      all += sums[w];
    }
    mine += __popc(mask & ((1u << lane) - 1));
    if (on) {
      l.pos[t] = mine;
      l.rows[mine] = static_cast<int>(t);
    }
    before += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) l.count[0] = before;
}

// A warp per token: the rows that count to their places, zeros to dx and loss of
// the others; warps from T on: zeros to the gathered rows behind the last.
template <typename TX>
__global__ void __launch_bounds__(kThreads)
    loss_gather_kernel(const TX* __restrict__ x, Lists l, long long T, int d, TX* __restrict__ xg,
                       float* __restrict__ loss, TX* __restrict__ dx) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32;
  const long long t = blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32;
  if (t >= 2 * T) return;
  TX zero;
  from_f(zero, 0.f);
  if (t >= T) {
    const long long r = t - T;
    if (r >= *l.count)
      for (int c = lane; c < d; c += 32) xg[r * d + c] = zero;
    return;
  }
  const int at = l.pos[t];
  if (at >= 0) {
    for (int c = lane; c < d; c += 32) xg[static_cast<long long>(at) * d + c] = x[t * d + c];
    return;
  }
  if (lane == 0) loss[t] = 0.f;
  if (dx != nullptr)
    for (int c = lane; c < d; c += 32) dx[t * d + c] = zero;
}

// A CTA per gathered row of the block: its loss from the fp32 logits z, and in
// place of them dz where the gradients are wanted (rows that do not count: 0).
__global__ void __launch_bounds__(kThreads)
    loss_rows_kernel(float* __restrict__ z, Lists l, long long first, int V, int top,
                     float inv_tau, float tau, const float* __restrict__ weights, bool grad,
                     float* __restrict__ loss) {
  pdl_wait();
  pdl_trigger();
  __shared__ float ms[kThreads / 32], ss[kThreads / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long r = first + blockIdx.x;
  float* row = z + static_cast<long long>(blockIdx.x) * V;
  const int n = *l.count;
  if (r >= n) {
    if (grad)
      for (int v = threadIdx.x; v < V; v += kThreads) row[v] = 0.f;
    return;
  }
  float m = -INFINITY;
  for (int v = threadIdx.x; v < V; v += kThreads) m = fmaxf(m, row[v]);
  m = warp_max(m);
  if (lane == 0) ms[warp] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) m = fmaxf(m, ms[w]);
  float s = 0.f;
  for (int v = threadIdx.x; v < V; v += kThreads) s += expf((row[v] - m) * inv_tau);
  s = warp_sum(s);
  if (lane == 0) ss[warp] = s;
  __syncthreads();
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) s += ss[w];
  const long long t = l.rows[r], base = t * top;
  const float log_s = logf(s);
  if (warp == 0) {
    float sum = 0.f;
    for (int k = lane; k < top; k += 32) {
      const int i = l.index[base + k];
      if (i >= 0) sum += l.p[base + k] * (log_s - (row[i] - m) * inv_tau);
    }
    sum = warp_sum(sum);
    if (lane == 0) loss[t] = tau * tau * (l.ent[t] + sum);
  }
  if (!grad) return;
  const float scale = (weights != nullptr ? weights[t] : 1.f / static_cast<float>(n)) * tau;
  __syncthreads();
  for (int v = threadIdx.x; v < V; v += kThreads)
    row[v] = scale * (expf((row[v] - m) * inv_tau) / s);
  __syncthreads();
  if (threadIdx.x == 0)
    for (int k = 0; k < top; ++k) {
      const int i = l.index[base + k];
      if (i >= 0) row[i] -= scale * l.p[base + k];
    }
}

// total = sum over the tokens that count of w loss, in 64 bits, one CTA.
__global__ void __launch_bounds__(kOrderThreads)
    loss_total_kernel(const float* __restrict__ loss, const float* __restrict__ weights, Lists l,
                      long long T, float* __restrict__ total) {
  pdl_wait();
  pdl_trigger();
  __shared__ double sums[32];
  double sum = 0.0;
  for (long long t = threadIdx.x; t < T; t += kOrderThreads)
    if (l.pos[t] >= 0) sum += (weights != nullptr ? weights[t] : 1.0) * loss[t];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < kOrderThreads / 32; ++w) sum += sums[w];
    if (weights == nullptr) sum /= max(1, *l.count);
    *total = static_cast<float>(sum);
  }
}

// out[m][n] = sum_k A(m, k) B(k, n) in fp32, element strides; accumulated onto
// out32 and / or rounded into out (row m at rows[m], only the first *limit).
struct Product {
  const void* A;
  const void* B;
  long long am, ak, bk, bn;
  long long M;
  int N;
  long long K;
  float* out32;
  bool add;
  void* out;
  const int* rows;
  const int* limit;
  long long first;
};

template <typename TA, typename TB, typename TO>
__global__ void __launch_bounds__(256) loss_product_kernel(const Product p) {
  pdl_wait();
  pdl_trigger();
  __shared__ float as[16][65], bs[16][65];
  const TA* A = static_cast<const TA*>(p.A);
  const TB* B = static_cast<const TB*>(p.B);
  const long long m0 = blockIdx.y * 64ll, n0 = blockIdx.x * 64ll;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  float acc[4][4] = {};
  for (long long k0 = 0; k0 < p.K; k0 += 16) {
    for (int e = threadIdx.x; e < 1024; e += 256) {
      const int k = p.ak == 1 ? e % 16 : e / 64, m = p.ak == 1 ? e / 16 : e % 64;
      as[k][m] = m0 + m < p.M && k0 + k < p.K ? to_f(A[(m0 + m) * p.am + (k0 + k) * p.ak]) : 0.f;
      const int kb = p.bk == 1 ? e % 16 : e / 64, n = p.bk == 1 ? e / 16 : e % 64;
      bs[kb][n] =
          n0 + n < p.N && k0 + kb < p.K ? to_f(B[(n0 + n) * p.bn + (k0 + kb) * p.bk]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = as[k][ty * 4 + i], b[i] = bs[k][tx * 4 + i];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
    }
    __syncthreads();
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m >= p.M || n >= p.N || (p.limit != nullptr && p.first + m >= *p.limit)) continue;
      float v = acc[i][j];
      if (p.add) v += p.out32[m * p.N + n];
      if (p.out32 != nullptr) p.out32[m * p.N + n] = v;
      if (p.out != nullptr) {
        const long long row = p.rows != nullptr ? p.rows[p.first + m] : m;
        from_f(static_cast<TO*>(p.out)[row * p.N + n], v);
      }
    }
}

template <typename TA, typename TB, typename TO>
cudaError_t product(const Product& p, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((p.N + 63) / 64), static_cast<unsigned>((p.M + 63) / 64));
  prof_begin("loss_product", s);
  const cudaError_t e =
      launch_pdl(loss_product_kernel<TA, TB, TO>, grid, dim3(256), 0, s, p);
  prof_end("loss_product", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

constexpr size_t kBlockBytes = size_t{1} << 31;  // of logits at a time

struct Plan {
  long long block;
  size_t count = 0, pos, rows, index, p, ent, xg, z, acc, total;
  Plan(const LossArgs& a, bool want_dw) {
    const size_t T = static_cast<size_t>(a.T);
    block = a.block > 0 ? a.block
                        : static_cast<long long>(kBlockBytes / (4 * static_cast<size_t>(a.V)));
    block = std::max<long long>(1, std::min<long long>(block, a.T));
    block = std::min<long long>(block, 64ll * 65535);
    size_t at = 256;
    const auto take = [&](size_t bytes) {
      const size_t here = at;
      at += round256(bytes);
      return here;
    };
    pos = take(4 * T);
    rows = take(4 * T);
    index = take(4 * T * a.top);
    p = take(4 * T * a.top);
    ent = take(4 * T);
    xg = take((a.is_bf16 ? 2 : 4) * T * a.d);
    z = take(4 * static_cast<size_t>(block) * a.V);
    acc = take(want_dw && a.is_bf16 ? 4 * static_cast<size_t>(a.V) * a.d : 0);
    total = at;
  }
};

template <typename T>
cudaError_t run(const LossArgs& a, char* ws, cudaStream_t s) {
  const Plan plan(a, a.dW != nullptr);
  Lists l;
  l.count = reinterpret_cast<int*>(ws + plan.count);
  l.pos = reinterpret_cast<int*>(ws + plan.pos);
  l.rows = reinterpret_cast<int*>(ws + plan.rows);
  l.index = reinterpret_cast<int*>(ws + plan.index);
  l.p = reinterpret_cast<float*>(ws + plan.p);
  l.ent = reinterpret_cast<float*>(ws + plan.ent);
  T* xg = reinterpret_cast<T*>(ws + plan.xg);
  float* z = reinterpret_cast<float*>(ws + plan.z);
  float* acc = a.is_bf16 ? reinterpret_cast<float*>(ws + plan.acc) : static_cast<float*>(a.dW);
  const float inv_tau = 1.f / a.tau;
  const unsigned warps = kThreads / 32;
  cudaError_t e;
  const auto launched = [&](const char* tag, auto&& call) {
    prof_begin(tag, s);
    cudaError_t err = call();
    prof_end(tag, s);
    return err != cudaSuccess ? err : cudaGetLastError();
  };
  e = launched("loss_entries", [&] {
    return launch_pdl(loss_entries_kernel, dim3(static_cast<unsigned>((a.T + warps - 1) / warps)),
                      dim3(kThreads), 0, s, a.indices, a.index_bytes, a.top_logits, a.top_bf16,
                      a.T, a.top, a.V, inv_tau, l, device_status_ptr());
  });
  if (e != cudaSuccess) return e;
  e = launched("loss_order", [&] {
    return launch_pdl(loss_order_kernel, dim3(1), dim3(kOrderThreads), 0, s, l, a.T);
  });
  if (e != cudaSuccess) return e;
  e = launched("loss_gather", [&] {
    return launch_pdl(loss_gather_kernel<T>,
                      dim3(static_cast<unsigned>((2 * a.T + warps - 1) / warps)), dim3(kThreads),
                      0, s, static_cast<const T*>(a.x), l, a.T, a.d, xg, a.loss,
                      static_cast<T*>(a.dx));
  });
  if (e != cudaSuccess) return e;
  const bool grad = a.dx != nullptr || a.dW != nullptr;
  for (long long first = 0; first < a.T; first += plan.block) {
    const long long rows = std::min(plan.block, a.T - first);
    const T* xb = xg + first * a.d;
    Product p = {};
    p.A = xb, p.am = a.d, p.ak = 1;
    p.B = a.W, p.bk = 1, p.bn = a.d;
    p.M = rows, p.N = a.V, p.K = a.d;
    p.out32 = z;
    if ((e = product<T, T, T>(p, s)) != cudaSuccess) return e;
    e = launched("loss_rows", [&] {
      return launch_pdl(loss_rows_kernel, dim3(static_cast<unsigned>(rows)), dim3(kThreads), 0, s,
                        z, l, first, a.V, a.top, inv_tau, a.tau, a.weights, grad, a.loss);
    });
    if (e != cudaSuccess) return e;
    if (a.dx != nullptr) {
      Product q = {};
      q.A = z, q.am = a.V, q.ak = 1;
      q.B = a.W, q.bk = a.d, q.bn = 1;
      q.M = rows, q.N = a.d, q.K = a.V;
      q.out = a.dx, q.rows = l.rows, q.limit = l.count, q.first = first;
      if ((e = product<float, T, T>(q, s)) != cudaSuccess) return e;
    }
    if (a.dW != nullptr) {
      Product q = {};
      q.A = z, q.am = 1, q.ak = a.V;
      q.B = xb, q.bk = a.d, q.bn = 1;
      q.M = a.V, q.N = a.d, q.K = rows;
      q.out32 = acc, q.add = first > 0;
      q.out = a.is_bf16 && first + plan.block >= a.T ? a.dW : nullptr;
      if ((e = product<float, T, T>(q, s)) != cudaSuccess) return e;
    }
  }
  return launched("loss_total", [&] {
    return launch_pdl(loss_total_kernel, dim3(1), dim3(kOrderThreads), 0, s,
                      static_cast<const float*>(a.loss), a.weights, l, a.T, a.total);
  });
}

}  // namespace

size_t head_loss_scratch(const LossArgs& a, bool want_dx, bool want_dw) {
  (void)want_dx;
  return Plan(a, want_dw).total;
}

cudaError_t head_loss(const LossArgs& a, void* scratch, cudaStream_t s) {
  char* ws = static_cast<char*>(scratch);
  return a.is_bf16 ? run<bf16>(a, ws, s) : run<float>(a, ws, s);
}

}  // namespace poetx
