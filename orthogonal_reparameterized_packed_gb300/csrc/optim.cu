// The end of a training step over many tensors: the global gradient norm,
// the clipped gradients, and Adam with the clip applied as it reads them.
//
//   norm  = sqrt(sum over all tensors of g^2)
//   scale = min(1, max_norm / (norm + 1e-6))
//   clip: out = scale g;  Adam: poetx_adam_update's step on scale g
//
// Every tensor is cut into chunks of at most kChunk elements; chunk c of the
// whole list is found by a binary search over the tensors' first chunks, so
// lists of any sizes spread evenly over the grid.  The lists travel in the
// kernel parameters: no table in device memory, nothing kept between calls.
//
// Pass one leaves one partial sum per CTA in the workspace.  The pass that
// needs the norm adds the partials itself, in every CTA and in the same order
// (no atomics, no counter to reset, the same bits in every CTA), so a clip
// is two launches.  All of it is bound by memory traffic.
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "poetx.h"
#include "ptx.cuh"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;       // elements: 8 16-byte loads in flight per thread (fp32)
constexpr int kMaxTensors = 512;   // per launch: the table is at most 24 KB of parameters
constexpr int kMaxCtas = 1024;     // partial sums per launch
constexpr float kClipEps = 1e-6f;  // guards the division when the norm is 0

struct TensorTable {
  int n;
  unsigned chunks;
  const void* grad[kMaxTensors];
  long long count[kMaxTensors];
  unsigned first[kMaxTensors];  // the tensor's first chunk
  unsigned char bf16[kMaxTensors];
};

struct ClipTable {
  TensorTable t;
  void* out[kMaxTensors];
};

struct AdamTable {
  TensorTable t;
  float* theta[kMaxTensors];
  float* m[kMaxTensors];
  float* v[kMaxTensors];
};

// The last tensor whose first chunk is <= c (empty tensors own no chunk).
__device__ __forceinline__ int find_tensor(const TensorTable& t, unsigned c) {
  int lo = 0, hi = t.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (t.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& o, float x) { o = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }

template <typename T>
struct alignas(16) Vec {
  static constexpr int N = 16 / sizeof(T);
  T x[N];
};

// Elements of p before its first 16-byte boundary, at most n.
template <typename T>
__device__ __forceinline__ int head_elements(const T* p, int n) {
  const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15u);
  return off == 0 ? 0 : min(n, static_cast<int>((16 - off) / sizeof(T)));
}

// Sum of squares of this thread's share of p[0..n).  The squares are added in
// fp32 (at most kChunk / kThreads + 2 of them, so the sum keeps about 2^-22
// of its value); sums that overflowed fp32, or are so small that squares may
// have been lost below its range, are taken again in 64 bits, so every finite
// gradient has a finite and accurate norm.
template <typename T>
__device__ __forceinline__ double chunk_sumsq(const T* p, int n) {
  const int head = head_elements(p, n);
  const int nv = (n - head) / Vec<T>::N;
  const int tail = head + nv * Vec<T>::N;
  const Vec<T>* pv = reinterpret_cast<const Vec<T>*>(p + head);
  float s = 0.f;
  unsigned any = 0;
  auto add = [&](T x) {
    const float f = to_f(x);
    s = fmaf(f, f, s);
    any |= __float_as_uint(f);
  };
#pragma unroll 8
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    const Vec<T> q = pv[i];
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) add(q.x[j]);
  }
  const int i0 = threadIdx.x;  // at most 7 elements on either side
  if (i0 < head) add(p[i0]);
  if (tail + i0 < n) add(p[tail + i0]);
  if (s >= 1e-24f && s <= 3e38f) return static_cast<double>(s);
  if ((any & 0x7fffffffu) == 0) return 0.0;
  double d = 0.0;
  for (int i = threadIdx.x; i < nv; i += kThreads)
    for (int j = 0; j < Vec<T>::N; ++j) {
      const double f = static_cast<double>(to_f(p[head + i * Vec<T>::N + j]));
      d += f * f;
    }
  if (i0 < head) d += static_cast<double>(to_f(p[i0])) * static_cast<double>(to_f(p[i0]));
  if (tail + i0 < n)
    d += static_cast<double>(to_f(p[tail + i0])) * static_cast<double>(to_f(p[tail + i0]));
  return d;
}

// Sum over the CTA, the same value in every thread, in a fixed order.
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warp_sum[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = v;
  __syncthreads();
  v = warp_sum[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) v += warp_sum[w];
  return v;
}

__global__ void __launch_bounds__(kThreads)
    sumsq_kernel(const __grid_constant__ TensorTable t, double* part) {
  pdl_wait();
  pdl_trigger();
  double acc = 0.0;
  for (unsigned c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const long long at = static_cast<long long>(c - t.first[i]) * kChunk;
    const int n = static_cast<int>(min(static_cast<long long>(kChunk), t.count[i] - at));
    acc += t.bf16[i] ? chunk_sumsq(static_cast<const __nv_bfloat16*>(t.grad[i]) + at, n)
                     : chunk_sumsq(static_cast<const float*>(t.grad[i]) + at, n);
  }
  acc = block_sum(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// The norm from the partial sums, the same bits in every CTA.
__device__ __forceinline__ double norm_of(const double* part, int parts) {
  double v = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) v += part[i];
  return sqrt(block_sum(v));
}

// min(1, max_norm / (norm + eps)); NaN where the norm is NaN (or inf over inf).
__device__ __forceinline__ float clip_scale(double norm, float max_norm) {
  const double s = static_cast<double>(max_norm) / (norm + static_cast<double>(kClipEps));
  return s > 1.0 ? 1.f : static_cast<float>(s);
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* part, int parts, float* norm) {
  pdl_wait();
  pdl_trigger();
  const double v = norm_of(part, parts);
  if (threadIdx.x == 0) *norm = static_cast<float>(v);
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* p, T* o, int n, float scale) {
  auto one = [&](T x) {
    T r;
    from_f(r, to_f(x) * scale);
    return r;
  };
  const bool same_phase =
      ((reinterpret_cast<uintptr_t>(p) ^ reinterpret_cast<uintptr_t>(o)) & 15u) == 0;
  const int head = same_phase ? head_elements(p, n) : n;
  const int nv = (n - head) / Vec<T>::N;
  const int tail = head + nv * Vec<T>::N;
  const Vec<T>* pv = reinterpret_cast<const Vec<T>*>(p + head);
  Vec<T>* ov = reinterpret_cast<Vec<T>*>(o + head);
#pragma unroll 4
  for (int i = threadIdx.x; i < nv; i += kThreads) {
    Vec<T> q = pv[i];
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) q.x[j] = one(q.x[j]);
    ov[i] = q;
  }
  for (int i = threadIdx.x; i < head; i += kThreads) o[i] = one(p[i]);
  for (int i = tail + threadIdx.x; i < n; i += kThreads) o[i] = one(p[i]);
}

// Chunks in descending order: the ones that pass one read last are still in
// the 129 MB L2 and are read from there before they are evicted.
__global__ void __launch_bounds__(kThreads)
    clip_kernel(const __grid_constant__ ClipTable a, const double* part, int parts, float max_norm,
                float* norm) {
  pdl_wait();
  pdl_trigger();
  const double nv = norm_of(part, parts);
  const float scale = clip_scale(nv, max_norm);
  if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(nv);
  const TensorTable& t = a.t;
  for (unsigned c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const unsigned r = t.chunks - 1 - c;
    const int i = find_tensor(t, r);
    const long long at = static_cast<long long>(r - t.first[i]) * kChunk;
    const int n = static_cast<int>(min(static_cast<long long>(kChunk), t.count[i] - at));
    if (scale == 1.f && t.grad[i] == a.out[i]) continue;  // times one, in place
    if (t.bf16[i])
      scale_chunk(static_cast<const __nv_bfloat16*>(t.grad[i]) + at,
                  static_cast<__nv_bfloat16*>(a.out[i]) + at, n, scale);
    else
      scale_chunk(static_cast<const float*>(t.grad[i]) + at, static_cast<float*>(a.out[i]) + at, n,
                  scale);
  }
}

// poetx_adam_update's step on scale * g, the roundings written out so that an
// element's result does not depend on the loop (vector or scalar) it is met in.
__device__ __forceinline__ void adam_one(float& th, float g, float& m, float& v,
                                         const AdamHyper& h, float scale) {
  g = __fmul_rn(g, scale);
  m = fmaf(h.beta1, m, __fmul_rn(1.f - h.beta1, g));
  v = fmaf(h.beta2, v, __fmul_rn(__fmul_rn(1.f - h.beta2, g), g));
  const float step = (m / h.bc1) / (sqrtf(v / h.bc2) + h.eps);
  th = fmaf(-h.lr, fmaf(h.wd, th, step), th);
}

// parts = 0: no clip.
__global__ void __launch_bounds__(kThreads)
    adam_many_kernel(const __grid_constant__ AdamTable a, const AdamHyper h, const double* part,
                     int parts, float max_norm, float* norm) {
  pdl_wait();
  pdl_trigger();
  float scale = 1.f;
  if (parts > 0) {
    const double nv = norm_of(part, parts);
    scale = clip_scale(nv, max_norm);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = static_cast<float>(nv);
  }
  const TensorTable& t = a.t;
  for (unsigned c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const unsigned r = t.chunks - 1 - c;  // as in clip_kernel
    const int i = find_tensor(t, r);
    const long long at = static_cast<long long>(r - t.first[i]) * kChunk;
    const int n = static_cast<int>(min(static_cast<long long>(kChunk), t.count[i] - at));
    const float* g = static_cast<const float*>(t.grad[i]) + at;
    float* th = a.theta[i] + at;
    float* m = a.m[i] + at;
    float* v = a.v[i] + at;
    const uintptr_t gp = reinterpret_cast<uintptr_t>(g);
    const bool same_phase = (((gp ^ reinterpret_cast<uintptr_t>(th)) |
                              (gp ^ reinterpret_cast<uintptr_t>(m)) |
                              (gp ^ reinterpret_cast<uintptr_t>(v))) &
                             15u) == 0;
    const int head = same_phase ? head_elements(g, n) : n;
    const int n4 = (n - head) / 4;
#pragma unroll 2
    for (int j = threadIdx.x; j < n4; j += kThreads) {
      const float4 gj = reinterpret_cast<const float4*>(g + head)[j];
      float4 tj = reinterpret_cast<float4*>(th + head)[j];
      float4 mj = reinterpret_cast<float4*>(m + head)[j];
      float4 vj = reinterpret_cast<float4*>(v + head)[j];
      adam_one(tj.x, gj.x, mj.x, vj.x, h, scale);
      adam_one(tj.y, gj.y, mj.y, vj.y, h, scale);
      adam_one(tj.z, gj.z, mj.z, vj.z, h, scale);
      adam_one(tj.w, gj.w, mj.w, vj.w, h, scale);
      reinterpret_cast<float4*>(th + head)[j] = tj;
      reinterpret_cast<float4*>(m + head)[j] = mj;
      reinterpret_cast<float4*>(v + head)[j] = vj;
    }
    for (int j = threadIdx.x; j < head; j += kThreads) adam_one(th[j], g[j], m[j], v[j], h, scale);
    for (int j = head + 4 * n4 + threadIdx.x; j < n; j += kThreads)
      adam_one(th[j], g[j], m[j], v[j], h, scale);
  }
}

// Fills the table from tensors [at, at + kMaxTensors) of the list, empty ones
// left out (`index` gives their places); returns where the next launch begins.
// The caller has checked that all counts add up to at most 2^42 (2^29 chunks).
int fill_table(TensorTable& t, int* index, int at, int n, const void* const* grads,
               const int64_t* counts, const int* dtypes) {
  t.n = 0;
  unsigned long long chunks = 0;
  for (; at < n && t.n < kMaxTensors; ++at) {
    if (counts[at] == 0) continue;
    t.grad[t.n] = grads[at];
    t.count[t.n] = counts[at];
    t.first[t.n] = static_cast<unsigned>(chunks);
    t.bf16[t.n] = dtypes != nullptr && dtypes[at] == POETX_BF16;
    index[t.n++] = at;
    chunks += (static_cast<unsigned long long>(counts[at]) + kChunk - 1) / kChunk;
  }
  t.chunks = static_cast<unsigned>(chunks);
  return at;
}

int grid_for(unsigned chunks, int per_sm) {
  const int most = std::min(kMaxCtas, per_sm * sm_count());
  return static_cast<int>(std::min<unsigned>(chunks, static_cast<unsigned>(most)));
}

// Pass one over the whole list; returns the number of partial sums.
cudaError_t sumsq_pass(int n, const void* const* grads, const int64_t* counts, const int* dtypes,
                       double* part, int* parts, cudaStream_t s) {
  TensorTable t;
  int index[kMaxTensors];
  *parts = 0;
  for (int at = 0; at < n;) {
    at = fill_table(t, index, at, n, grads, counts, dtypes);
    if (t.n == 0) continue;
    const int grid = grid_for(t.chunks, 6);
    prof_begin("grad_sumsq", s);
    cudaError_t e = launch_pdl(sumsq_kernel, dim3(grid), dim3(kThreads), 0, s, t, part + *parts);
    prof_end("grad_sumsq", s);
    if (e != cudaSuccess) return e;
    *parts += grid;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_norm_scratch(int n) {
  const long long launches = (static_cast<long long>(n) + kMaxTensors - 1) / kMaxTensors;
  return static_cast<size_t>(launches > 0 ? launches : 1) * kMaxCtas * sizeof(double);
}

cudaError_t grad_norm(int n, const void* const* grads, const int64_t* counts, const int* dtypes,
                      float* norm, void* scratch, cudaStream_t s) {
  double* part = static_cast<double*>(scratch);
  int parts = 0;
  cudaError_t e = sumsq_pass(n, grads, counts, dtypes, part, &parts, s);
  if (e != cudaSuccess) return e;
  prof_begin("grad_norm", s);
  e = launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(part),
                 parts, norm);
  prof_end("grad_norm", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t clip_grads(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                       const int* dtypes, float max_norm, float* norm, void* scratch,
                       cudaStream_t s) {
  double* part = static_cast<double*>(scratch);
  int parts = 0;
  cudaError_t e = sumsq_pass(n, grads, counts, dtypes, part, &parts, s);
  if (e != cudaSuccess) return e;
  if (parts == 0) return grad_norm(0, grads, counts, dtypes, norm, scratch, s);  // norm = 0
  ClipTable a;
  int index[kMaxTensors];
  for (int at = 0; at < n;) {
    at = fill_table(a.t, index, at, n, grads, counts, dtypes);
    if (a.t.n == 0) continue;
    for (int i = 0; i < a.t.n; ++i) a.out[i] = outs[index[i]];
    prof_begin("grad_clip", s);
    e = launch_pdl(clip_kernel, dim3(grid_for(a.t.chunks, 6)), dim3(kThreads), 0, s, a,
                   static_cast<const double*>(part), parts, max_norm, norm);
    prof_end("grad_clip", s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t adam_update_many(int n, float* const* theta, const float* const* grads,
                             float* const* m, float* const* v, const int64_t* counts,
                             const AdamHyper& h, float max_norm, float* norm, void* scratch,
                             cudaStream_t s) {
  const void* const* gr = reinterpret_cast<const void* const*>(grads);
  double* part = static_cast<double*>(scratch);
  int parts = 0;
  cudaError_t e;
  if (max_norm >= 0.f) {
    e = sumsq_pass(n, gr, counts, nullptr, part, &parts, s);
    if (e != cudaSuccess) return e;
    if (parts == 0) return grad_norm(0, gr, counts, nullptr, norm, scratch, s);
  }
  AdamTable a;
  int index[kMaxTensors];
  for (int at = 0; at < n;) {
    at = fill_table(a.t, index, at, n, gr, counts, nullptr);
    if (a.t.n == 0) continue;
    for (int i = 0; i < a.t.n; ++i) {
      a.theta[i] = theta[index[i]];
      a.m[i] = m[index[i]];
      a.v[i] = v[index[i]];
    }
    prof_begin("adam_many", s);
    e = launch_pdl(adam_many_kernel, dim3(grid_for(a.t.chunks, 6)), dim3(kThreads), 0, s, a, h,
                   static_cast<const double*>(part), parts, max_norm, norm);
    prof_end("adam_many", s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace poetx
