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
//
// Squares are added in fp32, at most kChunk / kThreads + 2 at a time; those
// sums, and everything after them, as pairs of fp32 (hi + lo, two-sum), about
// 2^-45 of the total.  (In fp64, which this GPU runs at 1/64 of the rate, the
// closing sums alone took several microseconds per launch.)  Where a sum of
// squares is too large or too small for that it is taken again in fp64 and
// kept apart, so that every finite gradient has a finite and accurate norm.
#include <algorithm>
#include <cstdint>
#include <cstring>

#include "internal.h"
#include "poetx.h"
#include "ptx.cuh"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kChunk = 8192;       // elements
constexpr int kFlight = kChunk / 4 / kThreads;  // a thread's 16-byte vectors of one (fp32)
constexpr int kMaxTensors = 512;   // per launch: the table is at most 24 KB of parameters
constexpr int kFewTensors = 32;
// CTAs per SM.  The norm and the clip have a whole chunk in registers, all its
// loads in flight (336 gradients of 261,120: norm 53.6 us, 6.55 TB/s; 8 CTAs of 32
// registers 60.2; clip 164 against 176); Adam has one vector of each array, and
// every warp that an SM can hold.
constexpr int kSumPerSm = 4, kClipPerSm = 3, kAdamPerSm = 8;
constexpr int kMaxCtas = 2048;     // partial sums per launch
constexpr float kClipEps = 1e-6f;  // guards the division when the norm is 0

// CAP tensors of one launch.  The parameters of a launch cost time by their
// size, so short lists take a small table.
template <int CAP>
struct TensorTable {
  int n;
  unsigned chunks;
  const void* grad[CAP];
  long long count[CAP];
  unsigned first[CAP];  // the tensor's first chunk
  unsigned char bf16[CAP];
};

template <int CAP>
struct ClipTable {
  TensorTable<CAP> t;
  void* out[CAP];
};

template <int CAP>
struct AdamTable {
  TensorTable<CAP> t;
  float* theta[CAP];
  float* m[CAP];
  float* v[CAP];
};

// A sum of squares: hi + lo, and what had to be added in fp64.
struct Sum {
  float hi, lo;
  double wide;
};

// The last tensor whose first chunk is <= c (empty tensors own no chunk).
template <int CAP>
__device__ __forceinline__ int find_tensor(const TensorTable<CAP>& t, unsigned c) {
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

// hi + lo += x, the rounding error of hi + x kept in lo (two-sum).
__device__ __forceinline__ void add_to(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}

// acc += the sum of squares of this thread's share of p[0..n).
template <typename T>
__device__ __forceinline__ void chunk_sumsq(const T* p, int n, Sum& acc) {
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
  constexpr int FLIGHT = kChunk / Vec<T>::N / kThreads;
  Vec<T> q[FLIGHT];
#pragma unroll
  for (int k = 0; k < FLIGHT; ++k) {
    const int i = threadIdx.x + k * kThreads;
    if (i < nv)
      q[k] = pv[i];
    else
      memset(&q[k], 0, sizeof(q[k]));
  }
#pragma unroll
  for (int k = 0; k < FLIGHT; ++k)
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) add(q[k].x[j]);
  const int i0 = threadIdx.x;  // at most 7 elements on either side
  if (i0 < head) add(p[i0]);
  if (tail + i0 < n) add(p[tail + i0]);
  // 2^42 elements are 2^29 chunks: sums of up to 1e28 each stay inside fp32, and
  // squares that fp32 loses (below 1e-38) are nothing beside 1e-24
  if (s >= 1e-24f && s <= 1e28f) {
    add_to(acc.hi, acc.lo, s);
    return;
  }
  if ((any & 0x7fffffffu) == 0) return;
  double d = 0.0;
  auto add_wide = [&](T x) {
    const double f = static_cast<double>(to_f(x));
    d += f * f;
  };
  for (int i = threadIdx.x; i < nv; i += kThreads)
    for (int j = 0; j < Vec<T>::N; ++j) add_wide(p[head + i * Vec<T>::N + j]);
  if (i0 < head) add_wide(p[i0]);
  if (tail + i0 < n) add_wide(p[tail + i0]);
  acc.wide += d;
}

// The CTA's total, the same bits in every thread (it goes by the warps' first
// lanes), in a fixed order.
__device__ __forceinline__ Sum block_sum(Sum v) {
  __shared__ Sum warp_sum[kThreads / 32];
  const bool wide = __syncthreads_or(v.wide != 0.0);  // NaN counts
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float hi = __shfl_xor_sync(0xffffffffu, v.hi, o);
    const float lo = __shfl_xor_sync(0xffffffffu, v.lo, o);
    add_to(v.hi, v.lo, hi);
    v.lo = __fadd_rn(v.lo, lo);
    if (wide) v.wide += __shfl_xor_sync(0xffffffffu, v.wide, o);
  }
  if (threadIdx.x % 32 == 0) warp_sum[threadIdx.x / 32] = v;
  __syncthreads();
  v = warp_sum[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) {
    add_to(v.hi, v.lo, warp_sum[w].hi);
    v.lo = __fadd_rn(v.lo, warp_sum[w].lo);
    if (wide) v.wide += warp_sum[w].wide;
  }
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kSumPerSm)
    sumsq_kernel(const __grid_constant__ TensorTable<CAP> t, Sum* part) {
  pdl_wait();
  pdl_trigger();
  Sum acc = {0.f, 0.f, 0.0};
  for (unsigned c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    const int i = find_tensor(t, c);
    const long long at = static_cast<long long>(c - t.first[i]) * kChunk;
    const int n = static_cast<int>(min(static_cast<long long>(kChunk), t.count[i] - at));
    if (t.bf16[i])
      chunk_sumsq(static_cast<const __nv_bfloat16*>(t.grad[i]) + at, n, acc);
    else
      chunk_sumsq(static_cast<const float*>(t.grad[i]) + at, n, acc);
  }
  acc = block_sum(acc);
  if (threadIdx.x == 0) part[blockIdx.x] = acc;
}

// The norm from the partial sums and min(1, max_norm / (norm + eps)), the same
// bits in every thread of every CTA.  The scale is NaN where the norm is (or
// where both are infinite).
__device__ __forceinline__ float2 norm_and_scale(const Sum* part, int parts, float max_norm) {
  Sum v = {0.f, 0.f, 0.0};
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    const Sum p = part[i];
    add_to(v.hi, v.lo, p.hi);
    v.lo = __fadd_rn(v.lo, p.lo);
    if (p.wide != 0.0) v.wide += p.wide;
  }
  v = block_sum(v);
  float norm, scale;
  if (v.wide != 0.0) {
    const double d = sqrt(v.wide + static_cast<double>(v.hi) + static_cast<double>(v.lo));
    norm = static_cast<float>(d);
    scale = static_cast<float>(static_cast<double>(max_norm) / (d + static_cast<double>(kClipEps)));
  } else {
    norm = sqrtf(v.hi + v.lo);
    scale = max_norm / (norm + kClipEps);
  }
  return make_float2(norm, scale > 1.f ? 1.f : scale);
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const Sum* part, int parts, float* norm) {
  pdl_wait();
  pdl_trigger();
  const float2 v = norm_and_scale(part, parts, 0.f);
  if (threadIdx.x == 0) *norm = v.x;
}

// Chunk r of a clip: where it is, and each thread's vectors of it.
struct ClipChunk {
  const void* p;
  void* o;
  int n, head, nv;  // head elements before the first of nv vectors; no vector: head = n
  bool bf16;
  uint4 vec[kFlight];

  template <int CAP>
  __device__ __forceinline__ ClipChunk(const ClipTable<CAP>& a, unsigned r) {
    const TensorTable<CAP>& t = a.t;
    const int i = find_tensor(t, r);
    const long long at = static_cast<long long>(r - t.first[i]) * kChunk;
    n = static_cast<int>(min(static_cast<long long>(kChunk), t.count[i] - at));
    bf16 = t.bf16[i];
    const int size = bf16 ? 2 : 4, per = 16 / size;
    p = static_cast<const char*>(t.grad[i]) + at * size;
    o = static_cast<char*>(a.out[i]) + at * size;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(p), oa = reinterpret_cast<uintptr_t>(o);
    const int off = static_cast<int>(pa & 15u);
    head = ((pa ^ oa) & 15u) != 0 ? n : off == 0 ? 0 : min(n, (16 - off) / size);
    nv = (n - head) / per;
    const uint4* pv = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + head * size);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int v = threadIdx.x + k * kThreads;
      if (v < nv) vec[k] = pv[v];
    }
  }

  template <typename T>
  __device__ __forceinline__ void scaled(float scale) const {
    const T* g = static_cast<const T*>(p);
    T* out = static_cast<T*>(o);
    auto one = [&](T x) {
      T r;
      from_f(r, to_f(x) * scale);
      return r;
    };
    Vec<T>* ov = reinterpret_cast<Vec<T>*>(out + head);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      const int v = threadIdx.x + k * kThreads;
      if (v >= nv) break;
      Vec<T> q;
      memcpy(&q, &vec[k], 16);
#pragma unroll
      for (int j = 0; j < Vec<T>::N; ++j) q.x[j] = one(q.x[j]);
      ov[v] = q;
    }
    for (int i = threadIdx.x; i < head; i += kThreads) out[i] = one(g[i]);
    for (int i = head + nv * Vec<T>::N + threadIdx.x; i < n; i += kThreads) out[i] = one(g[i]);
  }
};

// Chunks in descending order: the ones that pass one read last are still in
// the 129 MB L2 and are read from there before they are evicted.  The first one's
// loads are on their way while the partial sums are added up.
template <int CAP>
__global__ void __launch_bounds__(kThreads, kClipPerSm)
    clip_kernel(const __grid_constant__ ClipTable<CAP> a, const Sum* part, int parts,
                float max_norm, float* norm) {
  pdl_wait();
  pdl_trigger();
  const unsigned chunks = a.t.chunks;
  float scale = 1.f;
  for (unsigned c = blockIdx.x; c < chunks; c += gridDim.x) {
    const ClipChunk k(a, chunks - 1 - c);
    if (c == blockIdx.x) {
      const float2 ns = norm_and_scale(part, parts, max_norm);
      scale = ns.y;
      if (c == 0 && threadIdx.x == 0) *norm = ns.x;
    }
    if (scale == 1.f && k.p == k.o) continue;  // times one, in place
    if (k.bf16)
      k.template scaled<__nv_bfloat16>(scale);
    else
      k.template scaled<float>(scale);
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

// parts = 0: no clip.  One vector of each array in flight per thread and 64 warps
// per SM: 336 vectors of 261,120 take 375 us, 6.55 TB/s of their 28 bytes per
// parameter (two in flight at 48 warps 429, four at 32 warps 371 but the passes
// over the gradients alone then lose more).
template <int CAP>
__global__ void __launch_bounds__(kThreads)
    adam_many_kernel(const __grid_constant__ AdamTable<CAP> a, const AdamHyper h, const Sum* part,
                     int parts, float max_norm, float* norm) {
  pdl_wait();
  pdl_trigger();
  float scale = 1.f;
  if (parts > 0) {
    const float2 ns = norm_and_scale(part, parts, max_norm);
    scale = ns.y;
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = ns.x;
  }
  const TensorTable<CAP>& t = a.t;
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

// Fills the table from the list's tensors from `at` on, empty ones left out
// (`index` gives their places); returns where the next launch begins.  The
// caller has checked that all counts add up to at most 2^42 (2^29 chunks).
template <int CAP>
int fill_table(TensorTable<CAP>& t, int* index, int at, int n, const void* const* grads,
               const int64_t* counts, const int* dtypes) {
  t.n = 0;
  unsigned long long chunks = 0;
  for (; at < n && t.n < CAP; ++at) {
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
template <int CAP>
cudaError_t sumsq_pass(int n, const void* const* grads, const int64_t* counts, const int* dtypes,
                       Sum* part, int* parts, cudaStream_t s) {
  TensorTable<CAP> t;
  int index[CAP];
  *parts = 0;
  for (int at = 0; at < n;) {
    at = fill_table(t, index, at, n, grads, counts, dtypes);
    if (t.n == 0) continue;
    const int grid = grid_for(t.chunks, kSumPerSm);
    prof_begin("grad_sumsq", s);
    cudaError_t e =
        launch_pdl(sumsq_kernel<CAP>, dim3(grid), dim3(kThreads), 0, s, t, part + *parts);
    prof_end("grad_sumsq", s);
    if (e != cudaSuccess) return e;
    *parts += grid;
  }
  return cudaSuccess;
}

cudaError_t norm_pass(const Sum* part, int parts, float* norm, cudaStream_t s) {
  prof_begin("grad_norm", s);
  const cudaError_t e = launch_pdl(norm_kernel, dim3(1), dim3(kThreads), 0, s, part, parts, norm);
  prof_end("grad_norm", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int CAP>
cudaError_t clip_pass(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                      const int* dtypes, float max_norm, float* norm, Sum* part, cudaStream_t s) {
  int parts = 0;
  cudaError_t e = sumsq_pass<CAP>(n, grads, counts, dtypes, part, &parts, s);
  if (e != cudaSuccess) return e;
  if (parts == 0) return norm_pass(part, 0, norm, s);  // nothing to clip: norm = 0
  ClipTable<CAP> a;
  int index[CAP];
  for (int at = 0; at < n;) {
    at = fill_table(a.t, index, at, n, grads, counts, dtypes);
    if (a.t.n == 0) continue;
    for (int i = 0; i < a.t.n; ++i) a.out[i] = outs[index[i]];
    prof_begin("grad_clip", s);
    e = launch_pdl(clip_kernel<CAP>, dim3(grid_for(a.t.chunks, kClipPerSm)), dim3(kThreads), 0, s,
                   a, static_cast<const Sum*>(part), parts, max_norm, norm);
    prof_end("grad_clip", s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int CAP>
cudaError_t adam_pass(int n, float* const* theta, const void* const* grads, float* const* m,
                      float* const* v, const int64_t* counts, const AdamHyper& h, float max_norm,
                      float* norm, Sum* part, cudaStream_t s) {
  int parts = 0;
  cudaError_t e;
  if (max_norm >= 0.f) {
    e = sumsq_pass<CAP>(n, grads, counts, nullptr, part, &parts, s);
    if (e != cudaSuccess) return e;
    if (parts == 0) return norm_pass(part, 0, norm, s);
  }
  AdamTable<CAP> a;
  int index[CAP];
  for (int at = 0; at < n;) {
    at = fill_table(a.t, index, at, n, grads, counts, nullptr);
    if (a.t.n == 0) continue;
    for (int i = 0; i < a.t.n; ++i) {
      a.theta[i] = theta[index[i]];
      a.m[i] = m[index[i]];
      a.v[i] = v[index[i]];
    }
    prof_begin("adam_many", s);
    e = launch_pdl(adam_many_kernel<CAP>, dim3(grid_for(a.t.chunks, kAdamPerSm)), dim3(kThreads), 0,
                   s, a, h, static_cast<const Sum*>(part), parts, max_norm, norm);
    prof_end("adam_many", s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t grad_norm_scratch(int n) {
  const long long launches = (static_cast<long long>(n) + kMaxTensors - 1) / kMaxTensors;
  return static_cast<size_t>(launches > 0 ? launches : 1) * kMaxCtas * sizeof(Sum);
}

cudaError_t grad_norm(int n, const void* const* grads, const int64_t* counts, const int* dtypes,
                      float* norm, void* scratch, cudaStream_t s) {
  Sum* part = static_cast<Sum*>(scratch);
  int parts = 0;
  const cudaError_t e =
      n <= kFewTensors ? sumsq_pass<kFewTensors>(n, grads, counts, dtypes, part, &parts, s)
                       : sumsq_pass<kMaxTensors>(n, grads, counts, dtypes, part, &parts, s);
  return e != cudaSuccess ? e : norm_pass(part, parts, norm, s);
}

cudaError_t clip_grads(int n, const void* const* grads, void* const* outs, const int64_t* counts,
                       const int* dtypes, float max_norm, float* norm, void* scratch,
                       cudaStream_t s) {
  Sum* part = static_cast<Sum*>(scratch);
  return n <= kFewTensors
             ? clip_pass<kFewTensors>(n, grads, outs, counts, dtypes, max_norm, norm, part, s)
             : clip_pass<kMaxTensors>(n, grads, outs, counts, dtypes, max_norm, norm, part, s);
}

cudaError_t adam_update_many(int n, float* const* theta, const float* const* grads,
                             float* const* m, float* const* v, const int64_t* counts,
                             const AdamHyper& h, float max_norm, float* norm, void* scratch,
                             cudaStream_t s) {
  const void* const* gr = reinterpret_cast<const void* const*>(grads);
  Sum* part = static_cast<Sum*>(scratch);
  return n <= kFewTensors
             ? adam_pass<kFewTensors>(n, theta, gr, m, v, counts, h, max_norm, norm, part, s)
             : adam_pass<kMaxTensors>(n, theta, gr, m, v, counts, h, max_norm, norm, part, s);
}

}  // namespace poetx
