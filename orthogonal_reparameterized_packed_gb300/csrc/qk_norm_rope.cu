// RMS norm of every query and key head and the rotary embedding, one pass
// over q and k each way.
//
// For a head row x[0..D) of token t, with r = 1 / sqrt(mean(x^2) + eps) and
// n_i = gamma_i r x_i, the first `rot` features are rotated in pairs (a, b)
//   y_a = n_a c - n_b s,  y_b = n_b c + n_a s,   (c, s) = tables[position][pair]
// and the rest pass through.  Pairs: (i, i + rot/2), or (2i, 2i + 1).
// Backward, with dn the transposed rotation of dy and g_i = gamma_i dn_i:
//   dx_i = r (g_i - x_i r^2 mean_j(g_j x_j)),   dgamma_i = sum over rows dn_i r x_i
// All of it in fp32, rounded once at the store; r is formed again in the
// backward pass (x is read there in any case).
//
// A row is cut into slots of two V-element vectors that hold whole pairs, so
// no lane needs another's elements to rotate; the G lanes of a row share only
// the sums.  What bounds it is memory traffic: 2 (forward) or 3 (backward)
// passes over q and k.
#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "poetx.h"
#include "ptx.cuh"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 512;

template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& o, float x) { o = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }

// Slot s of a row: the vectors at o0 and o1; `turns`: its pairs are rotated,
// with the trigonometric entries [s V, s V + V).
struct Slot {
  int o0, o1;
  bool turns, has0, has1;
};

template <int V>
__device__ __forceinline__ Slot slot_of(int s, int D, int rot, int interleaved) {
  Slot w;
  const int nrot = rot / 2 / V;
  w.turns = s < nrot;
  if (w.turns) {
    w.o0 = interleaved ? 2 * s * V : s * V;
    w.o1 = interleaved ? w.o0 + V : rot / 2 + s * V;
  } else {
    w.o0 = rot + (s - nrot) * 2 * V;
    w.o1 = w.o0 + V;
  }
  w.has0 = w.o0 < D;
  w.has1 = w.o1 < D;
  return w;
}

// (a, b) <- the rotation of the slot's 2 V values; sgn = -1: transposed.
template <int V>
__device__ __forceinline__ void turn(float (&a)[V], float (&b)[V], const float (&c)[V],
                                     const float (&s)[V], bool adjacent, float sgn) {
  if (V == 1 || !adjacent) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float u = a[j], w = b[j], sn = sgn * s[j];
      a[j] = u * c[j] - w * sn;
      b[j] = w * c[j] + u * sn;
    }
  } else {
#pragma unroll
    for (int j = 0; j + 1 < V; j += 2) {
      const float sa = sgn * s[j / 2], sb = sgn * s[V / 2 + j / 2];
      const float ua = a[j], wa = a[j + 1], ub = b[j], wb = b[j + 1];
      a[j] = ua * c[j / 2] - wa * sa;
      a[j + 1] = wa * c[j / 2] + ua * sa;
      b[j] = ub * c[V / 2 + j / 2] - wb * sb;
      b[j + 1] = wb * c[V / 2 + j / 2] + ub * sb;
    }
  }
}

template <int V>
__device__ __forceinline__ void load_f32(float (&o)[V], const float* p) {
  // the tables and weights are fp32 arrays of any 4-byte alignment
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = __ldg(p + j);
}

template <typename T, int V>
__device__ __forceinline__ void load_row(float (&o)[V], const T* p, bool has) {
  if (has) {
    const Pack<T, V> q = *reinterpret_cast<const Pack<T, V>*>(p);
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = to_f(q.x[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 0.f;
  }
}

template <typename T, int V>
__device__ __forceinline__ void store_row(T* p, const float (&v)[V], bool has) {
  if (!has) return;
  Pack<T, V> q;
#pragma unroll
  for (int j = 0; j < V; ++j) from_f(q.x[j], v[j]);
  *reinterpret_cast<Pack<T, V>*>(p) = q;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The table row of token t, or -1 where its position is outside the table.
__device__ __forceinline__ long long table_row(const QkNormRopeArgs& a, long long t) {
  if (a.rot == 0) return 0;
  const long long p = a.positions != nullptr ? a.positions[t] : t;
  return p >= 0 && p < a.table_rows ? p : -1;
}

// One side (q or k) as the kernels see it.
template <typename T>
struct Side {
  const T* x;
  const T* g;
  T* out;
  const float* gamma;
  long long ld_x, ld_g, ld_out;
  int heads;
};

template <typename T>
__device__ __forceinline__ Side<T> side_of(const QkNormRopeArgs& a, bool is_k) {
  Side<T> s;
  s.x = static_cast<const T*>(is_k ? a.k : a.q);
  s.g = static_cast<const T*>(is_k ? a.gk : a.gq);
  s.out = static_cast<T*>(is_k ? a.out_k : a.out_q);
  s.gamma = is_k ? a.gamma_k : a.gamma_q;
  s.ld_x = is_k ? a.ld_k : a.ld_q;
  s.ld_g = is_k ? a.ld_gk : a.ld_gq;
  s.ld_out = is_k ? a.ld_out_k : a.ld_out_q;
  s.heads = is_k ? a.hk : a.hq;
  return s;
}

// One warp per item: 32 / G heads of one side of one token, NS slots per lane.
template <typename T, int V, int G, int NS>
__global__ void __launch_bounds__(kThreads) qk_forward_kernel(const QkNormRopeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int R = 32 / G;  // rows per warp
  const int lane = threadIdx.x % 32, li = lane % G, row = lane / G;
  const int iq = (a.hq + R - 1) / R, ik = (a.hk + R - 1) / R;
  const long long items = a.T * (iq + ik);
  const long long warps = static_cast<long long>(gridDim.x) * kWarps;
  for (long long it = blockIdx.x * static_cast<long long>(kWarps) + threadIdx.x / 32; it < items;
       it += warps) {
    const long long t = it / (iq + ik);
    const int e = static_cast<int>(it % (iq + ik));
    const bool is_k = e >= iq;
    const Side<T> sd = side_of<T>(a, is_k);
    const int head = (is_k ? e - iq : e) * R + row;
    const bool live = head < sd.heads;
    const long long tr = table_row(a, t);
    if (tr < 0 && lane == 0) atomicCAS(a.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
    const T* x = sd.x + t * sd.ld_x + static_cast<long long>(head) * a.D;
    T* out = sd.out + t * sd.ld_out + static_cast<long long>(head) * a.D;
    float v0[NS][V], v1[NS][V];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const Slot w = slot_of<V>(li + G * j, a.D, a.rot, a.interleaved);
      load_row<T, V>(v0[j], x + w.o0, live && w.has0);
      load_row<T, V>(v1[j], x + w.o1, live && w.has1);
#pragma unroll
      for (int i = 0; i < V; ++i) ss = fmaf(v0[j][i], v0[j][i], fmaf(v1[j][i], v1[j][i], ss));
    }
    ss = group_sum<G>(ss);
    const float r = 1.f / sqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int s = li + G * j;
      const Slot w = slot_of<V>(s, a.D, a.rot, a.interleaved);
      if (!w.has0) continue;
      float gm[V];
#pragma unroll
      for (int i = 0; i < V; ++i) v0[j][i] *= r, v1[j][i] *= r;
      if (sd.gamma != nullptr) {
        load_f32<V>(gm, sd.gamma + w.o0);
#pragma unroll
        for (int i = 0; i < V; ++i) v0[j][i] *= gm[i];
        if (w.has1) {
          load_f32<V>(gm, sd.gamma + w.o1);
#pragma unroll
          for (int i = 0; i < V; ++i) v1[j][i] *= gm[i];
        }
      }
      if (w.turns && tr >= 0) {
        float cs[V], sn[V];
        load_f32<V>(cs, a.cos_table + tr * (a.rot / 2) + s * V);
        load_f32<V>(sn, a.sin_table + tr * (a.rot / 2) + s * V);
        turn<V>(v0[j], v1[j], cs, sn, a.interleaved != 0, 1.f);
      }
      if (tr < 0) {
#pragma unroll
        for (int i = 0; i < V; ++i) v0[j][i] = v1[j][i] = 0.f;
      }
      store_row<T, V>(out + w.o0, v0[j], live && w.has0);
      store_row<T, V>(out + w.o1, v1[j], live && w.has1);
    }
  }
}

// As the forward, but a CTA stays with one side (blockIdx.y: 0 q, 1 k) and
// keeps its lanes' sums of dgamma in registers over all its items; they go to
// part[side][CTA][D], added up by qk_dgamma_kernel in a fixed order.
template <typename T, int V, int G, int NS>
__global__ void __launch_bounds__(kThreads) qk_backward_kernel(const QkNormRopeArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int R = 32 / G;
  __shared__ float acc[kMaxD];
  const int lane = threadIdx.x % 32, li = lane % G, row = lane / G;
  const bool is_k = blockIdx.y != 0;
  const Side<T> sd = side_of<T>(a, is_k);
  const int per_token = (sd.heads + R - 1) / R;
  const long long items = a.T * per_token;
  const long long warps = static_cast<long long>(gridDim.x) * kWarps;
  float dg0[NS][V] = {}, dg1[NS][V] = {};
  for (long long it = blockIdx.x * static_cast<long long>(kWarps) + threadIdx.x / 32; it < items;
       it += warps) {
    const long long t = it / per_token;
    const int head = static_cast<int>(it % per_token) * R + row;
    const bool live = head < sd.heads;
    const long long tr = table_row(a, t);
    if (tr < 0 && lane == 0) atomicCAS(a.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
    const T* x = sd.x + t * sd.ld_x + static_cast<long long>(head) * a.D;
    const T* g = sd.g + t * sd.ld_g + static_cast<long long>(head) * a.D;
    T* out = sd.out + t * sd.ld_out + static_cast<long long>(head) * a.D;
    float x0[NS][V], x1[NS][V], g0[NS][V], g1[NS][V];
    float ss = 0.f, gx = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const int s = li + G * j;
      const Slot w = slot_of<V>(s, a.D, a.rot, a.interleaved);
      load_row<T, V>(x0[j], x + w.o0, live && w.has0);
      load_row<T, V>(x1[j], x + w.o1, live && w.has1);
      // a token whose position is outside the table has no gradient
      load_row<T, V>(g0[j], g + w.o0, live && w.has0 && tr >= 0);
      load_row<T, V>(g1[j], g + w.o1, live && w.has1 && tr >= 0);
      if (w.turns && tr >= 0) {
        float cs[V], sn[V];
        load_f32<V>(cs, a.cos_table + tr * (a.rot / 2) + s * V);
        load_f32<V>(sn, a.sin_table + tr * (a.rot / 2) + s * V);
        turn<V>(g0[j], g1[j], cs, sn, a.interleaved != 0, -1.f);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        ss = fmaf(x0[j][i], x0[j][i], fmaf(x1[j][i], x1[j][i], ss));
      }
    }
    ss = group_sum<G>(ss);
    const float r = 1.f / sqrtf(ss / static_cast<float>(a.D) + a.eps);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const Slot w = slot_of<V>(li + G * j, a.D, a.rot, a.interleaved);
      float m0[V], m1[V];
#pragma unroll
      for (int i = 0; i < V; ++i) m0[i] = m1[i] = 1.f;
      if (sd.gamma != nullptr) {
        if (w.has0) load_f32<V>(m0, sd.gamma + w.o0);
        if (w.has1) load_f32<V>(m1, sd.gamma + w.o1);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (tr >= 0) {
          dg0[j][i] = fmaf(g0[j][i], x0[j][i] * r, dg0[j][i]);
          dg1[j][i] = fmaf(g1[j][i], x1[j][i] * r, dg1[j][i]);
        }
        g0[j][i] *= m0[i];
        g1[j][i] *= m1[i];
        gx = fmaf(g0[j][i], x0[j][i], fmaf(g1[j][i], x1[j][i], gx));
      }
    }
    gx = group_sum<G>(gx);
    const float k = r * r * gx / static_cast<float>(a.D);
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      const Slot w = slot_of<V>(li + G * j, a.D, a.rot, a.interleaved);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        g0[j][i] = tr >= 0 ? r * (g0[j][i] - x0[j][i] * k) : 0.f;
        g1[j][i] = tr >= 0 ? r * (g1[j][i] - x1[j][i] * k) : 0.f;
      }
      store_row<T, V>(out + w.o0, g0[j], live && w.has0);
      store_row<T, V>(out + w.o1, g1[j], live && w.has1);
    }
  }
  // the CTA's sum, warp by warp in order (rows of a warp by shuffles)
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int o = 16; o >= G; o >>= 1) {
        dg0[j][i] += __shfl_xor_sync(0xffffffffu, dg0[j][i], o);
        dg1[j][i] += __shfl_xor_sync(0xffffffffu, dg1[j][i], o);
      }
  for (int wp = 0; wp < kWarps; ++wp) {
    if (threadIdx.x / 32 == wp && row == 0) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const Slot w = slot_of<V>(li + G * j, a.D, a.rot, a.interleaved);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (w.has0) acc[w.o0 + i] = (wp == 0 ? 0.f : acc[w.o0 + i]) + dg0[j][i];
          if (w.has1) acc[w.o1 + i] = (wp == 0 ? 0.f : acc[w.o1 + i]) + dg1[j][i];
        }
      }
    }
    __syncthreads();
  }
  float* part = a.part + (static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * a.D;
  for (int i = threadIdx.x; i < a.D; i += kThreads) part[i] = acc[i];
}

// dgamma[i] = sum over the CTAs' partial sums, in order; one warp per feature.
__global__ void __launch_bounds__(kThreads)
    qk_dgamma_kernel(const float* part, int ctas, int D, float* dgamma_q, float* dgamma_k) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x * kWarps + threadIdx.x / 32;
  float* out = blockIdx.y == 0 ? dgamma_q : dgamma_k;
  if (i >= D || out == nullptr) return;
  const float* p = part + static_cast<long long>(blockIdx.y) * ctas * D + i;
  double v = 0.0;
  for (int c = threadIdx.x % 32; c < ctas; c += 32) v += p[static_cast<long long>(c) * D];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (threadIdx.x % 32 == 0) out[i] = static_cast<float>(v);
}

// CTAs of the backward pass per side (fixed by the sizes: the sums' order is
// the same from run to run).
int backward_ctas(int hq, int hk, long long T) {
  const long long rows = T * std::max(hq, hk);
  return static_cast<int>(std::max<long long>(
      1, std::min<long long>(2 * sm_count(), (rows + kWarps - 1) / kWarps)));
}

template <typename T>
cudaError_t forward(const QkNormRopeArgs& a, cudaStream_t s) {
  const long long items = a.T * (a.hq + a.hk);
  const int grid = static_cast<int>(
      std::min<long long>((items + kWarps - 1) / kWarps, 16ll * sm_count()));
  return launch_pdl(qk_forward_kernel<T, 1, 32, kMaxD / 64>, dim3(grid), dim3(kThreads), 0, s, a);
}

template <typename T>
cudaError_t backward(const QkNormRopeArgs& a, int ctas, cudaStream_t s) {
  return launch_pdl(qk_backward_kernel<T, 1, 32, kMaxD / 64>, dim3(ctas, a.hk > 0 ? 2 : 1),
                    dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t qk_norm_rope_forward(const QkNormRopeArgs& a, bool is_bf16, cudaStream_t s) {
  prof_begin("qk_norm_rope", s);
  const cudaError_t e = is_bf16 ? forward<__nv_bfloat16>(a, s) : forward<float>(a, s);
  prof_end("qk_norm_rope", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t qk_norm_rope_scratch(int hq, int hk, int D, long long T) {
  return static_cast<size_t>(backward_ctas(hq, hk, T)) * 2 * D * sizeof(float);
}

cudaError_t qk_norm_rope_backward(const QkNormRopeArgs& a, bool is_bf16, cudaStream_t s) {
  const int ctas = backward_ctas(a.hq, a.hk, a.T);
  prof_begin("qk_norm_rope_bwd", s);
  cudaError_t e =
      is_bf16 ? backward<__nv_bfloat16>(a, ctas, s) : backward<float>(a, ctas, s);
  prof_end("qk_norm_rope_bwd", s);
  if (e != cudaSuccess) return e;
  prof_begin("qk_dgamma", s);
  e = launch_pdl(qk_dgamma_kernel, dim3((a.D + kWarps - 1) / kWarps, a.hk > 0 ? 2 : 1),
                 dim3(kThreads), 0, s, static_cast<const float*>(a.part), ctas, a.D, a.dgamma_q,
                 a.dgamma_k);
  prof_end("qk_dgamma", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace poetx
