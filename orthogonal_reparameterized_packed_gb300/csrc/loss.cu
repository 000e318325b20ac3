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
#include <climits>
#include <cstdint>

#include "internal.h"
#include "linear.h"
#include "linear_planes.cuh"
#include "loss.h"
#include "poetx.h"
#include "ptx.cuh"

namespace poetx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kOrderThreads = 1024;
constexpr int kOrderDeep = 8;  // tokens of a thread in flight

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

// Entries (index, p) of a warp in ascending order of the index; n a power of two,
// entries from `top` on are INT_MAX.
__device__ __forceinline__ void sort_entries(int* key, float* val, int n, int lane) {
  for (int size = 2; size <= n; size *= 2)
    for (int stride = size / 2; stride > 0; stride /= 2) {
      for (int i = lane; i < n / 2; i += 32) {
        const int a = 2 * i - (i & (stride - 1)), b = a + stride;
        const bool up = (a & size) == 0;
        const int ka = key[a], kb = key[b];
        if (up ? ka > kb : ka < kb) {
          const float va = val[a], vb = val[b];
          key[a] = kb, key[b] = ka;
          val[a] = vb, val[b] = va;
        }
      }
      __syncwarp();
    }
}

constexpr int kEntryWarps = 4;
constexpr int kMostEntries = 1024;

// The entries of a token, a warp each: p = softmax of the teacher's logits at tau
// over the entries that are there, sorted by their indices; those of one index become
// one, behind the places that hold none.  Differences are divided by tau, not the
// logits: the type's lowest value stays finite.
__global__ void __launch_bounds__(32 * kEntryWarps)
    loss_entries_kernel(const void* indices, int index_bytes, const void* logits, bool logits_bf16,
                        long long T, int top, int V, float inv_tau, LossRows l, int* status) {
  __shared__ int keys[kEntryWarps][kMostEntries];
  __shared__ float vals[kEntryWarps][kMostEntries];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long t = blockIdx.x * static_cast<long long>(kEntryWarps) + warp;
  if (t >= T) return;
  const long long base = t * top;
  int* key = keys[warp];
  float* val = vals[warp];
  int padded = 1;
  while (padded < top) padded *= 2;
  bool outside = false, any = false;
  float m = -INFINITY;
  for (int k = lane; k < padded; k += 32) {
    int at = INT_MAX;
    float v = 0.f;
    if (k < top) {
      const long long i = index_at(indices, index_bytes, base + k);
      v = logits_bf16 ? to_f(static_cast<const bf16*>(logits)[base + k])
                      : static_cast<const float*>(logits)[base + k];
      outside |= i >= V;
      const bool there = i >= 0 && i < V && !(v == -INFINITY);
      at = there ? static_cast<int>(i) : -1;
      any |= there;
      if (there) m = fmaxf(m, v);
    }
    key[k] = at;
    val[k] = v;
  }
  m = warp_max(m);
  any = __any_sync(0xffffffffu, any);
  outside = __any_sync(0xffffffffu, outside);
  float sum = 0.f;
  for (int k = lane; k < top; k += 32)
    if (key[k] >= 0) sum += expf((val[k] - m) * inv_tau);
  const float log_sum = logf(warp_sum(sum));
  float ent = 0.f, best = -1.f;
  int lead = INT_MAX;
  for (int k = lane; k < top; k += 32) {
    float p = 0.f;
    if (key[k] >= 0) {
      const float log_p = (val[k] - m) * inv_tau - log_sum;
      p = expf(log_p);
      if (!(p == 0.f)) ent += p * log_p;
      if (!(p <= best)) best = p, lead = key[k];
    }
    val[k] = p;
  }
  ent = warp_sum(ent);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {  // the largest p, of equal ones the lowest index
    const float other = __shfl_xor_sync(0xffffffffu, best, o);
    const int at = __shfl_xor_sync(0xffffffffu, lead, o);
    if (other > best || (other == best && at < lead)) best = other, lead = at;
  }
  __syncwarp();
  sort_entries(key, val, padded, lane);
  // the first of an index, with the sum of its p
  const auto first_of = [&](int k) {
    return k < top && key[k] >= 0 && (k == 0 || key[k - 1] != key[k]);
  };
  int heads = 0;
  for (int k = lane; k < padded; k += 32) heads += first_of(k);
  int to = top - __reduce_add_sync(0xffffffffu, heads);
  for (int k = lane; k < to; k += 32) {
    l.index[base + k] = -1;
    l.p[base + k] = 0.f;
  }
  for (int k0 = 0; k0 < top; k0 += 32) {
    const int k = k0 + lane;
    const bool head = first_of(k);
    const unsigned mask = __ballot_sync(0xffffffffu, head);
    if (head) {
      float all = val[k];
      for (int q = k + 1; q < top && key[q] == key[k]; ++q) all += val[q];
      const long long at = base + to + __popc(mask & ((1u << lane) - 1));
      l.index[at] = key[k];
      l.p[at] = all;
    }
    to += __popc(mask);
  }
  if (lane == 0) {
    l.pos[t] = any ? 0 : -1;
    l.ent[t] = ent;
    l.lead[t] = lead < V ? lead : 0;
    if (outside) atomicCAS(status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
  }
}

// pos[t] (0 or -1) -> the number of tokens before t that count, or -1; token its
// inverse; the largest weight; the blocks' flags and the counter of finished CTAs
// cleared.  For the cross entropy also the entries: the targets.  One CTA,
// kOrderThreads * kOrderDeep tokens at a time.
__global__ void __launch_bounds__(kOrderThreads)
    loss_order_kernel(LossRows l, long long T, const float* __restrict__ weights, int blocks,
                      const void* targets, int index_bytes, int V, int* status) {
  __shared__ int sums[kOrderDeep][32];
  __shared__ float largest[32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  int before = 0;
  float most = 0.f;
  bool outside = false;
  for (long long t0 = 0; t0 < T; t0 += kOrderThreads * kOrderDeep) {
    bool on[kOrderDeep];
    unsigned mask[kOrderDeep];
    long long at[kOrderDeep];
#pragma unroll
    for (int i = 0; i < kOrderDeep; ++i) {
      const long long t = t0 + i * kOrderThreads + threadIdx.x;
      at[i] = t >= T ? -1 : targets != nullptr ? index_at(targets, index_bytes, t) : l.pos[t];
    }
#pragma unroll
    for (int i = 0; i < kOrderDeep; ++i) {
      const long long t = t0 + i * kOrderThreads + threadIdx.x;
      on[i] = at[i] >= 0;
      if (targets != nullptr) {
        outside |= at[i] >= V;
        on[i] &= at[i] < V;
        if (t < T) {
          l.index[t] = l.lead[t] = on[i] ? static_cast<int>(at[i]) : -1;
          l.p[t] = 1.f;
          l.ent[t] = 0.f;
        }
      }
      mask[i] = __ballot_sync(0xffffffffu, on[i]);
      if (lane == 0) sums[i][warp] = __popc(mask[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kOrderDeep; ++i) {
      if (t0 + i * kOrderThreads >= T) break;
      const long long t = t0 + i * kOrderThreads + threadIdx.x;
      const int of_warp = sums[i][lane];
      const int all = __reduce_add_sync(0xffffffffu, of_warp);
      const int mine = before + __reduce_add_sync(0xffffffffu, lane < warp ? of_warp : 0) +
                       __popc(mask[i] & ((1u << lane) - 1));
      if (t < T) l.pos[t] = on[i] ? mine : -1;
      if (on[i]) {
        l.token[mine] = static_cast<int>(t);
        if (weights != nullptr) most = fmaxf(most, fabsf(weights[t]));
      }
      before += all;
    }
    __syncthreads();
  }
  for (int b = threadIdx.x; b < blocks; b += kOrderThreads) l.again[b] = 0;
  most = warp_max(most);
  if (lane == 0) largest[warp] = most;
  outside = __syncthreads_or(outside);
  if (threadIdx.x == 0) {
    for (int w = 0; w < 32; ++w) most = fmaxf(most, largest[w]);
    *l.count = before;
    *l.done = 0;
    *l.most = weights == nullptr ? 1.f / static_cast<float>(max(1, before))
              : most > 0.f       ? most
                                 : 1.f;
    if (outside) atomicCAS(status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
  }
}

// How far above its lead entry's exponent a row's reference lies, and the largest
// logit's exponent that may lie above the reference (below it: never by more than
// kAbove but for rounding), in powers of 2.  The terms are then between 2^-126 and
// 2^44: no sum or product of V of them leaves fp32's or bf16's range, and the
// largest is at least 2^-28.  A token whose loss is above (28 + 44) log 2 = 50 does
// not fit; its block is taken again with the largest logit as the reference.
constexpr float kAbove = 28.f, kFits = 44.f;

// V consecutive values.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

// What loss_gather_kernel does in loss_order_kernel's place for up to kStartTokens.
struct StartArgs {
  const void* targets;  // null: distillation, pos is 0 or -1
  int index_bytes, V, blocks;
  const float* weights;
  int* status;
};

constexpr long long kStartTokens = 2048;

// A warp per token: the tokens that count to their rows, zeros to dx and loss of
// the others; warps from T on: zeros to the rows behind the last, to all of them or
// up to a multiple of 64.  unit: log2(e) / tau where references are wanted, else 0.
// V values (16 bytes) at a time.  START: up to kStartTokens tokens every CTA counts
// those before its own, which saves the launch that orders them but costs by the square
// of the tokens.  Counted here / ordered by a launch, us: losses of 256 -> 1000 with 128
// tokens 15.7 / 17.6, 1024 17.3 / 18.5, 2048 20.5 / 20.7; of 1024 -> 4000 with 1024 22.6 /
// 24.4, 2048 29.7 / 29.5, with gradients 71.6 / 72.3.  4096 tokens of both would take 28.9 /
// 27.0 and 42.1 / 40.3, 8192 47.4 / 38.8 and 72.0 / 63.4.
template <typename TX, int V, bool START>
__global__ void __launch_bounds__(kThreads)
    loss_gather_kernel(const TX* __restrict__ x, const TX* __restrict__ W, LossRows l, long long T,
                       int d, TX* __restrict__ xg, long long ldx, bool zero_all, float unit,
                       float* __restrict__ loss, TX* __restrict__ dx, const StartArgs start) {
  using P = Pack<TX, V>;
  __shared__ int counts[2][kThreads / 32];
  __shared__ float largest[kThreads / 32];
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long t0 = blockIdx.x * static_cast<long long>(kThreads / 32), t = t0 + warp;
  long long n, at = -1, lead = 0;
  if (START) {
    const auto index_of = [&](long long i) {  // -1: does not count
      if (start.targets == nullptr) return static_cast<long long>(l.pos[i]);
      const long long v = index_at(start.targets, start.index_bytes, i);
      return v < start.V ? v : -1ll;
    };
    int before = 0, all = 0;
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kStartTokens / kThreads; ++i) {
      const long long u = i * kThreads + threadIdx.x;
      if (u >= T || index_of(u) < 0) continue;
      ++all;
      before += u < t0;
      if (blockIdx.x == 0 && start.weights != nullptr)
        most = fmaxf(most, fabsf(start.weights[u]));
    }
    all = __reduce_add_sync(0xffffffffu, all);
    before = __reduce_add_sync(0xffffffffu, before);
    most = warp_max(most);
    if (lane == 0) counts[0][warp] = all, counts[1][warp] = before, largest[warp] = most;
    __syncthreads();
    all = before = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      all += counts[0][w];
      before += counts[1][w];
      most = fmaxf(most, largest[w]);
    }
    n = all;
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i < start.blocks; i += kThreads) l.again[i] = 0;
      if (threadIdx.x == 0) {
        *l.count = all;
        *l.done = 0;
        *l.most = start.weights == nullptr ? 1.f / static_cast<float>(max(1, all))
                  : most > 0.f             ? most
                                           : 1.f;
      }
    }
    // the tokens of this CTA before the warp's
    const long long first = t0 + lane < T && lane < warp ? index_of(t0 + lane) : -1;
    const long long own = t < T ? index_of(t) : -1;
    before += __popc(__ballot_sync(0xffffffffu, first >= 0));
    if (own >= 0) at = before;
    if (t < T && lane == 0 && start.targets != nullptr) {
      l.index[t] = own >= 0 ? static_cast<int>(own) : -1;
      l.p[t] = 1.f;
      l.ent[t] = 0.f;
      if (index_at(start.targets, start.index_bytes, t) >= start.V)
        atomicCAS(start.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
    }
    if (own >= 0 && lane == 0) l.token[at] = static_cast<int>(t);
    lead = start.targets != nullptr ? own : own >= 0 ? l.lead[t] : 0;
  } else {
    n = *l.count;
    if (t < T) {
      at = l.pos[t];
      lead = l.lead[t];
    }
  }
  const auto at_row = [&](auto* base, long long row, long long ld, int c) {
    return base + row * ld + c;
  };
  P zero;
#pragma unroll
  for (int j = 0; j < V; ++j) from_f(zero.x[j], 0.f);
  if (t >= T) {
    const long long r = t - T;
    if (r >= n && r < (zero_all ? T : (n + 63) / 64 * 64))
      for (int c = lane * V; c < d; c += 32 * V)
        *reinterpret_cast<P*>(at_row(xg, r, ldx, c)) = zero;
    return;
  }
  if (at >= 0) {
    float dot = 0.f;
#pragma unroll 4
    for (int c = lane * V; c < d; c += 32 * V) {
      const P v = *reinterpret_cast<const P*>(at_row(x, t, d, c));
      *reinterpret_cast<P*>(at_row(xg, at, ldx, c)) = v;
      if (unit > 0.f) {
        const P w = *reinterpret_cast<const P*>(at_row(W, lead, d, c));
#pragma unroll
        for (int j = 0; j < V; ++j) dot = fmaf(to_f(v.x[j]), to_f(w.x[j]), dot);
      }
    }
    if (unit > 0.f) {
      dot = warp_sum(dot);
      if (lane == 0) l.ref[at] = fmaf(dot, unit, kAbove);
    }
    return;
  }
  if (lane == 0) loss[t] = 0.f;
  if (dx != nullptr)
    for (int c = lane * V; c < d; c += 32 * V) *reinterpret_cast<P*>(at_row(dx, t, d, c)) = zero;
}

// What becomes of a block's statistics.
struct FinishArgs {
  LossRows rows;
  const float2* part;
  long long ldp, first, block;
  int parts, top, d;
  float unit, tau;
  const float* weights;
  float* loss;
  bf16* E;  // null: no gradients
  long long lde;
  bf16* x;  // the block's rows; null: no dW
  long long ldx;
  bool second, last;  // last: of the call; total is taken behind it
  bool direct;        // the rows are the tokens, also those that do not count,
  const void* targets;  // and (not null) the entries are the targets, not looked over yet
  int target_bytes, V;
  int* status;
  long long T;
  float* total;
};

// total, from the parts (w loss of some rows, in 64 bits, in order) divided by `by`,
// by one CTA.
template <int THREADS>
__device__ void sum_total(const LossRows& l, long long count, float by, float* total) {
  __shared__ double sums[THREADS / 32];
  double sum = 0.0;
#pragma unroll 4
  for (long long i = threadIdx.x; i < count; i += THREADS) sum += __ldcg(l.totals + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (threadIdx.x % 32 == 0) sums[threadIdx.x / 32] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    sum = 0.0;
    for (int w = 0; w < THREADS / 32; ++w) sum += sums[w];
    *total = static_cast<float>(sum / by);
  }
}

// The same where this kernel wrote the parts, every CTA's by its thread 0: the CTA
// that comes last adds them up.
template <int THREADS>
__device__ void total_behind(const LossRows& l, long long count, float by, float* total) {
  __shared__ bool mine;
  if (threadIdx.x == 0) {
    __threadfence();
    mine = atomicAdd(l.done, 1) == static_cast<int>(gridDim.x) - 1;
  }
  __syncthreads();
  if (!mine) return;
  __threadfence();
  sum_total<THREADS>(l, count, by, total);
}

constexpr int kFinishRows = 4;  // 32-byte sectors of the parts

// kFinishRows rows per CTA.  The parts of their sums (all threads), then a warp per row:
// its loss, its factor, and in E the entries' terms e - p sum.  A row whose reference
// does not fit sets its block's flag.  The second pass does this again where the flag is
// set, and scales the rows of x for dW.
__device__ __forceinline__ void finish_rows(const FinishArgs& a) {
  constexpr int R = kFinishRows;
  __shared__ float2 sums[kThreads / 32][R];
  __shared__ double totals[R];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int count = a.direct ? 0 : *a.rows.count;
  const long long n = max(0ll, min(a.block, (a.direct ? a.T : count) - a.first));
  const long long r0 = blockIdx.x * static_cast<long long>(R);
  if (r0 >= n) return;
  int* again = a.rows.again + a.first / a.block;
  const bool own = a.E == nullptr;  // every part has its own reference
  const long long row = r0 + warp, r = a.first + row;  // of the first R warps
  const bool on = warp < R && row < n;
  if (!a.second || *again != 0) {
    // what the row needs besides its statistics, first
    long long t = 0, base = 0;
    bool counts = false;
    float weight = 0.f, ent = 0.f, ref = 0.f, p0 = 0.f, z0 = 0.f;
    int i0 = -1;
    if (on) {
      t = a.direct ? r : a.rows.token[r];
      base = t * a.top;
      if (a.targets != nullptr) {
        const long long i = index_at(a.targets, a.target_bytes, t);
        counts = i >= 0 && i < a.V;
        if (i >= a.V && lane == 0) atomicCAS(a.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
        if (lane == 0 && counts) {
          i0 = static_cast<int>(i);
          p0 = 1.f;
          z0 = a.rows.z[t];
        }
      } else {
        if (lane < a.top) {
          i0 = a.rows.index[base + lane];
          p0 = a.rows.p[base + lane];
          z0 = i0 >= 0 ? a.rows.z[base + lane] : 0.f;
        }
        counts = !a.direct || a.rows.pos[t] >= 0;
        ent = a.rows.ent[t];
      }
      if (counts) weight = a.weights != nullptr ? a.weights[t] : 1.f;
      if (!own) ref = a.rows.ref[r];
    }
    const int j = threadIdx.x % R;
    float m = -INFINITY, s = 0.f;
    const auto add = [&](float m2, float s2) {
      if (own) {
        const float top = fmaxf(m, m2);
        // a largest of the row's that is -inf or equal has the factor 1
        s = s * (m == top ? 1.f : exp2f((m - top) * a.unit)) +
            s2 * (m2 == top ? 1.f : exp2f((m2 - top) * a.unit));
        m = top;
      } else {
        m = fmaxf(m, m2);
        s += s2;
      }
    };
    if (r0 + j < n)
#pragma unroll 4
      for (int i = threadIdx.x / R; i < a.parts; i += kThreads / R) {
        const float2 v = a.part[i * a.ldp + r0 + j];
        add(v.x, v.y);
      }
#pragma unroll
    for (int o = R; o < 32; o *= 2) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), s2 = __shfl_xor_sync(0xffffffffu, s, o);
      add(m2, s2);
    }
    if (lane < R) sums[warp][lane] = make_float2(m, s);
    __syncthreads();
    m = -INFINITY, s = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) add(sums[w][warp % R].x, sums[w][warp % R].y);
    if (on) {
      if (own) ref = m == -INFINITY ? 0.f : m * a.unit;
      // log2 s = log_f + at_s, with the whole number apart: next to a reference 2^28 away
      // it would cost a small loss 1e-6 of rounding.  An infinite logit: the sum is
      // infinite too.
      int whole = 0;
      float f = m == INFINITY ? 1.f : frexpf(s, &whole);
      if (f < 0.70710678f) f *= 2.f, --whole;
      const float log_f = log2f(f), at_s = static_cast<float>(whole);
      float sum = 0.f, both = 0.f, square = 0.f;
      for (int k = lane; k < a.top; k += 32) {
        const int i = k == lane ? i0 : a.rows.index[base + k];
        if (i < 0) continue;
        const float p = k == lane ? p0 : a.rows.p[base + k];
        const float over = fmaf(k == lane ? z0 : a.rows.z[base + k], a.unit, -ref);
        if (!(p == 0.f)) sum += p * (log_f + (at_s - over));
        if (!own) {
          const float term = exp2f(over) / s - p;
          const bf16 kept = __float2bfloat16_rn(term * s);
          a.E[row * a.lde + i] = kept;
          both = fmaf(term, term, both);
          square = fmaf(__bfloat162float(kept) / s, term, square);
        }
      }
      sum = warp_sum(sum);
      both = warp_sum(both);
      square = warp_sum(square);
      if (lane == 0) {
        const float loss = counts ? a.tau * a.tau * (ent + 0.69314718056f * sum) : 0.f;
        a.loss[t] = loss;
        totals[warp] = counts ? static_cast<double>(weight) * loss : 0.0;
        if (!own) {
          // The row's factor takes up what the rounding of its entries' terms has in
          // common (least squares; for one entry all of it): these are most of the
          // gradient, and their errors would be a whole row's of dx and dW.
          // That is within a rounding, 2^-8, of 1; beyond 2^-7 all of them are next to nothing
          // (rounded to 0, or the squares are), and the factor stays as it is.
          float fit = both / square;
          if (!(fabsf(fit - 1.f) <= 0.0078125f)) fit = 1.f;
          a.rows.scale[r] = make_float2(
              a.tau / s * fit, a.weights != nullptr ? weight : 1.f / static_cast<float>(count));
          const float above = m * a.unit - ref;
          if (!a.second && (above > kFits || above < -2.f * kAbove)) {
            a.rows.ref[r] = m * a.unit;
            *again = 1;
          }
        }
      }
    }
  }
  if (!a.second || *again != 0) {
    __syncthreads();
    if (threadIdx.x == 0) {
      double sum = 0.0;
      for (int i = 0; i < min(static_cast<long long>(R), n - r0); ++i) sum += totals[i];
      a.rows.totals[(a.first + r0) / R] = sum;
    }
  }
  if (!a.second || a.x == nullptr) return;
  __syncthreads();
  // the rows of x, all threads
  const bool vec = a.d % 8 == 0;
  const int pieces = vec ? a.d / 8 : a.d;
  const int rows = static_cast<int>(min(static_cast<long long>(R), n - r0));
  const float most = *a.rows.most;
  float by[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float2 f = i < rows ? a.rows.scale[a.first + r0 + i] : make_float2(0.f, 0.f);
    by[i] = f.x * (f.y / most);
  }
  bf16* x = a.x + r0 * a.ldx;
  for (int c = threadIdx.x; c < pieces; c += kThreads) {
    if (vec) {
      Pack<bf16, 8> v[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < rows) v[i] = *reinterpret_cast<const Pack<bf16, 8>*>(x + i * a.ldx + 8 * c);
#pragma unroll
      for (int i = 0; i < R; ++i) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[i].x[k] = __float2bfloat16_rn(__bfloat162float(v[i].x[k]) * by[i]);
        if (i < rows) *reinterpret_cast<Pack<bf16, 8>*>(x + i * a.ldx + 8 * c) = v[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < rows)
          x[i * a.ldx + c] = __float2bfloat16_rn(__bfloat162float(x[i * a.ldx + c]) * by[i]);
    }
  }
}

__global__ void __launch_bounds__(kThreads, 4) loss_finish_kernel(const FinishArgs a) {
  pdl_wait();
  pdl_trigger();
  finish_rows(a);
  if (!a.last) return;
  long long tokens;  // that count
  if (a.direct) {  // T is kFewTokens at most
    long long i = -1;
    if (threadIdx.x < a.T)
      i = a.targets != nullptr ? index_at(a.targets, a.target_bytes, threadIdx.x)
                               : a.rows.pos[threadIdx.x];
    tokens = __syncthreads_count(i >= 0 && i < a.V);
  } else {
    tokens = *a.rows.count;
  }
  const long long count = ((a.direct ? a.T : tokens) + kFinishRows - 1) / kFinishRows;
  const float by = a.weights == nullptr ? static_cast<float>(max(1ll, tokens)) : 1.f;
  if (!a.second || a.rows.again[a.first / a.block] != 0)
    total_behind<kThreads>(a.rows, count, by, a.total);
  else if (blockIdx.x == gridDim.x - 1)  // the parts are the last kernel's
    sum_total<kThreads>(a.rows, count, by, a.total);
}

// Where a block's dz goes as planes too (null: it does not), for rows of the block.
struct DzPlanes {
  bf16* planes;
  int* flags;
  long long rows, stride, pitch;
};

// A CTA per row of the block: its loss from the fp32 logits z, and in place of them dz
// where the gradients are wanted (rows that do not count, and those behind the block's:
// 0), and its planes.  Two passes over the row, 16 bytes at a time.
template <int THREADS>
__device__ __forceinline__ void loss_row(float* __restrict__ z, long long ld, const LossRows& l,
                                         long long first, int V, int top, float inv_tau, float tau,
                                         const float* __restrict__ weights, bool grad,
                                         float* __restrict__ loss, const DzPlanes& dz) {
  __shared__ float ms[THREADS / 32], ss[THREADS / 32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long r = first + blockIdx.x;
  float* row = z + static_cast<long long>(blockIdx.x) * ld;
  const int n = *l.count;
  constexpr int kStep = 8 * THREADS;  // values at a time, two quads of a thread
  bf16* planes = dz.planes + static_cast<long long>(blockIdx.x) * dz.pitch;
  if (r >= n || blockIdx.x >= dz.rows) {
    for (int v = 4 * threadIdx.x; grad && v < V; v += 4 * THREADS) {
      float zero[4] = {0.f, 0.f, 0.f, 0.f};
      if (blockIdx.x < dz.rows)
        *reinterpret_cast<float4*>(row + v) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (dz.planes != nullptr) store_planes(planes + v, dz.stride, zero);
    }
    if (dz.planes != nullptr && threadIdx.x == 0 && blockIdx.x < dz.rows) dz.flags[blockIdx.x] = 0;
    return;
  }
  // this thread's eight values from v0 on; behind the row's end -inf
  const auto load = [&](int v0, float (&x)[8]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = v0 + 4 * (threadIdx.x + h * THREADS);
      float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      if (v < V) q = *reinterpret_cast<const float4*>(row + v);
      x[4 * h] = q.x, x[4 * h + 1] = q.y, x[4 * h + 2] = q.z, x[4 * h + 3] = q.w;
      if (v + 3 >= V) {
#pragma unroll
        for (int j = 1; j < 4; ++j)
          if (v + j >= V) x[4 * h + j] = -INFINITY;
      }
    }
  };
  // largest and sum in one pass
  float m = -INFINITY, s = 0.f;
  for (int v0 = 0; v0 < V; v0 += kStep) {
    float x[8], top_x = m;
    load(v0, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) top_x = fmaxf(top_x, x[j]);
    if (m < top_x) {
      s *= expf((m - top_x) * inv_tau);
      m = top_x;
    }
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < 8; ++j) s += expf((x[j] - ref) * inv_tau);
  }
  const float mine = m;
  m = warp_max(m);
  if (lane == 0) ms[warp] = m;
  __syncthreads();
  for (int w = 0; w < THREADS / 32; ++w) m = fmaxf(m, ms[w]);
  if (mine < m) s *= expf((mine - m) * inv_tau);
  s = warp_sum(s);
  if (lane == 0) ss[warp] = s;
  __syncthreads();
  s = 0.f;
  for (int w = 0; w < THREADS / 32; ++w) s += ss[w];
  const long long t = l.token[r], base = t * top;
  if (warp == 0) {
    // an infinite logit: the sum is infinite too
    const float log_s = m == INFINITY ? 0.f : logf(s);
    float sum = 0.f;
    for (int k = lane; k < top; k += 32) {
      const int i = l.index[base + k];
      const float p = l.p[base + k];
      if (i >= 0 && !(p == 0.f)) sum += p * (log_s - (row[i] - m) * inv_tau);
    }
    sum = warp_sum(sum);
    if (lane == 0) {  // thread 0
      const float of_row = tau * tau * (l.ent[t] + sum);
      loss[t] = of_row;
      l.totals[r] = (weights != nullptr ? weights[t] : 1.0) * of_row;
    }
  }
  if (!grad) return;
  const float scale = (weights != nullptr ? weights[t] : 1.f / static_cast<float>(n)) * tau;
  __syncthreads();
  const float over = scale / s;
  // Below 2^-109 the products on the tensor cores do not take a value: it is 0 where that is
  // next to nothing, 2^-45 of the row's factor; a smaller factor leaves it to the CUDA cores.
  const float least = dz.planes != nullptr && fabsf(scale) >= 5.4210108624e-20f  // 2^-64
                          ? 1.5407439555e-33f
                          : 0.f;
  bool bad = false;
  for (int v0 = 0; v0 < V; v0 += kStep) {
    float x[8];
    load(v0, x);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float term = over * expf((x[j] - m) * inv_tau);
      x[j] = fabsf(term) < least ? 0.f : term;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int v = v0 + 4 * (threadIdx.x + h * THREADS);
      if (v >= V) continue;
      float q[4] = {x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]};
      *reinterpret_cast<float4*>(row + v) = make_float4(q[0], q[1], q[2], q[3]);
      if (dz.planes == nullptr) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) bad |= outside_planes(q[j]);
      store_planes(planes + v, dz.stride, q);
    }
  }
  __syncthreads();
  for (int k = threadIdx.x; k < top; k += THREADS) {
    const int i = l.index[base + k];
    if (i < 0) continue;
    const float term = row[i] - scale * l.p[base + k];
    row[i] = term;
    if (dz.planes == nullptr) continue;
    bad |= outside_planes(term);
    store_planes(planes + i, dz.stride, term);
  }
  if (dz.planes == nullptr) return;
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) dz.flags[blockIdx.x] = bad;
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS)
    loss_rows_kernel(float* __restrict__ z, long long ld, LossRows l, long long first, int V,
                     int top, float inv_tau, float tau, const float* __restrict__ weights,
                     bool grad, float* __restrict__ loss, const DzPlanes dz, bool last,
                     float* __restrict__ total) {
  pdl_wait();
  pdl_trigger();
  loss_row<THREADS>(z, ld, l, first, V, top, inv_tau, tau, weights, grad, loss, dz);
  if (last)
    total_behind<THREADS>(l, *l.count,
                          weights == nullptr ? static_cast<float>(max(1, *l.count)) : 1.f, total);
}

// dx of the block's rows, the sum of `slices` products (the first alone where the
// product's flag `whole` says that the CUDA cores made it), to their tokens.
__global__ void __launch_bounds__(kThreads)
    loss_scatter_kernel(const float* __restrict__ rows, int slices, const int* __restrict__ whole,
                        LossRows l, long long first, long long block, int d,
                        float* __restrict__ dx) {
  pdl_wait();
  pdl_trigger();
  const long long r = blockIdx.x;
  const int c = blockIdx.y * kThreads + threadIdx.x;
  if (first + r >= *l.count || c >= d) return;
  const long long t = l.token[first + r];
  if (slices > 1 && *whole != 0) slices = 1;
  float v = 0.f;
#pragma unroll 8
  for (int i = 0; i < slices; ++i) v += rows[(i * block + r) * d + c];
  dx[t * d + c] = v;
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }
long long round64(long long n) { return (n + 63) / 64 * 64; }

constexpr size_t kBlockBytes = size_t{1} << 31;  // of a block's terms
constexpr size_t kCutBytes = size_t{64} << 20;  // of fp32 dx's slices
constexpr long long kFewTokens = 64;

// Elements between rows of d features as TMA operands (16-byte multiples).
long long pitch_of(int d, bool is_bf16) { return !is_bf16 || d % 8 == 0 ? d : round64(d); }

// Where everything lies in the workspace.
struct Plan {
  long long block;  // rows taken at a time, a multiple of 64
  int blocks;
  long long ldx, lde, ldp;
  size_t meta = 0, again, pos, token, index, p, ent, lead, z, totals, ref, scale, xg, wp, terms,
         part, acc, cut, x_planes, z_planes, scratch, total;
  Plan(const LossArgs& a, bool want_dx, bool want_dw) {
    const size_t T = static_cast<size_t>(a.T), es = a.is_bf16 ? 2 : 4;
    const bool grad = want_dx || want_dw;
    lde = a.is_bf16 ? round64(a.V) : (a.V + 3) / 4 * 4;  // 16-byte rows
    ldx = pitch_of(a.d, a.is_bf16);
    block = a.block > 0
                ? a.block
                : static_cast<long long>(kBlockBytes / es / static_cast<size_t>(lde) / 64 * 64);
    block = std::max(64ll, std::min(round64(block), round64(a.T)));
    blocks = static_cast<int>((a.T + block - 1) / block);
    ldp = block;
    size_t at = 256;
    const auto take = [&](size_t bytes) {
      const size_t here = at;
      at += round256(bytes);
      return here;
    };
    again = take(4 * static_cast<size_t>(blocks));
    pos = take(4 * T);
    token = take(4 * T);
    index = take(4 * T * a.top);
    p = take(4 * T * a.top);
    ent = take(4 * T);
    lead = take(4 * T);
    z = take(4 * T * a.top);
    totals = take(8 * T);
    ref = take(4 * T);
    scale = take(8 * T);
    xg = take(es * static_cast<size_t>(round64(a.T)) * ldx);
    wp = take(ldx != a.d ? es * static_cast<size_t>(a.V) * ldx : 0);
    terms = take(!a.is_bf16 || grad ? es * static_cast<size_t>(block) * lde : 0);
    part = take(a.is_bf16 ? sizeof(float2) * static_cast<size_t>(loss_parts(a.V)) * ldp : 0);
    acc = take(want_dw && a.is_bf16 && blocks > 1 ? 4 * static_cast<size_t>(a.V) * a.d : 0);
    cut = take(a.is_bf16 && ((want_dx && loss_cuts(a.V)) || (want_dw && loss_cuts(block)))
                   ? loss_cut_bytes()
               : !a.is_bf16 && want_dx
                   ? std::max(4 * static_cast<size_t>(block) * a.d,
                              std::min(kCutBytes,
                                       4 * kMaxFp32Slices * static_cast<size_t>(block) * a.d))
                   : 0);
    const bool planes = want_dw && !a.is_bf16;
    x_planes = take(planes ? linear_planes_bytes(block, a.d) : 0);
    z_planes = take(grad && !a.is_bf16 ? linear_planes_bytes(block, a.V) : 0);
    scratch = take(a.is_bf16 ? 0 : fp32_scratch(a, grad, want_dw));
    total = at;
  }

  // The largest of the products' scratch, for blocks of any number of rows: of the
  // logits', without x's planes where dW keeps them; with gradients also W's for dx.
  size_t fp32_scratch(const LossArgs& a, bool grad, bool want_dw) const {
    LinearProduct g;
    g.M = block, g.N = a.V, g.K = a.d;
    return std::max(want_dw ? 0 : linear_split_scratch_up_to(g),
                    grad ? linear_split_b_scratch(g) : 0);
  }
};

template <typename F>
cudaError_t launched(const char* tag, cudaStream_t s, F&& call) {
  prof_begin(tag, s);
  const cudaError_t e = call();
  prof_end(tag, s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned warps_grid(long long warps) {
  return static_cast<unsigned>((warps + kThreads / 32 - 1) / (kThreads / 32));
}

// rows of d features onto rows of ld: 16-byte multiples, which TMA needs.
__global__ void __launch_bounds__(kThreads)
    loss_pad_kernel(const bf16* __restrict__ in, int d, bf16* __restrict__ out, long long ld,
                    long long rows) {
  pdl_wait();
  pdl_trigger();
  const long long r = blockIdx.x * static_cast<long long>(kThreads / 32) + threadIdx.x / 32;
  if (r >= rows) return;
  for (int c = threadIdx.x % 32; c < d; c += 32) out[r * ld + c] = in[r * d + c];
}

// Losses alone of a few tokens: from x as it lies, the weight streamed once.  The
// rows do not touch each other, so tokens that do not count may run along.  In graphs
// behind a flush of L2, streamed / on CTA pairs: 2048 -> 32000, one token 43 / 56 us,
// 64 46 / 57; 4096 -> 128256, one 181 / 207, 64 197 / 214.  From 65 to 128 tokens it is
// 52 / 56 and 224 / 217, but the tile's accumulators are too wide for several of them,
// which the losses' precision takes.
bool few_form(const LossArgs& a) {
  return a.is_bf16 && a.dx == nullptr && a.dW == nullptr && a.T <= kFewTokens && a.d % 8 == 0;
}

cudaError_t few_logits(const LossArgs& a, const LossProducts& p, cudaStream_t s) {
  LossColumns c;
  c.part = p.part;
  c.ldp = p.ldp;
  c.unit = p.unit;
  c.index = p.rows.index;
  c.targets = a.top_logits == nullptr ? a.indices : nullptr;
  c.target_bytes = a.index_bytes;
  c.z = p.rows.z;
  c.top = a.top;
  c.done = p.rows.done;
  LinearProduct g;
  g.A = a.x;
  g.B = a.W;
  g.lda = g.ldb = a.d;
  g.M = a.T, g.N = a.V, g.K = a.d;
  g.loss = &c;
  g.tag = "loss_stream";
  return linear_stream(g, s);
}

cudaError_t run_bf16(const LossArgs& a, const Plan& plan, const LossRows& l, char* ws,
                     cudaStream_t s) {
  const bool direct = few_form(a);
  const bool grad = a.dx != nullptr || a.dW != nullptr;
  bf16* xg = reinterpret_cast<bf16*>(ws + plan.xg);
  bf16* E = grad ? reinterpret_cast<bf16*>(ws + plan.terms) : nullptr;
  cudaError_t e;
  LossProducts g;
  g.W = a.W;
  g.ldw = g.ldx = plan.ldx;
  if (plan.ldx != a.d) {
    bf16* wp = reinterpret_cast<bf16*>(ws + plan.wp);
    g.W = wp;
    e = launched("loss_pad", s, [&] {
      return launch_pdl(loss_pad_kernel, dim3(warps_grid(a.V)), dim3(kThreads), 0, s,
                        static_cast<const bf16*>(a.W), a.d, wp, plan.ldx,
                        static_cast<long long>(a.V));
    });
    if (e != cudaSuccess) return e;
  }
  g.E = E;
  g.lde = plan.lde;
  g.part = reinterpret_cast<float2*>(ws + plan.part);
  g.ldp = plan.ldp;
  g.unit = 1.44269504089f / a.tau;
  g.block = plan.block;
  g.d = a.d;
  g.V = a.V;
  g.top = a.top;
  g.dx = a.dx;
  g.dW = a.dW;
  g.acc = plan.blocks > 1 ? reinterpret_cast<float*>(ws + plan.acc) : nullptr;
  g.parts = reinterpret_cast<float*>(ws + plan.cut);
  g.schedule = ws + plan.meta + 64;
  g.rows = l;
  FinishArgs f = {};
  f.direct = direct;
  f.targets = direct && a.top_logits == nullptr ? a.indices : nullptr;
  f.target_bytes = a.index_bytes;
  f.V = a.V;
  f.status = device_status_ptr();
  f.rows = l;
  f.part = g.part;
  f.ldp = g.ldp;
  f.block = plan.block;
  f.parts = direct ? (a.V + 127) / 128 : loss_parts(a.V);
  f.top = a.top;
  f.d = a.d;
  f.unit = g.unit;
  f.tau = a.tau;
  f.weights = a.weights;
  f.loss = a.loss;
  f.E = E;
  f.lde = g.lde;
  f.ldx = g.ldx;
  f.T = a.T;
  f.total = a.total;
  for (int b = 0; b < plan.blocks; ++b) {
    bf16* xb = xg + b * plan.block * plan.ldx;
    g.first = f.first = b * plan.block;
    g.x = xb;
    g.x_rows = std::min(plan.block, round64(a.T) - g.first);
    for (int pass = 0; pass < (grad ? 2 : 1); ++pass) {
      e = direct ? few_logits(a, g, s) : loss_logits(g, pass > 0, s);
      if (e != cudaSuccess) return e;
      f.second = pass > 0;
      f.x = a.dW != nullptr ? xb : nullptr;
      f.last = b == plan.blocks - 1 && (!grad || pass == 1);
      e = launched("loss_finish", s, [&] {
        return launch_pdl(
            loss_finish_kernel,
            dim3(static_cast<unsigned>((plan.block + kFinishRows - 1) / kFinishRows)),
            dim3(kThreads), 0, s, f);
      });
      if (e != cudaSuccess) return e;
    }
    if (a.dx != nullptr && (e = loss_dx(g, s)) != cudaSuccess) return e;
    if (a.dW != nullptr && (e = loss_dw(g, s)) != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// fp32: the products of linear_fp32 on a block's logits, which become dz in place.  Rows
// that do not count are 0.  dz' planes are made along with it (a launch of their own: 515
// tokens, 1000 -> 10007 268 us, not 261; 333 tokens, 768 -> 30001 387, not 377), x's for
// the logits, and dW takes both as they lie (dz transposed and split again: 21 and 41 us
// more).
cudaError_t run_f32(const LossArgs& a, const Plan& plan, const LossRows& l, char* ws,
                    cudaStream_t s) {
  float* xg = reinterpret_cast<float*>(ws + plan.xg);
  float* z = reinterpret_cast<float*>(ws + plan.terms);
  void* scratch = ws + plan.scratch;
  float* out = reinterpret_cast<float*>(ws + plan.cut);
  const bool grad = a.dx != nullptr || a.dW != nullptr;
  char* x_planes = a.dW != nullptr ? ws + plan.x_planes : nullptr;
  char* z_planes = ws + plan.z_planes;
  cudaError_t e;
  bool ready = false;  // W's planes are in the scratch
  for (long long first = 0; first < a.T; first += plan.block) {
    const long long rows = std::min(plan.block, a.T - first);
    float* xb = xg + first * a.d;
    const int slices = a.dx != nullptr ? linear_split_slices(rows, a.d, a.V, kCutBytes) : 1;
    const bool split_dx =
        a.dx != nullptr && (slices > 1 || linear_split_pays(rows, a.d, a.V));
    const bool split_dw =
        a.dW != nullptr && linear_split_pays(a.V, a.d, static_cast<int>(rows));
    const bool x_ready = linear_split_pays(rows, a.V, a.d);  // the logits made its planes
    DzPlanes dz = {};
    dz.rows = rows;
    if (split_dx || split_dw) {
      const Fp32Planes at = linear_planes_at(z_planes, rows, a.V);
      dz.planes = static_cast<bf16*>(at.planes);
      dz.flags = at.flags;
      dz.pitch = at.pitch;
      dz.stride = at.plane_rows * at.pitch;
    }
    LinearProduct g;
    g.A = xb;
    g.B = a.W;
    g.y = z;
    g.pitch_y = plan.lde;
    g.M = rows, g.N = a.V, g.K = a.d;
    g.b_ready = ready;
    g.a_planes = x_planes;
    g.tag = "loss_logits";
    if ((e = linear_fp32(g, scratch, s)) != cudaSuccess) return e;
    ready |= x_ready;
    e = launched("loss_rows", s, [&] {
      // long rows take 512 threads, four CTAs on an SM: 333 of 30001 28 us (with 1024
      // a second wave), 515 of 10007 19; short ones 256
      const bool wide = a.V > 8192;
      return launch_pdl(wide ? loss_rows_kernel<512> : loss_rows_kernel<kThreads>,
                        dim3(static_cast<unsigned>(dz.planes != nullptr ? round64(rows) : rows)),
                        dim3(wide ? 512 : kThreads), 0, s, z, plan.lde, l, first, a.V, a.top,
                        1.f / a.tau, a.tau, a.weights, grad, a.loss, dz, first + rows >= a.T,
                        a.total);
    });
    if (e != cudaSuccess) return e;
    if (a.dx != nullptr) {
      LinearProduct q;
      q.A = z;
      q.pitch_a = plan.lde;
      q.B = a.W;
      q.b_mn = true;
      q.slices = slices;
      q.b_ready = ready;
      q.a_planes = z_planes;
      q.a_ready = true;
      q.y = out;
      q.M = rows, q.N = a.d, q.K = a.V;
      q.tag = "loss_dx";
      if ((e = linear_fp32(q, scratch, s)) != cudaSuccess) return e;
      ready |= split_dx;
      e = launched("loss_scatter", s, [&] {
        return launch_pdl(loss_scatter_kernel,
                          dim3(static_cast<unsigned>(rows),
                               static_cast<unsigned>((a.d + kThreads - 1) / kThreads)),
                          dim3(kThreads), 0, s,
                          static_cast<const float*>(out), q.slices,
                          static_cast<const int*>(scratch), l, first, rows, a.d,
                          static_cast<float*>(a.dx));
      });
      if (e != cudaSuccess) return e;
    }
    if (a.dW != nullptr) {
      LinearProduct q;
      q.A = z;
      q.pitch_a = plan.lde;
      q.B = xb;
      q.a_mn = q.b_mn = true;
      q.residual = first > 0 ? a.dW : nullptr;
      q.y = a.dW;
      q.M = a.V, q.N = a.d, q.K = static_cast<int>(rows);
      q.tag = "loss_dw";
      if (split_dw) {
        if (!x_ready && (e = linear_split_planes(xb, rows, a.d, a.d, x_planes, s)) != cudaSuccess)
          return e;
        e = linear_split_turned(q, z_planes, x_planes, s);
      } else {
        e = linear_simt(q, s);
      }
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

template <typename TX, int V>
cudaError_t run_gather(const LossArgs& a, const Plan& plan, const LossRows& l, char* ws,
                       cudaStream_t s) {
  const bool grad = a.dx != nullptr || a.dW != nullptr;
  const bool start = a.T <= kStartTokens;
  StartArgs st;
  st.targets = a.top_logits == nullptr ? a.indices : nullptr;
  st.index_bytes = a.index_bytes;
  st.V = a.V;
  st.blocks = plan.blocks;
  st.weights = a.weights;
  st.status = device_status_ptr();
  cudaError_t e;
  if (!start) {
    e = launched("loss_order", s, [&] {
      return launch_pdl(loss_order_kernel, dim3(1), dim3(kOrderThreads), 0, s, l, a.T, a.weights,
                        plan.blocks, st.targets, a.index_bytes, a.V, st.status);
    });
    if (e != cudaSuccess) return e;
  }
  return launched("loss_gather", s, [&] {
    return launch_pdl(start ? loss_gather_kernel<TX, V, true> : loss_gather_kernel<TX, V, false>,
                      dim3(warps_grid(a.T + round64(a.T))), dim3(kThreads), 0, s,
                      static_cast<const TX*>(a.x), static_cast<const TX*>(a.W), l, a.T, a.d,
                      reinterpret_cast<TX*>(ws + plan.xg), plan.ldx, !a.is_bf16,
                      a.is_bf16 && grad ? 1.44269504089f / a.tau : 0.f, a.loss,
                      static_cast<TX*>(a.dx), st);
  });
}

}  // namespace

size_t head_loss_scratch(const LossArgs& a, bool want_dx, bool want_dw) {
  return Plan(a, want_dx, want_dw).total;
}

cudaError_t head_loss(const LossArgs& a, void* scratch, cudaStream_t s) {
  char* ws = static_cast<char*>(scratch);
  const Plan plan(a, a.dx != nullptr, a.dW != nullptr);
  LossRows l;
  l.count = reinterpret_cast<int*>(ws + plan.meta);
  l.most = reinterpret_cast<float*>(ws + plan.meta + 4);
  l.again = reinterpret_cast<int*>(ws + plan.again);
  l.pos = reinterpret_cast<int*>(ws + plan.pos);
  l.token = reinterpret_cast<int*>(ws + plan.token);
  l.index = reinterpret_cast<int*>(ws + plan.index);
  l.p = reinterpret_cast<float*>(ws + plan.p);
  l.ent = reinterpret_cast<float*>(ws + plan.ent);
  l.lead = reinterpret_cast<int*>(ws + plan.lead);
  l.z = reinterpret_cast<float*>(ws + plan.z);
  l.totals = reinterpret_cast<double*>(ws + plan.totals);
  l.ref = reinterpret_cast<float*>(ws + plan.ref);
  l.scale = reinterpret_cast<float2*>(ws + plan.scale);
  l.done = reinterpret_cast<int*>(ws + plan.meta + 8);
  cudaError_t e = cudaSuccess;
  const bool ce = a.top_logits == nullptr;
  if (!ce) {
    e = launched("loss_entries", s, [&] {
      return launch_pdl(loss_entries_kernel,
                        dim3(static_cast<unsigned>((a.T + kEntryWarps - 1) / kEntryWarps)),
                        dim3(32 * kEntryWarps), 0, s, a.indices, a.index_bytes, a.top_logits,
                        a.top_bf16, a.T, a.top, a.V, 1.f / a.tau, l, device_status_ptr());
    });
    if (e != cudaSuccess) return e;
  }
  // the kernels of few_logits take targets or entries as they are
  if (few_form(a))
    e = cudaSuccess;
  else if (a.is_bf16)
    e = a.d % 8 == 0 ? run_gather<bf16, 8>(a, plan, l, ws, s)
                     : run_gather<bf16, 1>(a, plan, l, ws, s);
  else
    e = a.d % 4 == 0 ? run_gather<float, 4>(a, plan, l, ws, s)
                     : run_gather<float, 1>(a, plan, l, ws, s);
  if (e != cudaSuccess) return e;
  return a.is_bf16 ? run_bf16(a, plan, l, ws, s) : run_f32(a, plan, l, ws, s);
}

}  // namespace poetx
