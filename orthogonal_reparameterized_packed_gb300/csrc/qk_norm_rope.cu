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
// the sums, and a warp works on 32 / G heads of a token at once.  A warp goes
// through the heads of its token with the table row and gamma in registers
// (few tokens: through a part of them, so that every SM has work).  What
// bounds it is memory traffic: 2 (forward) or 3 (backward) passes over q and k.
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>

#include "internal.h"
#include "poetx.h"
#include "ptx.cuh"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxD = 512;
constexpr int kForwardPerSm = 2;   // CTAs per SM that the registers are cut for
constexpr int kBackwardPerSm = 2;

// V elements as the memory holds them.
template <typename T, int V>
struct alignas(sizeof(T) * V) Pack {
  T x[V];
};

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float& o, float x) { o = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }

template <typename T, int V>
__device__ __forceinline__ void unpack(float (&o)[V], const Pack<T, V>& q) {
  if constexpr (sizeof(T) == 2 && V > 1) {
    uint32_t w[V / 2];
    memcpy(w, &q, sizeof(w));
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      o[2 * j] = __uint_as_float(w[j] << 16);
      o[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = to_f(q.x[j]);
  }
}

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float (&v)[V]) {
  Pack<T, V> q;
  if constexpr (sizeof(T) == 2 && V > 1) {
    uint32_t w[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * j], v[2 * j + 1]);
      memcpy(&w[j], &h, 4);
    }
    memcpy(&q, w, sizeof(w));
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) from_f(q.x[j], v[j]);
  }
  return q;
}

// Slot s of a row: the vectors at o0 and o1; `turns`: its pairs are rotated,
// with the trigonometric entries [s V, s V + V).
struct Slot {
  int o0, o1;
  bool turns, has0, has1;
};

// FULL: every lane has whole slots and all of them turn.
template <int V, bool INTER, bool FULL>
__device__ __forceinline__ Slot slot_of(int s, int D, int rot) {
  Slot w;
  const int nrot = rot / 2 / V;
  w.turns = FULL || s < nrot;
  if (w.turns) {
    w.o0 = INTER ? 2 * s * V : s * V;
    w.o1 = INTER ? w.o0 + V : rot / 2 + s * V;
  } else {
    w.o0 = rot + (s - nrot) * 2 * V;
    w.o1 = w.o0 + V;
  }
  w.has0 = FULL || w.o0 < D;
  w.has1 = FULL || w.o1 < D;
  return w;
}

// Where value j of the slot's first (b = 0) or second vector finds its pair:
// half by half, value j of the other vector; interleaved vectors hold whole
// pairs, (2i, 2i + 1), the first vector's with table entries [0, V/2) and the
// second's with [V/2, V).
template <int V, bool INTER>
struct Pairs {
  static constexpr bool ADJACENT = INTER && V > 1;  // V = 1: a slot is one pair either way
  // table entry of pair i = 0 .. V - 1, and its two members' (vector, value)
  static constexpr int vec_a(int i) { return ADJACENT ? (i >= V / 2) : 0; }
  static constexpr int vec_b(int i) { return ADJACENT ? (i >= V / 2) : 1; }
  static constexpr int at_a(int i) { return ADJACENT ? 2 * (i % (V / 2 > 0 ? V / 2 : 1)) : i; }
  static constexpr int at_b(int i) { return ADJACENT ? at_a(i) + 1 : i; }
};

// V floats; V >= 4: from a 16-byte aligned address.
template <int V>
__device__ __forceinline__ void load_f32(float (&o)[V], const float* p) {
  if (V % 4 == 0) {
#pragma unroll
    for (int j = 0; j + 3 < V; j += 4) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p + j));
      o[j] = q.x, o[j + 1] = q.y, o[j + 2] = q.z, o[j + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = __ldg(p + j);
  }
}

// The next rows of a warp on their way to shared memory while it works on the
// current ones: STAGES groups of N vectors per lane.  Every lane copies and
// reads only its own vectors, so the ring needs no barrier.  (It is the bytes
// in flight that bound these kernels: with the next group in registers
// instead, 126 of them left 16 warps per SM and the backward pass at 3.9 TB/s.)
// Vectors of two bytes cannot be copied this way and are read when needed.
template <typename T, int V, int N>
struct Rows {
  static constexpr int BYTES = sizeof(T) * V;
  static constexpr bool ASYNC = BYTES >= 4;
  static constexpr int STAGES = !ASYNC ? 1 : N * BYTES <= 64 ? 4 : 2;
  static constexpr int SMEM = ASYNC ? kWarps * STAGES * N * 32 * BYTES : 0;  // of a CTA

  uint32_t base;         // this lane's first vector
  Pack<T, V> direct[N];  // !ASYNC

  __device__ __forceinline__ explicit Rows(uint8_t* smem) {
    base = smem_u32(smem) + (threadIdx.x / 32) * (STAGES * N * 32 * BYTES) +
           (threadIdx.x % 32) * BYTES;
  }
  __device__ __forceinline__ uint32_t at(int stage, int n) const {
    return base + static_cast<uint32_t>((stage * N + n) * 32 * BYTES);
  }
  // Vector n of a stage from p; zeros where there is none.
  __device__ __forceinline__ void fetch(int stage, int n, const T* p, bool has) {
    if constexpr (BYTES == 16) {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at(stage, n)), "l"(p),
                   "r"(has ? 16 : 0)
                   : "memory");
    } else if constexpr (ASYNC) {
      asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(at(stage, n)), "l"(p),
                   "n"(BYTES), "r"(has ? BYTES : 0)
                   : "memory");
    } else {
      if (has)
        direct[n] = *reinterpret_cast<const Pack<T, V>*>(p);
      else
        memset(&direct[n], 0, sizeof(direct[n]));
    }
  }
  __device__ __forceinline__ static void commit() {
    if constexpr (ASYNC) asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // The oldest of the STAGES groups has arrived.
  __device__ __forceinline__ static void wait() {
    if constexpr (ASYNC) asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
  }
  __device__ __forceinline__ void read(int stage, int n, float (&o)[V]) const {
    Pack<T, V> q;
    if constexpr (BYTES == 16) {
      uint32_t w[4];
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                   : "r"(at(stage, n))
                   : "memory");
      memcpy(&q, w, 16);
    } else if constexpr (ASYNC) {
      uint32_t w[BYTES / 4];
#pragma unroll
      for (int i = 0; i < BYTES / 4; ++i)
        asm volatile("ld.shared.b32 %0, [%1];"
                     : "=r"(w[i])
                     : "r"(at(stage, n) + 4 * i)
                     : "memory");
      memcpy(&q, w, BYTES);
    } else {
      q = direct[n];
    }
    unpack<T, V>(o, q);
  }
};

// gamma's values of a slot (ones where there is no gamma).
template <int V>
__device__ __forceinline__ void load_gamma(float (&m)[2][V], const float* gamma, const Slot& w) {
#pragma unroll
  for (int i = 0; i < V; ++i) m[0][i] = m[1][i] = 1.f;
  if (gamma == nullptr) return;
  if (w.has0) load_f32<V>(m[0], gamma + w.o0);
  if (w.has1) load_f32<V>(m[1], gamma + w.o1);
}

// The slot's table entries of row tr (1 and 0 where nothing turns).
template <int V>
__device__ __forceinline__ void load_trig(float (&c)[V], float (&s)[V], const QkNormRopeArgs& a,
                                          long long tr, int slot, const Slot& w) {
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 1.f, s[i] = 0.f;
  if (!w.turns) return;
  load_f32<V>(c, a.cos_table + tr * (a.rot / 2) + slot * V);
  load_f32<V>(s, a.sin_table + tr * (a.rot / 2) + slot * V);
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

// A warp's way through its items, `chunk` of the groups of one token each, q's
// groups (iq of them) before k's; stepped without divisions.
struct Walk {
  int items, step, step_t, step_c, chunk, chunks, iq, groups;
  int it, t, c;       // the item: token t, its c-th chunk
  int g, end, after;  // group g of [.., end) of a side; k's groups that follow
  bool is_k;

  __device__ __forceinline__ Walk(int first, int step_, int items_, int chunk_, int chunks_,
                                  int iq_, int groups_)
      : items(items_), step(step_), chunk(chunk_), chunks(chunks_), iq(iq_), groups(groups_) {
    step_t = step / chunks;
    step_c = step - step_t * chunks;
    it = first;
    t = first / chunks;
    c = first - t * chunks;
    enter();
  }
  __device__ __forceinline__ void enter() {
    const int first = c * chunk, last = min(groups, first + chunk);
    is_k = first >= iq;
    g = is_k ? first - iq : first;
    end = is_k ? last - iq : min(last, iq);
    after = is_k ? 0 : last - iq;
  }
  __device__ __forceinline__ bool live() const { return it < items; }
  // To the next group; true where it is of another token or side.
  __device__ __forceinline__ bool next() {
    if (++g < end) return false;
    if (after > 0) {
      is_k = true;
      g = 0;
      end = after;
      after = 0;
      return true;
    }
    it += step;
    t += step_t;
    c += step_c;
    if (c >= chunks) {
      c -= chunks;
      ++t;
    }
    enter();
    return true;
  }
};

// Items of groups of 32 / G heads of one token (q's groups, then k's), NS slots
// per lane.  gamma and the table row are multiplied once per token and side,
// so that a value costs three operations: y_a = r (x_a (g_a c) - x_b (g_b s)).
template <typename T, int V, int G, int NS, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, NS == 1 ? kForwardPerSm : 1)
    qk_forward_kernel(const QkNormRopeArgs a, int chunk, int chunks) {
  pdl_wait();
  pdl_trigger();
  using P = Pairs<V, INTER>;
  using Ring = Rows<T, V, 2 * NS>;
  constexpr int R = 32 / G;  // rows per warp
  extern __shared__ __align__(16) uint8_t smem[];
  Ring ring(smem);
  const int lane = threadIdx.x % 32, li = lane % G, row = lane / G;
  const int iq = (a.hq + R - 1) / R, groups = iq + (a.hk + R - 1) / R;
  const float inv_d = 1.f / static_cast<float>(a.D);
  Slot w[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) w[j] = slot_of<V, INTER, FULL>(li + G * j, a.D, a.rot);
  Walk now(static_cast<int>(blockIdx.x) * kWarps + threadIdx.x / 32,
           static_cast<int>(gridDim.x) * kWarps, static_cast<int>(a.T) * chunks, chunk, chunks, iq,
           groups);
  Walk ahead = now;
  bool fresh = true;  // the group ahead begins another token or side
  const T* x = nullptr;
  int x_head = 0;
  auto fetch = [&](int stage) {
    if (ahead.live()) {
      if (fresh) {
        x_head = ahead.g * R + row;
        x = static_cast<const T*>(ahead.is_k ? a.k : a.q) +
            ahead.t * (ahead.is_k ? a.ld_k : a.ld_q) + x_head * a.D;
      }
      const bool live = x_head < (ahead.is_k ? a.hk : a.hq);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        ring.fetch(stage, 2 * j, x + w[j].o0, live && (FULL || w[j].has0));
        ring.fetch(stage, 2 * j + 1, x + w[j].o1, live && (FULL || w[j].has1));
      }
      x_head += R;
      x += R * a.D;
      fresh = ahead.next();
    }
    Ring::commit();
  };
  if (Ring::ASYNC)
    for (int s = 0; s < Ring::STAGES; ++s) fetch(s);
  // own[v][i] x[v][i] is the value's own part, cross[v][i] x[v][i] its partner's
  float own[NS][2][V], cross[NS][2][V];
  long long tr = -1;
  bool turned = true;  // another token or side than the last group's
  T* out = nullptr;
  int head = 0;
  for (int stage = 0; now.live(); stage = stage + 1 == Ring::STAGES ? 0 : stage + 1) {
    if (turned) {
      head = now.g * R + row;
      out = static_cast<T*>(now.is_k ? a.out_k : a.out_q) +
            now.t * (now.is_k ? a.ld_out_k : a.ld_out_q) + head * a.D;
      tr = table_row(a, now.t);
      if (tr >= 0) {
        const float* gamma = now.is_k ? a.gamma_k : a.gamma_q;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          float cs[V], sn[V], m[2][V];
          load_trig<V>(cs, sn, a, tr, li + G * j, w[j]);
          load_gamma<V>(m, gamma, w[j]);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            own[j][P::vec_a(i)][P::at_a(i)] = m[P::vec_a(i)][P::at_a(i)] * cs[i];
            own[j][P::vec_b(i)][P::at_b(i)] = m[P::vec_b(i)][P::at_b(i)] * cs[i];
            cross[j][P::vec_a(i)][P::at_a(i)] = m[P::vec_a(i)][P::at_a(i)] * sn[i];
            cross[j][P::vec_b(i)][P::at_b(i)] = -m[P::vec_b(i)][P::at_b(i)] * sn[i];
          }
        }
      } else if (lane == 0) {
        atomicCAS(a.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
      }
    }
    if (!Ring::ASYNC) fetch(stage);
    Ring::wait();
    float v[NS][2][V];
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      ring.read(stage, 2 * j, v[j][0]);
      ring.read(stage, 2 * j + 1, v[j][1]);
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i)
        ss = fmaf(v[j][0][i], v[j][0][i], fmaf(v[j][1][i], v[j][1][i], ss));
    if (Ring::ASYNC) fetch(stage);
    const bool live = head < (now.is_k ? a.hk : a.hq);
    ss = group_sum<G>(ss);
    const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
    if (tr < 0) {  // outside the table: zeros
      const float zero[V] = {};
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        if (live && w[j].has0) *reinterpret_cast<Pack<T, V>*>(out + w[j].o0) = pack<T, V>(zero);
        if (live && w[j].has1) *reinterpret_cast<Pack<T, V>*>(out + w[j].o1) = pack<T, V>(zero);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        float y[2][V];
        if (FULL || w[j].turns) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float xa = v[j][P::vec_a(i)][P::at_a(i)];
            const float xb = v[j][P::vec_b(i)][P::at_b(i)];
            y[P::vec_a(i)][P::at_a(i)] = r * fmaf(xa, own[j][P::vec_a(i)][P::at_a(i)],
                                                  xb * cross[j][P::vec_b(i)][P::at_b(i)]);
            y[P::vec_b(i)][P::at_b(i)] = r * fmaf(xb, own[j][P::vec_b(i)][P::at_b(i)],
                                                  xa * cross[j][P::vec_a(i)][P::at_a(i)]);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < V; ++i) y[h][i] = r * (v[j][h][i] * own[j][h][i]);
        }
        if (live && (FULL || w[j].has0))
          *reinterpret_cast<Pack<T, V>*>(out + w[j].o0) = pack<T, V>(y[0]);
        if (live && (FULL || w[j].has1))
          *reinterpret_cast<Pack<T, V>*>(out + w[j].o1) = pack<T, V>(y[1]);
      }
    }
    head += R;
    out += R * a.D;
    turned = now.next();
  }
}

// As the forward, but a CTA stays with one side (the first ctas_q CTAs with q)
// and keeps its lanes' sums of dgamma in registers over all its items; they go
// to part[CTA][D], added up by qk_dgamma_kernel in a fixed order.  A token's
// heads are cut into `chunks` items of `chunk` groups.
template <typename T, int V, int G, int NS, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, NS == 1 ? kBackwardPerSm : 1)
    qk_backward_kernel(const QkNormRopeArgs a, int ctas_q, int chunk_q, int chunks_q, int chunk_k,
                       int chunks_k) {
  pdl_wait();
  pdl_trigger();
  using P = Pairs<V, INTER>;
  using Ring = Rows<T, V, 4 * NS>;
  constexpr int R = 32 / G;
  extern __shared__ __align__(16) uint8_t smem[];
  Ring ring(smem);
  __shared__ float acc[kMaxD];
  const int lane = threadIdx.x % 32, li = lane % G, row = lane / G;
  const bool is_k = static_cast<int>(blockIdx.x) >= ctas_q;
  const Side<T> sd = side_of<T>(a, is_k);
  const int cta = static_cast<int>(blockIdx.x) - (is_k ? ctas_q : 0);
  const int ctas = is_k ? static_cast<int>(gridDim.x) - ctas_q : ctas_q;
  const int groups = (sd.heads + R - 1) / R;
  const int chunk = is_k ? chunk_k : chunk_q, chunks = is_k ? chunks_k : chunks_q;
  const float inv_d = 1.f / static_cast<float>(a.D);
  Slot w[NS];
  float m[NS][2][V];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    w[j] = slot_of<V, INTER, FULL>(li + G * j, a.D, a.rot);
    load_gamma<V>(m[j], sd.gamma, w[j]);
  }
  Walk now(cta * kWarps + threadIdx.x / 32, ctas * kWarps, static_cast<int>(a.T) * chunks, chunk,
           chunks, groups, groups);
  Walk ahead = now;
  bool fresh = true;  // the group ahead begins another token
  const T* x = nullptr;
  const T* dy = nullptr;
  int x_head = 0;
  auto fetch = [&](int stage) {
    if (ahead.live()) {
      if (fresh) {
        x_head = ahead.g * R + row;
        x = sd.x + ahead.t * sd.ld_x + x_head * a.D;
        dy = sd.g + ahead.t * sd.ld_g + x_head * a.D;
      }
      const bool live = x_head < sd.heads;
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        ring.fetch(stage, 4 * j, x + w[j].o0, live && (FULL || w[j].has0));
        ring.fetch(stage, 4 * j + 1, x + w[j].o1, live && (FULL || w[j].has1));
        ring.fetch(stage, 4 * j + 2, dy + w[j].o0, live && (FULL || w[j].has0));
        ring.fetch(stage, 4 * j + 3, dy + w[j].o1, live && (FULL || w[j].has1));
      }
      x_head += R;
      x += R * a.D;
      dy += R * a.D;
      fresh = ahead.next();
    }
    Ring::commit();
  };
  if (Ring::ASYNC)
    for (int s = 0; s < Ring::STAGES; ++s) fetch(s);
  float dg[NS][2][V] = {};
  float cs[NS][V], sn[NS][V];
  long long tr = -1;
  bool turned = true;  // another token than the last group's
  T* out = nullptr;
  int head = 0;
  for (int stage = 0; now.live(); stage = stage + 1 == Ring::STAGES ? 0 : stage + 1) {
    if (turned) {
      head = now.g * R + row;
      out = sd.out + now.t * sd.ld_out + head * a.D;
      tr = table_row(a, now.t);
      if (tr >= 0) {
#pragma unroll
        for (int j = 0; j < NS; ++j) load_trig<V>(cs[j], sn[j], a, tr, li + G * j, w[j]);
      } else if (lane == 0) {
        atomicCAS(a.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
      }
    }
    if (!Ring::ASYNC) fetch(stage);
    Ring::wait();
    float v[NS][2][V], dn[NS][2][V];
    float ss = 0.f, gx = 0.f;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      float d[2][V];
      ring.read(stage, 4 * j, v[j][0]);
      ring.read(stage, 4 * j + 1, v[j][1]);
      ring.read(stage, 4 * j + 2, d[0]);
      ring.read(stage, 4 * j + 3, d[1]);
      if (FULL || w[j].turns) {  // the rotation transposed
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float da = d[P::vec_a(i)][P::at_a(i)], db = d[P::vec_b(i)][P::at_b(i)];
          dn[j][P::vec_a(i)][P::at_a(i)] = fmaf(da, cs[j][i], db * sn[j][i]);
          dn[j][P::vec_b(i)][P::at_b(i)] = fmaf(db, cs[j][i], -da * sn[j][i]);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < V; ++i) dn[j][h][i] = d[h][i];
      }
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < V; ++i) {
          ss = fmaf(v[j][h][i], v[j][h][i], ss);
          gx = fmaf(dn[j][h][i] * m[j][h][i], v[j][h][i], gx);
        }
    }
    if (Ring::ASYNC) fetch(stage);
    const bool live = head < sd.heads;
    ss = group_sum<G>(ss);
    gx = group_sum<G>(gx);
    if (tr < 0) {  // outside the table: no gradient
      const float zero[V] = {};
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        if (live && w[j].has0) *reinterpret_cast<Pack<T, V>*>(out + w[j].o0) = pack<T, V>(zero);
        if (live && w[j].has1) *reinterpret_cast<Pack<T, V>*>(out + w[j].o1) = pack<T, V>(zero);
      }
    } else {
      const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
      const float k = r * (r * r * gx * inv_d);
#pragma unroll
      for (int j = 0; j < NS; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float rd = r * dn[j][h][i];
            dg[j][h][i] = fmaf(rd, v[j][h][i], dg[j][h][i]);
            dn[j][h][i] = fmaf(rd, m[j][h][i], -v[j][h][i] * k);
          }
        if (live && (FULL || w[j].has0))
          *reinterpret_cast<Pack<T, V>*>(out + w[j].o0) = pack<T, V>(dn[j][0]);
        if (live && (FULL || w[j].has1))
          *reinterpret_cast<Pack<T, V>*>(out + w[j].o1) = pack<T, V>(dn[j][1]);
      }
    }
    head += R;
    out += R * a.D;
    turned = now.next();
  }
  // the CTA's sum, warp by warp in order (rows of a warp by shuffles)
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int o = 16; o >= G; o >>= 1)
          dg[j][h][i] += __shfl_xor_sync(0xffffffffu, dg[j][h][i], o);
  for (int wp = 0; wp < kWarps; ++wp) {
    if (threadIdx.x / 32 == wp && row == 0) {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          if (w[j].has0) acc[w[j].o0 + i] = (wp == 0 ? 0.f : acc[w[j].o0 + i]) + dg[j][0][i];
          if (w[j].has1) acc[w[j].o1 + i] = (wp == 0 ? 0.f : acc[w[j].o1 + i]) + dg[j][1][i];
        }
      }
    }
    __syncthreads();
  }
  float* part = a.part + static_cast<long long>(blockIdx.x) * a.D;
  for (int i = threadIdx.x; i < a.D; i += kThreads) part[i] = acc[i];
}

// dgamma[i] = sum over the CTAs' partial sums in a fixed order: 32 features a
// CTA, its eight warps take every eighth partial sum each.  In fp32: the few
// hundred additions lose less than the partial sums did (in fp64, which this
// GPU runs at 1/64 of the rate, the launch took 14 us instead of 2).
__global__ void __launch_bounds__(kThreads)
    qk_dgamma_kernel(const float* part, int ctas_q, int ctas_k, int D, float* dgamma_q,
                     float* dgamma_k) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sums[kWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i = blockIdx.x * 32 + lane;
  const bool is_k = blockIdx.y != 0;
  float* out = is_k ? dgamma_k : dgamma_q;
  if (out == nullptr) return;
  const float* p = part + (is_k ? static_cast<long long>(ctas_q) * D : 0) + i;
  const int ctas = is_k ? ctas_k : ctas_q;
  float v = 0.f;
  if (i < D)
#pragma unroll 8
    for (int c = warp; c < ctas; c += kWarps) v += p[static_cast<long long>(c) * D];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || i >= D) return;
#pragma unroll
  for (int w = 1; w < kWarps; ++w) v += sums[w][lane];
  out[i] = v;
}

// CTAs of the backward pass, shared out between q and k by their heads (fixed
// by the sizes: the sums' order is the same from run to run).
struct BackwardGrid {
  int q, k;
  BackwardGrid(int hq, int hk, long long T) {
    const long long rows = T * (hq + hk);
    const long long most = std::max<long long>(2, std::min<long long>(kBackwardPerSm * sm_count(),
                                                                     rows / kWarps + 2));
    k = hk == 0 ? 0
                : static_cast<int>(std::max<long long>(1, (most * hk + (hq + hk) / 2) / (hq + hk)));
    q = static_cast<int>(std::max<long long>(1, most - k));
  }
};

// A token's groups cut into `count` items of `size` (the last may have fewer,
// none is empty): as many as give every warp about eight, so that the last
// round of items is a small part of the whole.  T * count fits 32 bits.
struct Chunks {
  int size, count;
  Chunks(long long T, int groups, long long warps) {
    const long long wanted = std::max<long long>(1, 8 * warps / std::max<long long>(T, 1));
    const int most = static_cast<int>(std::min<long long>(std::max(groups, 1), wanted));
    size = (std::max(groups, 1) + most - 1) / most;
    count = (std::max(groups, 1) + size - 1) / size;
  }
};

// Lets a kernel use more shared memory than the default limit of 48 KiB for
// all of it; `done`: the kernel's own flags, one per device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (bytes <= 32 * 1024 || done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

template <typename T, int V, int G, int NS, bool INTER, bool FULL>
cudaError_t forward(const QkNormRopeArgs& a, cudaStream_t s) {
  constexpr int R = 32 / G;
  const int groups = (a.hq + R - 1) / R + (a.hk + R - 1) / R;
  const long long warps = static_cast<long long>(kForwardPerSm) * kWarps * sm_count();
  const Chunks cut(a.T, groups, warps);
  const long long items = a.T * cut.count;
  const int grid = static_cast<int>(
      std::min<long long>((items + kWarps - 1) / kWarps, warps / kWarps));
  auto* kernel = qk_forward_kernel<T, V, G, NS, INTER, FULL>;
  constexpr int smem = Rows<T, V, 2 * NS>::SMEM;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, s, a, cut.size, cut.count);
}

template <typename T, int V, int G, int NS, bool INTER, bool FULL>
cudaError_t backward(const QkNormRopeArgs& a, const BackwardGrid& n, cudaStream_t s) {
  constexpr int R = 32 / G;
  const Chunks cq(a.T, (a.hq + R - 1) / R, static_cast<long long>(kWarps) * n.q);
  const Chunks ck(a.T, (a.hk + R - 1) / R, static_cast<long long>(kWarps) * n.k);
  auto* kernel = qk_backward_kernel<T, V, G, NS, INTER, FULL>;
  constexpr int smem = Rows<T, V, 4 * NS>::SMEM;
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(n.q + n.k), dim3(kThreads), smem, s, a, n.q, cq.size,
                    cq.count, ck.size, ck.count);
}

// The widest vectors (at most 16 bytes) that the sizes, pointers and strides
// allow: halves of the rotated part and whole rows in multiples of V, fp32
// tables and gamma on 16 bytes where V >= 4.
template <typename T>
int vector_width(const QkNormRopeArgs& a) {
  uintptr_t bits = 0, wide = 0;
  for (const void* p : {a.q, a.gq, static_cast<const void*>(a.out_q)})
    bits |= reinterpret_cast<uintptr_t>(p);
  bits |= static_cast<uintptr_t>(a.ld_q | a.ld_gq | a.ld_out_q) * sizeof(T);
  if (a.hk > 0) {
    for (const void* p : {a.k, a.gk, static_cast<const void*>(a.out_k)})
      bits |= reinterpret_cast<uintptr_t>(p);
    bits |= static_cast<uintptr_t>(a.ld_k | a.ld_gk | a.ld_out_k) * sizeof(T);
  }
  for (const float* p : {a.gamma_q, a.gamma_k}) wide |= reinterpret_cast<uintptr_t>(p);
  if (a.rot > 0)
    wide |= reinterpret_cast<uintptr_t>(a.cos_table) | reinterpret_cast<uintptr_t>(a.sin_table);
  for (int v = static_cast<int>(16 / sizeof(T)); v > 1; v /= 2)
    if (a.D % v == 0 && (a.rot / 2) % v == 0 && bits % (v * sizeof(T)) == 0 &&
        (v < 4 || wide % 16 == 0))
      return v;
  return 1;
}

// Slots of a row: whole pairs of vectors of the rotated part, then of the rest.
int slots_of(const QkNormRopeArgs& a, int v) { return a.rot / 2 / v + (a.D - a.rot + 2 * v - 1) / (2 * v); }

// call(V, G, NS) for the row's slots: G lanes, a power of two, of NS slots each.
#define QK_BY_SLOTS(slots, call)                                             \
  do {                                                                       \
    if (v == 8) {                                                            \
      if ((slots) <= 4) return call(8, 4, 1);                                \
      if ((slots) <= 8) return call(8, 8, 1);                                \
      if ((slots) <= 16) return call(8, 16, 1);                              \
      return call(8, 32, 1);                                                 \
    }                                                                        \
    if (v == 4) {                                                            \
      if ((slots) <= 8) return call(4, 8, 1);                                \
      if ((slots) <= 16) return call(4, 16, 1);                              \
      if ((slots) <= 32) return call(4, 32, 1);                              \
      return call(4, 32, 2);                                                 \
    }                                                                        \
    if (v == 2) {                                                            \
      if ((slots) <= 32) return call(2, 32, 1);                              \
      return call(2, 32, 4);                                                 \
    }                                                                        \
    return call(1, 32, 8);                                                   \
  } while (0)

// Both passes (n null: forward), by the pairs' layout and, for the widest
// vectors, by whether every lane has a whole turning slot.
template <typename T, int V, int G, int NS>
cudaError_t by_layout(const QkNormRopeArgs& a, const BackwardGrid* n, cudaStream_t s) {
  if constexpr (sizeof(T) * V == 16 && NS == 1) {
    if (a.rot == a.D && slots_of(a, V) == G) {
      if (n == nullptr)
        return a.interleaved ? forward<T, V, G, NS, true, true>(a, s)
                             : forward<T, V, G, NS, false, true>(a, s);
      return a.interleaved ? backward<T, V, G, NS, true, true>(a, *n, s)
                           : backward<T, V, G, NS, false, true>(a, *n, s);
    }
  }
  if (n == nullptr)
    return a.interleaved ? forward<T, V, G, NS, true, false>(a, s)
                         : forward<T, V, G, NS, false, false>(a, s);
  return a.interleaved ? backward<T, V, G, NS, true, false>(a, *n, s)
                       : backward<T, V, G, NS, false, false>(a, *n, s);
}

template <typename T>
cudaError_t run(const QkNormRopeArgs& a, const BackwardGrid* n, cudaStream_t s) {
  const int v = vector_width<T>(a);
#define CALL(V, G, NS) by_layout<T, sizeof(T) * V <= 16 ? V : 4, G, NS>(a, n, s)
  QK_BY_SLOTS(slots_of(a, v), CALL);
#undef CALL
}

}  // namespace

cudaError_t qk_norm_rope_forward(const QkNormRopeArgs& a, bool is_bf16, cudaStream_t s) {
  prof_begin("qk_norm_rope", s);
  const cudaError_t e = is_bf16 ? run<__nv_bfloat16>(a, nullptr, s) : run<float>(a, nullptr, s);
  prof_end("qk_norm_rope", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

size_t qk_norm_rope_scratch(int hq, int hk, int D, long long T) {
  const BackwardGrid n(hq, hk, T);
  return static_cast<size_t>(n.q + n.k) * D * sizeof(float);
}

cudaError_t qk_norm_rope_backward(const QkNormRopeArgs& a, bool is_bf16, cudaStream_t s) {
  const BackwardGrid n(a.hq, a.hk, a.T);
  prof_begin("qk_norm_rope_bwd", s);
  cudaError_t e = is_bf16 ? run<__nv_bfloat16>(a, &n, s) : run<float>(a, &n, s);
  prof_end("qk_norm_rope_bwd", s);
  if (e != cudaSuccess) return e;
  if (a.dgamma_q == nullptr && a.dgamma_k == nullptr) return cudaGetLastError();
  prof_begin("qk_dgamma", s);
  e = launch_pdl(qk_dgamma_kernel, dim3((a.D + 31) / 32, a.hk > 0 ? 2 : 1),
                 dim3(kThreads), 0, s, static_cast<const float*>(a.part), n.q, n.k, a.D,
                 a.dgamma_q, a.dgamma_k);
  prof_end("qk_dgamma", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace poetx
