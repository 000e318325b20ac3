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
// the sums, and a warp works on 32 / G heads of a token at once: a group.  What
// bounds it is memory traffic, 2 (forward) or 3 (backward) passes over q and k:
// 16384 tokens of 40 heads of 128, bf16, take 55.8 us forward (6.0 TB/s) and 84.2
// backward (6.0), in fp32 half as many tokens 54 and 82.7.  (Alternatives below
// were measured before the sums of dgamma took their present form, 4 us less.)
#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <type_traits>

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

// Slot s of a row: the vectors at o0 and o1, apart by half of the rotated part,
// so that the lanes' vectors are next to each other; `turns`: its pairs are
// rotated, with V table entries from e0 and e1, a half of them each.
struct Slot {
  int o0, o1, e0, e1;
  bool turns, has0, has1;
};

// FULL: every lane has whole slots and all of them turn.
template <int V, bool INTER, bool FULL>
__device__ __forceinline__ Slot slot_of(int s, int D, int rot) {
  Slot w;
  const int nrot = rot / 2 / V;
  w.turns = FULL || s < nrot;
  if (w.turns) {
    const bool pair = INTER && V == 1;
    w.o0 = pair ? 2 * s : s * V;
    w.o1 = pair ? 2 * s + 1 : rot / 2 + s * V;
    w.e0 = INTER ? w.o0 / 2 : w.o0;
    w.e1 = INTER ? w.o1 / 2 : w.o0 + V / 2;
  } else {
    w.o0 = rot + (s - nrot) * 2 * V;
    w.o1 = w.o0 + V;
    w.e0 = w.e1 = 0;
  }
  w.has0 = FULL || w.o0 < D;
  w.has1 = FULL || w.o1 < D;
  return w;
}

// A slot's values as the arithmetic holds them: V pairs, members a and b apart,
// two pairs to a register pair (fma.rn.f32x2; singly for V = 1).  Half by half, a
// is the slot's first vector and b its second; interleaved, the vectors hold
// whole pairs (a0 b0 a1 b1 ..).
template <int V>
struct Vals {
  using E = std::conditional_t<(V > 1), f32x2, float>;
  static constexpr int N = V > 1 ? V / 2 : 1;
  E a[N], b[N];
};

__device__ __forceinline__ void join(f32x2& o, float lo, float hi) { o = f32x2_of(lo, hi); }
__device__ __forceinline__ void join(float& o, float lo, float) { o = lo; }
__device__ __forceinline__ void part(f32x2 v, float& lo, float& hi) { f32x2_split(v, lo, hi); }
__device__ __forceinline__ void part(float v, float& lo, float&) { lo = v; }
__device__ __forceinline__ f32x2 mul(f32x2 a, f32x2 b) { return f32x2_mul(a, b); }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ f32x2 mad(f32x2 a, f32x2 b, f32x2 c) { return f32x2_fma(a, b, c); }
__device__ __forceinline__ float mad(float a, float b, float c) { return fmaf(a, b, c); }
template <typename E>
__device__ __forceinline__ E both(float x) {
  E o;
  join(o, x, x);
  return o;
}
__device__ __forceinline__ float total(f32x2 v) {
  float lo, hi;
  f32x2_split(v, lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float total(float v) { return v; }

// The two vectors of a slot as values, and back.
template <int V, bool INTER>
__device__ __forceinline__ Vals<V> values(const float (&x)[2][V]) {
  Vals<V> o;
  auto at = [&](int i) { return i < V ? x[0][i] : x[1][i - V]; };  // of both, end to end
#pragma unroll
  for (int j = 0; j < Vals<V>::N; ++j) {
    if (INTER) {
      join(o.a[j], at(4 * j), V > 1 ? at(4 * j + 2) : 0.f);
      join(o.b[j], at(4 * j + 1), V > 1 ? at(4 * j + 3) : 0.f);
    } else {
      join(o.a[j], at(2 * j), V > 1 ? at(2 * j + 1) : 0.f);
      join(o.b[j], at(V + 2 * j), V > 1 ? at(V + 2 * j + 1) : 0.f);
    }
  }
  return o;
}
template <int V, bool INTER>
__device__ __forceinline__ void vectors(float (&x)[2][V], const Vals<V>& o) {
  auto at = [&](int i) -> float& { return i < V ? x[0][i] : x[1][i - V]; };
  float unused;
#pragma unroll
  for (int j = 0; j < Vals<V>::N; ++j) {
    if (INTER) {
      part(o.a[j], at(4 * j), V > 1 ? at(4 * j + 2) : unused);
      part(o.b[j], at(4 * j + 1), V > 1 ? at(4 * j + 3) : unused);
    } else {
      part(o.a[j], at(2 * j), V > 1 ? at(2 * j + 1) : unused);
      part(o.b[j], at(V + 2 * j), V > 1 ? at(V + 2 * j + 1) : unused);
    }
  }
}

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
// reads only its own vectors, so the ring needs no barrier.  Two groups of 16
// warps keep the memory busy; four are slower (16384 x 40 heads of 128: forward
// 62 against 55.5 us, backward 97.6 against 88), as are the next group in
// registers and 24 warps of 80 registers (forward 83).  Vectors of two bytes
// cannot be copied this way and are read when needed.
template <typename T, int V, int N>
struct Rows {
  static constexpr int BYTES = sizeof(T) * V;
  static constexpr bool ASYNC = BYTES >= 4;
  static constexpr int STAGES = ASYNC ? 2 : 1;
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
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // The oldest of the STAGES groups has arrived.
  __device__ __forceinline__ static void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
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
template <int V, bool INTER>
__device__ __forceinline__ Vals<V> load_gamma(const float* gamma, const Slot& w) {
  float m[2][V];
#pragma unroll
  for (int i = 0; i < V; ++i) m[0][i] = m[1][i] = 1.f;
  if (gamma != nullptr) {
    if (w.has0) load_f32<V>(m[0], gamma + w.o0);
    if (w.has1) load_f32<V>(m[1], gamma + w.o1);
  }
  return values<V, INTER>(m);
}

// A slot's table entries (1 and 0 where nothing turns).
template <int V>
struct Trig {
  using E = typename Vals<V>::E;
  static constexpr int N = Vals<V>::N;
  E c[N], s[N];
};

// cos, sin: the token's rows in shared memory.
template <int V>
__device__ __forceinline__ Trig<V> load_trig(const float* cos, const float* sin, const Slot& w) {
  constexpr int H = V > 1 ? V / 2 : 1;
  float c[V], s[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = 1.f, s[i] = 0.f;
  if (w.turns) {
#pragma unroll
    for (int i = 0; i < V; i += H) {
      const int e = i == 0 ? w.e0 : w.e1;
      memcpy(c + i, __builtin_assume_aligned(cos + e, 4 * H), 4 * H);
      memcpy(s + i, __builtin_assume_aligned(sin + e, 4 * H), 4 * H);
    }
  }
  Trig<V> t;
#pragma unroll
  for (int j = 0; j < Trig<V>::N; ++j) {
    constexpr int H = V > 1 ? 1 : 0;  // the second of two pairs
    join(t.c[j], c[2 * j], c[2 * j + H]);
    join(t.s[j], s[2 * j], s[2 * j + H]);
  }
  return t;
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
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

enum class New { nothing, side, token };

// A warp's way through its share of all groups (T tokens' `groups` each, the
// first iq of them q's, the rest k's): consecutive ones, so that the shares
// differ by one group at most and a token's table row serves all its heads.
// (Whole tokens in turn: backward 97 us for 16384 tokens, 16.8 for 1024; in
// shares 88 and 14.4.)
struct Walk {
  int left, iq, groups;
  int t, g, end;  // token t's group g of [0, end) of a side
  bool is_k;

  __device__ __forceinline__ Walk(int warp, int warps, long long T, int iq_, int groups_)
      : iq(iq_), groups(groups_) {
    const long long total = T * groups, first = total * warp / warps;
    left = static_cast<int>(total * (warp + 1) / warps - first);
    t = static_cast<int>(first / groups);
    g = static_cast<int>(first - static_cast<long long>(t) * groups);
    is_k = g >= iq;
    end = is_k ? groups - iq : iq;
    if (is_k) g -= iq;
  }
  __device__ __forceinline__ bool live() const { return left > 0; }
  // To the next group; what is new there.
  __device__ __forceinline__ New next() {
    --left;
    if (++g < end) return New::nothing;
    g = 0;
    if (!is_k && groups > iq) {
      is_k = true;
      end = groups - iq;
      return New::side;
    }
    is_k = false;
    end = iq;
    ++t;
    return New::token;
  }
};

// The table rows of a warp's tokens on their way to shared memory, with the
// groups that they turn: SLOTS tokens (one is started per group at most, and a
// row is read before the group STAGES later is fetched).  Positions are read 32
// tokens at a time.  (With loads at the token's first group
// instead, a warp stood still twice per token for a trip to memory: backward 98
// us instead of 88, heads of 64 65 instead of 52.)
template <int V, int SLOTS>
struct Tables {
  static constexpr int bytes(int half) {
    return kWarps * SLOTS * 2 * ((half + 3) & ~3) * 4;
  }

  const QkNormRopeArgs& a;
  float* rows;  // this warp's slots: a row of each table
  int half, pitch, count, slot, ahead_slot;
  int position;  // of the lane's token among 32; -1: outside the table
  uint32_t valid;

  __device__ __forceinline__ Tables(const QkNormRopeArgs& a_, uint8_t* smem)
      : a(a_), half(a_.rot / 2), pitch((a_.rot / 2 + 3) & ~3), count(0), slot(SLOTS - 1),
        ahead_slot(SLOTS - 1), position(-1), valid(0) {
    rows = reinterpret_cast<float*>(smem) + (threadIdx.x / 32) * SLOTS * 2 * pitch;
  }
  __device__ __forceinline__ void positions(const Walk& w) {
    const long long t = w.t + static_cast<long long>(threadIdx.x % 32);
    position = -1;
    if (t < a.T) {
      const int p = a.rot == 0 ? 0 : a.positions != nullptr ? a.positions[t] : static_cast<int>(t);
      if (a.rot == 0 || (p >= 0 && p < a.table_rows)) position = p;
    }
  }
  // The rows of the token that w enters.
  __device__ __forceinline__ void fetch(const Walk& w) {
    if (count == 32) {
      positions(w);
      count = 0;
    }
    const int p = __shfl_sync(0xffffffffu, position, count);
    __syncwarp();  // every lane has read the slot (a shuffle orders no memory)
    ++count;
    ahead_slot = ahead_slot + 1 == SLOTS ? 0 : ahead_slot + 1;
    valid = p >= 0 ? valid | 1u << ahead_slot : valid & ~(1u << ahead_slot);
    if (p < 0) return;
    float* to = rows + ahead_slot * 2 * pitch;
    const float* cos = a.cos_table + static_cast<long long>(p) * half;
    const float* sin = a.sin_table + static_cast<long long>(p) * half;
    constexpr int W = V % 4 == 0 ? 4 : 1;  // floats per copy (vector_width: 16-byte rows)
    for (int i = (threadIdx.x % 32) * W; i < 2 * half; i += 32 * W) {
      const float* from = i < half ? cos + i : sin + (i - half);
      const uint32_t dst = smem_u32(to + (i < half ? i : i - half + pitch));
      if constexpr (W == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(from) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(from) : "memory");
    }
  }
  // To the rows of the next token; whether its position is in the table.
  __device__ __forceinline__ bool enter() {
    slot = slot + 1 == SLOTS ? 0 : slot + 1;
    return (valid >> slot & 1u) != 0;
  }
  __device__ __forceinline__ const float* cos() const { return rows + slot * 2 * pitch; }
  __device__ __forceinline__ const float* sin() const { return cos() + pitch; }
};

// Groups of 32 / G heads of one token (q's, then k's), NS slots per lane.  gamma
// and the table row are multiplied once per token and side, so that a value costs
// three operations: y_a = r (x_a (g_a c) - x_b (g_b s)).
template <typename T, int V, int G, int NS, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, NS == 1 ? kForwardPerSm : 1)
    qk_forward_kernel(const QkNormRopeArgs a) {
  pdl_wait();
  pdl_trigger();
  using W = Vals<V>;
  using E = typename W::E;
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
           static_cast<int>(gridDim.x) * kWarps, a.T, iq, groups);
  Walk ahead = now;
  Tables<V, Ring::STAGES> tables(a, smem + Ring::SMEM);
  tables.positions(now);
  New fresh = New::token;  // at the group ahead
  const T* x = nullptr;
  int x_head = 0;
  auto fetch = [&](int stage) {
    if (ahead.live()) {
      if (fresh != New::nothing) {
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
      if (fresh == New::token) tables.fetch(ahead);
      x_head += R;
      x += R * a.D;
      fresh = ahead.next();
    }
    Ring::commit();
  };
  if (Ring::ASYNC)
    for (int s = 0; s < Ring::STAGES; ++s) fetch(s);
  // a value's output is r (own x + cross (its partner's x)); cross is indexed by
  // the value that it multiplies
  W own[NS], cross[NS];
  const E minus = both<E>(-1.f);
  bool valid = false;
  New turned = New::token;
  T* out = nullptr;
  int head = 0;
  for (int stage = 0; now.live(); stage = stage + 1 == Ring::STAGES ? 0 : stage + 1) {
    if (!Ring::ASYNC) fetch(stage);
    Ring::wait();
    if (turned != New::nothing) {
      head = now.g * R + row;
      out = static_cast<T*>(now.is_k ? a.out_k : a.out_q) +
            now.t * (now.is_k ? a.ld_out_k : a.ld_out_q) + head * a.D;
      if (turned == New::token) {
        valid = tables.enter();
        __syncwarp();  // the other lanes' copies of the rows
      }
      if (valid) {
        const float* gamma = now.is_k ? a.gamma_k : a.gamma_q;
#pragma unroll
        for (int j = 0; j < NS; ++j) {
          const Trig<V> t = load_trig<V>(tables.cos(), tables.sin(), w[j]);
          const W m = load_gamma<V, INTER>(gamma, w[j]);
#pragma unroll
          for (int i = 0; i < W::N; ++i) {
            own[j].a[i] = mul(m.a[i], t.c[i]);
            own[j].b[i] = mul(m.b[i], t.c[i]);
            cross[j].a[i] = mul(m.a[i], t.s[i]);
            cross[j].b[i] = mul(m.b[i], mul(minus, t.s[i]));
          }
        }
      } else if (lane == 0) {
        atomicCAS(a.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
      }
    }
    W v[NS];
    E sq_a = both<E>(0.f), sq_b = sq_a;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      float x2[2][V];
      ring.read(stage, 2 * j, x2[0]);
      ring.read(stage, 2 * j + 1, x2[1]);
      v[j] = values<V, INTER>(x2);
#pragma unroll
      for (int i = 0; i < W::N; ++i) {
        sq_a = mad(v[j].a[i], v[j].a[i], sq_a);
        sq_b = mad(v[j].b[i], v[j].b[i], sq_b);
      }
    }
    if (Ring::ASYNC) fetch(stage);
    const bool live = head < (now.is_k ? a.hk : a.hq);
    const float ss = group_sum<G>(total(sq_a) + total(sq_b));
    const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
    if (!valid) {  // outside the table: zeros
      const float zero[V] = {};
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        if (live && w[j].has0) *reinterpret_cast<Pack<T, V>*>(out + w[j].o0) = pack<T, V>(zero);
        if (live && w[j].has1) *reinterpret_cast<Pack<T, V>*>(out + w[j].o1) = pack<T, V>(zero);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        const E rr = both<E>(r);
        W o;
        if (FULL || w[j].turns) {
#pragma unroll
          for (int i = 0; i < W::N; ++i) {
            const E xa = v[j].a[i], xb = v[j].b[i];
            o.a[i] = mul(rr, mad(xa, own[j].a[i], mul(xb, cross[j].b[i])));
            o.b[i] = mul(rr, mad(xb, own[j].b[i], mul(xa, cross[j].a[i])));
          }
        } else {
#pragma unroll
          for (int i = 0; i < W::N; ++i) {
            o.a[i] = mul(rr, mul(v[j].a[i], own[j].a[i]));
            o.b[i] = mul(rr, mul(v[j].b[i], own[j].b[i]));
          }
        }
        float y[2][V];
        vectors<V, INTER>(y, o);
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
// and keeps its lanes' sums of dgamma in registers over all its groups; they go
// to part[CTA][D], added up by qk_dgamma_kernel in a fixed order.  The table
// entries are read from shared memory for every group: in registers they spill.
template <typename T, int V, int G, int NS, bool INTER, bool FULL>
__global__ void __launch_bounds__(kThreads, NS == 1 ? kBackwardPerSm : 1)
    qk_backward_kernel(const QkNormRopeArgs a, int ctas_q) {
  pdl_wait();
  pdl_trigger();
  using W = Vals<V>;
  using E = typename W::E;
  using Ring = Rows<T, V, 4 * NS>;
  constexpr int R = 32 / G;
  extern __shared__ __align__(16) uint8_t smem[];
  Ring ring(smem);
  __shared__ float acc[kWarps][kMaxD];
  const int lane = threadIdx.x % 32, li = lane % G, row = lane / G;
  const bool is_k = static_cast<int>(blockIdx.x) >= ctas_q;
  const Side<T> sd = side_of<T>(a, is_k);
  const int cta = static_cast<int>(blockIdx.x) - (is_k ? ctas_q : 0);
  const int ctas = is_k ? static_cast<int>(gridDim.x) - ctas_q : ctas_q;
  const int groups = (sd.heads + R - 1) / R;
  const float inv_d = 1.f / static_cast<float>(a.D);
  Slot w[NS];
  W m[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    w[j] = slot_of<V, INTER, FULL>(li + G * j, a.D, a.rot);
    m[j] = load_gamma<V, INTER>(sd.gamma, w[j]);
  }
  Walk now(cta * kWarps + threadIdx.x / 32, ctas * kWarps, a.T, groups, groups);
  Walk ahead = now;
  Tables<V, Ring::STAGES> tables(a, smem + Ring::SMEM);
  tables.positions(now);
  New fresh = New::token;  // at the group ahead
  const T* x = nullptr;
  const T* dy = nullptr;
  int x_head = 0;
  auto fetch = [&](int stage) {
    if (ahead.live()) {
      if (fresh != New::nothing) {
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
      if (fresh == New::token) tables.fetch(ahead);
      x_head += R;
      x += R * a.D;
      dy += R * a.D;
      fresh = ahead.next();
    }
    Ring::commit();
  };
  if (Ring::ASYNC)
    for (int s = 0; s < Ring::STAGES; ++s) fetch(s);
  W dg[NS];
#pragma unroll
  for (int j = 0; j < NS; ++j)
#pragma unroll
    for (int i = 0; i < W::N; ++i) dg[j].a[i] = dg[j].b[i] = both<E>(0.f);
  const E minus = both<E>(-1.f);
  bool valid = false;
  New turned = New::token;
  T* out = nullptr;
  int head = 0;
  for (int stage = 0; now.live(); stage = stage + 1 == Ring::STAGES ? 0 : stage + 1) {
    if (!Ring::ASYNC) fetch(stage);
    Ring::wait();
    if (turned != New::nothing) {
      head = now.g * R + row;
      out = sd.out + now.t * sd.ld_out + head * a.D;
      valid = tables.enter();
      __syncwarp();  // the other lanes' copies of the rows
      if (!valid && lane == 0) atomicCAS(a.status, 0, static_cast<int>(POETX_ERR_INVALID_ARG));
    }
    W v[NS], dn[NS];
    E sq_a = both<E>(0.f), sq_b = sq_a, gx_a = sq_a, gx_b = sq_a;
#pragma unroll
    for (int j = 0; j < NS; ++j) {
      float x2[2][V], d2[2][V];
      ring.read(stage, 4 * j, x2[0]);
      ring.read(stage, 4 * j + 1, x2[1]);
      ring.read(stage, 4 * j + 2, d2[0]);
      ring.read(stage, 4 * j + 3, d2[1]);
      v[j] = values<V, INTER>(x2);
      const W d = values<V, INTER>(d2);
      if (valid && (FULL || w[j].turns)) {  // the rotation transposed
        const Trig<V> t = load_trig<V>(tables.cos(), tables.sin(), w[j]);
#pragma unroll
        for (int i = 0; i < W::N; ++i) {
          dn[j].a[i] = mad(d.a[i], t.c[i], mul(d.b[i], t.s[i]));
          dn[j].b[i] = mad(minus, mul(d.a[i], t.s[i]), mul(d.b[i], t.c[i]));
        }
      } else {
        dn[j] = d;
      }
#pragma unroll
      for (int i = 0; i < W::N; ++i) {
        sq_a = mad(v[j].a[i], v[j].a[i], sq_a);
        sq_b = mad(v[j].b[i], v[j].b[i], sq_b);
        gx_a = mad(mul(dn[j].a[i], m[j].a[i]), v[j].a[i], gx_a);
        gx_b = mad(mul(dn[j].b[i], m[j].b[i]), v[j].b[i], gx_b);
      }
    }
    if (Ring::ASYNC) fetch(stage);
    const bool live = head < sd.heads;
    const float ss = group_sum<G>(total(sq_a) + total(sq_b));
    const float gx = group_sum<G>(total(gx_a) + total(gx_b));
    if (!valid) {  // outside the table: no gradient
      const float zero[V] = {};
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        if (live && w[j].has0) *reinterpret_cast<Pack<T, V>*>(out + w[j].o0) = pack<T, V>(zero);
        if (live && w[j].has1) *reinterpret_cast<Pack<T, V>*>(out + w[j].o1) = pack<T, V>(zero);
      }
    } else {
      const float r = rsqrtf(fmaf(ss, inv_d, a.eps));
      const E rr = both<E>(r), k = both<E>(-(r * (r * r * gx * inv_d)));
#pragma unroll
      for (int j = 0; j < NS; ++j) {
        W o;
#pragma unroll
        for (int i = 0; i < W::N; ++i) {
          const E ra = mul(rr, dn[j].a[i]), rb = mul(rr, dn[j].b[i]);
          dg[j].a[i] = mad(ra, v[j].a[i], dg[j].a[i]);
          dg[j].b[i] = mad(rb, v[j].b[i], dg[j].b[i]);
          o.a[i] = mad(ra, m[j].a[i], mul(v[j].a[i], k));
          o.b[i] = mad(rb, m[j].b[i], mul(v[j].b[i], k));
        }
        float y[2][V];
        vectors<V, INTER>(y, o);
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
  // the CTA's sum over its warps in order (rows of a warp by shuffles)
  float sums[NS][2][V];
#pragma unroll
  for (int j = 0; j < NS; ++j) {
    vectors<V, INTER>(sums[j], dg[j]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < V; ++i)
#pragma unroll
        for (int o = 16; o >= G; o >>= 1)
          sums[j][h][i] += __shfl_xor_sync(0xffffffffu, sums[j][h][i], o);
  }
  if (row == 0) {
#pragma unroll
    for (int j = 0; j < NS; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (w[j].has0) acc[threadIdx.x / 32][w[j].o0 + i] = sums[j][0][i];
        if (w[j].has1) acc[threadIdx.x / 32][w[j].o1 + i] = sums[j][1][i];
      }
  }
  __syncthreads();
  float* part = a.part + static_cast<long long>(blockIdx.x) * a.D;
  for (int i = threadIdx.x; i < a.D; i += kThreads) {
    float v = acc[0][i];
#pragma unroll
    for (int wp = 1; wp < kWarps; ++wp) v += acc[wp][i];
    part[i] = v;
  }
}

// dgamma[i] = sum over the CTAs' partial sums in a fixed order: 32 features a
// CTA, its 32 warps take every 32nd partial sum each, all their loads in flight
// (8 warps: backward of 1024 tokens 14.4 us, 32: 12.8; with the CTA's own sums in
// one round instead of warp after warp 10.4).  In fp32: the few hundred additions
// lose less than the partial sums did (in fp64, which this GPU runs at 1/64 of the
// rate, the launch took 14 us instead of 2).
constexpr int kGammaWarps = 32;
constexpr int kGammaFlight = 10;

__global__ void __launch_bounds__(32 * kGammaWarps)
    qk_dgamma_kernel(const float* part, int ctas_q, int ctas_k, int D, float* dgamma_q,
                     float* dgamma_k) {
  pdl_wait();
  pdl_trigger();
  __shared__ float sums[kGammaWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int i = blockIdx.x * 32 + lane;
  const bool is_k = blockIdx.y != 0;
  float* out = is_k ? dgamma_k : dgamma_q;
  if (out == nullptr) return;
  const float* p = part + (is_k ? static_cast<long long>(ctas_q) * D : 0) + i;
  const int ctas = is_k ? ctas_k : ctas_q;
  float v = 0.f;
  if (i < D)
    for (int c0 = warp; c0 < ctas; c0 += kGammaWarps * kGammaFlight) {
      float x[kGammaFlight];
#pragma unroll
      for (int n = 0; n < kGammaFlight; ++n) {
        const int c = c0 + n * kGammaWarps;
        x[n] = c < ctas ? p[static_cast<long long>(c) * D] : 0.f;
      }
#pragma unroll
      for (int n = 0; n < kGammaFlight; ++n) v += x[n];
    }
  sums[warp][lane] = v;
  __syncthreads();
  if (warp != 0 || i >= D) return;
#pragma unroll
  for (int w = 1; w < kGammaWarps; ++w) v += sums[w][lane];
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
  const int grid = static_cast<int>(
      std::min<long long>((a.T * groups + kWarps - 1) / kWarps, warps / kWarps));
  auto* kernel = qk_forward_kernel<T, V, G, NS, INTER, FULL>;
  using Ring = Rows<T, V, 2 * NS>;
  using Rot = Tables<V, Ring::STAGES>;
  const int smem = Ring::SMEM + Rot::bytes(a.rot / 2);
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel),
                                   Ring::SMEM + Rot::bytes(kMaxD / 2), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(grid), dim3(kThreads), smem, s, a);
}

template <typename T, int V, int G, int NS, bool INTER, bool FULL>
cudaError_t backward(const QkNormRopeArgs& a, const BackwardGrid& n, cudaStream_t s) {
  auto* kernel = qk_backward_kernel<T, V, G, NS, INTER, FULL>;
  using Ring = Rows<T, V, 4 * NS>;
  using Rot = Tables<V, Ring::STAGES>;
  const int smem = Ring::SMEM + Rot::bytes(a.rot / 2);
  static std::atomic<bool> done[64];
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel),
                                   Ring::SMEM + Rot::bytes(kMaxD / 2), done);
  if (e != cudaSuccess) return e;
  return launch_pdl(kernel, dim3(n.q + n.k), dim3(kThreads), smem, s, a, n.q);
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
int slots_of(const QkNormRopeArgs& a, int v) {
  return a.rot / 2 / v + (a.D - a.rot + 2 * v - 1) / (2 * v);
}

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
                 dim3(32 * kGammaWarps), 0, s, static_cast<const float*>(a.part), n.q, n.k, a.D,
                 a.dgamma_q, a.dgamma_k);
  prof_end("qk_dgamma", s);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace poetx
