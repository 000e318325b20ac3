// The matrix products of poetx_linear_* in fp32, on the CUDA cores:
//   C[M][N] = act(A B + bias) + residual,  A [M][K], B(k, n) = W[n][k] or W[k][n]
//   (the latter also with A [K][M])
// Tiles of 16 RM x 128, 256 threads, RM x 8 outputs each (RM = 8, 4, 2: the
// tile's rows by the number of tokens), K in steps of 16 (64 for few rows, where
// the bytes in flight count): the next step's operands come into registers
// while this one's FMAs run.  The FMAs are issued
// two at a time (fma.rn.f32x2, pairs along N): what bounds the kernel is the
// FMA rate, and issue slots are what a plain FMA loop lacks for its loads.
// Every output sums K in order (within a K slice).
//
// Up to 16 tokens (FLAT): tiles of 8 x 128, every thread all 8 rows of 8
// columns for every 16th k, added up over the threads at the end.  The tile's
// share of the weight is then read from shared memory once and not 16 times,
// which bounded the other form (4096 x 4096, one token: 62 us).
//
// Few tiles: K is split over a cluster of up to 8 CTAs (any number; powers of two
// in the FLAT form) whose partial tiles are added through distributed shared
// memory, in rank order, rank r finishing the r-th share of the rows.
#include <algorithm>
#include <atomic>

#include "internal.h"
#include "linear.h"
#include "linear_fp32.cuh"
#include "ptx.cuh"

namespace poetx {
namespace {

constexpr int kThreads = 256;
constexpr int kTN = 128;
constexpr int kLdb = kTN + 4;  // rows of the staged tiles start on 16 bytes
constexpr int kMaxSplits = 8;

struct SimtArgs {
  const float* A;
  const float* B;
  Fp32Epilogue epi;
  long long M, lda;
  int N, K, splits, k_slice;
  const int* all_rows;   // null: every row; otherwise every row where it is not 0,
  const int* row_flags;  // and else the rows with one of their `segs` flags set
  int segs;
  bool vec_a, vec_b;  // 16-byte rows of A, of B
};

template <int RM, bool FLAT>
struct Shape {
  static constexpr int TM = FLAT ? RM : 16 * RM;
  static constexpr int TK = FLAT || RM < 4 ? 64 : RM < 8 ? 32 : 16;
  static constexpr int LDA = TM + 4;
  static constexpr int STAGE = TK * (LDA + kLdb) * 4;  // one K step of both operands
  static constexpr int PART = (FLAT ? 4 : 1) * TM * kLdb * 4;  // partial tiles, over the stages
  static constexpr int SMEM = 2 * STAGE > PART ? 2 * STAGE : PART;
};

// Four consecutive floats at row r, from column c, of a [rows][cols] array;
// zeros outside.
__device__ __forceinline__ float4 load4(const float* p, long long r, long long rows, int c,
                                        int cols, long long ld, bool vec) {
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r >= rows) return v;
  const float* q = p + r * ld + c;
  if (vec && c + 3 < cols) return __ldg(reinterpret_cast<const float4*>(q));
  if (c < cols) v.x = __ldg(q);
  if (c + 1 < cols) v.y = __ldg(q + 1);
  if (c + 2 < cols) v.z = __ldg(q + 2);
  if (c + 3 < cols) v.w = __ldg(q + 3);
  return v;
}

// Where piece e of a [ROWS][4 KQ] operand step lies: its row and its quad of K.
// Long steps: neighbouring lanes take the two halves of a 32-byte sector, then
// the next row, so that the transposed stores to rows of a multiple of 4 floats
// meet 32 different banks (4096 x 4096, one token: 31 -> 23 us).  Short steps: a
// row's four quads side by side (two lanes a bank).
template <int ROWS, int KQ>
__device__ __forceinline__ void piece(int e, int& row, int& quad) {
  if (KQ <= 4) {
    row = e / KQ;
    quad = e % KQ;
    return;
  }
  constexpr int RL = ROWS < 16 ? ROWS : 16;
  const int low = e / 2 % RL, rest = e / (2 * RL);
  quad = rest % (KQ / 2) * 2 + e % 2;
  row = rest / (KQ / 2) * RL + low;
}

__device__ __forceinline__ bool flagged(const SimtArgs& p, long long m) {
  int bad = 0;
  for (int i = 0; i < p.segs; ++i) bad |= p.row_flags[m * p.segs + i];
  return bad != 0;
}

__device__ __forceinline__ void finish(const SimtArgs& p, long long m, int n, float4 acc) {
  if (m >= p.M || n >= p.N) return;
  if (p.all_rows != nullptr && *p.all_rows == 0 && !flagged(p, m)) return;
  finish4(p.epi, m, n, acc);
}

// Grid: x = N tile * splits + slice (a cluster along x), y = row tile.
// A_KM: A is [K][M].
template <int RM, bool A_KM, bool B_KN, bool FLAT>
__global__ void __launch_bounds__(kThreads, 2) linear_simt_kernel(const SimtArgs p) {
  using S = Shape<RM, FLAT>;
  constexpr int TM = S::TM, LDA = S::LDA, kTK = S::TK;
  constexpr int KQ = kTK / 4;  // 4-wide pieces of a row's K step
  constexpr int VEC = RM >= 4 ? 4 : RM;  // consecutive rows of a thread
  extern __shared__ __align__(16) float smem[];
  pdl_wait();
  pdl_trigger();
  if (p.all_rows != nullptr && *p.all_rows == 0) {
    // the same for all CTAs of a cluster: they have the same rows
    const long long m = static_cast<long long>(blockIdx.y) * S::TM + threadIdx.x;
    if (!__syncthreads_or(threadIdx.x < S::TM && m < p.M && flagged(p, m))) return;
  }
  const int slice = static_cast<int>(blockIdx.x) % p.splits;
  const int n0 = static_cast<int>(blockIdx.x) / p.splits * kTN;
  const long long m0 = static_cast<long long>(blockIdx.y) * TM;
  const int k0 = slice * p.k_slice, k1 = min(p.K, k0 + p.k_slice);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int tx = lane % 8 + 8 * (warp % 2), ty = lane / 8 + 4 * (warp / 2);

  constexpr int QA = TM * kTK / 4;                        // 4-wide pieces of A's step
  constexpr int NA = (QA + kThreads - 1) / kThreads;      // of this thread
  constexpr int NB = kTN * kTK / 4 / kThreads;
  float4 ra[NA], rb[NB];
  auto fetch = [&](int k) {
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int e = threadIdx.x + q * kThreads;
      ra[q] = make_float4(0.f, 0.f, 0.f, 0.f);
      int row, quad;
      piece<TM, KQ>(e, row, quad);
      if (QA % kThreads == 0 || e < QA)
        ra[q] = A_KM ? load4(p.A, k + e / (TM / 4), k1, static_cast<int>(m0) + e % (TM / 4) * 4,
                             static_cast<int>(p.M), p.lda, p.vec_a)
                     : load4(p.A, m0 + row, p.M, k + quad * 4, k1, p.lda, p.vec_a);
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int e = threadIdx.x + q * kThreads;
      int row, quad;
      piece<kTN, KQ>(e, row, quad);
      rb[q] = B_KN ? load4(p.B, k + e / 32, k1, n0 + e % 32 * 4, p.N, p.N, p.vec_b)
                   : load4(p.B, n0 + row, p.N, k + quad * 4, k1, p.K, p.vec_b);
    }
  };
  auto stage = [&](float* as, float* bs) {
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      const int e = threadIdx.x + q * kThreads;
      if (A_KM && (QA % kThreads == 0 || e < QA)) {
        *reinterpret_cast<float4*>(as + e / (TM / 4) * LDA + e % (TM / 4) * 4) = ra[q];
      } else if (QA % kThreads == 0 || e < QA) {
        int row, quad;
        piece<TM, KQ>(e, row, quad);
        float* d = as + quad * 4 * LDA + row;
        d[0] = ra[q].x, d[LDA] = ra[q].y, d[2 * LDA] = ra[q].z, d[3 * LDA] = ra[q].w;
      }
    }
#pragma unroll
    for (int q = 0; q < NB; ++q) {
      const int e = threadIdx.x + q * kThreads;
      if (B_KN) {
        *reinterpret_cast<float4*>(bs + e / 32 * kLdb + e % 32 * 4) = rb[q];
      } else {
        int row, quad;
        piece<kTN, KQ>(e, row, quad);
        float* d = bs + quad * 4 * kLdb + row;
        d[0] = rb[q].x, d[kLdb] = rb[q].y, d[2 * kLdb] = rb[q].z, d[3 * kLdb] = rb[q].w;
      }
    }
  };

  f32x2 acc[RM][4];
#pragma unroll
  for (int i = 0; i < RM; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0ull;  // two zeros
  if (k0 < k1) {
    fetch(k0);
    stage(smem, smem + kTK * LDA);
  }
  __syncthreads();
  int buf = 0;
  for (int k = k0; k < k1; k += kTK) {
    const bool more = k + kTK < k1;
    if (more) fetch(k + kTK);
    const float* as = smem + buf * (S::STAGE / 4);
    const float* bs = as + kTK * LDA;
#pragma unroll 16
    for (int kk = FLAT ? ty : 0; kk < kTK; kk += FLAT ? 16 : 1) {
      float a[RM];
#pragma unroll
      for (int h = 0; h < RM / VEC; ++h) {
        const float* src = as + kk * LDA + (FLAT ? h * 4 : h * 64 + ty * VEC);
        if (VEC == 4) {
          const float4 q = *reinterpret_cast<const float4*>(src);
          a[4 * h] = q.x, a[4 * h + 1] = q.y, a[4 * h + 2] = q.z, a[4 * h + 3] = q.w;
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) a[i] = src[i];
        }
      }
      f32x2 b[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const ulonglong2 q =
            *reinterpret_cast<const ulonglong2*>(bs + kk * kLdb + h * 64 + tx * 4);
        b[2 * h] = q.x;
        b[2 * h + 1] = q.y;
      }
#pragma unroll
      for (int i = 0; i < RM; ++i) {
        const f32x2 aa = f32x2_of(a[i], a[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = f32x2_fma(aa, b[j], acc[i][j]);
      }
    }
    buf ^= 1;
    if (more) stage(smem + buf * (S::STAGE / 4), smem + buf * (S::STAGE / 4) + kTK * LDA);
    __syncthreads();
  }

  if (FLAT) {
    // over the warp's four k groups by shuffles, then over the four pairs of
    // warps through shared memory (the last step ended with a barrier)
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[4];
        f32x2_split(acc[i][2 * h], v[0], v[1]);
        f32x2_split(acc[i][2 * h + 1], v[2], v[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] += __shfl_xor_sync(0xffffffffu, v[j], 8);
          v[j] += __shfl_xor_sync(0xffffffffu, v[j], 16);
        }
        if (lane < 8)
          *reinterpret_cast<float4*>(smem + (warp / 2 * TM + i) * kLdb + h * 64 + tx * 4) =
              make_float4(v[0], v[1], v[2], v[3]);
      }
    __syncthreads();
    static_assert(!FLAT || TM * 32 == kThreads, "one piece of a row per thread");
    float4* mine = reinterpret_cast<float4*>(smem + warp * kLdb + lane * 4);
    float4 v = mine[0];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 q = mine[w * TM * kLdb / 4];
      v.x += q.x, v.y += q.y, v.z += q.z, v.w += q.w;
    }
    mine[0] = v;  // row `warp` of the first tile: read by this thread only
  } else {
    auto row_of = [&](int i) { return i / VEC * 64 + ty * VEC + i % VEC; };
    // to the tile over the stages (the last step ended with a barrier)
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float4 v;
        f32x2_split(acc[i][2 * h], v.x, v.y);
        f32x2_split(acc[i][2 * h + 1], v.z, v.w);
        *reinterpret_cast<float4*>(smem + row_of(i) * kLdb + h * 64 + tx * 4) = v;
      }
  }
  // the epilogue goes through the tile in a loop: whole rows per warp, and one
  // copy of its code
  if (p.splits == 1) {
    __syncthreads();
#pragma unroll 1
    for (int e = threadIdx.x; e < TM * 32; e += kThreads)
      finish(p, m0 + e / 32, n0 + e % 32 * 4,
             *reinterpret_cast<const float4*>(smem + e / 32 * kLdb + e % 32 * 4));
    return;
  }
  cluster_sync();  // every slice's partial tile is written
  // FLAT: the slices divide its eight rows (any number of them costs registers
  // that the main loop needs: 4096 x 4096, one token 25.8 us instead of 24)
  const int share = FLAT ? TM / p.splits : (TM + p.splits - 1) / p.splits;
#pragma unroll 1
  for (int e = threadIdx.x; e < share * 32; e += kThreads) {
    const int r = slice * share + e / 32, c = e % 32 * 4;
    if (!FLAT && r >= TM) break;
    const uint32_t at = smem_u32(smem + r * kLdb + c);
    float4 q[kMaxSplits];
#pragma unroll
    for (int s = 0; s < kMaxSplits; ++s)
      if (s < p.splits) {
        if (s == slice) {
          q[s] = *reinterpret_cast<const float4*>(smem + r * kLdb + c);
        } else {
          const uint32_t peer = map_peer(at, static_cast<uint32_t>(s));
          asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                       : "=f"(q[s].x), "=f"(q[s].y), "=f"(q[s].z), "=f"(q[s].w)
                       : "r"(peer)
                       : "memory");
        }
      }
    float4 v = q[0];
#pragma unroll
    for (int s = 1; s < kMaxSplits; ++s)
      if (s < p.splits) v.x += q[s].x, v.y += q[s].y, v.z += q[s].z, v.w += q[s].w;
    finish(p, m0 + r, n0 + c, v);
  }
  cluster_sync();  // no CTA leaves while a peer still reads its tile
}

// How K is cut for a grid of some tiles.
struct Slices {
  int count, length;
  double us;  // of the main loop
};

// Slices of whole K steps (`step`), so that the SM with the most CTAs has the
// least to do: per_k us per k for one CTA, 1.9 times that for two, and 0.1 us per
// slice for adding them up.  Clusters of up to six CTAs get an SM per CTA up to
// 128 of 152 CTAs (64 tiles in two slices, 32 in four, 20 in six; 35 tiles in four
// ran two to an SM while others stayed empty), clusters of seven or eight up to 64
// (8 tiles in eight slices, not 12).  powers: powers of two only.
Slices slices_for(long long tiles, int K, int step, double per_k, bool powers) {
  Slices best = {};
  for (int n = 1; n <= kMaxSplits; ++n) {
    const int length = ((K + n - 1) / n + step - 1) / step * step;
    const long long ctas = tiles * n, sms = sm_count();
    if (n > 1 && ctas > 2 * sms) break;
    if (powers && (n & (n - 1)) != 0) continue;
    if (n > 1 && static_cast<long long>(length) * (n - 1) >= K) continue;  // an empty slice
    const long long apart = n == 1 ? sms : n <= 6 ? sms * 128 / 152 : sms * 64 / 152;
    const long long rounds = (ctas + 2 * sms - 1) / (2 * sms);
    const double us =
        per_k * length * (ctas <= apart ? 1.0 : 1.9 * static_cast<double>(rounds)) + 0.1 * n;
    if (n == 1 || us < 0.97 * best.us) best = {n, length, us};
  }
  return best;
}

// us per k of a CTA's tile, measured (1024 of K in one slice).
constexpr double kPerK8 = 0.105, kPerK4 = 0.067, kPerK2 = 0.052, kPerKFlat = 0.03;

template <int RM, bool A_KM, bool B_KN, bool FLAT>
cudaError_t launch(const LinearProduct& g, long long m_first, long long rows, double per_k,
                   cudaStream_t stream) {
  using S = Shape<RM, FLAT>;
  auto* kernel = linear_simt_kernel<RM, A_KM, B_KN, FLAT>;
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
    if (e != cudaSuccess) return e;
    ready[dev].store(true, std::memory_order_relaxed);
  }
  SimtArgs p;
  p.lda = g.pitch_a > 0 ? g.pitch_a : A_KM ? g.M : g.K;
  p.A = static_cast<const float*>(g.A) + m_first * (A_KM ? 1 : p.lda);
  p.B = static_cast<const float*>(g.B);
  p.epi = fp32_epilogue(g, m_first);
  p.M = rows;
  p.N = g.N;
  p.K = g.K;
  p.all_rows = g.all_rows;
  p.row_flags = g.row_flags != nullptr ? g.row_flags + m_first * g.segs : nullptr;
  p.segs = g.segs;
  p.vec_a = p.lda % 4 == 0;
  p.vec_b = (B_KN ? g.N : g.K) % 4 == 0;
  const int n_tiles = (g.N + kTN - 1) / kTN;
  const long long m_tiles = (rows + S::TM - 1) / S::TM;
  const Slices cut = slices_for(n_tiles * m_tiles, g.K, S::TK, per_k, FLAT);
  const int splits = cut.count;
  p.splits = splits;
  p.k_slice = cut.length;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n_tiles * splits), static_cast<unsigned>(m_tiles));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = splits > 1 ? 2 : 1;
  prof_begin(g.tag, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  prof_end(g.tag, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int RM, bool FLAT = false>
cudaError_t by_major(const LinearProduct& g, long long m, long long rows, double per_k,
                     cudaStream_t s) {
  if (g.a_mn) return launch<RM, true, true, FLAT>(g, m, rows, per_k, s);
  return g.b_mn ? launch<RM, false, true, FLAT>(g, m, rows, per_k, s)
                : launch<RM, false, false, FLAT>(g, m, rows, per_k, s);
}

}  // namespace

cudaError_t linear_simt(const LinearProduct& g, cudaStream_t s) {
  // at most 2^19 rows a launch: the grid's y extent is 16 bits
  constexpr long long kRows = 1 << 19;
  for (long long m = 0; m < g.M; m += kRows) {
    const long long rows = std::min(kRows, g.M - m);
    const long long tiles = (g.N + kTN - 1) / kTN;
    const auto us = [&](int tm, int step, double per_k) {
      return slices_for(tiles * ((rows + tm - 1) / tm), g.K, step, per_k, false).us;
    };
    cudaError_t e;
    // the fewest rows that hold the tokens; beyond 64, tiles of 128 rows unless
    // the main loop of 64 is clearly shorter (300 x 4096 -> 512: 51 against 71 us)
    const bool half = rows <= 64 || us(64, Shape<4, false>::TK, kPerK4) <
                                        0.93 * us(128, Shape<8, false>::TK, kPerK8);
    if (rows <= 16)
      e = by_major<8, true>(g, m, rows, kPerKFlat, s);
    else if (rows <= 32)
      e = by_major<2>(g, m, rows, kPerK2, s);
    else if (half)
      e = by_major<4>(g, m, rows, kPerK4, s);
    else
      e = by_major<8>(g, m, rows, kPerK8, s);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace poetx
