// The matrix products of poetx_linear_* in fp32 on the tensor cores.
//
// Every fp32 value is the sum of three bf16 numbers, x = x1 + x2 + x3, each the
// rounding of what the ones before leave (24 bits in all), so
//   x w = x1 w1 + (x1 w2 + x2 w1) + (x1 w3 + x2 w2 + x3 w1) + O(2^-24 |x w|)
// and an fp32 product is six bf16 products with fp32 accumulation.  The tensor
// core's accumulation truncates (a sum of 1 and 64 terms of 0.75 ulp is 1), which
// would bias long sums; so the six products of every 128 of K, the small ones
// first, are accumulated on their own, and those partial sums are added up in
// registers with round-to-nearest: 2e-7 to 4e-7 of the result, as a plain fp32
// product has (cuBLAS: 4e-7 to 1e-6 on the same inputs).
//
// x and W are split into three bf16 planes each in the workspace first, which
// takes 0 and magnitudes from 2^-109 to 2^60.  Below, the third plane's bits fall
// under bf16's smallest number, 2^-133; up to 2^60, 128 products of two stay
// under 2^128, so that no partial sum meets an infinite one of the other sign (beyond,
// a product of small parts can leave the range before the main one does, and the
// infinity had the wrong sign).  Where a value is outside, or not finite, the
// split sets the flag of its token (of all, where it is W's), this kernel leaves
// those rows alone and linear_simt, enqueued behind it, computes them; its tiles
// without such rows return at once.
//
// The kernel is linear_pair's with another epilogue: CTA pairs, tiles of 256 x 128 to
// 256 (tile_width), 64-wide K steps in a TMA ring, one step per pair of planes;
// 16 epilogue warps (a quarter of the columns each) drain one of two TMEM
// accumulators into registers while the next 128 of K go into the other.
#include <algorithm>
#include <mutex>

#include "internal.h"
#include "linear.h"
#include "linear_fp32.cuh"
#include "linear_planes.cuh"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace poetx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kEpiWarps = 16;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kA = BM * BK * 2;     // this CTA's 128 rows, one K step
constexpr int kSlot = 32 * 16 * 4;  // an epilogue warp's 32 rows x 16 columns
constexpr int kStaging = kEpiWarps * kSlot;

template <int BN>
struct Shape {
  static constexpr int B = (BN / 2) * BK * 2;  // this CTA's half of B, one K step
  static constexpr int STAGE = kA + B;
  static constexpr int STAGES = BN == 256 ? 6 : 8;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int SMEM = RING + kStaging + 256;
  static constexpr uint32_t TMEM_COLS = 2 * BN;
  static constexpr int COLS = BN / 4;  // columns of an epilogue warp
  static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

constexpr int kGroupM = 8;
constexpr int kProducts = 6;
constexpr int kChunkSteps = 2;  // K steps accumulated by the tensor core in one go

// Product p = 0 .. 5, the smallest first: planes (2,0) (0,2) (1,1) (1,0) (0,1)
// (0,0) of A and B, four bits each.
__device__ __forceinline__ int plane_a(int p) { return (0x001102 >> (4 * p)) & 3; }
__device__ __forceinline__ int plane_b(int p) { return (0x010120 >> (4 * p)) & 3; }

struct SplitArgs {
  int m_pairs, n_tiles, k_steps, N;
  int width;  // of a tile, BN at most
  int slices, slice_steps;  // of K; a slice's outputs are M N values behind the last's
  int plane_rows_a, plane_rows_b;  // rows between planes of A, of B
  long long M;
  Fp32Epilogue epi;
  int segs;              // flags per row of A
  const int* row_flags;  // A's: rows with one that is not 0 are left to linear_simt
  int b_count, a_count;  // flags of B (quads), and of A as [K][M]: then all rows are
  const int *b_flags, *a_flags;
  int* all;              // set here: whether any of those is
  int* status;
};

// Unit u: its tile and K steps; all tiles of a slice before the next.
__device__ __forceinline__ void unit_tile(int u, const SplitArgs& p, int& mp, int& nt, int& slice,
                                          int& begin, int& end) {
  const int tiles = p.m_pairs * p.n_tiles;
  slice = u / tiles;
  u -= slice * tiles;
  begin = slice * p.slice_steps;
  end = min(p.k_steps, begin + p.slice_steps);
  const int per_group = kGroupM * p.n_tiles;
  const int g = u / per_group, r = u - g * per_group;
  const int rows = min(kGroupM, p.m_pairs - g * kGroupM);
  mp = g * kGroupM + r % rows;
  nt = r / rows;
}

template <int BN, bool A_MN, bool B_MN>
__global__ void __launch_bounds__(kThreads, 1)
    linear_split_kernel(const __grid_constant__ CUtensorMap tmA,
                        const __grid_constant__ CUtensorMap tmB, const SplitArgs p) {
  using S = Shape<BN>;
  constexpr int kStages = S::STAGES, kStage = S::STAGE, kRing = S::RING, kBN = BN;
  extern __shared__ __align__(1024) uint8_t base[];  // 128B-swizzled tiles start on 1024 bytes
  if ((smem_u32(base) & 1023u) != 0) {  // the declared alignment, which the tiles rely on
    if (threadIdx.x == 0) atomicCAS(p.status, 0, static_cast<int>(POETX_ERR_CUDA));
    return;
  }
  uint8_t* ring = base;  // stage s: A (16 KiB), then this CTA's half of B
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(base + kRing + kStaging);  // leader
  uint64_t* empty_bar = full_bar + kStages;   // each CTA: its slot is free
  uint64_t* tfull_bar = empty_bar + kStages;  // [2] each CTA: accumulator ready
  uint64_t* tempty_bar = tfull_bar + 2;       // [2] leader: accumulator drained
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int first = static_cast<int>(cluster_id_x());
  const int step = static_cast<int>(cluster_count_x());

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull_bar[a], 1);
      mbar_init(&tempty_bar[a], 2 * kEpiWarps);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, S::TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();
  int bad = 0;
  for (int i = threadIdx.x; i < p.b_count / 4; i += kThreads) {
    const int4 q = reinterpret_cast<const int4*>(p.b_flags)[i];
    bad |= q.x | q.y | q.z | q.w;
  }
  if (A_MN)
    for (int i = threadIdx.x; i < p.a_count; i += kThreads) bad |= p.a_flags[i];
  bad = __syncthreads_or(bad);
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.all = bad;
  const int units = bad != 0 ? 0 : p.m_pairs * p.n_tiles * p.slices;

  const uint32_t full0 = map_peer(smem_u32(full_bar), 0);
  const uint32_t tempty0 = map_peer(smem_u32(tempty_bar), 0);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // (here and in the MMA warp one elected lane issues, as in linear_pair)
    int stage = 0;
    uint32_t phase = 0;
    long long issued = 0;
    // bytes of a step; an MN-major B comes in boxes of 64 columns
    const uint32_t half = static_cast<uint32_t>(B_MN ? kBN : p.width) / 2;
    const uint32_t tx = 2 * (kA + half * BK * 2);
    bool ok = true;
    for (int u = first; u < units && ok; u += step) {
      int mp, nt, slice, begin, end;
      unit_tile(u, p, mp, nt, slice, begin, end);
      const int a_row = mp * 2 * BM + static_cast<int>(rank) * BM;
      const int b_n = nt * p.width + static_cast<int>(rank) * (p.width / 2);
      for (int k0 = begin; k0 < end && ok; k0 += kChunkSteps) {
        const int k1 = min(end, k0 + kChunkSteps);
        for (int pr = 0; pr < kProducts && ok; ++pr) {
          const int ra = plane_a(pr) * p.plane_rows_a;
          const int rb = plane_b(pr) * p.plane_rows_b;
          for (int ks = k0; ks < k1; ++ks) {
            if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag)) {
              record_timeout(p.status, abort_flag);
              ok = false;
              break;
            }
            if (elect_one()) {
              if (leader) mbar_arrive_expect_tx(&full_bar[stage], tx);
              uint8_t* a_dst = ring + stage * kStage;
              uint8_t* b_dst = a_dst + kA;
              const uint32_t bar = full0 + static_cast<uint32_t>(stage * 8);
              if (!A_MN) {
                tma_load_2d_pair(a_dst, &tmA, bar, ks * BK, ra + a_row);
              } else {
                tma_load_2d_pair(a_dst, &tmA, bar, a_row, ra + ks * BK);
                tma_load_2d_pair(a_dst + 8192, &tmA, bar, a_row + 64, ra + ks * BK);
              }
              if (!B_MN) {
                tma_load_2d_pair(b_dst, &tmB, bar, ks * BK, rb + b_n);
              } else {
                tma_load_2d_pair(b_dst, &tmB, bar, b_n, rb + ks * BK);
                if (BN == 256)
                  tma_load_2d_pair(b_dst + 8192, &tmB, bar, b_n + 64, rb + ks * BK);
              }
            }
            __syncwarp();
            ++issued;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
      }
    }
    // every slot this CTA filled is released again before it leaves
    const int outstanding = issued < kStages ? static_cast<int>(issued) : kStages;
    int st = stage;
    uint32_t ph = phase;
    for (int n = 0; n < outstanding; ++n) {
      if (--st < 0) {
        st = kStages - 1;
        ph ^= 1;
      }
      const unsigned long long t0 = global_timer_ns();
      while (!mbar_try_wait_cluster(&empty_bar[st], ph) &&
             global_timer_ns() - t0 < (ok ? kWaitLimitNs : 10000000ull)) {
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // -------------------------------------------------- MMA issuer (pair)
      const uint32_t IDESC = instr_desc_bf16(2 * BM, p.width, A_MN, B_MN);
      const uint32_t empty_own = smem_u32(empty_bar);
      const uint32_t tfull_own = smem_u32(tfull_bar);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      bool any_mma = false;
      for (int u = first; u < units && ok; u += step) {
        int mp, nt, slice, begin, end;
        unit_tile(u, p, mp, nt, slice, begin, end);
        for (int k0 = begin; k0 < end && ok; k0 += kChunkSteps) {
          const int steps = (min(end, k0 + kChunkSteps) - k0) * kProducts;
          if (!mbar_wait_cluster(&tempty_bar[acc], acc_phase ^ 1, abort_flag)) {
            record_timeout(p.status, abort_flag);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * kBN);
          for (int i = 0; i < steps; ++i) {
            if (!mbar_wait(&full_bar[stage], phase, abort_flag)) {
              record_timeout(p.status, abort_flag);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_base = smem_u32(ring) + stage * kStage;
            const uint64_t adesc0 = smem_desc_sw128(a_base, A_MN ? 8192 : 16, 1024);
            const uint64_t bdesc0 = smem_desc_sw128(a_base + kA, B_MN ? 8192 : 16, 1024);
            if (elect_one()) {
#pragma unroll
              for (int j = 0; j < BK / 16; ++j)
                umma_bf16_pair(d_tmem, adesc0 + j * (A_MN ? 128 : 2),
                               bdesc0 + j * (B_MN ? 128 : 2), IDESC,
                               (i > 0 || j > 0) ? 1u : 0u);
              umma_commit_both(empty_own + static_cast<uint32_t>(stage * 8));
            }
            __syncwarp();
            any_mma = true;
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          if (elect_one()) umma_commit_both(tfull_own + static_cast<uint32_t>(acc * 8));
          __syncwarp();
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
      }
      if (!ok && any_mma) {
        // the MMAs in flight finish before TMEM is released
        if (elect_one()) umma_commit_pair(smem_u32(drain_bar));
        __syncwarp();
        const unsigned long long t0 = global_timer_ns();
        while (!mbar_try_wait(drain_bar, 0) && global_timer_ns() - t0 < 10000000ull) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 2;
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const int side = ew >> 2;      // its quarter of the tile's columns
    float* slot = reinterpret_cast<float*>(base + kRing + ew * kSlot);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = first; u < units && ok; u += step) {
      int mp, nt, slice, begin, end;
      unit_tile(u, p, mp, nt, slice, begin, end);
      const long long row0 = static_cast<long long>(mp) * 2 * BM + rank * BM + quarter * 32;
      const int col0 = nt * p.width + side * S::COLS;
      const int cols = min(p.N, (nt + 1) * p.width) - col0;  // of this warp that are the tile's
      float sum[S::COLS / 16][16] = {};
      for (int k0 = begin; k0 < end; k0 += kChunkSteps) {
        const bool got = mbar_wait_cluster(&tfull_bar[acc], acc_phase, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          record_timeout(p.status, abort_flag);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t t_base = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                static_cast<uint32_t>(acc * kBN + side * S::COLS);
#pragma unroll
        for (int q = 0; q < S::COLS / 16; ++q) {
          uint32_t r[16];
          tmem_load_16(t_base + q * 16, r);
#pragma unroll
          for (int j = 0; j < 16; ++j) sum[q][j] += __uint_as_float(r[j]);
        }
        tc_fence_before();
        __syncwarp();
        // the accumulator is free again once both CTAs' epilogue warps have read it
        if (lane == 0) mbar_arrive_remote_relaxed(tempty0 + static_cast<uint32_t>(acc * 8));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
      if (!ok) break;
      // this lane's row: outside, or left to linear_simt
      int skip = row0 + lane >= p.M;
      if (!skip)
        for (int i = 0; i < p.segs; ++i) skip |= p.row_flags[(row0 + lane) * p.segs + i];
      // 16 columns at a time through the warp's staging tile, so that four lanes
      // write 64 bytes of a row (pieces of 16 bytes xor-swizzled by the row)
      // (one copy of the epilogue's code: sixteen unrolled ones, with every
      // activation in each, cost 10 us of instruction fetches)
#pragma unroll 1
      for (int q = 0; q < S::COLS / 16 && q * 16 < cols; ++q) {
        __syncwarp();
#pragma unroll
        for (int s = 0; s < S::COLS / 16; ++s)
          if (s == q) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<float4*>(slot + lane * 16 + ((j ^ (lane >> 1)) & 3) * 4) =
                  make_float4(sum[s][4 * j], sum[s][4 * j + 1], sum[s][4 * j + 2],
                              sum[s][4 * j + 3]);
          }
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + lane / 4, n = col0 + q * 16 + lane % 4 * 4;
          const float4 v =
              *reinterpret_cast<const float4*>(slot + r * 16 + ((lane % 4 ^ (r >> 1)) & 3) * 4);
          const int no = __shfl_sync(0xffffffffu, skip, r);
          if (p.slices == 1) {
            if (no == 0 && n < p.N) finish4(p.epi, row0 + r, n, v);
          } else if (row0 + r < p.M && n < p.N && (no == 0 || slice > 0)) {
            // a row of linear_simt's is whole in the first slice, 0 in the others
            const float4 part = no == 0 ? v : make_float4(0.f, 0.f, 0.f, 0.f);
            finish4(p.epi, slice * p.M + row0 + r, n, part);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal or read it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, S::TMEM_COLS);
  }
}

// One operand: in [rows][cols] fp32 -> planes [3][plane_rows][pitch] bf16, rows
// from `rows` to plane_rows zero (columns past cols are not read by any tile);
// flag[r][segs]: whether a value of the row's segment of kSegment columns is
// neither 0 nor of a magnitude that the planes take.  Of B a flag per CTA, `flags` of
// them, is enough: one for every row (30001) made each CTA of the product read them
// for 20 us.
constexpr int kSegment = 1024;

struct SplitOperand {
  const float* in;
  bf16* planes;
  int* flag;   // null: none
  int* whole;  // the CTAs'; null: none
  long long rows, ld, plane_rows, pitch;
  int cols, segs;
};

constexpr int kSplitThreads = 256;

// Both operands, a warp per segment of a row.  Five CTAs on an SM: with the 57 registers
// that the compiler takes otherwise four fit, and the copies in flight are too few (2048 x
// 2048 and 5632 x 2048: 25.8 / 28.2 us, 513 x 1537 and 2049 x 1537: 10.4 / 14.5).
__global__ void __launch_bounds__(kSplitThreads, 5)
    split_planes_kernel(const SplitOperand a, const SplitOperand b, int flags) {
  pdl_wait();
  pdl_trigger();
  bool bad_a = false, bad_b = false;
  const int lane = threadIdx.x % 32;
  const long long items_a = a.plane_rows * a.segs, items = items_a + b.plane_rows * b.segs;
  for (long long it = blockIdx.x * static_cast<long long>(kSplitThreads / 32) + threadIdx.x / 32;
       it < items; it += static_cast<long long>(gridDim.x) * (kSplitThreads / 32)) {
    const bool first = it < items_a;
    const SplitOperand& o = first ? a : b;
    const long long at = first ? it : it - items_a;
    const long long r = at / o.segs;
    const int c0 = static_cast<int>(at - r * o.segs) * kSegment;
    const int c1 = min(o.cols, c0 + kSegment);
    const float* in = o.in + r * o.ld;
    const bool vec = o.ld % 4 == 0;
    bool bad = false;
#pragma unroll 4
    for (int c = c0 + lane * 4; c < c1; c += 128) {
      float v[4] = {0.f, 0.f, 0.f, 0.f};
      if (r < o.rows) {
        if (vec) {
          const float4 q = *reinterpret_cast<const float4*>(in + c);
          v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
          if (c + 3 >= o.cols) {  // what lies between the rows is nothing
#pragma unroll
            for (int j = 1; j < 4; ++j)
              if (c + j >= o.cols) v[j] = 0.f;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (c + j < o.cols) v[j] = in[c + j];
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) bad |= outside_planes(v[j]);
      // rows are a multiple of 64 elements apart: 8 bytes fit, padding included
      store_planes(o.planes + r * o.pitch + c, o.plane_rows * o.pitch, v);
    }
    bad = __any_sync(0xffffffffu, bad);
    (first ? bad_a : bad_b) |= bad;
    if (o.flag != nullptr && lane == 0) o.flag[at] = bad;
  }
  const auto whole = [&](int* to, bool bad) {
    if (to == nullptr) return;
    bad = __syncthreads_or(bad);
    if (blockIdx.x == 0)
      for (int i = gridDim.x + threadIdx.x; i < flags; i += kSplitThreads) to[i] = 0;
    if (threadIdx.x == 0) to[blockIdx.x] = bad;
  };
  whole(a.whole, bad_a);
  whole(b.whole, bad_b);
}

size_t round256(size_t n) { return (n + 255) & ~static_cast<size_t>(255); }

long long b_plane_rows(const LinearProduct& g) {
  // [K][N]: rows to a whole K step, so that no tile meets the next plane's rows; [N][K]
  // the same, for a next product with the array the other way round (b_ready)
  return ((g.b_mn ? g.K : g.N) + BK - 1ll) / BK * BK;
}

int b_cols(const LinearProduct& g) { return g.b_mn ? g.N : g.K; }

// Rows of planes start on 128 bytes: rows of 2000 bytes made the loads a third
// slower than the products (1000^3: 750 cycles a step instead of 512).
long long pitch64(int cols) { return (static_cast<long long>(cols) + 63) / 64 * 64; }

int segments(int cols) { return (cols + kSegment - 1) / kSegment; }

int split_ctas() { return 8 * sm_count(); }

size_t planes_bytes(long long plane_rows, int cols) {
  return round256(static_cast<size_t>(kPlanes) * plane_rows * pitch64(cols) * 2);
}

// a, b: their planes and flags; A_MN: a is [K][M].
template <int BN, bool A_MN, bool B_MN>
cudaError_t launch(const LinearProduct& g, const SplitOperand& a, const SplitOperand& b, int width,
                   int* all, cudaStream_t stream) {
  constexpr int kSmem = Shape<BN>::SMEM;
  auto* kernel = linear_split_kernel<BN, A_MN, B_MN>;
  static bool ready[64] = {false};
  static int max_clusters[64] = {0};
  static std::mutex mu;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  int cmax;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      cfg.gridDim = dim3(2 * sm_count());
      cfg.numAttrs = 1;
      int n = 0;
      e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
      if (e != cudaSuccess) return e;
      if (n < 1) return cudaErrorLaunchOutOfResources;
      max_clusters[dev] = n;
      ready[dev] = true;
    }
    cmax = max_clusters[dev];
  }
  SplitArgs p;
  p.plane_rows_a = static_cast<int>(a.plane_rows);
  p.plane_rows_b = static_cast<int>(b.plane_rows);
  CUtensorMap tmA, tmB;
  if (!make_map(&tmA, a.planes, kPlanes * a.plane_rows, a.cols, a.pitch, 2, 64, A_MN ? 64 : BM) ||
      !make_map(&tmB, b.planes, kPlanes * b.plane_rows, b.cols, b.pitch, 2, 64,
                B_MN ? 64 : width / 2))
    return cudaErrorInvalidValue;
  p.m_pairs = static_cast<int>((g.M + 2 * BM - 1) / (2 * BM));
  p.width = width;
  p.n_tiles = (g.N + width - 1) / width;
  p.k_steps = (g.K + BK - 1) / BK;
  p.slices = g.slices;
  p.slice_steps = (p.k_steps + g.slices - 1) / g.slices;
  p.N = g.N;
  p.M = g.M;
  p.epi = fp32_epilogue(g, 0);
  p.all = all;
  p.row_flags = A_MN ? nullptr : a.flag;
  p.segs = A_MN ? 0 : a.segs;
  p.b_count = split_ctas();
  p.b_flags = b.whole;
  p.a_count = A_MN ? g.K : 0;
  p.a_flags = a.flag;
  p.status = device_status_ptr();
  const int clusters = static_cast<int>(
      std::min<long long>(static_cast<long long>(p.m_pairs) * p.n_tiles * p.slices, cmax));
  cfg.gridDim = dim3(2 * clusters);
  cfg.numAttrs = 2;
  prof_begin(g.tag, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tmA, tmB, p);
  prof_end(g.tag, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

namespace {

// The width of the tiles: a narrower one of as many rounds over the clusters leaves less
// of the last round empty; a step is taken to lie between those of 128 and of 256 wide
// (loop_us) in proportion.  256 or 128 / any: 515 tokens, 1000 -> 10007 116 / 106 us, 333
// tokens, 768 -> 30001 186 / 168, 2048 tokens, 2048 -> 5632 224 / 199, 4096^3 545 / 508,
// 300 tokens, 2048 -> 8192 105 / 101.  Of a [K][N] B, which comes in boxes of 64 columns,
// multiples of 32: its loads stay those of 256 (dx of 515 tokens, 10007 <- 1000 116 / 111,
// of 2048, 5632 <- 2048 224 / 209, 4096^3 543 / 507).  linear_split_pays keeps to 128 and
// 256.
int tile_width(const LinearProduct& g) {
  const long long m_pairs = (g.M + 2 * BM - 1) / (2 * BM), clusters = std::max(1, sm_count() / 2);
  int best = 256;
  double least = 0.0;
  for (int w = 256; w >= 128; w -= g.b_mn ? 32 : 16) {
    const long long rounds = (g.slices * m_pairs * ((g.N + w - 1) / w) + clusters - 1) / clusters;
    const double us = static_cast<double>(rounds) * (0.53 + 1.18 / 256.0 * w);
    if (w == 256 || us < 0.98 * least) {
      least = us;
      best = w;
    }
  }
  return best;
}

// Microseconds of the products' main loops: a 64-wide step of the six products
// takes 1.71 us in a 256-wide tile, 1.12 in a 128-wide one (see linear_pair).
double loop_us(long long M, int N, int K, int slices) {
  const long long m_pairs = (M + 2 * BM - 1) / (2 * BM), clusters = std::max(1, sm_count() / 2);
  const long long wide = (slices * m_pairs * ((N + 255) / 256) + clusters - 1) / clusters;
  const long long thin = (slices * m_pairs * ((N + 127) / 128) + clusters - 1) / clusters;
  const long long steps = (K + BK - 1) / BK;
  return std::min(1.12 * thin, 1.71 * wide) * ((steps + slices - 1) / slices);
}

// With 4 bytes written and read per output and slice.
double split_us(long long M, int N, int K, int slices = 1) {
  return 18.0 + loop_us(M, N, K, slices) + 10e-6 * K * (static_cast<double>(M) + N) / 6.0 +
         (slices > 1 ? 2e-6 * slices * M * N : 0.0);
}

}  // namespace

// By the measured costs of both: here the loops above, 18 us for three launches
// and the pipeline's ends, and 10 bytes per element of the operands for their
// planes; linear_simt 8 us and 45 TFLOP/s.  They cross near 1000^3.
bool linear_split_pays(long long M, int N, int K) {
  return split_us(M, N, K) < 8.0 + 2e-6 * M * N * K / 45.0;
}

// A slice has at least four K steps, none is empty.  333 x 30001 -> 768 (6 tiles of
// 256, 12 of 128, 469 steps): on the CUDA cores 459 us, in 8 slices 103, in 12 90.
int linear_split_slices(long long M, int N, int K, size_t most_bytes) {
  const int steps = (K + BK - 1) / BK;
  int best = 1;
  double least = split_us(M, N, K);
  for (int n = 2; n <= kMaxFp32Slices && steps / n >= 4; ++n) {
    if (4ull * n * M * N > most_bytes) break;
    if ((steps + n - 1) / n * (n - 1) >= steps) continue;
    const double us = split_us(M, N, K, n);
    if (us < least) {
      least = us;
      best = n;
    }
  }
  // linear_simt, with at most eight slices of its own: at least 0.05 us (up to 16 tokens
  // 0.03) for a k of one (512 x 128256 -> 64: 1900 us, here 310 with
  // the operands' planes)
  const double simt =
      8.0 + std::max(2e-6 * M * N * K / 45.0, (M <= 16 ? 0.03 : 0.05) * K / 8.0);
  return split_us(M, N, K, best) < simt ? best : 1;
}

namespace {

long long up64(long long n) { return (n + 63) / 64 * 64; }

size_t flag_bytes(long long rows, int cols) {
  return round256(static_cast<size_t>(rows * segments(cols)) * sizeof(int));
}

// The word that says whether the CUDA cores take everything, and from the second 16 bytes
// on the CTAs' flags.
size_t all_flag_bytes() { return round256((4 + split_ctas()) * sizeof(int)); }

SplitOperand operand(const void* in, long long rows, int cols, long long ld,
                     long long plane_rows) {
  SplitOperand o = {};
  o.in = static_cast<const float*>(in);
  o.rows = rows;
  o.cols = cols;
  o.ld = ld > 0 ? ld : cols;
  o.plane_rows = plane_rows;
  o.segs = segments(cols);
  o.pitch = pitch64(cols);
  return o;
}

// An operand that is kept, at a place of linear_planes_bytes: a word that says whether
// the CUDA cores take all of it, the CTAs' flags, the rows', the planes.
SplitOperand kept(void* at, const void* in, long long rows, int cols, long long ld) {
  SplitOperand o = operand(in, rows, cols, ld, up64(rows));
  char* c = static_cast<char*>(at);
  o.whole = reinterpret_cast<int*>(c) + 4;
  o.flag = reinterpret_cast<int*>(c + all_flag_bytes());
  o.planes = reinterpret_cast<bf16*>(c + all_flag_bytes() + flag_bytes(o.plane_rows, cols));
  return o;
}

// The planes of a, and of b unless it is null.
cudaError_t split(const SplitOperand& a, const SplitOperand* b, cudaStream_t s) {
  const SplitOperand other = b != nullptr ? *b : operand(nullptr, 0, 1, 1, 0);
  const int grid = static_cast<int>(std::min<long long>(
      (a.plane_rows * a.segs + other.plane_rows * other.segs + 7) / 8, split_ctas()));
  prof_begin("linear_split_planes", s);
  const cudaError_t e = launch_pdl(split_planes_kernel, dim3(grid), dim3(kSplitThreads), 0, s, a,
                                   other, split_ctas());
  prof_end("linear_split_planes", s);
  return e;
}

}  // namespace

size_t linear_planes_bytes(long long rows, int cols) {
  return all_flag_bytes() + flag_bytes(up64(rows), cols) + planes_bytes(up64(rows), cols);
}

Fp32Planes linear_planes_at(void* at, long long rows, int cols) {
  const SplitOperand o = kept(at, nullptr, rows, cols, 0);
  return {o.planes, o.flag, o.plane_rows, o.pitch};
}

size_t linear_split_b_scratch(const LinearProduct& g) {
  return all_flag_bytes() + planes_bytes(b_plane_rows(g), b_cols(g));
}

// B's flags and planes come first: their place depends on B alone.
size_t linear_split_scratch(const LinearProduct& g) {
  return linear_split_b_scratch(g) + flag_bytes(g.M, g.K) + planes_bytes(g.M, g.K);
}

// Whether this form is taken does not grow with the rows: a new pair of row tiles
// can add a round over the clusters, and linear_simt wins.  But within a pair both
// costs are linear in the rows, so its first and its last row decide; the scratch
// grows with the rows, so the last pair that has any bounds it.
size_t linear_split_scratch_up_to(const LinearProduct& g) {
  LinearProduct at = g;
  while (at.M > 0) {
    const long long first = (at.M - 1) / (2 * BM) * (2 * BM) + 1;
    if (linear_split_pays(at.M, g.N, g.K) || linear_split_pays(first, g.N, g.K))
      return linear_split_scratch(at);
    at.M = first - 1;
  }
  return 0;
}

cudaError_t linear_split(const LinearProduct& g, void* scratch, cudaStream_t s) {
  int* all = static_cast<int*>(scratch);
  SplitOperand a, b = operand(g.B, g.b_mn ? g.K : g.N, b_cols(g), 0, b_plane_rows(g));
  b.whole = all + 4;
  b.planes = reinterpret_cast<bf16*>(static_cast<char*>(scratch) + all_flag_bytes());
  if (g.a_planes != nullptr) {
    a = kept(g.a_planes, g.A, g.M, g.K, g.pitch_a);
    if (g.a_ready) a.segs = 1;
  } else {
    char* at = static_cast<char*>(scratch) + linear_split_b_scratch(g);
    a = operand(g.A, g.M, g.K, g.pitch_a, g.M);
    a.flag = reinterpret_cast<int*>(at);
    a.planes = reinterpret_cast<bf16*>(at + flag_bytes(g.M, g.K));
  }
  cudaError_t e = cudaSuccess;
  if (!g.a_ready)
    e = split(a, g.b_ready ? nullptr : &b, s);
  else if (!g.b_ready)
    e = split(b, nullptr, s);
  if (e != cudaSuccess) return e;
  const int w = tile_width(g);
  e = w == 128 ? g.b_mn ? launch<128, false, true>(g, a, b, w, all, s)
                        : launch<128, false, false>(g, a, b, w, all, s)
      : g.b_mn ? launch<256, false, true>(g, a, b, w, all, s)
               : launch<256, false, false>(g, a, b, w, all, s);
  if (e != cudaSuccess) return e;
  LinearProduct again = g;
  again.all_rows = all;
  again.row_flags = a.flag;
  again.slices = 1;
  again.segs = a.segs;
  again.tag = "linear_rows";
  return linear_simt(again, s);
}

cudaError_t linear_split_planes(const float* in, long long rows, int cols, long long ld, void* at,
                                cudaStream_t s) {
  const SplitOperand o = kept(at, in, rows, cols, ld);
  return split(o, nullptr, s);
}

cudaError_t linear_split_turned(const LinearProduct& g, void* a_planes, void* b_planes,
                                cudaStream_t s) {
  const SplitOperand a = kept(a_planes, nullptr, g.K, static_cast<int>(g.M), 0),
                     b = kept(b_planes, nullptr, g.K, g.N, 0);
  const int w = tile_width(g);
  int* all = static_cast<int*>(a_planes);
  const cudaError_t e = w == 128 ? launch<128, true, true>(g, a, b, w, all, s)
                                 : launch<256, true, true>(g, a, b, w, all, s);
  if (e != cudaSuccess) return e;
  LinearProduct again = g;
  again.all_rows = all;
  again.tag = "linear_rows";
  return linear_simt(again, s);
}

}  // namespace poetx
