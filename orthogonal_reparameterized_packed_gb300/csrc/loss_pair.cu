// The products of the head's losses in bf16, on CTA pairs (loss.h):
//   logits  z = x W^T with the softmax's statistics in the epilogue
//   dx      dx = E W, each row times its factor, stored to its token's row
//   dw      dW = E^T x
// The kernel is linear_pair's with other epilogues: clusters of two CTAs compute
// tiles of 256 x 256 with tcgen05.mma.cta_group::2 over 64-wide K steps from a TMA
// ring, two TMEM accumulators; warp 0 loads, warp 1 issues the MMAs, and behind their
// warpgroup 16 epilogue warps take 64 columns of a 32-row quarter each.  dw's A is E as
// it lies, [rows][V]: an MN-major operand.  The rows are counted on the GPU: tiles
// behind the last row are not computed.
//
// The logits are never stored.  A tile's epilogue takes each z once: its
// exponential relative to the row's reference, the sum and the largest of 64
// columns; a token's entries are sorted, so that a warp finds those of its 64 columns
// by bisection.
//
// Every wait is bounded as in gemm_pair.cu.
#include <algorithm>
#include <climits>
#include <mutex>

#include "internal.h"
#include "loss.h"
#include "poetx.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace poetx {
namespace {

using bf16 = __nv_bfloat16;

// kLogits leaves the terms, kStats the statistics alone
enum Kind { kLogits, kStats, kDx, kDw };

constexpr int BN = 256;
constexpr int kA = BM * BK * 2;        // this CTA's 128 rows, one K step
constexpr int kB = (BN / 2) * BK * 2;  // this CTA's half of B, one K step
constexpr int kStage = kA + kB;
constexpr int kStages = 6;
constexpr int kRing = kStages * kStage;
constexpr int kSides = BN / 64;  // of 64 columns, four warps each
constexpr int kEpiWarps = 4 * kSides;
constexpr int kThreads = 128 + 32 * kEpiWarps;  // warps 2 and 3 have no role
constexpr int kChunk = 32;  // columns that a warp stages at a time
constexpr int kSlot = 32 * kChunk * 2;
constexpr int kSmem = kRing + kEpiWarps * kSlot + 256;
constexpr int kGroupM = 8;
constexpr uint32_t kAcc = 256;  // TMEM columns of an accumulator
constexpr int kLeastShare = 8;   // K steps of a slice
constexpr int kMaxSlices = 64;
constexpr int kSlots = 4;        // slices' tiles per cluster at most
constexpr float kCutCost = 20.f;
// The tensor core's accumulation truncates: over 2048 of K a logit comes out 4e-6 of
// itself too small, and the losses were 2.4e-6 off where a product rounded to nearest
// leaves 8e-7.  So the logits take some K steps at a time, and the epilogue adds those up
// in registers.  A piece of k features loses k 1.0e-9 of itself (measured, 256 to 768):
// 12 steps at a time 7.5e-7, 8 5e-7, 4 2.6e-7.  Shorter pieces leave the epilogue of the
// tile before less time, which the first two of them hide.  12 / 8 / 4 / 2 steps, us: one
// row of tiles, which W's bytes bound, losses of 256 tokens 1024 -> 32000 29.4 / 29.6 / 30.5 /
// 31.8, 2048 -> 32000 45.2 / 45.3 / 45.7 / 47.5, 4096 -> 128256 205 / 207 / 213 / 219; 1024 tokens
// 54.4 / 54.4 / 60.4 / 68.5, 90.0 / 89.9 / 95.9 / 107, 644 / 650 / 671 / 736.
constexpr int kDrain = 8;
constexpr int kDrainOneRow = 4;  // of tiles
static_assert(kSmem <= 227 * 1024, "shared memory per CTA");

// The order of the work.  Whole rounds of tiles over the clusters come first; the
// tiles of the last round (`rest`) are cut into `slices` of their K steps, all of one
// slice before the next, so that what runs at one time still shares its operands
// through L2 (parts of equal length at any K took 187 us where uncut tiles took 145:
// 1638 rows, d = 2048, V = 32000).  A slice's tile is kept in fp32, [256][256], and
// added up by loss_sum_kernel.
struct Schedule {
  int whole, rest, slices, share, k_steps, clusters, rows, drain;

  // In units of a K step (0.28 us): the rounds of the rest and, when it is cut, 0.4
  // for a slice's tile written and read and kCutCost for the launch.
  __device__ void plan(int tiles, int steps, int clusters_, bool may_cut) {
    whole = tiles;
    rest = 0;
    slices = 1;
    share = k_steps = steps;
    clusters = clusters_;
    const int left = tiles % clusters;
    if (!may_cut || left == 0) return;
    float best = static_cast<float>(steps);
    for (int i = 4; i <= 2 * kMaxSlices; i += i & (i - 1) ? i / 3 : i / 2) {  // 2, 3, 4, 6, 8, 12 ..
      const int n = i / 2, len = (steps + n - 1) / n;
      if (n * left > kSlots * clusters || len < kLeastShare) break;
      const float cost = static_cast<float>((n * left + clusters - 1) / clusters * len) +
                         0.4f * static_cast<float>(n * left) + kCutCost;
      if (cost < best && len * (n - 1) < steps) {
        best = cost;
        slices = n;
        share = len;
      }
    }
    if (slices > 1) {
      whole = tiles - left;
      rest = left;
    }
  }
  // Item i of cluster c: its tile, its K steps and where a slice goes (-1: whole).
  __device__ __forceinline__ bool item(int i, int c, int& tile, int& k0, int& k1,
                                       int& slot) const {
    const long long u = static_cast<long long>(i) * clusters + c;
    slot = -1;
    k0 = 0;
    k1 = k_steps;
    if (u < whole) {
      tile = static_cast<int>(u);
      return true;
    }
    if (u - whole >= static_cast<long long>(rest) * slices) return false;
    slot = static_cast<int>(u - whole);
    const int slice = slot / rest;
    tile = whole + slot - slice * rest;
    k0 = slice * share;
    k1 = min(k_steps, k0 + share);
    return true;
  }
};

struct PairArgs {
  int n_tiles, N, K, top;
  long long M;           // kDw: the output's rows
  long long first, block;
  long long ld, ldp;
  const int* only;       // null, or nothing is done while it is 0
  float unit;
  bool vec;              // output rows are 16-byte aligned
  float2* part;
  bf16* out;             // dx or dW
  float* acc;
  float* parts;          // of tiles cut along K; null: none is
  Schedule* schedule;    // what loss_sum_kernel goes by
  LossRows rows;
  int* status;
};

__device__ __forceinline__ void unit_tile(int u, int m_pairs, int n_tiles, int& mp, int& nt) {
  const int per_group = kGroupM * n_tiles;
  const int g = u / per_group, r = u - g * per_group;
  const int rows = min(kGroupM, m_pairs - g * kGroupM);
  mp = g * kGroupM + r % rows;
  nt = r / rows;
}

// A warp's staging tile: 32 rows of 64 bytes as TMA's 64-byte swizzle lays them out.
struct Staged {
  uint8_t* base;

  __device__ __forceinline__ uint4* piece(int row, int q) const {  // 16 bytes
    return reinterpret_cast<uint4*>(base + row * 64 + ((q ^ (row >> 1 & 3)) << 4));
  }
  __device__ __forceinline__ bf16* value(int row, int col) const {
    return reinterpret_cast<bf16*>(piece(row, col >> 3)) + (col & 7);
  }
};

// 16 values of this thread's row -> pieces 2 part, 2 part + 1 of its staging row
__device__ __forceinline__ void stage_part(const Staged& slot, int lane, int part,
                                           const float (&v)[16]) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    uint32_t w[4];
#pragma unroll
    for (int h = 0; h < 4; ++h)
      w[h] = pack_bf16x2(__float_as_uint(v[8 * q + 2 * h]), __float_as_uint(v[8 * q + 2 * h + 1]));
    st_shared_v4(slot.piece(lane, 2 * part + q), w[0], w[1], w[2], w[3]);
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Registers.  The logits' epilogue keeps 64 sums a thread and takes 112 (512 threads),
// the first warpgroup keeps 32 (128): 61440, which is what 640 threads have at the
// launch with 96 each.  With 96 in the epilogue the sums spilled, and the product took
// twice the time.  Fewer at the launch would make the epilogue wait for ever: launch()
// refuses that.
constexpr int kLaunchRegisters = 96;
static_assert(kThreads == 640 && 512 * 112 + 128 * 32 <= kThreads * kLaunchRegisters, "registers");

__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 32;");
}
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 112;");
}

template <int KIND>
__global__ void __launch_bounds__(kThreads, 1)
    loss_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ CUtensorMap tmB,
                     const __grid_constant__ CUtensorMap tmOut, const PairArgs p) {
  constexpr bool LOGITS = KIND == kLogits || KIND == kStats, STORE = KIND == kLogits;
  constexpr bool A_MN = KIND == kDw, B_MN = !LOGITS;
  extern __shared__ __align__(1024) uint8_t base[];  // 128B-swizzled tiles start on 1024 bytes
  if ((smem_u32(base) & 1023u) != 0) {  // the declared alignment, which the tiles rely on
    if (threadIdx.x == 0) atomicCAS(p.status, 0, static_cast<int>(POETX_ERR_CUDA));
    return;
  }
  uint8_t* ring = base;  // stage s: A (16 KiB), then this CTA's half of B
  uint8_t* staging = base + kRing;
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(staging + kEpiWarps * kSlot);  // leader
  uint64_t* empty_bar = full_bar + kStages;   // each CTA: its slot is free
  uint64_t* tfull_bar = empty_bar + kStages;  // [2] each CTA: accumulator ready
  uint64_t* tempty_bar = tfull_bar + 2;       // [2] leader: accumulator drained
  uint64_t* drain_bar = tempty_bar + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  Schedule* schedule = reinterpret_cast<Schedule*>(tmem_slot + 2);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int first_unit = static_cast<int>(cluster_id_x());
  const int step = static_cast<int>(cluster_count_x());

  if (STORE && p.only != nullptr) {  // the same for every CTA, before anything is set up
    pdl_wait();
    if (*p.only == 0) return;
  }
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
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * kAcc);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  // the same for every thread of the grid
  const long long counted = *p.rows.count;
  const long long n = max(0ll, min(p.block, counted - p.first));  // rows of this block
  const long long M = KIND == kDw ? p.M : n;
  const int m_pairs = static_cast<int>((M + 2 * BM - 1) / (2 * BM));
  const int k_steps = static_cast<int>(((KIND == kDw ? n : p.K) + BK - 1) / BK);
  int units = m_pairs * p.n_tiles;
  if (KIND == kDw && n == 0 && p.first > 0) units = 0;  // the block before was the last
  const bool products = k_steps > 0;  // dW without a row is 0
  if (threadIdx.x == 0) {
    schedule->rows = static_cast<int>(n);
    schedule->drain = m_pairs > 1 ? kDrain : kDrainOneRow;  // of the logits
    schedule->plan(units, k_steps, step, !LOGITS && p.parts != nullptr);
    if (blockIdx.x == 0 && p.parts != nullptr) *p.schedule = *schedule;
  }
  __syncthreads();
  const Schedule& todo = *schedule;

  const uint32_t full0 = map_peer(smem_u32(full_bar), 0);
  const uint32_t tempty0 = map_peer(smem_u32(tempty_bar), 0);

  if (warp < 4) {  // the same for each warpgroup, as setmaxnreg needs
    if (LOGITS) registers_down();
    if (warp == 0) {
      // ------------------------------------------------------------ producer
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      int tile, ks0, ks1, part_slot;
      for (int i = 0; products && ok && todo.item(i, first_unit, tile, ks0, ks1, part_slot); ++i) {
        int mp, nt;
        unit_tile(tile, m_pairs, p.n_tiles, mp, nt);
        const int a_row = mp * 2 * BM + static_cast<int>(rank) * BM;
        const int b_n = nt * BN + static_cast<int>(rank) * (BN / 2);
        for (int ks = ks0; ks < ks1; ++ks) {
          if (!mbar_wait(&empty_bar[stage], phase ^ 1, abort_flag)) {
            record_timeout(p.status, abort_flag);
            ok = false;
            break;
          }
          if (elect_one()) {
            if (leader) mbar_arrive_expect_tx(&full_bar[stage], 2 * kStage);
            uint8_t* a_dst = ring + stage * kStage;
            uint8_t* b_dst = a_dst + kA;
            const uint32_t bar = full0 + static_cast<uint32_t>(stage * 8);
            if (!A_MN) {
              tma_load_2d_pair(a_dst, &tmA, bar, ks * BK, a_row);
            } else {
              tma_load_2d_pair(a_dst, &tmA, bar, a_row, ks * BK);
              tma_load_2d_pair(a_dst + 8192, &tmA, bar, a_row + 64, ks * BK);
            }
            if (!B_MN) {
              tma_load_2d_pair(b_dst, &tmB, bar, ks * BK, b_n);
            } else {
              tma_load_2d_pair(b_dst, &tmB, bar, b_n, ks * BK);
              tma_load_2d_pair(b_dst + 8192, &tmB, bar, b_n + 64, ks * BK);
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
      // every slot this CTA filled is released again before it leaves
      const int outstanding = issued < kStages ? static_cast<int>(issued) : kStages;
      int st = stage;
      uint32_t ph = phase;
      for (int i = 0; i < outstanding; ++i) {
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
        constexpr uint32_t IDESC = instr_desc_bf16(2 * BM, BN, A_MN, B_MN);
        const uint32_t empty_own = smem_u32(empty_bar);
        const uint32_t tfull_own = smem_u32(tfull_bar);
        int stage = 0;
        uint32_t phase = 0;
        int acc = 0;
        uint32_t acc_phase = 0;
        bool ok = true;
        bool any_mma = false;
        int tile, ks0, ks1, part_slot;
        for (int i = 0;
             products && ok && todo.item(i, first_unit, tile, ks0, ks1, part_slot); ++i) {
          const int piece = LOGITS ? todo.drain : ks1 - ks0;
          for (int kc = ks0; kc < ks1 && ok; kc += piece) {
            const int kc1 = min(ks1, kc + piece);
            if (!mbar_wait_cluster(&tempty_bar[acc], acc_phase ^ 1, abort_flag)) {
              record_timeout(p.status, abort_flag);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc) * kAcc;
            for (int ks = kc; ks < kc1; ++ks) {
              if (!mbar_wait(&full_bar[stage], phase, abort_flag)) {
                record_timeout(p.status, abort_flag);
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t a_base = smem_u32(ring) + stage * kStage;
              const uint32_t b_base = a_base + kA;
              // 16 of K: 32 bytes along a K-major row, 16 rows of 128 bytes MN-major
              const uint64_t adesc0 = smem_desc_sw128(a_base, A_MN ? 8192 : 16, 1024);
              const uint64_t bdesc0 = smem_desc_sw128(b_base, B_MN ? 8192 : 16, 1024);
              if (elect_one()) {
#pragma unroll
                for (int j = 0; j < BK / 16; ++j)
                  umma_bf16_pair(d_tmem, adesc0 + j * (A_MN ? 128 : 2),
                                 bdesc0 + j * (B_MN ? 128 : 2), IDESC,
                                 (ks > kc || j > 0) ? 1u : 0u);
                // the slot is free in both CTAs once the MMAs have read it
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
    }
  } else {
    // ------------------------------------------------------------ epilogue
    if (LOGITS) registers_up();
    const int ew = warp - 4;
    const int quarter = warp & 3;  // the TMEM lanes this warp may read
    const int side = ew >> 2;      // its 64 columns
    const Staged slot{staging + ew * kSlot};
    int acc = 0;
    uint32_t acc_phase = 0;
    bool stores_pending = false;
    const float most = KIND == kDw ? *p.rows.most : 0.f;
    const bool last = KIND != kDw || p.acc == nullptr || p.first + p.block >= counted;

    const auto staging_free = [&]() {
      if (stores_pending && lane == 0) bulk_wait_read_all();
      __syncwarp();
    };
    // The staged chunk by TMA; the staging tile may be written again after
    // staging_free().
    const auto store_tma = [&](long long row0, int col) {
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(&tmOut, slot.base, col, static_cast<int>(row0));
        bulk_commit();
      }
      stores_pending = true;
    };
    // The staged chunk with plain stores, row r to output row `to` of lane r (-1:
    // none); rows of 16-byte pieces, or an odd length value by value.
    const auto store_rows = [&](int to, int col) {
      __syncwarp();
      if (p.vec) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + lane / 4, q = lane % 4;
          const int row = __shfl_sync(0xffffffffu, to, r);
          if (row >= 0 && col + q * 8 < p.N)
            *reinterpret_cast<uint4*>(p.out + static_cast<long long>(row) * p.ld + col + q * 8) =
                *slot.piece(r, q);
        }
      } else {
        for (int r = 0; r < 32; ++r) {
          const int row = __shfl_sync(0xffffffffu, to, r);
          if (row >= 0 && col + lane < p.N)
            p.out[static_cast<long long>(row) * p.ld + col + lane] = *slot.value(r, lane);
        }
      }
      __syncwarp();
    };

    if (LOGITS) {
      // Nothing but the sums lives through the main loop: registers are short.
      const volatile Schedule* plan = schedule;
      for (int u = first_unit; u < plan->whole; u += plan->clusters) {
        const int chunks = (plan->k_steps + plan->drain - 1) / plan->drain;
        float z[64];
        bool got = true;
        for (int kc = 0; kc < chunks; ++kc) {
          got = __all_sync(0xffffffffu,
                           mbar_wait_cluster(&tfull_bar[acc], acc_phase, abort_flag));
          if (!got) break;
          tc_fence_after();
          const uint32_t t_side = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                  static_cast<uint32_t>(acc) * kAcc +
                                  static_cast<uint32_t>(side * 64);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t r[16];
            tmem_load_16(t_side + q * 16, r);
            if (kc == 0) {
#pragma unroll
              for (int j = 0; j < 16; ++j) z[16 * q + j] = __uint_as_float(r[j]);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j) z[16 * q + j] += __uint_as_float(r[j]);
            }
          }
          tc_fence_before();
          __syncwarp();
          // the accumulator is free again once both CTAs' epilogue warps have read it
          if (lane == 0) mbar_arrive_remote_relaxed(tempty0 + static_cast<uint32_t>(acc * 8));
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1;
        }
        if (!got) {
          record_timeout(p.status, abort_flag);
          break;
        }
        int at_unit = u;
        asm volatile("" : "+r"(at_unit));  // what follows is computed here, not before
        const int rows = plan->rows;
        int mp, nt;
        unit_tile(at_unit, (rows + 2 * BM - 1) / (2 * BM), p.n_tiles, mp, nt);
        const int row0 = mp * 2 * BM + static_cast<int>(rank) * BM + quarter * 32;
        const int side_col = nt * BN + side * 64;
        const int row = row0 + lane;
        const int in = p.N - side_col;  // columns in the vocabulary
        // E's rows behind the last are written up to a whole K step of dW
        if (row0 >= (rows + BK - 1) / BK * BK || in <= 0) continue;
        const bool on = row < rows;
        float ref = 0.f;
        int token = 0, k = p.top, next = INT_MAX;  // the row's next entry from side_col on
        if (on) {
          token = p.rows.token[p.first + row];
          if (STORE) ref = p.rows.ref[p.first + row];
          const int* idx = p.rows.index + static_cast<long long>(token) * p.top;
          int lo = 0;
          while (lo < k) {
            const int mid = (lo + k) >> 1;
            if (idx[mid] < side_col)
              lo = mid + 1;
            else
              k = mid;
          }
          if (k < p.top) next = idx[k];
        }
        if (in < 64) {
#pragma unroll
          for (int j = 0; j < 64; ++j)
            if (j >= in) z[j] = -INFINITY;
        }
        if (STORE && !on) {  // rows behind the last: their terms are 0, whatever W holds
#pragma unroll
          for (int j = 0; j < 64; ++j) z[j] = -INFINITY;
        }
        float sum = 0.f, top_z = -INFINITY;
        if (!STORE) {  // the reference is the largest of the 64 columns
#pragma unroll
          for (int j = 0; j < 64; j += 4)
            top_z = fmaxf(top_z, fmaxf(fmaxf(z[j], z[j + 1]), fmaxf(z[j + 2], z[j + 3])));
          ref = top_z == -INFINITY ? 0.f : top_z * p.unit;
        }
#pragma unroll
        for (int c = 0; c < 64; c += kChunk) {
          if (c >= in) break;
          if (stores_pending) staging_free();
          // the logits at this row's entries
          const int end = min(side_col + c + kChunk, p.N);
          while (__any_sync(0xffffffffu, next < end)) {
            const int at = next - side_col;
            float of_entry = 0.f;
#pragma unroll
            for (int j = c; j < c + kChunk; ++j)
              if (j == at) of_entry = z[j];
            if (next < end) {
              const long long to = static_cast<long long>(token) * p.top + k;
              p.rows.z[to] = of_entry;
              next = ++k < p.top ? p.rows.index[to + 1] : INT_MAX;
            }
          }
#pragma unroll
          for (int j = c; j < c + kChunk; j += 4) {
            if (STORE)
              top_z = fmaxf(top_z, fmaxf(fmaxf(z[j], z[j + 1]), fmaxf(z[j + 2], z[j + 3])));
#pragma unroll
            for (int i = j; i < j + 4; ++i) z[i] = exp2_fast(fmaf(z[i], p.unit, -ref));
            sum += (z[j] + z[j + 1]) + (z[j + 2] + z[j + 3]);
          }
          if (STORE) {
#pragma unroll
            for (int q = 0; q < kChunk / 8; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int h = 0; h < 4; ++h)
                w[h] = pack_bf16x2(__float_as_uint(z[c + 8 * q + 2 * h]),
                                   __float_as_uint(z[c + 8 * q + 2 * h + 1]));
              st_shared_v4(slot.piece(lane, q), w[0], w[1], w[2], w[3]);
            }
            store_tma(row0, side_col + c);
          }
        }
        if (on)
          p.part[(static_cast<long long>(nt) * kSides + side) * p.ldp + row] =
              make_float2(top_z, sum);
      }
    }

    int tile, ks0, ks1, part_slot;
    for (int i = 0; !LOGITS && todo.item(i, first_unit, tile, ks0, ks1, part_slot); ++i) {
      int mp, nt;
      unit_tile(tile, m_pairs, p.n_tiles, mp, nt);
      const long long row0 = static_cast<long long>(mp) * 2 * BM + rank * BM + quarter * 32;
      const int side_col = nt * BN + side * 64;
      const long long row = row0 + lane;
      const bool live = row0 < M && side_col < p.N;  // the same for the whole warp
      const bool on = row < M;
      // what the row needs besides the accumulator, under the main loop
      int token = -1;
      float2 scale = make_float2(0.f, 0.f);
      if (KIND == kDx && live && on) {
        token = p.rows.token[p.first + row];
        scale = p.rows.scale[p.first + row];
      }
      if (KIND == kDw && p.acc != nullptr && p.first > 0 && live && on) {
        // the sums of the blocks before, into L2 under the main loop
        const float* sums = p.acc + row * p.N + side_col;
        for (int c = 0; c < 64 && side_col + c < p.N; c += 32)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(sums + c));
      }
      if (products) {
        const bool got = mbar_wait_cluster(&tfull_bar[acc], acc_phase, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          record_timeout(p.status, abort_flag);
          break;
        }
        tc_fence_after();
      }
      const uint32_t t_side = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                              static_cast<uint32_t>(acc) * kAcc + static_cast<uint32_t>(side * 64);
      if (part_slot >= 0 && live) {
        float* to = p.parts + static_cast<long long>(part_slot) * 2 * BM * BN +
                    (rank * BM + quarter * 32 + lane) * BN + side * 64;
#pragma unroll 1
        for (int c = 0; c < 64; c += 16) {
          uint32_t r[16];
          tmem_load_16(t_side + c, r);
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<uint4*>(to + c + j) = make_uint4(r[j], r[j + 1], r[j + 2], r[j + 3]);
        }
      }
#pragma unroll 1
      for (int c = 0; c < 64 && live && part_slot < 0; c += kChunk) {
        const int col = side_col + c;
        if (col >= p.N) break;
        if (stores_pending) staging_free();
        float* acc_row = nullptr;
        if (KIND == kDw && p.acc != nullptr)
          acc_row = p.acc + row * p.N + col;
#pragma unroll 1
        for (int part = 0; part < kChunk / 16; ++part) {
          float v[16];
          if (products) {
            uint32_t r[16];
            tmem_load_16(t_side + c + part * 16, r);
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0.f;
          }
          const int in = p.N - col - part * 16;
          if (KIND == kDx) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = v[j] * scale.x * scale.y;
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] *= most;
            if (acc_row != nullptr && on) {
              float* at = acc_row + part * 16;
              if (p.vec) {  // whole quads are inside
#pragma unroll
                for (int j = 0; j < 16; j += 4) {
                  if (j >= in) continue;
                  float4* quad = reinterpret_cast<float4*>(at + j);
                  if (p.first > 0) {
                    const float4 q = *quad;
                    v[j] += q.x, v[j + 1] += q.y, v[j + 2] += q.z, v[j + 3] += q.w;
                  }
                  if (!last) *quad = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
                }
              } else {
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  if (j < in) {
                    if (p.first > 0) v[j] += at[j];
                    if (!last) at[j] = v[j];
                  }
              }
            }
          }
          stage_part(slot, lane, part, v);
        }
        if (KIND == kDx) {
          store_rows(token, col);
        } else if (last) {
          if (p.vec)
            store_tma(row0, col);
          else
            store_rows(on ? static_cast<int>(row) : -1, col);
        } else {
          __syncwarp();
        }
      }
      if (products) {
        tc_fence_before();
        __syncwarp();
        // the accumulator is free again once both CTAs' epilogue warps have read it
        if (lane == 0) mbar_arrive_remote_relaxed(tempty0 + static_cast<uint32_t>(acc * 8));
        acc ^= 1;
        if (acc == 0) acc_phase ^= 1;
      }
    }
    if (lane == 0 && stores_pending) bulk_wait_all();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal or read it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kAcc);
  }
}

// The tiles that were cut along K: their slices added up in order, then
// what the epilogue does.  A CTA takes four rows of a tile, a thread four
// columns.
constexpr int kSumRows = 4;
constexpr int kSumThreads = 256;

template <int KIND>
__global__ void __launch_bounds__(kSumThreads) loss_sum_kernel(const PairArgs p) {
  pdl_wait();
  pdl_trigger();
  const int rest = p.schedule->rest, slices = p.schedule->slices, whole = p.schedule->whole;
  const long long counted = *p.rows.count;
  const long long M = KIND == kDw ? p.M : max(0ll, min(p.block, counted - p.first));
  const int m_pairs = static_cast<int>((M + 2 * BM - 1) / (2 * BM));
  const bool last = KIND != kDw || p.acc == nullptr || p.first + p.block >= counted;
  constexpr int kPieces = 2 * BM / kSumRows;
  for (int item = blockIdx.x; item < rest * kPieces; item += gridDim.x) {
    const int j = item / kPieces;
    int mp, nt;
    unit_tile(whole + j, m_pairs, p.n_tiles, mp, nt);
    const int col = threadIdx.x % 64 * 4, to_col = nt * BN + col;
    const int in = min(4, p.N - to_col);
    const int r = item % kPieces * kSumRows + threadIdx.x / 64;
    const long long row = static_cast<long long>(mp) * 2 * BM + r;
    if (row >= M || in <= 0) continue;
    const float* part = p.parts + static_cast<long long>(j) * 2 * BM * BN + r * BN + col;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int i = 0; i < slices; ++i) {
      const float4 q =
          *reinterpret_cast<const float4*>(part + static_cast<long long>(i) * rest * 2 * BM * BN);
      v[0] += q.x, v[1] += q.y, v[2] += q.z, v[3] += q.w;
    }
    long long to = row;
    if (KIND == kDx) {
      to = p.rows.token[p.first + row];
      const float2 scale = p.rows.scale[p.first + row];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = v[i] * scale.x * scale.y;
    } else {
      const float most = *p.rows.most;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] *= most;
        if (p.acc == nullptr || i >= in) continue;
        float* sum = p.acc + row * p.N + to_col + i;
        if (p.first > 0) v[i] += *sum;
        if (!last) *sum = v[i];
      }
    }
    if (!last) continue;
    bf16* out = p.out + to * p.ld + to_col;
    if (p.vec) {
      *reinterpret_cast<uint2*>(out) =
          make_uint2(pack_bf16x2(__float_as_uint(v[0]), __float_as_uint(v[1])),
                     pack_bf16x2(__float_as_uint(v[2]), __float_as_uint(v[3])));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < in) out[i] = __float2bfloat16_rn(v[i]);
    }
  }
}

template <int KIND>
cudaError_t sum_slices(const PairArgs& p, cudaStream_t stream) {
  prof_begin("loss_sum", stream);
  const cudaError_t e =
      launch_pdl(loss_sum_kernel<KIND>, dim3(8 * static_cast<unsigned>(sm_count())),
                 dim3(kSumThreads), 0, stream, p);
  prof_end("loss_sum", stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int KIND>
cudaError_t launch(const CUtensorMap& tmA, const CUtensorMap& tmB, const CUtensorMap& tmOut,
                   const PairArgs& p, long long most_units, const char* tag,
                   cudaStream_t stream) {
  auto* kernel = loss_pair_kernel<KIND>;
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
      if (KIND == kLogits || KIND == kStats) {
        cudaFuncAttributes has;
        e = cudaFuncGetAttributes(&has, kernel);
        if (e != cudaSuccess) return e;
        if (has.numRegs < kLaunchRegisters) return cudaErrorLaunchOutOfResources;
      }
      max_clusters[dev] = n;
      ready[dev] = true;
    }
    cmax = max_clusters[dev];
  }
  // tiles that may be cut keep every cluster busy
  cfg.gridDim = dim3(
      2 * static_cast<unsigned>(p.parts != nullptr ? cmax : std::min<long long>(most_units, cmax)));
  cfg.numAttrs = 2;
  prof_begin(tag, stream);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tmA, tmB, tmOut, p);
  prof_end(tag, stream);
  if (e == cudaSuccess) e = cudaGetLastError();
  if constexpr (KIND == kDx || KIND == kDw) {
    if (e == cudaSuccess && p.parts != nullptr) e = sum_slices<KIND>(p, stream);
  }
  return e;
}

PairArgs common(const LossProducts& g) {
  PairArgs p = {};
  p.top = g.top;
  p.first = g.first;
  p.block = g.block;
  p.unit = g.unit;
  p.rows = g.rows;
  p.status = device_status_ptr();
  return p;
}

long long pairs(long long rows) { return (rows + 2 * BM - 1) / (2 * BM); }

}  // namespace

bool loss_cuts(long long K) { return (K + BK - 1) / BK > static_cast<long long>(kCutCost); }

size_t loss_cut_bytes() {
  return static_cast<size_t>(sm_count() / 2 + 1) * kSlots * 2 * BM * BN * sizeof(float);
}

int loss_parts(int V) { return (V + 63) / 64; }

cudaError_t loss_logits(const LossProducts& g, bool only_again, cudaStream_t s) {
  PairArgs p = common(g);
  CUtensorMap tmA, tmB, tmE;
  if (!make_map(&tmA, g.x, g.x_rows, g.d, g.ldx, 2, 64, BM) ||
      !make_map(&tmB, g.W, g.V, g.d, g.ldw, 2, 64, BN / 2))
    return cudaErrorInvalidValue;
  tmE = tmA;  // a stand-in: not used
  const bool store = g.E != nullptr;
  if (store && !make_map(&tmE, g.E, g.block, g.V, g.lde, 2, kChunk, 32, 64))
    return cudaErrorInvalidValue;
  p.n_tiles = (g.V + BN - 1) / BN;
  p.N = g.V;
  p.K = g.d;
  p.part = g.part;
  p.ldp = g.ldp;
  if (only_again) p.only = g.rows.again + g.first / g.block;
  const long long tiles = pairs(g.block) * p.n_tiles;
  if (!store) return launch<kStats>(tmA, tmB, tmE, p, tiles, "loss_logits", s);
  return launch<kLogits>(tmA, tmB, tmE, p, tiles, only_again ? "loss_logits_again" : "loss_logits",
                         s);
}

cudaError_t loss_dx(const LossProducts& g, cudaStream_t s) {
  PairArgs p = common(g);
  CUtensorMap tmA, tmB;
  if (!make_map(&tmA, g.E, g.block, g.V, g.lde, 2, 64, BM) ||
      !make_map(&tmB, g.W, g.V, g.d, g.ldw, 2, 64, 64))
    return cudaErrorInvalidValue;
  p.n_tiles = (g.d + BN - 1) / BN;
  p.N = g.d;
  p.K = g.V;
  p.parts = loss_cuts(g.V) ? g.parts : nullptr;
  p.schedule = static_cast<Schedule*>(g.schedule);
  p.out = static_cast<bf16*>(g.dx);
  p.ld = g.d;
  p.vec = g.d % 8 == 0;
  return launch<kDx>(tmA, tmB, tmA, p, pairs(g.block) * p.n_tiles, "loss_dx", s);
}

cudaError_t loss_dw(const LossProducts& g, cudaStream_t s) {
  PairArgs p = common(g);
  CUtensorMap tmA, tmB, tmOut;
  if (!make_map(&tmA, g.E, g.block, g.V, g.lde, 2, 64, 64) ||
      !make_map(&tmB, g.x, g.x_rows, g.d, g.ldx, 2, 64, 64))
    return cudaErrorInvalidValue;
  tmOut = tmA;
  p.vec = g.d % 8 == 0;
  if (p.vec && !make_map(&tmOut, g.dW, g.V, g.d, g.d, 2, kChunk, 32, 64))
    return cudaErrorInvalidValue;
  p.n_tiles = (g.d + BN - 1) / BN;
  p.N = g.d;
  p.M = g.V;
  p.out = static_cast<bf16*>(g.dW);
  p.acc = g.acc;
  p.parts = loss_cuts(g.block) ? g.parts : nullptr;
  p.schedule = static_cast<Schedule*>(g.schedule);
  p.ld = g.d;
  return launch<kDw>(tmA, tmB, tmOut, p, pairs(g.V) * p.n_tiles, "loss_dw", s);
}

}  // namespace poetx
