// The matrix products of poetx_linear_* for many tokens, bf16, on CTA pairs:
//   C[M][N] = act(A B^T + bias) + residual   (A [M][K]; B [N][K] or, MN-major, [K][N])
// Each cluster of two CTAs computes tiles of 256 x 256, 224, 192 or 128 with
// tcgen05.mma.cta_group::2 over 64-wide K steps (a TMA ring of six to eight
// stages per CTA; five instead of six cost 3 us in 79 at 4096^3); two TMEM
// accumulators let a tile's epilogue run under the next tile's main loop.
//
// Roles, per CTA (576 threads, fewer with narrower tiles):
//   warp 0      TMA producer
//   warp 1      TMEM allocation; in the leader CTA the MMAs
//               (in both the whole warp runs the loop and one elected lane
//               issues, which keeps addresses and descriptors in uniform
//               registers: with the loop inside `lane == 0` a K step took 570
//               cycles of issue, more than the 512 its MMAs take)
//   the others  epilogue: a warp for 64 columns of each 32-row quarter of the
//               accumulator, 32 at a time: bias, (z,) activation and residual
//               in fp32 on the accumulator's values, one rounding, through a
//               2 KiB staging tile per warp.  The residual comes into the same
//               staging tile by TMA; a tile's first chunk is asked for while
//               its main loop still runs.  (Half as many warps with twice the
//               columns: 2048 -> 2048, T = 8192 with gelu 49.8 us instead of
//               47.3; staging tiles of 4 KiB leave five stages.)
// Rows that are not a multiple of 16 bytes apart (an odd number of output
// features) cannot be TMA tiles: there the staging tile is filled and emptied
// with plain loads and stores, a row at a time so that they coalesce.
//
// Tile order: kGroupM pairs of row tiles, then the next column: the tiles that
// run at one time (76 on 152 SMs) form a block of about 8 x 9, whose operands
// are 17 panels; in row order a wide B (14336 features: 56 tiles) would be read
// from HBM again in every round.
//
// Every wait is bounded as in gemm_pair.cu.
#include <algorithm>
#include <mutex>

#include "activation.cuh"
#include "internal.h"
#include "linear.h"
#include "ptx.cuh"
#include "tc_common.cuh"

namespace poetx {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kA = BM * BK * 2;      // this CTA's 128 rows, one K step
constexpr int kChunk = 32;           // columns that a warp stages at a time
constexpr int kSlot = 32 * kChunk * 2;

template <int BN, bool B_MN>
struct Shape {
  // this CTA's half of B, one K step (MN-major: whole 64-column boxes)
  static constexpr int B = B_MN ? (BN / 2 + 63) / 64 * 64 * BK * 2 : (BN / 2) * BK * 2;
  static constexpr int STAGE = kA + B;
  static constexpr int SIDES = (BN + 63) / 64;  // of 64 columns, four warps each
  static constexpr int EPI_WARPS = 4 * SIDES;
  static constexpr int THREADS = 64 + 32 * EPI_WARPS;
  static constexpr int STAGING = EPI_WARPS * kSlot;
  static constexpr int BIAS = EPI_WARPS * kChunk * 4;
  static constexpr int STAGES = (227 * 1024 - STAGING - BIAS - 512) / STAGE;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int SMEM = RING + STAGING + BIAS + 512;
  static constexpr uint32_t ACC = BN > 128 ? 256 : 128;  // TMEM columns of an accumulator
  static_assert(BN % 32 == 0 && (STAGE & 1023) == 0, "tiles on 1024 bytes");
};

constexpr int kGroupM = 8;

struct PairArgs {
  int m_pairs, n_tiles, k_steps, N;
  long long M, ld;
  int act, tma_rows;  // tma_rows: output rows are 16-byte aligned
  const float* bias;
  const bf16* residual;
  bf16* y;
  bf16* z;
  int* status;
};

__device__ __forceinline__ void unit_tile(int u, const PairArgs& p, int& mp, int& nt) {
  const int per_group = kGroupM * p.n_tiles;
  const int g = u / per_group, r = u - g * per_group;
  const int rows = min(kGroupM, p.m_pairs - g * kGroupM);
  mp = g * kGroupM + r % rows;
  nt = r / rows;
}

template <int ACT>
__device__ __forceinline__ void act_all(float (&v)[16]) {
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = act_f<ACT, true>(v[j]);
}

__device__ __forceinline__ void apply_act(int act, float (&v)[16]) {
  switch (act) {  // uniform over the grid
    case POETX_ACT_RELU: act_all<POETX_ACT_RELU>(v); break;
    case POETX_ACT_SILU: act_all<POETX_ACT_SILU>(v); break;
    case POETX_ACT_GELU: act_all<POETX_ACT_GELU>(v); break;
    case POETX_ACT_GELU_TANH: act_all<POETX_ACT_GELU_TANH>(v); break;
    default: break;
  }
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

template <int BN, bool B_MN>
__global__ void __launch_bounds__(Shape<BN, B_MN>::THREADS, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                       const __grid_constant__ CUtensorMap tmB,
                       const __grid_constant__ CUtensorMap tmY,
                       const __grid_constant__ CUtensorMap tmZ,
                       const __grid_constant__ CUtensorMap tmR, const PairArgs p) {
  using S = Shape<BN, B_MN>;
  constexpr int kStages = S::STAGES, kStage = S::STAGE, kRing = S::RING, kBN = BN;
  constexpr int kEpiWarps = S::EPI_WARPS;
  extern __shared__ __align__(1024) uint8_t base[];  // 128B-swizzled tiles start on 1024 bytes
  if ((smem_u32(base) & 1023u) != 0) {  // the declared alignment, which the tiles rely on
    if (threadIdx.x == 0) atomicCAS(p.status, 0, static_cast<int>(POETX_ERR_CUDA));
    return;
  }
  uint8_t* ring = base;  // stage s: A (16 KiB), then this CTA's half of B
  uint8_t* staging = base + kRing;
  float* bias_s = reinterpret_cast<float*>(staging + S::STAGING);
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(staging + S::STAGING + S::BIAS);  // leader
  uint64_t* empty_bar = full_bar + kStages;  // each CTA: its slot is free
  uint64_t* tfull_bar = empty_bar + kStages;  // [2] each CTA: accumulator ready
  uint64_t* tempty_bar = tfull_bar + 2;       // [2] leader: accumulator drained
  uint64_t* res_bar = tempty_bar + 2;         // [kEpiWarps] residual chunk arrived
  uint64_t* drain_bar = res_bar + kEpiWarps;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int units = p.m_pairs * p.n_tiles;
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
    for (int w = 0; w < kEpiWarps; ++w) mbar_init(&res_bar[w], 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * S::ACC);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers exist before either signals the other
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  const uint32_t full0 = map_peer(smem_u32(full_bar), 0);
  const uint32_t tempty0 = map_peer(smem_u32(tempty_bar), 0);

  if (warp == 0) {
    {
      // ---------------------------------------------------------- producer
      int stage = 0;
      uint32_t phase = 0;
      long long issued = 0;
      bool ok = true;
      for (int u = first; u < units && ok; u += step) {
        int mp, nt;
        unit_tile(u, p, mp, nt);
        const int a_row = mp * 2 * BM + static_cast<int>(rank) * BM;
        const int b_n = nt * kBN + static_cast<int>(rank) * (kBN / 2);
        for (int ks = 0; ks < p.k_steps; ++ks) {
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
            tma_load_2d_pair(a_dst, &tmA, bar, ks * BK, a_row);
            if (!B_MN) {
              tma_load_2d_pair(b_dst, &tmB, bar, ks * BK, b_n);
            } else {
              tma_load_2d_pair(b_dst, &tmB, bar, b_n, ks * BK);
              if (BN > 128) tma_load_2d_pair(b_dst + 8192, &tmB, bar, b_n + 64, ks * BK);
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
    }
  } else if (warp == 1) {
    if (leader) {
      // -------------------------------------------------- MMA issuer (pair)
      constexpr uint32_t IDESC = instr_desc_bf16(2 * BM, kBN, false, B_MN);
      const uint32_t empty_own = smem_u32(empty_bar);
      const uint32_t tfull_own = smem_u32(tfull_bar);
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      bool any_mma = false;
      for (int u = first; u < units && ok; u += step) {
        if (!mbar_wait_cluster(&tempty_bar[acc], acc_phase ^ 1, abort_flag)) {
          record_timeout(p.status, abort_flag);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc) * S::ACC;
        for (int ks = 0; ks < p.k_steps; ++ks) {
          if (!mbar_wait(&full_bar[stage], phase, abort_flag)) {
            record_timeout(p.status, abort_flag);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_base = smem_u32(ring) + stage * kStage;
          const uint32_t b_base = a_base + kA;
          // 16 of K: 32 bytes along a K-major row, 16 rows of 128 bytes MN-major
          const uint64_t adesc0 = smem_desc_sw128(a_base, 16, 1024);
          const uint64_t bdesc0 = smem_desc_sw128(b_base, B_MN ? 8192 : 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < BK / 16; ++j)
              umma_bf16_pair(d_tmem, adesc0 + j * 2, bdesc0 + j * (B_MN ? 128 : 2), IDESC,
                             (ks > 0 || j > 0) ? 1u : 0u);
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
    const int side = ew >> 2;      // its 64 (at the end of a 224-wide tile 32) columns
    const Staged slot{staging + ew * kSlot};
    int acc = 0;
    uint32_t acc_phase = 0;
    uint32_t res_phase = 0;
    bool res_pending = false;
    bool stores_pending = false;

    // The residual chunk at (row0, col) into the staging tile, which must be free.
    auto fetch_residual = [&](long long row0, int col) {
      if (p.tma_rows) {
        if (lane == 0) {
          mbar_arrive_expect_tx(&res_bar[ew], kSlot);
          tma_load_2d(slot.base, &tmR, &res_bar[ew], col, static_cast<int>(row0));
        }
        res_pending = true;
      } else {
        for (int r = 0; r < 32 && row0 + r < p.M; ++r)
          if (col + lane < p.N)
            *slot.value(r, lane) = p.residual[(row0 + r) * p.ld + col + lane];
        __syncwarp();
      }
    };
    // The staged chunk to `out`; the staging tile may be written again after
    // staging_free().
    auto store_chunk = [&](const CUtensorMap* map, bf16* out, long long row0, int col) {
      if (p.tma_rows) {
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(map, slot.base, col, static_cast<int>(row0));
          bulk_commit();
        }
        stores_pending = true;
      } else {
        __syncwarp();
        for (int r = 0; r < 32 && row0 + r < p.M; ++r)
          if (col + lane < p.N) out[(row0 + r) * p.ld + col + lane] = *slot.value(r, lane);
        __syncwarp();
      }
    };
    // 16 columns of z: the accumulator plus the chunk's bias
    auto load_z = [&](float (&v)[16], uint32_t taddr, const float* bias_w, int part) {
      uint32_t r[16];
      tmem_load_16(taddr + part * 16, r);
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
      if (p.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < 16; j += 4) {
          const float4 b = *reinterpret_cast<const float4*>(bias_w + part * 16 + j);
          v[j] += b.x, v[j + 1] += b.y, v[j + 2] += b.z, v[j + 3] += b.w;
        }
      }
    };
    auto staging_free = [&]() {
      if (stores_pending && lane == 0) bulk_wait_read_all();
      __syncwarp();
    };

    for (int u = first; u < units; u += step) {
      int mp, nt;
      unit_tile(u, p, mp, nt);
      const long long row0 = static_cast<long long>(mp) * 2 * BM + rank * BM + quarter * 32;
      const int side_col = nt * kBN + side * 64;
      const bool live = row0 < p.M && side_col < p.N;  // the same for the whole warp
      if (p.residual != nullptr && live) {
        staging_free();
        fetch_residual(row0, side_col);
      }
      const bool got = mbar_wait_cluster(&tfull_bar[acc], acc_phase, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        record_timeout(p.status, abort_flag);
        break;
      }
      tc_fence_after();
      bool timed_out = false;
#pragma unroll 1
      for (int c = 0; c < 64 && live; c += kChunk) {
        const int col = side_col + c;
        if (side * 64 + c >= BN || col >= p.N) break;
        const uint32_t t_chunk = tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) +
                                 static_cast<uint32_t>(acc) * S::ACC +
                                 static_cast<uint32_t>(side * 64 + c);
        if (c > 0 && p.residual != nullptr) {
          staging_free();
          fetch_residual(row0, col);
        }
        float* bias_w = bias_s + ew * kChunk;
        if (p.bias != nullptr) {
          __syncwarp();
          bias_w[lane] = col + lane < p.N ? __ldg(p.bias + col + lane) : 0.f;
          __syncwarp();
        }
        if (p.residual == nullptr) staging_free();
        if (p.residual != nullptr && p.tma_rows) {
          const bool have = mbar_wait(&res_bar[ew], res_phase, abort_flag);
          if (!__all_sync(0xffffffffu, have)) {
            timed_out = true;
            break;
          }
          res_phase ^= 1;
          res_pending = false;
        }
        uint4 res[kChunk / 8];
        if (p.residual != nullptr && p.z != nullptr) {  // z takes the staging tile first
#pragma unroll
          for (int q = 0; q < kChunk / 8; ++q) res[q] = *slot.piece(lane, q);
          __syncwarp();
        }
        if (p.z != nullptr) {
#pragma unroll 1
          for (int part = 0; part < kChunk / 16; ++part) {
            float v[16];
            load_z(v, t_chunk, bias_w, part);
            stage_part(slot, lane, part, v);
          }
          store_chunk(&tmZ, p.z, row0, col);
          staging_free();
          if (p.residual != nullptr) {
#pragma unroll
            for (int q = 0; q < kChunk / 8; ++q)
              st_shared_v4(slot.piece(lane, q), res[q].x, res[q].y, res[q].z, res[q].w);
          }
        }
#pragma unroll 1
        for (int part = 0; part < kChunk / 16; ++part) {
          float v[16];
          load_z(v, t_chunk, bias_w, part);
          apply_act(p.act, v);
          if (p.residual != nullptr) {  // this thread's own row: read, added, written over
#pragma unroll
            for (int q = 0; q < 2; ++q) {
              const uint4 r = *slot.piece(lane, 2 * part + q);
              const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f =
                    __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
                v[8 * q + 2 * i] += f.x;
                v[8 * q + 2 * i + 1] += f.y;
              }
            }
          }
          stage_part(slot, lane, part, v);
        }
        store_chunk(&tmY, p.y, row0, col);
      }
      if (timed_out) {
        record_timeout(p.status, abort_flag);
        break;
      }
      tc_fence_before();
      __syncwarp();
      // the accumulator is free again once both CTAs' epilogue warps have read it
      if (lane == 0) mbar_arrive_remote(tempty0 + static_cast<uint32_t>(acc * 8));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1;
    }
    if (lane == 0 && stores_pending) bulk_wait_all();
    if (res_pending) {  // only after a timeout: the load in flight lands before the CTA leaves
      const unsigned long long t0 = global_timer_ns();
      while (!mbar_try_wait(&res_bar[ew], res_phase) && global_timer_ns() - t0 < 10000000ull) {
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no CTA leaves while its peer may still signal or read it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * S::ACC);
  }
}

template <int BN, bool B_MN>
cudaError_t launch(const LinearProduct& g, cudaStream_t stream) {
  using S = Shape<BN, B_MN>;
  constexpr int kSmem = S::SMEM, kBN = BN;
  auto* kernel = linear_pair_kernel<BN, B_MN>;
  static bool ready[64] = {false};
  static int max_clusters[64] = {0};
  static std::mutex mu;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(S::THREADS);
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

  CUtensorMap tmA, tmB, tmY, tmZ, tmR;
  PairArgs p;
  p.tma_rows = g.ld % 8 == 0;
  if (!make_map(&tmA, g.A, g.M, g.K, g.lda, 2, 64, BM)) return cudaErrorInvalidValue;
  if (!(B_MN ? make_map(&tmB, g.B, g.K, g.N, g.ldb, 2, 64, 64)
             : make_map(&tmB, g.B, g.N, g.K, g.ldb, 2, 64, kBN / 2)))
    return cudaErrorInvalidValue;
  tmY = tmZ = tmR = tmA;  // stand-ins where a tensor is absent: never used
  if (p.tma_rows) {
    const auto map = [&](CUtensorMap* m, const void* at) {
      return at == nullptr || make_map(m, at, g.M, g.N, g.ld, 2, kChunk, 32, 64);
    };
    if (!map(&tmY, g.y) || !map(&tmZ, g.z) || !map(&tmR, g.residual))
      return cudaErrorInvalidValue;
  }
  p.m_pairs = static_cast<int>((g.M + 2 * BM - 1) / (2 * BM));
  p.n_tiles = (g.N + kBN - 1) / kBN;
  p.k_steps = (g.K + BK - 1) / BK;
  p.N = g.N;
  p.M = g.M;
  p.ld = g.ld;
  p.act = g.act;
  p.bias = g.bias;
  p.residual = static_cast<const bf16*>(g.residual);
  p.y = static_cast<bf16*>(g.y);
  p.z = static_cast<bf16*>(g.z);
  p.status = device_status_ptr();
  const int clusters = static_cast<int>(
      std::min<long long>(static_cast<long long>(p.m_pairs) * p.n_tiles, cmax));
  cfg.gridDim = dim3(2 * clusters);
  cfg.numAttrs = 2;
  prof_begin(g.tag, stream);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tmA, tmB, tmY, tmZ, tmR, p);
  prof_end(g.tag, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

namespace {

template <int BN>
cudaError_t by_layout(const LinearProduct& g, cudaStream_t s) {
  return g.b_mn ? launch<BN, true>(g, s) : launch<BN, false>(g, s);
}

}  // namespace

// The width of the tiles: the one whose rounds over the clusters take the least
// time, at 0.28 us for a 64-wide K step of a 256-wide tile (bound by the MMAs),
// 0.25 for 224, 0.23 for 192 and 0.17 for 128 (bound by the operands' loads).
// Bare products, us, of 256 / 224 / 192 / 128: 4096^3 78.7 / 73.4 / 76.1 / 85.0
// (4, 4, 5 and 7 rounds); 2048 -> 5632, T = 2048 32.5 / 30.1 / 32.1 / 33.4;
// 2048 -> 2048, T = 8192 44.8 / 49.5 / 43.8 / 47.8.
cudaError_t linear_pair(const LinearProduct& g, cudaStream_t s) {
  if (g.M <= 0 || g.N <= 0 || g.K <= 0) return cudaSuccess;
  const long long m_pairs = (g.M + 2 * BM - 1) / (2 * BM);
  const long long clusters = std::max(1, sm_count() / 2);
  const auto cost = [&](int width, int step) {
    return (m_pairs * ((g.N + width - 1) / width) + clusters - 1) / clusters * step;
  };
  const long long c256 = cost(256, 28), c224 = cost(224, 25), c192 = cost(192, 23),
                  c128 = cost(128, 17);
  const long long best = std::min(std::min(c256, c224), std::min(c192, c128));
  if (c256 == best) return by_layout<256>(g, s);
  if (c224 == best) return by_layout<224>(g, s);
  if (c192 == best) return by_layout<192>(g, s);
  return by_layout<128>(g, s);
}

}  // namespace poetx
