// The matrix products of poetx_linear_* for few tokens, bf16: the weight is
// read once and everything else is small, so the kernel is built round the
// weight's stream from memory.
//
// The weight's output features are the MMA's M (tiles of 128), the tokens its
// N (BT = 16 .. 256, the rest zero-filled by TMA): one tcgen05.mma covers 128
// features x BT tokens x 16.  K is split over the CTAs of a cluster (up to 8),
// so that a 4096 x 4096 weight still keeps every SM loading; each CTA streams
// its slice of the weight tile through a TMA ring.  The slices' fp32 partial
// tiles are then added through distributed shared memory, in rank order: CTA r
// finalises the tokens [r BT / S, (r + 1) BT / S) with bias, activation and
// residual and stores them, a warp per token (256 contiguous bytes).  No
// workspace, no atomics, the same bits on every run.
//
// Two CTAs fit on an SM (BT <= 128): one fills its ring while the other adds
// and stores.
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

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

template <int BT>
struct Shape {
  static constexpr int A = BM * BK * 2;
  static constexpr int B = BT * BK * 2;
  static constexpr int STAGE = A + B;
  static constexpr int CTAS = BT <= 128 ? 2 : 1;  // per SM
  static constexpr int STAGES = (CTAS == 2 ? 108 * 1024 : 216 * 1024) / STAGE;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int PART = BT * BM * 4;  // the partial tile, over the ring when it is done
  static constexpr int SMEM = RING + 256;
  static constexpr uint32_t TMEM_COLS = BT < 32 ? 32 : BT;
  static_assert(PART <= RING, "the partial tile fits the ring");
  static_assert(CTAS * (SMEM + 1024) <= 228 * 1024, "shared memory per SM");
};

struct StreamArgs {
  int N;  // output features (the MMA's M)
  int k_steps, splits, act;
  long long T, ld;
  const float* bias;
  const bf16* residual;
  bf16* y;
  bf16* z;
  int* status;
};

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void apply_act4(int act, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    switch (act) {  // uniform over the grid
      case POETX_ACT_RELU: v[j] = act_f<POETX_ACT_RELU, true>(v[j]); break;
      case POETX_ACT_SILU: v[j] = act_f<POETX_ACT_SILU, true>(v[j]); break;
      case POETX_ACT_GELU: v[j] = act_f<POETX_ACT_GELU, true>(v[j]); break;
      case POETX_ACT_GELU_TANH: v[j] = act_f<POETX_ACT_GELU_TANH, true>(v[j]); break;
      default: break;
    }
  }
}

// Four consecutive outputs at `at`, `live` of them inside the row.
__device__ __forceinline__ void store4(bf16* out, long long at, const float (&v)[4], int live,
                                       bool vec) {
  if (vec && live == 4) {
    *reinterpret_cast<uint2*>(out + at) =
        make_uint2(pack_bf16x2(__float_as_uint(v[0]), __float_as_uint(v[1])),
                   pack_bf16x2(__float_as_uint(v[2]), __float_as_uint(v[3])));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) out[at + j] = __float2bfloat16_rn(v[j]);
  }
}

// Adds the slices' partial values of features n .. n + 3 for this CTA's tokens,
// in rank order, and finishes them: one warp per token, U tokens at a time so
// that U x SPLITS remote loads are in flight.
template <int BT, int SPLITS, int U>
__device__ __forceinline__ void finish(const StreamArgs& p, const float* part, long long t0,
                                       int slice, int t_end, int n) {
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int live_n = min(4, p.N - n);
  const bool vec = p.ld % 4 == 0;
  float b4[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.bias != nullptr)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live_n) b4[j] = __ldg(p.bias + n + j);
  for (int t = slice * (BT / SPLITS) + warp; t < t_end; t += kWarps * U) {
    float4 q[U][SPLITS];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u * kWarps >= t_end) continue;
      const float* at = part + (t + u * kWarps) * BM + 4 * lane;
#pragma unroll
      for (int r = 0; r < SPLITS; ++r)
        q[u][r] = r == slice ? *reinterpret_cast<const float4*>(at)
                             : ld_cluster_f32x4(map_peer(smem_u32(at), static_cast<uint32_t>(r)));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u * kWarps >= t_end || live_n <= 0) continue;
      float v[4] = {q[u][0].x, q[u][0].y, q[u][0].z, q[u][0].w};
#pragma unroll
      for (int r = 1; r < SPLITS; ++r)
        v[0] += q[u][r].x, v[1] += q[u][r].y, v[2] += q[u][r].z, v[3] += q[u][r].w;
      const long long o = (t0 + t + u * kWarps) * p.ld + n;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] += b4[j];
      if (p.z != nullptr) store4(p.z, o, v, live_n, vec);
      apply_act4(p.act, v);
      if (p.residual != nullptr) {
        if (vec && live_n == 4) {
          const uint2 w = *reinterpret_cast<const uint2*>(p.residual + o);
          const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.x));
          const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w.y));
          v[0] += lo.x, v[1] += lo.y, v[2] += hi.x, v[3] += hi.y;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < live_n) v[j] += __bfloat162float(p.residual[o + j]);
        }
      }
      store4(p.y, o, v, live_n, vec);
    }
  }
}

// Grid: x = feature tile * splits + slice (a cluster along x), y = token tile.
template <int BT, bool A_MN>
__global__ void __launch_bounds__(kThreads, Shape<BT>::CTAS)
    linear_stream_kernel(const __grid_constant__ CUtensorMap tmW,
                         const __grid_constant__ CUtensorMap tmX, const StreamArgs p) {
  using S = Shape<BT>;
  extern __shared__ __align__(1024) uint8_t base[];
  if ((smem_u32(base) & 1023u) != 0) {  // the declared alignment, which the tiles rely on
    if (threadIdx.x == 0) atomicCAS(p.status, 0, static_cast<int>(POETX_ERR_CUDA));
    return;
  }
  uint64_t* full_bar = reinterpret_cast<uint64_t*>(base + S::RING);
  uint64_t* empty_bar = full_bar + S::STAGES;
  uint64_t* done_bar = empty_bar + S::STAGES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done_bar + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  const int slice = static_cast<int>(blockIdx.x) % p.splits;
  const int n0 = static_cast<int>(blockIdx.x) / p.splits * BM;
  const long long t0 = static_cast<long long>(blockIdx.y) * BT;
  const int live_t = static_cast<int>(min(static_cast<long long>(BT), p.T - t0));
  const int per = (p.k_steps + p.splits - 1) / p.splits;
  const int k_begin = slice * per;
  const int steps = max(0, min(p.k_steps, k_begin + per) - k_begin);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S::STAGES; ++s) {
      mbar_init(&full_bar[s], 1);
      mbar_init(&empty_bar[s], 1);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmW);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, S::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  pdl_trigger();

  // In both roles the whole warp runs the loop and one elected lane issues, so
  // that addresses and descriptors stay in uniform registers.
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    int issued = 0, st = 0;
    uint32_t phase = 1;
    for (; issued < steps; ++issued) {
      if (!mbar_wait(&empty_bar[st], phase, abort_flag)) {
        record_timeout(p.status, abort_flag);
        break;
      }
      if (elect_one()) {
        uint8_t* a_dst = base + st * S::STAGE;
        const int k = (k_begin + issued) * BK;
        mbar_arrive_expect_tx(&full_bar[st], S::STAGE);
        if (!A_MN) {
          tma_load_2d(a_dst, &tmW, &full_bar[st], k, n0);
        } else {
          tma_load_2d(a_dst, &tmW, &full_bar[st], n0, k);
          tma_load_2d(a_dst + 8192, &tmW, &full_bar[st], n0 + 64, k);
        }
        tma_load_2d(a_dst + S::A, &tmX, &full_bar[st], k, static_cast<int>(t0));
      }
      __syncwarp();
      if (++st == S::STAGES) {
        st = 0;
        phase ^= 1;
      }
    }
    // after a timeout the copies in flight land before the CTA leaves (bounded)
    if (issued < steps)
      for (int i = max(0, issued - S::STAGES); i < issued; ++i) {
        const unsigned long long w0 = global_timer_ns();
        while (!mbar_try_wait(&full_bar[i % S::STAGES],
                              static_cast<uint32_t>(i / S::STAGES) & 1) &&
               global_timer_ns() - w0 < 10000000ull) {
        }
      }
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    constexpr uint32_t IDESC = instr_desc_bf16(BM, BT, A_MN, false);
    int st = 0;
    uint32_t phase = 0;
    for (int i = 0; i < steps; ++i) {
      if (!mbar_wait(&full_bar[st], phase, abort_flag)) {
        record_timeout(p.status, abort_flag);
        break;
      }
      tc_fence_after();
      const uint32_t a_base = smem_u32(base) + st * S::STAGE;
      // 16 of K: 32 bytes along a K-major row, 16 rows of 128 bytes MN-major
      const uint64_t adesc0 = smem_desc_sw128(a_base, A_MN ? 8192 : 16, 1024);
      const uint64_t bdesc0 = smem_desc_sw128(a_base + S::A, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int j = 0; j < BK / 16; ++j)
          umma_bf16(tmem, adesc0 + j * (A_MN ? 128 : 2), bdesc0 + j * 2, IDESC,
                    (i > 0 || j > 0) ? 1u : 0u);
        umma_commit(&empty_bar[st]);
      }
      __syncwarp();
      if (++st == S::STAGES) {
        st = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) umma_commit(done_bar);  // also after a timeout: what was issued finishes first
  }
  __syncwarp();
  // the accumulator is complete and the ring free for the partial tile
  if (!mbar_wait(done_bar, 0, abort_flag, 2 * kWaitLimitNs)) record_timeout(p.status, abort_flag);
  tc_fence_after();
  float* part = reinterpret_cast<float*>(base);  // [BT tokens][BM features]
  {  // two warps per 32-feature quarter, alternate groups of 16 tokens
    const int quarter = warp & 3;
    const uint32_t t_base = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    float* col = part + quarter * 32 + lane;
#pragma unroll 2
    for (int c = (warp >> 2) * 16; c < live_t; c += 32) {
      uint32_t r[16];
      tmem_load_16(t_base + c, r);
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (c + j < live_t) col[(c + j) * BM] = steps > 0 ? __uint_as_float(r[j]) : 0.f;
    }
    tc_fence_before();
  }
  if (p.splits > 1)
    cluster_sync();  // every slice's partial tile is written
  else
    __syncthreads();

  // tokens [slice BT / splits, (slice + 1) BT / splits)
  const int t_end = min(live_t, (slice + 1) * (BT / p.splits));
  switch (p.splits) {
    case 1: finish<BT, 1, 2>(p, part, t0, slice, t_end, n0 + 4 * lane); break;
    case 2: finish<BT, 2, 2>(p, part, t0, slice, t_end, n0 + 4 * lane); break;
    case 4: finish<BT, 4, 1>(p, part, t0, slice, t_end, n0 + 4 * lane); break;
    default: finish<BT, 8, 1>(p, part, t0, slice, t_end, n0 + 4 * lane);
  }
  __syncthreads();
  if (p.splits > 1) cluster_sync();  // no CTA leaves while a peer still reads its tile
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, S::TMEM_COLS);
  }
}

// Slices of K.  Two CTAs share an SM where BT <= 128: up to 7/4 CTAs per SM
// (4096 -> 14336 features, one token: 112 / 224 / 448 CTAs take 21.5 / 20.8 / 22.8
// us; 14336 -> 4096: 128 / 256 CTAs 21.4 / 20.4; 2048 -> 5632: 88 / 176 / 352
// CTAs 7.2 / 6.8 / 10.2).  The closing sum costs by BT: a slice has at least
// four K steps, eight for BT = 128 (2048 -> 2048: 9.1 with four, 7.7 with eight),
// and beyond one CTA per SM eight, sixteen for BT >= 64 (4096 -> 4096, T = 128:
// 13.5 with eight, 12.1 in half as many slices).  One CTA per SM (BT = 256): as
// long as every cluster is resident at one time; clusters of eight do not fill
// the GPU's processing clusters (2048 -> 2048, T = 256: 8 slices ran in two waves,
// 19.2 us; 4 take 10.0).
int split_count(long long tiles, int k_steps, int bt, const int (&most)[4]) {
  int s = 1;
  for (int i = 1; i < 4; ++i) {
    const int next = 2 * s, per_slice = k_steps / next;
    const long long ctas = tiles * next;
    if (bt > 128) {
      if (per_slice < 4 || tiles > most[i]) break;
    } else {
      if (per_slice < (bt >= 128 ? 8 : 4) || 4 * ctas > 7ll * sm_count()) break;
      if (ctas > sm_count() && per_slice < (bt >= 64 ? 16 : 8)) break;
    }
    s = next;
  }
  return s;
}

template <int BT, bool A_MN>
cudaError_t launch(const LinearProduct& g, cudaStream_t stream) {
  using S = Shape<BT>;
  auto* kernel = linear_stream_kernel<BT, A_MN>;
  static bool ready[64] = {false};
  static int most[64][4] = {};  // clusters of 1, 2, 4, 8 CTAs resident at one time
  static std::mutex mu;
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!ready[dev]) {
      cudaError_t e =
          cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::SMEM);
      if (e != cudaSuccess) return e;
      cfg.numAttrs = 1;
      for (int i = 1; i < 4; ++i) {
        attr[0].val.clusterDim.x = 1u << i;
        cfg.gridDim = dim3(1u << i);
        e = cudaOccupancyMaxActiveClusters(&most[dev][i], kernel, &cfg);
        if (e != cudaSuccess) return e;
      }
      ready[dev] = true;
    }
  }
  CUtensorMap tmW, tmX;
  if (!(A_MN ? make_map(&tmW, g.B, g.K, g.N, g.ldb, 2, 64, 64)
             : make_map(&tmW, g.B, g.N, g.K, g.ldb, 2, 64, BM)))
    return cudaErrorInvalidValue;
  if (!make_map(&tmX, g.A, g.M, g.K, g.lda, 2, 64, BT)) return cudaErrorInvalidValue;
  StreamArgs p;
  p.N = g.N;
  p.k_steps = (g.K + BK - 1) / BK;
  p.act = g.act;
  p.T = g.M;
  p.ld = g.ld;
  p.bias = g.bias;
  p.residual = static_cast<const bf16*>(g.residual);
  p.y = static_cast<bf16*>(g.y);
  p.z = static_cast<bf16*>(g.z);
  p.status = device_status_ptr();
  const int n_tiles = (g.N + BM - 1) / BM;
  const long long t_tiles = (g.M + BT - 1) / BT;
  p.splits = split_count(n_tiles * t_tiles, p.k_steps, BT, most[dev]);
  cfg.gridDim = dim3(static_cast<unsigned>(n_tiles * p.splits), static_cast<unsigned>(t_tiles));
  attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
  cfg.numAttrs = 2;
  prof_begin(g.tag, stream);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tmW, tmX, p);
  prof_end(g.tag, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool A_MN>
cudaError_t run(const LinearProduct& g, cudaStream_t s) {
  if (g.M <= 16) return launch<16, A_MN>(g, s);
  if (g.M <= 32) return launch<32, A_MN>(g, s);
  if (g.M <= 64) return launch<64, A_MN>(g, s);
  if (g.M <= 128) return launch<128, A_MN>(g, s);
  return launch<256, A_MN>(g, s);
}

}  // namespace

cudaError_t linear_stream(const LinearProduct& g, cudaStream_t s) {
  if (g.M <= 0 || g.N <= 0 || g.K <= 0) return cudaSuccess;
  return g.b_mn ? run<true>(g, s) : run<false>(g, s);
}

}  // namespace poetx
