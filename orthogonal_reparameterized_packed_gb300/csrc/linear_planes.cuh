// An fp32 value as the sum of three bf16 ones (linear_split.cu), for the kernels that
// make such planes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace poetx {
namespace {

constexpr int kPlanes = 3;
constexpr unsigned kLeastBits = (127u - 109u) << 23, kMostBits = (127u + 60u) << 23;

// Whether v is neither 0 nor of a magnitude that the planes take; infinities and NaN
// have larger bits than 2^60.
__device__ __forceinline__ bool outside_planes(float v) {
  const unsigned u = __float_as_uint(v) & 0x7fffffffu;
  return u != 0 && u - kLeastBits > kMostBits - kLeastBits;
}

// Four values to the planes, 8 bytes each, which lie `stride` elements apart.
__device__ __forceinline__ void store_planes(__nv_bfloat16* at, long long stride, float (&v)[4]) {
#pragma unroll
  for (int s = 0; s < kPlanes; ++s) {
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __nv_bfloat162 q = __floats2bfloat162_rn(v[2 * h], v[2 * h + 1]);
      const float2 f = __bfloat1622float2(q);
      v[2 * h] -= f.x;  // exact: the rounding error of a bf16 rounding
      v[2 * h + 1] -= f.y;
      w[h] = *reinterpret_cast<const uint32_t*>(&q);
    }
    *reinterpret_cast<uint2*>(at + s * stride) = make_uint2(w[0], w[1]);
  }
}

__device__ __forceinline__ void store_planes(__nv_bfloat16* at, long long stride, float v) {
#pragma unroll
  for (int s = 0; s < kPlanes; ++s) {
    const __nv_bfloat16 q = __float2bfloat16_rn(v);
    at[s * stride] = q;
    v -= __bfloat162float(q);
  }
}

}  // namespace
}  // namespace poetx
