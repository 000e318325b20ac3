// The epilogue that the fp32 products share.
#pragma once

#include "activation.cuh"
#include "linear.h"

namespace poetx {
namespace {

struct Fp32Epilogue {
  const float* bias;
  const float* residual;
  float* y;
  float* z;
  long long ld;  // between rows
  int N, act;
  bool vec_n;  // 16-byte rows
};

// Of the product's rows from m_first on.
Fp32Epilogue fp32_epilogue(const LinearProduct& g, long long m_first) {
  const long long ld = g.pitch_y > 0 ? g.pitch_y : g.N;
  auto at = [&](const void* base) {
    return static_cast<const float*>(base) + (base != nullptr ? m_first * ld : 0);
  };
  Fp32Epilogue e;
  e.ld = ld;
  e.bias = g.bias;
  e.residual = at(g.residual);
  e.y = const_cast<float*>(at(g.y));
  e.z = const_cast<float*>(at(g.z));
  e.N = g.N;
  e.act = g.act;
  e.vec_n = ld % 4 == 0;
  return e;
}

__device__ __forceinline__ void apply4(int act, float (&v)[4]) {
  auto each = [&](auto f) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = f(v[j]);
  };
  switch (act) {  // uniform over the grid
    case POETX_ACT_RELU: each([](float x) { return act_f<POETX_ACT_RELU, false>(x); }); break;
    case POETX_ACT_SILU: each([](float x) { return act_f<POETX_ACT_SILU, false>(x); }); break;
    case POETX_ACT_GELU: each([](float x) { return act_f<POETX_ACT_GELU, false>(x); }); break;
    case POETX_ACT_GELU_TANH:
      each([](float x) { return act_f<POETX_ACT_GELU_TANH, false>(x); });
      break;
    default: break;
  }
}

// Outputs (m, n .. n + 3), n < N a multiple of 4.
__device__ __forceinline__ void finish4(const Fp32Epilogue& p, long long m, int n, float4 acc) {
  float v[4] = {acc.x, acc.y, acc.z, acc.w};
  const long long at = m * p.ld + n;
  if (p.vec_n) {  // all four are inside the pitch (a bias only comes without one)
    if (p.bias != nullptr) {
      const float4 b = __ldg(reinterpret_cast<const float4*>(p.bias + n));
      v[0] += b.x, v[1] += b.y, v[2] += b.z, v[3] += b.w;
    }
    if (p.z != nullptr) *reinterpret_cast<float4*>(p.z + at) = make_float4(v[0], v[1], v[2], v[3]);
    apply4(p.act, v);
    if (p.residual != nullptr) {
      const float4 r = *reinterpret_cast<const float4*>(p.residual + at);
      v[0] += r.x, v[1] += r.y, v[2] += r.z, v[3] += r.w;
    }
    *reinterpret_cast<float4*>(p.y + at) = make_float4(v[0], v[1], v[2], v[3]);
    return;
  }
  const int live = min(4, p.N - n);
  if (p.bias != nullptr)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) v[j] += __ldg(p.bias + n + j);
  if (p.z != nullptr)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < live) p.z[at + j] = v[j];
  apply4(p.act, v);
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (j < live) p.y[at + j] = p.residual != nullptr ? v[j] + p.residual[at + j] : v[j];
}

}  // namespace
}  // namespace poetx
