// Epilogue of zdit_linear: out = residual + act(acc + bias), fp32 until the one rounding of
// the store.
#pragma once
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace zdit {

// SiLU y / (1 + e^-y).  GELU y Phi(y) = y erfc(-y / sqrt 2) / 2 (erfc keeps the tail of
// large negative y, where 1 + erf cancels).  Its tanh form with u = sqrt(2 / pi)
// (y + 0.044715 y^3): y (1 + tanh u) / 2 = y / (1 + e^-2u), which does not cancel either.
// __fdividef is within 2 ulp for divisors up to 2^126 and 0 beyond, the limit here.
template <int ACT>
__device__ __forceinline__ float linear_act(float y) {
  if constexpr (ACT == ZDIT_ACT_SILU) return __fdividef(y, 1.0f + __expf(-y));
  if constexpr (ACT == ZDIT_ACT_GELU_TANH) {
    const float u2 = 1.5957691216057308f * fmaf(0.044715f * y * y, y, y);
    return __fdividef(y, 1.0f + __expf(-u2));
  }
  if constexpr (ACT == ZDIT_ACT_GELU) return 0.5f * y * erfcf(-0.7071067811865476f * y);
  return y;
}

// The activation is chosen once per W values: a choice per value would put W copies of
// every function into the unrolled epilogue, which then misses the instruction cache
// (measured: 47 instead of 12 us for a 1000 x 1000 x 1000 product).
template <int W>
__device__ __forceinline__ void linear_act_all(float (&v)[W], int act) {
  if (act == ZDIT_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = linear_act<ZDIT_ACT_SILU>(v[j]);
  } else if (act == ZDIT_ACT_GELU_TANH) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = linear_act<ZDIT_ACT_GELU_TANH>(v[j]);
  } else if (act == ZDIT_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = linear_act<ZDIT_ACT_GELU>(v[j]);
  }
}

__device__ __forceinline__ void add_bf16x2(uint32_t u, float& a, float& b) {
  a += __uint_as_float(u << 16);
  b += __uint_as_float(u & 0xffff0000u);
}

// Stores W (a multiple of 4) consecutive columns of one row, starting at col0: accesses of up
// to 16 bytes when all W are inside N and the rows are aligned (e.vec), else one by one.
template <int W>
__device__ __forceinline__ void linear_store(const LinearEpi& e, int row, int col0, int N, const float (&v)[W]) {
  const int64_t at = (int64_t)row * e.ld_out + col0;
  if (e.vec && col0 + W <= N) {
    if (e.out_f32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(e.out) + at);
#pragma unroll
      for (int j = 0; j < W / 4; ++j) d[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else if constexpr (W % 8 == 0) {
      uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(e.out) + at);
#pragma unroll
      for (int j = 0; j < W / 8; ++j)
        d[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                          pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    } else {
      uint2* d = reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(e.out) + at);
#pragma unroll
      for (int j = 0; j < W / 4; ++j)
        d[j] = make_uint2(pack_bf16x2(v[4 * j], v[4 * j + 1]), pack_bf16x2(v[4 * j + 2], v[4 * j + 3]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < W; ++j)
    if (col0 + j < N) {
      if (e.out_f32)
        static_cast<float*>(e.out)[at + j] = v[j];
      else
        static_cast<__nv_bfloat16*>(e.out)[at + j] = __float2bfloat16_rn(v[j]);
    }
}

// Four columns of the residual (zeros past N).
__device__ __forceinline__ void linear_residual4(const LinearEpi& e, int row, int col0, int N, float (&r)[4]) {
  const int64_t at = (int64_t)row * e.ld_res + col0;
  if (e.vec && col0 + 4 <= N) {
    if (e.res_f32) {
      const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + at);
      r[0] = f.x; r[1] = f.y; r[2] = f.z; r[3] = f.w;
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(e.residual) + at);
      r[0] = __uint_as_float(u.x << 16);
      r[1] = __uint_as_float(u.x & 0xffff0000u);
      r[2] = __uint_as_float(u.y << 16);
      r[3] = __uint_as_float(u.y & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    r[j] = 0.f;
    if (col0 + j < N)
      r[j] = e.res_f32 ? static_cast<const float*>(e.residual)[at + j]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[at + j]);
  }
}

// The whole epilogue of W (a multiple of 8) consecutive columns of one row, starting at col0;
// accesses as in linear_store.
template <int W>
__device__ __forceinline__ void linear_finish(const LinearEpi& e, int row, int col0, int N, float (&v)[W]) {
  const bool vec = e.vec && col0 + W <= N;
  if (e.bias != nullptr) {
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (vec || col0 + j < N) v[j] += __ldg(e.bias + col0 + j);
  }
  linear_act_all<W>(v, e.act);
  if (vec) {
    if (e.residual != nullptr) {
      const int64_t ra = (int64_t)row * e.ld_res + col0;
      if (e.res_f32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + ra);
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
          const float4 r = s[j];
          v[4 * j] += r.x; v[4 * j + 1] += r.y; v[4 * j + 2] += r.z; v[4 * j + 3] += r.w;
        }
      } else {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.residual) + ra);
#pragma unroll
        for (int j = 0; j < W / 8; ++j) {
          const uint4 u = s[j];
          add_bf16x2(u.x, v[8 * j], v[8 * j + 1]);
          add_bf16x2(u.y, v[8 * j + 2], v[8 * j + 3]);
          add_bf16x2(u.z, v[8 * j + 4], v[8 * j + 5]);
          add_bf16x2(u.w, v[8 * j + 6], v[8 * j + 7]);
        }
      }
    }
    linear_store<W>(e, row, col0, N, v);
    return;
  }
  if (e.residual != nullptr) {
    const int64_t ra = (int64_t)row * e.ld_res + col0;
#pragma unroll
    for (int j = 0; j < W; ++j)
      if (col0 + j < N)
        v[j] += e.res_f32 ? static_cast<const float*>(e.residual)[ra + j]
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[ra + j]);
  }
  linear_store<W>(e, row, col0, N, v);
}

}  // namespace zdit
