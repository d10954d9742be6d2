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
__device__ __forceinline__ float linear_act(float y, int act) {
  if (act == ZDIT_ACT_SILU) return y / (1.0f + __expf(-y));
  if (act == ZDIT_ACT_GELU_TANH) {
    const float u2 = 1.5957691216057308f * fmaf(0.044715f * y * y, y, y);
    return y / (1.0f + __expf(-u2));
  }
  if (act == ZDIT_ACT_GELU) return 0.5f * y * erfcf(-0.7071067811865476f * y);
  return y;
}

__device__ __forceinline__ float linear_load(const void* p, int64_t at, int f32) {
  return f32 ? static_cast<const float*>(p)[at] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}
__device__ __forceinline__ void linear_store(void* p, int64_t at, int f32, float v) {
  if (f32)
    static_cast<float*>(p)[at] = v;
  else
    static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

// W consecutive columns of one row, starting at col0 (a multiple of W): 16-byte accesses
// when all W are inside N and the rows are aligned (e.vec), else one by one.
template <int W>
__device__ __forceinline__ void linear_finish_row(const LinearEpi& e, int row, int col0, int N, float (&v)[W]) {
  if (e.vec && col0 + W <= N) {
    if (e.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] += __ldg(e.bias + col0 + j);
    }
    if (e.act != ZDIT_ACT_NONE) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = linear_act(v[j], e.act);
    }
    if (e.residual != nullptr) {
      const int64_t at = (int64_t)row * e.ld_res + col0;
      if (e.res_f32) {
        const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(e.residual) + at);
#pragma unroll
        for (int j = 0; j < W / 4; ++j) {
          const float4 r = s[j];
          v[4 * j] += r.x; v[4 * j + 1] += r.y; v[4 * j + 2] += r.z; v[4 * j + 3] += r.w;
        }
      } else {
        const uint4* s = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.residual) + at);
#pragma unroll
        for (int j = 0; j < W / 8; ++j) {
          const uint4 u = s[j];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[8 * j + 2 * i] += __uint_as_float(w[i] << 16);
            v[8 * j + 2 * i + 1] += __uint_as_float(w[i] & 0xffff0000u);
          }
        }
      }
    }
    const int64_t at = (int64_t)row * e.ld_out + col0;
    if (e.out_f32) {
      float4* d = reinterpret_cast<float4*>(static_cast<float*>(e.out) + at);
#pragma unroll
      for (int j = 0; j < W / 4; ++j) d[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    } else {
      uint4* d = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(e.out) + at);
#pragma unroll
      for (int j = 0; j < W / 8; ++j)
        d[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                          pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < W; ++j) {
    const int col = col0 + j;
    if (col < N) {
      float y = v[j];
      if (e.bias != nullptr) y += __ldg(e.bias + col);
      y = linear_act(y, e.act);
      if (e.residual != nullptr) y += linear_load(e.residual, (int64_t)row * e.ld_res + col, e.res_f32);
      linear_store(e.out, (int64_t)row * e.ld_out + col, e.out_f32, y);
    }
  }
}

}  // namespace zdit
