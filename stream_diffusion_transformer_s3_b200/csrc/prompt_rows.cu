// Row kernels of the prompt operators (bandwidth-bound, fp32 or fp64 arithmetic):
//   rope_scaled  : cos / sin of one position per token, scaled frequencies
//   qk_norm_rope : per-head RMSNorm of q and k, then the rotation, one read and one write
#include <cuda_bf16.h>

#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace zdit {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kMaxPairs = 256;

struct RopeScaledParams {
  const int* pos;
  int64_t T;
  int pairs;
  double theta, factor, original_len, beta_fast, beta_slow;
  int kind;
  float magnitude;
  float* cs;
  float* sn;
};

__device__ double scaled_frequency(const RopeScaledParams& p, int i) {
  const double d = 2.0 * p.pairs;
  if (p.kind == ZDIT_ROPE_SCALE_NTK) {
    const double base = p.theta * pow(p.factor, d / (d - 2.0));
    return pow(base, -2.0 * i / d);
  }
  const double w = pow(p.theta, -2.0 * i / d);
  if (p.kind == ZDIT_ROPE_SCALE_LINEAR) return w / p.factor;
  if (p.kind == ZDIT_ROPE_SCALE_YARN) {
    const double turns = p.original_len * w * 0.15915494309189535;  // 1 / 2 pi
    const double g = fmin(fmax((turns - p.beta_slow) / (p.beta_fast - p.beta_slow), 0.0), 1.0);
    return w * (g + (1.0 - g) / p.factor);
  }
  return w;
}

// cos and sin of an angle given in double.  The angle is reduced by the nearest multiple
// n of pi/2 in double with pi/2 split in two parts (Cody and Waite): n < 2^31 * 2/pi * w_0,
// and the second part carries the product to ~2^-75 of n, so the remainder is good to
// |angle| 2^-53.  The remainder (|r| <= pi/4) is rounded to fp32, an error of at most
// 2^-25 absolute, below the half step 2^-25 of outputs in [1/2, 1]; then the fp32 sine and
// cosine.  A double sincos costs ~40 FP64 operations per element, this ~5.
__device__ __forceinline__ void sincos_of(double x, float& s, float& c) {
  const double n = rint(x * 0.63661977236758134);
  double r = fma(-n, 1.5707963267948966, x);
  r = fma(-n, 6.123233995736766e-17, r);
  float sr, cr;
  sincosf((float)r, &sr, &cr);
  const int q = (int)((long long)n & 3);
  s = (q & 1) ? cr : sr;
  c = (q & 1) ? sr : cr;
  if (q & 2) s = -s;
  if (q == 1 || q == 2) c = -c;
}

// A row of `pairs` values per token, VEC consecutive ones per thread, `tpr` threads per row
// (a power of two): 256 / tpr rows per CTA and step.  The frequencies are formed once per
// CTA, so the grid is a few CTAs per SM that stride over the rows.
template <int VEC>
__global__ void __launch_bounds__(kRopeThreads) rope_scaled_kernel(const RopeScaledParams p, int tpr) {
  __shared__ double omega[kMaxPairs];
  for (int i = threadIdx.x; i < p.pairs; i += kRopeThreads) omega[i] = scaled_frequency(p, i);
  griddep_wait();
  griddep_trigger();
  __syncthreads();
  const int lane = threadIdx.x & (tpr - 1);
  const int rows = kRopeThreads / tpr;
  for (int64_t t = (int64_t)blockIdx.x * rows + threadIdx.x / tpr; t < p.T; t += (int64_t)gridDim.x * rows) {
    const double pos = (double)p.pos[t];
    for (int i = lane * VEC; i < p.pairs; i += tpr * VEC) {
      float c[VEC], s[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        sincos_of(pos * omega[i + e], s[e], c[e]);
        c[e] *= p.magnitude;
        s[e] *= p.magnitude;
      }
      const int64_t at = t * p.pairs + i;
      if constexpr (VEC == 4) {
        *reinterpret_cast<float4*>(p.cs + at) = make_float4(c[0], c[1], c[2], c[3]);
        *reinterpret_cast<float4*>(p.sn + at) = make_float4(s[0], s[1], s[2], s[3]);
      } else {
        p.cs[at] = c[0];
        p.sn[at] = s[0];
      }
    }
  }
}

// ------------------------------------------------------------------------------ q / k norm + rotation
constexpr int kQkThreads = 256;

struct QkParams {
  int64_t units;  // T * (n_q + n_k)
  int n_q, n_k, head_dim, pairs;
  const void *q, *k;
  void *qo, *ko;
  int64_t q_rs, q_hs, k_rs, k_hs, qo_rs, qo_hs, ko_rs, ko_hs;
  const float *w_q, *w_k, *cos, *sin;
  float eps, inv_dim;
  int in_f32, out_f32;
};

__device__ __forceinline__ void load8(const void* base, int64_t at, bool f32, float (&v)[8]) {
  if (f32) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = s[0], b = s[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
}

__device__ __forceinline__ void store8(void* base, int64_t at, bool f32, const float (&v)[8]) {
  if (f32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// A group of G lanes (a power of two >= head_dim / 8) holds one head, 8 elements a lane,
// so each head is read and written once in 16-byte accesses and its sum of squares is a
// shuffle reduction.  HALF pairs (i, i + pairs): when pairs is a multiple of 8 the partner
// elements are one other lane's (shuffles); otherwise they go through shared memory (MODE
// 2).  Interleaved pairs are a lane's own (MODE 0).
enum { PAIR_OWN = 0, PAIR_SHUFFLE = 1, PAIR_SHARED = 2 };

template <int G, int MODE>
__global__ void __launch_bounds__(kQkThreads) qk_norm_rope_kernel(const QkParams p) {
  __shared__ float xs[MODE == PAIR_SHARED ? kQkThreads * 8 : 1];
  griddep_wait();
  griddep_trigger();
  const int lane = threadIdx.x & (G - 1);
  const int64_t unit = (int64_t)blockIdx.x * (kQkThreads / G) + threadIdx.x / G;
  const int heads = p.n_q + p.n_k;
  const bool live = unit < p.units && lane * 8 < p.head_dim;
  const int64_t t = unit / heads;
  int h = (int)(unit - t * heads);
  const bool is_q = h < p.n_q;
  if (!is_q) h -= p.n_q;
  const int e0 = lane * 8;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) {
    if (is_q)
      load8(p.q, t * p.q_rs + h * p.q_hs + e0, p.in_f32, v);
    else
      load8(p.k, t * p.k_rs + h * p.k_hs + e0, p.in_f32, v);
  }
  const float* w = is_q ? p.w_q : p.w_k;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if (w != nullptr && live) {
    const float r = 1.0f / sqrtf(fmaf(ss, p.inv_dim, p.eps));
    float wv[8];
    load8(w, e0, true, wv);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * wv[i];
  }
  if (p.pairs > 0) {
    const float* cs = p.cos + t * p.pairs;
    const float* sn = p.sin + t * p.pairs;
    if constexpr (MODE == PAIR_OWN) {
      const int i0 = e0 / 2;
      if (live && i0 < p.pairs) {
        float c[4], s[4];
        if ((p.pairs & 3) == 0) {
          const float4 c4 = *reinterpret_cast<const float4*>(cs + i0), s4 = *reinterpret_cast<const float4*>(sn + i0);
          c[0] = c4.x; c[1] = c4.y; c[2] = c4.z; c[3] = c4.w;
          s[0] = s4.x; s[1] = s4.y; s[2] = s4.z; s[3] = s4.w;
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool in = i0 + i < p.pairs;
            c[i] = in ? cs[i0 + i] : 1.f;
            s[i] = in ? sn[i0 + i] : 0.f;
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = v[2 * i], b = v[2 * i + 1];
          if (i0 + i < p.pairs) {
            v[2 * i] = a * c[i] - b * s[i];
            v[2 * i + 1] = a * s[i] + b * c[i];
          }
        }
      }
    } else if constexpr (MODE == PAIR_SHUFFLE) {
      const int step = p.pairs / 8;  // lanes between partners
      const bool lo = lane < step, hi = !lo && lane < 2 * step;
      const int src = lo ? lane + step : (hi ? lane - step : lane);
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, v[i], src, G);
      if (live && (lo || hi)) {
        const int i0 = lo ? e0 : e0 - p.pairs;
        float c[8], s[8];
        load8(cs, i0, true, c);
        load8(sn, i0, true, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lo ? v[i] * c[i] - o[i] * s[i] : o[i] * s[i] + v[i] * c[i];
      }
    } else {
      float* x = xs + (threadIdx.x / G) * (G * 8);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[e0 + i] = v[i];
      __syncwarp();
      if (live) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int e = e0 + i;
          if (e < p.pairs)
            v[i] = v[i] * cs[e] - x[e + p.pairs] * sn[e];
          else if (e < 2 * p.pairs)
            v[i] = x[e - p.pairs] * sn[e - p.pairs] + v[i] * cs[e - p.pairs];
        }
      }
    }
  }
  if (live) {
    if (is_q)
      store8(p.qo, t * p.qo_rs + h * p.qo_hs + e0, p.out_f32, v);
    else
      store8(p.ko, t * p.ko_rs + h * p.ko_hs + e0, p.out_f32, v);
  }
}

template <int G>
cudaError_t launch_qk_group(const QkParams& p, int mode, cudaStream_t s) {
  const int64_t per = kQkThreads / G;
  const dim3 grid((unsigned)((p.units + per - 1) / per));
  switch (mode) {
    case PAIR_OWN: return launch_dependent(qk_norm_rope_kernel<G, PAIR_OWN>, grid, dim3(kQkThreads), 0, s, p);
    case PAIR_SHUFFLE: return launch_dependent(qk_norm_rope_kernel<G, PAIR_SHUFFLE>, grid, dim3(kQkThreads), 0, s, p);
    default: return launch_dependent(qk_norm_rope_kernel<G, PAIR_SHARED>, grid, dim3(kQkThreads), 0, s, p);
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

// Heads of a buffer that is written must not overlap one another: either the rows contain
// the heads (token-major) or the heads contain the rows (head-major).
bool heads_disjoint(const zdit_heads& h, int64_t rows, int heads, int head_dim) {
  if (heads > 1 && h.head_stride < head_dim) return false;
  if (rows > 1 && h.row_stride < head_dim) return false;
  if (heads <= 1 || rows <= 1) return true;
  const int64_t lim = INT64_MAX / 4;
  if (h.row_stride > lim / rows || h.head_stride > lim / heads) return false;
  return h.row_stride >= (heads - 1) * h.head_stride + head_dim || h.head_stride >= (rows - 1) * h.row_stride + head_dim;
}

}  // namespace zdit

using namespace zdit;

extern "C" {

ZDIT_API zdit_status zdit_rope_table_scaled(const int32_t* pos, int64_t T, int32_t rotary_dim, float theta,
                                            const zdit_rope_scaling* scaling, float* cos_out, float* sin_out,
                                            void* stream) {
  zdit_rope_scaling sc = {ZDIT_ROPE_SCALE_NONE, 1.f, 1.f, 32.f, 1.f, 1.f};
  if (scaling != nullptr) sc = *scaling;
  if (!pos || !cos_out || !sin_out || T < 0 || !(theta >= 1.f) || !std::isfinite(theta)) return ZDIT_ERR_INVALID_ARG;
  if (sc.kind < ZDIT_ROPE_SCALE_NONE || sc.kind > ZDIT_ROPE_SCALE_YARN) return ZDIT_ERR_INVALID_ARG;
  if (!(sc.magnitude > 0.f) || !std::isfinite(sc.magnitude)) return ZDIT_ERR_INVALID_ARG;
  if (sc.kind != ZDIT_ROPE_SCALE_NONE && (!(sc.factor >= 1.f) || !std::isfinite(sc.factor)))
    return ZDIT_ERR_INVALID_ARG;
  if (sc.kind == ZDIT_ROPE_SCALE_YARN &&
      (!(sc.original_len > 0.f) || !std::isfinite(sc.original_len) || !(sc.beta_slow >= 0.f) ||
       !(sc.beta_fast > sc.beta_slow) || !std::isfinite(sc.beta_fast)))
    return ZDIT_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim % 2 || rotary_dim > 2 * kMaxPairs) return ZDIT_ERR_SHAPE;
  if (sc.kind == ZDIT_ROPE_SCALE_NTK && rotary_dim < 4) return ZDIT_ERR_SHAPE;
  if (T > INT64_MAX / (8 * kMaxPairs)) return ZDIT_ERR_SHAPE;
  if (!aligned16(cos_out) || !aligned16(sin_out) || (reinterpret_cast<uintptr_t>(pos) & 3)) return ZDIT_ERR_ALIGNMENT;
  if (T == 0) return ZDIT_OK;
  if (!device_ok()) return ZDIT_ERR_UNSUPPORTED;
  RopeScaledParams p;
  p.pos = pos; p.T = T; p.pairs = rotary_dim / 2; p.theta = theta; p.factor = sc.factor;
  p.original_len = sc.original_len; p.beta_fast = sc.beta_fast; p.beta_slow = sc.beta_slow; p.kind = sc.kind;
  p.magnitude = sc.magnitude; p.cs = cos_out; p.sn = sin_out;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int vec = p.pairs % 4 == 0 ? 4 : 1;
  int tpr = 1;
  while (tpr < kRopeThreads && tpr * vec < p.pairs) tpr *= 2;
  const int64_t rows = kRopeThreads / tpr;
  const int64_t want = (T + rows - 1) / rows, most = (int64_t)num_sms() * 8;
  const dim3 grid((unsigned)(want < most ? want : most));
  ProfScope ps(PROF_ROPE, 0.0, 8.0 * T * p.pairs + 4.0 * T, s);
  const cudaError_t e = vec == 4 ? launch_dependent(rope_scaled_kernel<4>, grid, dim3(kRopeThreads), 0, s, p, tpr)
                                 : launch_dependent(rope_scaled_kernel<1>, grid, dim3(kRopeThreads), 0, s, p, tpr);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ZDIT_OK : ZDIT_ERR_CUDA;
}

ZDIT_API zdit_status zdit_qk_norm_rope(const zdit_qk_norm_rope_args* a, void* stream) {
  if (a == nullptr || a->T < 0 || a->n_q <= 0 || a->n_k < 0) return ZDIT_ERR_INVALID_ARG;
  if (!a->q.ptr || !a->q_out.ptr || (a->n_k > 0 && (!a->k.ptr || !a->k_out.ptr))) return ZDIT_ERR_INVALID_ARG;
  if (a->in_dtype < 0 || a->in_dtype > 1 || a->out_dtype < 0 || a->out_dtype > 1) return ZDIT_ERR_INVALID_ARG;
  if (a->layout != ZDIT_ROPE_INTERLEAVED && a->layout != ZDIT_ROPE_HALF) return ZDIT_ERR_INVALID_ARG;
  if ((a->w_q || a->w_k) && (!(a->eps >= 0.f) || !std::isfinite(a->eps))) return ZDIT_ERR_INVALID_ARG;
  if (a->head_dim < 8 || a->head_dim % 8 || a->head_dim > 256) return ZDIT_ERR_SHAPE;
  if (a->rotary_dim < 0 || a->rotary_dim % 2 || a->rotary_dim > a->head_dim) return ZDIT_ERR_SHAPE;
  if (a->rotary_dim > 0 && (!a->cos || !a->sin)) return ZDIT_ERR_INVALID_ARG;
  const int64_t heads = (int64_t)a->n_q + a->n_k;
  if (heads > (1 << 20) || a->T > (int64_t(1) << 33) / heads) return ZDIT_ERR_SHAPE;
  const zdit_heads* hs[4] = {&a->q, &a->q_out, &a->k, &a->k_out};
  for (int i = 0; i < 4; ++i) {
    const int n = i < 2 ? a->n_q : a->n_k;
    if (n == 0) continue;
    const int64_t unit = (i & 1 ? a->out_dtype : a->in_dtype) == ZDIT_T_F32 ? 4 : 8;
    if (hs[i]->row_stride < 0 || hs[i]->head_stride < 0) return ZDIT_ERR_SHAPE;
    if (!aligned16(hs[i]->ptr) || (a->T > 1 && hs[i]->row_stride % unit) || (n > 1 && hs[i]->head_stride % unit))
      return ZDIT_ERR_ALIGNMENT;
    if ((i & 1) && !heads_disjoint(*hs[i], a->T, n, a->head_dim)) return ZDIT_ERR_SHAPE;
  }
  if (!aligned16(a->w_q) || !aligned16(a->w_k) || !aligned16(a->cos) || !aligned16(a->sin)) return ZDIT_ERR_ALIGNMENT;
  if (a->T == 0) return ZDIT_OK;
  if (!device_ok()) return ZDIT_ERR_UNSUPPORTED;
  QkParams p;
  p.units = a->T * heads; p.n_q = a->n_q; p.n_k = a->n_k; p.head_dim = a->head_dim; p.pairs = a->rotary_dim / 2;
  p.q = a->q.ptr; p.k = a->k.ptr; p.qo = a->q_out.ptr; p.ko = a->k_out.ptr;
  p.q_rs = a->q.row_stride; p.q_hs = a->q.head_stride; p.k_rs = a->k.row_stride; p.k_hs = a->k.head_stride;
  p.qo_rs = a->q_out.row_stride; p.qo_hs = a->q_out.head_stride;
  p.ko_rs = a->k_out.row_stride; p.ko_hs = a->k_out.head_stride;
  p.w_q = a->w_q; p.w_k = a->w_k; p.cos = a->cos; p.sin = a->sin; p.eps = a->eps; p.inv_dim = 1.0f / a->head_dim;
  p.in_f32 = a->in_dtype == ZDIT_T_F32; p.out_f32 = a->out_dtype == ZDIT_T_F32;
  const int mode = a->layout == ZDIT_ROPE_INTERLEAVED ? PAIR_OWN : (p.pairs % 8 == 0 ? PAIR_SHUFFLE : PAIR_SHARED);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double elems = (double)p.units * p.head_dim;
  ProfScope ps(PROF_NORM_MOD, 7.0 * elems,
               elems * ((p.in_f32 ? 4 : 2) + (p.out_f32 ? 4 : 2)) + 8.0 * a->T * p.pairs, s);
  cudaError_t e;
  if (a->head_dim <= 64) e = launch_qk_group<8>(p, mode, s);
  else if (a->head_dim <= 128) e = launch_qk_group<16>(p, mode, s);
  else e = launch_qk_group<32>(p, mode, s);
  return e == cudaSuccess && cudaGetLastError() == cudaSuccess ? ZDIT_OK : ZDIT_ERR_CUDA;
}

}  // extern "C"
