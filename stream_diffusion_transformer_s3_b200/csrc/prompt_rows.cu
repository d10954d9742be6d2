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
  double log2_base;  // w_i = 2^(-2i/d log2_base) before LINEAR / YARN scaling
  double factor, original_len, beta_fast, beta_slow;
  int kind;
  float magnitude;
  float* cs;
  float* sn;
};

// (exp2 of a product instead of a power: its relative error grows with the exponent, but
// pos * w carries it times w log2(1/w) <= 0.54, so the angle is as good: |pos| 2^-53.)
__device__ double scaled_frequency(const RopeScaledParams& p, int i) {
  const double w = exp2(-(double)i / p.pairs * p.log2_base);
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
// 2^-25 absolute, below the half step 2^-25 of outputs in [1/2, 1]; then the Taylor series
// of sine and cosine to r^9 and r^10 (first terms left out: r^11/11! < 1.8e-9 and r^12/12!
// < 1.2e-10).  About 30 instructions an element; a double sincos takes ~40 FP64 operations.
__device__ __forceinline__ void sincos_of(double x, float& s, float& c) {
  const double n = rint(x * 0.63661977236758134);
  double rd = fma(-n, 1.5707963267948966, x);
  rd = fma(-n, 6.123233995736766e-17, rd);
  const float r = (float)rd, q = r * r;
  float ps = fmaf(q, 1.0f / 362880.0f, -1.0f / 5040.0f);
  ps = fmaf(q, ps, 1.0f / 120.0f);
  ps = fmaf(q, ps, -1.0f / 6.0f);
  const float sr = fmaf(r * q, ps, r);
  float pc = fmaf(q, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  pc = fmaf(q, pc, -1.0f / 720.0f);
  pc = fmaf(q, pc, 1.0f / 24.0f);
  pc = fmaf(q, pc, -0.5f);
  const float cr = fmaf(q, pc, 1.0f);
  const int k = (int)((long long)n & 3);  // quadrant
  s = (k & 1) ? cr : sr;
  c = (k & 1) ? sr : cr;
  if (k & 2) s = -s;
  if ((k + 1) & 2) c = -c;
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
  int64_t T;
  int tokens;  // tokens per CTA
  int n_q, n_k, head_dim, pairs;
  const void *q, *k;
  void *qo, *ko;
  int64_t q_rs, q_hs, k_rs, k_hs, qo_rs, qo_hs, ko_rs, ko_hs;
  const float *w_q, *w_k, *cos, *sin;
  float eps, inv_dim;
  int in_f32, out_f32;
};

// v = v * r * w for the 8 values of a chunk.
__device__ __forceinline__ void scale8(float (&v)[8], float r, const float4* w, int chunks) {
  const float4 w0 = w[0], w1 = w[chunks];
  v[0] = v[0] * r * w0.x; v[1] = v[1] * r * w0.y; v[2] = v[2] * r * w0.z; v[3] = v[3] * r * w0.w;
  v[4] = v[4] * r * w1.x; v[5] = v[5] * r * w1.y; v[6] = v[6] * r * w1.z; v[7] = v[7] * r * w1.w;
}

template <bool F32>
__device__ __forceinline__ void store8(char* at, const float (&v)[8]) {
  if constexpr (F32) {
    float4* d = reinterpret_cast<float4*>(at);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// A group of G lanes takes one head of `tokens` consecutive tokens.  Lane l holds two chunks
// of 8 elements, at 8 l and at 8 (C + l), C = ceil(head_dim / 16) <= G: each head is read and
// written once in 16-byte accesses, its sum of squares is a shuffle reduction, and the pairs
// (i, i + head_dim / 2) of a wholly rotated head are a lane's own.  Neighbouring groups take
// neighbouring heads, so a CTA reads whole stretches of a row.
// The kernel is bound by instructions before it is bound by memory.  16381 x 40 heads of
// 128, bf16, a quarter rotated: 87 us with 8 elements a lane and the head and token of every
// 16 bytes found by division, 80 us with each group staying on its head (addresses advancing
// by a row), 69 us with 16 elements a lane, 67 us with the norm weights in shared memory and
// the registers of four CTAs per SM (two tokens in flight per lane: 73 us, four: 103 us, their
// registers cost more threads), 63 us (5.3 TB/s) with types and pairing as template arguments
// and the weights laid out so that no two lanes of a read share a bank.
enum {
  PAIR_OWN = 0,     // interleaved: pairs inside a chunk, tables in multiples of 4 pairs
  PAIR_LOCAL = 1,   // halves of the whole head: element i of both chunks
  PAIR_SHUFFLE = 2, // halves inside the first chunks: another lane's elements
  PAIR_SHARED = 3,  // any other split: through shared memory
  PAIR_ODD = 4      // interleaved, any number of pairs
};
// The rotation tables of one lane and token: N pairs from i0; ODD: one by one, the identity
// past the last.
template <int N, bool ODD>
__device__ __forceinline__ void load_pairs(const float* cs, const float* sn, int i0, int pairs, float (&c)[N],
                                           float (&s)[N]) {
  if constexpr (!ODD) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 c4 = *reinterpret_cast<const float4*>(cs + i0 + i), s4 = *reinterpret_cast<const float4*>(sn + i0 + i);
      c[i] = c4.x; c[i + 1] = c4.y; c[i + 2] = c4.z; c[i + 3] = c4.w;
      s[i] = s4.x; s[i + 1] = s4.y; s[i + 2] = s4.z; s[i + 3] = s4.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = i0 + i < pairs;
      c[i] = in ? cs[i0 + i] : 1.f;
      s[i] = in ? sn[i0 + i] : 0.f;
    }
  }
}

template <bool ODD>
__device__ __forceinline__ void rotate_own(float (&v)[8], const float (&c)[4], const float (&s)[4], int i0, int pairs) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float x = v[2 * i], y = v[2 * i + 1];
    if (!ODD || i0 + i < pairs) {
      v[2 * i] = x * c[i] - y * s[i];
      v[2 * i + 1] = x * s[i] + y * c[i];
    }
  }
}

template <bool F32>
struct RawChunk {
  uint4 u[F32 ? 2 : 1];
  __device__ __forceinline__ void load(const char* p, bool live) {
    u[0] = make_uint4(0, 0, 0, 0);
    if constexpr (F32) u[1] = make_uint4(0, 0, 0, 0);
    if (live) {
      u[0] = reinterpret_cast<const uint4*>(p)[0];
      if constexpr (F32) u[1] = reinterpret_cast<const uint4*>(p)[1];
    }
  }
  __device__ __forceinline__ void unpack(float (&v)[8]) const {
    const uint32_t a[4] = {u[0].x, u[0].y, u[0].z, u[0].w};
    if constexpr (F32) {
      const uint32_t b[4] = {u[1].x, u[1].y, u[1].z, u[1].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = __uint_as_float(a[i]);
        v[4 + i] = __uint_as_float(b[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
      }
    }
  }
};

template <int G, int MODE, bool F32, bool OUT_F32>
__global__ void __launch_bounds__(kQkThreads, 4) qk_norm_rope_kernel(const QkParams p) {
  __shared__ float xs[MODE == PAIR_SHARED ? kQkThreads * 16 : 1];
  // norm weights: the first halves of all chunks of 8, then the second halves, so that
  // neighbouring lanes read neighbouring 16 bytes
  __shared__ float4 ws[2][64];
  constexpr int ES = F32 ? 4 : 2, OES = OUT_F32 ? 4 : 2;
  constexpr bool OWN = MODE == PAIR_OWN || MODE == PAIR_ODD;
  const int lane = threadIdx.x & (G - 1);
  const int chunks = (p.head_dim + 15) / 16;  // C
  const int ea = lane * 8, eb = (chunks + lane) * 8;
  const int heads = p.n_q + p.n_k;
  const int64_t group = (int64_t)blockIdx.x * (kQkThreads / G) + threadIdx.x / G;
  const int64_t block = group / heads;  // of `tokens` tokens
  int h = (int)(group - block * heads);
  const int64_t t0 = block * p.tokens;
  const int n = t0 < p.T && lane < chunks ? (int)(p.T - t0 < p.tokens ? p.T - t0 : p.tokens) : 0;
  const bool has_b = eb < p.head_dim;
  const bool is_q = h < p.n_q;
  if (!is_q) h -= p.n_q;
  const int64_t rs = is_q ? p.q_rs : p.k_rs, ors = is_q ? p.qo_rs : p.ko_rs;
  const char* src = static_cast<const char*>(is_q ? p.q : p.k) + ((is_q ? h * p.q_hs : h * p.k_hs) + t0 * rs + ea) * ES;
  char* dst = static_cast<char*>(is_q ? p.qo : p.ko) + ((is_q ? h * p.qo_hs : h * p.ko_hs) + t0 * ors + ea) * OES;
  const int64_t src_step = rs * ES, dst_step = ors * OES;
  const int src_b = chunks * 8 * ES, dst_b = chunks * 8 * OES;  // to the second chunk
  const float* w = is_q ? p.w_q : p.w_k;
  const bool norms = p.w_q != nullptr || p.w_k != nullptr;
  const int step = p.pairs / 8;  // PAIR_SHUFFLE: lanes between partners
  const bool lo = lane < step, hi = !lo && lane < 2 * step;
  const int partner = lo ? lane + step : (hi ? lane - step : lane);
  const int i0 = OWN ? ea / 2 : MODE == PAIR_SHUFFLE && hi ? ea - p.pairs : ea;  // first pair of chunk a
  const bool rotates = OWN ? i0 < p.pairs : MODE == PAIR_LOCAL ? true : (lo || hi);
  const bool rotates_b = OWN && has_b && eb / 2 < p.pairs;
  const float* cs = p.cos + t0 * p.pairs;
  const float* sn = p.sin + t0 * p.pairs;
  griddep_wait();
  griddep_trigger();
  for (int i = threadIdx.x; i < 2 * p.head_dim; i += kQkThreads) {
    const int k = i >= p.head_dim;
    const float* src_w = k ? p.w_k : p.w_q;
    const int e = i - k * p.head_dim;
    if (src_w != nullptr) reinterpret_cast<float*>(&ws[k][(e >> 2 & 1) * (p.head_dim / 8) + e / 8])[e & 3] = src_w[e];
  }
  __syncthreads();
  const float4* wsm = ws[is_q ? 0 : 1];

  // (the same number of steps for every group: shuffles and __syncwarp need whole warps)
  constexpr int TAB = OWN ? 4 : MODE == PAIR_SHARED ? 1 : 8;
  constexpr int TAB_B = OWN ? 4 : 1;
  RawChunk<F32> ra, rb;
  float c[TAB], s[TAB], cb[TAB_B], sb[TAB_B];
  auto request = [&](bool live) {  // the head and table rows that src, cs and sn point at
    ra.load(src, live);
    rb.load(src + src_b, live && has_b);
    if constexpr (MODE != PAIR_SHARED) {
      if (live && rotates) load_pairs<TAB, MODE == PAIR_ODD>(cs, sn, i0, p.pairs, c, s);
      if constexpr (OWN)
        if (live && rotates_b) load_pairs<4, MODE == PAIR_ODD>(cs, sn, eb / 2, p.pairs, cb, sb);
    }
  };
  for (int k = 0; k < p.tokens; ++k) {
    const bool live = k < n;
    request(live);
    float a[8], b[8];
    ra.unpack(a);
    rb.unpack(b);
    const float *cs_now = cs, *sn_now = sn;
    src += src_step;
    cs += p.pairs;
    sn += p.pairs;
    if (norms) {
      float ss = 0.f, sq = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(a[i], a[i], ss);
        sq = fmaf(b[i], b[i], sq);
      }
      ss += sq;
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (w != nullptr) {
        const float r = rsqrtf(fmaf(ss, p.inv_dim, p.eps));
        scale8(a, r, wsm + (n > 0 ? lane : 0), p.head_dim / 8);
        scale8(b, r, wsm + (has_b ? chunks + lane : 0), p.head_dim / 8);
      }
    }
    if constexpr (OWN) {
      if (rotates) rotate_own<MODE == PAIR_ODD>(a, c, s, i0, p.pairs);
      if (rotates_b) rotate_own<MODE == PAIR_ODD>(b, cb, sb, eb / 2, p.pairs);
    } else if constexpr (MODE == PAIR_LOCAL) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x = a[i], y = b[i];
        a[i] = x * c[i] - y * s[i];
        b[i] = x * s[i] + y * c[i];
      }
    } else if constexpr (MODE == PAIR_SHUFFLE) {
      if (p.pairs > 0) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(0xffffffffu, a[i], partner, G);
        if (rotates) {
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] = fmaf(a[i], c[i], lo ? -o[i] * s[i] : o[i] * s[i]);
        }
      }
    } else {
      float* x = xs + (threadIdx.x / G) * (G * 16);
      __syncwarp();  // the previous token's readers are done
      // (only lanes that hold elements: lane l >= C would write where lane l - C's second chunk is)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (lane < chunks) x[ea + i] = a[i];
        if (has_b) x[eb + i] = b[i];
      }
      __syncwarp();
      if (live) {
        auto turn = [&](float v, int e) {
          if (e < p.pairs) return v * cs_now[e] - x[e + p.pairs] * sn_now[e];
          if (e < 2 * p.pairs) return x[e - p.pairs] * sn_now[e - p.pairs] + v * cs_now[e - p.pairs];
          return v;
        };
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          a[i] = turn(a[i], ea + i);
          b[i] = turn(b[i], eb + i);
        }
      }
    }
    if (live) {
      store8<OUT_F32>(dst, a);
      if (has_b) store8<OUT_F32>(dst + dst_b, b);
    }
    dst += dst_step;
  }
}

template <int G, int MODE>
cudaError_t launch_qk_mode(const QkParams& p, cudaStream_t s) {
  const int64_t groups = (p.T + p.tokens - 1) / p.tokens * (p.n_q + p.n_k), per = kQkThreads / G;
  const dim3 grid((unsigned)((groups + per - 1) / per)), block(kQkThreads);
  if (p.in_f32)
    return p.out_f32 ? launch_dependent(qk_norm_rope_kernel<G, MODE, true, true>, grid, block, 0, s, p)
                     : launch_dependent(qk_norm_rope_kernel<G, MODE, true, false>, grid, block, 0, s, p);
  return p.out_f32 ? launch_dependent(qk_norm_rope_kernel<G, MODE, false, true>, grid, block, 0, s, p)
                   : launch_dependent(qk_norm_rope_kernel<G, MODE, false, false>, grid, block, 0, s, p);
}

template <int G>
cudaError_t launch_qk_group(const QkParams& p, int mode, cudaStream_t s) {
  switch (mode) {
    case PAIR_OWN: return launch_qk_mode<G, PAIR_OWN>(p, s);
    case PAIR_LOCAL: return launch_qk_mode<G, PAIR_LOCAL>(p, s);
    case PAIR_SHUFFLE: return launch_qk_mode<G, PAIR_SHUFFLE>(p, s);
    case PAIR_ODD: return launch_qk_mode<G, PAIR_ODD>(p, s);
    default: return launch_qk_mode<G, PAIR_SHARED>(p, s);
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
  if (cos_out == sin_out) return ZDIT_ERR_INVALID_ARG;
  if (!device_ok()) return ZDIT_ERR_UNSUPPORTED;
  RopeScaledParams p;
  p.pos = pos; p.T = T; p.pairs = rotary_dim / 2; p.factor = sc.factor;
  p.log2_base = std::log2((double)theta);
  if (sc.kind == ZDIT_ROPE_SCALE_NTK)
    p.log2_base += (double)rotary_dim / (rotary_dim - 2.0) * std::log2((double)sc.factor);
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
  return launch_status(e);
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
  // one buffer for input and output: in place only where every element keeps its address
  for (int i = 0; i < 4; i += 2) {
    const int n = i == 0 ? a->n_q : a->n_k;
    if (n > 0 && hs[i]->ptr == hs[i + 1]->ptr &&
        (a->in_dtype != a->out_dtype || (a->T > 1 && hs[i]->row_stride != hs[i + 1]->row_stride) ||
         (n > 1 && hs[i]->head_stride != hs[i + 1]->head_stride)))
      return ZDIT_ERR_INVALID_ARG;
  }
  if (a->n_k > 0 && (a->q_out.ptr == a->k_out.ptr || a->q_out.ptr == a->k.ptr || a->k_out.ptr == a->q.ptr))
    return ZDIT_ERR_INVALID_ARG;
  if (!aligned16(a->w_q) || !aligned16(a->w_k) || !aligned16(a->cos) || !aligned16(a->sin)) return ZDIT_ERR_ALIGNMENT;
  if (a->T == 0) return ZDIT_OK;
  if (!device_ok()) return ZDIT_ERR_UNSUPPORTED;
  QkParams p;
  p.T = a->T;
  // tokens per group: 1 while that gives no more than about two waves of CTAs, up to 8
  const int64_t lanes = a->T * heads * (a->head_dim <= 64 ? 4 : a->head_dim <= 128 ? 8 : 16);
  const int64_t fill = lanes / ((int64_t)num_sms() * 2048 * 2);
  p.tokens = (int)(fill < 1 ? 1 : fill > 8 ? 8 : fill);
  p.n_q = a->n_q; p.n_k = a->n_k; p.head_dim = a->head_dim; p.pairs = a->rotary_dim / 2;
  p.q = a->q.ptr; p.k = a->k.ptr; p.qo = a->q_out.ptr; p.ko = a->k_out.ptr;
  p.q_rs = a->q.row_stride; p.q_hs = a->q.head_stride; p.k_rs = a->k.row_stride; p.k_hs = a->k.head_stride;
  p.qo_rs = a->q_out.row_stride; p.qo_hs = a->q_out.head_stride;
  p.ko_rs = a->k_out.row_stride; p.ko_hs = a->k_out.head_stride;
  p.w_q = a->w_q; p.w_k = a->w_k; p.cos = a->cos; p.sin = a->sin; p.eps = a->eps; p.inv_dim = 1.0f / a->head_dim;
  p.in_f32 = a->in_dtype == ZDIT_T_F32; p.out_f32 = a->out_dtype == ZDIT_T_F32;
  const int half = (a->head_dim + 15) / 16 * 8;  // first element of the second chunks
  const int mode = a->layout == ZDIT_ROPE_INTERLEAVED          ? (p.pairs % 4 == 0 ? PAIR_OWN : PAIR_ODD)
                   : p.pairs == half && a->rotary_dim == a->head_dim ? PAIR_LOCAL
                   : p.pairs % 8 == 0 && a->rotary_dim <= half ? PAIR_SHUFFLE
                                                               : PAIR_SHARED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const double elems = (double)a->T * heads * p.head_dim;
  ProfScope ps(PROF_NORM_MOD, 7.0 * elems,
               elems * ((p.in_f32 ? 4 : 2) + (p.out_f32 ? 4 : 2)) + 8.0 * a->T * p.pairs, s);
  cudaError_t e;
  if (a->head_dim <= 64) e = launch_qk_group<4>(p, mode, s);
  else if (a->head_dim <= 128) e = launch_qk_group<8>(p, mode, s);
  else e = launch_qk_group<16>(p, mode, s);
  return launch_status(e);
}

}  // extern "C"
