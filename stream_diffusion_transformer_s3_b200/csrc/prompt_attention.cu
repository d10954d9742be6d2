// Causal attention with grouped heads over packed prompts, for sm_100a (head dim 64 or 128).
//
//   O_i = sum_j p_ij V_j,  p_i = softmax_j(scale q_i . k_j),  j <= i + kv_len - q_len
//
// The `group` query heads that share a key head are packed into one 128-row tile: a tile
// holds 128 / group consecutive tokens, row r = (token r / group, head r % group), which a
// 3-D TMA box (64 columns x group heads x tokens) delivers as consecutive rows.  So K and V
// are read once per key head, a single token fills `group` rows instead of one, and the mask
// is a limit on the key index that depends on the row's token alone.
//
// One CTA takes one query tile (sequence, 128 rows, key head, part of the keys), two CTAs per
// SM, so that one CTA's set-up, loads and output overlap the other's work; 64-key tiles with S
// double-buffered in TMEM, so that S of the next tile is ready when the softmax finishes the
// last one.  7 warps: 0-3 softmax, one thread per row; 4 loads Q and K; 5 issues the MMAs; 6
// loads V (its own warp: a V stage still in use never delays the next K).
// TMEM columns: S buffers [0, 64) and [64, 128), O [128, +HD).  P (bf16 pairs) is written over
// the first columns of its S and feeds the PV product from there.  Softmax in fp32: a running
// maximum that moves only when a row grows by more than 16 (log2 units; P <= 2^16 keeps bf16's
// relative precision), and the sum of the unrounded P.  P is rounded to bf16 because both operands
// of a product have V's type (splitting it into two bf16 halves would double that product): the
// outputs are then 1.8e-3 to 2.3e-3 off in the norm, against 1.5e-3 to 1.7e-3 for an fp32 P, where
// only the stored result is rounded.
// Per 128 x 64 unit the tensor core works 8 x 48 + 4 x 64 = 640 clocks (S reads both operands
// from shared memory, 48 clocks a step instead of 32), the exponentials take 512, and shared
// memory moves 32 KB of K and V in and 64 KB of operands out, 768.  A unit of a long prompt
// takes about 1120 clocks (16384 tokens, 32 heads on 8: tensor pipe 57% active, 2.0 to 2.1 ms,
// 1.05 to 1.1 PFLOP/s; under the power cap 2.15 to 2.2 ms), so no unit is saturated: the rest
// is the hand-over between softmax and MMA of the two CTAs.  A short item is mostly set-up, load
// latency and output (one key tile 4.3 us, each further one 0.7 us), two of them at a time on an
// SM (24 captions of 8 to 512 tokens, 32 heads on 8: 34 us, 2.5 times the floor of their products
// and bytes).
// Measured and not kept: two query tiles and 128-key tiles per CTA, one CTA per SM (half the K
// and V traffic, but it waits for its own softmax: 1.0 to 1.6 times slower from 300 to 16384
// tokens with 8 key heads); a persistent kernel that loads the next item while it finishes the
// last (its bookkeeping costs 1 us an item and the static shares are uneven: 1.2 to 1.4 times
// slower).
//
// Keys are split over CTAs when the items do not fill the GPU: each part writes its normalised
// O (fp32) with its maximum and sum to the workspace, and a second kernel joins the parts of a
// row in a fixed order.
#include <algorithm>
#include <climits>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace zdit {

bool make_tmap_bf16_heads(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t heads, uint64_t head_dim,
                          uint64_t row_stride, uint64_t head_stride, uint32_t box_heads, uint32_t box_rows);
bool heads_disjoint(const zdit_heads& h, int64_t rows, int heads, int head_dim);

namespace {

constexpr int TILE = 128;       // rows of a query tile
constexpr int KTILE = 64;       // keys of a key tile
constexpr int THREADS = 224;
constexpr int WARP_QK = 4, WARP_MMA = 5, WARP_V = 6;
constexpr int kMaxSeqs = 128;
constexpr float kRescaleThreshold = 16.0f;  // log2 units

// Per-sequence plan, in the order the items are launched (longest key range first).
struct Plan {
  int n;  // sequences with query rows
  int item0[kMaxSeqs + 1];  // first item (per key head) of sequence i; item0[n] = all
  int q0[kMaxSeqs], q_len[kMaxSeqs], kv0[kMaxSeqs], kv_len[kMaxSeqs];
  int tiles[kMaxSeqs];      // query tiles
  int parts[kMaxSeqs];      // key splits
  int chunk[kMaxSeqs];      // keys of a part, a multiple of KTILE
  int part0[kMaxSeqs];      // first partial row of the sequence in the workspace (parts > 1)
  int join0[kMaxSeqs + 1];  // first joined row (token, head) among sequences with parts > 1
};

struct PParams {
  int n_kv, group, tokens;  // tokens per query tile
  int causal;
  int heads_first;          // grid (key heads, items) instead of (items, key heads)
  float scale_log2;
  __nv_bfloat16* o;
  int64_t o_rs, o_hs;
  const __nv_bfloat16* v;   // read again only for infinities and NaN at masked places
  int64_t v_rs, v_hs;
  float* part_o;    // [rows][HD] normalised partial outputs
  float2* part_ml;  // [rows] (maximum in log2 units, sum)
  int* err;
};

template <int HD>
struct Cfg {
  static constexpr int Q_HALF = TILE * 128;              // 64 columns x 128 rows
  static constexpr int Q_BYTES = (HD / 64) * Q_HALF;
  static constexpr int HALF = KTILE * 128;               // 64 columns x 64 keys, 8 KB
  static constexpr int TILE_BYTES = (HD / 64) * HALF;
  static constexpr int ST = HD == 128 ? 2 : 4;           // ring depth of K and of V (32 KB each)
  static constexpr int OFF_K = Q_BYTES;
  static constexpr int OFF_V = OFF_K + ST * TILE_BYTES;
  static constexpr int OFF_BAR = OFF_V + ST * TILE_BYTES;
  static constexpr int SMEM = 1024 + OFF_BAR + 256;      // two CTAs fit an SM
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint64_t pk2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpk2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Largest key index allowed for query token `tok` of a sequence (-1: none).
__device__ __forceinline__ int last_key(int tok, int q_len, int kv_len, int causal) {
  return causal ? min(tok + kv_len - q_len, kv_len - 1) : kv_len - 1;
}

// Index of the sequence that item `item` (per key head) belongs to.
__device__ __forceinline__ int find_item(const Plan& plan, int item) {
  int lo = 0, hi = plan.n;  // plan.item0[lo] <= item < plan.item0[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan.item0[mid] <= item) lo = mid; else hi = mid;
  }
  return lo;
}

template <int N>
__device__ __forceinline__ float row_max(const float (&s)[N]) {
  float m8[8];  // independent chains of 3-input max
#pragma unroll
  for (int e = 0; e < 8; ++e) m8[e] = fmaxf(s[e], s[8 + e]);
#pragma unroll
  for (int e = 16; e < N; e += 16)
#pragma unroll
    for (int k = 0; k < 8; ++k) m8[k] = fmax3(m8[k], s[e + k], s[e + 8 + k]);
  return fmaxf(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], fmax3(m8[5], m8[6], m8[7])));
}

// P = exp2(s scale - m_use) of one row over a tile of N logits, stored as bf16 pairs over the
// tile's first columns of TMEM; returns the sum of the unrounded P.
template <int N>
__device__ __forceinline__ float row_exp(const float (&s)[N], float scale_log2, float m_use, uint32_t tS) {
  const uint64_t sc2 = pk2(scale_log2, scale_log2);
  const uint64_t nm2 = pk2(-m_use, -m_use);
  uint64_t sum4[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int e4 = 0; e4 < N / 32; ++e4) {
    uint32_t pk[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const uint64_t x2 = fma2(pk2(s[e4 * 32 + 2 * e], s[e4 * 32 + 2 * e + 1]), sc2, nm2);
      float a, b;
      unpk2(x2, a, b);
      const float p0 = ex2(a), p1 = ex2(b);
      sum4[e & 3] = add2(sum4[e & 3], pk2(p0, p1));
      pk[e] = pack_bf16x2(p0, p1);
    }
    tmem_st16(tS + e4 * 16, pk);
  }
  float a0, a1, a2, a3, a4, a5, a6, a7;
  unpk2(sum4[0], a0, a1);
  unpk2(sum4[1], a2, a3);
  unpk2(sum4[2], a4, a5);
  unpk2(sum4[3], a6, a7);
  return ((a0 + a1) + (a2 + a3)) + ((a4 + a5) + (a6 + a7));
}

// O (HD columns of TMEM) *= alpha.
template <int HD>
__device__ __forceinline__ void scale_o(uint32_t tO, float alpha) {
#pragma unroll 1
  for (int e = 0; e < HD / 16; ++e) {
    uint32_t r[16];
    tmem_ld16(tO + e * 16, r);
    tmem_ld_wait();
#pragma unroll
    for (int k = 0; k < 16; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * alpha);
    tmem_st16(tO + e * 16, r);
  }
}

// A key that a row may not see has P = 0, but 0 times an infinity or NaN in its row of V is
// not 0.  So a V tile in shared memory is cleaned before a product that some row may not see
// all of: rows from `valid` on (past the end of the sequence) are cleared, and with `scan`
// infinities and NaN are taken out; returns whether any were (they are added back, in the
// epilogue, to the rows that do see them).  It costs 5% on a batch of short prompts (32.6 us
// without, 34.3 with, 24 captions of 8 to 512 tokens) and nothing where few tiles are masked; to
// look at the outputs instead, and do an item with a NaN again, measured the same.  Half row t <
// 128 (at head_dim 64 every other half of its pieces); the order of the 16-byte pieces spreads
// eight rows over all banks.
template <int HD>
__device__ __forceinline__ bool clean_v_tile(uint8_t* v_tile, int half_bytes, int t, int valid, bool scan) {
  constexpr int PIECES = HD / 16;  // 16-byte pieces of half a row
  const int row = t & 63, h = t >> 6;
  uint8_t* base = v_tile + (HD == 64 ? 0 : h * half_bytes) + row * 128;
  auto at = [&](int e) { return base + ((e + row + (HD == 64 ? h * PIECES : 0)) & 7) * 16; };
  if (row >= valid) {
#pragma unroll
    for (int e = 0; e < PIECES; ++e) *reinterpret_cast<uint4*>(at(e)) = make_uint4(0, 0, 0, 0);
    return false;
  }
  if (!scan) return false;
  // adding one unit of the exponent's last place carries into the sign bit exactly where the
  // exponent is all ones
  uint32_t found = 0;
#pragma unroll
  for (int e = 0; e < PIECES; ++e) {
    const uint4 u = *reinterpret_cast<const uint4*>(at(e));
    found |= ((u.x & 0x7f807f80u) + 0x00800080u) | ((u.y & 0x7f807f80u) + 0x00800080u) |
             ((u.z & 0x7f807f80u) + 0x00800080u) | ((u.w & 0x7f807f80u) + 0x00800080u);
  }
  if ((found & 0x80008000u) == 0) return false;
  for (int e = 0; e < PIECES; ++e)
    for (int k = 0; k < 8; ++k) {
      uint16_t* x = reinterpret_cast<uint16_t*>(at(e)) + k;
      if ((*x & 0x7f80u) == 0x7f80u) *x = 0;
    }
  return true;
}

// One warp's 32 finished rows as bf16, staged in shared memory (row pitch padded against
// bank conflicts) and stored as whole rows; off: element offset of this lane's row in o, -1
// for none.  take(e4, v) yields 32 columns of the row.
template <int HD, typename Take>
__device__ __forceinline__ void store_rows(uint8_t* stage, int lane, long long off, __nv_bfloat16* o, Take take) {
  constexpr int PITCH = 2 * HD + 16;
  for (int e4 = 0; e4 < HD / 32; ++e4) {
    float v[32];
    take(e4, v);
    uint4* dst = reinterpret_cast<uint4*>(stage + lane * PITCH + e4 * 64);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      dst[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                          pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
  }
  __syncwarp();
  constexpr int LPR = HD / 8;  // lanes per row
#pragma unroll 4
  for (int it = 0; it < LPR; ++it) {
    const int r = it * (32 / LPR) + lane / LPR;
    const long long ro = __shfl_sync(0xffffffffu, off, r);
    const uint4 v = *reinterpret_cast<const uint4*>(stage + r * PITCH + (lane % LPR) * 16);
    if (ro >= 0) *reinterpret_cast<uint4*>(o + ro + (lane % LPR) * 8) = v;
  }
}

template <int HD>
__global__ void __launch_bounds__(THREADS, 2)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                              const __grid_constant__ CUtensorMap tmV, const __grid_constant__ Plan plan,
                              const PParams p) {
  using C = Cfg<HD>;
  constexpr int ST = C::ST;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;
  uint64_t* pv_done = bars + 1;     // one phase per PV product
  uint64_t* mma_done = bars + 2;
  uint64_t* s_full = bars + 3;      // [2]
  uint64_t* p_full = bars + 5;      // [2]
  uint64_t* k_full = bars + 7;      // [ST]
  uint64_t* k_empty = k_full + ST;  // [ST]
  uint64_t* v_full = k_empty + ST;  // [ST]
  uint64_t* v_empty = v_full + ST;  // [ST]
  uint64_t* v_clean = v_empty + ST; // [ST] one phase per cleaned tile of the stage
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(v_clean + ST);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* bad_v = abort_flag + 1;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // Item of this CTA: the items of a head come by decreasing work, either head after head or
  // all heads of an item next to each other (see launch_prompt).  No division on the way to
  // the first load unless keys are split.
  const int kvh = p.heads_first ? blockIdx.x : blockIdx.y;
  const int item = p.heads_first ? blockIdx.y : blockIdx.x;
  const int sq = find_item(plan, item);
  const int q_len = plan.q_len[sq], kv_len = plan.kv_len[sq], kv0 = plan.kv0[sq], q0 = plan.q0[sq];
  const int parts = plan.parts[sq];
  int tile = item - plan.item0[sq], part = 0, key_first = 0;
  if (parts > 1) {
    const int t = tile / parts;
    part = tile - t * parts;
    tile = t;
    key_first = part * plan.chunk[sq];
  }
  const int tok0 = (plan.tiles[sq] - 1 - tile) * p.tokens;  // later rows see more keys: first
  // key tiles of this item; the first that some of its rows see more of than others; the first
  // whose V rows need cleaning (those, and the one that the sequence ends in)
  int n, masked, clean_from;
  {
    const int first = last_key(tok0, q_len, kv_len, p.causal);
    const int lk = last_key(min(tok0 + p.tokens, q_len) - 1, q_len, kv_len, p.causal);
    const int end = parts > 1 ? min(lk + 1, key_first + plan.chunk[sq]) : lk + 1;
    n = end > key_first ? (end - key_first + KTILE - 1) / KTILE : 0;
    masked = first < lk ? max(first + 1 - key_first, 0) / KTILE : n;
    clean_from = min(masked, key_first + n * KTILE > kv_len ? n - 1 : n);
  }
  auto load_k = [&](int i) {
    uint8_t* sK = smem + C::OFF_K + (i % ST) * C::TILE_BYTES;
    mbar_arrive_expect_tx(&k_full[i % ST], C::TILE_BYTES);
    for (int c = 0; c < HD / 64; ++c)
      tma_load_3d(sK + c * C::HALF, &tmK, &k_full[i % ST], c * 64, kvh, kv0 + key_first + i * KTILE);
  };
  auto load_v = [&](int i) {
    uint8_t* sV = smem + C::OFF_V + (i % ST) * C::TILE_BYTES;
    mbar_arrive_expect_tx(&v_full[i % ST], C::TILE_BYTES);
    for (int c = 0; c < HD / 64; ++c)
      tma_load_3d(sV + c * C::HALF, &tmV, &v_full[i % ST], c * 64, kvh, kv0 + key_first + i * KTILE);
  };

  if (warp == WARP_QK && lane == 0) {
    mbar_init(q_full, 1);
    mbar_init(pv_done, 1);
    mbar_init(mma_done, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    for (int i = 0; i < ST; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&v_clean[i], 1);
    }
    *abort_flag = 0;
    *bad_v = 0;
    fence_barrier_init();
    griddep_wait();  // Q, K, V of the predecessor are complete
    // this thread made the barriers: its first loads need not wait for the others
    if (n > 0) {
      mbar_arrive_expect_tx(q_full, (uint32_t)(p.group * p.tokens * 128 * (HD / 64)));
      for (int c = 0; c < HD / 64; ++c)
        tma_load_3d(smem + c * C::Q_HALF, &tmQ, q_full, c * 64, kvh * p.group, q0 + tok0);
      for (int i = 0; i < min(n, ST); ++i) load_k(i);
      for (int i = 0; i < min(n, ST); ++i) load_v(i);
    }
  }
  if (warp == WARP_MMA) tmem_alloc(tmem_slot, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();     // (every thread: the outputs and the workspace are free)
  griddep_trigger();  // every CTA has started: the successor may launch

  if (warp == WARP_QK) {
    if (lane == 0) {
      // ------------------------------------------------------------ K (and Q above)
      int issued = min(n, ST);
      for (; issued < n; ++issued) {
        if (!mbar_wait(&k_empty[issued % ST], ((issued / ST) & 1) ^ 1, abort_flag, p.err)) break;
        load_k(issued);
      }
      if (*abort_flag && n > 0) {  // let copies in flight land before shared memory is released
        int dummy = 0;
        mbar_wait(q_full, 0, &dummy);
        for (int i = max(issued - ST, 0); i < issued; ++i) mbar_wait(&k_full[i % ST], (i / ST) & 1, &dummy);
      }
    }
  } else if (warp == WARP_V) {
    // ------------------------------------------------------------ V
    // The warp cleans tile i while the softmax works on it, then one lane loads tile i + ST when
    // the PV product of tile i is done.  A barrier only tells the phase before the current one
    // from the current one, so whoever waits for a tile of a stage must not be a round ahead of
    // it: this warp has loaded the tile that it waits for, and it cannot clean the next one of
    // the stage before the MMA thread has taken this one.  (No other warp can help: it could be
    // ahead of the loads.)
    int issued = min(n, ST);
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      if (i >= clean_from) {
        ok = __all_sync(0xffffffffu, mbar_wait(&v_full[i % ST], (i / ST) & 1, abort_flag, p.err));
        if (!ok) break;
        uint8_t* sV = smem + C::OFF_V + (i % ST) * C::TILE_BYTES;
        const int valid = kv_len - key_first - i * KTILE;
        bool bad = false;
        // (as a loop: its four turns unrolled made the 24 captions' call 38.4 us instead of 34.2)
#pragma unroll 1
        for (int t = 0; t < 128; t += 32) bad |= clean_v_tile<HD>(sV, C::HALF, t + lane, valid, i >= masked);
        if (bad) *bad_v = 1;
        // (the tensor core has to see what was written; mostly nothing was)
        if (__any_sync(0xffffffffu, bad || valid < KTILE)) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_clean[i % ST]);
      }
      if (issued < n) {  // tile i + ST
        if (lane == 0) {
          ok = mbar_wait(&v_empty[i % ST], (i / ST) & 1, abort_flag, p.err);
          if (ok) load_v(issued);
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++issued;
      }
    }
    if (lane == 0 && *abort_flag) {
      int dummy = 0;
      for (int i = max(issued - ST, 0); i < issued; ++i) mbar_wait(&v_full[i % ST], (i / ST) & 1, &dummy);
    }
  } else if (warp == WARP_MMA) {
    if (lane == 0 && n > 0) {
      // ------------------------------------------------------------ MMA issuer
      const uint32_t id_s = idesc_bf16_f32(TILE, KTILE);            // Q, K both K-major
      const uint32_t id_o = idesc_bf16_f32(TILE, HD, false, true);  // P from TMEM, V MN-major
      const uint64_t dq = sdesc_kmajor_sw128(smem_u32(smem));
      const uint64_t dk = sdesc_kmajor_sw128(smem_u32(smem + C::OFF_K));
      const uint64_t dv = sdesc_mnmajor_sw128(smem_u32(smem + C::OFF_V), C::HALF, 1024);
      constexpr uint64_t kTileDesc = C::TILE_BYTES >> 4;
      bool ok = mbar_wait(q_full, 0, abort_flag, p.err);
      // S_i into buffer i & 1: after PV of tile i - 2, which read P from the same columns
      auto sk = [&](int i) -> bool {
        if (!mbar_wait(&k_full[i % ST], (i / ST) & 1, abort_flag, p.err)) return false;
        tc_fence_after();
        const uint64_t kb = dk + (i % ST) * kTileDesc;
        const uint32_t d = tmem + (i & 1) * KTILE;
#pragma unroll
        for (int k = 0; k < HD / 16; ++k)
          umma_bf16_ss(d, dq + (uint64_t)(((k >> 2) * C::Q_HALF + (k & 3) * 32) >> 4),
                       kb + (uint64_t)(((k >> 2) * C::HALF + (k & 3) * 32) >> 4), id_s, k != 0 ? 1u : 0u);
        umma_commit(&s_full[i & 1]);
        umma_commit(&k_empty[i % ST]);
        return true;
      };
      if (ok) ok = sk(0);
      if (ok && n > 1) ok = sk(1);
      for (int i = 0; ok && i < n; ++i) {
        if (!(ok = mbar_wait(&p_full[i & 1], (i >> 1) & 1, abort_flag, p.err))) break;
        if (!(ok = mbar_wait(&v_full[i % ST], (i / ST) & 1, abort_flag, p.err))) break;
        if (i >= clean_from && !(ok = mbar_wait(&v_clean[i % ST], ((i - clean_from) / ST) & 1, abort_flag, p.err)))
          break;
        tc_fence_after();
        const uint64_t vb = dv + (i % ST) * kTileDesc;
        const uint32_t pa = tmem + (i & 1) * KTILE;
#pragma unroll
        for (int k = 0; k < KTILE / 16; ++k)
          umma_bf16_ts(tmem + 2 * KTILE, pa + k * 8, vb + (uint64_t)((k * 16 * 128) >> 4), id_o, (i | k) != 0 ? 1u : 0u);
        umma_commit(pv_done);
        umma_commit(&v_empty[i % ST]);
        if (i + 2 < n) ok = sk(i + 2);
      }
      umma_commit(mma_done);
      int dummy = 0;
      mbar_wait(mma_done, 0, &dummy);
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int row = warp * 32 + lane;
    const int tok = tok0 + row / p.group;
    const int head = kvh * p.group + row % p.group;
    const bool live = row < p.group * p.tokens && tok < q_len;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const int lim = live ? last_key(tok, q_len, kv_len, p.causal) : kv_len - 1;
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tO = tmem + lane_off + 2 * KTILE;
    float m_ref = -INFINITY, l_sum = 0.f;
    bool ok = true;
    for (int i = 0; i < n; ++i) {
      const int key0 = key_first + i * KTILE;
      ok = __all_sync(0xffffffffu, mbar_wait(&s_full[i & 1], (i >> 1) & 1, abort_flag, p.err));
      if (!ok) break;
      tc_fence_after();
      if (warp_live) {
        const uint32_t tS = tmem + lane_off + (i & 1) * KTILE;
        float s[KTILE];
#pragma unroll
        for (int e4 = 0; e4 < KTILE / 32; ++e4) {
          uint32_t r[32];
          tmem_ld32(tS + e4 * 32, r);
#pragma unroll
          for (int e = 0; e < 32; ++e) s[e4 * 32 + e] = __uint_as_float(r[e]);
        }
        tmem_ld_wait();
        const int valid = lim - key0;  // last allowed column of this tile
        if (valid < KTILE - 1) {
#pragma unroll
          for (int e = 0; e < KTILE; ++e)
            if (e > valid) s[e] = -INFINITY;
        }
        const float mx = row_max<KTILE>(s) * p.scale_log2;
        float alpha = 1.f;
        bool move = false;
        if (i == 0) {
          m_ref = mx;
        } else if (mx > m_ref + kRescaleThreshold) {
          alpha = ex2(m_ref - mx);
          m_ref = mx;
          move = true;
        }
        if (__any_sync(0xffffffffu, move)) {
          // the previous PV may still be adding to O (phase i - 1; the one before it completed
          // before this S, which was issued after it)
          ok = __all_sync(0xffffffffu, mbar_wait(pv_done, (i - 1) & 1, abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
          scale_o<HD>(tO, alpha);
        }
        l_sum = l_sum * alpha + row_exp<KTILE>(s, p.scale_log2, m_ref == -INFINITY ? 0.f : m_ref, tS);
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[i & 1]);
    }
    // ------------------------------------------------------------ epilogue
    // (pv_done could be two phases behind here, which its parity does not show)
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(mma_done, 0, abort_flag, p.err));
    tc_fence_after();
    if (ok && warp_live) {
      const float inv = l_sum == 0.f ? 0.f : 1.0f / l_sum;
      auto take = [&](int e4, float (&v)[32]) {  // 32 columns of the finished row
        if (n > 0) {
          uint32_t r[32];
          tmem_ld32(tO + e4 * 32, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(r[e]) * inv;
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = 0.f;
        }
      };
      if (parts > 1) {
        const int64_t at = (int64_t)plan.part0[sq] + ((int64_t)part * q_len + tok) * (p.n_kv * p.group) + head;
        if (live) p.part_ml[at] = make_float2(m_ref, l_sum);
        // through shared memory (every product is done: Q and the rings are idle), so that a
        // store instruction writes four whole lines instead of 16 bytes of 32 (100 tokens, 32 heads
        // on 8, 2000 keys: 17.3 -> 15.0 us; single tokens, 4 rows of a tile: 36.9 -> 37.2 us)
        constexpr int PITCH = 128 + 16;
        uint8_t* stage = smem + warp * 32 * PITCH;
        const long long off = live ? at * HD : -1;
        const int rows = __popc(__ballot_sync(0xffffffffu, live));  // the live rows come first
        for (int e4 = 0; e4 < HD / 32; ++e4) {
          float v[32];
          take(e4, v);
          float4* dst = reinterpret_cast<float4*>(stage + lane * PITCH);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          __syncwarp();
#pragma unroll
          for (int it = 0; it < 8; ++it) {
            if (it * 4 >= rows) break;
            const int r = it * 4 + lane / 8;
            const long long ro = __shfl_sync(0xffffffffu, off, r);
            const float4 f = *reinterpret_cast<const float4*>(stage + r * PITCH + (lane % 8) * 16);
            if (ro >= 0) *reinterpret_cast<float4*>(p.part_o + ro + e4 * 32 + (lane % 8) * 4) = f;
          }
          __syncwarp();
        }
      } else {
        // every product is done: Q and the rings are idle
        store_rows<HD>(smem + warp * 32 * (2 * HD + 16), lane,
                       live ? (q0 + (int64_t)tok) * p.o_rs + head * p.o_hs : -1, p.o, take);
      }
      if (*bad_v != 0) {
        // infinities and NaN were taken out of V: added to the stored rows that see them
        __syncwarp();
        for (int j = key_first + masked * KTILE; live && j <= min(lim, key_first + n * KTILE - 1); ++j) {
          const __nv_bfloat16* vp = p.v + (kv0 + (int64_t)j) * p.v_rs + kvh * p.v_hs;
          for (int e = 0; e < HD; ++e) {
            const float x = __bfloat162float(vp[e]);
            if (isfinite(x)) continue;
            if (parts > 1) {
              const int64_t at = (int64_t)plan.part0[sq] + ((int64_t)part * q_len + tok) * (p.n_kv * p.group) + head;
              p.part_o[at * HD + e] += x;
            } else {
              __nv_bfloat16* op = p.o + (q0 + (int64_t)tok) * p.o_rs + head * p.o_hs + e;
              *op = __float2bfloat16_rn(__bfloat162float(*op) + x);
            }
          }
        }
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == WARP_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// Joins the parts of a split row: O = sum_s w_s O_s / sum_s w_s, w_s = l_s 2^(m_s - max m).
// WPR warps per (token, head) row; warp w of a row takes the parts w, w + WPR, ..., and the
// warps' sums are added in order (the result does not depend on timing).  A chain of
// dependent loads, so everything that does not come from the parts is found before the wait,
// and the partial rows are requested together with their maxima.  Four warps a row while the
// rows are few (32 parts of 4 rows: 8 us with one warp, 2 us with four), one when they fill the
// GPU by themselves (2664 rows of 10 parts: 8.7 us with four, 5.4 us with one; two warps a row,
// or 5 or 16 parts requested at a time, are within 10% of that or slower).
constexpr int kJoinThreads = 128;
template <int HD, int WPR>
__global__ void __launch_bounds__(kJoinThreads)
    prompt_join_kernel(const __grid_constant__ Plan plan, const PParams p) {
  constexpr int V = HD / 32, AHEAD = WPR == 1 ? 8 : 4, ROWS = kJoinThreads / 32 / WPR;
  __shared__ float sh[WPR > 1 ? WPR : 1][HD + 2];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % WPR;
  const int total = plan.join0[plan.n];
  const int r = blockIdx.x * ROWS + (threadIdx.x >> 5) / WPR;
  const bool live = r < total;
  int lo = 0, hi = plan.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (plan.join0[mid] <= r) lo = mid; else hi = mid;
  }
  const int H = p.n_kv * p.group;
  const int64_t rows = (int64_t)plan.q_len[lo] * H;
  const int parts = live ? plan.parts[lo] : 0;
  const int rr = r - plan.join0[lo];
  const int64_t at = (int64_t)plan.part0[lo] + rr;
  const int tok = rr / H, head = rr - tok * H;
  __nv_bfloat16* dst = p.o + (plan.q0[lo] + (int64_t)tok) * p.o_rs + head * p.o_hs + lane * V;
  griddep_wait();
  griddep_trigger();
  // this warp's parts, AHEAD at a time, with a running maximum
  float m = -INFINITY, den = 0.f, acc[V] = {};
  for (int s0 = warp; s0 < parts; s0 += AHEAD * WPR) {
    float2 ml[AHEAD];
    float v[AHEAD][V];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      const int s = s0 + j * WPR;
      ml[j] = make_float2(-INFINITY, 0.f);
      if (s < parts) {
        const int64_t a = at + s * rows;
        ml[j] = p.part_ml[a];
        const float* src = p.part_o + a * HD + lane * V;
        if constexpr (V == 4) {
          const float4 f = *reinterpret_cast<const float4*>(src);
          v[j][0] = f.x; v[j][1] = f.y; v[j][2] = f.z; v[j][3] = f.w;
        } else {
          const float2 f = *reinterpret_cast<const float2*>(src);
          v[j][0] = f.x; v[j][1] = f.y;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (ml[j].y == 0.f) continue;  // no key of this part is allowed for the row
      const float mn = fmaxf(m, ml[j].x);
      const float f = m == -INFINITY ? 0.f : ex2(m - mn), w = ml[j].y * ex2(ml[j].x - mn);
      den = den * f + w;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(w, v[j][e], acc[e] * f);
      m = mn;
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) sh[warp][lane * V + e] = acc[e];
    if (lane == 0) {
      sh[warp][HD] = m;
      sh[warp][HD + 1] = den;
    }
    __syncthreads();
    if (warp != 0) return;
    m = -INFINITY;
#pragma unroll
    for (int w = 0; w < WPR; ++w) m = sh[w][HD + 1] == 0.f ? m : fmaxf(m, sh[w][HD]);
    den = 0.f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) {
      if (sh[w][HD + 1] == 0.f) continue;
      const float f = ex2(sh[w][HD] - m);
      den = fmaf(sh[w][HD + 1], f, den);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(sh[w][lane * V + e], f, acc[e]);
    }
  }
  if (!live) return;
  const float inv = den == 0.f ? 0.f : 1.0f / den;
  if constexpr (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv),
                                                pack_bf16x2(acc[2] * inv, acc[3] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(acc[0] * inv, acc[1] * inv);
}

// Keys of a part (INT_MAX: not split): the length that gives the earliest end when the parts
// run over two slots per SM.  Costs in keys (0.01 us, what a key takes in a part of its own):
// 400 for a part's set-up and output, 250 for the join and 6 for each part that it goes
// through.  (One row group, head_dim 128, us split / not: 256 keys 7.1 / 6.9, 448 keys 6.2 / 9.1.)
template <typename Seq>
int choose_part(const Seq* seq, int n, int tokens, int n_kv, int64_t sms) {
  constexpr int kMinPart = 128, kPartCost = 400, kJoinCost = 250, kJoinPartCost = 6;
  const int64_t slots = 2 * sms;
  int longest = 1;
  int64_t items = 0;
  for (int i = 0; i < n; ++i) {
    longest = std::max(longest, seq[i].kl);
    items += (int64_t)((seq[i].ql + tokens - 1) / tokens) * n_kv;
  }
  if (items >= slots || longest <= 2 * kMinPart) return INT_MAX;
  int64_t best_cost = (int64_t)longest + kPartCost;  // not split: no join either
  int best = INT_MAX;
  for (int c = kMinPart; c < longest; c += std::max(KTILE, c / 4 / KTILE * KTILE)) {
    int64_t m = 0;
    int big = 0;
    for (int i = 0; i < n; ++i) {
      const int parts = std::max(1, (seq[i].kl + c - 1) / c);
      m += (int64_t)((seq[i].ql + tokens - 1) / tokens) * n_kv * parts;
      big = std::max(big, (seq[i].kl + parts - 1) / parts);
    }
    const int64_t cost = (m + slots - 1) / slots * (big + kPartCost) + kJoinCost + kJoinPartCost * (longest / c);
    if (cost < best_cost) {
      best_cost = cost;
      best = c;
    }
  }
  return best;
}

struct HostPlan {
  Plan p;
  int tokens, group;
  int64_t q_rows, kv_rows, part_rows;
  double pairs;  // allowed (query, key) pairs, for the profiler
};

// Kernel, items, splits and workspace rows of a call; false on invalid lengths.
bool make_plan(const zdit_prompt_attention_args& a, HostPlan* h) {
  if (a.batch <= 0 || a.batch > kMaxSeqs || !a.q_len || a.n_kv_heads <= 0 || a.n_heads <= 0 ||
      a.n_heads % a.n_kv_heads || a.n_heads / a.n_kv_heads > 64 || (a.head_dim != 64 && a.head_dim != 128) ||
      a.n_heads > 65535 || a.causal < 0 || a.causal > 1)
    return false;
  h->group = a.n_heads / a.n_kv_heads;
  h->tokens = TILE / h->group;
  struct Seq { int q0, ql, kv0, kl; };
  Seq seq[kMaxSeqs];
  int n = 0;
  int64_t q = 0, kv = 0;
  h->kv_rows = 0;
  h->pairs = 0;
  for (int b = 0; b < a.batch; ++b) {
    const int64_t ql = a.q_len[b], kl = a.kv_len ? a.kv_len[b] : ql, k0 = a.kv_start ? a.kv_start[b] : kv;
    if (ql < 0 || kl < 0 || k0 < 0 || k0 + kl > (1 << 30) || q + ql > (1 << 30)) return false;
    if (!a.kv_start) kv += kl;
    h->kv_rows = std::max(h->kv_rows, k0 + kl);
    if (ql > 0) {
      seq[n++] = Seq{(int)q, (int)ql, (int)k0, (int)kl};
      double seen = (double)ql * kl;  // allowed pairs
      if (a.causal) seen = kl >= ql ? seen - 0.5 * ql * (ql - 1.0) : 0.5 * kl * (kl + 1.0);
      h->pairs += seen;
    }
    q += ql;
  }
  h->q_rows = q;
  const int64_t sms = num_sms();
  // Longest key range first: its items start early.
  std::sort(seq, seq + n, [](const Seq& x, const Seq& y) { return x.kl != y.kl ? x.kl > y.kl : x.q0 < y.q0; });
  const int part_keys = choose_part(seq, n, h->tokens, a.n_kv_heads, sms);
  int64_t items = 0, parts_rows = 0, join = 0;
  Plan& p = h->p;
  p.n = n;
  for (int i = 0; i < n; ++i) {
    const Seq& s = seq[i];
    const int parts = part_keys == INT_MAX ? 1 : std::max(1, (s.kl + part_keys - 1) / part_keys);
    p.item0[i] = (int)items;
    p.tiles[i] = (s.ql + h->tokens - 1) / h->tokens;
    p.q0[i] = s.q0; p.q_len[i] = s.ql; p.kv0[i] = s.kv0; p.kv_len[i] = s.kl; p.parts[i] = parts;
    p.chunk[i] = ((s.kl + parts - 1) / parts + KTILE - 1) / KTILE * KTILE;  // parts of equal length
    p.part0[i] = (int)parts_rows;
    p.join0[i] = (int)join;
    items += (int64_t)p.tiles[i] * parts;
    if (parts > 1) {
      join += (int64_t)s.ql * a.n_heads;
      parts_rows += (int64_t)s.ql * a.n_heads * parts;
    }
    if (items > INT_MAX || parts_rows > INT_MAX || join > INT_MAX) return false;
  }
  p.item0[n] = (int)items;
  p.join0[n] = (int)join;
  h->part_rows = parts_rows;
  return true;
}

size_t plan_bytes(const HostPlan& h, int head_dim) {
  if (h.part_rows == 0) return 0;
  const size_t ml = ((size_t)h.part_rows * sizeof(float2) + 255) / 256 * 256;
  return ml + (size_t)h.part_rows * head_dim * sizeof(float);
}

template <int HD>
zdit_status launch_prompt(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const HostPlan& h,
                          PParams p, cudaStream_t s) {
  const int H = p.n_kv * p.group;
  {
    ProfScope ps(PROF_ATTENTION, 4.0 * HD * H * h.pairs,
                 2.0 * HD * (2.0 * H * h.q_rows + 2.0 * p.n_kv * h.kv_rows), s);
    // Head after head keeps one head's keys in L2 while its items run (30 heads, 16384 tokens: 2.08
    // against 2.17 ms; 16 on 2, 2 of 8192: 504 against 529 us); but with few waves the last head's
    // longest items would end the launch alone, so then the longest items of all heads come first
    // (32 on 8, 2 prompts of 1024 tokens: 27 against 37 us; 8 heads, 2 of 4096: 70 against 106).
    // Causal, 1 to 30 key heads, 1 to 120 prompts of 8 to 32768 tokens, time of head after head over
    // heads first: 0.99 to 1.51 below 9 waves, 0.95 to 1.08 above but for one (30 heads, 120 of 300
    // tokens: 1.32).  Unmasked items of a sequence are all alike (0.90 to 1.04; short prompts of 30
    // heads 1.3).
    const int64_t items = h.p.item0[h.p.n];
    p.heads_first = p.causal && items * p.n_kv < 9 * (int64_t)num_sms();
    const dim3 grid = p.heads_first ? dim3((unsigned)p.n_kv, (unsigned)items) : dim3((unsigned)items, (unsigned)p.n_kv);
    // per launch: the shared-memory opt-in belongs to the current context
    cudaError_t e =
        cudaFuncSetAttribute(prompt_attn_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<HD>::SMEM);
    if (e == cudaSuccess)
      e = launch_dependent(prompt_attn_kernel<HD>, grid, dim3(THREADS), Cfg<HD>::SMEM, s, tq, tk, tv, h.p, p);
    if (e != cudaSuccess) return launch_status(e);
  }
  const int join = h.p.join0[h.p.n];
  if (join > 0) {
    ProfScope ps(PROF_ATTENTION, 0.0, (4.0 * HD + 8.0) * h.part_rows + 2.0 * HD * join, s);
    const dim3 block(kJoinThreads);
    const cudaError_t e =
        join > 8 * num_sms()
            ? launch_dependent(prompt_join_kernel<HD, 1>, dim3((unsigned)((join + 3) / 4)), block, 0, s, h.p, p)
            : launch_dependent(prompt_join_kernel<HD, 4>, dim3((unsigned)join), block, 0, s, h.p, p);
    if (e != cudaSuccess) return launch_status(e);
  }
  return launch_status(cudaSuccess);
}

}  // namespace

}  // namespace zdit

using namespace zdit;

extern "C" {

ZDIT_API size_t zdit_prompt_attention_workspace_bytes(const zdit_prompt_attention_args* a) {
  HostPlan h;
  if (a == nullptr || !make_plan(*a, &h)) return 0;
  return plan_bytes(h, a->head_dim);
}

ZDIT_API zdit_status zdit_prompt_attention(const zdit_prompt_attention_args* a, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  if (a == nullptr || !a->q_len) return ZDIT_ERR_INVALID_ARG;
  if (!(a->scale >= 0.f) || !std::isfinite(a->scale) || a->causal < 0 || a->causal > 1) return ZDIT_ERR_INVALID_ARG;
  HostPlan h;
  if (!make_plan(*a, &h)) return ZDIT_ERR_SHAPE;
  if (h.q_rows > 0 && (!a->q.ptr || !a->o.ptr)) return ZDIT_ERR_INVALID_ARG;
  if (h.kv_rows > 0 && (!a->k.ptr || !a->v.ptr)) return ZDIT_ERR_INVALID_ARG;
  if (a->o.ptr != nullptr && (a->o.ptr == a->q.ptr || a->o.ptr == a->k.ptr || a->o.ptr == a->v.ptr))
    return ZDIT_ERR_INVALID_ARG;
  const zdit_heads* hs[4] = {&a->q, &a->k, &a->v, &a->o};
  for (int i = 0; i < 4; ++i) {
    const int n = (i == 0 || i == 3) ? a->n_heads : a->n_kv_heads;
    const int64_t rows = (i == 0 || i == 3) ? h.q_rows : h.kv_rows;
    const int64_t lim = int64_t(1) << 38;  // strides of a tensor map are below 2^40 bytes
    if ((rows > 1 && (hs[i]->row_stride < a->head_dim || hs[i]->row_stride > lim)) ||
        (n > 1 && (hs[i]->head_stride < a->head_dim || hs[i]->head_stride > lim)))
      return ZDIT_ERR_SHAPE;
    if ((reinterpret_cast<uintptr_t>(hs[i]->ptr) & 15) || (rows > 1 && hs[i]->row_stride % 8) ||
        (n > 1 && hs[i]->head_stride % 8))
      return ZDIT_ERR_ALIGNMENT;
  }
  if (!heads_disjoint(a->o, h.q_rows, a->n_heads, a->head_dim)) return ZDIT_ERR_SHAPE;
  const size_t need = plan_bytes(h, a->head_dim);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return ZDIT_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return ZDIT_ERR_ALIGNMENT;
  }
  if (h.q_rows == 0) return ZDIT_OK;
  if (!device_ok()) return ZDIT_ERR_UNSUPPORTED;
  PParams p;
  p.n_kv = a->n_kv_heads; p.group = h.group; p.tokens = h.tokens; p.causal = a->causal;
  const float scale = a->scale == 0.f ? 1.0f / sqrtf((float)a->head_dim) : a->scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o = static_cast<__nv_bfloat16*>(a->o.ptr); p.o_rs = a->o.row_stride; p.o_hs = a->o.head_stride;
  p.v = static_cast<const __nv_bfloat16*>(a->v.ptr); p.v_rs = a->v.row_stride; p.v_hs = a->v.head_stride;
  p.part_ml = static_cast<float2*>(workspace);
  p.part_o = need ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) +
                                             ((size_t)h.part_rows * sizeof(float2) + 255) / 256 * 256) : nullptr;
  p.err = device_error_ptr();
  CUtensorMap tq, tk, tv;
  if (h.kv_rows == 0) {
    // no sequence has a key: no K or V tile is loaded, the maps only have to be valid
    if (!make_tmap_bf16_heads(&tk, a->q.ptr, 1, 1, a->head_dim, a->head_dim, a->head_dim, 1, KTILE))
      return ZDIT_ERR_CUDA;
    tv = tk;
  } else if (!make_tmap_bf16_heads(&tk, a->k.ptr, h.kv_rows, a->n_kv_heads, a->head_dim, a->k.row_stride,
                                   a->k.head_stride, 1, KTILE) ||
             !make_tmap_bf16_heads(&tv, a->v.ptr, h.kv_rows, a->n_kv_heads, a->head_dim, a->v.row_stride,
                                   a->v.head_stride, 1, KTILE)) {
    return ZDIT_ERR_CUDA;
  }
  if (!make_tmap_bf16_heads(&tq, a->q.ptr, h.q_rows, a->n_heads, a->head_dim, a->q.row_stride, a->q.head_stride,
                            h.group, h.tokens))
    return ZDIT_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  return a->head_dim == 64 ? launch_prompt<64>(tq, tk, tv, h, p, s) : launch_prompt<128>(tq, tk, tv, h, p, s);
}

}  // extern "C"
