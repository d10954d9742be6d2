// zdit_linear: out = residual + act(a . w^T + bias).
//
// Two kernels.  Many rows: the persistent projection GEMM of gemm.cu with the epilogue of
// linear_epi.cuh.  Few rows: the kernel below, which is bound by streaming w once.  There
// the weights are the 128-row operand of the tensor core and the rows of a its N side (16 to
// 160 columns, a multiple of 16), so a tile computes 128 output features for all rows with
// no padding of M to 128, and N / 128 tiles times `split` parts of K spread the weights
// over the SMs.  The parts of one tile are a cluster: each leaves its fp32 partial tile in
// its own shared memory and every CTA adds up its share of the rows over the cluster's
// shared memory, in rank order (the result does not depend on timing, and there is no
// workspace to clear or share).  At 133 x 9728 x 2560 (17.8 us) making the products takes 12 us,
// moving them to shared memory 1.4, and adding them up and storing 4, of which the distance of
// the peers' memory is 1.2; so the more rows the fewer parts.  Sending the rows to their owners
// with bulk copies instead is no faster (19.3 against 18.0 us, 1 x 2560 x 4096 8.4 against 7.5).
// Bias and residual are fetched while the products are made (19.1 -> 17.8 us with the
// accumulator read 16 instead of 8 columns at a time; 2048 deep, 2560 wide, 64 rows: 8.3 -> 7.7).
//
// Warp roles (320 threads): warp 0 loads (TMA ring), warp 1 issues the MMAs, warps 2-9 move
// the accumulator (TMEM lane = feature, column = row of a).
#include <algorithm>
#include <cmath>

#include "internal.h"
#include "linear_epi.cuh"
#include "ptx.cuh"

namespace zdit {

bool make_tmap_bf16_2d(CUtensorMap* m, const void* ptr, uint64_t rows, uint64_t cols, uint64_t ld_elems,
                       uint32_t box_rows, uint32_t box_cols);

namespace {

constexpr int FT = 128;              // features per tile
constexpr int BK = 64;               // K slice
constexpr int W_TILE = FT * BK * 2;  // 16 KB
constexpr int EPI_WARPS = 8;         // two per TMEM lane group
constexpr int THREADS = 64 + 32 * EPI_WARPS;
constexpr int kRing = 110 * 1024;    // shared memory of the ring: two CTAs fit an SM
constexpr int kMaxStages = 8;
constexpr int kMaxSplit = 8;         // portable cluster size
constexpr int kMaxRowTile = 160;     // rows of a in one tile
constexpr int kMaxSmem = 1024 + kRing;  // of any plan; the partial tiles lie over the idle ring
static_assert(kMaxRowTile * FT * 4 <= kRing, "partial tile");

struct FewParams {
  int M, N;
  int row_tile;  // rows of a per tile (UMMA N)
  int slices;    // K slices in all
  int split;     // CTAs per tile
  int stages;
  int group;     // K slices per ring stage
  uint32_t tmem_cols;
  LinearEpi e;
  int* err;
};

__device__ __forceinline__ uint32_t map_cluster(uint32_t addr, uint32_t cta) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(cta));
  return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// 32 lanes x 8 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
}

// Adds the residual to and stores n <= 8 rows of one feature: element offsets res and out, a
// row further each.  Types are told apart outside the loops and addresses advance by a row:
// with one value a lane and row, every instruction here counts.
template <typename T>
__device__ __forceinline__ void add_rows(const T* p, int64_t step, int n, float (&v)[8]) {
  T t[8];
#pragma unroll
  for (int j = 0; j < 8; ++j, p += step)
    if (j < n) t[j] = *p;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < n) v[j] += static_cast<float>(t[j]);
}
template <typename T>
__device__ __forceinline__ void store_rows(T* p, int64_t step, int n, const float (&v)[8]) {
  if (n == 8) {
#pragma unroll
    for (int j = 0; j < 8; ++j, p += step) *p = static_cast<T>(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j, p += step)
      if (j < n) *p = static_cast<T>(v[j]);
  }
}
__device__ __forceinline__ void finish_rows(const LinearEpi& e, int64_t res, int64_t out, int n, float (&v)[8]) {
  if (e.residual != nullptr) {
    if (e.res_f32)
      add_rows(static_cast<const float*>(e.residual) + res, e.ld_res, n, v);
    else
      add_rows(static_cast<const __nv_bfloat16*>(e.residual) + res, e.ld_res, n, v);
  }
  if (e.out_f32)
    store_rows(static_cast<float*>(e.out) + out, e.ld_out, n, v);
  else
    store_rows(static_cast<__nv_bfloat16*>(e.out) + out, e.ld_out, n, v);
}

__global__ void __launch_bounds__(THREADS)
    linear_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmA,
                      const FewParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  __shared__ uint64_t bars[2 * kMaxStages + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ volatile int abort_flag;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = bars;
  uint64_t* empty = bars + kMaxStages;
  uint64_t* done = bars + 2 * kMaxStages;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int tile = blockIdx.x / p.split;
  const int rank = blockIdx.x - tile * p.split;
  const int f0 = tile * FT;
  const int r0 = blockIdx.y * p.row_tile;
  const int k_lo = (int)((int64_t)p.slices * rank / p.split), k_hi = (int)((int64_t)p.slices * (rank + 1) / p.split);
  const int n = k_hi - k_lo;  // >= 1: split <= slices
  const int slice_bytes = W_TILE + p.row_tile * BK * 2;
  const int stage_bytes = p.group * slice_bytes;

  // The loads of this CTA, by thread 0.  (Stage and phase are counted: a division by the
  // run-time ring depth would cost more than the slice it serves.)
  int st = 0, k_at = k_lo * BK, left = n;
  uint32_t phase = 0, armed = 0;
  uint8_t* dst = smem;
  auto load_stage = [&]() {
    const int g = min(p.group, left);
    mbar_arrive_expect_tx(&full[st], g * slice_bytes);
    for (int j = 0; j < g; ++j) tma_load_2d(dst + j * slice_bytes, &tmW, &full[st], k_at + j * BK, f0);
    for (int j = 0; j < g; ++j) tma_load_2d(dst + j * slice_bytes + W_TILE, &tmA, &full[st], k_at + j * BK, r0);
    armed = (armed & ~(1u << st)) | (phase << st) | (0x10000u << st);
    left -= g;
    k_at += g * BK;
    dst += stage_bytes;
    if (++st == p.stages) {
      st = 0;
      phase ^= 1;
      dst = smem;
    }
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(done, 1);
    abort_flag = 0;
    fence_barrier_init();
    griddep_wait();
    // this thread made the barriers: its first stage need not wait for the others (0.1 to 0.2 us
    // of every call; the whole ring before the others start costs up to 0.6 us instead)
    load_stage();
  }
  if (warp == 1) tmem_alloc(&tmem_slot, p.tmem_cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  griddep_wait();
  griddep_trigger();

  if (warp == 0 && lane == 0) {
    while (left > 0 && mbar_wait(&empty[st], phase ^ 1, &abort_flag, p.err)) load_stage();
    if (abort_flag) {  // let copies in flight land before shared memory is released
      int dummy = 0;
      for (int i = 0; i < p.stages; ++i)
        if (armed & (0x10000u << i)) mbar_wait(&full[i], (armed >> i) & 1, &dummy);
    }
  } else if (warp == 1 && lane == 0) {
    const uint32_t idesc = idesc_bf16_f32(FT, p.row_tile);
    const uint64_t w0 = sdesc_kmajor_sw128(smem_u32(smem));
    const uint64_t stage_desc = stage_bytes >> 4, slice_desc = slice_bytes >> 4;  // linear in the address
    uint32_t acc = 0;
    uint64_t ws = w0;
    while (left > 0) {
      if (!mbar_wait(&full[st], phase, &abort_flag, p.err)) break;
      tc_fence_after();
      const int g = min(p.group, left);
      uint64_t w = ws;
      for (int j = 0; j < g; ++j, w += slice_desc) {
        const uint64_t a = w + (W_TILE >> 4);
#pragma unroll
        for (int k = 0; k < BK / 16; ++k) {
          umma_bf16_ss(tmem, w + k * 2, a + k * 2, idesc, acc);
          acc = 1u;
        }
      }
      umma_commit(&empty[st]);
      left -= g;
      ws += stage_desc;
      if (++st == p.stages) {
        st = 0;
        phase ^= 1;
        ws = w0;
      }
    }
    umma_commit(done);  // every MMA issued: the ring is idle once it fires
    int dummy = 0;
    mbar_wait(done, 0, &dummy);
  }
  // split: rows rank, rank + split, ... of the tile are this CTA's, 4 features per lane.  What
  // the first of them need beside the products is fetched while the products are made.
  constexpr int kRows = 2;
  const int rows = min(p.row_tile, p.M - r0);
  const int f4 = f0 + lane * 4;
  int r = rank + (warp - 2) * p.split;
  float bias[4] = {}, res[kRows][4] = {};
  auto fetch = [&](int row) {
    if (p.e.residual == nullptr) return;
#pragma unroll
    for (int i = 0; i < kRows; ++i)
      if (row + i * EPI_WARPS * p.split < rows)
        linear_residual4(p.e, r0 + row + i * EPI_WARPS * p.split, f4, p.N, res[i]);
  };
  const int lg = warp & 3, half = (warp - 2) >> 2;  // TMEM lane group; which of its two warps
  const int f1 = f0 + lg * 32 + lane;               // unsplit: the lane's one feature
  if (warp >= 2 && p.split == 1) {
    if (p.e.bias != nullptr && f1 < p.N) bias[0] = __ldg(p.e.bias + f1);
  } else if (warp >= 2) {
    if (p.e.bias != nullptr) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (f4 + j < p.N) bias[j] = __ldg(p.e.bias + f4 + j);
    }
    fetch(r);
  }
  __syncthreads();  // (the other warps wait here, not in a polling loop)
  const uint32_t t0 = tmem + ((uint32_t)(lg * 32) << 16);
  if (p.split == 1) {
    // straight from the accumulator, 8 rows of one feature per lane at a time
    if (warp >= 2 && !abort_flag) {
      tc_fence_after();
      for (int c = half * 8; c < rows; c += 16) {
        uint32_t t[8];
        __syncwarp();
        tmem_ld8(t0 + c, t);
        tmem_ld_wait();
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(t[j]) + bias[0];
        linear_act_all<8>(v, p.e.act);
        const int64_t row = r0 + c;
        if (f1 < p.N) finish_rows(p.e, row * p.e.ld_res + f1, row * p.e.ld_out + f1, min(8, rows - c), v);
      }
    }
    tc_fence_before();
    __syncthreads();
  } else {
    // the partial tile, [row][128 features] fp32, over the idle ring
    float* part = reinterpret_cast<float*>(smem);
    if (warp >= 2 && !abort_flag) {
      tc_fence_after();
      float* col = part + lg * 32 + lane;
      for (int c = half * 16; c < rows; c += 32) {
        uint32_t t[16];
        tmem_ld16(t0 + c, t);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) col[(c + j) * FT] = __uint_as_float(t[j]);
      }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();  // partial tiles of the whole cluster are visible
    if (warp >= 2 && !abort_flag) {
      // a warp adds up kRows rows at a time, all loads of the cluster in flight at once
      const uint32_t base = smem_u32(part) + lane * 16;
      const int step = EPI_WARPS * p.split;
      uint32_t peer[kMaxSplit];
#pragma unroll
      for (int s = 0; s < kMaxSplit; ++s) peer[s] = map_cluster(base, s < p.split ? s : rank);
      for (; r < rows; r += kRows * step) {
        float4 q[kRows][kMaxSplit];
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int s = 0; s < kMaxSplit; ++s)
            q[i][s] = s < p.split && r + i * step < rows ? ld_cluster_f4(peer[s] + (r + i * step) * (FT * 4))
                                                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          if (r + i * step >= rows) break;
          float v[4] = {q[i][0].x, q[i][0].y, q[i][0].z, q[i][0].w};
#pragma unroll
          for (int s = 1; s < kMaxSplit; ++s) {
            v[0] += q[i][s].x; v[1] += q[i][s].y; v[2] += q[i][s].z; v[3] += q[i][s].w;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += bias[j];
          linear_act_all<4>(v, p.e.act);
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] += res[i][j];
          linear_store<4>(p.e, r0 + r + i * step, f4, p.N, v);
        }
        fetch(r + kRows * step);
      }
    }
    __syncwarp();
    cluster_sync();  // no CTA leaves while a peer may still read its tile
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }
}

// How the few-row kernel covers a problem.
struct FewPlan {
  int row_tile, row_tiles, split, stages, group, smem;
  uint32_t tmem_cols;
};

// Whether the few-row kernel takes a problem, and how.
// One row tile (M <= 160): always.  From 256 to 152000 features by K of 64 to 10240 it is 0.98 to 7
// times as fast as the GEMM where two CTAs per SM hold all of it, and 0.92 to 1.44 times where CTAs
// follow one another (us few rows / GEMM: 1 row 256 x 10240 9 / 64, 24576 x 10240 80 / 138,
// 33000 x 4096 44 / 63, 151936 x 2560 120 / 150; 160 rows 60000 x 1504 46 / 56; the losses: 100 rows
// 60000 x 1504 42 / 39, 100000 x 136 22.6 / 21.0).
// Otherwise by expected times in us:
//   few rows   3.0 + slices per part * (0.30 + 0.0012 row_tile) * load + the finish: 0.018 a row
//              unsplit, else 0.8 + 0.04 a row and CTA on the SM (the cluster's shared memory)
//              load: 1 up to one CTA per SM, 1.2 up to 1.6 (two CTAs fill each other's gaps);
//              more are not taken (250 rows 24576 x 2560: 48 / 44, 500 rows 12000 x 2560: 50 / 40;
//              300 rows 12000 x 2560, 1.9 CTAs per SM, would gain: 25 / 36)
//   GEMM       10 + 0.34 a slice and wave of its 256-wide tiles (measured 0.26 to 0.44)
// and in both no less than the time to read w at 6.6 TB/s.  Of 24 problems measured with 170 to 500
// rows, 4000 x 4096 to 20000 x 1000, two are not given to the faster kernel and split within 10%: the
// one above and 500 rows 4000 x 4096, 23 / 27.  us few rows / GEMM at 2560 x 4096: 512 rows 20 / 27;
// 9728 x 2560: 512 rows 57 / 35; 3840 x 10240: 266 rows 48 / 56; 7680 x 10240: 256 rows 51 / 78.
// Parts: 1 x 256 x 10240 45 us with one, 9 with eight; clusters of 5 to 7 pack badly into the GPCs
// (6144 x 2560, 1 row: 6 parts 16.6 us, 3 parts 9.9).
bool plan_few(int64_t M, int64_t N, int64_t K, FewPlan* f) {
  const double sms = num_sms(), slices = (double)((K + BK - 1) / BK), read_w = 2.0 * N * K / 6.6e6;
  const double wide_tiles = (double)(M > 256 ? (M + 255) / 256 : (M + 127) / 128) * ((N + 255) / 256);
  const double gemm = 10.0 + std::max(0.34 * slices * std::ceil(wide_tiles / (M > 256 ? sms / 2 : sms)), read_w);
  const int64_t row_tiles = M <= kMaxRowTile ? 1 : (M + 127) / 128;
  const double tiles = (double)((N + FT - 1) / FT) * row_tiles;
  f->row_tiles = (int)row_tiles;
  f->row_tile = (int)(((M + row_tiles - 1) / row_tiles + 15) / 16 * 16);
  f->split = 0;
  double best = row_tiles == 1 ? INFINITY : gemm;
  const int sizes[] = {1, 2, 3, 4, 8};
  for (const int s : sizes) {
    const double ctas = tiles * s / sms;  // per SM
    if ((ctas > 1.63 && (s > 1 || row_tiles > 1)) || (s > 1 && slices < 2 * s)) break;
    const double stream =
        std::max(std::ceil(slices / s) * (0.30 + 0.0012 * f->row_tile) * (ctas <= 1 ? 1.0 : 1.2), read_w);
    const double finish = s == 1 ? 0.018 * f->row_tile : 0.8 + 0.04 * f->row_tile * std::max(1.0, ctas);
    if (3.0 + stream + finish < best) {
      best = 3.0 + stream + finish;
      f->split = s;
    }
  }
  if (f->split == 0) return false;
  // Two slices per stage while the rows are few (fewer waits: 1 row 7.9 -> 7.5 us); one when
  // the row tile takes its share of the ring.
  f->group = f->row_tile <= 32 ? 2 : 1;
  const int stage = f->group * (W_TILE + f->row_tile * BK * 2);
  f->stages = std::min(kRing / stage, kMaxStages);
  f->smem = 1024 + std::max(f->stages * stage, f->split > 1 ? f->row_tile * FT * 4 : 0);
  f->tmem_cols = 32;
  while (f->tmem_cols < (uint32_t)f->row_tile) f->tmem_cols *= 2;
  return true;
}

zdit_status launch_few(const zdit_linear_args& a, const LinearEpi& e, const FewPlan& f, cudaStream_t s) {
  CUtensorMap tw, ta;
  if (!make_tmap_bf16_2d(&tw, a.w, a.N, a.K, a.ldw, FT, BK) ||
      !make_tmap_bf16_2d(&ta, a.a, a.M, a.K, a.lda, f.row_tile, BK))
    return ZDIT_ERR_CUDA;
  // the opt-in is state of the context that all host threads share: always the largest, so that
  // no call takes away what another one is about to launch with
  const cudaError_t opt_in =
      cudaFuncSetAttribute(linear_few_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (opt_in != cudaSuccess) return launch_status(opt_in);
  FewParams p;
  p.M = (int)a.M; p.N = (int)a.N; p.row_tile = f.row_tile; p.slices = (int)((a.K + BK - 1) / BK); p.split = f.split;
  p.stages = f.stages; p.group = f.group; p.tmem_cols = f.tmem_cols; p.e = e; p.err = device_error_ptr();
  const double rw = (e.out_f32 ? 4.0 : 2.0) + (e.residual ? (e.res_f32 ? 4.0 : 2.0) : 0.0);
  ProfScope ps(PROF_GEMM_OTHER, 2.0 * a.M * a.N * (double)a.K,
               2.0 * ((double)a.M * a.K + (double)a.N * a.K) + rw * a.M * a.N, s);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.N + FT - 1) / FT * f.split), (unsigned)f.row_tiles);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = f.smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = f.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return launch_status(cudaLaunchKernelEx(&cfg, linear_few_kernel, tw, ta, p));
}

}  // namespace

}  // namespace zdit

using namespace zdit;

extern "C" {

ZDIT_API zdit_status zdit_linear(const zdit_linear_args* args, void* stream) {
  if (args == nullptr || args->M < 0 || args->N < 0 || args->K < 0) return ZDIT_ERR_INVALID_ARG;
  // the stride of a single row leads nowhere: any value is allowed, and one that keeps the
  // tensor maps and the wide stores valid takes its place
  const int64_t most = int64_t(1) << 30;
  zdit_linear_args one = *args;
  if (one.M == 1) {
    one.lda = (std::min(one.K, most) + 7) / 8 * 8;
    one.ld_out = one.ld_residual = (std::min(one.N, most) + 7) / 8 * 8;
  }
  if (one.N == 1) one.ldw = (std::min(one.K, most) + 7) / 8 * 8;
  const zdit_linear_args* a = &one;
  if (a->act < ZDIT_ACT_NONE || a->act > ZDIT_ACT_GELU || a->out_dtype < 0 || a->out_dtype > 1 ||
      (a->residual && (a->residual_dtype < 0 || a->residual_dtype > 1)))
    return ZDIT_ERR_INVALID_ARG;
  if (a->N < 1 || a->K < 1 || a->M > most || a->N > most || a->K > most || a->lda > most || a->ldw > most)
    return ZDIT_ERR_SHAPE;
  if (a->M == 0) return ZDIT_OK;
  if (!a->a || !a->w || !a->out) return ZDIT_ERR_INVALID_ARG;
  if (a->lda < a->K || a->ldw < a->K || a->ld_out < a->N || (a->residual && a->ld_residual < a->N))
    return ZDIT_ERR_SHAPE;
  const uintptr_t oa = reinterpret_cast<uintptr_t>(a->out), ra = reinterpret_cast<uintptr_t>(a->residual);
  const int oe = a->out_dtype == ZDIT_T_F32 ? 4 : 2, re = a->residual_dtype == ZDIT_T_F32 ? 4 : 2;
  if (((reinterpret_cast<uintptr_t>(a->a) | reinterpret_cast<uintptr_t>(a->w)) & 15) || a->lda % 8 || a->ldw % 8)
    return ZDIT_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(a->bias) & 3) || oa % oe || (a->residual && ra % re)) return ZDIT_ERR_ALIGNMENT;
  if (a->residual == a->out && (oe != re || a->ld_residual != a->ld_out)) return ZDIT_ERR_INVALID_ARG;
  if (a->a == a->out || a->w == a->out) return ZDIT_ERR_INVALID_ARG;
  if (!device_ok()) return ZDIT_ERR_UNSUPPORTED;
  LinearEpi e{};
  e.bias = a->bias; e.residual = a->residual; e.out = a->out; e.ld_res = a->ld_residual; e.ld_out = a->ld_out;
  e.act = a->act; e.res_f32 = re == 4; e.out_f32 = oe == 4;
  e.vec = oa % 16 == 0 && a->ld_out * oe % 16 == 0 &&
          (!a->residual || (ra % 16 == 0 && a->ld_residual * re % 16 == 0));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  FewPlan f;
  if (plan_few(a->M, a->N, a->K, &f)) return launch_few(*a, e, f, s);
  GemmArgs g{};
  g.A = a->a; g.B = a->w; g.M = (int)a->M; g.N = (int)a->N; g.K = (int)a->K; g.lda = (int)a->lda; g.ldb = (int)a->ldw;
  g.epi = EPI_LINEAR; g.out = a->out; g.lin = e;
  return launch_gemm(g, s);
}

}  // extern "C"
