// zdit_linear: out = residual + act(a . w^T + bias).
#include <cmath>

#include "internal.h"
#include "linear_epi.cuh"
#include "ptx.cuh"

using namespace zdit;

extern "C" {

ZDIT_API zdit_status zdit_linear(const zdit_linear_args* a, void* stream) {
  if (a == nullptr || a->M < 0 || a->N < 0 || a->K < 0) return ZDIT_ERR_INVALID_ARG;
  if (a->act < ZDIT_ACT_NONE || a->act > ZDIT_ACT_GELU || a->out_dtype < 0 || a->out_dtype > 1 ||
      (a->residual && (a->residual_dtype < 0 || a->residual_dtype > 1)))
    return ZDIT_ERR_INVALID_ARG;
  const int64_t most = int64_t(1) << 30;
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
  if (!device_ok()) return ZDIT_ERR_UNSUPPORTED;
  GemmArgs g{};
  g.A = a->a; g.B = a->w; g.M = (int)a->M; g.N = (int)a->N; g.K = (int)a->K; g.lda = (int)a->lda; g.ldb = (int)a->ldw;
  g.epi = EPI_LINEAR; g.out = a->out;
  g.lin.bias = a->bias; g.lin.residual = a->residual; g.lin.out = a->out; g.lin.ld_res = a->ld_residual;
  g.lin.ld_out = a->ld_out; g.lin.act = a->act; g.lin.res_f32 = re == 4; g.lin.out_f32 = oe == 4;
  g.lin.vec = oa % 16 == 0 && a->ld_out * oe % 16 == 0 &&
              (!a->residual || (ra % 16 == 0 && a->ld_residual * re % 16 == 0));
  return launch_gemm(g, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
