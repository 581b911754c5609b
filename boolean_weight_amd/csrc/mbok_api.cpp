// C ABI of the MBOK library: argument validation and dispatch.  Every check
// runs on the host before anything is enqueued; nothing here allocates,
// synchronises or keeps state.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "../../include/mbok.h"
#include "mbok_adamw.h"
#include "mbok_launch.h"
#include "mbok_linear.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Checks a descriptor that may have been filled by hand.
int check_desc(const mbok_desc* d) {
  if (!d) return MBOK_ERR_INVALID_ARG;
  if (d->m < 1 || d->m > (1 << 24)) return MBOK_ERR_SHAPE;
  if (d->n < MBOK_GROUP || d->n > (1 << 20) || d->n % MBOK_GROUP) return MBOK_ERR_SHAPE;
  if (d->K < 1 || d->K > MBOK_MAX_K) return MBOK_ERR_UNSUPPORTED;
  if (d->group != MBOK_GROUP) return MBOK_ERR_UNSUPPORTED;
  if (d->alpha_dtype != MBOK_F32 && d->alpha_dtype != MBOK_F16) return MBOK_ERR_DTYPE;
  if (d->layout != MBOK_LAYOUT_L64) return MBOK_ERR_UNSUPPORTED;
  return MBOK_OK;
}

// largest leading dimension of the fine-tuning calls: T rows of it stay far
// inside 63-bit element offsets
constexpr int64_t kMaxLd = int64_t(1) << 32;

size_t alpha_size(int32_t dt) { return dt == MBOK_F16 ? 2 : 4; }

bool float_dtype(int32_t t) { return t == MBOK_F32 || t == MBOK_F16 || t == MBOK_BF16; }

}  // namespace

extern "C" {

int mbok_desc_init(mbok_desc* d, int32_t m, int32_t n, int32_t K, int32_t alpha_dtype) {
  if (!d) return MBOK_ERR_INVALID_ARG;
  mbok_desc t;
  t.m = m;
  t.n = n;
  t.K = K;
  t.group = MBOK_GROUP;
  t.alpha_dtype = alpha_dtype;
  t.layout = MBOK_LAYOUT_L64;
  const int st = check_desc(&t);
  if (st != MBOK_OK) return st;
  *d = t;
  return MBOK_OK;
}

size_t mbok_packed_bytes(const mbok_desc* d) {
  if (check_desc(d) != MBOK_OK) return 0;
  const size_t m_pad = ((size_t)d->m + MBOK_ROW_BLOCK - 1) / MBOK_ROW_BLOCK * MBOK_ROW_BLOCK;
  const size_t G = (size_t)d->n / MBOK_GROUP;
  return (size_t)d->K * m_pad * (size_t)d->n / 8 +
         (size_t)d->K * m_pad * G * alpha_size(d->alpha_dtype);
}

size_t mbok_alpha_bytes(const mbok_desc* d) {
  if (check_desc(d) != MBOK_OK) return 0;
  return (size_t)d->K * (size_t)d->m * ((size_t)d->n / MBOK_GROUP) * alpha_size(d->alpha_dtype);
}

int mbok_residual_binarize(const mbok_desc* d, const float* W, int64_t ldw, int8_t* signs,
                           void* alpha, int32_t* flag, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!W || !signs || !alpha) return MBOK_ERR_INVALID_ARG;
  if (ldw < d->n) return MBOK_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(signs, 16) || !aligned(alpha, 16) || (ldw % 4) != 0)
    return MBOK_ERR_ALIGN;
  if (flag && !aligned(flag, 4)) return MBOK_ERR_ALIGN;
  return mbok::launch_residual_binarize(d, W, ldw, signs, alpha, flag, (hipStream_t)stream);
}

int mbok_residual_energy(const mbok_desc* d, const float* W, int64_t ldw, double* row_energy,
                         double* layer_energy, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!W || !row_energy || !layer_energy) return MBOK_ERR_INVALID_ARG;
  if (ldw < d->n) return MBOK_ERR_INVALID_ARG;
  if (!aligned(W, 16) || (ldw % 4) != 0 || !aligned(row_energy, 8) || !aligned(layer_energy, 8))
    return MBOK_ERR_ALIGN;
  return mbok::launch_residual_energy(d, W, ldw, row_energy, layer_energy, (hipStream_t)stream);
}

int mbok_allocate_kernels(int32_t L, const int64_t* sizes, const double* errors, int32_t kmax,
                          int64_t budget, int32_t* K_out) {
  if (!sizes || !errors || !K_out || L < 1 || kmax < 1 || kmax > MBOK_MAX_K || budget < 0)
    return MBOK_ERR_INVALID_ARG;
  for (int32_t l = 0; l < L; ++l) {
    if (sizes[l] < 1 || sizes[l] > (int64_t(1) << 44)) return MBOK_ERR_INVALID_ARG;
    for (int32_t k = 0; k < kmax; ++k) {
      const double e = errors[(size_t)l * kmax + k];
      if (!std::isfinite(e) || e < 0.0) return MBOK_ERR_INVALID_ARG;
    }
  }
  return mbok::allocate_kernels(L, sizes, errors, kmax, budget, K_out);
}

size_t mbok_svid_workspace_bytes(const mbok_desc* d) {
  if (check_desc(d) != MBOK_OK) return 0;
  return mbok::svid_workspace_bytes(d);
}

int mbok_svid_decompose(const mbok_desc* d, const float* W, int64_t ldw, int8_t* signs,
                        void* s_out, void* s_in, int32_t iters, void* workspace, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!W || !signs || !s_out || !s_in || !workspace) return MBOK_ERR_INVALID_ARG;
  if (ldw < d->n || iters < 1 || iters > MBOK_MAX_SVID_ITERS) return MBOK_ERR_INVALID_ARG;
  if (!aligned(W, 16) || (ldw % 4) != 0 || !aligned(signs, 16) || !aligned(s_out, 4) ||
      !aligned(s_in, 4) || !aligned(workspace, 256))
    return MBOK_ERR_ALIGN;
  return mbok::launch_svid_decompose(d, W, ldw, signs, s_out, s_in, iters, workspace,
                                     (hipStream_t)stream);
}

int mbok_svid_pack(const mbok_desc* d, const int8_t* signs, const void* s_out, void* packed,
                   void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!signs || !s_out || !packed) return MBOK_ERR_INVALID_ARG;
  if (!aligned(signs, 16) || !aligned(s_out, 4) || !aligned(packed, 16)) return MBOK_ERR_ALIGN;
  return mbok::launch_svid_pack(d, signs, s_out, packed, (hipStream_t)stream);
}

size_t mbok_svid_gemv_workspace_bytes(const mbok_desc* d) {
  (void)d;
  return 0;
}

int mbok_svid_gemv(const mbok_desc* d, const void* packed, const void* s_in, const void* x,
                   int32_t x_dtype, float* y, void* workspace, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !s_in || !x || !y) return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_BF16 && x_dtype != MBOK_F32) return MBOK_ERR_DTYPE;
  if (!aligned(packed, 16) || !aligned(s_in, 16) || !aligned(x, 16) || !aligned(y, 4) ||
      (workspace && !aligned(workspace, 256)))
    return MBOK_ERR_ALIGN;
  // the fp4 x fp8 form by default; MBOK_SVID_VARIANT=skinny selects the bf16
  // +-1 form (measurements)
  const char* v = getenv("MBOK_SVID_VARIANT");
  if (v && strcmp(v, "skinny") == 0)
    return mbok::launch_svid_skinny(d, packed, x, x_dtype, s_in, y, (hipStream_t)stream);
  return mbok::launch_svid_f4(d, packed, x, x_dtype, s_in, y, (hipStream_t)stream);
}

int mbok_refit(const mbok_desc* d, const float* W, int64_t ldw, int8_t* signs, void* alpha,
               int32_t rounds, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!W || !signs || !alpha) return MBOK_ERR_INVALID_ARG;
  if (ldw < d->n) return MBOK_ERR_INVALID_ARG;
  if (rounds < 0 || rounds > MBOK_MAX_REFIT_ROUNDS || rounds > mbok::refit_max_rounds())
    return MBOK_ERR_INVALID_ARG;
  if (!aligned(W, 16) || !aligned(signs, 16) || !aligned(alpha, 16) || (ldw % 4) != 0)
    return MBOK_ERR_ALIGN;
  return mbok::launch_refit(d, W, ldw, signs, alpha, rounds, (hipStream_t)stream);
}

int mbok_pack(const mbok_desc* d, const int8_t* signs, const void* alpha, void* packed,
              void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!signs || !alpha || !packed) return MBOK_ERR_INVALID_ARG;
  if (!aligned(signs, 16) || !aligned(alpha, 16) || !aligned(packed, 16)) return MBOK_ERR_ALIGN;
  return mbok::launch_pack(d, signs, alpha, packed, (hipStream_t)stream);
}

size_t mbok_gemv_workspace_bytes(const mbok_desc* d) {
  if (check_desc(d) != MBOK_OK) return 0;
  return mbok::gemv_workspace_bytes(d);
}

int mbok_gemv(const mbok_desc* d, const void* packed, const void* x, int32_t x_dtype, float* y,
              void* workspace, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !x || !y) return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_BF16 && x_dtype != MBOK_F32) return MBOK_ERR_DTYPE;
  if (!aligned(packed, 16) || !aligned(x, 16) || !aligned(y, 4)) return MBOK_ERR_ALIGN;
  if (workspace && !aligned(workspace, 256)) return MBOK_ERR_ALIGN;
  return mbok::launch_gemv(d, packed, x, x_dtype, y, workspace, (hipStream_t)stream);
}

size_t mbok_gemvt_workspace_bytes(const mbok_desc* d) {
  if (check_desc(d) != MBOK_OK) return 0;
  return mbok::gemvt_workspace_bytes(d);
}

int mbok_gemvt(const mbok_desc* d, const void* packed, const void* g, int32_t g_dtype, float* dx,
               void* workspace, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !g || !dx) return MBOK_ERR_INVALID_ARG;
  if (g_dtype != MBOK_BF16 && g_dtype != MBOK_F32) return MBOK_ERR_DTYPE;
  if (!aligned(packed, 16) || !aligned(g, g_dtype == MBOK_BF16 ? 2 : 4) || !aligned(dx, 4))
    return MBOK_ERR_ALIGN;
  if (workspace && !aligned(workspace, 256)) return MBOK_ERR_ALIGN;
  return mbok::launch_gemvt(d, packed, g, g_dtype, dx, workspace, (hipStream_t)stream);
}

size_t mbok_gemvt_scratch_bytes(void) { return mbok::gemvt_scratch_bytes(); }

int mbok_gemvt_noalloc(const mbok_desc* d, const void* packed, const void* g, int32_t g_dtype,
                       float* dx, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !g || !dx) return MBOK_ERR_INVALID_ARG;
  if (g_dtype != MBOK_BF16 && g_dtype != MBOK_F32) return MBOK_ERR_DTYPE;
  if (!aligned(packed, 16) || !aligned(g, g_dtype == MBOK_BF16 ? 2 : 4) || !aligned(dx, 4))
    return MBOK_ERR_ALIGN;
  return mbok::launch_gemvt_noalloc(d, packed, g, g_dtype, dx, (hipStream_t)stream);
}

static int gemm_checked(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                        int64_t T, int64_t ldx, float* Y, int64_t ldy, int passes,
                        void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !X || !Y) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_T) return MBOK_ERR_SHAPE;
  if (ldx < d->n || ldy < d->m) return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_BF16) return MBOK_ERR_DTYPE;
  if (!aligned(packed, 16) || !aligned(X, 16) || (ldx % 8) != 0 || !aligned(Y, 4))
    return MBOK_ERR_ALIGN;
  return mbok::launch_gemm(d, packed, X, T, ldx, Y, ldy, passes, (hipStream_t)stream);
}

int mbok_gemm(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype, int64_t T,
              int64_t ldx, float* Y, int64_t ldy, void* stream) {
  return gemm_checked(d, packed, X, x_dtype, T, ldx, Y, ldy, 1, stream);
}

int mbok_gemm_precise(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                      int64_t T, int64_t ldx, float* Y, int64_t ldy, void* stream) {
  return gemm_checked(d, packed, X, x_dtype, T, ldx, Y, ldy, 2, stream);
}

static int gemmt_checked(const mbok_desc* d, const void* packed, const void* dY, int64_t T,
                         int64_t lddy, void* dX, int64_t lddx, void* workspace, int passes,
                         void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !dY || !dX) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_T) return MBOK_ERR_SHAPE;
  if (lddy < d->m || lddx < d->n || lddy > kMaxLd || lddx > kMaxLd) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(dY, 2) || !aligned(dX, 16) || (lddx % 8) != 0 ||
      (workspace && !aligned(workspace, 256)))
    return MBOK_ERR_ALIGN;
  return mbok::launch_gemmt(d, packed, dY, T, lddy, dX, lddx, workspace, passes,
                            (hipStream_t)stream);
}

int mbok_gemmt(const mbok_desc* d, const void* packed, const void* dY, int64_t T, int64_t lddy,
               void* dX, int64_t lddx, void* workspace, void* stream) {
  return gemmt_checked(d, packed, dY, T, lddy, dX, lddx, workspace, 1, stream);
}

int mbok_gemmt_precise(const mbok_desc* d, const void* packed, const void* dY, int64_t T,
                       int64_t lddy, void* dX, int64_t lddx, void* workspace, void* stream) {
  return gemmt_checked(d, packed, dY, T, lddy, dX, lddx, workspace, 2, stream);
}

size_t mbok_gemmt_workspace_bytes(const mbok_desc* d, int64_t T) {
  if (check_desc(d) != MBOK_OK || T < 1 || T > MBOK_MAX_T) return 0;
  return mbok::gemmt_workspace_bytes(d, T);
}

int mbok_scale_grad(const mbok_desc* d, const void* packed, const void* dY, int64_t T,
                    int64_t lddy, const void* X, int64_t ldx, float* dalpha, int32_t accumulate,
                    void* workspace, void* stream) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !dY || !X || !dalpha) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_T) return MBOK_ERR_SHAPE;
  if (lddy < d->m || ldx < d->n || lddy > kMaxLd || ldx > kMaxLd) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(dY, 2) || !aligned(X, 16) || (ldx % 8) != 0 ||
      !aligned(dalpha, 4) || (workspace && !aligned(workspace, 256)))
    return MBOK_ERR_ALIGN;
  return mbok::launch_scale_grad(d, packed, dY, T, lddy, X, ldx, dalpha, accumulate != 0,
                                 workspace, (hipStream_t)stream);
}

size_t mbok_scale_grad_workspace_bytes(const mbok_desc* d, int64_t T) {
  if (check_desc(d) != MBOK_OK || T < 1 || T > MBOK_MAX_T) return 0;
  return mbok::scale_grad_workspace_bytes(d, T);
}

int mbok_gated_stack(const mbok_desc* d, mbok_desc* stacked) {
  int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!stacked) return MBOK_ERR_INVALID_ARG;
  if (d->m > (1 << 23)) return MBOK_ERR_SHAPE;
  *stacked = mbok::gated_stacked(d);
  return MBOK_OK;
}

int mbok_gated_pack(const mbok_desc* d, const int8_t* signs_gate, const void* alpha_gate,
                    const int8_t* signs_up, const void* alpha_up, void* packed, void* stream) {
  mbok_desc stacked;
  int st = mbok_gated_stack(d, &stacked);
  if (st != MBOK_OK) return st;
  if (!signs_gate || !alpha_gate || !signs_up || !alpha_up || !packed)
    return MBOK_ERR_INVALID_ARG;
  if (!aligned(signs_gate, 16) || !aligned(alpha_gate, 16) || !aligned(signs_up, 16) ||
      !aligned(alpha_up, 16) || !aligned(packed, 16))
    return MBOK_ERR_ALIGN;
  return mbok::launch_gated_pack(d, signs_gate, alpha_gate, signs_up, alpha_up, packed,
                                 (hipStream_t)stream);
}

static int gated_checked(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                         int64_t T, int64_t ldx, int32_t act, void* H, int64_t ldh, void* pre,
                         int64_t ldpre, int passes, void* stream) {
  mbok_desc stacked;
  int st = mbok_gated_stack(d, &stacked);
  if (st != MBOK_OK) return st;
  if (!packed || !X || !H) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_T) return MBOK_ERR_SHAPE;
  if (act != MBOK_ACT_SILU && act != MBOK_ACT_GELU) return MBOK_ERR_INVALID_ARG;
  if (ldx < d->n || ldh < d->m || ldx > kMaxLd || ldh > kMaxLd) return MBOK_ERR_INVALID_ARG;
  if (pre && (ldpre < stacked.m || ldpre > kMaxLd)) return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_BF16) return MBOK_ERR_DTYPE;
  if (!aligned(packed, 16) || !aligned(X, 16) || (ldx % 8) != 0 || !aligned(H, 2) ||
      (pre && (!aligned(pre, 16) || (ldpre % 8) != 0)))
    return MBOK_ERR_ALIGN;
  return mbok::launch_gated(d, packed, X, T, ldx, act, H, ldh, pre, ldpre, passes,
                            (hipStream_t)stream);
}

int mbok_gated(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype, int64_t T,
               int64_t ldx, int32_t act, void* H, int64_t ldh, void* pre, int64_t ldpre,
               void* stream) {
  return gated_checked(d, packed, X, x_dtype, T, ldx, act, H, ldh, pre, ldpre, 1, stream);
}

int mbok_gated_precise(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                       int64_t T, int64_t ldx, int32_t act, void* H, int64_t ldh, void* pre,
                       int64_t ldpre, void* stream) {
  return gated_checked(d, packed, X, x_dtype, T, ldx, act, H, ldh, pre, ldpre, 2, stream);
}

static int gated_backward_checked(const mbok_desc* d, const void* packed, const void* pre,
                                  int64_t ldpre, const void* dH, int64_t lddh, int64_t T,
                                  int32_t act, void* dpre, int64_t lddpre, void* dX, int64_t lddx,
                                  void* workspace, int passes, void* stream) {
  mbok_desc stacked;
  int st = mbok_gated_stack(d, &stacked);
  if (st != MBOK_OK) return st;
  if (!packed || !pre || !dH || !dpre) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_T) return MBOK_ERR_SHAPE;
  if (act != MBOK_ACT_SILU && act != MBOK_ACT_GELU) return MBOK_ERR_INVALID_ARG;
  if (ldpre < stacked.m || lddpre < stacked.m || lddh < d->m || ldpre > kMaxLd ||
      lddpre > kMaxLd || lddh > kMaxLd)
    return MBOK_ERR_INVALID_ARG;
  if (dX && (lddx < d->n || lddx > kMaxLd)) return MBOK_ERR_INVALID_ARG;
  if (dpre == pre && lddpre != ldpre) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(pre, 16) || !aligned(dpre, 16) || (ldpre % 8) != 0 ||
      (lddpre % 8) != 0 || !aligned(dH, 2) ||
      (dX && (!aligned(dX, 16) || (lddx % 8) != 0)) || (workspace && !aligned(workspace, 256)))
    return MBOK_ERR_ALIGN;
  return mbok::launch_gated_backward(d, packed, pre, ldpre, dH, lddh, T, act, dpre, lddpre, dX,
                                     lddx, workspace, passes, (hipStream_t)stream);
}

int mbok_gated_backward(const mbok_desc* d, const void* packed, const void* pre, int64_t ldpre,
                        const void* dH, int64_t lddh, int64_t T, int32_t act, void* dpre,
                        int64_t lddpre, void* dX, int64_t lddx, void* workspace, void* stream) {
  return gated_backward_checked(d, packed, pre, ldpre, dH, lddh, T, act, dpre, lddpre, dX, lddx,
                                workspace, 1, stream);
}

int mbok_gated_backward_precise(const mbok_desc* d, const void* packed, const void* pre,
                                int64_t ldpre, const void* dH, int64_t lddh, int64_t T,
                                int32_t act, void* dpre, int64_t lddpre, void* dX, int64_t lddx,
                                void* workspace, void* stream) {
  return gated_backward_checked(d, packed, pre, ldpre, dH, lddh, T, act, dpre, lddpre, dX, lddx,
                                workspace, 2, stream);
}

static int check_distill(const mbok_distill_desc* d) {
  // below 2^-126 the kernels' fp32 factor log2(e) / tau is not finite
  if (!d || !std::isnormal(d->temperature) || !(d->temperature > 0.f))
    return MBOK_ERR_INVALID_ARG;
  if (d->vocab < 1 || d->vocab > MBOK_MAX_VOCAB || d->top < 1 || d->top > MBOK_MAX_TOP)
    return MBOK_ERR_SHAPE;
  return MBOK_OK;
}

int mbok_distill_desc_init(mbok_distill_desc* d, int32_t vocab, int32_t top, float temperature) {
  if (!d) return MBOK_ERR_INVALID_ARG;
  const mbok_distill_desc t = {vocab, top, temperature};
  const int st = check_distill(&t);
  if (st != MBOK_OK) return st;
  *d = t;
  return MBOK_OK;
}

// what mbok_distill and mbok_distill_backward check alike
static int check_distill_args(const mbok_distill_desc* d, const mbok::DistillArgs& a) {
  const int st = check_distill(d);
  if (st != MBOK_OK) return st;
  if (!a.Z || !a.t_logits || !a.t_index) return MBOK_ERR_INVALID_ARG;
  if (a.T < 1 || a.T > MBOK_MAX_DISTILL_ROWS) return MBOK_ERR_SHAPE;
  if (a.ldz < d->vocab || a.ldt < d->top || a.ldz > kMaxLd || a.ldt > kMaxLd)
    return MBOK_ERR_INVALID_ARG;
  if (a.dZ && (a.lddz < d->vocab || a.lddz > kMaxLd)) return MBOK_ERR_INVALID_ARG;
  if (!float_dtype(a.z_dtype) || !float_dtype(a.t_dtype)) return MBOK_ERR_DTYPE;
  if (a.dZ && a.dz_dtype != a.z_dtype && a.dz_dtype != MBOK_BF16) return MBOK_ERR_DTYPE;
  if (a.dZ == a.Z && (a.dz_dtype != a.z_dtype || a.lddz != a.ldz)) return MBOK_ERR_INVALID_ARG;
  auto size = [](int32_t t) { return t == MBOK_F32 ? 4 : 2; };
  if (!aligned(a.Z, size(a.z_dtype)) || !aligned(a.t_logits, size(a.t_dtype)) ||
      !aligned(a.t_index, 4) || !aligned(a.t_lse, 4) || !aligned(a.weight, 4) ||
      (a.dZ && !aligned(a.dZ, size(a.dz_dtype))))
    return MBOK_ERR_ALIGN;
  return MBOK_OK;
}

int mbok_distill(const mbok_distill_desc* d, const void* Z, int32_t z_dtype, int64_t T,
                 int64_t ldz, const void* t_logits, int32_t t_dtype, const int32_t* t_index,
                 int64_t ldt, const float* t_lse, const float* weight, float* loss, float* stats,
                 void* dZ, int32_t dz_dtype, int64_t lddz, void* stream) {
  const mbok::DistillArgs a = {Z, z_dtype, T, ldz, t_logits, t_dtype, t_index, ldt,
                               t_lse, weight, dZ, dz_dtype, lddz};
  const int st = check_distill_args(d, a);
  if (st != MBOK_OK) return st;
  if (!loss) return MBOK_ERR_INVALID_ARG;
  if (!aligned(loss, 4) || (stats && !aligned(stats, 16))) return MBOK_ERR_ALIGN;
  return mbok::launch_distill(d, a, loss, stats, (hipStream_t)stream);
}

int mbok_distill_backward(const mbok_distill_desc* d, const void* Z, int32_t z_dtype, int64_t T,
                          int64_t ldz, const void* t_logits, int32_t t_dtype,
                          const int32_t* t_index, int64_t ldt, const float* t_lse,
                          const float* weight, const float* stats, const float* dloss, void* dZ,
                          int32_t dz_dtype, int64_t lddz, void* stream) {
  const mbok::DistillArgs a = {Z, z_dtype, T, ldz, t_logits, t_dtype, t_index, ldt,
                               t_lse, weight, dZ, dz_dtype, lddz};
  const int st = check_distill_args(d, a);
  if (st != MBOK_OK) return st;
  if (!stats || !dloss || !dZ) return MBOK_ERR_INVALID_ARG;
  if (!aligned(stats, 16) || !aligned(dloss, 4)) return MBOK_ERR_ALIGN;
  return mbok::launch_distill_backward(d, a, stats, dloss, (hipStream_t)stream);
}

static int linear_checked(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                          int64_t T, int64_t ldx, const void* bias, int32_t bias_dtype,
                          int32_t act, const void* residual, int64_t ldr, void* Y,
                          int32_t y_dtype, int64_t ldy, void* pre, int64_t ldpre, int passes,
                          void* stream) {
  const int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !X || !Y) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_T) return MBOK_ERR_SHAPE;
  if (act != MBOK_ACT_SILU && act != MBOK_ACT_GELU && act != MBOK_ACT_NONE)
    return MBOK_ERR_INVALID_ARG;
  if (ldx < d->n || ldy < d->m || ldx > kMaxLd || ldy > kMaxLd) return MBOK_ERR_INVALID_ARG;
  if (residual && (ldr < d->m || ldr > kMaxLd || (residual == Y && ldr != ldy)))
    return MBOK_ERR_INVALID_ARG;
  if (pre && (ldpre < d->m || ldpre > kMaxLd)) return MBOK_ERR_INVALID_ARG;
  if (x_dtype != MBOK_BF16 || (y_dtype != MBOK_BF16 && y_dtype != MBOK_F32) ||
      (bias && !float_dtype(bias_dtype)))
    return MBOK_ERR_DTYPE;
  const uintptr_t ys = y_dtype == MBOK_F32 ? 4 : 2;
  if (!aligned(packed, 16) || !aligned(X, 16) || (ldx % 8) != 0 || !aligned(Y, ys) ||
      !aligned(residual, ys) || !aligned(bias, bias_dtype == MBOK_F32 ? 4 : 2) ||
      !aligned(pre, 2))
    return MBOK_ERR_ALIGN;
  const mbok::LinearOut out = {Y, ldy, residual, ldr, reinterpret_cast<uint16_t*>(pre), ldpre,
                               bias, d->m, act, y_dtype == MBOK_F32, bias_dtype};
  return mbok::launch_linear(d, packed, X, T, ldx, out, passes, (hipStream_t)stream);
}

int mbok_linear(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                int64_t T, int64_t ldx, const void* bias, int32_t bias_dtype, int32_t act,
                const void* residual, int64_t ldr, void* Y, int32_t y_dtype, int64_t ldy,
                void* pre, int64_t ldpre, void* stream) {
  return linear_checked(d, packed, X, x_dtype, T, ldx, bias, bias_dtype, act, residual, ldr, Y,
                        y_dtype, ldy, pre, ldpre, 1, stream);
}

int mbok_linear_precise(const mbok_desc* d, const void* packed, const void* X, int32_t x_dtype,
                        int64_t T, int64_t ldx, const void* bias, int32_t bias_dtype,
                        int32_t act, const void* residual, int64_t ldr, void* Y,
                        int32_t y_dtype, int64_t ldy, void* pre, int64_t ldpre, void* stream) {
  return linear_checked(d, packed, X, x_dtype, T, ldx, bias, bias_dtype, act, residual, ldr, Y,
                        y_dtype, ldy, pre, ldpre, 2, stream);
}

static int linear_backward_checked(const mbok_desc* d, const void* packed, const void* pre,
                                   int64_t ldpre, const void* dY, int64_t lddy, int64_t T,
                                   int32_t act, void* dpre, int64_t lddpre, float* dbias,
                                   int32_t accumulate, void* dX, int64_t lddx, void* workspace,
                                   int passes, void* stream) {
  const int st = check_desc(d);
  if (st != MBOK_OK) return st;
  if (!packed || !dY) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_T) return MBOK_ERR_SHAPE;
  if (lddy < d->m || lddy > kMaxLd) return MBOK_ERR_INVALID_ARG;
  if (act == MBOK_ACT_NONE) {
    if (pre || dpre || (!dbias && !dX)) return MBOK_ERR_INVALID_ARG;
  } else if (act == MBOK_ACT_SILU || act == MBOK_ACT_GELU) {
    if (!pre || !dpre || ldpre < d->m || lddpre < d->m || ldpre > kMaxLd || lddpre > kMaxLd ||
        (dpre == pre && lddpre != ldpre) || (dpre == dY && lddpre != lddy))
      return MBOK_ERR_INVALID_ARG;
  } else {
    return MBOK_ERR_INVALID_ARG;
  }
  if (dX && (lddx < d->n || lddx > kMaxLd)) return MBOK_ERR_INVALID_ARG;
  if (!aligned(packed, 16) || !aligned(dY, 2) || !aligned(pre, 2) || !aligned(dpre, 2) ||
      !aligned(dbias, 4) || (dX && (!aligned(dX, 16) || (lddx % 8) != 0)) ||
      !aligned(workspace, 256))
    return MBOK_ERR_ALIGN;
  const mbok::LinearGrad g = {dY, lddy, pre, ldpre, dpre, lddpre, dbias, dX, lddx};
  return mbok::launch_linear_backward(d, packed, g, T, act, accumulate, workspace, passes,
                                      (hipStream_t)stream);
}

int mbok_linear_backward(const mbok_desc* d, const void* packed, const void* pre, int64_t ldpre,
                         const void* dY, int64_t lddy, int64_t T, int32_t act, void* dpre,
                         int64_t lddpre, float* dbias, int32_t accumulate, void* dX,
                         int64_t lddx, void* workspace, void* stream) {
  return linear_backward_checked(d, packed, pre, ldpre, dY, lddy, T, act, dpre, lddpre, dbias,
                                 accumulate, dX, lddx, workspace, 1, stream);
}

int mbok_linear_backward_precise(const mbok_desc* d, const void* packed, const void* pre,
                                 int64_t ldpre, const void* dY, int64_t lddy, int64_t T,
                                 int32_t act, void* dpre, int64_t lddpre, float* dbias,
                                 int32_t accumulate, void* dX, int64_t lddx, void* workspace,
                                 void* stream) {
  return linear_backward_checked(d, packed, pre, ldpre, dY, lddy, T, act, dpre, lddpre, dbias,
                                 accumulate, dX, lddx, workspace, 2, stream);
}

size_t mbok_linear_backward_workspace_bytes(const mbok_desc* d, int64_t T) {
  if (check_desc(d) != MBOK_OK || T < 1 || T > MBOK_MAX_T) return 0;
  return mbok::linear_backward_workspace_bytes(d, T);
}

static int check_rows_desc(int32_t vocab, float temperature) {
  // as check_distill
  if (!std::isnormal(temperature) || !(temperature > 0.f)) return MBOK_ERR_INVALID_ARG;
  return vocab < 1 || vocab > MBOK_MAX_VOCAB ? MBOK_ERR_SHAPE : MBOK_OK;
}

int mbok_logp_desc_init(mbok_logp_desc* d, int32_t vocab, float temperature) {
  if (!d) return MBOK_ERR_INVALID_ARG;
  const int st = check_rows_desc(vocab, temperature);
  if (st != MBOK_OK) return st;
  *d = mbok_logp_desc{vocab, temperature};
  return MBOK_OK;
}

// what the calls on rows of logits check alike
static int check_rows(int32_t vocab, const mbok::RowArgs& a) {
  if (!a.Z || !a.label) return MBOK_ERR_INVALID_ARG;
  if (a.T < 1 || a.T > MBOK_MAX_DISTILL_ROWS) return MBOK_ERR_SHAPE;
  if (a.ldz < vocab || a.ldz > kMaxLd) return MBOK_ERR_INVALID_ARG;
  if (a.dZ && (a.lddz < vocab || a.lddz > kMaxLd)) return MBOK_ERR_INVALID_ARG;
  if (!float_dtype(a.z_dtype)) return MBOK_ERR_DTYPE;
  if (a.dZ && a.dz_dtype != a.z_dtype && a.dz_dtype != MBOK_BF16) return MBOK_ERR_DTYPE;
  if (a.dZ == a.Z && (a.dz_dtype != a.z_dtype || a.lddz != a.ldz)) return MBOK_ERR_INVALID_ARG;
  auto size = [](int32_t t) { return t == MBOK_F32 ? 4 : 2; };
  if (!aligned(a.Z, size(a.z_dtype)) || !aligned(a.label, 4) ||
      (a.dZ && !aligned(a.dZ, size(a.dz_dtype))))
    return MBOK_ERR_ALIGN;
  return MBOK_OK;
}

int mbok_logp(const mbok_logp_desc* d, const void* Z, int32_t z_dtype, int64_t T, int64_t ldz,
              const int32_t* label, float* logp, float* stats, void* stream) {
  if (!d) return MBOK_ERR_INVALID_ARG;
  int st = check_rows_desc(d->vocab, d->temperature);
  if (st != MBOK_OK) return st;
  const mbok::RowArgs a = {Z, z_dtype, T, ldz, label, nullptr, z_dtype, 0};
  st = check_rows(d->vocab, a);
  if (st != MBOK_OK) return st;
  if (!logp) return MBOK_ERR_INVALID_ARG;
  if (!aligned(logp, 4) || !aligned(stats, 16)) return MBOK_ERR_ALIGN;
  return mbok::launch_logp(d, a, logp, stats, (hipStream_t)stream);
}

int mbok_logp_backward(const mbok_logp_desc* d, const void* Z, int32_t z_dtype, int64_t T,
                       int64_t ldz, const int32_t* label, const float* stats,
                       const float* dlogp, void* dZ, int32_t dz_dtype, int64_t lddz,
                       void* stream) {
  if (!d || !dZ) return MBOK_ERR_INVALID_ARG;
  int st = check_rows_desc(d->vocab, d->temperature);
  if (st != MBOK_OK) return st;
  const mbok::RowArgs a = {Z, z_dtype, T, ldz, label, dZ, dz_dtype, lddz};
  st = check_rows(d->vocab, a);
  if (st != MBOK_OK) return st;
  if (!stats || !dlogp) return MBOK_ERR_INVALID_ARG;
  if (!aligned(stats, 16) || !aligned(dlogp, 4)) return MBOK_ERR_ALIGN;
  return mbok::launch_logp_backward(d, a, stats, dlogp, (hipStream_t)stream);
}

static int check_policy(const mbok_policy_desc* d) {
  if (!d || !(d->clip_low >= 0.f && d->clip_low <= 1.f) || !(d->clip_high >= 0.f) ||
      !(d->kl >= 0.f) || !std::isfinite(d->kl))
    return MBOK_ERR_INVALID_ARG;
  return check_rows_desc(d->vocab, d->temperature);
}

int mbok_policy_desc_init(mbok_policy_desc* d, int32_t vocab, float temperature, float clip_low,
                          float clip_high, float kl) {
  if (!d) return MBOK_ERR_INVALID_ARG;
  const mbok_policy_desc t = {vocab, temperature, clip_low, clip_high, kl};
  const int st = check_policy(&t);
  if (st != MBOK_OK) return st;
  *d = t;
  return MBOK_OK;
}

int mbok_policy(const mbok_policy_desc* d, const void* Z, int32_t z_dtype, int64_t T,
                int64_t ldz, const int32_t* label, const float* advantage,
                const float* old_logp, const float* ref_logp, const float* weight, float* loss,
                float* logp, float* stats, float* dlogp, void* dZ, int32_t dz_dtype,
                int64_t lddz, void* stream) {
  int st = check_policy(d);
  if (st != MBOK_OK) return st;
  const mbok::RowArgs a = {Z, z_dtype, T, ldz, label, dZ, dz_dtype, lddz};
  st = check_rows(d->vocab, a);
  if (st != MBOK_OK) return st;
  if (!advantage || !loss) return MBOK_ERR_INVALID_ARG;
  if (!aligned(advantage, 4) || !aligned(old_logp, 4) || !aligned(ref_logp, 4) ||
      !aligned(weight, 4) || !aligned(loss, 4) || !aligned(logp, 4) || !aligned(stats, 16) ||
      !aligned(dlogp, 4))
    return MBOK_ERR_ALIGN;
  return mbok::launch_policy(d, a, advantage, old_logp, ref_logp, weight, loss, logp, stats,
                             dlogp, (hipStream_t)stream);
}

static int check_preference(const mbok_preference_desc* d) {
  if (!d || !(d->beta > 0.f) || !std::isfinite(d->beta) ||
      !(d->smoothing >= 0.f && d->smoothing <= 0.5f) || !std::isfinite(d->margin))
    return MBOK_ERR_INVALID_ARG;
  return d->vocab < 1 || d->vocab > MBOK_MAX_VOCAB ? MBOK_ERR_SHAPE : MBOK_OK;
}

int mbok_preference_desc_init(mbok_preference_desc* d, float beta, float smoothing,
                              float margin, int32_t mean, int32_t vocab) {
  if (!d) return MBOK_ERR_INVALID_ARG;
  const mbok_preference_desc t = {beta, smoothing, margin, mean != 0, vocab};
  const int st = check_preference(&t);
  if (st != MBOK_OK) return st;
  *d = t;
  return MBOK_OK;
}

int mbok_preference(const mbok_preference_desc* d, const int32_t* offsets, int64_t pairs,
                    const float* logp, const float* ref_logp, const int32_t* label, int64_t T,
                    const float* weight, float* loss, float* dlogp, void* stream) {
  const int st = check_preference(d);
  if (st != MBOK_OK) return st;
  if (!offsets || !logp || !loss) return MBOK_ERR_INVALID_ARG;
  if (T < 1 || T > MBOK_MAX_DISTILL_ROWS || pairs < 1 || pairs > MBOK_MAX_PAIRS)
    return MBOK_ERR_SHAPE;
  if (!aligned(offsets, 4) || !aligned(logp, 4) || !aligned(ref_logp, 4) ||
      !aligned(label, 4) || !aligned(weight, 4) || !aligned(loss, 4) || !aligned(dlogp, 4))
    return MBOK_ERR_ALIGN;
  return mbok::launch_preference(d, offsets, pairs, logp, ref_logp, label, T, weight, loss, dlogp,
                                 (hipStream_t)stream);
}

namespace {

struct Range {
  uintptr_t from, to;
};

bool overlap(std::vector<Range>& r) {
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.from < b.from; });
  for (size_t i = 1; i < r.size(); ++i)
    if (r[i].from < r[i - 1].to) return true;
  return false;
}

// whether a range of `a` meets one of `b`; both are sorted, b's do not overlap
bool meet(const std::vector<Range>& a, const std::vector<Range>& b) {
  for (const Range& x : a) {
    auto it = std::upper_bound(b.begin(), b.end(), x.from,
                               [](uintptr_t v, const Range& y) { return v < y.to; });
    if (it != b.end() && it->from < x.to) return true;
  }
  return false;
}

// One tensor's arguments; adds what it writes and reads to the lists.
int check_adamw_tensor(const mbok_adamw_tensor& t, std::vector<Range>& written,
                       std::vector<Range>& read) {
  if (!t.param || !t.grad || !t.m || !t.v || t.count < 1 || !(t.weight_decay >= 0.0) ||
      !std::isfinite(t.weight_decay))
    return MBOK_ERR_INVALID_ARG;
  if (t.count > MBOK_MAX_ADAMW_VALUES) return MBOK_ERR_SHAPE;
  if (!float_dtype(t.grad_dtype)) return MBOK_ERR_DTYPE;
  if (t.state_dtype != MBOK_F32 && t.state_dtype != MBOK_E4M3) return MBOK_ERR_DTYPE;
  const bool eight = t.state_dtype == MBOK_E4M3;
  if (eight != (t.m_scale != nullptr) || eight != (t.v_scale != nullptr))
    return MBOK_ERR_INVALID_ARG;
  const uintptr_t n = (uintptr_t)t.count, gs = t.grad_dtype == MBOK_F32 ? 4 : 2;
  if (!aligned(t.param, 4) || !aligned(t.grad, gs) || (!eight && (!aligned(t.m, 4) ||
      !aligned(t.v, 4))) || !aligned(t.m_scale, 4) || !aligned(t.v_scale, 4))
    return MBOK_ERR_ALIGN;
  auto add = [](std::vector<Range>& to, const void* p, uintptr_t bytes) {
    to.push_back(Range{(uintptr_t)p, (uintptr_t)p + bytes});
  };
  add(written, t.param, 4 * n);
  add(written, t.m, eight ? n : 4 * n);
  add(written, t.v, eight ? n : 4 * n);
  if (eight) {
    const uintptr_t blocks = (n + MBOK_ADAMW_BLOCK - 1) / MBOK_ADAMW_BLOCK;
    add(written, t.m_scale, 4 * blocks);
    add(written, t.v_scale, 4 * blocks);
  }
  add(read, t.grad, gs * n);
  if (t.layer) {
    const int st = check_desc(t.layer);
    if (st != MBOK_OK) return st;
    if (!t.out) return MBOK_ERR_INVALID_ARG;
    if (t.count != (int64_t)t.layer->K * t.layer->m * (t.layer->n / MBOK_GROUP))
      return MBOK_ERR_SHAPE;
    if (!aligned(t.out, 16)) return MBOK_ERR_ALIGN;
    add(written, t.out, mbok_packed_bytes(t.layer));
  } else if (t.out) {
    if (!float_dtype(t.out_dtype)) return MBOK_ERR_DTYPE;
    const uintptr_t os = t.out_dtype == MBOK_F32 ? 4 : 2;
    if (!aligned(t.out, os)) return MBOK_ERR_ALIGN;
    add(written, t.out, os * n);
  }
  return MBOK_OK;
}

// Checks the tensors; the values a workgroup takes, the number of workgroups and
// their LDS.
int plan_adamw(const mbok_adamw_tensor* tensors, int32_t n, mbok_adamw_plan* plan,
               int* part) try {
  if (!tensors) return MBOK_ERR_INVALID_ARG;
  if (n < 1 || n > MBOK_MAX_ADAMW_TENSORS) return MBOK_ERR_SHAPE;
  std::vector<Range> written, read;
  int64_t values = 0;
  for (int32_t i = 0; i < n; ++i) {
    const int st = check_adamw_tensor(tensors[i], written, read);
    if (st != MBOK_OK) return st;
    values += tensors[i].count;
    if (values > MBOK_MAX_ADAMW_VALUES) return MBOK_ERR_SHAPE;
  }
  if (overlap(written) || meet(read, written)) return MBOK_ERR_INVALID_ARG;
  *part = mbok::adamw_part(values);
  int64_t parts = 0;
  plan->lds_bytes = 0;
  for (int32_t i = 0; i < n; ++i) {
    parts += (tensors[i].count + *part - 1) / *part;
    if (tensors[i].layer)
      plan->lds_bytes = std::max(
          plan->lds_bytes, mbok::adamw_layer_lds(tensors[i].layer->n / MBOK_GROUP, *part));
  }
  plan->tensors = n;
  plan->parts = (int32_t)parts;
  plan->table_bytes =
      (int64_t)n * sizeof(mbok::AdamTensor) + parts * (int64_t)sizeof(mbok::AdamPart);
  return MBOK_OK;
} catch (const std::bad_alloc&) {  // the lists of ranges
  return MBOK_ERR_SCRATCH;
}

}  // namespace

size_t mbok_adamw_table_bytes(const mbok_adamw_tensor* tensors, int32_t n) {
  mbok_adamw_plan plan;
  int part;
  return plan_adamw(tensors, n, &plan, &part) == MBOK_OK ? (size_t)plan.table_bytes : 0;
}

int mbok_adamw_plan_init(mbok_adamw_plan* plan, const mbok_adamw_tensor* tensors, int32_t n,
                         void* table) {
  if (!plan || !table) return MBOK_ERR_INVALID_ARG;
  mbok_adamw_plan p;
  int part;
  const int st = plan_adamw(tensors, n, &p, &part);
  if (st != MBOK_OK) return st;
  char* at = reinterpret_cast<char*>(table);
  for (int32_t i = 0; i < n; ++i, at += sizeof(mbok::AdamTensor)) {
    const mbok_adamw_tensor& t = tensors[i];
    mbok::AdamTensor a = {};
    a.param = t.param;
    a.grad = t.grad;
    a.m = t.m;
    a.v = t.v;
    a.m_scale = t.m_scale;
    a.v_scale = t.v_scale;
    a.out = t.out;
    a.decay = t.weight_decay;
    a.salt = mbok::adamw_salt(i);
    a.grad_dtype = t.grad_dtype;
    a.state_dtype = t.state_dtype;
    a.out_dtype = t.out_dtype;
    if (t.layer) {
      const size_t alphas = mbok_packed_bytes(t.layer);
      const size_t m_pad =
          ((size_t)t.layer->m + MBOK_ROW_BLOCK - 1) / MBOK_ROW_BLOCK * MBOK_ROW_BLOCK;
      a.groups = t.layer->n / MBOK_GROUP;
      a.kernels = t.layer->K;
      a.rows = t.layer->m;
      a.out_dtype = t.layer->alpha_dtype;
      a.out = reinterpret_cast<char*>(t.out) + alphas -
              m_pad * a.kernels * a.groups * alpha_size(a.out_dtype);
    }
    memcpy(at, &a, sizeof(a));
  }
  for (int32_t i = 0; i < n; ++i)
    for (int64_t s = 0; s < tensors[i].count; s += part, at += sizeof(mbok::AdamPart)) {
      const mbok::AdamPart a = {s, i, (int32_t)std::min<int64_t>(part, tensors[i].count - s)};
      memcpy(at, &a, sizeof(a));
    }
  *plan = p;
  return MBOK_OK;
}

int mbok_adamw(const mbok_adamw_plan* plan, const void* table, const mbok_adamw_step* step,
               const float* live, void* stream) {
  if (!plan || !table || !step) return MBOK_ERR_INVALID_ARG;
  if (plan->tensors < 1 || plan->tensors > MBOK_MAX_ADAMW_TENSORS || plan->parts < 1 ||
      plan->parts >= (1 << 24) || plan->lds_bytes < 0 || plan->lds_bytes > 65536 ||
      plan->table_bytes != (int64_t)plan->tensors * (int64_t)sizeof(mbok::AdamTensor) +
                               (int64_t)plan->parts * (int64_t)sizeof(mbok::AdamPart))
    return MBOK_ERR_INVALID_ARG;
  if (!std::isfinite(step->lr) || !(step->beta1 >= 0.0 && step->beta1 < 1.0) ||
      !(step->beta2 >= 0.0 && step->beta2 < 1.0) || !(step->eps >= 0x1p-126) ||
      !std::isfinite((float)step->eps) || std::isnan(step->grad_scale) || step->step < 1 ||
      step->step >= (int64_t(1) << 53))
    return MBOK_ERR_INVALID_ARG;
  if (!aligned(table, 16) || !aligned(live, 4)) return MBOK_ERR_ALIGN;
  return mbok::launch_adamw(plan, table, step, live, (hipStream_t)stream);
}

const char* mbok_status_str(int status) {
  switch (status) {
    case MBOK_OK: return "MBOK_OK: success";
    case MBOK_ERR_INVALID_ARG: return "MBOK_ERR_INVALID_ARG: null pointer, unknown enum or bad leading dimension";
    case MBOK_ERR_SHAPE: return "MBOK_ERR_SHAPE: m, n or T out of range, or n not a multiple of 128";
    case MBOK_ERR_DTYPE: return "MBOK_ERR_DTYPE: element type not accepted by this call";
    case MBOK_ERR_ALIGN: return "MBOK_ERR_ALIGN: pointer or leading dimension misaligned";
    case MBOK_ERR_HIP: return "MBOK_ERR_HIP: the HIP runtime rejected a launch";
    case MBOK_ERR_UNSUPPORTED: return "MBOK_ERR_UNSUPPORTED: K, group or layout outside what the library runs";
    case MBOK_ERR_INFEASIBLE: return "MBOK_ERR_INFEASIBLE: no kernel allocation fits the bit budget";
    case MBOK_ERR_SCRATCH: return "MBOK_ERR_SCRATCH: the call needs more scratch than the library's static scratch holds";
  }
  return "unknown status";
}

const char* mbok_version(void) { return "mbok 0.1.0 gfx950"; }

}  // extern "C"
