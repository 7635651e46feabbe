// C ABI of the operators around an adapted projection (lq_block.h): argument
// validation and dispatch to the kernels.
#include <cmath>

#include "block.h"
#include "check.h"
#include "dispatch.h"
#include "mx.h"

using namespace lq;

namespace {

constexpr int64_t kLim = (int64_t)1 << 31;

int check_to(const void* p, size_t bytes, const char* name) {
  REQUIRE((uintptr_t)p % bytes == 0, LQ_ERR_INVALID_ARG, "%s is not aligned to %zu bytes", name,
          bytes);
  return LQ_OK;
}

// ------------------------------------------------------------------ norm

// at most 2^35 elements, padding included (M not negative)
bool norm_fits(int64_t M, int64_t K) {
  return K >= 1 && K <= 65536 && M <= ((int64_t)1 << 35) / (cdiv(K, kMxB) * kMxB);
}

int check_norm(int64_t M, int64_t K, lq_dtype dt, const void* W, lq_dtype wdt, float eps) {
  REQUIRE(dt == LQ_F32 || dt == LQ_BF16, LQ_ERR_INVALID_ARG, "bad dtype %d", (int)dt);
  REQUIRE(wdt == LQ_F32 || wdt == LQ_BF16, LQ_ERR_INVALID_ARG, "bad gain dtype %d", (int)wdt);
  REQUIRE(M >= 0 && K >= 1, LQ_ERR_INVALID_ARG, "%lld x %lld elements", (long long)M,
          (long long)K);
  REQUIRE(norm_fits(M, K), LQ_ERR_UNSUPPORTED,
          "%lld x %lld elements: K <= 65536 and at most 2^35 elements", (long long)M,
          (long long)K);
  REQUIRE(std::isfinite(eps) && eps >= 0.0f, LQ_ERR_INVALID_ARG, "eps = %g", (double)eps);
  REQUIRE(W != nullptr, LQ_ERR_INVALID_ARG, "W is NULL");
  return check_to(W, wdt == LQ_F32 ? 4 : 2, "W");
}

// -------------------------------------------------------------- adapters

// The first of the shape rules that the sizes break, or NULL: one place for the
// calls and the workspace sizes
const char* broken_rule(int64_t M, int64_t N, int64_t K, int64_t r, int64_t slots) {
  if (M < 0 || N < 1 || K < 1 || r < 1 || slots < 1) return "sizes must be positive";
  if (K % 64 || N % 64) return "N and K must be multiples of 64";
  if (K > 65536 || N > 65536) return "N, K <= 65536";
  if (r > 64) return "rank outside [1, 64]";
  if (slots > LQ_ADAPTERS_MAX_SLOTS) return "more than 4096 places";
  if (M >= kLim || M * K >= kLim || M * N >= kLim || M * r >= kLim)
    return "M*K, M*N and M*r must be below 2^31 elements";
  return nullptr;
}

int check_pool(const lq_adapter_pool* q, int64_t M, const int32_t* rows) {
  REQUIRE(q != nullptr, LQ_ERR_INVALID_ARG, "pool is NULL");
  REQUIRE(M >= 0 && q->N >= 1 && q->K >= 1 && q->r >= 1 && q->slots >= 1, LQ_ERR_INVALID_ARG,
          "M=%lld N=%lld K=%lld r=%d slots=%d", (long long)M, (long long)q->N, (long long)q->K,
          (int)q->r, (int)q->slots);
  const char* rule = broken_rule(M, q->N, q->K, q->r, q->slots);
  REQUIRE(!rule, LQ_ERR_UNSUPPORTED, "%s (M=%lld N=%lld K=%lld r=%d slots=%d)", rule,
          (long long)M, (long long)q->N, (long long)q->K, (int)q->r, (int)q->slots);
  if (M == 0) return LQ_OK;
  REQUIRE(q->A && q->B && q->scales, LQ_ERR_INVALID_ARG, "the pool's A, B or scales is NULL");
  REQUIRE(rows != nullptr, LQ_ERR_INVALID_ARG, "rows is NULL");
  int rc = check_to(q->A, 16, "A");
  if (!rc) rc = check_to(q->B, 16, "B");
  if (!rc) rc = check_to(q->ranks, 4, "ranks");
  if (!rc) rc = check_to(q->scales, 4, "scales");
  if (!rc) rc = check_to(rows, 4, "rows");
  return rc;
}

// ------------------------------------------------------------------ head

const char* broken_head_rule(int64_t M, int64_t V, int64_t K, int64_t kt) {
  if (K % 64 || K < 64 || K > 16384) return "K must be a multiple of 64, at most 16384";
  if (V < 1 || V > (1 << 20)) return "vocabulary outside [1, 2^20]";
  if (kt < 1 || kt > 128) return "targets per row outside [1, 128]";
  if (M < 0 || M >= kLim || M * K >= kLim || V * K >= kLim || M * kt >= kLim)
    return "M*K, V*K and M*kt must be below 2^31 elements";
  return nullptr;
}

}  // namespace

extern "C" {

int lq_rmsnorm_fwd(const void* X, const void* R, int64_t M, int64_t K, lq_dtype dt,
                   const void* W, lq_dtype wdt, float eps, void* H_out, void* Y,
                   int32_t format, uint8_t* codes, uint8_t* scales, float* rstd_out,
                   hipStream_t stream) {
  int rc = check_norm(M, K, dt, W, wdt, eps);
  if (rc) return rc;
  REQUIRE(Y || codes, LQ_ERR_INVALID_ARG, "nothing to write: Y and codes are NULL");
  if (codes) {
    REQUIRE(format == LQ_MX_FP4 || format == LQ_MX_FP8, LQ_ERR_INVALID_ARG,
            "unknown MX format %d", (int)format);
    REQUIRE(scales != nullptr, LQ_ERR_INVALID_ARG, "codes without scales");
    if ((rc = check_to(codes, 16, "codes"))) return rc;
  }
  REQUIRE(!H_out || H_out != Y, LQ_ERR_INVALID_ARG, "H_out and Y are the same buffer");
  if (M == 0) return LQ_OK;
  REQUIRE(X != nullptr, LQ_ERR_INVALID_ARG, "X is NULL");
  const size_t e = dt == LQ_F32 ? 4 : 2;
  if ((rc = check_to(X, e, "X")) || (rc = check_to(R, e, "R")) ||
      (rc = check_to(H_out, e, "H_out")) || (rc = check_to(Y, e, "Y")) ||
      (rc = check_to(rstd_out, 4, "rstd_out")))
    return rc;
  return dispatch::rmsnorm_fwd(X, R, M, K, dt, W, wdt, eps, H_out, Y, format, codes, scales,
                               rstd_out, stream);
}

size_t lq_rmsnorm_bwd_workspace(int64_t M, int64_t K) {
  return M <= 0 || !norm_fits(M, K) ? 0 : dispatch::rmsnorm_part_bytes(M, K);
}

int lq_rmsnorm_bwd(const void* dY, const void* H, int64_t M, int64_t K, lq_dtype dt,
                   const void* W, lq_dtype wdt, float eps, const float* rstd, const void* dH,
                   void* dX, float* dW, int32_t accumulate, void* ws, size_t ws_bytes,
                   hipStream_t stream) {
  int rc = check_norm(M, K, dt, W, wdt, eps);
  if (rc) return rc;
  REQUIRE(dX || dW, LQ_ERR_INVALID_ARG, "nothing to compute: dX and dW are NULL");
  if ((rc = check_to(dW, 4, "dW"))) return rc;
  if (M == 0) return dW && !accumulate ? launch_zero_f32(dW, K, stream) : LQ_OK;
  REQUIRE(dY && H, LQ_ERR_INVALID_ARG, "dY or H is NULL");
  const size_t e = dt == LQ_F32 ? 4 : 2;
  if ((rc = check_to(dY, e, "dY")) || (rc = check_to(H, e, "H")) ||
      (rc = check_to(dH, e, "dH")) || (rc = check_to(dX, e, "dX")) ||
      (rc = check_to(rstd, 4, "rstd")) || (rc = check_to(ws, 16, "ws")))
    return rc;
  if (dW) {
    const size_t need = dispatch::rmsnorm_part_bytes(M, K);
    REQUIRE(ws != nullptr && ws_bytes >= need, LQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu",
            ws_bytes, need);
  }
  return dispatch::rmsnorm_bwd(dY, H, M, K, dt, W, wdt, eps, rstd, dH, dX, dW, accumulate,
                               (float*)ws, stream);
}

size_t lq_adapters_workspace_size(int32_t op, int64_t M, int64_t N, int64_t K, int64_t r,
                                  int32_t slots) {
  if (M <= 0 || broken_rule(M, N, K, r, slots)) return 0;
  if (op == LQ_ADAPTERS_OP_FWD) return dispatch::adapters_fwd_ws(M, N, K, r, slots);
  if (op == LQ_ADAPTERS_OP_BWD) return dispatch::adapters_bwd_ws(M, N, K, r, slots);
  return 0;
}

int lq_adapters_fwd(const void* X, int64_t M, const lq_adapter_pool* pool, const int32_t* rows,
                    const void* Y_in, void* Y_out, float* T_out, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  int rc = check_pool(pool, M, rows);
  if (rc || M == 0) return rc;
  REQUIRE(X && Y_in && Y_out, LQ_ERR_INVALID_ARG, "X, Y_in or Y_out is NULL");
  if ((rc = check_to(X, 16, "X")) || (rc = check_to(Y_in, 16, "Y_in")) ||
      (rc = check_to(Y_out, 16, "Y_out")) || (rc = check_to(T_out, 4, "T_out")) ||
      (rc = check_to(ws, 16, "ws")))
    return rc;
  const size_t need = dispatch::adapters_fwd_ws(M, pool->N, pool->K, pool->r, pool->slots);
  REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need), LQ_ERR_WORKSPACE,
          "workspace %zu bytes, need %zu", ws_bytes, need);
  return dispatch::adapters_fwd(X, M, *pool, rows, Y_in, Y_out, T_out, ws, stream);
}

int lq_adapters_bwd(const void* dY, const void* X, int64_t M, const lq_adapter_pool* pool,
                    const int32_t* rows, const float* T_saved, const void* dX_in, void* dX_out,
                    float* dA, float* dB, int32_t accumulate, void* ws, size_t ws_bytes,
                    hipStream_t stream) {
  int rc = check_pool(pool, M, rows);
  if (rc) return rc;
  REQUIRE((dA == nullptr) == (dB == nullptr), LQ_ERR_INVALID_ARG,
          "dA and dB must both be given or both be NULL");
  REQUIRE((dX_in == nullptr) == (dX_out == nullptr), LQ_ERR_INVALID_ARG,
          "dX_in and dX_out must both be given or both be NULL");
  REQUIRE(dA || dX_out, LQ_ERR_INVALID_ARG, "nothing to compute: dX_out, dA and dB are NULL");
  if ((rc = check_to(dA, 16, "dA")) || (rc = check_to(dB, 16, "dB"))) return rc;
  const int64_t N = pool->N, K = pool->K, r = pool->r, slots = pool->slots;
  if (M == 0) {
    if (accumulate || !dA) return LQ_OK;
    if ((rc = launch_zero_f32(dA, slots * r * K, stream))) return rc;
    return launch_zero_f32(dB, slots * r * N, stream);
  }
  REQUIRE(dY && (X || !dA), LQ_ERR_INVALID_ARG, "dY or X is NULL");
  if ((rc = check_to(dY, 16, "dY")) || (rc = check_to(X, 16, "X")) ||
      (rc = check_to(dX_in, 16, "dX_in")) || (rc = check_to(dX_out, 16, "dX_out")) ||
      (rc = check_to(T_saved, 4, "T_saved")) || (rc = check_to(ws, 16, "ws")))
    return rc;
  const size_t need = dispatch::adapters_bwd_ws(M, N, K, r, pool->slots);
  REQUIRE(ws != nullptr && ws_bytes >= need, LQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu",
          ws_bytes, need);
  return dispatch::adapters_bwd(dY, X, M, *pool, rows, T_saved, dX_in, dX_out, dA, dB, accumulate,
                                ws, stream);
}

size_t lq_head_loss_workspace(int64_t M, int64_t V, int64_t K, int32_t kt, int32_t need_dh) {
  return M <= 0 || broken_head_rule(M, V, K, kt)
             ? 0
             : dispatch::head_loss_ws(M, V, K, kt, need_dh != 0);
}

int lq_head_loss(const void* H, int64_t M, const lq_weight* W0, const int32_t* targets,
                 const float* p, int32_t kt, const float* w, float logit_scale, float* loss,
                 float* lse, void* dH, void* ws, size_t ws_bytes, hipStream_t stream) {
  REQUIRE(W0 != nullptr, LQ_ERR_INVALID_ARG, "W0 is NULL");
  REQUIRE(W0->kind == LQ_WEIGHT_DENSE && W0->dtype == LQ_BF16, LQ_ERR_UNSUPPORTED,
          "the head is a dense bf16 weight");
  const int64_t V = W0->N, K = W0->K;
  REQUIRE(M >= 0 && V >= 1 && K >= 1, LQ_ERR_INVALID_ARG, "M=%lld V=%lld K=%lld", (long long)M,
          (long long)V, (long long)K);
  const char* rule = broken_head_rule(M, V, K, kt);
  REQUIRE(!rule, LQ_ERR_UNSUPPORTED, "%s (M=%lld V=%lld K=%lld kt=%d)", rule, (long long)M,
          (long long)V, (long long)K, (int)kt);
  REQUIRE(std::isfinite(logit_scale), LQ_ERR_INVALID_ARG, "logit_scale = %g", (double)logit_scale);
  REQUIRE(loss || lse || dH, LQ_ERR_INVALID_ARG, "nothing to compute: loss, lse and dH are NULL");
  if (M == 0) return LQ_OK;
  REQUIRE(H && W0->dense && targets, LQ_ERR_INVALID_ARG, "H, W0's data or targets is NULL");
  int rc;
  if ((rc = check_to(H, 16, "H")) || (rc = check_to(W0->dense, 16, "W0")) ||
      (rc = check_to(dH, 16, "dH")) || (rc = check_to(ws, 16, "ws")) ||
      (rc = check_to(targets, 4, "targets")) || (rc = check_to(p, 4, "p")) ||
      (rc = check_to(w, 4, "w")) || (rc = check_to(loss, 4, "loss")) || (rc = check_to(lse, 4, "lse")))
    return rc;
  const size_t need = dispatch::head_loss_ws(M, V, K, kt, dH != nullptr);
  REQUIRE(ws != nullptr && ws_bytes >= need, LQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu",
          ws_bytes, need);
  return dispatch::head_loss(H, M, V, K, W0->dense, targets, p, kt, w, logit_scale, loss, lse, dH,
                             ws, stream);
}

}  // extern "C"
