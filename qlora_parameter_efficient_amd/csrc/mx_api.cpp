// C ABI of the MX operators (lq_mx.h): argument validation, workspace carving
// and dispatch to the kernels.
#include "check.h"
#include "dispatch.h"
#include "mx.h"

using namespace lq;

namespace lq {

int mx_check_aligned(const void* p, const char* name) {
  REQUIRE(((uintptr_t)p & 15) == 0, LQ_ERR_INVALID_ARG, "%s is not 16-byte aligned", name);
  return LQ_OK;
}

int mx_check_tensor(const lq_mx_tensor* q, const char* name, int32_t formats, int64_t rows,
                    int64_t cols) {
  REQUIRE(q != nullptr, LQ_ERR_INVALID_ARG, "%s is NULL", name);
  REQUIRE(q->format == LQ_MX_FP4 || q->format == LQ_MX_FP8, LQ_ERR_INVALID_ARG,
          "%s has unknown MX format %d", name, (int)q->format);
  REQUIRE(q->format & formats, LQ_ERR_UNSUPPORTED, "%s in MX format %d is not supported here",
          name, (int)q->format);
  REQUIRE(q->rows == rows && q->cols == cols, LQ_ERR_INVALID_ARG,
          "%s is %lld x %lld, expected %lld x %lld", name, (long long)q->rows,
          (long long)q->cols, (long long)rows, (long long)cols);
  REQUIRE(q->codes && q->scales, LQ_ERR_INVALID_ARG, "%s has a NULL buffer", name);
  // rows of whole 64-column groups start at even addresses, also in a tensor that
  // begins at a row of another
  REQUIRE((uintptr_t)q->scales % 2 == 0, LQ_ERR_INVALID_ARG, "%s has scales at an odd address",
          name);
  return mx_check_aligned(q->codes, name);
}

}  // namespace lq

namespace {

constexpr int64_t kMaxRank = 64;
constexpr int64_t kMaxElems = (int64_t)1 << 35;

// No more elements than the codec takes, padding included (sizes not negative)
bool codec_fits(int64_t rows, int64_t cols) {
  return cols == 0 || (cols <= kMaxElems && rows <= kMaxElems / (cdiv(cols, kMxB) * kMxB));
}

size_t up256(size_t b) { return (b + 255) & ~(size_t)255; }

// The first of the layer's shape rules that the sizes break, or NULL: one place
// for the calls and for the workspace sizes, which are asked for before a call
// has checked anything.  M, N and K are positive, or M is 0.
const char* broken_rule(int64_t M, int64_t N, int64_t K, int64_t r, int64_t rmin) {
  const int64_t lim = (int64_t)1 << 31;
  if (K % 64 || N % 64) return "N and K must be multiples of 64";
  if (K > 65536 || N > 65536) return "N, K <= 65536";
  if (M >= lim || M * K >= lim || M * N >= lim) return "M*K and M*N must be below 2^31 elements";
  if (r < rmin || r > kMaxRank) return rmin ? "rank outside [1, 64]" : "rank outside [0, 64]";
  return nullptr;
}

int check_layer(const lq_mx_tensor* W0, int64_t M, int64_t r, int64_t rmin) {
  REQUIRE(W0 != nullptr, LQ_ERR_INVALID_ARG, "W0 is NULL");
  const int64_t N = W0->rows, K = W0->cols;
  REQUIRE(N > 0 && K > 0, LQ_ERR_INVALID_ARG, "W0 is %lld x %lld", (long long)N, (long long)K);
  REQUIRE(M >= 0, LQ_ERR_INVALID_ARG, "M = %lld", (long long)M);
  int rc = mx_check_tensor(W0, "W0", LQ_MX_FP4, N, K);
  if (rc) return rc;
  const char* rule = broken_rule(M, N, K, r, rmin);
  REQUIRE(!rule, LQ_ERR_UNSUPPORTED, "%s (M=%lld N=%lld K=%lld r=%lld)", rule, (long long)M,
          (long long)N, (long long)K, (long long)r);
  return LQ_OK;
}

// Workspace of the forward: [T][the path's part].  Either input kind may be
// given at M <= LQ_MX_ROWS_BF16, so the size covers both.
size_t fwd_part_bytes(int64_t M, int64_t N, int64_t K, int64_t r) {
  const size_t g = dispatch::mx_gemm_ws_bytes(M, N, K);
  const size_t s = M <= LQ_MX_ROWS_BF16 ? dispatch::mx_stream_ws_bytes(M, K, r) : 0;
  return g > s ? g : s;
}

// dX of a dense or NF4 base whose kind is not known: the large-tile product's
// part, or that of the split dX of a dense base
size_t big_dx_bytes(int64_t M, int64_t N, int64_t K) {
  const size_t a = dispatch::big_dx_eligible(M, N, K) ? dispatch::big_dx_ws_bytes(M, N, K) : 0;
  const size_t b = dispatch::mx_dx_ws_bytes(M, N, K);
  return a > b ? a : b;
}

}  // namespace

extern "C" {

size_t lq_mx_codes_bytes(int32_t format, int64_t rows, int64_t cols) {
  if ((format != LQ_MX_FP4 && format != LQ_MX_FP8) || rows < 0 || cols < 0) return 0;
  return !codec_fits(rows, cols) ? 0 : (size_t)(rows * mx_pitch(format, cols));
}

size_t lq_mx_scales_bytes(int64_t rows, int64_t cols) {
  return rows < 0 || cols < 0 || !codec_fits(rows, cols) ? 0 : (size_t)(rows * mx_spitch(cols));
}

int lq_mx_quantize(const void* X, lq_dtype xdt, int64_t rows, int64_t cols, int32_t format,
                   uint8_t* codes, uint8_t* scales, hipStream_t stream) {
  REQUIRE(X && codes && scales, LQ_ERR_INVALID_ARG, "X, codes or scales is NULL");
  REQUIRE(xdt == LQ_F32 || xdt == LQ_BF16, LQ_ERR_INVALID_ARG, "bad dtype %d", (int)xdt);
  REQUIRE(format == LQ_MX_FP4 || format == LQ_MX_FP8, LQ_ERR_INVALID_ARG,
          "unknown MX format %d", (int)format);
  REQUIRE(rows >= 1 && cols >= 1, LQ_ERR_INVALID_ARG, "%lld x %lld elements", (long long)rows,
          (long long)cols);
  REQUIRE(codec_fits(rows, cols), LQ_ERR_UNSUPPORTED, "%lld x %lld elements: more than 2^35",
          (long long)rows, (long long)cols);
  REQUIRE((uintptr_t)X % (xdt == LQ_F32 ? 4 : 2) == 0, LQ_ERR_INVALID_ARG, "X is misaligned");
  const int rc = mx_check_aligned(codes, "codes");
  if (rc) return rc;
  return dispatch::mx_quantize(X, xdt, rows, cols, format, codes, scales, stream);
}

int lq_mx_dequantize(const lq_mx_tensor* q, void* out, lq_dtype odt, hipStream_t stream) {
  REQUIRE(q != nullptr && out != nullptr, LQ_ERR_INVALID_ARG, "q or out is NULL");
  REQUIRE(odt == LQ_F32 || odt == LQ_BF16, LQ_ERR_INVALID_ARG, "bad dtype %d", (int)odt);
  REQUIRE(q->format == LQ_MX_FP4 || q->format == LQ_MX_FP8, LQ_ERR_INVALID_ARG,
          "unknown MX format %d", (int)q->format);
  REQUIRE(q->rows >= 1 && q->cols >= 1, LQ_ERR_INVALID_ARG, "%lld x %lld elements",
          (long long)q->rows, (long long)q->cols);
  REQUIRE(codec_fits(q->rows, q->cols), LQ_ERR_UNSUPPORTED, "%lld x %lld elements: more than 2^35",
          (long long)q->rows, (long long)q->cols);
  REQUIRE(q->codes && q->scales, LQ_ERR_INVALID_ARG, "q has a NULL buffer");
  REQUIRE((uintptr_t)out % (odt == LQ_F32 ? 4 : 2) == 0, LQ_ERR_INVALID_ARG, "out is misaligned");
  const int rc = mx_check_aligned(q->codes, "codes");
  if (rc) return rc;
  return dispatch::mx_dequantize(*q, out, odt, stream);
}

size_t lq_mx_workspace_size(int32_t op, int64_t M, int64_t N, int64_t K, int64_t r) {
  // 0 too for the sizes that the operators refuse
  if (M <= 0 || N <= 0 || K <= 0 || broken_rule(M, N, K, r, op == LQ_MX_OP_FWD ? 0 : 1)) return 0;
  const bool grads = op < LQ_MX_NO_GRADS;
  const int32_t kind = grads ? op : op - LQ_MX_NO_GRADS;
  if (!grads && kind == LQ_MX_OP_FWD) return 0;
  switch (kind) {
    case LQ_MX_OP_FWD:
      return up256((size_t)(M * r) * 4) + fwd_part_bytes(M, N, K, r);
    case LQ_MX_OP_BWD:
      return mx_bwd_ws(M, N, K, r, grads).rest + dispatch::mx_dx_ws_bytes(M, N, K);
    case LQ_MX_OP_BWD_CKPT:
      return mx_bwd_ws(M, N, K, r, grads).rest + big_dx_bytes(M, N, K);
    case LQ_MX_OP_BWD_CKPT_FUSED:
      return mx_bwd_ws(M, N, K, r, grads).rest;
    default:
      return 0;
  }
}

int lq_mx_lora_fwd(const void* X, const lq_mx_tensor* Xq, int64_t M, const lq_mx_tensor* W0,
                   const void* A, const void* B, int64_t r, float scale, void* Y, float* T_out,
                   void* ws, size_t ws_bytes, hipStream_t stream) {
  int rc = check_layer(W0, M, r, 0);
  if (rc) return rc;
  const int64_t N = W0->rows, K = W0->cols;
  if (M == 0) return LQ_OK;
  REQUIRE((X == nullptr) != (Xq == nullptr), LQ_ERR_INVALID_ARG,
          "exactly one of X and Xq must be given");
  REQUIRE(Y != nullptr, LQ_ERR_INVALID_ARG, "Y is NULL");
  REQUIRE(r == 0 || (A && B), LQ_ERR_INVALID_ARG, "A or B is NULL with rank %lld", (long long)r);
  REQUIRE(!X || M <= LQ_MX_ROWS_BF16, LQ_ERR_UNSUPPORTED,
          "bf16 X of %lld rows: more than %d take an MX tensor", (long long)M, LQ_MX_ROWS_BF16);
  if (Xq && (rc = mx_check_tensor(Xq, "Xq", LQ_MX_FP4 | LQ_MX_FP8, M, K))) return rc;
  if ((rc = mx_check_aligned(X, "X")) || (rc = mx_check_aligned(Y, "Y")) ||
      (rc = mx_check_aligned(ws, "ws")) || (r && (rc = mx_check_aligned(A, "A"))) ||
      (r && (rc = mx_check_aligned(B, "B"))))
    return rc;
  REQUIRE((uintptr_t)T_out % 4 == 0, LQ_ERR_INVALID_ARG, "T_out is misaligned");
  const size_t need = lq_mx_workspace_size(LQ_MX_OP_FWD, M, N, K, r);
  REQUIRE(need == 0 || (ws != nullptr && ws_bytes >= need), LQ_ERR_WORKSPACE,
          "workspace %zu bytes, need %zu", ws_bytes, need);
  char* part = (char*)ws + up256((size_t)(M * r) * 4);
  if (X)
    return dispatch::mx_stream_fwd(X, M, *W0, A, B, r, scale, Y, r ? T_out : nullptr, (float*)part,
                                   stream);
  float* T = T_out ? T_out : (float*)ws;
  if (r && (rc = dispatch::mx_shrink(*Xq, A, r, T, stream))) return rc;
  return dispatch::mx_gemm(*Xq, *W0, T, B, r, scale, Y, part, stream);
}

int lq_mx_lora_bwd(const void* dY, const lq_mx_tensor* Xq, int64_t M, const lq_mx_tensor* W0,
                   const void* A, const void* B, int64_t r, float scale, const float* T_saved,
                   void* dX, float* dA, float* dB, int32_t accumulate, void* ws,
                   size_t ws_bytes, hipStream_t stream) {
  int rc = check_layer(W0, M, r, 1);
  if (rc) return rc;
  const int64_t N = W0->rows, K = W0->cols;
  REQUIRE(A && B, LQ_ERR_INVALID_ARG, "A or B is NULL");
  REQUIRE((dA == nullptr) == (dB == nullptr), LQ_ERR_INVALID_ARG,
          "dA and dB must both be given or both be NULL");
  REQUIRE(dA || dX, LQ_ERR_INVALID_ARG, "nothing to compute: dX, dA and dB are NULL");
  if (M == 0) {
    if (accumulate || !dA) return LQ_OK;
    if ((rc = launch_zero_f32(dA, r * K, stream))) return rc;
    return launch_zero_f32(dB, N * r, stream);
  }
  REQUIRE(dY != nullptr, LQ_ERR_INVALID_ARG, "dY is NULL");
  if (dA && (rc = mx_check_tensor(Xq, "Xq", LQ_MX_FP4 | LQ_MX_FP8, M, K))) return rc;
  if ((rc = mx_check_aligned(dY, "dY")) || (rc = mx_check_aligned(dX, "dX")) ||
      (rc = mx_check_aligned(A, "A")) || (rc = mx_check_aligned(B, "B")) ||
      (rc = mx_check_aligned(ws, "ws")) || (rc = mx_check_aligned(T_saved, "T_saved")))
    return rc;
  const MxBwdWs w = mx_bwd_ws(M, N, K, r, dA != nullptr);
  const size_t need = w.rest + (dX ? dispatch::mx_dx_ws_bytes(M, N, K) : 0);
  REQUIRE(ws != nullptr && ws_bytes >= need, LQ_ERR_WORKSPACE, "workspace %zu bytes, need %zu",
          ws_bytes, need);
  char* base = (char*)ws;
  float* U = (float*)(base + w.u);
  if ((rc = dispatch::mx_u(dY, M, N, B, r, base + w.bt, U, stream))) return rc;
  if (dX) rc = dispatch::mx_dx(dY, M, *W0, U, A, r, scale, dX, base + w.rest, stream);
  if (rc || !dA) return rc;
  const float* T = T_saved;
  if (!T) {
    float* Tw = (float*)(base + w.t);
    if ((rc = dispatch::mx_shrink(*Xq, A, r, Tw, stream))) return rc;
    T = Tw;
  }
  return dispatch::mx_grads(*Xq, U, dY, T, N, r, scale, accumulate, dA, dB, base + w.part, stream);
}

}  // extern "C"
