/*
 * lq_block.h -- what stands around the adapted projections of a decoder block
 * on AMD Instinct MI355X (gfx950): the norm that feeds them, the adapters of
 * many requests beside one projection, and the loss at the end.  Part of
 * liblq.so; the conventions of lq.h (row-major, contiguous device pointers
 * owned by the caller, work enqueued on the caller's stream, no allocation, no
 * synchronisation, negative lq_status on a refused call, lq_last_error()) hold
 * here too.  Sums are float32; results do not depend on the order in which
 * workgroups run.
 */
#ifndef LQ_BLOCK_H
#define LQ_BLOCK_H

#include "lq_mx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------ RMS norm */

/*
 * Root-mean-square norm of the rows of H = X + R (R NULL: H = X), K columns:
 *   H  = round(X + R) to dt
 *   y  = H w / sqrt(mean(H^2) + eps),  mean over the row's K columns
 *   X, R     M x K of dt (LQ_BF16 or LQ_F32); R may be NULL
 *   W        gain w, K of wdt (LQ_BF16 or LQ_F32)
 *   H_out    optional M x K of dt: receives H (the residual stream)
 *   Y        optional M x K of dt: receives y, rounded once
 *   codes, scales, format   optional: y as an MX tensor (lq_mx.h; LQ_MX_FP8 or
 *            LQ_MX_FP4), quantised from float32 y by lq_mx_quantize's rule;
 *            codes NULL: none (scales and format are then not read)
 *   rstd_out optional M float32: 1 / sqrt(mean(H^2) + eps), for lq_rmsnorm_bwd
 * Rows whose H^2 leave float32's range are off as that sum is (|H| past 1e19: y is 0).
 * One of Y and codes at least.  H_out and Y may be X or R (the same pointer;
 * not both the same buffer); any other overlap of outputs with inputs or each
 * other is outside the contract.
 * Requires 1 <= K <= 65536, M >= 0 (0: no-op), at most 2^35 elements with the
 * rows padded to 32 columns, eps >= 0 and finite; pointers aligned to their
 * elements, codes to 16 bytes.
 */
int lq_rmsnorm_fwd(const void* X, const void* R, int64_t M, int64_t K, lq_dtype dt,
                   const void* W, lq_dtype wdt, float eps, void* H_out, void* Y,
                   int32_t format, uint8_t* codes, uint8_t* scales, float* rstd_out,
                   hipStream_t stream);

/*
 * Backward of lq_rmsnorm_fwd (an MX output is taken as the identity, the usual
 * straight-through reading).  With c = rstd of the row and g = dY w:
 *   dX = c (g - H c^2 mean(g H)) + dH     (also the gradient of R)
 *   dW = sum over rows of dY H c
 *   dY, H    M x K of dt; H as H_out gave it (X where there was no R)
 *   rstd     optional M float32 from rstd_out; NULL: formed from H and eps
 *   dH       optional M x K of dt: the gradient that reaches H by its other
 *            uses (the residual stream)
 *   dX       optional M x K of dt; may be dY, dH or H (the same pointer)
 *   dW       optional K float32; accumulate = 1 adds into it
 *   ws       lq_rmsnorm_bwd_workspace(M, K) bytes where dW is given
 * One of dX and dW at least.  Limits as lq_rmsnorm_fwd; M = 0 writes zeros to
 * dW unless accumulate is set.  dW is summed in a fixed order.
 */
int lq_rmsnorm_bwd(const void* dY, const void* H, int64_t M, int64_t K, lq_dtype dt,
                   const void* W, lq_dtype wdt, float eps, const float* rstd, const void* dH,
                   void* dX, float* dW, int32_t accumulate, void* ws, size_t ws_bytes,
                   hipStream_t stream);

/* Workspace of lq_rmsnorm_bwd with dW, in bytes; 0 for sizes that it refuses.  The
 * workspace of M rows is enough for fewer. */
size_t lq_rmsnorm_bwd_workspace(int64_t M, int64_t K);

/* -------------------------------- adapters of many requests, one projection */

/*
 * Low-rank adapters for one N x K projection, in ``slots`` places that the
 * caller loads and replaces while serving ([FT] "Serving many adapters at
 * once: the multi-tenant problem": many adapters resident beside one base, a
 * batch that mixes them).
 *   A       device slots x r x K bf16;  B  device slots x N x r bf16
 *   ranks   optional device int32[slots]: the rank in use, clamped to 0 .. r
 *           (NULL: r everywhere).  A's rows and B's columns past it are not
 *           part of the adapter: they may hold anything, NaN included
 *   scales  device float[slots]: each adapter's alpha / rank
 * Beside lq_lora_fwd_multi_ranks: that call forms the shared product too and rounds the
 * sum once, for segments given by the host and ranks of 64 together.  Here the rows
 * come in any order, places are loaded while serving, there is a backward, and the
 * base is any call's output, rounded before the adapters are added.
 */
typedef struct lq_adapter_pool {
  int32_t slots;
  int32_t r;
  int64_t N;
  int64_t K;
  const void* A;
  const void* B;
  const int32_t* ranks;
  const float* scales;
} lq_adapter_pool;

/*
 * Adds each row's adapter to a shared projection's output:
 *   Y_out[i] = Y_in[i] + scales[a] (X[i] A_a^T) B_a^T,   a = rows[i]
 *   X       M x K bf16
 *   rows    device int32[M]: the row's place in the pool, in any order; a value
 *           outside [0, slots) means no adapter, Y_out[i] = Y_in[i]
 *   Y_in    M x N bf16, e.g. of lq_lora_fwd or lq_mx_lora_fwd or a plain
 *           product; Y_out  M x N bf16, the same pointer or a buffer apart
 *           (in place, a row without an adapter is not touched)
 *   T_out   optional M x r float32: T[i] = X[i] A_a^T, zero past the adapter's
 *           rank and for rows without one (T_saved of lq_adapters_bwd)
 *   ws      lq_adapters_workspace_size(LQ_ADAPTERS_OP_FWD, M, N, K, r, slots) bytes
 *           (NULL where that is 0)
 * Ranks, scales and rows are read on the device: a captured call follows their
 * values at each replay.  T is float32 and enters its product with B in two
 * bf16 parts (2^-16 of its value); a row's non-finite elements stay in that row.
 * Requires K % 64 == 0, N % 64 == 0, N, K <= 65536, M K, M N and M r < 2^31,
 * 1 <= r <= 64, 1 <= slots <= 4096; X, A, B, Y_in, Y_out and ws 16-byte
 * aligned.  M = 0 is a no-op.
 */
int lq_adapters_fwd(const void* X, int64_t M, const lq_adapter_pool* pool, const int32_t* rows,
                    const void* Y_in, void* Y_out, float* T_out, void* ws, size_t ws_bytes,
                    hipStream_t stream);

/*
 * Backward of lq_adapters_fwd.  With U[i] = dY[i] B_a, a = rows[i]:
 *   dX_out[i] = dX_in[i] + scales[a] U[i] A_a     (bf16; dX_in: the gradient
 *               that came through the shared projection; the same pointer or a
 *               buffer apart; dX_in and dX_out may both be NULL)
 *   dA[a] = scales[a] sum over the adapter's rows of U[i]^T X[i]   (slots x r x K float32)
 *   dB[a] = scales[a] sum over its rows of dY[i]^T T[i]            (slots x N x r float32)
 *   dA and dB are given together or both NULL; they cover every place: zeros
 *   where no row has the adapter and past its rank.  accumulate = 1 adds
 *   instead (such entries then stay as they are).
 *   T_saved   optional T_out of the forward (NULL: recomputed)
 *   ws        lq_adapters_workspace_size(LQ_ADAPTERS_OP_BWD, ...) bytes
 * dA and dB are float32 sums, in a fixed order, of products with float32 U and
 * T (carried as three bf16 parts, so that nothing of their 24 bits is lost).  A
 * non-finite element makes the sums that it enters non-finite.
 * Without dA and dB X is not read.  The workspace and the time of the first launch grow
 * with slots, since factors are turned by place.  M = 0 writes zeros to dA and dB unless
 * accumulate is set.  Other rules as lq_adapters_fwd (dY, dX: 16-byte aligned).
 */
int lq_adapters_bwd(const void* dY, const void* X, int64_t M, const lq_adapter_pool* pool,
                    const int32_t* rows, const float* T_saved, const void* dX_in, void* dX_out,
                    float* dA, float* dB, int32_t accumulate, void* ws, size_t ws_bytes,
                    hipStream_t stream);

#define LQ_ADAPTERS_MAX_SLOTS 4096
#define LQ_ADAPTERS_OP_FWD 0
#define LQ_ADAPTERS_OP_BWD 1
/* Workspace in bytes; 0 for M = 0, for sizes that the call refuses, and for
 * forwards of few rows that need none.  The workspace of M rows is enough for
 * fewer. */
size_t lq_adapters_workspace_size(int32_t op, int64_t M, int64_t N, int64_t K, int64_t r,
                                  int32_t slots);

/* ------------------------------------------------- loss of a head */

/*
 * Softmax cross entropy of a frozen head over a vocabulary of V = W0->N
 * entries, from its input H, without keeping the logits z = c H W0^T
 * (c = logit_scale; 1 / temperature for distillation):
 *   lse[i]  = log sum over v of exp(z[i][v])
 *   loss[i] = sum over the targets j of row i of p[i][j] (lse[i] - z[i][t[i][j]])
 *   dH[i]   = d (sum over rows of w[i] loss[i]) / d H[i]
 *           = w[i] c (P_i softmax(z[i]) - sum over j of p[i][j] e(t[i][j])) W0,
 *             P_i = sum over j of p[i][j]
 * One label per row: kt = 1, p NULL (weights 1).  A teacher's top kt entries:
 * their indices and probabilities; the same index twice counts twice.
 *   H        M x K bf16;  W0  dense bf16, V x K (no gradient: the base is frozen)
 *   targets  device int32[M x kt]: a value outside [0, V) is no target; a row
 *            without any has loss 0 and dH 0 whatever H and w hold there
 *   p        optional device float[M x kt]
 *   w        optional device float[M]: the row's share of the total (1 / rows for
 *            a mean); NULL: 1.  Read for dH only
 *   loss, lse  optional device float[M];  dH  optional M x K bf16
 *   ws       lq_head_loss_workspace(M, V, K, kt, dH != NULL) bytes (more is not used)
 * Infinite logits: lse is +inf with a logit of +inf, -inf where all are -inf, NaN
 * with a NaN; loss follows from it, and dH of such a row is NaN.
 * One of loss, lse and dH at least.  The logits of one piece of rows at a time
 * are held in ws as float32; the gradient with respect to them enters its
 * product with W0 as bf16, over the row's largest entry (which is then exact).
 * Requires K % 64 == 0, 64 <= K <= 16384, 1 <= V <= 2^20, 1 <= kt <= 128,
 * M K < 2^31 and V K < 2^31; H, W0, dH and ws 16-byte aligned.  M = 0 is a no-op.
 */
int lq_head_loss(const void* H, int64_t M, const lq_weight* W0, const int32_t* targets,
                 const float* p, int32_t kt, const float* w, float logit_scale, float* loss,
                 float* lse, void* dH, void* ws, size_t ws_bytes, hipStream_t stream);

/* Workspace in bytes; 0 for M = 0 and for sizes that the call refuses.  The
 * workspace of M rows is enough for fewer. */
size_t lq_head_loss_workspace(int64_t M, int64_t V, int64_t K, int32_t kt, int32_t need_dh);

#ifdef __cplusplus
}
#endif
#endif /* LQ_BLOCK_H */
