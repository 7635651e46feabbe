/*
 * lq_mx.h -- microscaled (MX) tensors for the adapted linear layer on AMD
 * Instinct MI355X (gfx950): 8-bit and 4-bit floating point with one
 * power-of-two scale per 32 elements, the form gfx950's matrix cores multiply
 * directly.  Part of liblq.so; the conventions of lq.h (row-major device
 * pointers owned by the caller, work enqueued on the caller's stream, no
 * allocation, no synchronisation, negative lq_status on a refused call,
 * lq_last_error()) hold here too.
 *
 * What it is for: the frozen base W0 in 4 bits without a table (MXFP4, 4.25
 * bits per weight), and the layer's input kept in 8 bits (MXFP8) for the
 * backward, the activation checkpoint.  A layer on an MXFP4 base multiplies
 * that same checkpoint in its forward, so the gradients of lq_mx_lora_bwd are
 * those of the forward as it was computed (the quantiser itself is taken as
 * the identity, the usual straight-through reading).
 */
#ifndef LQ_MX_H
#define LQ_MX_H

#include "lq.h"

#ifdef __cplusplus
extern "C" {
#endif

#define LQ_MX_BLOCK 32
/* Element formats (named by their bits):
 *   LQ_MX_FP4  E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives, code =
 *              sign << 3 | magnitude index; two codes per byte, element 2j in
 *              the low nibble
 *   LQ_MX_FP8  E4M3 (bias 7, subnormals m 2^-9, largest 448, 0x7F / 0xFF NaN) */
#define LQ_MX_FP4 4
#define LQ_MX_FP8 8

/*
 * A rows x cols matrix of MX elements.  Every row is padded to kp =
 * 32 ceil(cols / 32) columns; a block is 32 consecutive columns of one row.
 *   codes   rows x kp / 2 bytes (FP4) or rows x kp bytes (FP8), row-major;
 *           padding columns hold code 0
 *   scales  rows x kp / 32 bytes, row-major: scale byte b stands for
 *           2^(b - 127), b = 255 for NaN (every element of the block is NaN)
 * Element value = value of its code times its block's scale.
 * Consecutive rows of a tensor are a tensor: both pointers at their first row.
 * The layer's calls take codes at multiples of 16 bytes and scales at even
 * addresses, which every such row has where cols % 64 == 0.
 */
typedef struct lq_mx_tensor {
  int32_t format;            /* LQ_MX_FP4 / LQ_MX_FP8                            */
  int32_t reserved;          /* 0                                               */
  int64_t rows;
  int64_t cols;
  const uint8_t* codes;
  const uint8_t* scales;
} lq_mx_tensor;

/* Bytes of a tensor's two buffers (0 for a bad format, a negative size or more
 * elements than lq_mx_quantize takes). */
size_t lq_mx_codes_bytes(int32_t format, int64_t rows, int64_t cols);
size_t lq_mx_scales_bytes(int64_t rows, int64_t cols);

/*
 * Quantise X (rows x cols of xdt, LQ_BF16 or LQ_F32) into codes and scales
 * (laid out as in lq_mx_tensor).  Per block, with amax = max |x|:
 *   e = the smallest integer in [-127, 127] with amax <= largest 2^e (largest
 *       = 6 or 448), b = e + 127
 *   code = the element nearest x 2^-e, ties to the even code
 * so no element is clipped and every one is off by at most half a step.  (The
 * OCP MX text takes e from the exponent of amax alone, which clips the top of
 * a block; the stored format is the same.)  A block that holds an infinity or
 * a NaN gets b = 255 and zero codes.  Results are bit-exact functions of the
 * input.  rows, cols >= 1; at most 2^35 elements, padding included; X aligned
 * to its element, codes to 16 bytes (scales: any address here).
 */
int lq_mx_quantize(const void* X, lq_dtype xdt, int64_t rows, int64_t cols, int32_t format,
                   uint8_t* codes, uint8_t* scales, hipStream_t stream);

/*
 * Element values of q to ``out`` (rows x cols of odt, LQ_BF16 or LQ_F32).
 * Exact in both types, but for bf16 values below 2^-126, which are rounded
 * to nearest even, and values of 2^128 (elements rounded up at the top of
 * float32's range), which are infinite.
 */
int lq_mx_dequantize(const lq_mx_tensor* q, void* out, lq_dtype odt, hipStream_t stream);

/*
 * Forward of the layer on an MXFP4 base:
 *   Y = X W0^T + s (X A^T) B^T
 * with X either bf16 values (X, M x K; M <= LQ_MX_ROWS_BF16) or an MX tensor
 * (Xq, M x K, either format): exactly one of X and Xq is given.
 *   W0     N x K, LQ_MX_FP4
 *   A, B   r x K and N x r bf16; r = 0: no adapter (A and B unused)
 *   Y      M x N bf16
 *   T_out  optional M x r float32: receives T = X A^T for lq_mx_lora_bwd
 *   ws     lq_mx_workspace_size(LQ_MX_OP_FWD, M, N, K, r) bytes
 * Products are summed in float32; with an MX X they are formed by the scaled
 * matrix instructions, whose sums inside one group of 64 products keep about
 * 14 bits below the largest.  T is formed from the exact element values in
 * float32 and enters its product with B in two bf16 parts, 2^-16 of its value.
 * Requires K % 64 == 0, N % 64 == 0, N, K <= 65536, M K and M N < 2^31,
 * 0 <= r <= 64, every pointer 16-byte aligned but T_out (4) and the scales of
 * W0 and Xq (2; on multiples of 16, K % 512 == 0, they load fastest).  M = 0 is
 * a no-op.
 */
#define LQ_MX_ROWS_BF16 64
int lq_mx_lora_fwd(const void* X, const lq_mx_tensor* Xq, int64_t M, const lq_mx_tensor* W0,
                   const void* A, const void* B, int64_t r, float scale, void* Y, float* T_out,
                   void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * Backward of lq_mx_lora_fwd from the MX tensor its forward multiplied:
 *   dX = dY W0 + s (dY B) A      (optional, M x K bf16)
 *   dA = s (dY B)^T Xq           (r x K float32)
 *   dB = s dY^T T, T = Xq A^T    (N x r float32)
 * dA and dB are given together or both NULL (Xq and T_saved are then not
 * read, and Xq may be NULL); dX, dA and dB all NULL is refused.  accumulate =
 * 1 adds into dA and dB.  T_saved: T_out of the forward, or NULL (recomputed).
 *   ws  lq_mx_workspace_size(LQ_MX_OP_BWD, M, N, K, r) bytes (without dA and dB,
 *       LQ_MX_OP_BWD + LQ_MX_NO_GRADS)
 * The weight enters as its exact bf16 values, s U its product with A in two
 * bf16 parts (2^-16 of its value); dA and dB are sums in float32
 * of products with float32 T and U = dY B (carried as three bf16 parts, so
 * that nothing of their 24 bits is lost), in a fixed order.  1 <= r <= 64;
 * other rules as lq_mx_lora_fwd (T_saved: 16).  A non-finite element of dY or
 * Xq makes the sums it enters non-finite.  M = 0 writes zeros to dA and dB
 * unless accumulate is set.
 */
int lq_mx_lora_bwd(const void* dY, const lq_mx_tensor* Xq, int64_t M, const lq_mx_tensor* W0,
                   const void* A, const void* B, int64_t r, float scale, const float* T_saved,
                   void* dX, float* dA, float* dB, int32_t accumulate, void* ws,
                   size_t ws_bytes, hipStream_t stream);

/*
 * lq_lora_bwd (lq.h) from a checkpoint of the layer's input: the backward of
 * the dense bf16 or NF4 layer with Xq, the MX tensor of X, in the place of X.
 * dX does not depend on X: it is formed as lq_lora_bwd forms it, or for a dense
 * base where that is faster as lq_mx_lora_bwd does.  dA and dB (and T, where
 * T_saved is NULL) are those of the restored input, summed as in lq_mx_lora_bwd.
 *   ws  at least lq_mx_workspace_size(LQ_MX_OP_BWD_CKPT_FUSED, M, N, K, r) bytes
 *       (without dA and dB, + LQ_MX_NO_GRADS); lq_lora_bwd_ckpt_workspace bytes
 *       let dX take its fastest path, whose results may differ in their
 *       rounding.  LQ_MX_OP_BWD_CKPT is enough for that whatever W0 is: it holds
 *       a bf16 copy of W0, which only some NF4 weights use.
 * Other arguments and rules as lq_lora_bwd with dt = LQ_BF16.
 */
int lq_lora_bwd_ckpt(const void* dY, const lq_mx_tensor* Xq, int64_t M, const lq_weight* W0,
                     const void* A, const void* B, int64_t r, float scale, const float* T_saved,
                     void* dX, float* dA, float* dB, int32_t accumulate, void* ws,
                     size_t ws_bytes, hipStream_t stream);

/* Bytes with which lq_lora_bwd_ckpt takes its fastest path: of W0 only kind, N
 * and K are read; need_dx, need_grads: whether dX, and dA and dB, are given.  0
 * for sizes that the call refuses. */
size_t lq_lora_bwd_ckpt_workspace(int64_t M, const lq_weight* W0, int64_t r, int32_t need_dx,
                                  int32_t need_grads);

/* Workspace of an operator (LQ_MX_OP_*), in bytes; 0 where none is needed and
 * for sizes that the operator refuses.  LQ_MX_NO_GRADS added to a backward's op:
 * its calls without dA and dB. */
#define LQ_MX_OP_FWD 0
#define LQ_MX_OP_BWD 1
#define LQ_MX_OP_BWD_CKPT 2
#define LQ_MX_OP_BWD_CKPT_FUSED 3
#define LQ_MX_NO_GRADS 16
size_t lq_mx_workspace_size(int32_t op, int64_t M, int64_t N, int64_t K, int64_t r);

#ifdef __cplusplus
}
#endif
#endif /* LQ_MX_H */
