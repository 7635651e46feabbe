// Launchers of the operators around an adapted projection (lq_block.h), called
// by the ABI layer.  Arguments are already validated.
#pragma once

#include "../../include/lq_block.h"
#include "common.h"

namespace lq {
namespace dispatch {

size_t rmsnorm_part_bytes(int64_t M, int64_t K);
int rmsnorm_fwd(const void* X, const void* R, int64_t M, int64_t K, lq_dtype dt, const void* W,
                lq_dtype wdt, float eps, void* H, void* Y, int32_t fmt, uint8_t* codes,
                uint8_t* scales, float* rstd, hipStream_t st);
int rmsnorm_bwd(const void* dY, const void* H, int64_t M, int64_t K, lq_dtype dt, const void* W,
                lq_dtype wdt, float eps, const float* rstd, const void* dH, void* dX, float* dW,
                int accumulate, float* part, hipStream_t st);

size_t adapters_fwd_ws(int64_t M, int64_t N, int64_t K, int64_t r, int32_t slots);
size_t adapters_bwd_ws(int64_t M, int64_t N, int64_t K, int64_t r, int32_t slots);
int adapters_fwd(const void* X, int64_t M, const lq_adapter_pool& q, const int32_t* rows,
                 const void* Y_in, void* Y_out, float* T_out, void* ws, hipStream_t st);
int adapters_bwd(const void* dY, const void* X, int64_t M, const lq_adapter_pool& q,
                 const int32_t* rows, const float* T_saved, const void* dX_in, void* dX_out,
                 float* dA, float* dB, int accumulate, void* ws, hipStream_t st);

size_t head_loss_ws(int64_t M, int64_t V, int64_t K, int32_t kt, bool need_dh);
int head_loss(const void* H, int64_t M, int64_t V, int64_t K, const void* W, const int32_t* t,
              const float* p, int32_t kt, const float* w, float scale, float* loss, float* lse,
              void* dH, void* ws, hipStream_t st);

}  // namespace dispatch
}  // namespace lq
