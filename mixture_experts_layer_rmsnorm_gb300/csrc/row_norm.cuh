// row_norm.cuh -- RMS norm and layer norm of rows, and their gradients (internal).
#pragma once

#include <cuda_runtime.h>
#include <cstdint>

namespace moe {

constexpr int kNormMaxH = 16384;
// CTAs of the gradient kernel at most: each leaves a partial sum of the weight's (and bias's) gradient
__host__ __device__ constexpr int norm_max_ctas(int H) { return H <= 1024 ? 1280 : H <= 4096 ? 640 : 320; }

struct RowNormArgs {
  int64_t rows;
  int H;
  float eps;
  int type;         // of x, y, dy, dx: 0 bf16, 1 fp16, 2 fp32
  int weight_type;  // of weight, bias: `type` or 2
  const void* x;
  int64_t ldx;
  const void* weight;  // [H], or null: ones
  const void* bias;    // layer norm: [H], or null
  void* y;             // forward
  int64_t ldy;
  float* mean;  // [rows]; forward: written unless null
  float* rstd;
  // gradient
  const void* dy;
  int64_t lddy;
  void* dx;
  int64_t lddx;
  void* dweight;  // [H] of dweight_type, or null
  void* dbias;
  int dweight_type;
  int accumulate;   // dweight, dbias (fp32): added to what they hold
  float* partials;  // [norm_max_ctas(H)][2][H]
};
cudaError_t launch_row_norm(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream);
cudaError_t launch_row_norm_grad(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream);

}  // namespace moe
