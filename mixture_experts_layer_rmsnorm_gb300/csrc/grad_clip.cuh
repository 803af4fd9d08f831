// grad_clip.cuh -- the norm of many tensors together, and their clipping (internal).
#pragma once

#include <cuda_runtime.h>
#include <cstddef>
#include <cstdint>

namespace moe {

struct GradTensor {
  const void* src;
  void* dst;
  int64_t n;
  uint8_t type, dst_type;  // 0 bf16, 1 fp16, 2 fp32
  uint8_t vec, dst_vec;    // addresses on 16-byte borders
};

// Tensors go to the kernels as parameters, so that a call is complete in itself (captured, replayed, several at
// once): as many of them as fit 32,764 bytes a launch, or kGradFew where that is all, since many bytes of parameters
// cost host time (norm and clipping in place, us on the host without / with kGradFew: 33 tensors 14.8 / 11.6, 300 18.7 /
// 14.5; but a still smaller table, of 32 tensors, costs more: 3 tensors 12.3 to 14.1 instead of 9.7 to 12.0).
constexpr int kGradTensors = 1600;  // of the norm, and clipped in place
constexpr int kGradApart = 1150;    // clipped into other tensors
constexpr int kGradFew = 300;
constexpr int kGradCtas = 640;       // of a launch, at most: a partial sum each
constexpr int64_t kGradChunk = 16384;  // elements

inline int64_t grad_launches(int64_t tensors) { return tensors > 0 ? (tensors + kGradTensors - 1) / kGradTensors : 1; }
inline size_t grad_partial_bytes(int64_t tensors) {
  return static_cast<size_t>(grad_launches(tensors)) * kGradCtas * sizeof(double);
}

// norm [1] from the tensors (empty ones left out)
cudaError_t launch_grad_norm(const GradTensor* t, int64_t n, float* norm, double* partials, int num_sms,
                             cudaStream_t stream);
// clipping by a norm that is there (partials null), or by the one that it computes and writes (n > 0)
cudaError_t launch_grad_clip(const GradTensor* t, int64_t n, float* norm, double* partials, double max_norm, double eps,
                             int num_sms, cudaStream_t stream);

}  // namespace moe
