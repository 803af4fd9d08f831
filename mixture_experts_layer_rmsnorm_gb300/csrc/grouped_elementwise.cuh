// grouped_elementwise.cuh -- 16-byte vectors of bf16 / fp16 and their fp32 values.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace moe {

cudaError_t launch_swiglu(bool fp16, const void* h, int64_t ldh, void* act, int64_t ldact, int64_t rows, int I,
                          cudaStream_t stream);
cudaError_t launch_swiglu_grad(bool fp16, const void* h, int64_t ldh, const void* dact, int64_t lddact, void* dh,
                               int64_t lddh, int64_t rows, int I, cudaStream_t stream);

#ifdef __CUDACC__

template <bool FP16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (FP16) {
      const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = p.x;
      f[2 * i + 1] = p.y;
    } else {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}

template <bool FP16>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (FP16) {
      const __half2 p = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    } else {
      const __nv_bfloat162 p = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

#endif  // __CUDACC__

}  // namespace moe
