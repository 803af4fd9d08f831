// k_grad_clip.cu -- the norm of all elements of many tensors, and the tensors times
//   f = min(1, max_norm / (norm + eps))
// the step between the gradients and the optimizer.  bf16, fp16 and fp32 tensors of
// any size together.
//
// Squares are summed in fp32 for 64 elements at most, the rest in fp64; the CTAs' sums
// are added in a fixed order.  A vector of 8 whose squares leave fp32's normal range
// (magnitudes above 2^60 or all below 2^-45) is summed in fp64, so no finite
// gradients overflow and none vanish.
//
// HBM-bound.  Tensors are cut into chunks of 16384 elements; CTAs walk the chunks of
// all tensors with the grid's stride, so sizes do not matter.  The clipping walks them
// backwards: what the norm read last still lies in the L2.  Where nothing is clipped
// in place, it reads the norm and ends.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "grad_clip.cuh"
#include "grouped_elementwise.cuh"
#include "moe_kernels.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kVecs = static_cast<int>(kGradChunk / (8 * kThreads)), kBatch = 4;
static_assert(kVecs % kBatch == 0, "whole batches");

template <int N>
struct Table {
  int n, chunks;
  GradTensor t[N];
};

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& table, int chunk) {
  int lo = 0, hi = table.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (table.t[mid].first <= chunk)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <int TYPE>
struct Vec {  // 8 elements
  uint4 raw[TYPE == 2 ? 2 : 1];
  __device__ __forceinline__ void load(const void* base, int64_t at, bool keep) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (TYPE == 2 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (TYPE == 2 ? 2 : 1); ++i) raw[i] = keep ? __ldcg(p + i) : __ldcs(p + i);
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    if constexpr (TYPE == 2) {
      const uint4 &a = raw[0], &b = raw[1];
      f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
      f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
    } else {
      unpack8<TYPE == 1>(raw[0], f);
    }
  }
};

template <int TYPE>
__device__ __forceinline__ float value_at(const void* p, int64_t i) {
  if (TYPE == 2) return static_cast<const float*>(p)[i];
  if (TYPE == 1) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ void put_at(void* p, int type, int64_t i, float v) {
  if (type == 2)
    static_cast<float*>(p)[i] = v;
  else if (type == 1)
    static_cast<__half*>(p)[i] = __float2half_rn(v);
  else
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void put8(void* p, int type, int64_t i, const float (&v)[8]) {
  if (type == 2) {
    uint4* q = reinterpret_cast<uint4*>(static_cast<float*>(p) + i);
    q[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    q[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = type == 1 ? pack8<true>(v) : pack8<false>(v);
  }
}

// ------------------------------------------------------------------ norm

// What 8 squares add: to `part` in fp32, or to `far` in fp64.
template <int TYPE>
__device__ __forceinline__ void add_squares(const float (&f)[8], float& part, double& far) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s = __fmaf_rn(f[i], f[i], s);
  if (TYPE == 1 || (s < 0x1p120f && s > 0x1p-90f)) {  // (fp16's squares all lie inside)
    part += s;
    return;
  }
  float top = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(f[i]));
  if (s == 0.0f && top == 0.0f) return;  // zeros
#pragma unroll 1
  for (int i = 0; i < 8; ++i) far += static_cast<double>(f[i]) * static_cast<double>(f[i]);
}

template <int TYPE>
__device__ __forceinline__ double chunk_squares(const GradTensor& t, int64_t from) {
  const int64_t n = min(t.n - from, kGradChunk);
  float part = 0.0f;
  double far = 0.0;
  if (t.vec) {
#pragma unroll
    for (int b = 0; b < kVecs; b += kBatch) {
      Vec<TYPE> v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t at = static_cast<int64_t>((b + i) * kThreads + threadIdx.x) * 8;
        if (at + 8 <= n) v[i].load(t.src, from + at, true);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t at = static_cast<int64_t>((b + i) * kThreads + threadIdx.x) * 8;
        float f[8];
        if (at + 8 <= n) {
          v[i].values(f);
        } else if (at < n) {
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = at + j < n ? value_at<TYPE>(t.src, from + at + j) : 0.0f;
        } else {
          continue;
        }
        add_squares<TYPE>(f, part, far);
      }
    }
  } else {
    for (int64_t at = threadIdx.x; at < n; at += 8 * kThreads) {  // 8 elements a CTA's width apart
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = at + j * kThreads < n ? value_at<TYPE>(t.src, from + at + j * kThreads) : 0.0f;
      add_squares<TYPE>(f, part, far);
    }
  }
  return static_cast<double>(part) + far;
}

// the sum over the CTA, in thread 0
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warp_sum[kThreads / 32];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < kThreads / 32; ++w) v += warp_sum[w];
  return v;
}

// norm: written where this CTA is the only one
template <int N>
__global__ void __launch_bounds__(kThreads) grad_squares_kernel(const __grid_constant__ Table<N> table, double* partials,
                                                                float* norm) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
  for (int c = blockIdx.x; c < table.chunks; c += gridDim.x) {
    const GradTensor& t = table.t[tensor_of(table, c)];
    const int64_t from = static_cast<int64_t>(c - t.first) * kGradChunk;
    sum += t.type == 2 ? chunk_squares<2>(t, from) : t.type == 1 ? chunk_squares<1>(t, from) : chunk_squares<0>(t, from);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) {
    partials[blockIdx.x] = sum;
    if (norm) *norm = static_cast<float>(sqrt(sum));
  }
}

__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const double* partials, int n, float* norm) {
  pdl_wait();
  pdl_launch_dependents();
  double sum = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kThreads) sum += __ldcg(partials + i);
  sum = block_sum(sum);
  if (threadIdx.x == 0) *norm = static_cast<float>(sqrt(sum));
}

// ------------------------------------------------------------------ clipping

template <int TYPE>
__device__ __forceinline__ void clip_chunk(const GradTensor& t, int64_t from, float factor) {
  const int64_t n = min(t.n - from, kGradChunk);
  if (t.vec && t.dst_vec) {
#pragma unroll 1
    for (int b = 0; b < kVecs; b += kBatch) {
      Vec<TYPE> v[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t at = static_cast<int64_t>((b + i) * kThreads + threadIdx.x) * 8;
        if (at + 8 <= n) v[i].load(t.src, from + at, false);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int64_t at = static_cast<int64_t>((b + i) * kThreads + threadIdx.x) * 8;
        if (at + 8 <= n) {
          float f[8];
          v[i].values(f);
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], factor);
          put8(t.dst, t.dst_type, from + at, f);
        } else {
          for (int64_t j = at; j < n; ++j) put_at(t.dst, t.dst_type, from + j, __fmul_rn(value_at<TYPE>(t.src, from + j), factor));
        }
      }
    }
  } else {
    for (int64_t at = threadIdx.x; at < n; at += 8 * kThreads) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = at + j * kThreads < n ? value_at<TYPE>(t.src, from + at + j * kThreads) : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j * kThreads < n) put_at(t.dst, t.dst_type, from + at + j * kThreads, __fmul_rn(f[j], factor));
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads) grad_clip_kernel(const __grid_constant__ Table<N> table, const float* norm,
                                                             double max_norm, double eps) {
  pdl_wait();
  pdl_launch_dependents();
  const float total = __ldcg(norm);
  float factor = 1.0f;
  if (total < __int_as_float(0x7F800000)) {  // (a norm that is no number clips nothing)
    const double f = max_norm / (static_cast<double>(total) + eps);
    if (f < 1.0) factor = static_cast<float>(f);
  }
  for (int i = blockIdx.x; i < table.chunks; i += gridDim.x) {
    const int c = table.chunks - 1 - i;
    const GradTensor& t = table.t[tensor_of(table, c)];
    if (factor == 1.0f && t.dst == t.src) continue;
    const int64_t from = static_cast<int64_t>(c - t.first) * kGradChunk;
    if (t.type == 2)
      clip_chunk<2>(t, from, factor);
    else if (t.type == 1)
      clip_chunk<1>(t, from, factor);
    else
      clip_chunk<0>(t, from, factor);
  }
}

// ------------------------------------------------------------------ launches

// Calls f(table, CTAs) for each launch's tensors.
template <int N, typename F>
cudaError_t each_launch(const GradTensor* t, int64_t n, int num_sms, F&& f) {
  for (int64_t i = 0; i < n; i += N) {
    Table<N> table;
    table.n = static_cast<int>(n - i < N ? n - i : N);
    std::memcpy(table.t, t + i, table.n * sizeof(GradTensor));
    const GradTensor& last = table.t[table.n - 1];
    table.chunks = last.first + static_cast<int>((last.n + kGradChunk - 1) / kGradChunk);
    int ctas = num_sms * 4 < kGradCtas ? num_sms * 4 : kGradCtas;
    if (ctas > table.chunks) ctas = table.chunks;
    const cudaError_t e = f(table, ctas);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
cudaError_t norm_of(const GradTensor* t, int64_t n, float* norm, double* partials, int num_sms, cudaStream_t stream) {
  int sums = 0;
  const bool alone = n <= N;
  bool done = false;
  cudaError_t e = each_launch<N>(t, n, num_sms, [&](const Table<N>& table, int ctas) {
    done = alone && ctas == 1;
    double* to = partials + sums;
    sums += ctas;
    return launch_pdl(grad_squares_kernel<N>, dim3(ctas), dim3(kThreads), 0, stream, table, to,
                      done ? norm : static_cast<float*>(nullptr));
  });
  if (e != cudaSuccess || done) return e;
  return launch_pdl(grad_norm_kernel, dim3(1), dim3(kThreads), 0, stream, static_cast<const double*>(partials), sums, norm);
}

template <int N>
cudaError_t clip(const GradTensor* t, int64_t n, const float* norm, double max_norm, double eps, int num_sms,
                 cudaStream_t stream) {
  return each_launch<N>(t, n, num_sms, [&](const Table<N>& table, int ctas) {
    return launch_pdl(grad_clip_kernel<N>, dim3(ctas), dim3(kThreads), 0, stream, table, norm, max_norm, eps);
  });
}

}  // namespace

cudaError_t launch_grad_norm(const GradTensor* t, int64_t n, float* norm, double* partials, int num_sms,
                             cudaStream_t stream) {
  return n <= kGradFew ? norm_of<kGradFew>(t, n, norm, partials, num_sms, stream)
                       : norm_of<kGradTensors>(t, n, norm, partials, num_sms, stream);
}

cudaError_t launch_grad_clip(const GradTensor* t, int64_t n, const float* norm, double max_norm, double eps, int num_sms,
                             cudaStream_t stream) {
  return n <= kGradFew ? clip<kGradFew>(t, n, norm, max_norm, eps, num_sms, stream)
                       : clip<kGradTensors>(t, n, norm, max_norm, eps, num_sms, stream);
}

}  // namespace moe
