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
// all tensors with the grid's stride, so sizes do not matter.  A thread has eight loads
// of 16 bytes in flight, four CTAs an SM (two: 598 for 584 us; six with four loads: 585;
// loads of 32 bytes for fp32: 630).  The clipping walks the chunks backwards: what the
// norm read last still lies in the L2 (loads that mark lines for eviction: 990 for 976 us).
// Where nothing is clipped in place, it reads the norm and ends.
// Beyond 1000 tensors a call is several launches of alike many: the later ones read what
// no launch of the call writes, so they begin beside the one before and wait for it at
// their end (1200 tensors of 25,000: 40 -> 33 us for the norm, 27 with the loads above).
//   24 tensors, 1.07 G elements: norm 584 us in fp32 (1.08 of a copy's rate), 302 in bf16
//   and clipping bf16 to bf16 976 together (1.00), 0.54 G fp32 to bf16 788 (1.02)
//   1200 tensors of 25,000: norm 27 us (fp32), with nothing to clip 37; bf16 clipped 42
//   (the floors are 18, 18 and 27: launches of 32 KB of parameters are the rest)
// Each chunk's tensor comes from kernel parameters: from device memory the compiler has
// to take it for different in each thread (norm of 1.07 G fp32 elements: 1130 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstring>

#include "grad_clip.cuh"
#include "grouped_elementwise.cuh"
#include "moe_kernels.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kCtas = 4;  // of an SM
constexpr int kLoads = 8;                 // of 16 bytes, in flight in a thread

// Elements of a 16-byte vector, and vectors of a thread in a chunk.
template <int TYPE>
constexpr int kWidth = TYPE == 2 ? 4 : 8;
template <int TYPE>
constexpr int kVecs = static_cast<int>(kGradChunk / (kWidth<TYPE> * kThreads));
static_assert(kVecs<0> % kLoads == 0 && kVecs<2> % kLoads == 0, "whole batches");

template <int N>
struct Table {
  int n, chunks;
  bool in_place;  // all of them
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

template <int TYPE>
__device__ __forceinline__ void values(const uint4& raw, float (&f)[kWidth<TYPE>]) {
  if constexpr (TYPE == 2)
    f[0] = __uint_as_float(raw.x), f[1] = __uint_as_float(raw.y), f[2] = __uint_as_float(raw.z), f[3] = __uint_as_float(raw.w);
  else
    unpack8<TYPE == 1>(raw, f);
}

template <int W>
__device__ __forceinline__ void put(void* p, int type, int64_t i, const float (&v)[W]) {
  if (type == 2) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
#pragma unroll
    for (int j = 0; j < W / 4; ++j) q[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + i;
    if constexpr (W == 8) {
      *reinterpret_cast<uint4*>(q) = type == 1 ? pack8<true>(v) : pack8<false>(v);
    } else {
      union {
        __half2 h[2];
        __nv_bfloat162 b[2];
        uint2 u;
      } o;
      if (type == 1)
        o.h[0] = __floats2half2_rn(v[0], v[1]), o.h[1] = __floats2half2_rn(v[2], v[3]);
      else
        o.b[0] = __floats2bfloat162_rn(v[0], v[1]), o.b[1] = __floats2bfloat162_rn(v[2], v[3]);
      *reinterpret_cast<uint2*>(q) = o.u;
    }
  }
}

// The loads of a batch: vectors a CTA's width apart, those beyond n read as zeros.
template <int TYPE, bool WHOLE>
__device__ __forceinline__ void load_batch(const void* base, int b, int n, uint4 (&raw)[kLoads]) {
  const uint4* p = static_cast<const uint4*>(base);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = (b + i) * kThreads + threadIdx.x;
    if (WHOLE || (at + 1) * kWidth<TYPE> <= n)
      raw[i] = __ldcg(p + at);
    else
      raw[i] = make_uint4(0, 0, 0, 0);
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
#pragma unroll
  for (int i = 0; i < 8; ++i) far += static_cast<double>(f[i]) * static_cast<double>(f[i]);
}

template <int TYPE, bool WHOLE>
__device__ __forceinline__ void vector_squares(const void* src, int n, float& part, double& far) {
#pragma unroll 1
  for (int b = 0; b < kVecs<TYPE>; b += kLoads) {
    if (!WHOLE && b * kThreads * kWidth<TYPE> >= n) break;
    uint4 raw[kLoads];
    load_batch<TYPE, WHOLE>(src, b, n, raw);
#pragma unroll
    for (int i = 0; i < kLoads; i += 8 / kWidth<TYPE>) {
      float f[8];
      if constexpr (TYPE == 2) {
        float lo[4], hi[4];
        values<2>(raw[i], lo);
        values<2>(raw[i + 1], hi);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = lo[j], f[4 + j] = hi[j];
      } else {
        values<TYPE>(raw[i], f);
      }
      add_squares<TYPE>(f, part, far);
    }
  }
}

template <int TYPE>
__device__ __forceinline__ double chunk_squares(const GradTensor& t, int64_t from) {
  constexpr int kSize = TYPE == 2 ? 4 : 2;
  const void* src = static_cast<const char*>(t.src) + from * kSize;
  const int n = static_cast<int>(min(t.n - from, kGradChunk));
  float part = 0.0f;
  double far = 0.0;
  if (t.vec && n == kGradChunk) {
    vector_squares<TYPE, true>(src, n, part, far);
  } else if (t.vec) {
    vector_squares<TYPE, false>(src, n, part, far);
    const int at = n / kWidth<TYPE> * kWidth<TYPE> + threadIdx.x;
    if (at < n) {
      const double x = value_at<TYPE>(src, at);
      far += x * x;
    }
  } else {
#pragma unroll 1
    for (int at = threadIdx.x; at < n; at += 8 * kThreads) {  // 8 elements a CTA's width apart
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = at + j * kThreads < n ? value_at<TYPE>(src, at + j * kThreads) : 0.0f;
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
__global__ void __launch_bounds__(kThreads, kCtas) grad_squares_kernel(const __grid_constant__ Table<N> table, double* partials,
                                                                float* norm, bool first) {
  if (first) {
    pdl_wait();
    pdl_launch_dependents();
  }
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
  if (!first) {
    pdl_wait();
    pdl_launch_dependents();
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

template <int TYPE, bool WHOLE>
__device__ __forceinline__ void clip_vectors(const void* src, void* dst, int dst_type, int n, float factor) {
#pragma unroll 1
  for (int b = 0; b < kVecs<TYPE>; b += kLoads) {
    if (!WHOLE && b * kThreads * kWidth<TYPE> >= n) break;
    uint4 raw[kLoads];
    load_batch<TYPE, WHOLE>(src, b, n, raw);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = ((b + i) * kThreads + threadIdx.x) * kWidth<TYPE>;
      float f[kWidth<TYPE>];
      values<TYPE>(raw[i], f);
#pragma unroll
      for (int j = 0; j < kWidth<TYPE>; ++j) f[j] = __fmul_rn(f[j], factor);
      if (WHOLE || at + kWidth<TYPE> <= n) put(dst, dst_type, at, f);
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void clip_chunk(const GradTensor& t, int64_t from, float factor) {
  const void* src = static_cast<const char*>(t.src) + from * (TYPE == 2 ? 4 : 2);
  void* dst = static_cast<char*>(t.dst) + from * (t.dst_type == 2 ? 4 : 2);
  const int n = static_cast<int>(min(t.n - from, kGradChunk));
  const bool vec = t.vec && t.dst_vec;
  if (vec && n == kGradChunk) {
    clip_vectors<TYPE, true>(src, dst, t.dst_type, n, factor);
  } else if (vec) {
    clip_vectors<TYPE, false>(src, dst, t.dst_type, n, factor);
    const int at = n / kWidth<TYPE> * kWidth<TYPE> + threadIdx.x;
    if (at < n) put_at(dst, t.dst_type, at, __fmul_rn(value_at<TYPE>(src, at), factor));
  } else {
#pragma unroll 1
    for (int at = threadIdx.x; at < n; at += 8 * kThreads) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = at + j * kThreads < n ? value_at<TYPE>(src, at + j * kThreads) : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j * kThreads < n) put_at(dst, t.dst_type, at + j * kThreads, __fmul_rn(f[j], factor));
    }
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, kCtas) grad_clip_kernel(const __grid_constant__ Table<N> table, const float* norm,
                                                             double max_norm, double eps, bool first) {
  if (first) {
    pdl_wait();
    pdl_launch_dependents();
  }
  const float total = __ldcg(norm);
  float factor = 1.0f;
  if (total < __int_as_float(0x7F800000)) {  // (a norm that is no number clips nothing)
    const double f = max_norm / (static_cast<double>(total) + eps);
    if (f < 1.0) factor = static_cast<float>(f);
  }
  const bool nothing = factor == 1.0f && table.in_place;
  for (int i = nothing ? table.chunks : blockIdx.x; i < table.chunks; i += gridDim.x) {
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
  if (!first) {
    pdl_wait();
    pdl_launch_dependents();
  }
}

// ------------------------------------------------------------------ launches

// Calls f(table, CTAs) for each launch's tensors.
template <int N, typename F>
cudaError_t each_launch(const GradTensor* t, int64_t n, int num_sms, F&& f) {
  const int64_t launches = (n + N - 1) / N, each = launches > 0 ? (n + launches - 1) / launches : 1;
  for (int64_t i = 0; i < n; i += each) {
    Table<N> table;
    table.n = static_cast<int>(n - i < each ? n - i : each);
    std::memcpy(table.t, t + i, table.n * sizeof(GradTensor));
    table.chunks = 0;
    table.in_place = true;
    for (int j = 0; j < table.n; ++j) {
      table.t[j].first = table.chunks;
      table.chunks += static_cast<int>((table.t[j].n + kGradChunk - 1) / kGradChunk);
      if (table.t[j].dst != table.t[j].src) table.in_place = false;
    }
    int ctas = num_sms * kCtas < kGradCtas ? num_sms * kCtas : kGradCtas;
    if (ctas > table.chunks) ctas = table.chunks;
    const cudaError_t e = f(table, ctas, i == 0);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N>
cudaError_t norm_of(const GradTensor* t, int64_t n, float* norm, double* partials, int num_sms, cudaStream_t stream) {
  int sums = 0;
  const bool alone = n <= N;
  bool done = false;
  cudaError_t e = each_launch<N>(t, n, num_sms, [&](const Table<N>& table, int ctas, bool first) {
    done = alone && ctas == 1;
    double* to = partials + sums;
    sums += ctas;
    return launch_pdl(grad_squares_kernel<N>, dim3(ctas), dim3(kThreads), 0, stream, table, to,
                      done ? norm : static_cast<float*>(nullptr), first);
  });
  if (e != cudaSuccess || done) return e;
  return launch_pdl(grad_norm_kernel, dim3(1), dim3(kThreads), 0, stream, static_cast<const double*>(partials), sums, norm);
}

template <int N>
cudaError_t clip(const GradTensor* t, int64_t n, const float* norm, double max_norm, double eps, int num_sms,
                 cudaStream_t stream) {
  return each_launch<N>(t, n, num_sms, [&](const Table<N>& table, int ctas, bool first) {
    return launch_pdl(grad_clip_kernel<N>, dim3(ctas), dim3(kThreads), 0, stream, table, norm, max_norm, eps, first);
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
