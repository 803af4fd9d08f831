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
// Where nothing is clipped in place, it ends there.  Norm and clipping in one call: each CTA
// of the clipping adds the sums itself (a launch less; one warp does, see block_sum).
// Beyond 1600 tensors (1150 into others) a call is several launches of alike many: the later
// ones read what no launch of the call writes, so they begin beside the one before and wait
// for it at their end (two launches for 1200 tensors of 25,000: 40 -> 33 us for the norm).
//   24 tensors, 1.07 G elements: norm 590 us in fp32 (1.07 of a copy's rate), 302 in bf16;
//   with the clipping, bf16 to bf16 971 (0.98), 0.54 G fp32 to bf16 788 (1.00)
//   1200 tensors of 25,000: norm 25 us (fp32), and nothing to clip 27; bf16 clipped 38
//   (the floors are 18, 18 and 27: launches of 32 KB of parameters are the rest)
// Each chunk's tensor comes from kernel parameters, alike for all threads.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

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

// The tensors of a launch, packed.
template <int N, bool APART>
struct Table {
  int n, chunks;
  bool in_place;        // all of them
  int first[N];         // a tensor's first chunk
  uint64_t meta[N];     // elements (48 bits), type (2), dst_type (2), vec, dst_vec
  const void* src[N];
  void* dst[APART ? N : 1];

  void put(int i, const GradTensor& t) {
    first[i] = chunks;
    meta[i] = static_cast<uint64_t>(t.n) | static_cast<uint64_t>(t.type) << 48 | static_cast<uint64_t>(t.dst_type) << 50 |
              static_cast<uint64_t>(t.vec) << 52 | static_cast<uint64_t>(t.dst_vec) << 53;
    src[i] = t.src;
    if (APART) dst[i] = t.dst;
    chunks += static_cast<int>((t.n + kGradChunk - 1) / kGradChunk);
    if (t.dst != t.src) in_place = false;
  }
  __device__ __forceinline__ GradTensor get(int i) const {
    const uint64_t m = meta[i];
    GradTensor t;
    t.src = src[i];
    t.dst = APART ? dst[i] : const_cast<void*>(src[i]);
    t.n = static_cast<int64_t>(m & 0xFFFFFFFFFFFFull);
    t.type = m >> 48 & 3, t.dst_type = m >> 50 & 3, t.vec = m >> 52 & 1, t.dst_vec = m >> 53 & 1;
    return t;
  }
};

template <typename T>
__device__ __forceinline__ int tensor_of(const T& table, int chunk) {
  int lo = 0, hi = table.n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (table.first[mid] <= chunk)
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

// What 8 squares add: to `part` in fp32, or to `sum` in fp64.
template <int TYPE>
__device__ __forceinline__ void add_squares(const float (&f)[8], float& part, double& sum) {
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
  for (int i = 0; i < 8; ++i) sum += static_cast<double>(f[i]) * static_cast<double>(f[i]);
}

template <int TYPE, bool WHOLE>
__device__ __forceinline__ void vector_squares(const void* src, int n, float& part, double& sum) {
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
      add_squares<TYPE>(f, part, sum);
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void chunk_squares(const GradTensor& t, int64_t from, double& sum) {
  constexpr int kSize = TYPE == 2 ? 4 : 2;
  const void* src = static_cast<const char*>(t.src) + from * kSize;
  const int n = static_cast<int>(min(t.n - from, kGradChunk));
  float part = 0.0f;
  if (t.vec && n == kGradChunk) {
    vector_squares<TYPE, true>(src, n, part, sum);
  } else if (t.vec) {
    vector_squares<TYPE, false>(src, n, part, sum);
    const int at = n / kWidth<TYPE> * kWidth<TYPE> + threadIdx.x;
    if (at < n) {
      const double x = value_at<TYPE>(src, at);
      sum += x * x;
    }
  } else {
#pragma unroll 1
    for (int at = threadIdx.x; at < n; at += 8 * kThreads) {  // 8 elements a CTA's width apart
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = at + j * kThreads < n ? value_at<TYPE>(src, at + j * kThreads) : 0.0f;
      add_squares<TYPE>(f, part, sum);
    }
  }
  sum += static_cast<double>(part);
}

// The sum over the CTA, in warp 0's threads, in a fixed order.  (An SM adds about two fp64
// numbers a clock, so 13 additions of one warp are cheaper than 5 of each and 8.)
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double all[kThreads];
  all[threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.x >= 32) return 0.0;
  v = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) v += all[w * 32 + threadIdx.x];
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  return v;
}

// The norm from n partial sums, by one warp, alike in every CTA.
__device__ __forceinline__ double norm_of_sums(const double* partials, int n) {
  double sum = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < n; i += 32) sum += __ldcg(partials + i);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  return sqrt(sum);
}

// norm: written where this CTA is the only one
template <int N, bool APART>
__global__ void __launch_bounds__(kThreads, kCtas)
    grad_squares_kernel(const __grid_constant__ Table<N, APART> table, double* partials, float* norm, bool first) {
  if (first) {
    pdl_wait();
    pdl_launch_dependents();
  }
  double sum = 0.0;
  for (int c = blockIdx.x; c < table.chunks; c += gridDim.x) {
    const int at = tensor_of(table, c);
    const GradTensor t = table.get(at);
    const int64_t from = static_cast<int64_t>(c - table.first[at]) * kGradChunk;
    if (t.type == 2)
      chunk_squares<2>(t, from, sum);
    else if (t.type == 1)
      chunk_squares<1>(t, from, sum);
    else
      chunk_squares<0>(t, from, sum);
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

__global__ void __launch_bounds__(32) grad_norm_kernel(const double* partials, int n, float* norm) {
  pdl_wait();
  pdl_launch_dependents();
  const double total = norm_of_sums(partials, n);
  if (threadIdx.x == 0) *norm = static_cast<float>(total);
}

// ------------------------------------------------------------------ clipping

// The factor f < 1 in two: below fp32's normal numbers, where f would lose bits (all below 2^-149, although f times a large
// element is an ordinary number), it is `first`, 1 at most, times a power of two.
struct Factor {
  float first, last;

  __device__ explicit Factor(double f) : first(1.0f), last(1.0f) {
    if (!(f < 1.0)) return;
    if (f >= 0x1p-126 || f == 0.0) {
      first = static_cast<float>(f);
      return;
    }
    int e;
    const double m = frexp(f, &e);  // m in [0.5, 1)
    const int last_e = e > -149 ? e : -149;
    first = static_cast<float>(ldexp(m, e - last_e));
    last = static_cast<float>(ldexp(1.0, last_e));
  }
  __device__ Factor(float first_, float last_) : first(first_), last(last_) {}
  __device__ __forceinline__ float times(float x) const { return __fmul_rn(__fmul_rn(x, first), last); }
};

template <int TYPE, bool WHOLE>
__device__ __forceinline__ void clip_vectors(const void* src, void* dst, int dst_type, int n, Factor factor) {
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
      for (int j = 0; j < kWidth<TYPE>; ++j) f[j] = factor.times(f[j]);
      if (WHOLE || at + kWidth<TYPE> <= n) put(dst, dst_type, at, f);
    }
  }
}

template <int TYPE>
__device__ __forceinline__ void clip_chunk(const GradTensor& t, int64_t from, Factor factor) {
  const void* src = static_cast<const char*>(t.src) + from * (TYPE == 2 ? 4 : 2);
  void* dst = static_cast<char*>(t.dst) + from * (t.dst_type == 2 ? 4 : 2);
  const int n = static_cast<int>(min(t.n - from, kGradChunk));
  const bool vec = t.vec && t.dst_vec;
  if (vec && n == kGradChunk) {
    clip_vectors<TYPE, true>(src, dst, t.dst_type, n, factor);
  } else if (vec) {
    clip_vectors<TYPE, false>(src, dst, t.dst_type, n, factor);
    const int at = n / kWidth<TYPE> * kWidth<TYPE> + threadIdx.x;
    if (at < n) put_at(dst, t.dst_type, at, factor.times(value_at<TYPE>(src, at)));
  } else {
#pragma unroll 1
    for (int at = threadIdx.x; at < n; at += 8 * kThreads) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = at + j * kThreads < n ? value_at<TYPE>(src, at + j * kThreads) : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j * kThreads < n) put_at(dst, t.dst_type, at + j * kThreads, factor.times(f[j]));
    }
  }
}

// sums > 0: from that many partial sums, and the first launch writes the norm; else the norm is read
template <int N, bool APART>
__global__ void __launch_bounds__(kThreads, kCtas)
    grad_clip_kernel(const __grid_constant__ Table<N, APART> table, const double* partials, int sums, float* norm,
                     double max_norm, double eps, bool first) {
  if (first) {
    pdl_wait();
    pdl_launch_dependents();
  }
  __shared__ float clipping[2];
  if (threadIdx.x < 32) {
    const double root = sums > 0 ? norm_of_sums(partials, sums) : __ldcg(norm);
    if (threadIdx.x == 0) {
      const float total = static_cast<float>(root);
      if (sums > 0 && first && blockIdx.x == 0) *norm = total;
      // The norm as the caller gets it, or, where finite elements have one beyond fp32, in 64 bits.  (One that is no number clips
      // nothing: an infinite or NaN gradient is for the caller to see in the norm, before or after.)
      const double by = total < __int_as_float(0x7F800000) ? total : root;
      const Factor f(by < __longlong_as_double(0x7FF0000000000000ll) ? max_norm / (by + eps) : 1.0);
      clipping[0] = f.first, clipping[1] = f.last;
    }
  }
  __syncthreads();
  const Factor factor(clipping[0], clipping[1]);
  const bool one = factor.first == 1.0f && factor.last == 1.0f;
  const bool nothing = one && table.in_place;
  for (int i = nothing ? table.chunks : blockIdx.x; i < table.chunks; i += gridDim.x) {
    const int c = table.chunks - 1 - i;
    const int at = tensor_of(table, c);
    const GradTensor t = table.get(at);
    if (one && t.dst == t.src) continue;
    const int64_t from = static_cast<int64_t>(c - table.first[at]) * kGradChunk;
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

// Calls f(table, CTAs, first launch) for each launch's tensors.
template <int N, bool APART, typename F>
cudaError_t each_launch(const GradTensor* t, int64_t n, int num_sms, F&& f) {
  static_assert(sizeof(Table<N, APART>) + 64 <= 32764, "a kernel's parameters");
  const int64_t launches = (n + N - 1) / N, each = launches > 0 ? (n + launches - 1) / launches : 1;
  for (int64_t i = 0; i < n; i += each) {
    Table<N, APART> table;
    table.n = static_cast<int>(n - i < each ? n - i : each);
    table.chunks = 0;
    table.in_place = true;
    for (int j = 0; j < table.n; ++j) table.put(j, t[i + j]);
    int ctas = num_sms * kCtas < kGradCtas ? num_sms * kCtas : kGradCtas;
    if (ctas > table.chunks) ctas = table.chunks;
    const cudaError_t e = f(table, ctas, i == 0);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

template <int N, bool APART>
cudaError_t squares(const Table<N, APART>& table, int ctas, double* partials, float* norm, bool first, cudaStream_t stream) {
  return launch_pdl(grad_squares_kernel<N, APART>, dim3(ctas), dim3(kThreads), 0, stream, table, partials, norm, first);
}

template <int N>
cudaError_t all_squares(const GradTensor* t, int64_t n, double* partials, int& sums, int num_sms, cudaStream_t stream) {
  sums = 0;
  return each_launch<N, false>(t, n, num_sms, [&](const Table<N, false>& table, int ctas, bool first) {
    sums += ctas;
    return squares(table, ctas, partials + (sums - ctas), nullptr, first, stream);
  });
}

template <int N>
cudaError_t norm_of(const GradTensor* t, int64_t n, float* norm, double* partials, int num_sms, cudaStream_t stream) {
  int sums = 0;
  bool done = false;
  cudaError_t e;
  if (n > 0 && n <= N) {
    e = each_launch<N, false>(t, n, num_sms, [&](const Table<N, false>& table, int ctas, bool first) {
      sums = ctas;
      done = ctas == 1;
      return squares(table, ctas, partials, done ? norm : nullptr, first, stream);
    });
  } else {
    e = all_squares<N>(t, n, partials, sums, num_sms, stream);
  }
  if (e != cudaSuccess || done) return e;
  return launch_pdl(grad_norm_kernel, dim3(1), dim3(32), 0, stream, static_cast<const double*>(partials), sums, norm);
}

// partials: null where the norm is there
template <int N, bool APART>
cudaError_t clip(const GradTensor* t, int64_t n, float* norm, double* partials, double max_norm, double eps, int num_sms,
                 cudaStream_t stream) {
  int sums = 0;
  if (partials && n > N) {
    const cudaError_t e = all_squares<kGradTensors>(t, n, partials, sums, num_sms, stream);
    if (e != cudaSuccess) return e;
  }
  return each_launch<N, APART>(t, n, num_sms, [&](const Table<N, APART>& table, int ctas, bool first) {
    if (partials && n <= N) {  // one table for both
      sums = ctas;
      const cudaError_t e = squares(table, ctas, partials, nullptr, first, stream);
      if (e != cudaSuccess) return e;
    }
    return launch_pdl(grad_clip_kernel<N, APART>, dim3(ctas), dim3(kThreads), 0, stream, table,
                      static_cast<const double*>(partials), sums, norm, max_norm, eps, first);
  });
}

}  // namespace

cudaError_t launch_grad_norm(const GradTensor* t, int64_t n, float* norm, double* partials, int num_sms,
                             cudaStream_t stream) {
  return n <= kGradFew ? norm_of<kGradFew>(t, n, norm, partials, num_sms, stream)
                          : norm_of<kGradTensors>(t, n, norm, partials, num_sms, stream);
}

cudaError_t launch_grad_clip(const GradTensor* t, int64_t n, float* norm, double* partials, double max_norm, double eps,
                             int num_sms, cudaStream_t stream) {
  if (n <= kGradFew) return clip<kGradFew, true>(t, n, norm, partials, max_norm, eps, num_sms, stream);
  bool apart = false;
  for (int64_t i = 0; i < n; ++i) apart = apart || t[i].dst != t[i].src;
  return apart ? clip<kGradApart, true>(t, n, norm, partials, max_norm, eps, num_sms, stream)
               : clip<kGradTensors, false>(t, n, norm, partials, max_norm, eps, num_sms, stream);
}

}  // namespace moe
