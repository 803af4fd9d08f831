// k_row_norm.cu -- the norm of rows, as the layer's first step computes it inside
// its router kernel ("4 · La fusion de noyaux", §4.2 "Réduction + élémentaire"), here for separate rows, with the
// layer norm beside it and the gradients of both:
//   n = (x - m) r,  r = 1 / sqrt(mean((x - m)^2) + eps),  y = n w + b
// with m the row's mean (layer) or 0 (rms, no b); and from dy, with e = dy w:
//   dx = r (e - mean(e) - n mean(e n))   (rms: without mean(e))
//   dw = sum over the rows of dy n,  db = sum of dy
// All sums in fp32.  The layer norm's variance comes from x - m, and what m's own
// rounding leaves, mean(x - m), is taken out too: rows far from zero lose nothing.
//
// HBM-bound: 2 (forward) and 3 (gradient) elements moved per element.  A row is
// held by 8, 16 or 32 lanes (H <= 1024; several rows a warp or a warp a row) or by a
// CTA; a thread takes vectors of 8 elements, neighbouring lanes neighbouring ones.
//
// Gradient.  A CTA walks rows with the grid's stride and keeps its threads' columns
// of dw and db in registers; the sums of all CTAs are added by a second kernel in a
// fixed order, so results repeat bit for bit.  Between a row's sums and its dx lies a
// reduction, so the next rows are loaded before it, into registers, packed.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grouped_elementwise.cuh"
#include "launch_config.cuh"
#include "moe_kernels.cuh"
#include "pdl.cuh"
#include "row_norm.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;    // of CTAs whose rows are held by 8, 16 or 32 lanes
constexpr int kRowThreads = 512;  // of CTAs that hold a row each, at most

template <int TYPE>
constexpr size_t kSize = TYPE == 2 ? 4 : 2;

// 8 elements of a type as fp32, from global or shared memory (16-byte aligned)
template <int TYPE>
__device__ __forceinline__ void load8(const void* p, float (&f)[8]) {
  const uint4* q = static_cast<const uint4*>(p);
  if constexpr (TYPE == 2) {
    const uint4 a = q[0], b = q[1];
    f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
  } else {
    unpack8<TYPE == 1>(q[0], f);
  }
}

template <int TYPE>
__device__ __forceinline__ void store8(void* p, const float (&f)[8]) {
  uint4* q = static_cast<uint4*>(p);
  if constexpr (TYPE == 2) {
    q[0] = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    q[1] = make_uint4(__float_as_uint(f[4]), __float_as_uint(f[5]), __float_as_uint(f[6]), __float_as_uint(f[7]));
  } else {
    q[0] = pack8<TYPE == 1>(f);
  }
}

// the weight's (bias's) 8 elements at `at`: fp32 or the rows' 16-bit type; or `none`
template <int TYPE>
__device__ __forceinline__ void load_weight8(const void* w, int weight_type, int64_t at, float none, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = none;
  } else if (weight_type == 2) {
    load8<2>(static_cast<const float*>(w) + at, f);
  } else {
    load8<TYPE == 2 ? 0 : TYPE>(static_cast<const uint16_t*>(w) + at, f);
  }
}

// Sums of N values over the L lanes of a row (xor butterfly), or (L = 0) over the
// CTA; every thread gets them.  buf: [2][16][N] floats, the halves in turn (`turn`), so
// that one barrier serves each sum.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* buf, int turn) {
#pragma unroll
  for (int d = (L ? L : 32) / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  if constexpr (L == 0) {
    float* b = buf + turn * 16 * N;
    const int warps = blockDim.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) b[(threadIdx.x >> 5) * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] += b[w * N + i];
  }
}

// ------------------------------------------------------------------ forward

// One row for each group of L lanes (L = 0: for the CTA), V vectors of 8 a thread.
template <int TYPE, int L, int V>
__global__ void __launch_bounds__(L ? kThreads : kRowThreads)
    row_norm_kernel(const __grid_constant__ RowNormArgs a, bool layer) {
  __shared__ float buf[2 * 16 * 2];
  pdl_wait();
  pdl_launch_dependents();
  const int lanes = L ? L : blockDim.x, lane = L ? threadIdx.x & (L - 1) : threadIdx.x, vecs = a.H / 8;
  const int64_t row = L ? static_cast<int64_t>(blockIdx.x) * (kThreads / (L ? L : 1)) + threadIdx.x / (L ? L : 1) : blockIdx.x;
  const bool mine = row < a.rows;
  const char* src = static_cast<const char*>(a.x) + static_cast<size_t>(row) * a.ldx * kSize<TYPE>;
  float x[V][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int at = v * lanes + lane;
    if (mine && at < vecs) {
      load8<TYPE>(src + static_cast<size_t>(at) * 8 * kSize<TYPE>, x[v]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[v][i] = 0.0f;
    }
  }
  const float inv_h = __fdiv_rn(1.0f, static_cast<float>(a.H));
  float m = 0.0f, shift = 0.0f, s[2] = {0.0f, 0.0f};
  if (layer) {
    float t[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) t[0] += x[v][i];
    row_sums<L>(t, buf + 32, 1);
    m = t[0] * inv_h;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (v * lanes + lane < vecs)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[v][i] -= m;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 8; ++i) s[0] += x[v][i];
  }
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) s[1] = __fmaf_rn(x[v][i], x[v][i], s[1]);
  row_sums<L>(s, buf, 0);
  if (layer) shift = s[0] * inv_h;  // (what the rounding of m left)
  float var = __fmaf_rn(-shift, shift, s[1] * inv_h);
  if (var < 0.0f) var = 0.0f;  // (NaN stays NaN)
  const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
  if (!mine) return;
  if (lane == 0) {
    if (layer && a.mean) a.mean[row] = m + shift;
    if (a.rstd) a.rstd[row] = r;
  }
  char* dst = static_cast<char*>(a.y) + static_cast<size_t>(row) * a.ldy * kSize<TYPE>;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int at = v * lanes + lane;
    if (at >= vecs) continue;
    float w[8], b[8];
    load_weight8<TYPE>(a.weight, a.weight_type, at * 8, 1.0f, w);
    load_weight8<TYPE>(a.bias, a.weight_type, at * 8, 0.0f, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = __fmaf_rn((x[v][i] - shift) * r, w[i], b[i]);
    store8<TYPE>(dst + static_cast<size_t>(at) * 8 * kSize<TYPE>, w);
  }
}

template <int TYPE, int L, int V>
cudaError_t forward(bool layer, const RowNormArgs& a, cudaStream_t stream) {
  const int threads = L ? kThreads : (a.H / 8 + 32 * V - 1) / (32 * V) * 32;
  const int64_t per = L ? kThreads / (L ? L : 1) : 1;
  return launch_pdl(row_norm_kernel<TYPE, L, V>, dim3(static_cast<unsigned>((a.rows + per - 1) / per)), dim3(threads), 0,
                    stream, a, layer);
}

template <int TYPE>
cudaError_t forward_of(bool layer, const RowNormArgs& a, cudaStream_t stream) {
  if (a.H <= 64) return forward<TYPE, 8, 1>(layer, a, stream);
  if (a.H <= 128) return forward<TYPE, 16, 1>(layer, a, stream);
  if (a.H <= 256) return forward<TYPE, 32, 1>(layer, a, stream);
  if (a.H <= 1024) return forward<TYPE, 32, 4>(layer, a, stream);
  if (a.H <= 8192) return forward<TYPE, 0, 2>(layer, a, stream);
  return forward<TYPE, 0, 4>(layer, a, stream);
}

// ------------------------------------------------------------------ gradient

// What a thread adds to dw and db goes out at the end: `out` [H] of `type`, or with `add` to what is there.
__device__ __forceinline__ void put_sum(void* out, int type, int accumulate, int64_t at, float v) {
  if (type == 2) {
    float* p = static_cast<float*>(out) + at;
    *p = accumulate ? *p + v : v;
  } else if (type == 1) {
    static_cast<__half*>(out)[at] = __float2half_rn(v);
  } else {
    static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(v);
  }
}

// A row's vectors as a thread holds them, packed, and the row's m and r.
template <int TYPE, int V>
struct RowData {
  static constexpr int kQuads = TYPE == 2 ? 2 : 1;  // of a vector
  uint4 x[V][kQuads], d[V][kQuads];
  float m, r;

  __device__ __forceinline__ void load(const RowNormArgs& a, bool layer, int64_t row, int lane, int lanes, int vecs) {
    if (row >= a.rows) return;
    const uint4* px = reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + static_cast<size_t>(row) * a.ldx * kSize<TYPE>);
    const uint4* pd =
        reinterpret_cast<const uint4*>(static_cast<const char*>(a.dy) + static_cast<size_t>(row) * a.lddy * kSize<TYPE>);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = v * lanes + lane;
      if (at < vecs) {
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
          x[v][q] = __ldcs(px + at * kQuads + q);
          d[v][q] = __ldcs(pd + at * kQuads + q);
        }
      }
    }
    m = layer ? __ldg(a.mean + row) : 0.0f;
    r = __ldg(a.rstd + row);
  }
  static __device__ __forceinline__ void unpack(const uint4 (&p)[kQuads], float (&f)[8]) {
    if constexpr (TYPE == 2) {
      f[0] = __uint_as_float(p[0].x), f[1] = __uint_as_float(p[0].y), f[2] = __uint_as_float(p[0].z);
      f[3] = __uint_as_float(p[0].w), f[4] = __uint_as_float(p[1].x), f[5] = __uint_as_float(p[1].y);
      f[6] = __uint_as_float(p[1].z), f[7] = __uint_as_float(p[1].w);
    } else {
      unpack8<TYPE == 1>(p[0], f);
    }
  }
};

// rows a thread holds beside the one it computes: as many as the registers take
template <int TYPE, int V>
constexpr int kAhead = V == 4 ? 0 : TYPE == 2 || V == 2 ? 1 : 2;

template <int TYPE, bool LAYER, int L, int V>
__global__ void __launch_bounds__(L ? kThreads : kRowThreads, L ? 2 : 1)
    row_norm_grad_kernel(const __grid_constant__ RowNormArgs a) {
  constexpr int kRows = L ? kThreads / (L ? L : 1) : 1;  // rows of a tile
  constexpr int A = kAhead<TYPE, V>;
  __shared__ float buf[2 * 16 * 2];
  __shared__ float all[L ? kThreads * 8 : 1];
  pdl_wait();
  pdl_launch_dependents();
  const int lanes = L ? L : blockDim.x, lane = L ? threadIdx.x & (L - 1) : threadIdx.x, vecs = a.H / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t tile = static_cast<int64_t>(blockIdx.x) * kRows;  // (a tile's rows are walked together: its first one decides)
  int64_t row = tile + (L ? threadIdx.x / (L ? L : 1) : 0);

  float dw[V][8], db[LAYER ? V : 1][8];
#pragma unroll
  for (int v = 0; v < V; ++v)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[v][i] = 0.0f;
      if (LAYER) db[LAYER ? v : 0][i] = 0.0f;
    }
  // the weight: kept where two vectors leave the registers for it, else read again (from L1)
  constexpr bool kKeep = V <= 2;
  float kept[kKeep ? V : 1][8];
  if constexpr (kKeep) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      load_weight8<TYPE>(v * lanes + lane < vecs ? a.weight : nullptr, a.weight_type, (v * lanes + lane) * 8, 1.0f, kept[v]);
  }
  const float inv_h = __fdiv_rn(1.0f, static_cast<float>(a.H));

  RowData<TYPE, V> data[A + 1];
#pragma unroll
  for (int k = 0; k < A; ++k) data[k].load(a, LAYER, row + k * stride, lane, lanes, vecs);
  int turn = 0;
  for (; tile < a.rows; tile += stride, row += stride) {
    data[A].load(a, LAYER, row + A * stride, lane, lanes, vecs);
    const RowData<TYPE, V>& now = data[0];
    const bool mine = row < a.rows;
    const float m = now.m, r = now.r;
    float c[2] = {0.0f, 0.0f};  // sums of e and e n
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (mine && v * lanes + lane < vecs) {
        float x[8], d[8], again[8];
        RowData<TYPE, V>::unpack(now.x[v], x);
        RowData<TYPE, V>::unpack(now.d[v], d);
        if constexpr (!kKeep) load_weight8<TYPE>(a.weight, a.weight_type, (v * lanes + lane) * 8, 1.0f, again);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float e = d[i] * (kKeep ? kept[kKeep ? v : 0][i] : again[i]);
          if (LAYER) c[0] += e;
          c[1] = __fmaf_rn(e, (LAYER ? x[i] - m : x[i]) * r, c[1]);
        }
      }
    }
    row_sums<L>(c, buf, turn);
    turn ^= 1;
    const float c0 = LAYER ? c[0] * inv_h : 0.0f, c1 = c[1] * inv_h;
    char* dst = static_cast<char*>(a.dx) + static_cast<size_t>(row) * a.lddx * kSize<TYPE>;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (mine && v * lanes + lane < vecs) {
        float x[8], d[8], again[8], o[8];
        RowData<TYPE, V>::unpack(now.x[v], x);
        RowData<TYPE, V>::unpack(now.d[v], d);
        if constexpr (!kKeep) load_weight8<TYPE>(a.weight, a.weight_type, (v * lanes + lane) * 8, 1.0f, again);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float n = (LAYER ? x[i] - m : x[i]) * r;
          const float e = d[i] * (kKeep ? kept[kKeep ? v : 0][i] : again[i]);
          o[i] = r * __fmaf_rn(-n, c1, e - c0);
          dw[v][i] = __fmaf_rn(d[i], n, dw[v][i]);
          if (LAYER) db[LAYER ? v : 0][i] += d[i];
        }
        store8<TYPE>(dst + static_cast<size_t>(v * lanes + lane) * 8 * kSize<TYPE>, o);
      }
    }
#pragma unroll
    for (int k = 0; k < A; ++k) data[k] = data[k + 1];
  }
  if (!a.dweight && !a.dbias) return;

  // One CTA alone writes the gradients, else its sums for the second kernel.
  const bool last = gridDim.x == 1;
  auto put = [&](int which, int64_t at, float v) {
    void* out = which ? a.dbias : a.dweight;
    if (!out) return;
    if (last)
      put_sum(out, a.dweight_type, a.accumulate, at, v);
    else
      a.partials[(static_cast<int64_t>(blockIdx.x) * 2 + which) * a.H + at] = v;
  };
  if constexpr (L == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = v * lanes + lane;
      if (at < vecs)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          put(0, at * 8 + i, dw[v][i]);
          if (LAYER) put(1, at * 8 + i, db[LAYER ? v : 0][i]);
        }
    }
  } else {
    // the tile's rows meet in shared memory: [kRows][H], 8 L >= H
#pragma unroll
    for (int which = 0; which < (LAYER ? 2 : 1); ++which) {
      __syncthreads();
      if (lane < vecs)
#pragma unroll
        for (int i = 0; i < 8; ++i)
          all[(threadIdx.x / (L ? L : 1)) * a.H + lane * 8 + i] = which ? db[0][i] : dw[0][i];
      __syncthreads();
      for (int h = threadIdx.x; h < a.H; h += kThreads) {
        float sum = 0.0f;
        for (int k = 0; k < kRows; ++k) sum += all[k * a.H + h];
        put(which, h, sum);
      }
    }
  }
}

// dw and db from the CTAs' sums: a CTA takes 32 columns of one of them, 16 sums at a time.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows) row_norm_sum_kernel(const __grid_constant__ RowNormArgs a, int n) {
  __shared__ float part[kSumRows][33];
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
  void* out = which ? a.dbias : a.dweight;
  if (!out) return;
  float sum = 0.0f;
  if (h < a.H)
#pragma unroll 4
    for (int p = threadIdx.y; p < n; p += kSumRows) sum += __ldcg(a.partials + (static_cast<int64_t>(p) * 2 + which) * a.H + h);
  part[threadIdx.y][threadIdx.x] = sum;
  __syncthreads();
  if (threadIdx.y == 0 && h < a.H) {
    for (int k = 1; k < kSumRows; ++k) sum += part[k][threadIdx.x];
    put_sum(out, a.dweight_type, a.accumulate, h, sum);
  }
}

cudaError_t sum_partials(const RowNormArgs& a, int n, cudaStream_t stream) {
  return launch_pdl(row_norm_sum_kernel, dim3((a.H + 31) / 32, 2), dim3(32, kSumRows), 0, stream, a, n);
}

template <int TYPE, bool LAYER, int L, int V>
cudaError_t gradient(const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kRows = L ? kThreads / (L ? L : 1) : 1;
  const int threads = L ? kThreads : (a.H / 8 + 32 * V - 1) / (32 * V) * 32;
  auto kernel = row_norm_grad_kernel<TYPE, LAYER, L, V>;
  static PerDevice config;  // registers a thread
  int regs = 0;
  cudaError_t e = config.get(
      [&](int& r) -> cudaError_t {
        cudaFuncAttributes attr;
        const cudaError_t ce = cudaFuncGetAttributes(&attr, kernel);
        r = attr.numRegs;
        return ce;
      },
      &regs);
  if (e != cudaSuccess) return e;
  // CTAs that are resident at once
  int per_sm = 65536 / (((regs + 7) & ~7) * threads);
  if (per_sm > 2048 / threads) per_sm = 2048 / threads;
  if (per_sm < 1) per_sm = 1;
  int64_t ctas = (a.rows + kRows - 1) / kRows;
  if (ctas > static_cast<int64_t>(num_sms) * per_sm) ctas = static_cast<int64_t>(num_sms) * per_sm;
  if (ctas > norm_max_ctas(a.H)) ctas = norm_max_ctas(a.H);
  e = launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(threads), 0, stream, a);
  if (e != cudaSuccess || ctas == 1 || (!a.dweight && !a.dbias)) return e;
  return sum_partials(a, static_cast<int>(ctas), stream);
}

template <int TYPE, bool LAYER>
cudaError_t gradient_of(const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  if (a.H <= 64) return gradient<TYPE, LAYER, 8, 1>(a, num_sms, stream);
  if (a.H <= 128) return gradient<TYPE, LAYER, 16, 1>(a, num_sms, stream);
  if (a.H <= 256) return gradient<TYPE, LAYER, 32, 1>(a, num_sms, stream);
  if (a.H <= 4096) return gradient<TYPE, LAYER, 0, 1>(a, num_sms, stream);
  if (a.H <= 8192) return gradient<TYPE, LAYER, 0, 2>(a, num_sms, stream);
  return gradient<TYPE, LAYER, 0, 4>(a, num_sms, stream);
}

template <int TYPE>
cudaError_t gradient_of(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  return layer ? gradient_of<TYPE, true>(a, num_sms, stream) : gradient_of<TYPE, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_row_norm(bool layer, const RowNormArgs& a, cudaStream_t stream) {
  return a.type == 2   ? forward_of<2>(layer, a, stream)
         : a.type == 1 ? forward_of<1>(layer, a, stream)
                       : forward_of<0>(layer, a, stream);
}

cudaError_t launch_row_norm_grad(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows == 0) return sum_partials(a, 0, stream);  // (sums of nothing)
  return a.type == 2   ? gradient_of<2>(layer, a, num_sms, stream)
         : a.type == 1 ? gradient_of<1>(layer, a, num_sms, stream)
                       : gradient_of<0>(layer, a, num_sms, stream);
}

}  // namespace moe
