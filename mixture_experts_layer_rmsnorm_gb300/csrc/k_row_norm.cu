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
// reduction: what dx needs (n and e) is held in registers, so that the next row's loads can
// take this one's place before it; the row after that is asked into the L2 (one bulk
// prefetch each of x and dy; 16384 rows of 4096, bf16: 79 -> 69 us).
//
// Measured (bf16, inputs not in the L2; of the measured copy rate): forward, rms 16384 x 4096 45 us (0.88), 4096 x
// 7168 22 (0.78); gradient, rms 16384 x 4096 69 (0.86), 4096 x 7168 38 (0.67), 163840 x 128 27 (0.68), layer 16384 x 4096
// 88 (0.67), 6141 x 1408 23 (0.33).  What is missing is latency: a row's barrier, and 5 us of the second kernel.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "grouped_elementwise.cuh"
#include "launch_config.cuh"
#include "moe_kernels.cuh"
#include "pdl.cuh"
#include "row_norm.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;     // of CTAs whose rows are held by 8, 16 or 32 lanes
constexpr int kRowThreads = 512;  // of CTAs that hold a row each, at most
constexpr int kWarps = kRowThreads / 32;

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

template <int TYPE, int Q>
__device__ __forceinline__ void unpack(const uint4 (&p)[Q], float (&f)[8]) {
  if constexpr (TYPE == 2) {
    f[0] = __uint_as_float(p[0].x), f[1] = __uint_as_float(p[0].y), f[2] = __uint_as_float(p[0].z);
    f[3] = __uint_as_float(p[0].w), f[4] = __uint_as_float(p[1].x), f[5] = __uint_as_float(p[1].y);
    f[6] = __uint_as_float(p[1].z), f[7] = __uint_as_float(p[1].w);
  } else {
    unpack8<TYPE == 1>(p[0], f);
  }
}

// Sums of N values over the L lanes of a row (xor butterfly), or (L = 0) over the
// CTA; every thread gets them.  buf: [2][kWarps][N] floats, the halves in turn (`turn`), so
// that one barrier serves each sum.
template <int L, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float* buf, int turn) {
#pragma unroll
  for (int d = (L ? L : 32) / 2; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xFFFFFFFFu, v[i], d);
  if constexpr (L == 0) {
    float* b = buf + turn * kWarps * N;
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

// One row at a time for each group of L lanes (L = 0: for the CTA), V vectors of 8 a thread, kept packed: the more
// a thread holds, the fewer warps a row's sums have to join (4096 rows of 7168, bf16: 62, 35, 25, 22 us with 1, 2,
// 4, 8 vectors).  Rows of up to 256 elements are walked with the grid's stride, the weight in registers and the next row
// on its way (163840 rows of 128, bf16: 18.2 instead of 20.9 us; with more vectors it costs: 65536 x 1024 55 -> 63 us).
template <int TYPE, int L, int V>
__global__ void __launch_bounds__(L || V == 8 ? kThreads : kRowThreads)
    row_norm_kernel(const __grid_constant__ RowNormArgs a, bool layer) {
  constexpr int Q = TYPE == 2 ? 2 : 1, kGroups = L ? kThreads / (L ? L : 1) : 1;  // Q: 16-byte pieces of a vector
  constexpr bool kWalk = L > 0 && V == 1;  // over rows, weight and bias in registers (else they are read from L1)
  __shared__ float buf[2 * kWarps * 2];
  pdl_wait();
  pdl_launch_dependents();
  const int lanes = L ? L : blockDim.x, lane = L ? threadIdx.x & (L - 1) : threadIdx.x, vecs = a.H / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kGroups;
  int64_t tile = static_cast<int64_t>(blockIdx.x) * kGroups;  // (a tile's rows are walked together: its first one decides)
  int64_t row = tile + (L ? threadIdx.x / (L ? L : 1) : 0);
  uint4 x[V][Q];
  auto load = [&](int64_t at_row) {
    const uint4* src = reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + static_cast<size_t>(at_row) * a.ldx * kSize<TYPE>);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = v * lanes + lane;
#pragma unroll
      for (int q = 0; q < Q; ++q) x[v][q] = at_row < a.rows && at < vecs ? __ldcs(src + at * Q + q) : make_uint4(0, 0, 0, 0);
    }
  };
  load(row);
  float w[kWalk ? V : 1][8], b[kWalk ? V : 1][8];
  if constexpr (kWalk) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const bool in = v * lanes + lane < vecs;
      load_weight8<TYPE>(in ? a.weight : nullptr, a.weight_type, (v * lanes + lane) * 8, 1.0f, w[v]);
      load_weight8<TYPE>(in ? a.bias : nullptr, a.weight_type, (v * lanes + lane) * 8, 0.0f, b[v]);
    }
  }
  const float inv_h = __fdiv_rn(1.0f, static_cast<float>(a.H));
  for (; tile < a.rows; tile += stride, row += stride) {
    uint4 now[V][Q];
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int q = 0; q < Q; ++q) now[v][q] = x[v][q];
    if constexpr (kWalk) load(row + stride);
    float m = 0.0f, shift = 0.0f, s[2] = {0.0f, 0.0f};
    if (layer) {
      float t[1] = {0.0f};
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        unpack<TYPE>(now[v], f);
        float part = 0.0f;  // (sums of 8, then of those: fewer roundings one after the other)
#pragma unroll
        for (int i = 0; i < 8; ++i) part += f[i];
        t[0] += part;
      }
      row_sums<L>(t, buf + 2 * kWarps, 1);
      m = t[0] * inv_h;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (v * lanes + lane >= vecs) continue;
      float f[8];
      unpack<TYPE>(now[v], f);
      float part[2] = {0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float d = layer ? f[i] - m : f[i];
        if (layer) part[0] += d;
        part[1] = __fmaf_rn(d, d, part[1]);
      }
      s[0] += part[0], s[1] += part[1];
    }
    if (layer) {
      row_sums<L>(s, buf, 0);
      shift = s[0] * inv_h;  // (what the rounding of m left)
    } else {
      float t[1] = {s[1]};
      row_sums<L>(t, buf, 0);
      s[1] = t[0];
    }
    float var = __fmaf_rn(-shift, shift, s[1] * inv_h);
    if (var < 0.0f) var = 0.0f;  // (NaN stays NaN)
    const float r = __fdiv_rn(1.0f, __fsqrt_rn(var + a.eps));
    if (row < a.rows) {
      if (lane == 0) {
        if (layer && a.mean) a.mean[row] = m + shift;
        if (a.rstd) a.rstd[row] = r;
      }
      char* dst = static_cast<char*>(a.y) + static_cast<size_t>(row) * a.ldy * kSize<TYPE>;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int at = v * lanes + lane;
        if (at >= vecs) continue;
        float f[8];
        unpack<TYPE>(now[v], f);
        if constexpr (!kWalk) {
          load_weight8<TYPE>(a.weight, a.weight_type, at * 8, 1.0f, w[0]);
          load_weight8<TYPE>(a.bias, a.weight_type, at * 8, 0.0f, b[0]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[i] = __fmaf_rn(((layer ? f[i] - m : f[i]) - shift) * r, w[kWalk ? v : 0][i], b[kWalk ? v : 0][i]);
        store8<TYPE>(dst + static_cast<size_t>(at) * 8 * kSize<TYPE>, f);
      }
    }
    if constexpr (!kWalk) break;
  }
}

template <int TYPE, int L, int V>
cudaError_t forward(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  const int threads = L ? kThreads : (a.H / 8 + 32 * V - 1) / (32 * V) * 32;
  const int64_t per = L ? kThreads / (L ? L : 1) : 1;
  int64_t ctas = (a.rows + per - 1) / per;
  if (L && V == 1 && ctas > static_cast<int64_t>(num_sms) * 4) ctas = static_cast<int64_t>(num_sms) * 4;  // (those resident)
  return launch_pdl(row_norm_kernel<TYPE, L, V>, dim3(static_cast<unsigned>(ctas)), dim3(threads), 0, stream, a, layer);
}

template <int TYPE>
cudaError_t forward_of(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  if (a.H <= 64) return forward<TYPE, 8, 1>(layer, a, num_sms, stream);
  if (a.H <= 128) return forward<TYPE, 16, 1>(layer, a, num_sms, stream);
  if (a.H <= 256) return forward<TYPE, 32, 1>(layer, a, num_sms, stream);
  if (a.H <= 512) return forward<TYPE, 32, 2>(layer, a, num_sms, stream);
  if (a.H <= 1024) return forward<TYPE, 32, 4>(layer, a, num_sms, stream);
  if (TYPE == 2 || a.H <= 2048) return forward<TYPE, 0, 4>(layer, a, num_sms, stream);
  return forward<TYPE, 0, 8>(layer, a, num_sms, stream);
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
};

// MAX: threads of a CTA at most, MIN: CTAs of that size that an SM holds at least.
template <int TYPE, bool LAYER, int L, int V, int MAX, int MIN>
__global__ void __launch_bounds__(MAX, MIN)
    row_norm_grad_kernel(const __grid_constant__ RowNormArgs a) {
  constexpr int kRows = L ? kThreads / (L ? L : 1) : 1;  // rows of a tile
  __shared__ float buf[2 * kWarps * 2];
  __shared__ float all[L ? kThreads * 8 * V : 1];
  pdl_wait();
  pdl_launch_dependents();
  const int lanes = L ? L : blockDim.x, lane = L ? threadIdx.x & (L - 1) : threadIdx.x, vecs = a.H / 8;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t tile = static_cast<int64_t>(blockIdx.x) * kRows;  // (a tile's rows are walked together: its first one decides)
  int64_t row = tile + (L ? threadIdx.x / (L ? L : 1) : 0);

  constexpr bool kHold = V <= 2;  // n, e and the weight stay in registers; else they are worked out (read) again
  float dw[V][8], db[LAYER ? V : 1][8], w[kHold ? V : 1][8];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (kHold)
      load_weight8<TYPE>(v * lanes + lane < vecs ? a.weight : nullptr, a.weight_type, (v * lanes + lane) * 8, 1.0f,
                         w[kHold ? v : 0]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      dw[v][i] = 0.0f;
      if (LAYER) db[LAYER ? v : 0][i] = 0.0f;
    }
  }
  const float inv_h = __fdiv_rn(1.0f, static_cast<float>(a.H));

  RowData<TYPE, V> data;
  data.load(a, LAYER, row, lane, lanes, vecs);
  int turn = 0;
  for (; tile < a.rows; tile += stride, row += stride) {
    if (L == 0 && threadIdx.x < 2 && row + 2 * stride < a.rows) {
      const char* p = threadIdx.x ? static_cast<const char*>(a.dy) + static_cast<size_t>(row + 2 * stride) * a.lddy * kSize<TYPE>
                                  : static_cast<const char*>(a.x) + static_cast<size_t>(row + 2 * stride) * a.ldx * kSize<TYPE>;
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(static_cast<uint32_t>(a.H * static_cast<int>(kSize<TYPE>))) : "memory");
    }
    const bool mine = row < a.rows;
    const float m = data.m, r = data.r;
    float n[V][8], e[V][8], c[2] = {0.0f, 0.0f};  // c: the sums of e n and e
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (mine && v * lanes + lane < vecs) {
        float x[8], d[8];
        unpack<TYPE>(data.x[v], x);
        unpack<TYPE>(data.d[v], d);
        if constexpr (!kHold) load_weight8<TYPE>(a.weight, a.weight_type, (v * lanes + lane) * 8, 1.0f, w[0]);
        float part[2] = {0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[v][i] = (LAYER ? x[i] - m : x[i]) * r;
          e[v][i] = d[i] * w[kHold ? v : 0][i];
          part[0] = __fmaf_rn(e[v][i], n[v][i], part[0]);
          dw[v][i] = __fmaf_rn(d[i], n[v][i], dw[v][i]);
          if (LAYER) {
            part[1] += e[v][i];
            db[LAYER ? v : 0][i] += d[i];
          }
        }
        c[0] += part[0];
        if (LAYER) c[1] += part[1];
      }
    }
    // the next row's loads, whose place has just become free, before the sums are joined
    if constexpr (kHold) data.load(a, LAYER, row + stride, lane, lanes, vecs);
    if constexpr (LAYER) {
      row_sums<L>(c, buf, turn);
    } else {
      float one[1] = {c[0]};
      row_sums<L>(one, buf, turn);
      c[0] = one[0];
    }
    turn ^= 1;
    const float c1 = c[0] * inv_h, c0 = LAYER ? c[1] * inv_h : 0.0f;
    char* dst = static_cast<char*>(a.dx) + static_cast<size_t>(row) * a.lddx * kSize<TYPE>;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (mine && v * lanes + lane < vecs) {
        float o[8];
        if constexpr (!kHold) {
          float x[8], d[8];
          unpack<TYPE>(data.x[v], x);
          unpack<TYPE>(data.d[v], d);
          load_weight8<TYPE>(a.weight, a.weight_type, (v * lanes + lane) * 8, 1.0f, w[0]);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            n[v][i] = (LAYER ? x[i] - m : x[i]) * r;
            e[v][i] = d[i] * w[0][i];
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = r * __fmaf_rn(-n[v][i], c1, LAYER ? e[v][i] - c0 : e[v][i]);
        store8<TYPE>(dst + static_cast<size_t>(v * lanes + lane) * 8 * kSize<TYPE>, o);
      }
    }
    if constexpr (!kHold) data.load(a, LAYER, row + stride, lane, lanes, vecs);
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
    // the tile's rows meet in shared memory: [kRows][H], 8 L V >= H
#pragma unroll
    for (int which = 0; which < (LAYER ? 2 : 1); ++which) {
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int at = v * lanes + lane;
        if (at < vecs)
#pragma unroll
          for (int i = 0; i < 8; ++i)
            all[(threadIdx.x / (L ? L : 1)) * a.H + at * 8 + i] = which ? db[LAYER ? v : 0][i] : dw[v][i];
      }
      __syncthreads();
      for (int h = threadIdx.x; h < a.H; h += kThreads) {
        float sum = 0.0f;
        for (int k = 0; k < kRows; ++k) sum += all[k * a.H + h];
        put(which, h, sum);
      }
    }
  }
}

// dw and db from the CTAs' sums: a CTA takes 32 columns of one of them, 32 sums at a time.
constexpr int kSumRows = 32;
__global__ void __launch_bounds__(32 * kSumRows) row_norm_sum_kernel(const __grid_constant__ RowNormArgs a, int n) {
  __shared__ float part[kSumRows][33];
  pdl_wait();
  pdl_launch_dependents();
  const int h = blockIdx.x * 32 + threadIdx.x, which = blockIdx.y;
  void* out = which ? a.dbias : a.dweight;
  if (!out) return;
  float sum = 0.0f;
  if (h < a.H)
#pragma unroll 8
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

template <int TYPE, bool LAYER, int L, int V, int MAX, int MIN>
cudaError_t gradient(const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  constexpr int kRows = L ? kThreads / (L ? L : 1) : 1;
  const int threads = L ? kThreads : (a.H / 8 + 32 * V - 1) / (32 * V) * 32;
  auto kernel = row_norm_grad_kernel<TYPE, LAYER, L, V, MAX, MIN>;
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
  constexpr int kMin = LAYER ? 3 : 4;
  if (a.H <= 64) return gradient<TYPE, LAYER, 8, 1, kThreads, kMin>(a, num_sms, stream);
  if (a.H <= 128) return gradient<TYPE, LAYER, 16, 1, kThreads, kMin>(a, num_sms, stream);
  if (a.H <= 256) return gradient<TYPE, LAYER, 32, 1, kThreads, kMin>(a, num_sms, stream);
  if (a.H <= 512) return gradient<TYPE, LAYER, 32, 2, kThreads, 2>(a, num_sms, stream);
  // Registers for two CTAs an SM where a CTA is near 256 threads (layer norm, 16384 rows of 4096, bf16: 102 -> 89 us;
  // below, they are as many without the limit: 16384 rows of 2048 50 us, 55 with it)
  if (a.H <= 2048) return gradient<TYPE, LAYER, 0, 2, 256, 1>(a, num_sms, stream);
  if (a.H <= 4096) return gradient<TYPE, LAYER, 0, 2, 256, 2>(a, num_sms, stream);
  if (a.H <= 8192) return gradient<TYPE, LAYER, 0, 2, 512, 1>(a, num_sms, stream);
  return gradient<TYPE, LAYER, 0, 4, 512, 1>(a, num_sms, stream);
}

template <int TYPE>
cudaError_t gradient_of(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  return layer ? gradient_of<TYPE, true>(a, num_sms, stream) : gradient_of<TYPE, false>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_row_norm(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  return a.type == 2   ? forward_of<2>(layer, a, num_sms, stream)
         : a.type == 1 ? forward_of<1>(layer, a, num_sms, stream)
                       : forward_of<0>(layer, a, num_sms, stream);
}

cudaError_t launch_row_norm_grad(bool layer, const RowNormArgs& a, int num_sms, cudaStream_t stream) {
  if (a.rows == 0) return sum_partials(a, 0, stream);  // (sums of nothing)
  return a.type == 2   ? gradient_of<2>(layer, a, num_sms, stream)
         : a.type == 1 ? gradient_of<1>(layer, a, num_sms, stream)
                       : gradient_of<0>(layer, a, num_sms, stream);
}

}  // namespace moe
