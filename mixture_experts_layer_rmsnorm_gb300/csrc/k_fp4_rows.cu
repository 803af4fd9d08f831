// k_fp4_rows.cu -- rows to 4 bits and back: MXFP4 (E2M1 codes, one E8M0 scale
// per 32 elements) and NVFP4 (E2M1 codes, one E4M3 scale per 16, one fp32
// scale per row or per group), with the definitions of the layer's weight
// quantizers:
//   MXFP4  E = floor(log2(amax)) - 2 clamped to [-127, 127] (-127 for zeros),
//          code = E2M1(x / 2^E)
//   NVFP4  g = amax_row (or group) / 2688 (1 for zeros), s = E4M3(amax / (6 g)),
//          code = E2M1(x / (s g)), 0 where s g = 0; each step one fp32 operation
// E2M1: nearest, ties to the even code, at most 6.  Beyond them: a block
// (MXFP4) or a row / group (NVFP4) that holds a NaN or an infinity gets a NaN
// scale, so the values it stands for are NaN.
//
// HBM-bound: an element is read once and half a byte plus its share of the scale written.  TPR
// threads share a row, 8 elements (16 bytes of 16-bit input) per load, a warp's
// loads and code stores contiguous; up to kHold vectors per thread stay in
// registers between NVFP4's row maximum and the codes.  The division x / (s g)
// decides codes, so it has to be the rounded quotient; only its side of a
// code's border matters, so x times the rounded reciprocal (within 2 ulps of
// the quotient) decides unless it lies within 8 ulps of a border, where the
// quotient itself is taken.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "grouped_elementwise.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kHold = 4;  // vectors of 8 elements a thread holds

struct RowPlace {
  bool on;
  int group;
  int64_t tile_row;
  int in_tile;
};

// The group and scale place of row p (warp-collective, the same p in a warp):
// two rounds of 32 comparisons find the group among up to 1024.  Rows of no
// group, and places that lists out of order could lead to, are off.
__device__ __forceinline__ RowPlace place_of(const Fp4RowsArgs& a, int64_t p, int lane) {
  RowPlace r{false, 0, 0, 0};
  int64_t start, count;
  if (a.offsets) {
    const int step = (a.G + 31) / 32;
    int at = lane * step;
    const unsigned m1 = __ballot_sync(0xFFFFFFFFu, at < a.G && __ldg(a.offsets + at) <= p);
    if (m1 == 0) return r;
    const int first = (31 - __clz(m1)) * step;
    int g = first;
    for (int base = 0; base < step; base += 32) {  // (one round up to 1024 groups)
      at = first + base + lane;
      const unsigned m2 = __ballot_sync(0xFFFFFFFFu, base + lane < step && at < a.G && __ldg(a.offsets + at) <= p);
      if (m2) g = first + base + 31 - __clz(m2);
    }
    start = __ldg(a.offsets + g);
    count = a.counts ? __ldg(a.counts + g) : __ldg(a.offsets + g + 1) - start;
    r.group = g;
    r.tile_row = start / 128 + g;
  } else {
    const int64_t R = a.rows / a.G;
    r.group = static_cast<int>(p / R);
    start = r.group * R;
    count = a.counts ? __ldg(a.counts + r.group) : R;
    if (count > R) count = R;
    r.tile_row = r.group * ((R + 127) / 128);
  }
  const int64_t within = p - start;
  r.tile_row += within / 128;
  r.in_tile = static_cast<int>(within % 128);
  r.on = start >= 0 && within >= 0 && within < count && r.tile_row < a.tile_rows;
  return r;
}

// byte offset of a chunk's word (4 blocks) of a row
__device__ __forceinline__ size_t word_offset(const RowPlace& r, int chunks, int chunk) {
  return (static_cast<size_t>(r.tile_row) * chunks + chunk) * 512 + (r.in_tile & 31) * 16 + (r.in_tile >> 5) * 4;
}

template <int TYPE>
__device__ __forceinline__ void load8(const void* row, int v, uint4 (&raw)[TYPE == 2 ? 2 : 1]) {
  const uint4* p = static_cast<const uint4*>(row) + static_cast<int64_t>(v) * (TYPE == 2 ? 2 : 1);
  raw[0] = __ldg(p);
  if (TYPE == 2) raw[TYPE == 2 ? 1 : 0] = __ldg(p + 1);
}

template <int TYPE>
__device__ __forceinline__ void values8(const uint4 (&raw)[TYPE == 2 ? 2 : 1], float (&f)[8]) {
  if (TYPE == 2) {
    const uint4& hi = raw[TYPE == 2 ? 1 : 0];
    f[0] = __uint_as_float(raw[0].x), f[1] = __uint_as_float(raw[0].y), f[2] = __uint_as_float(raw[0].z);
    f[3] = __uint_as_float(raw[0].w), f[4] = __uint_as_float(hi.x), f[5] = __uint_as_float(hi.y);
    f[6] = __uint_as_float(hi.z), f[7] = __uint_as_float(hi.w);
  } else {
    unpack8<TYPE == 1>(raw[0], f);
  }
}

// largest magnitude as fp32 bits: infinities and NaN are the largest of all
__device__ __forceinline__ uint32_t amax8(const float (&f)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  return m;
}

// eight E2M1 codes (nearest, ties to even, saturating): element i in bits 4i .. 4i + 3
__device__ __forceinline__ uint32_t codes8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

constexpr uint32_t kInfBits = 0x7F800000u;

__device__ __forceinline__ float nv_global(uint32_t amax) {
  if (amax >= kInfBits) return __uint_as_float(0x7FC00000u);
  return amax ? __fdiv_rn(__uint_as_float(amax), 2688.0f) : 1.0f;
}

__device__ __forceinline__ uint32_t e4m3_of(float u) {  // u >= 0
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(u));
  return r & 0xFFu;
}
__device__ __forceinline__ float e4m3_to(uint32_t c) {  // sign 0; 0x7F is NaN
  const uint32_t e = (c >> 3) & 15u, m = c & 7u;
  if (c == 0x7Fu) return __uint_as_float(0x7FC00000u);
  return e ? __uint_as_float(((e + 120u) << 23) | (m << 20)) : static_cast<float>(m) * 0x1p-9f;
}

// One block's part of 8 elements: the block maximum's scale byte and the codes.
template <Fp4Format F>
__device__ __forceinline__ uint32_t encode8(const float (&x)[8], uint32_t amax, float g, float six_g, uint32_t& scale) {
  if (F == Fp4Format::kMx) {
    int e = static_cast<int>(amax >> 23) - 127 - 2;  // (a subnormal maximum clamps too)
    e = e < -127 ? -127 : e;
    scale = amax >= kInfBits ? 255u : static_cast<uint32_t>(e + 127);
    // 2^-e, exact; e <= 126
    const float inv = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = x[i] * inv;
    return codes8(y);
  }
  scale = g == g ? e4m3_of(__fdiv_rn(__uint_as_float(amax), six_g)) : 0x7Fu;
  const float d = __fmul_rn(e4m3_to(scale), g);
  if (!(d > 0.0f)) return 0u;
  float y[8];
  // every border of E2M1 (0.25 .. 5) has its last 21 bits clear
  const float inv = __frcp_rn(d);
  bool near = !(d > 0x1p-100f && d < 0x1p100f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    y[i] = x[i] * inv;
    near |= ((__float_as_uint(y[i]) + 8u) & 0x1FFFFFu) < 16u && fabsf(y[i]) > 0.125f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], d);
  }
  return codes8(y);
}

// TPR threads per row.  NVFP4 per row: the row's maximum first; per group: from
// gscale, which then holds the maxima's bits.
template <Fp4Format F, int TYPE, int TPR>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(const __grid_constant__ Fp4RowsArgs a) {
  constexpr int kRows = kThreads / TPR, kWarpsPerRow = TPR / 32;
  __shared__ uint32_t warp_max[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % TPR;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const int vecs = a.K / 8;
  const bool in = p < a.rows;
  const char* src = static_cast<const char*>(a.src) + (in ? p : 0) * a.ld * (TYPE == 2 ? 4 : 2);
  uint4 held[kHold][TYPE == 2 ? 2 : 1];
  const RowPlace r = in ? place_of(a, p, lane) : RowPlace{false, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (r.on && t + i * TPR < vecs) load8<TYPE>(src, t + i * TPR, held[i]);
  float g = 1.0f;
  if (F == Fp4Format::kNv) {
    uint32_t m = 0;
    if (!a.per_group) {
      if (r.on) {
#pragma unroll
        for (int i = 0; i < kHold; ++i)
          if (t + i * TPR < vecs) {
            float x[8];
            values8<TYPE>(held[i], x);
            m = max(m, amax8(x));
          }
        for (int v = t + kHold * TPR; v < vecs; v += TPR) {
          uint4 raw[TYPE == 2 ? 2 : 1];
          load8<TYPE>(src, v, raw);
          float x[8];
          values8<TYPE>(raw, x);
          m = max(m, amax8(x));
        }
      }
      m = __reduce_max_sync(0xFFFFFFFFu, m);
      if (kWarpsPerRow > 1) {
        if (lane == 0) warp_max[warp] = m;
        __syncthreads();
        const int w0 = warp / kWarpsPerRow * kWarpsPerRow;
#pragma unroll
        for (int w = 0; w < kWarpsPerRow; ++w) m = max(m, warp_max[w0 + w]);
      }
      g = nv_global(m);
      if (r.on && t == 0) a.gscale[p] = g;
    } else if (r.on) {
      g = nv_global(__float_as_uint(__ldcg(a.gscale + r.group)));
    }
  }
  if (!r.on) return;  // (whole warps)
  const float six_g = __fmul_rn(6.0f, g);
  const int chunks = (a.K + fp4_chunk(F) - 1) / fp4_chunk(F);
  constexpr int kLanesPerBlock = fp4_block(F) / 8, kLanesPerWord = 4 * kLanesPerBlock;
  uint8_t* codes = a.codes + p * (a.K / 2);
  auto emit = [&](int v, const float (&x)[8], bool on) {
    uint32_t m = on ? amax8(x) : 0u;
#pragma unroll
    for (int o = 1; o < kLanesPerBlock; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    uint32_t sc;
    const uint32_t w = encode8<F>(x, m, g, six_g, sc);
    if (on) *reinterpret_cast<uint32_t*>(codes + v * 4) = w;
    // four blocks' bytes to one word; blocks past K are zeros
    sc = on ? sc << (8 * ((lane / kLanesPerBlock) & 3)) : 0u;
#pragma unroll
    for (int o = kLanesPerBlock; o < kLanesPerWord; o <<= 1) sc |= __shfl_xor_sync(0xFFFFFFFFu, sc, o);
    if (on && lane % kLanesPerWord == 0)
      *reinterpret_cast<uint32_t*>(a.scales + word_offset(r, chunks, v * 8 / fp4_chunk(F))) = sc;
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    if (i * TPR + (t & ~31) >= vecs) break;  // (whole warps)
    const bool on = t + i * TPR < vecs;
    float x[8];
    if (on) values8<TYPE>(held[i], x);
    else
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    emit(t + i * TPR, x, on);
  }
  for (int v0 = kHold * TPR + (t & ~31); v0 < vecs; v0 += TPR) {
    const int v = v0 + lane;
    const bool on = v < vecs;
    uint4 raw[TYPE == 2 ? 2 : 1];
    float x[8];
    if (on) {
      load8<TYPE>(src, v, raw);
      values8<TYPE>(raw, x);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = 0.0f;
    }
    emit(v, x, on);
  }
}

// Largest magnitude of every group's rows into gscale's bits (zero before).
template <int TYPE>
__global__ void __launch_bounds__(kThreads) fp4_group_amax_kernel(const __grid_constant__ Fp4RowsArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (p >= a.rows) return;
  const RowPlace r = place_of(a, p, lane);
  if (!r.on) return;
  const char* src = static_cast<const char*>(a.src) + p * a.ld * (TYPE == 2 ? 4 : 2);
  uint32_t m = 0;
#pragma unroll 4
  for (int v = lane; v < a.K / 8; v += 32) {
    uint4 raw[TYPE == 2 ? 2 : 1];
    load8<TYPE>(src, v, raw);
    float x[8];
    values8<TYPE>(raw, x);
    m = max(m, amax8(x));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (lane == 0) atomicMax(reinterpret_cast<unsigned int*>(a.gscale) + r.group, m);
}

// maxima -> scales, in place
__global__ void fp4_group_scale_kernel(float* gscale, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) gscale[i] = nv_global(__float_as_uint(gscale[i]));
}

// eight codes -> their values
__device__ __forceinline__ void decode8(uint32_t w, float (&f)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

template <Fp4Format F, int TYPE, int TPR>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const __grid_constant__ Fp4RowsArgs a) {
  const int lane = threadIdx.x & 31, t = threadIdx.x % TPR;
  const int64_t p = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (p >= a.rows) return;
  const RowPlace r = place_of(a, p, lane);
  if (!r.on) return;
  const int vecs = a.K / 8, chunks = (a.K + fp4_chunk(F) - 1) / fp4_chunk(F);
  const uint8_t* codes = a.codes + p * (a.K / 2);
  char* dst = static_cast<char*>(a.dst) + p * a.ld * (TYPE == 2 ? 4 : 2);
  const float g = F == Fp4Format::kNv ? __ldg(a.gscale + (a.per_group ? r.group : p)) : 1.0f;
#pragma unroll 4
  for (int v = t; v < vecs; v += TPR) {
    const uint32_t w = __ldcs(reinterpret_cast<const uint32_t*>(codes) + v);
    const int block = v * 8 / fp4_block(F);
    const uint32_t sc = a.scales[word_offset(r, chunks, block / 4) + (block & 3)];
    float f[8];
    decode8(w, f);
    if (F == Fp4Format::kMx) {
      // 2^(sc - 127); the smallest is subnormal, 255 stands for NaN
      const float s = sc == 255u ? __uint_as_float(0x7FC00000u) : sc ? __uint_as_float(sc << 23) : 0x1p-127f;
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], s);
    } else {
      const float s = e4m3_to(sc);  // times a code: exact
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(__fmul_rn(f[i], s), g);
    }
    if (TYPE == 2) {
      float4* o = reinterpret_cast<float4*>(dst) + 2 * v;
      o[0] = make_float4(f[0], f[1], f[2], f[3]);
      o[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      reinterpret_cast<uint4*>(dst)[v] = pack8<TYPE == 1>(f);
    }
  }
}

template <Fp4Format F, int TYPE, int TPR>
cudaError_t quantize_t(const Fp4RowsArgs& a, cudaStream_t stream) {
  constexpr int rows = kThreads / TPR;
  fp4_quantize_kernel<F, TYPE, TPR><<<static_cast<unsigned>((a.rows + rows - 1) / rows), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <Fp4Format F, int TYPE>
cudaError_t quantize(const Fp4RowsArgs& a, cudaStream_t stream) {
  if (F == Fp4Format::kNv && a.per_group) {
    cudaError_t e = cudaMemsetAsync(a.gscale, 0, sizeof(float) * a.G, stream);
    if (e != cudaSuccess) return e;
    fp4_group_amax_kernel<TYPE><<<static_cast<unsigned>((a.rows + 7) / 8), kThreads, 0, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  // a row's vectors fit the registers of its threads, up to 8192 elements
  const int vecs = a.K / 8;
  const cudaError_t e = vecs <= 32 * kHold   ? quantize_t<F, TYPE, 32>(a, stream)
                        : vecs <= 64 * kHold ? quantize_t<F, TYPE, 64>(a, stream)
                        : vecs <= 128 * kHold ? quantize_t<F, TYPE, 128>(a, stream)
                                              : quantize_t<F, TYPE, 256>(a, stream);
  if (e != cudaSuccess || F != Fp4Format::kNv || !a.per_group) return e;
  fp4_group_scale_kernel<<<(a.G + 127) / 128, 128, 0, stream>>>(a.gscale, a.G);
  return cudaGetLastError();
}

template <Fp4Format F, int TYPE>
cudaError_t dequantize(const Fp4RowsArgs& a, cudaStream_t stream) {
  if (a.K <= 1024)
    fp4_dequantize_kernel<F, TYPE, 32><<<static_cast<unsigned>((a.rows + 7) / 8), kThreads, 0, stream>>>(a);
  else
    fp4_dequantize_kernel<F, TYPE, 128><<<static_cast<unsigned>((a.rows + 1) / 2), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_quantize(Fp4Format f, const Fp4RowsArgs& a, cudaStream_t stream) {
  const bool mx = f == Fp4Format::kMx;
  switch (a.type) {
    case 0: return mx ? quantize<Fp4Format::kMx, 0>(a, stream) : quantize<Fp4Format::kNv, 0>(a, stream);
    case 1: return mx ? quantize<Fp4Format::kMx, 1>(a, stream) : quantize<Fp4Format::kNv, 1>(a, stream);
    default: return mx ? quantize<Fp4Format::kMx, 2>(a, stream) : quantize<Fp4Format::kNv, 2>(a, stream);
  }
}

cudaError_t launch_fp4_dequantize(Fp4Format f, const Fp4RowsArgs& a, cudaStream_t stream) {
  const bool mx = f == Fp4Format::kMx;
  switch (a.type) {
    case 0: return mx ? dequantize<Fp4Format::kMx, 0>(a, stream) : dequantize<Fp4Format::kNv, 0>(a, stream);
    case 1: return mx ? dequantize<Fp4Format::kMx, 1>(a, stream) : dequantize<Fp4Format::kNv, 1>(a, stream);
    default: return mx ? dequantize<Fp4Format::kMx, 2>(a, stream) : dequantize<Fp4Format::kNv, 2>(a, stream);
  }
}

}  // namespace moe
