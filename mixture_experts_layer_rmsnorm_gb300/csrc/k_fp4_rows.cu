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
// Bound: HBM asks for 2.56 bytes per 16-bit element, 14 instruction slots of an SM at the
// measured copy rate, so the instructions per element decide.  A thread takes 8
// elements (16 bytes of 16-bit input) at a time and kHold such vectors at once,
// all loads first; TPR threads share a row.
//   - The block maximum is taken on the packed 16-bit magnitudes, whose order
//     is that of their bits (NaN and infinities above all numbers).
//   - NVFP4's two quotients decide codes, so they have to be the rounded
//     quotients, but only their side of a code's border matters.  x times a
//     reciprocal lowered and raised by 2^-21 (more than all roundings of that product,
//     2^-22) brackets the quotient: if both ends get the same code, so does the quotient; else the
//     division is done.  Two products and conversions instead of a division.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp4.cuh"
#include "grouped_elementwise.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kHold = 4;  // vectors of 8 elements a thread holds

struct RowPlace {
  int group, tile_row, in_tile;
  bool on;
};

// The group and scale place of row p (warp-collective, the same p in a warp):
// two rounds of 32 comparisons find the group among up to 1024.  Rows of no
// group, and places that lists out of order could lead to, are off.
__device__ __forceinline__ RowPlace place_of(const Fp4RowsArgs& a, int p, int lane) {
  RowPlace r{0, 0, 0, false};
  int start, count;
  if (a.offsets) {
    const int step = (a.G + 31) / 32;
    int at = lane * step;
    const unsigned m1 = __ballot_sync(0xFFFFFFFFu, at < a.G && __ldg(a.offsets + at) <= p);
    if (m1 == 0) return r;
    int g = (31 - __clz(m1)) * step;
    if (step > 1) {
      at = g + lane;
      const unsigned m2 = __ballot_sync(0xFFFFFFFFu, lane < step && at < a.G && __ldg(a.offsets + at) <= p);
      if (m2) g += 31 - __clz(m2);
    }
    start = __ldg(a.offsets + g);
    const int end = __ldg(a.offsets + g + 1);
    count = a.counts ? __ldg(a.counts + g) : end - start;
    if (start < 0 || p < start) return r;
    r.group = g;
    r.tile_row = start / 128 + g;
  } else {
    const unsigned R = static_cast<unsigned>(a.rows) / static_cast<unsigned>(a.G);
    r.group = static_cast<int>(static_cast<unsigned>(p) / R);
    start = r.group * static_cast<int>(R);
    count = a.counts ? min(__ldg(a.counts + r.group), static_cast<int>(R)) : static_cast<int>(R);
    r.tile_row = r.group * static_cast<int>((R + 127) / 128);
  }
  const int within = p - start;
  r.tile_row += within >> 7;
  r.in_tile = within & 127;
  r.on = within < count && r.tile_row < a.tile_rows;
  return r;
}

// where a row's scale bytes are: block b at chunk b / 4 (512 bytes each), byte b % 4
__device__ __forceinline__ uint8_t* row_scales(const Fp4RowsArgs& a, const RowPlace& r, int chunks) {
  return a.scales + static_cast<size_t>(r.tile_row) * chunks * 512 + (r.in_tile & 31) * 16 + (r.in_tile >> 5) * 4;
}

template <int TYPE>
struct Vec {  // 8 elements
  uint4 raw[TYPE == 2 ? 2 : 1];
};

template <int TYPE>
__device__ __forceinline__ void load8(const void* row, int v, Vec<TYPE>& x) {
  const uint4* p = static_cast<const uint4*>(row) + static_cast<int64_t>(v) * (TYPE == 2 ? 2 : 1);
  x.raw[0] = __ldg(p);
  if constexpr (TYPE == 2) x.raw[1] = __ldg(p + 1);
}

template <int TYPE>
__device__ __forceinline__ void zero8(Vec<TYPE>& x) {
  x.raw[0] = make_uint4(0, 0, 0, 0);
  if constexpr (TYPE == 2) x.raw[1] = make_uint4(0, 0, 0, 0);
}

template <int TYPE>
__device__ __forceinline__ void values8(const Vec<TYPE>& x, float (&f)[8]) {
  if constexpr (TYPE == 2) {
    f[0] = __uint_as_float(x.raw[0].x), f[1] = __uint_as_float(x.raw[0].y), f[2] = __uint_as_float(x.raw[0].z);
    f[3] = __uint_as_float(x.raw[0].w), f[4] = __uint_as_float(x.raw[1].x), f[5] = __uint_as_float(x.raw[1].y);
    f[6] = __uint_as_float(x.raw[1].z), f[7] = __uint_as_float(x.raw[1].w);
  } else {
    unpack8<TYPE == 1>(x.raw[0], f);
  }
}

// Largest magnitudes as ordered bits: packed pairs of 16 bits, or fp32.
template <int TYPE>
__device__ __forceinline__ uint32_t max_mag(uint32_t a, uint32_t b) {
  return TYPE == 2 ? max(a, b) : __vmaxu2(a, b);
}
template <int TYPE>
__device__ __forceinline__ uint32_t mag8(const Vec<TYPE>& x) {
  if constexpr (TYPE == 2) {
    const uint4 &a = x.raw[0], &b = x.raw[1];
    constexpr uint32_t m = 0x7FFFFFFFu;
    return max(max(max(a.x & m, a.y & m), max(a.z & m, a.w & m)), max(max(b.x & m, b.y & m), max(b.z & m, b.w & m)));
  } else {
    const uint4& a = x.raw[0];
    constexpr uint32_t m = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(a.x & m, a.y & m), __vmaxu2(a.z & m, a.w & m));
  }
}
template <int TYPE>
__device__ __forceinline__ uint32_t mag_bits(uint32_t m) {  // of fp32
  if (TYPE == 2) return m;
  const uint32_t h = max(m >> 16, m & 0xFFFFu);
  return TYPE == 0 ? h << 16 : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
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

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float e4m3_to(uint32_t c) {  // 0x7F is NaN
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// What a row's NVFP4 codes need: g and 1 / (6 g) lowered and raised, or (far
// from 1, or no number) the sign that quotients are divided out.
struct NvRow {
  float g, six_g, r_lo, r_hi;
  bool plain;
};
constexpr float kLo = 1.0f - 0x1p-21f, kHi = 1.0f + 0x1p-21f;

__device__ __forceinline__ bool mid_range(float v) { return v > 0x1p-100f && v < 0x1p100f; }

__device__ __forceinline__ NvRow nv_row(float g) {
  NvRow r;
  r.g = g;
  r.six_g = __fmul_rn(6.0f, g);
  const float inv = __frcp_rn(r.six_g);
  r.r_lo = inv * kLo;
  r.r_hi = inv * kHi;
  r.plain = mid_range(r.six_g);
  return r;
}

// Codes and scale byte of 8 elements of a block whose largest magnitude has
// the fp32 bits `amax`.
template <Fp4Format F, int TYPE>
__device__ __forceinline__ uint32_t encode8(const Vec<TYPE>& v, uint32_t amax, const NvRow& nv, uint32_t& scale) {
  float x[8];
  if constexpr (F == Fp4Format::kMx) {
    int e = static_cast<int>(amax >> 23) - 127 - 2;  // (a subnormal maximum clamps too)
    e = e < -127 ? -127 : e;
    scale = amax >= kInfBits ? 255u : static_cast<uint32_t>(e + 127);
    // 2^-e; x 2^-e is exact down to magnitudes whose code is 0 either way
    const uint32_t inv = static_cast<uint32_t>(127 - e) << 23;
    if constexpr (TYPE == 0) {
      const uint32_t w[4] = {v.raw[0].x, v.raw[0].y, v.raw[0].z, v.raw[0].w};
      const uint32_t s2 = inv | (inv >> 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]),
                                         *reinterpret_cast<const __nv_bfloat162*>(&s2));
        const uint32_t b = *reinterpret_cast<const uint32_t*>(&p);
        x[2 * i] = __uint_as_float(b << 16);
        x[2 * i + 1] = __uint_as_float(b & 0xFFFF0000u);
      }
    } else {
      values8<TYPE>(v, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= __uint_as_float(inv);
    }
    return codes8(x);
  }
  const float top = __uint_as_float(amax);
  const uint32_t both = e4m3_pair(top * nv.r_lo, top * nv.r_hi);
  scale = both & 0xFFu;
  if (scale != both >> 8 || !nv.plain) scale = nv.g == nv.g ? e4m3_pair(__fdiv_rn(top, nv.six_g), 0.0f) & 0xFFu : 0x7Fu;
  const float d = __fmul_rn(e4m3_to(scale), nv.g);
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(d));
  values8<TYPE>(v, x);
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = x[i] * (inv * kLo);
    hi[i] = x[i] * (inv * kHi);
  }
  uint32_t w = codes8(lo);
  if (w != codes8(hi) || !mid_range(d)) {
    if (!(d > 0.0f)) return 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], d);
    w = codes8(x);
  }
  return w;
}

// TPR threads per row.  NVFP4 per row: the row's maximum first; per group: from
// gscale, which then holds the maxima's bits.
template <Fp4Format F, int TYPE, int TPR>
__global__ void __launch_bounds__(kThreads) fp4_quantize_kernel(const __grid_constant__ Fp4RowsArgs a) {
  constexpr int kRows = kThreads / TPR, kWarpsPerRow = TPR / 32;
  __shared__ uint32_t warp_max[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % TPR;
  const int64_t p64 = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const bool in = p64 < a.rows;
  const int p = in ? static_cast<int>(p64) : 0;
  const int vecs = a.K / 8;
  const char* src = static_cast<const char*>(a.src) + p * a.ld * (TYPE == 2 ? 4 : 2);
  Vec<TYPE> held[kHold];
  // (a row of no group is read in vain: its place is looked up meanwhile)
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    if (t + i * TPR < vecs)
      load8<TYPE>(src, t + i * TPR, held[i]);
    else
      zero8<TYPE>(held[i]);
  }
  const RowPlace r = place_of(a, p, lane);
  const bool row_on = in && r.on;
  NvRow nv{};
  if constexpr (F == Fp4Format::kNv) {
    float g;
    if (!a.per_group) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kHold; ++i) m = max_mag<TYPE>(m, mag8<TYPE>(held[i]));
      for (int v = t + kHold * TPR; v < vecs; v += TPR) {
        Vec<TYPE> x;
        load8<TYPE>(src, v, x);
        m = max_mag<TYPE>(m, mag8<TYPE>(x));
      }
      m = __reduce_max_sync(0xFFFFFFFFu, mag_bits<TYPE>(m));
      if (kWarpsPerRow > 1) {
        if (lane == 0) warp_max[warp] = m;
        __syncthreads();
        const int w0 = warp / kWarpsPerRow * kWarpsPerRow;
#pragma unroll
        for (int w = 0; w < kWarpsPerRow; ++w) m = max(m, warp_max[w0 + w]);
      }
      g = nv_global(m);
      if (row_on && t == 0) a.gscale[p] = g;
    } else {
      g = row_on ? nv_global(__float_as_uint(__ldcg(a.gscale + r.group))) : 1.0f;
    }
    nv = nv_row(g);
  }
  if (!row_on) return;  // (whole warps)
  const int chunks = (a.K + fp4_chunk(F) - 1) / fp4_chunk(F);
  constexpr int kLanesPerBlock = fp4_block(F) / 8;
  uint8_t* codes = a.codes + static_cast<size_t>(p) * (a.K / 2);
  uint8_t* scales = row_scales(a, r, chunks);
  auto emit = [&](int v, const Vec<TYPE>& x) {  // whole warps; a block's lanes are all below `vecs` or all not
    uint32_t m = mag8<TYPE>(x);
#pragma unroll
    for (int o = 1; o < kLanesPerBlock; o <<= 1) m = max_mag<TYPE>(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    uint32_t sc;
    const uint32_t w = encode8<F, TYPE>(x, mag_bits<TYPE>(m), nv, sc);
    if (v < vecs) {
      *reinterpret_cast<uint32_t*>(codes + v * 4) = w;
      const int block = v / kLanesPerBlock;
      if (lane % kLanesPerBlock == 0) scales[(block >> 2) * 512 + (block & 3)] = static_cast<uint8_t>(sc);
    }
  };
  const int w0 = t & ~31;  // the warp's first vector of a round
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (i * TPR + w0 < vecs) emit(t + i * TPR, held[i]);
  for (int v0 = kHold * TPR; v0 + w0 < vecs; v0 += kHold * TPR) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (v0 + t + i * TPR < vecs)
        load8<TYPE>(src, v0 + t + i * TPR, held[i]);
      else
        zero8<TYPE>(held[i]);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (v0 + i * TPR + w0 < vecs) emit(v0 + t + i * TPR, held[i]);
  }
  // blocks of the last chunk past K: zero scales
  const int blocks = a.K / fp4_block(F);
  if (t < chunks * 4 - blocks) scales[(chunks - 1) * 512 + ((blocks + t) & 3)] = 0;
}

// Largest magnitude of every group's rows into gscale's bits (zero before).
template <int TYPE>
__global__ void __launch_bounds__(kThreads) fp4_group_amax_kernel(const __grid_constant__ Fp4RowsArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t p64 = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (p64 >= a.rows) return;
  const int p = static_cast<int>(p64), vecs = a.K / 8;
  const char* src = static_cast<const char*>(a.src) + p * a.ld * (TYPE == 2 ? 4 : 2);
  uint32_t m = 0;
  for (int v0 = 0; v0 < vecs; v0 += kHold * 32) {
    Vec<TYPE> held[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (v0 + i * 32 + lane < vecs)
        load8<TYPE>(src, v0 + i * 32 + lane, held[i]);
      else
        zero8<TYPE>(held[i]);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) m = max_mag<TYPE>(m, mag8<TYPE>(held[i]));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, mag_bits<TYPE>(m));
  const RowPlace r = place_of(a, p, lane);
  if (r.on && lane == 0) atomicMax(reinterpret_cast<unsigned int*>(a.gscale) + r.group, m);
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
  const int64_t p64 = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (p64 >= a.rows) return;
  const int p = static_cast<int>(p64);
  const int vecs = a.K / 8, chunks = (a.K + fp4_chunk(F) - 1) / fp4_chunk(F);
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(a.codes + static_cast<size_t>(p) * (a.K / 2));
  uint32_t w[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i) w[i] = t + i * TPR < vecs ? __ldcs(codes + t + i * TPR) : 0u;
  const RowPlace r = place_of(a, p, lane);
  if (!r.on) return;
  const uint8_t* scales = row_scales(a, r, chunks);
  char* dst = static_cast<char*>(a.dst) + p * a.ld * (TYPE == 2 ? 4 : 2);
  const float g = F == Fp4Format::kNv ? __ldg(a.gscale + (a.per_group ? r.group : p)) : 1.0f;
  for (int v0 = 0; v0 < vecs; v0 += kHold * TPR) {
    uint32_t sc[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int v = v0 + t + i * TPR, block = v / (fp4_block(F) / 8);
      if (v0 > 0) w[i] = v < vecs ? __ldcs(codes + v) : 0u;
      sc[i] = v < vecs ? __ldg(scales + (block >> 2) * 512 + (block & 3)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int v = v0 + t + i * TPR;
      if (v >= vecs) break;
      float f[8];
      decode8(w[i], f);
      if constexpr (F == Fp4Format::kMx) {
        // 2^(sc - 127); the smallest is subnormal, 255 stands for NaN
        const float s =
            sc[i] == 255u ? __uint_as_float(0x7FC00000u) : sc[i] ? __uint_as_float(sc[i] << 23) : 0x1p-127f;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(f[j], s);
      } else {
        const float s = e4m3_to(sc[i]);  // times a code: exact
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __fmul_rn(__fmul_rn(f[j], s), g);
      }
      if constexpr (TYPE == 2) {
        float4* o = reinterpret_cast<float4*>(dst) + 2 * v;
        __stcs(o, make_float4(f[0], f[1], f[2], f[3]));
        __stcs(o + 1, make_float4(f[4], f[5], f[6], f[7]));
      } else {
        __stcs(reinterpret_cast<uint4*>(dst) + v, pack8<TYPE == 1>(f));
      }
    }
  }
}

template <Fp4Format F, int TYPE, int TPR>
cudaError_t quantize_t(const Fp4RowsArgs& a, cudaStream_t stream) {
  constexpr int rows = kThreads / TPR;
  fp4_quantize_kernel<F, TYPE, TPR><<<static_cast<unsigned>((a.rows + rows - 1) / rows), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// Threads per row.  Where a row's vectors have to be held at once (NVFP4's
// scale per row), as many as hold them, up to 8192 elements.  Else a warp per row, whose look-up of the
// row's place then serves most elements, unless there are too few rows to fill
// the GPU with warps.
template <Fp4Format F, int TYPE>
cudaError_t quantize(const Fp4RowsArgs& a, cudaStream_t stream) {
  const bool whole = F == Fp4Format::kNv && !a.per_group;
  if (F == Fp4Format::kNv && a.per_group) {
    cudaError_t e = cudaMemsetAsync(a.gscale, 0, sizeof(float) * a.G, stream);
    if (e != cudaSuccess) return e;
    fp4_group_amax_kernel<TYPE><<<static_cast<unsigned>((a.rows + 7) / 8), kThreads, 0, stream>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  const int vecs = a.K / 8;
  const cudaError_t e = vecs <= 32 * kHold || (!whole && a.rows >= 8192) ? quantize_t<F, TYPE, 32>(a, stream)
                        : vecs <= 64 * kHold                             ? quantize_t<F, TYPE, 64>(a, stream)
                        : vecs <= 128 * kHold                            ? quantize_t<F, TYPE, 128>(a, stream)
                                                                         : quantize_t<F, TYPE, 256>(a, stream);
  if (e != cudaSuccess || F != Fp4Format::kNv || !a.per_group) return e;
  fp4_group_scale_kernel<<<(a.G + 127) / 128, 128, 0, stream>>>(a.gscale, a.G);
  return cudaGetLastError();
}

template <Fp4Format F, int TYPE, int TPR>
cudaError_t dequantize_t(const Fp4RowsArgs& a, cudaStream_t stream) {
  constexpr int rows = kThreads / TPR;
  fp4_dequantize_kernel<F, TYPE, TPR><<<static_cast<unsigned>((a.rows + rows - 1) / rows), kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <Fp4Format F, int TYPE>
cudaError_t dequantize(const Fp4RowsArgs& a, cudaStream_t stream) {
  if (a.K <= 32 * 8 * kHold || a.rows >= 8192) return dequantize_t<F, TYPE, 32>(a, stream);
  return a.K <= 128 * 8 * kHold ? dequantize_t<F, TYPE, 128>(a, stream) : dequantize_t<F, TYPE, 256>(a, stream);
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
