// k_fp8_rows.cu -- rows and matrices to 8 bits and back.  128 elements of a row
// (rows), or a block of 128 x 128 (matrices), share one fp32 scale:
//   s = amax / 448 (1 where that is zero),  code = E4M3(x / s)
// each division one fp32 operation, codes to nearest with ties to even.  A block
// that holds a NaN or an infinity gets a NaN scale and codes of zero, so what it
// stands for is NaN.
//
// Bound: HBM.  A thread takes 16 elements at a time, 8 threads a row's block;
// all loads of a thread come first (four blocks along a row, or 4 rows of a
// matrix's block, which is read once and kept in registers while its maximum is found).
// From bf16, of a copy's rate: 65536 rows of 4096 117 us (1.01), 64 matrices of 4096 x
// 4096 471 us (1.01), 300 rows of 7168 4.5 us (latency).
// Quotients decide codes, so they have to be the rounded ones: one rounded
// reciprocal y = 1 / s serves 16 of them by Markstein's correction ("Computation of
// elementary functions on the IBM RISC System/6000", 1990): q = x y,
// r = x - q s (exact in a fused multiply-add), x / s = q + r y rounded, two elements an instruction.
// (The theorem excepts divisors whose significand is all ones, which s can have.  tests/test_quotients.py compares with
// divisions, nine dividends around each border of E4M3 for every ninth significand of the divisor, and was run for all 2^23:
// every quotient is the rounded one, those divisors' too.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.cuh"
#include "grouped_elementwise.cuh"
#include "launch_config.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kTileRows = kThreads / 8;  // 8 threads a block of a row
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr float kMaxCode = 448.0f;

// 16 elements of a row
template <int TYPE>
struct Vec {
  static constexpr int kQuads = TYPE == 2 ? 4 : 2;
  uint4 raw[kQuads];

  __device__ __forceinline__ void load(const void* row, int64_t vec) {
    const uint4* p = static_cast<const uint4*>(row) + vec * kQuads;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) raw[i] = __ldg(p + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) raw[i] = make_uint4(0, 0, 0, 0);
  }
  // elements 8 h .. 8 h + 7 as fp32
  __device__ __forceinline__ void values8(int h, float (&f)[8]) const {
    if constexpr (TYPE == 2) {
      const uint4 &a = raw[2 * h], &b = raw[2 * h + 1];
      f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
      f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
    } else {
      unpack8<TYPE == 1>(raw[h], f);
    }
  }
  // The largest magnitude as fp32 bits.  Magnitudes are ordered as their bits are (NaN and
  // infinities above all numbers), so 16-bit ones are compared packed in pairs.
  __device__ __forceinline__ uint32_t magnitude() const {
    constexpr uint32_t m = TYPE == 2 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const uint4& a = raw[i];
      if (TYPE == 2)
        r = max(max(max(r, a.x & m), a.y & m), max(a.z & m, a.w & m));
      else
        r = __vmaxu2(__vmaxu2(__vmaxu2(r, a.x & m), a.y & m), __vmaxu2(a.z & m, a.w & m));
    }
    if (TYPE == 2) return r;
    const uint32_t h = max(r >> 16, r & 0xFFFFu);
    return TYPE == 0 ? h << 16 : __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(h))));
  }
};

// four E4M3 codes (nearest, ties to even, saturating): element i in byte i
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// x becomes -(x / s), ny the negated rounded reciprocal.  (Negated, because with x = -0
// the residual is +0 and q + r y would lose the zero's sign.)
__device__ __forceinline__ void negated_quotients8(float (&x)[8], float s, float ny) {
#pragma unroll
  for (int i = 0; i < 8; i += 2)
    asm("{\n\t.reg .b64 x, d, n, q;\n\t"
        "mov.b64 x, {%0, %1};\n\t"
        "mov.b64 d, {%2, %2};\n\t"
        "mov.b64 n, {%3, %3};\n\t"
        "mul.rn.f32x2 q, x, n;\n\t"
        "fma.rn.f32x2 x, q, d, x;\n\t"
        "fma.rn.f32x2 x, x, n, q;\n\t"
        "mov.b64 {%0, %1}, x;\n\t}"
        : "+f"(x[i]), "+f"(x[i + 1])
        : "f"(s), "f"(ny));
}

// The scale of a block whose largest magnitude has the bits `amax`.
__device__ __forceinline__ float scale_of(uint32_t amax) {
  if (amax >= kInfBits) return __uint_as_float(0x7FC00000u);
  const float s = __fdiv_rn(__uint_as_float(amax), kMaxCode);
  return s > 0.0f ? s : 1.0f;
}

template <int TYPE>
__device__ __forceinline__ uint4 encode(const Vec<TYPE>& v, float s) {
  uint32_t w[4];
  if (s > 0x1p-80f && s < 0x1p80f) {  // no step below leaves fp32's normal range where it matters
    const float ny = -__frcp_rn(s);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8];
      v.values8(h, x);
      negated_quotients8(x, s, ny);
      w[2 * h] = codes4(x[0], x[1], x[2], x[3]) ^ 0x80808080u;
      w[2 * h + 1] = codes4(x[4], x[5], x[6], x[7]) ^ 0x80808080u;
    }
  } else if (s == s) {  // (the rare way: divisions)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[8];
      v.values8(h, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __fdiv_rn(x[i], s);
      w[2 * h] = codes4(x[0], x[1], x[2], x[3]);
      w[2 * h + 1] = codes4(x[4], x[5], x[6], x[7]);
    }
  } else {
    w[0] = w[1] = w[2] = w[3] = 0;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Rows: a CTA takes 32 rows x HOLD blocks, then the next 32 rows gridDim.y tiles on.
template <int TYPE, int HOLD>
__global__ void __launch_bounds__(kThreads) fp8_quantize_rows_kernel(const __grid_constant__ Fp8Args a) {
  pdl_wait();
  pdl_launch_dependents();
  const int part = threadIdx.x & 7, vecs = a.K / 16, b0 = blockIdx.x * HOLD;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * kTileRows + (threadIdx.x >> 3);;
       row += static_cast<int64_t>(gridDim.y) * kTileRows) {
    if (row - (threadIdx.x >> 3) >= a.rows) break;  // (uniform)
    const bool mine = row < a.rows;
    const size_t size = TYPE == 2 ? 4 : 2;
    const void* src = static_cast<const char*>(a.src) + static_cast<size_t>(row) * a.ld * size;
    Vec<TYPE> v[HOLD];
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int at = (b0 + i) * 8 + part;
      if (mine && at < vecs)
        v[i].load(src, at);
      else
        v[i].zero();
    }
    float s[HOLD];
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      uint32_t m = v[i].magnitude();
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
      const int at = (b0 + i) * 8 + part;
      s[i] = scale_of(m);
      if (mine && at < vecs)
        *reinterpret_cast<uint4*>(a.codes + static_cast<size_t>(row) * a.K + static_cast<size_t>(at) * 16) = encode(v[i], s[i]);
    }
    if (part == 0 && mine) {  // (lds is a multiple of 4: blocks past K get the 1 of zeros)
      float* to = a.scales + row * a.lds + b0;
      if constexpr (HOLD == 4)
        *reinterpret_cast<float4*>(to) = make_float4(s[0], s[1], s[2], s[3]);
      else
        *reinterpret_cast<float2*>(to) = make_float2(s[0], s[1]);
    }
  }
}

// Matrices: a CTA takes a block of 128 x 128, 4 rows a thread.
template <int TYPE>
__global__ void __launch_bounds__(kThreads) fp8_quantize_blocks_kernel(const __grid_constant__ Fp8Args a, int tiles,
                                                                       int kblocks) {
  __shared__ uint32_t warp_max[kThreads / 32];
  pdl_wait();
  pdl_launch_dependents();
  const int kb = static_cast<int>(blockIdx.x % static_cast<unsigned>(kblocks));
  const int mt = static_cast<int>(blockIdx.x / static_cast<unsigned>(kblocks)), g = mt / tiles, r0 = (mt - g * tiles) * 128;
  const int at = kb * 8 + (threadIdx.x & 7);
  const bool in = at < a.K / 16;
  const size_t size = TYPE == 2 ? 4 : 2;
  Vec<TYPE> v[4];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + i * kTileRows + (threadIdx.x >> 3);
    if (in && r < a.per)
      v[i].load(static_cast<const char*>(a.src) + static_cast<size_t>(g * a.per + r) * a.ld * size, at);
    else
      v[i].zero();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, v[i].magnitude());
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = max(m, warp_max[i]);
  const float s = scale_of(m);
  if (threadIdx.x == 0) a.scales[static_cast<size_t>(mt) * kblocks + kb] = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t r = r0 + i * kTileRows + (threadIdx.x >> 3);
    if (in && r < a.per)
      *reinterpret_cast<uint4*>(a.codes + static_cast<size_t>(g * a.per + r) * a.K + static_cast<size_t>(at) * 16) =
          encode(v[i], s);
  }
}

// Back: value = code * s, rounded to the output's type.  A thread's codes fill one store of
// 16 bytes; a warp takes HOLD runs of 32 such of a row, and loads them all first: 64 matrices
// of 4096 x 4096 to bf16 455 us (1.04 of a copy's rate), 65536 rows of 512 18 us (0.80).
// (16 codes a thread, its two stores apart: 570 to 640 us.  Grids of the SMs' size
// that walk the rows: 479 with eight CTAs an SM, 511 with two.)
template <int TYPE, int HOLD>
__global__ void __launch_bounds__(kThreads) fp8_dequantize_kernel(const __grid_constant__ Fp8Args a, int tiles,
                                                                  int kblocks) {
  constexpr int kCodes = TYPE == 2 ? 4 : 8;
  pdl_wait();
  pdl_launch_dependents();
  const int k0 = (static_cast<int>(blockIdx.x) * HOLD * 32 + (threadIdx.x & 31)) * kCodes;
  for (int64_t row = static_cast<int64_t>(blockIdx.y) * kWarps + (threadIdx.x >> 5); row < a.rows;
       row += static_cast<int64_t>(gridDim.y) * kWarps) {
    const float* sc = a.scales + row * a.lds;
    if (a.per) {
      const int64_t g = static_cast<uint32_t>(row) / static_cast<uint32_t>(a.per);
      sc = a.scales + (g * tiles + (row - g * a.per) / 128) * kblocks;
    }
    const uint8_t* src = a.codes + static_cast<size_t>(row) * a.K;
    uint2 c[HOLD];
    float s[HOLD];
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int k = k0 + i * 32 * kCodes;
      if (k >= a.K) continue;
      if constexpr (TYPE == 2)
        c[i].x = __ldg(reinterpret_cast<const uint32_t*>(src + k));
      else
        c[i] = __ldg(reinterpret_cast<const uint2*>(src + k));
      s[i] = __ldg(sc + k / 128);
    }
#pragma unroll
    for (int i = 0; i < HOLD; ++i) {
      const int k = k0 + i * 32 * kCodes;
      if (k >= a.K) continue;
      float f[kCodes];
#pragma unroll
      for (int j = 0; j < kCodes / 2; ++j) {
        uint32_t h;  // two codes to fp16, exactly
        const uint32_t w = j < 2 ? c[i].x : c[i].y;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w >> (16 * (j & 1)))));
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h));
        f[2 * j] = __fmul_rn(p.x, s[i]);
        f[2 * j + 1] = __fmul_rn(p.y, s[i]);
      }
      const size_t size = TYPE == 2 ? 4 : 2;
      uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(a.dst) + (static_cast<size_t>(row) * a.ld + k) * size);
      if constexpr (TYPE == 2)
        *dst = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
      else
        *dst = pack8<TYPE == 1>(f);
    }
  }
}

dim3 rows_grid(const Fp8Args& a, int hold) {
  const int64_t tiles = (a.rows + kTileRows - 1) / kTileRows, blocks = (a.K + 127) / 128;
  return dim3(static_cast<unsigned>((blocks + hold - 1) / hold), static_cast<unsigned>(tiles < 65535 ? tiles : 65535));
}

template <int TYPE>
cudaError_t quantize(const Fp8Args& a, cudaStream_t stream) {
  constexpr int kHold = TYPE == 2 ? 2 : 4;
  if (a.per) {
    const int64_t tiles = (a.per + 127) / 128, kblocks = (a.K + 127) / 128;
    return launch_pdl(fp8_quantize_blocks_kernel<TYPE>, dim3(static_cast<unsigned>(a.rows / a.per * tiles * kblocks)),
                      dim3(kThreads), 0, stream, a, static_cast<int>(tiles), static_cast<int>(kblocks));
  }
  return launch_pdl(fp8_quantize_rows_kernel<TYPE, kHold>, rows_grid(a, kHold), dim3(kThreads), 0, stream, a);
}

template <int TYPE>
cudaError_t dequantize(const Fp8Args& a, cudaStream_t stream) {
  constexpr int kHold = 4, kSpan = kHold * 32 * (TYPE == 2 ? 4 : 8);
  const int64_t tiles = (a.rows + kWarps - 1) / kWarps;
  const dim3 grid((a.K + kSpan - 1) / kSpan, static_cast<unsigned>(tiles < 65535 ? tiles : 65535));
  return launch_pdl(fp8_dequantize_kernel<TYPE, kHold>, grid, dim3(kThreads), 0, stream, a,
                    static_cast<int>(a.per ? (a.per + 127) / 128 : 0), (a.K + 127) / 128);
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8Args& a, cudaStream_t stream) {
  return a.type == 2 ? quantize<2>(a, stream) : a.type == 1 ? quantize<1>(a, stream) : quantize<0>(a, stream);
}

cudaError_t launch_fp8_dequantize(const Fp8Args& a, cudaStream_t stream) {
  return a.type == 2 ? dequantize<2>(a, stream) : a.type == 1 ? dequantize<1>(a, stream) : dequantize<0>(a, stream);
}

}  // namespace moe
