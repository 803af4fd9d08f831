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
// measured copy rate, so the instructions per element decide.  A thread takes 16
// elements at a time (a whole NVFP4 block, half an MXFP4 one: the scale is computed once for
// them) and hold_of(type) such vectors at once, all loads first; TPR threads share a row.
//   - The block maximum is taken on the packed 16-bit magnitudes, whose order
//     is that of their bits (NaN and infinities above all numbers).
//   - NVFP4's quotients decide codes, so they have to be the rounded quotients.
//     One rounded reciprocal y = 1 / d serves 16 of them by Markstein's correction
//     ("Computation of elementary functions on the IBM RISC System/6000", 1990):
//     q = x y, r = x - q d (exact in a fused multiply-add), x / d = q + r y rounded, on two elements an
//     instruction.  (The theorem excepts divisors whose significand is all ones, which d and 6 g
//     can have.  tests/test_quotients.py compares with divisions, nine dividends around each border of E2M1 and of E4M3
//     for every ninth significand of the divisor, and was run for all 2^23: every quotient is the rounded one, those divisors'
//     too.)  (Products with a lowered and a raised reciprocal, whose codes agree unless the
//     quotient lies at a border, cost a second conversion, the slowest
//     instruction here: 105 us for 134 M elements.)
// Measured, 134 M bf16 elements: NVFP4 65 us (0.78 of the copy rate), MXFP4 48 to
// 50 us (1.0); back to 16 bits 50 us, to fp32 88 us.  1.07 G elements to MXFP4 and back 755 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "fp4.cuh"
#include "grouped_elementwise.cuh"
#include "pdl.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// vectors of 16 elements a thread holds: 32 registers
__host__ __device__ constexpr int hold_of(int type) { return type == 2 ? 2 : 4; }

struct RowPlace {
  int group, tile_row, in_tile;
  bool on;
};

// The offsets of up to kOneRound groups, entry 32 i + lane in [i], for a kernel that reads
// them ahead of its row: the inverse with a warp per row (134 M elements 58 -> 52 us; with
// more warps per row, 1021 rows of 7168, 4.7 -> 5.0; the quantizer, whose registers are full,
// gains nothing).
constexpr int kOneRound = 256;
struct Offsets {
  int at[kOneRound / 32 + 1];
  __device__ __forceinline__ Offsets(const Fp4RowsArgs& a, int lane) {
#pragma unroll
    for (int i = 0; i <= kOneRound / 32; ++i)
      at[i] = a.offsets && a.G <= kOneRound && 32 * i + lane <= a.G ? __ldg(a.offsets + 32 * i + lane) : 0x7FFFFFFF;
  }
};
struct NoOffsets {
  __device__ __forceinline__ NoOffsets(const Fp4RowsArgs&, int) {}
};

// The group and scale place of row p (warp-collective, the same p in a warp): the
// last group that starts at p or before, from `off`, or in two rounds of 32
// comparisons among up to 1024.  Rows of no group, and places that lists out of order
// could lead to, are off.
template <typename Ahead>
__device__ __forceinline__ RowPlace place_of(const Fp4RowsArgs& a, const Ahead& off, int p, int lane) {
  constexpr bool kRead = std::is_same_v<Ahead, Offsets>;
  RowPlace r{0, 0, 0, false};
  int start, count;
  if (kRead && a.offsets && a.G <= kOneRound) {
    if constexpr (kRead) {
      int n = 0, from = -1, to = 0x7FFFFFFF;
#pragma unroll
      for (int i = 0; i <= kOneRound / 32; ++i) {
        const bool before = off.at[i] <= p;
        n += before && 32 * i + lane < a.G;
        from = before ? max(from, off.at[i]) : from;
        to = before ? to : min(to, off.at[i]);
      }
      const int g = __reduce_add_sync(0xFFFFFFFFu, n) - 1;
      start = __reduce_max_sync(0xFFFFFFFFu, from);
      to = __reduce_min_sync(0xFFFFFFFFu, to);  // the next group's start
      if (g < 0 || start < 0 || to == 0x7FFFFFFF) return r;
      count = a.counts ? __ldg(a.counts + g) : to - start;
      r.group = g;
      r.tile_row = start / 128 + g;
    }
  } else if (a.offsets) {
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

constexpr int kElems = 16;  // of a vector

template <int TYPE>
struct Vec {
  static constexpr int kQuads = TYPE == 2 ? 4 : 2;
  uint4 raw[kQuads];
};

template <int TYPE>
__device__ __forceinline__ void load_vec(const void* row, int v, Vec<TYPE>& x) {
  const uint4* p = static_cast<const uint4*>(row) + static_cast<int64_t>(v) * Vec<TYPE>::kQuads;
#pragma unroll
  for (int i = 0; i < Vec<TYPE>::kQuads; ++i) x.raw[i] = __ldg(p + i);
}

template <int TYPE>
__device__ __forceinline__ void zero_vec(Vec<TYPE>& x) {
#pragma unroll
  for (int i = 0; i < Vec<TYPE>::kQuads; ++i) x.raw[i] = make_uint4(0, 0, 0, 0);
}

// Elements 8 h .. 8 h + 7 as fp32.
template <int TYPE>
__device__ __forceinline__ void values8(const Vec<TYPE>& x, int h, float (&f)[8]) {
  if constexpr (TYPE == 2) {
    const uint4 &a = x.raw[2 * h], &b = x.raw[2 * h + 1];
    f[0] = __uint_as_float(a.x), f[1] = __uint_as_float(a.y), f[2] = __uint_as_float(a.z), f[3] = __uint_as_float(a.w);
    f[4] = __uint_as_float(b.x), f[5] = __uint_as_float(b.y), f[6] = __uint_as_float(b.z), f[7] = __uint_as_float(b.w);
  } else {
    unpack8<TYPE == 1>(x.raw[h], f);
  }
}

// Largest magnitudes as ordered bits: packed pairs of 16 bits, or fp32.
template <int TYPE>
__device__ __forceinline__ uint32_t max_mag(uint32_t a, uint32_t b) {
  return TYPE == 2 ? max(a, b) : __vmaxu2(a, b);
}
template <int TYPE>
__device__ __forceinline__ uint32_t mag_vec(const Vec<TYPE>& x) {
  constexpr uint32_t m = TYPE == 2 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < Vec<TYPE>::kQuads; ++i) {
    const uint4& a = x.raw[i];
    r = max_mag<TYPE>(r, max_mag<TYPE>(max_mag<TYPE>(a.x & m, a.y & m), max_mag<TYPE>(a.z & m, a.w & m)));
  }
  return r;
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

__device__ __forceinline__ uint32_t e4m3_of(float u) {  // u >= 0
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.0f), "f"(u));
  return r;
}
__device__ __forceinline__ float e4m3_to(uint32_t c) {  // 0x7F is NaN
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// What a row's NVFP4 codes need: g and the reciprocal of 6 g.  `plain`: g is so
// near 1 that no step below leaves fp32's normal range where it matters (else,
// or with no number, quotients are divided out).
struct NvRow {
  float g, six_g, inv_six_g;
  bool plain;
};

__device__ __forceinline__ NvRow nv_row(float g) {
  NvRow r;
  r.g = g;
  r.six_g = __fmul_rn(6.0f, g);
  r.inv_six_g = __frcp_rn(r.six_g);
  r.plain = g > 0x1p-80f && g < 0x1p80f;
  return r;
}

// a / d by Markstein's correction, y = the rounded 1 / d
__device__ __forceinline__ float quotient(float a, float d, float y) {
  const float q = __fmul_rn(a, y);
  return __fmaf_rn(__fmaf_rn(-q, d, a), y, q);
}

// The same for eight, negated: x becomes -(x / d), ny the negated reciprocal.
// (With x = -0 the residual is +0, so q + r y would lose the zero's sign; here
// every product of the last step has the sign of -0.)
__device__ __forceinline__ void negated_quotients8(float (&x)[8], float d, float ny) {
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
        : "f"(d), "f"(ny));
}

// The rare way: divisions.
__device__ __noinline__ uint32_t divided_codes(float x0, float x1, float x2, float x3, float x4, float x5, float x6,
                                               float x7, float d) {
  const float x[8] = {__fdiv_rn(x0, d), __fdiv_rn(x1, d), __fdiv_rn(x2, d), __fdiv_rn(x3, d),
                      __fdiv_rn(x4, d), __fdiv_rn(x5, d), __fdiv_rn(x6, d), __fdiv_rn(x7, d)};
  return codes8(x);
}

// Codes and scale byte of 16 elements of a block whose largest magnitude has
// the fp32 bits `amax`.
template <Fp4Format F, int TYPE>
__device__ __forceinline__ uint2 encode(const Vec<TYPE>& v, uint32_t amax, const NvRow& nv, uint32_t& scale) {
  uint32_t w[2];
  float x[8];
  if constexpr (F == Fp4Format::kMx) {
    int e = static_cast<int>(amax >> 23) - 127 - 2;  // (a subnormal maximum clamps too)
    e = e < -127 ? -127 : e;
    scale = amax >= kInfBits ? 255u : static_cast<uint32_t>(e + 127);
    // 2^-e; x 2^-e is exact down to magnitudes whose code is 0 either way
    const uint32_t inv = static_cast<uint32_t>(127 - e) << 23;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (TYPE == 0) {
        const uint32_t q[4] = {v.raw[h].x, v.raw[h].y, v.raw[h].z, v.raw[h].w};
        const uint32_t s2 = inv | (inv >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 p = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&q[i]),
                                           *reinterpret_cast<const __nv_bfloat162*>(&s2));
          const uint32_t b = *reinterpret_cast<const uint32_t*>(&p);
          x[2 * i] = __uint_as_float(b << 16);
          x[2 * i + 1] = __uint_as_float(b & 0xFFFF0000u);
        }
      } else {
        values8<TYPE>(v, h, x);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= __uint_as_float(inv);
      }
      w[h] = codes8(x);
    }
    return make_uint2(w[0], w[1]);
  }
  const float top = __uint_as_float(amax);
  if (!nv.plain) {  // (whole rows)
    scale = nv.g == nv.g ? e4m3_of(__fdiv_rn(top, nv.six_g)) : 0x7Fu;
    const float d = __fmul_rn(e4m3_to(scale), nv.g);
    if (!(d > 0.0f)) return make_uint2(0u, 0u);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      values8<TYPE>(v, h, x);
      w[h] = divided_codes(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], d);
    }
    return make_uint2(w[0], w[1]);
  }
  scale = e4m3_of(quotient(top, nv.six_g, nv.inv_six_g));
  const float d = __fmul_rn(e4m3_to(scale), nv.g), ny = -__frcp_rn(d);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    values8<TYPE>(v, h, x);
    negated_quotients8(x, d, ny);
    w[h] = codes8(x) ^ 0x88888888u;
  }
  return scale ? make_uint2(w[0], w[1]) : make_uint2(0u, 0u);
}

// TPR threads per row.  NVFP4 per row: the row's maximum first; per group: from
// gscale, which then holds the maxima's bits.
template <Fp4Format F, int TYPE, int TPR>
__global__ void __launch_bounds__(kThreads, 4) fp4_quantize_kernel(const __grid_constant__ Fp4RowsArgs a) {
  constexpr int kRows = kThreads / TPR, kWarpsPerRow = TPR / 32;
  pdl_wait();
  pdl_launch_dependents();
  __shared__ uint32_t warp_max[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = threadIdx.x % TPR;
  const int64_t p64 = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / TPR;
  const bool in = p64 < a.rows;
  const int p = in ? static_cast<int>(p64) : 0;
  const int vecs = a.K / kElems;
  const char* src = static_cast<const char*>(a.src) + p * a.ld * (TYPE == 2 ? 4 : 2);
  constexpr int kHold = hold_of(TYPE);
  Vec<TYPE> held[kHold];
  // (a row of no group is read in vain: its place is looked up meanwhile)
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    if (t + i * TPR < vecs)
      load_vec<TYPE>(src, t + i * TPR, held[i]);
    else
      zero_vec<TYPE>(held[i]);
  }
  const RowPlace r = place_of(a, NoOffsets(a, lane), p, lane);
  const bool row_on = in && r.on;
  NvRow nv{};
  if constexpr (F == Fp4Format::kNv) {
    float g;
    if (!a.per_group) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < kHold; ++i) m = max_mag<TYPE>(m, mag_vec<TYPE>(held[i]));
      for (int v0 = kHold * TPR + t; v0 < vecs; v0 += kHold * TPR) {
        Vec<TYPE> x[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          if (v0 + i * TPR < vecs)
            load_vec<TYPE>(src, v0 + i * TPR, x[i]);
          else
            zero_vec<TYPE>(x[i]);
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) m = max_mag<TYPE>(m, mag_vec<TYPE>(x[i]));
      }
      m = __reduce_max_sync(0xFFFFFFFFu, mag_bits<TYPE>(m));
      if (kWarpsPerRow > 1) {
        if (lane == 0) warp_max[warp] = m;
        // the row's warps alone (the whole block: 66.3 instead of 64.5 us for 134 M elements)
        asm volatile("barrier.sync %0, %1;" ::"r"(1 + warp / kWarpsPerRow), "n"(TPR) : "memory");
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
  constexpr int kLanesPerBlock = fp4_block(F) / kElems;
  uint8_t* codes = a.codes + static_cast<size_t>(p) * (a.K / 2);
  uint8_t* scales = row_scales(a, r, chunks);
  // this lane's places of vector t; one of TPR vectors further is whole chunks further
  constexpr int kScaleStep = TPR / kLanesPerBlock / 4 * 512;
  const int block = t / kLanesPerBlock;
  codes += t * 8;
  uint8_t* scale_at = scales + (block >> 2) * 512 + (block & 3);
  const bool scale_lane = lane % kLanesPerBlock == 0;
  auto emit = [&](int i, const Vec<TYPE>& x, bool on) {  // whole warps; a block's lanes are all on or all off
    uint32_t m = mag_vec<TYPE>(x);
#pragma unroll
    for (int o = 1; o < kLanesPerBlock; o <<= 1) m = max_mag<TYPE>(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    uint32_t sc;
    const uint2 w = encode<F, TYPE>(x, mag_bits<TYPE>(m), nv, sc);
    if (on) {
      *reinterpret_cast<uint2*>(codes + i * (TPR * 8)) = w;
      if (scale_lane) scale_at[i * kScaleStep] = static_cast<uint8_t>(sc);
    }
  };
  const int w0 = t & ~31;  // the warp's first vector of a round
#pragma unroll
  for (int i = 0; i < kHold; ++i)
    if (i * TPR + w0 < vecs) emit(i, held[i], t + i * TPR < vecs);
  for (int v0 = kHold * TPR; v0 + w0 < vecs; v0 += kHold * TPR) {
    codes += kHold * TPR * 8;
    scale_at += kHold * kScaleStep;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (v0 + t + i * TPR < vecs)
        load_vec<TYPE>(src, v0 + t + i * TPR, held[i]);
      else
        zero_vec<TYPE>(held[i]);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (v0 + i * TPR + w0 < vecs) emit(i, held[i], v0 + t + i * TPR < vecs);
  }
  // blocks of the last chunk past K: zero scales
  const int blocks = a.K / fp4_block(F);
  if (t < chunks * 4 - blocks) scales[(chunks - 1) * 512 + ((blocks + t) & 3)] = 0;
}

// Largest magnitude of every group's rows into gscale's bits (zero before).
template <int TYPE>
__global__ void __launch_bounds__(kThreads) fp4_group_amax_kernel(const __grid_constant__ Fp4RowsArgs a) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t p64 = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (p64 >= a.rows) return;
  const int p = static_cast<int>(p64), vecs = a.K / kElems;
  const char* src = static_cast<const char*>(a.src) + p * a.ld * (TYPE == 2 ? 4 : 2);
  constexpr int kHold = hold_of(TYPE);
  uint32_t m = 0;
  for (int v0 = 0; v0 < vecs; v0 += kHold * 32) {
    Vec<TYPE> held[kHold];
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      if (v0 + i * 32 + lane < vecs)
        load_vec<TYPE>(src, v0 + i * 32 + lane, held[i]);
      else
        zero_vec<TYPE>(held[i]);
    }
#pragma unroll
    for (int i = 0; i < kHold; ++i) m = max_mag<TYPE>(m, mag_vec<TYPE>(held[i]));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, mag_bits<TYPE>(m));
  const RowPlace r = place_of(a, NoOffsets(a, lane), p, lane);
  if (r.on && lane == 0) atomicMax(reinterpret_cast<unsigned int*>(a.gscale) + r.group, m);
}

// maxima -> scales, in place
__global__ void fp4_group_scale_kernel(float* gscale, int n) {
  pdl_wait();
  pdl_launch_dependents();
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) gscale[i] = nv_global(__float_as_uint(gscale[i]));
}

// four codes (16 bits) -> their values
__device__ __forceinline__ void decode4(uint32_t w, float* f) {
  uint32_t h[2];
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t}"
      : "=r"(h[0]), "=r"(h[1])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

constexpr int kAhead = 8;

// A thread writes 16 bytes at a time (8 elements of 16 bits or 4 of 32), so a
// warp's stores are contiguous; kAhead of them per round, their loads first.
template <Fp4Format F, int TYPE, int TPR>
__global__ void __launch_bounds__(kThreads) fp4_dequantize_kernel(const __grid_constant__ Fp4RowsArgs a) {
  constexpr int kVec = TYPE == 2 ? 4 : 8;
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, t = threadIdx.x % TPR;
  const int64_t p64 = static_cast<int64_t>(blockIdx.x) * (kThreads / TPR) + threadIdx.x / TPR;
  if (p64 >= a.rows) return;
  const int p = static_cast<int>(p64);
  const int vecs = a.K / kVec, chunks = (a.K + fp4_chunk(F) - 1) / fp4_chunk(F);
  const uint8_t* codes = a.codes + static_cast<size_t>(p) * (a.K / 2);
  auto load = [&](int v) -> uint32_t {
    if (v >= vecs) return 0u;
    return kVec == 8 ? __ldcs(reinterpret_cast<const uint32_t*>(codes) + v)
                     : static_cast<uint32_t>(__ldcs(reinterpret_cast<const unsigned short*>(codes) + v));
  };
  const std::conditional_t<TPR == 32, Offsets, NoOffsets> off(a, lane);
  uint32_t w[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) w[i] = load(t + i * TPR);
  const RowPlace r = place_of(a, off, p, lane);
  if (!r.on) return;
  const uint8_t* scales = row_scales(a, r, chunks);
  uint4* dst = reinterpret_cast<uint4*>(static_cast<char*>(a.dst) + p * a.ld * (TYPE == 2 ? 4 : 2));
  const float g = F == Fp4Format::kNv ? __ldg(a.gscale + (a.per_group ? r.group : p)) : 1.0f;
  for (int v0 = 0; v0 < vecs; v0 += kAhead * TPR) {
    uint32_t sc[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = v0 + t + i * TPR, block = v / (fp4_block(F) / kVec);
      if (v0 > 0) w[i] = load(v);
      sc[i] = v < vecs ? __ldg(scales + (block >> 2) * 512 + (block & 3)) : 0u;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int v = v0 + t + i * TPR;
      if (v >= vecs) break;
      float f[8];
      decode4(w[i], f);
      if (kVec == 8) decode4(w[i] >> 16, f + 4);
      if constexpr (F == Fp4Format::kMx) {
        // 2^(sc - 127); the smallest is subnormal, 255 stands for NaN
        const float s =
            sc[i] == 255u ? __uint_as_float(0x7FC00000u) : sc[i] ? __uint_as_float(sc[i] << 23) : 0x1p-127f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] = __fmul_rn(f[j], s);
      } else {
        const float s = e4m3_to(sc[i]);  // times a code: exact
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] = __fmul_rn(__fmul_rn(f[j], s), g);
      }
      if constexpr (TYPE == 2)
        __stcs(dst + v, make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                                   __float_as_uint(f[3])));
      else
        __stcs(dst + v, pack8<TYPE == 1>(f));
    }
  }
}

template <Fp4Format F, int TYPE, int TPR>
cudaError_t quantize_t(const Fp4RowsArgs& a, cudaStream_t stream) {
  constexpr int rows = kThreads / TPR;
  return launch_pdl(fp4_quantize_kernel<F, TYPE, TPR>, dim3(static_cast<unsigned>((a.rows + rows - 1) / rows)),
                    dim3(kThreads), 0, stream, a);
}

// Threads per row: as few as hold its vectors at once, `hold` each; more where there are
// few rows, up to `most` threads in all.
int threads_per_row(int vecs, int hold, int64_t rows, int64_t most) {
  int tpr = 32;
  while (tpr < 256 && vecs > tpr * hold) tpr *= 2;
  while (tpr < 256 && tpr < vecs && rows * tpr * 2 <= most) tpr *= 2;
  return tpr;
}
constexpr int64_t kResident = 152 * 1024;  // threads of the quantizer that run at once

template <Fp4Format F, int TYPE>
cudaError_t quantize(const Fp4RowsArgs& a, cudaStream_t stream) {
  const bool whole = F == Fp4Format::kNv && !a.per_group;
  if (F == Fp4Format::kNv && a.per_group) {
    cudaError_t e = cudaMemsetAsync(a.gscale, 0, sizeof(float) * a.G, stream);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};  // (after a memset: no programmatic dependency)
    cfg.gridDim = dim3(static_cast<unsigned>((a.rows + 7) / 8));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    if ((e = cudaLaunchKernelEx(&cfg, fp4_group_amax_kernel<TYPE>, a)) != cudaSuccess) return e;
  }
  const int vecs = a.K / kElems;
  // A scale per row asks for the row's maximum before any code, so all of its vectors are to be
  // held; else a warp, whose look-up of the place then serves most elements.  Measured (us, bf16,
  // 32 / 64 / 128 / 256 threads): NVFP4, 64 x 4096: 5.0 / 3.2 / 2.7 / 2.3, 1021 x 7168: 7.7 / 6.3 / 6.4 / 6.9,
  // 2048 x 4096: 6.6 / 6.4 / 7.7 / 9.6, 32768 x 4096: 71 / 65 / 93 / 127, 8192 x 8192: 44 / 42 / 35 / 45;
  // MXFP4, 64 x 4096: 3.1 / 2.2 / 1.9 / 1.8, 2048 x 4096: 4.3 / 4.2 / 4.4 / 5.7, 32768 x 4096: 48 / 49 / 55 / 79.
  cudaError_t e;
  switch (threads_per_row(vecs, whole ? hold_of(TYPE) : vecs, a.rows, kResident)) {
    case 32: e = quantize_t<F, TYPE, 32>(a, stream); break;
    case 64: e = quantize_t<F, TYPE, 64>(a, stream); break;
    case 128: e = quantize_t<F, TYPE, 128>(a, stream); break;
    default: e = quantize_t<F, TYPE, 256>(a, stream);
  }
  if (e != cudaSuccess || F != Fp4Format::kNv || !a.per_group) return e;
  return launch_pdl(fp4_group_scale_kernel, dim3((a.G + 127) / 128), dim3(128), 0, stream, a.gscale, a.G);
}

template <Fp4Format F, int TYPE, int TPR>
cudaError_t dequantize_t(const Fp4RowsArgs& a, cudaStream_t stream) {
  constexpr int rows = kThreads / TPR;
  return launch_pdl(fp4_dequantize_kernel<F, TYPE, TPR>, dim3(static_cast<unsigned>((a.rows + rows - 1) / rows)),
                    dim3(kThreads), 0, stream, a);
}

template <Fp4Format F, int TYPE>
cudaError_t dequantize(const Fp4RowsArgs& a, cudaStream_t stream) {
  // (its loads are in flight kAhead at a time.)  Measured (us, 32 / 64 / 128 / 256 threads): to fp32, 1021 x
  // 7168: 9.9 / 7.6 / 8.7 / 6.7, 32768 x 4096: 93 / 91 / 88 / 87, 8192 x 8192: 62 / 52 / 48 / 46; to 16 bits, 64 x 4096:
  // 3.4 / 2.6 / 2.2 / 2.2, 2048 x 4096: 4.7 / 5.7 / 4.6 / 6.3, 32768 x 4096: 52 / 50 / 52 / 78, 8192 x 8192: 30 / 33 / 26 /
  // 28, 32768 x 1408: 20 / 24 / 37 / 65.
  switch (threads_per_row(a.K / (TYPE == 2 ? 4 : 8), kAhead, a.rows, 2 * kResident)) {
    case 32: return dequantize_t<F, TYPE, 32>(a, stream);
    case 64: return dequantize_t<F, TYPE, 64>(a, stream);
    case 128: return dequantize_t<F, TYPE, 128>(a, stream);
    default: return dequantize_t<F, TYPE, 256>(a, stream);
  }
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
