// k_fp8_gemm.cu -- the grouped products on 8-bit operands (E4M3) whose fp32
// scales cover 128 elements of a row, or 128 x 128 of a matrix:
//   forward         y[p, :]  = x[p, :] w_g^T       (p in group g)
//   input gradient  dx[p, :] = dy[p, :] w_g
// The reduction is cut into the blocks b that share a scale:
//   y[p, f] = sum_b (sx[b, p] sw[f / 128, b]) D_b[p, f],  D_b = sum over the block of the codes' products
// Only D_b is the tensor core's (kind::f8f6f4, fp32 in TMEM, K = 32 an MMA); the
// scales are no powers of two, so D_b leaves TMEM block by block and is summed in
// registers, one fp32 multiply-add per element and block.  That sum rounds to nearest;
// the tensor core's own cuts towards zero stay inside a block of 128.  Scales whose product
// is no normal fp32 number meet the block's sum one after the other (one_factor).
//
// Units and work split as in k_grouped_gemm.cu and k_grouped_pair.cu; the input gradient
// reads the stored matrix as an MN-major operand.  A K-block is one block of scales, 128
// bytes of codes a row.
//
// Few rows a group: single CTAs, stream-K, the weights on the MMA's M side (128 features x
// 32 rows a unit), bound by HBM.
//
// More: units of 256 features, here with the rows on the MMA's M side, so that a TMEM
// lane is a row of x and an epilogue warp's 128 columns are one block of features: a
// thread multiplies a whole block with one scale.  (With the weights on the M side columns
// are rows with a scale each, and reading them from shared memory took half of the time: one
// group of 8192 rows, N = K = 8192: 772 us.)  MMAs of M = 128 (256 for pairs) take the same time for
// any number of rows.
//   single CTAs: units of 128 rows, bound by HBM where a group has no more
//   CTA pairs: units of 256 rows handed out on demand, where the mean group's units of 256 rows take less time
//   than its units of 128 (choose_fp8_plan: 129 to 256, 385 to 512 and above 640 rows a group)
//                                         pairs   single CTAs
//   64 x 100 rows, N = 8192, K = 4096      435    354 us
//   64 x 512 rows, N = K = 4096            450    510
//   8192 rows, N = K = 8192                422    480
//   - A block's MMAs (128 x 256 x 128 an SM) take 512 cycles at the FP8 rate.  The
//     eight epilogue warps read 128 x 256 accumulators for it and issue as many
//     multiply-adds, paired (fma.f32x2), 64 a thread; a load is under way while the one before it is summed.
//   - The sums take 128 registers of each epilogue thread: setmaxnreg moves them there.
//     What leads from one unit to the next is worked out anew for each, since registers kept for it
//     would spill, and any spill costs a quarter of the rate.
//   - TMEM holds two blocks of 256 columns: one is read while the next is computed.
// Bound: reading TMEM beside the MMAs that write it.  One group of 8192 rows, N = K = 8192, pairs: 421 us (412 to 438 over boxes; 2.6 PFLOP/s,
// 870 cycles a block); with a quarter of the multiply-adds 417, without reading TMEM 333.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bounded_wait.cuh"
#include "fp8.cuh"
#include "launch_config.cuh"
#include "pair_sched.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kABytes = 128 * 128;  // 128 features x 128 of the reduction

enum : int {
  kWaitSlotFree = 1,
  kWaitAccFree = 2,
  kWaitSlotFull = 3,
  kWaitAccFull = 4,
  kWaitPartials = 5,
  kWaitUnit = 10
};

// A stage's weights as the MMA reads them: K-major rows of 128 codes, or (input gradient)
// MN-major rows of 128 features.  Steps of K = 32.
template <bool DGRAD>
__device__ __forceinline__ uint64_t w_desc(uint32_t saddr) {
  return DGRAD ? sdesc_mnmajor_sw128(saddr, kABytes) : sdesc_kmajor_sw128(saddr);
}
template <bool DGRAD>
constexpr uint64_t kStepW = (DGRAD ? 32 * 128 : 32) >> 4;
constexpr uint64_t kStepX = 32 >> 4;

__device__ __forceinline__ uint16_t to16(float v, bool fp16) {
  return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// A block's sum times sx sw.  Where the product of the scales is a normal fp32 number, that is one factor.  Elsewhere the
// sum meets the larger scale, then the smaller one: it is 0 or lies in [2^-18, 2^25), so if it overflows with the
// larger scale the result does too (beyond fp32's largest product the smaller scale is above 1), and if it falls below the normal
// range with it the result vanishes (the scales are then below 2^-108).
__device__ __forceinline__ bool one_factor(float product) {
  return (__float_as_uint(product) << 1) - 0x01000000u < 0xFE000000u;  // (neither the lowest exponent nor the highest)
}
// The second factor (s) and the first from two scales; their product and 1 where one factor does.
__device__ __forceinline__ void two_factors(float& s, float& first) {
  const float product = __fmul_rn(s, first), a = s, b = first;
  const bool one = one_factor(product), a_larger = fabsf(a) > fabsf(b);
  first = one ? 1.0f : a_larger ? a : b;
  s = one ? product : a_larger ? b : a;
}

__device__ __forceinline__ uint64_t twice(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}

// The scales of a unit's features (one block of 128) along the reduction.
template <bool DGRAD>
__device__ __forceinline__ const float* feature_scales(const Fp8GemmArgs& a, int g, int feat) {
  const int fb = min(feat / 128, (DGRAD ? a.w_cols : a.w_rows) - 1);  // (features past the end are dropped)
  const float* m = a.w_scales + static_cast<int64_t>(g) * a.w_rows * a.w_cols;
  return DGRAD ? m + fb : m + static_cast<int64_t>(fb) * a.w_cols;
}

// ------------------------------------------------------------------ few rows: single CTAs

constexpr int kUnitRows = 32, kRowBox = 16;
constexpr int kStageBytes = kABytes + kUnitRows * 128;
constexpr int kStages = 10;
constexpr int kAccs = 4;
constexpr int kAhead = 3;  // blocks whose scales are loaded ahead
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = kAccs * kUnitRows;
constexpr int kBarBytes = 256;
constexpr int kTabBytes = 3 * (kGroupsSmem[0] + 1) * 4;
constexpr int kScaleBytes = 4 * 2 * 2 * kUnitRows * 4;  // per epilogue warp, two blocks, two factors
constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + kBarBytes + kScaleBytes + kTabBytes;
static_assert((2 * kStages + 2 * kAccs + 1) * 8 + 8 <= kBarBytes, "barrier area");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

template <bool DGRAD>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_small_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ Fp8GemmArgs args) {
  const GroupedGemmArgs& a = args.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + kAccs;
  uint64_t* done = tempty + kAccs;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  float* scales = reinterpret_cast<float*>(smem + kStages * kStageBytes + kBarBytes);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + kStages * kStageBytes + kBarBytes + kScaleBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = static_cast<int>(blockIdx.x), workers = static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);  // the epilogue warps
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();  // the plan kernel's tables
  const GroupedTables tables = grouped_tables(a, tab, kGroupsSmem[0], kThreads);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int total_units = tables.unit_off[a.G];
  const int kblocks = (a.R + 127) / 128;
  GroupedUnits units(tables, a.G, 1, kUnitRows);  // each thread walks its role's units
  GroupedRange rg(total_units, kblocks, worker, workers);
  int u, kb0, kb1;

  if (warp == 0) {
    // ---------------- TMA producer (one lane issues)
    const bool issue = elect_one();
    const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_last();
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      const int feat = un.tile * 128;
      const int rows = (un.n + kRowBox - 1) / kRowBox * kRowBox;  // whole boxes
      // a weight tile read by one token chunk only is streamed; by more, kept
      const uint64_t pol_w = units.chunks > 1 ? pol_keep : pol_stream;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          break;
        }
        if (issue) {
          uint8_t* sa = smem + stage * kStageBytes;
          uint64_t* bar = &full[stage];
          mbar_arrive_expect_tx(bar, kABytes + rows * 128);
          if constexpr (DGRAD)  // 128 rows of w x 128 of its columns, which are the features
            tma_load_3d(sa, &tm_w, bar, feat, kb * 128, un.g, pol_w);
          else
            tma_load_3d(sa, &tm_w, bar, kb * 128, feat, un.g, pol_w);
          for (int r = 0; r < rows; r += kRowBox)
            tma_load_2d(sa + kABytes + r * 128, &tm_x, bar, kb * 128, un.tok0 + r, pol_keep);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && issue) raise_timeout(a.err, abort_flag, kKernFp8Gemm, kWaitSlotFree);
    // every load issued has landed before the CTA exits
    for (int s = 0; s < kStages; ++s) {
      if (issued <= s) break;
      const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
      const int never = 0;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[s], par, kWaitTimeoutNs, &never))) break;
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: the whole warp walks the units, one lane issues
    const bool issue = elect_one();
    const uint32_t s0 = smem_u32(smem);
    const uint64_t a0 = w_desc<DGRAD>(s0), b0 = sdesc_kmajor_sw128(s0 + kABytes);
    int stage = 0, acc = 0, where = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      const uint32_t idesc = idesc_e4m3_f32(128, static_cast<uint32_t>((un.n + 15) & ~15), DGRAD, 0);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          where = kWaitAccFree;
          break;
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          where = kWaitSlotFull;
          break;
        }
        tc_fence_after();
        if (issue) {
          const uint64_t at = static_cast<uint64_t>(stage * (kStageBytes >> 4));
          const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kUnitRows);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_f8_ss(d, a0 + at + k * kStepW<DGRAD>, b0 + at + k * kStepX, idesc, k > 0);
          mma_commit(&empty[stage]);
          mma_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
        if (++acc == kAccs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
    if (!ok && issue) raise_timeout(a.err, abort_flag, kKernFp8Gemm, where);
    // all MMAs issued have finished before TMEM is released
    if (issue) mma_commit(done);
    __syncwarp();
    int dummy = 0;
    mbar_wait(done, 0, kWaitTimeoutNs, &dummy);
  } else {
    // ---------------- epilogue: warps 2..5, TMEM lane quarter = warp % 4; a lane
    // holds one feature's sums of all rows
    const int q = warp & 3;
    const int row = q * 32 + lane;  // this thread's TMEM lane = feature of the unit's 128
    const bool fp16 = a.fp16 != 0;
    float* s_buf = scales + (warp - 2) * 4 * kUnitRows;
    const int64_t w_step = DGRAD ? args.w_cols : 1;
    int acc = 0, where = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      const float* sw = feature_scales<DGRAD>(args, un.g, un.tile * 128);
      const float* sx = args.x_scales + (un.tok0 + lane) * args.ldxs;
      const bool valid = lane < un.n;
      float next[kAhead], next_w[kAhead];
      auto scales_of = [&](int kb, float& x, float& w) {
        if (kb < kb1) {
          w = __ldg(sw + kb * w_step);
          x = valid ? __ldg(sx + kb) : 0.0f;
        }
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k) scales_of(kb0 + k, next[k], next_w[k]);
      float sum[kUnitRows];
#pragma unroll
      for (int c = 0; c < kUnitRows; ++c) sum[c] = 0.0f;
      for (int kb = kb0; kb < kb1; ++kb) {
        float* s = s_buf + (kb & 1) * 2 * kUnitRows;  // (the other one may still be read by slower lanes)
        const float product = __fmul_rn(next[0], next_w[0]);
        s[lane] = product;
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) {
          next[k] = next[k + 1];
          next_w[k] = next_w[k + 1];
        }
        scales_of(kb + kAhead, next[kAhead - 1], next_w[kAhead - 1]);
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kUnitRows);
        // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
        const bool got = mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got && (one_factor(product) || !valid))) {
          if (!__all_sync(0xFFFFFFFFu, got)) {
            ok = false;
            where = kWaitAccFull;
            break;
          }
          // (rare) some row's scales are two factors: the sums meet the first one in TMEM
          tc_fence_after();
          float first = __ldg(sw + kb * w_step), second = valid ? __ldg(sx + kb) : 0.0f;
          two_factors(second, first);
          s[lane] = second;
          s[kUnitRows + lane] = first;
          __syncwarp();
#pragma unroll 1
          for (int c0 = 0; c0 < un.n; c0 += 16) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_row + c0, r);
            tmem_ld_wait(r);
#pragma unroll
            for (int j = 0; j < 16; ++j)
              r[j] = __float_as_uint(__fmul_rn(__uint_as_float(r[j]), s[kUnitRows + c0 + j]));
            tmem_st_32x32b(t_row + c0, r);
          }
          tmem_st_wait();
        }
        tc_fence_after();
        __syncwarp();
#pragma unroll
        for (int c0 = 0; c0 < kUnitRows; c0 += 16) {
          if (c0 >= un.n) break;
          uint32_t r[16];
          tmem_ld_32x32b_x16(t_row + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(s + c0 + j);
            sum[c0 + j] = __fmaf_rn(__uint_as_float(r[j]), v.x, sum[c0 + j]);
            sum[c0 + j + 1] = __fmaf_rn(__uint_as_float(r[j + 1]), v.y, sum[c0 + j + 1]);
            sum[c0 + j + 2] = __fmaf_rn(__uint_as_float(r[j + 2]), v.z, sum[c0 + j + 2]);
            sum[c0 + j + 3] = __fmaf_rn(__uint_as_float(r[j + 3]), v.w, sum[c0 + j + 3]);
          }
        }
        // hand the accumulator back to the MMA warp
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
        if (++acc == kAccs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) break;
      if (kb0 > 0) {
        // a later part of a unit that an earlier CTA started: hand over the partial sums
        float* slot = a.partials + static_cast<int64_t>(worker) * kUnitRows * 128 + row;
#pragma unroll
        for (int c = 0; c < kUnitRows; ++c)
          if (c < un.n) __stcg(slot + c * 128, sum[c]);
        __threadfence();
        __syncwarp();
        if (lane == 0) st_release(a.flags + worker * 4 + q, 1);
      } else {
        // this CTA finishes the unit: the CTAs after it whose (non-empty)
        // ranges start inside the unit hold its later K-blocks, as their first work
        int c_last = worker;
        if (kb1 < kblocks) {
          const int64_t unit_end = static_cast<int64_t>(u + 1) * kblocks;
          while (c_last + 1 < workers && rg.begin_of(c_last + 1) < unit_end) ++c_last;
        }
        if (!rg.wait_partials(a.flags + q, worker + 1, c_last, abort_flag)) {
          ok = false;
          where = kWaitPartials;
          break;
        }
        for (int c = worker + 1; c <= c_last; ++c) {
          if (rg.begin_of(c) == rg.begin_of(c + 1)) continue;  // empty range
          const float* slot = a.partials + static_cast<int64_t>(c) * kUnitRows * 128 + row;
#pragma unroll
          for (int j = 0; j < kUnitRows; ++j)
            if (j < un.n) sum[j] += __ldcg(slot + j * 128);
        }
        if (un.tile * 128 + row < a.F) {
          uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(un.tok0) * a.ldo + un.tile * 128 + row;
#pragma unroll
          for (int c = 0; c < kUnitRows; ++c)
            if (c < un.n) out[static_cast<int64_t>(c) * a.ldo] = to16(sum[c], fp16);
        }
      }
    }
    if (!ok && lane == 0) raise_timeout(a.err, abort_flag, kKernFp8Gemm, where);
  }

  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

// ------------------------------------------------------------------ more rows: single CTAs and CTA pairs

template <bool PAIR>
struct Large {
  static constexpr int kRows = PAIR ? 256 : 128;     // of a unit (pairs: half in each CTA)
  static constexpr int kFeatures = 256;              // of a unit (pairs: each CTA holds half of the weight tile)
  static constexpr int kWBoxes = PAIR ? 1 : 2;       // of 128 features
  static constexpr int kStageBytes = (1 + kWBoxes) * kABytes;
  static constexpr int kStages = PAIR ? 5 : 4;
  static constexpr int kEpiWarps = 8;                // two per TMEM lane quarter, 128 features each
  static constexpr int kRowsWarp = 2;                // 0 the weights' producer, 1 the MMA warp, 3 a pair's relay, the epilogue from 4
  static constexpr int kThreads = 32 * (4 + kEpiWarps);
  // registers: 168 a thread at launch; the first four warps give theirs up
  static constexpr int kLaunchRegs = 168, kControlRegs = 64, kEpiRegs = 216;
  static_assert(128 * kControlRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * kLaunchRegs, "register shares");
  static constexpr int kPass = PAIR ? 64 : 32;       // features of an output row that go out at once
  static constexpr int kOutRow = kPass * 2 + 16;     // (the rows in different banks)
  static constexpr int kOutBytes = kEpiWarps * 32 * kOutRow;
  static constexpr int kBarBytes = 256;
  static constexpr int kTabGroups = kGroupsSmem[1];
  static constexpr int kTabBytes = 3 * (kTabGroups + 1) * 4;
  static constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + kOutBytes + kBarBytes + kSchedBytes + kTabBytes;
  static_assert((2 * kStages + 5) * 8 + 8 <= kBarBytes, "barrier area");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

// the rows of a unit that a CTA holds (pairs: the first half in the even one)
template <bool PAIR>
struct Part {
  int from, n, loaded;  // loaded: one box of 128, or boxes of 32 (both CTAs alike)
  __device__ Part(int rows, uint32_t rank) {
    const int first = PAIR ? (rows + 1) / 2 : rows;
    from = rank ? first : 0;
    n = rank ? rows - first : first;
    loaded = first > 96 ? 128 : (first + 31) & ~31;
  }
};

template <int N>
__device__ __forceinline__ void set_registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// sum += (d0, d1) * s, both halves
__device__ __forceinline__ void fma2(uint64_t& sum, uint32_t d0, uint32_t d1, uint64_t s) {
  asm("{\n\t.reg .b64 d;\n\t"
      "mov.b64 d, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, d, %3, %0;\n\t}"
      : "+l"(sum)
      : "r"(d0), "r"(d1), "l"(s));
}

template <bool DGRAD, bool PAIR>
__global__ void __launch_bounds__(Large<PAIR>::kThreads, 1)
    fp8_large_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                     const __grid_constant__ CUtensorMap tm_x32, const __grid_constant__ Fp8GemmArgs args) {
  using C = Large<PAIR>;
  const GroupedGemmArgs& a = args.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* const outs = smem + C::kStages * C::kStageBytes;  // the epilogue warps' rows on their way out
  uint8_t* const bars = outs + C::kOutBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(bars);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;  // a block's MMAs are complete
  uint64_t* tempty = tfull + 2;          // it is read, by the epilogue (of both CTAs)
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const PairSched sched(bars + C::kBarBytes);
  int32_t* tab = reinterpret_cast<int32_t*>(bars + C::kBarBytes + kSchedBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], (PAIR ? 2 : 1) * C::kEpiWarps);
    }
    mbar_init(done, 1);
    if (PAIR) sched.init(2 + C::kEpiWarps);  // producers and epilogue
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
    prefetch_tensormap(&tm_x32);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, 2 * C::kFeatures);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, 2 * C::kFeatures);
      tmem_relinquish();
    }
  }
  pdl_wait();  // the plan kernel's tables
  const GroupedTables tables = grouped_tables(a, tab, C::kTabGroups, C::kThreads);
  tc_fence_before();
  if (PAIR)
    cluster_sync();  // the peer's barriers are initialised before any remote signal
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int kblocks = (a.R + 127) / 128;
  // Each warp's walk along the units: as the pair hands them out, or (single CTAs, whose units take the
  // same time each) with the grid's stride.  Only the place is kept.
  int place = PAIR ? 0 : static_cast<int>(blockIdx.x);
  uint32_t place_phase = 0;
  bool walked = true;  // no wait for a unit ran out
  auto next_unit = [&]() -> int {
    const int total = tables.unit_off[a.G];
    if constexpr (PAIR) {
      PairUnits walk(sched, total, kWaitTimeoutNs, abort_flag, leader, warp == 0);
      walk.slot = place;
      walk.phase = place_phase;
      const int u = walk.next();
      place = walk.slot;
      place_phase = walk.phase;
      walked = walked && walk.ok;
      return u;
    } else {
      const int u = place;
      place += static_cast<int>(gridDim.x);
      return u < total ? u : -1;
    }
  };

  if (warp < 4) {
    set_registers_down<C::kControlRegs>();
    if (warp == 0 || warp == C::kRowsWarp) {
      // ---------------- TMA producers: one warp for the weight tiles, one for the rows; one lane issues
      const bool weights = warp == 0, issue = elect_one();
      const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_last();
      const uint32_t full_cl = PAIR ? mapa_shared(smem_u32(full), 0) : 0u;  // both CTAs signal the even one
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int u; ok && (u = next_unit()) >= 0;) {
        GroupedUnits units(tables, a.G, 1, a.bn, true);
        const GroupedUnit un = units.at(u);
        const Part<PAIR> z(un.n, rank);
        const int feat = un.tile * C::kFeatures + static_cast<int>(rank) * 128, tok = un.tok0 + z.from;
        // a weight tile read by one chunk only is streamed; by more, kept
        const uint64_t pol_w = units.chunks > 1 ? pol_keep : pol_stream;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            break;
          }
          if (issue) {
            uint8_t* sa = smem + stage * C::kStageBytes;
            uint64_t* const bar = &full[stage];
            const uint32_t bar_cl = full_cl + 8u * stage;
            if (weights) {
              if (leader)
                mbar_arrive_expect_tx(bar, (PAIR ? 2 : 1) * (C::kWBoxes * kABytes + z.loaded * 128));
#pragma unroll
              for (int b = 0; b < C::kWBoxes; ++b) {
                // 128 features x 128 of the reduction; the input gradient's features are w's columns
                const int c0 = DGRAD ? feat + 128 * b : kb * 128, c1 = DGRAD ? kb * 128 : feat + 128 * b;
                if (PAIR)
                  tma_load_3d_pair(sa + kABytes, &tm_w, bar_cl, c0, c1, un.g, pol_w);
                else
                  tma_load_3d(sa + (1 + b) * kABytes, &tm_w, bar, c0, c1, un.g, pol_w);
              }
            } else if (z.loaded == 128) {
              if (PAIR)
                tma_load_2d_pair(sa, &tm_x, bar_cl, kb * 128, tok, pol_keep);
              else
                tma_load_2d(sa, &tm_x, bar, kb * 128, tok, pol_keep);
            } else {
              for (int r = 0; r < z.loaded; r += 32) {
                if (PAIR)
                  tma_load_2d_pair(sa + r * 128, &tm_x32, bar_cl, kb * 128, tok + r, pol_keep);
                else
                  tma_load_2d(sa + r * 128, &tm_x32, bar, kb * 128, tok + r, pol_keep);
              }
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == C::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!(ok && walked) && issue)
        raise_timeout(a.err, abort_flag, kKernFp8Gemm, walked ? kWaitSlotFree : kWaitUnit);
      // every load issued has been used before the CTA exits
      for (int s = 0; s < C::kStages; ++s) {
        if (issued <= s) break;
        const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
        const int never = 0;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], par, kWaitTimeoutNs, &never))) break;
      }
    } else if (warp == 1) {
      if (leader) {
        // ---------------- MMA issuer (for both CTAs): the whole warp walks the units, one lane issues
        const bool issue = elect_one();
        const uint32_t s0 = smem_u32(smem);
        const uint64_t a0 = sdesc_kmajor_sw128(s0), b0 = w_desc<DGRAD>(s0 + kABytes);
        const uint32_t idesc = idesc_e4m3_f32(PAIR ? 256 : 128, C::kFeatures, 0, DGRAD);
        int stage = 0, acc = 0, where = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        while (ok && next_unit() >= 0) {
          for (int kb = 0; kb < kblocks; ++kb) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
              ok = false;
              where = kWaitAccFree;
              break;
            }
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, kWaitTimeoutNs, abort_flag))) {
              ok = false;
              where = kWaitSlotFull;
              break;
            }
            tc_fence_after();
            if (issue) {
              const uint64_t at = static_cast<uint64_t>(stage * (C::kStageBytes >> 4));
              const uint32_t d = tmem_base + static_cast<uint32_t>(acc * C::kFeatures);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (PAIR)
                  mma_f8_ss_pair(d, a0 + at + k * kStepX, b0 + at + k * kStepW<DGRAD>, idesc, k > 0);
                else
                  mma_f8_ss(d, a0 + at + k * kStepX, b0 + at + k * kStepW<DGRAD>, idesc, k > 0);
              }
              if (PAIR) {
                mma_commit_pair_mc(&empty[stage], 0x3);
                mma_commit_pair_mc(&tfull[acc], 0x3);
              } else {
                mma_commit(&empty[stage]);
                mma_commit(&tfull[acc]);
              }
            }
            __syncwarp();
            if (++stage == C::kStages) {
              stage = 0;
              phase ^= 1u;
            }
            if (++acc == 2) {
              acc = 0;
              acc_phase ^= 1u;
            }
          }
        }
        if (!walked) where = kWaitUnit;
        if (!(ok && walked) && issue) raise_timeout(a.err, abort_flag, kKernFp8Gemm, where);
        // all MMAs issued have finished before TMEM is released
        if (issue) {
          if (PAIR)
            mma_commit_pair(done);
          else
            mma_commit(done);
        }
        __syncwarp();
        int dummy = 0;
        mbar_wait(done, 0, kWaitTimeoutNs, &dummy);
      } else if (lane == 0) {
        if (!sched.schedule(a.next_unit, tables.unit_off[a.G], kWaitTimeoutNs, abort_flag))
          raise_timeout(a.err, abort_flag, kKernFp8Gemm, kWaitUnit);
      }
    } else if (PAIR) {
      if (leader && lane == 0 && !sched.relay(tables.unit_off[a.G], kWaitTimeoutNs, abort_flag))
        raise_timeout(a.err, abort_flag, kKernFp8Gemm, kWaitUnit);
    }
  } else {
    set_registers_up<C::kEpiRegs>();
    // ---------------- epilogue: TMEM lane quarter = warp % 4; a quarter's two warps
    // take 128 features each, a lane one row
    const int q = warp & 3, col0 = (warp - 4) / 4 * 128;
    const bool fp16 = a.fp16 != 0;
    const uint32_t tempty_cl = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
    const uint32_t t_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(col0);
    const int64_t w_step = DGRAD ? args.w_cols : 1;
    int acc = 0, where = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u; ok && (u = next_unit()) >= 0;) {
      int tok, rows, feat;  // this warp's first row, its rows, its first feature
      const float *sx, *sw;
      {
        const GroupedUnit un = GroupedUnits(tables, a.G, 1, a.bn, true).at(u);
        const Part<PAIR> z(un.n, rank);
        feat = un.tile * C::kFeatures + col0;
        tok = un.tok0 + z.from + q * 32;
        rows = z.n - q * 32;
        sw = feature_scales<DGRAD>(args, un.g, feat);
        // (lanes without a row read another one's scales)
        sx = args.x_scales + (un.tok0 + min(z.from + q * 32 + lane, un.n - 1)) * args.ldxs;
      }
      float next_w = __ldg(sw), next_x = __ldg(sx);
      // a block's factor, and whether some lane's are two: asked for once the block before is summed (before the wait
      // for its own MMAs: 64 x 300 rows, N = K = 4096, input gradient 385 -> 401 us)
      float s = __fmul_rn(next_x, next_w);
      bool two = __any_sync(0xFFFFFFFFu, !one_factor(s));
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      for (int kb = 0; kb < kblocks; ++kb) {
        uint64_t s2 = twice(s);
        if (kb + 1 < kblocks) {  // the next block's, while this one's MMAs run
          next_w = __ldg(sw + (kb + 1) * w_step);
          next_x = __ldg(sx + kb + 1);
        }
        // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          where = kWaitAccFull;
          break;
        }
        tc_fence_after();
        __syncwarp();
        const uint32_t t = t_base + static_cast<uint32_t>(acc * C::kFeatures);
        if (two) {  // (rare) the sums meet their first factor in TMEM, 16 at a time: registers for it here would spill
          float second = __ldg(sx + kb), first = __ldg(sw + kb * w_step);
          two_factors(second, first);
          s2 = twice(second);
#pragma unroll 1
          for (uint32_t c = 0; c < 128; c += 16) {
            uint32_t d[16];
            tmem_ld_32x32b_x16(t + c, d);
            tmem_ld_wait(d);
#pragma unroll
            for (int i = 0; i < 16; ++i) d[i] = __float_as_uint(__fmul_rn(__uint_as_float(d[i]), first));
            tmem_st_32x32b(t + c, d);
          }
          tmem_st_wait();
        }
        uint32_t r[2][16];
        tmem_ld_32x32b_x16(t, r[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_ld_wait(r[c & 1]);
          if (c < 7) {
            tmem_ld_32x32b_x16(t + 16 * (c + 1), r[(c + 1) & 1]);
          } else {  // hand the accumulator back to the MMA thread
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              if (PAIR)
                mbar_arrive_remote(tempty_cl + 8u * acc);
              else
                mbar_arrive(&tempty[acc]);
            }
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) fma2(sum[8 * c + i / 2], r[c & 1][i], r[c & 1][i + 1], s2);
        }
        s = __fmul_rn(next_x, next_w);
        two = __any_sync(0xFFFFFFFFu, !one_factor(s));
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) break;
      // A pass's features of the 32 rows through shared memory, so that a store covers whole sectors of
      // few rows: 16-byte stores of 32 rows at once take 32 cycles each, copies of each row by TMA as long
      // (64 x 512 rows, N = K = 4096: 87 us of 560).
      constexpr int kLanes = C::kPass / 8, kPer = 32 / kLanes;  // lanes a row, rows a store
      uint8_t* const buf = outs + (warp - 4) * 32 * C::kOutRow;
      uint16_t* const out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(tok) * a.ldo + feat;
#pragma unroll
      for (int c = 0; c < 128; c += C::kPass) {
#pragma unroll
        for (int i = 0; i < C::kPass / 2; i += 4) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo, hi;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(sum[c / 2 + i + k]));
            w[k] = pack16(lo, hi, fp16);
          }
          *reinterpret_cast<uint4*>(buf + lane * C::kOutRow + 4 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
        const int at = c + 8 * (lane % kLanes);
        if (feat + at < a.F) {  // (F is a multiple of 8)
#pragma unroll
          for (int i = 0; i < 32; i += kPer) {
            const int r = i + lane / kLanes;
            if (r < rows)
              *reinterpret_cast<uint4*>(out + r * a.ldo + at) =
                  *reinterpret_cast<const uint4*>(buf + r * C::kOutRow + 16 * (lane % kLanes));
          }
        }
        __syncwarp();
      }
    }
    if (!walked) where = kWaitUnit;
    if (!(ok && walked) && lane == 0) raise_timeout(a.err, abort_flag, kKernFp8Gemm, where);
  }

  __syncthreads();
  if (PAIR) cluster_sync();  // both CTAs keep their shared memory, barriers and TMEM until both are done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, 2 * C::kFeatures);
    else
      tmem_dealloc(tmem_base, 2 * C::kFeatures);
  }
}

template <bool DGRAD, bool PAIR>
cudaError_t launch_large(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tx32, const Fp8GemmArgs& a,
                         int num_sms, cudaStream_t stream) {
  using C = Large<PAIR>;
  static PerDevice config;
  auto kernel = fp8_large_kernel<DGRAD, PAIR>;
  if constexpr (PAIR) return launch_pairs(kernel, config, C::kThreads, C::kSmemBytes, stream, tw, tx, tx32, a);
  return launch_ctas(kernel, config, num_sms, C::kThreads, C::kSmemBytes, stream, tw, tx, tx32, a);
}

template <bool DGRAD>
cudaError_t launch(Fp8Plan plan, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tx32,
                   const Fp8GemmArgs& a, int num_sms, cudaStream_t stream) {
  if (plan == Fp8Plan::kPairs) return launch_large<DGRAD, true>(tw, tx, tx32, a, num_sms, stream);
  if (plan == Fp8Plan::kSingle) return launch_large<DGRAD, false>(tw, tx, tx32, a, num_sms, stream);
  static PerDevice config;
  return launch_ctas(fp8_small_kernel<DGRAD>, config, num_sms < kMaxGemmCtas ? num_sms : kMaxGemmCtas, kThreads,
                     kSmemBytes, stream, tw, tx, a);
}

}  // namespace

int fp8_bn(Fp8Plan plan) {
  return plan == Fp8Plan::kSmall ? kUnitRows : plan == Fp8Plan::kSingle ? Large<false>::kRows : Large<true>::kRows;
}
int fp8_tile(Fp8Plan plan) { return plan == Fp8Plan::kSmall ? 128 : Large<true>::kFeatures; }
int fp8_tok_box(Fp8Plan plan) { return plan == Fp8Plan::kSmall ? kRowBox : 128; }

cudaError_t launch_fp8_gemm(GroupedOp op, Fp8Plan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                            const CUtensorMap& tm_x32, const Fp8GemmArgs& a, int num_sms, cudaStream_t stream) {
  return op == GroupedOp::kForward ? launch<false>(plan, tm_w, tm_x, tm_x32, a, num_sms, stream)
                                   : launch<true>(plan, tm_w, tm_x, tm_x32, a, num_sms, stream);
}

}  // namespace moe
