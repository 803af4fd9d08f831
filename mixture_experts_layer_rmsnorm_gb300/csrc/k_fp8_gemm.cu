// k_fp8_gemm.cu -- the grouped products on 8-bit operands (E4M3) whose fp32
// scales cover 128 elements of a row, or 128 x 128 of a matrix:
//   forward         y[p, :]  = x[p, :] w_g^T       (p in group g)
//   input gradient  dx[p, :] = dy[p, :] w_g
// The reduction is cut into the blocks b that share a scale:
//   y[p, f] = sum_b (sx[b, p] sw[f / 128, b]) D_b[p, f],  D_b = sum over the block of the codes' products
// Only D_b is the tensor core's (kind::f8f6f4, fp32 in TMEM, K = 32 an MMA); the
// scales are no powers of two, so D_b leaves TMEM block by block and is summed in
// registers, one fp32 multiply-add per element and block.  That sum rounds to nearest;
// the tensor core's own cuts towards zero stay inside a block of 128.
//
// Units and work split as in k_grouped_gemm.cu and k_grouped_pair.cu; the input gradient
// reads the stored matrix as an MN-major operand.  A K-block is one block of scales, 128
// bytes of codes a row.
//
// Few rows a group: single CTAs, stream-K, the weights on the MMA's M side (128 features x
// 32 rows a unit), bound by HBM.
//
// Many: CTA pairs, units of up to 256 rows x 256 features handed out on demand, here with
// the rows on the MMA's M side, so that a TMEM lane is a row of x and an epilogue
// warp's 128 columns are one block of features: a thread multiplies a whole block with one
// scale, which it has loaded ahead.  (With the weights on the M side columns are rows with a scale
// each, and reading them from shared memory, beside the tensor core's own reads, took
// half of the time: one group of 8192 rows, N = K = 8192: 772 us.)  MMAs of M = 256 take the same
// time for any number of rows, but up to 256 rows a group HBM bounds the product all the same.
//   - A block's MMAs (256 x 256 x 128) take 512 cycles at the FP8 rate.  In that time the
//     eight epilogue warps of each CTA read 128 x 256 accumulators and issue as many
//     multiply-adds, paired (fma.f32x2), 64 a thread; a load is under way while the one before it is summed.
//   - The sums take 128 registers of each epilogue thread: setmaxnreg moves them there.
//   - TMEM holds two blocks of 256 columns: one is read while the next is computed.
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
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = kAccs * kUnitRows;
constexpr int kBarBytes = 256;
constexpr int kTabBytes = 3 * (kGroupsSmem[0] + 1) * 4;
constexpr int kScaleBytes = 4 * 2 * kUnitRows * 4;  // per epilogue warp, two blocks
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
    float* s_buf = scales + (warp - 2) * 2 * kUnitRows;
    const int64_t w_step = DGRAD ? args.w_cols : 1;
    int acc = 0, where = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      const float* sw = feature_scales<DGRAD>(args, un.g, un.tile * 128) + kb0 * w_step;
      const float* sx = args.x_scales + kb0 * args.ldxs + un.tok0 + lane;
      const bool valid = lane < un.n;
      float sum[kUnitRows];
#pragma unroll
      for (int c = 0; c < kUnitRows; ++c) sum[c] = 0.0f;
      float next_x = valid ? __ldg(sx) : 0.0f, next_w = __ldg(sw);
      for (int kb = kb0; kb < kb1; ++kb) {
        float* s = s_buf + (kb & 1) * kUnitRows;  // (the other one may still be read by slower lanes)
        s[lane] = __fmul_rn(next_x, next_w);
        if (kb + 1 < kb1) {  // the next block's, while this one's MMAs run
          sx += args.ldxs;
          sw += w_step;
          next_x = valid ? __ldg(sx) : 0.0f;
          next_w = __ldg(sw);
        }
        // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          where = kWaitAccFull;
          break;
        }
        tc_fence_after();
        __syncwarp();
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kUnitRows);
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

// ------------------------------------------------------------------ many rows: CTA pairs

namespace pair {

constexpr int kRows = 256;                         // of a unit: half in each CTA
constexpr int kFeatures = 256;                     // of a unit: each CTA holds half of the weight tile
constexpr int kStageBytes = 2 * kABytes;
constexpr int kStages = 6;
constexpr int kEpiWarps = 8;                       // two per TMEM lane quarter, 128 features each
constexpr int kRowsWarp = 2;                       // 0 the weights' producer, 1 the MMA warp, 3 the relay, the epilogue from 4
constexpr int kThreads = 32 * (4 + kEpiWarps);
// registers: 168 a thread at launch; the first four warps give theirs up
constexpr int kLaunchRegs = 168, kControlRegs = 64, kEpiRegs = 216;
static_assert(128 * kControlRegs + 32 * kEpiWarps * kEpiRegs <= kThreads * kLaunchRegs, "register shares");
constexpr int kAhead = 3;                          // blocks whose scales are loaded ahead
constexpr int kBarBytes = 256;
constexpr int kTabBytes = 3 * (kGroupsSmem[1] + 1) * 4;
constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + kBarBytes + kSchedBytes + kTabBytes;
static_assert((2 * kStages + 5) * 8 + 8 <= kBarBytes, "barrier area");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

// the rows of a unit that a CTA holds: the first half in the even one
struct Half {
  int from, n, loaded;  // loaded: one box of 128, or boxes of 32
  __device__ Half(int rows, uint32_t rank) {
    const int first = (rows + 1) / 2;
    from = rank ? first : 0;
    n = rank ? rows - first : first;
    loaded = boxes(first);  // (both alike)
  }
  static __device__ __forceinline__ int boxes(int n) { return n > 96 ? 128 : (n + 31) & ~31; }
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

template <bool DGRAD>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ CUtensorMap tm_x32, const __grid_constant__ Fp8GemmArgs args) {
  const GroupedGemmArgs& a = args.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // a block's MMAs are complete
  uint64_t* tempty = tfull + 2;       // it is read, by the epilogue of both CTAs
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const PairSched sched(smem + kStages * kStageBytes + kBarBytes);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + kStages * kStageBytes + kBarBytes + kSchedBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);
    }
    mbar_init(done, 1);
    sched.init(2 + kEpiWarps);  // producers and epilogue
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
    prefetch_tensormap(&tm_x32);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 2 * kFeatures);
    tmem_relinquish_pair();
  }
  pdl_wait();  // the plan kernel's tables
  const GroupedTables tables = grouped_tables(a, tab, kGroupsSmem[1], kThreads);
  tc_fence_before();
  cluster_sync();  // the peer's barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int total_units = tables.unit_off[a.G];
  const int kblocks = (a.R + 127) / 128;

  if (warp < 4) {
    set_registers_down<kControlRegs>();
    GroupedUnits units(tables, a.G, 1, a.bn, true);  // each warp walks its role's units
    PairUnits walk(sched, total_units, kWaitTimeoutNs, abort_flag, leader, warp == 0);
    if (warp == 0 || warp == kRowsWarp) {
      // ---------------- TMA producers: one warp for the weight tiles, one for the rows; one lane issues
      const bool weights = warp == 0, issue = elect_one();
      const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_last();
      const uint32_t full_cl = mapa_shared(smem_u32(full), 0);  // both CTAs signal the even one
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      for (int u; ok && (u = walk.next()) >= 0;) {
        const GroupedUnit un = units.at(u);
        const Half z(un.n, rank);
        const int feat = un.tile * kFeatures + static_cast<int>(rank) * 128, tok = un.tok0 + z.from;
        // a weight tile read by one chunk only is streamed; by more, kept
        const uint64_t pol_w = units.chunks > 1 ? pol_keep : pol_stream;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            break;
          }
          if (issue) {
            uint8_t* sa = smem + stage * kStageBytes;
            const uint32_t bar = full_cl + 8u * stage;
            if (weights) {
              if (leader) mbar_arrive_expect_tx(&full[stage], 2 * (kABytes + z.loaded * 128));
              if constexpr (DGRAD)  // 128 rows of w x 128 of its columns, which are the features
                tma_load_3d_pair(sa + kABytes, &tm_w, bar, feat, kb * 128, un.g, pol_w);
              else
                tma_load_3d_pair(sa + kABytes, &tm_w, bar, kb * 128, feat, un.g, pol_w);
            } else if (z.loaded == 128) {
              tma_load_2d_pair(sa, &tm_x, bar, kb * 128, tok, pol_keep);
            } else {
              for (int r = 0; r < z.loaded; r += 32) tma_load_2d_pair(sa + r * 128, &tm_x32, bar, kb * 128, tok + r, pol_keep);
            }
          }
          __syncwarp();
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!(ok && walk.ok) && issue)
        raise_timeout(a.err, abort_flag, kKernFp8Gemm, walk.ok ? kWaitSlotFree : kWaitUnit);
      // every load issued has been used before the CTA exits
      for (int s = 0; s < kStages; ++s) {
        if (issued <= s) break;
        const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
        const int never = 0;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], par, kWaitTimeoutNs, &never))) break;
      }
    } else if (warp == 1) {
      if (leader) {
        // ---------------- MMA issuer for both CTAs: the whole warp walks the units, one lane issues
        const bool issue = elect_one();
        const uint32_t s0 = smem_u32(smem);
        const uint64_t a0 = sdesc_kmajor_sw128(s0), b0 = w_desc<DGRAD>(s0 + kABytes);
        const uint32_t idesc = idesc_e4m3_f32(256, kFeatures, 0, DGRAD);
        int stage = 0, acc = 0, where = 0;
        uint32_t phase = 0, acc_phase = 0;
        bool ok = true;
        for (int u; ok && (u = walk.next()) >= 0;) {
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
              const uint64_t at = static_cast<uint64_t>(stage * (kStageBytes >> 4));
              const uint32_t d = tmem_base + static_cast<uint32_t>(acc * kFeatures);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_f8_ss_pair(d, a0 + at + k * kStepX, b0 + at + k * kStepW<DGRAD>, idesc, k > 0);
              mma_commit_pair_mc(&empty[stage], 0x3);
              mma_commit_pair_mc(&tfull[acc], 0x3);
            }
            __syncwarp();
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
            if (++acc == 2) {
              acc = 0;
              acc_phase ^= 1u;
            }
          }
        }
        if (!walk.ok) where = kWaitUnit;
        if (!(ok && walk.ok) && issue) raise_timeout(a.err, abort_flag, kKernFp8Gemm, where);
        // all MMAs issued have finished before TMEM is released
        if (issue) mma_commit_pair(done);
        __syncwarp();
        int dummy = 0;
        mbar_wait(done, 0, kWaitTimeoutNs, &dummy);
      } else if (lane == 0) {
        if (!sched.schedule(a.next_unit, total_units, kWaitTimeoutNs, abort_flag))
          raise_timeout(a.err, abort_flag, kKernFp8Gemm, kWaitUnit);
      }
    } else {
      if (leader && lane == 0 && !sched.relay(total_units, kWaitTimeoutNs, abort_flag))
        raise_timeout(a.err, abort_flag, kKernFp8Gemm, kWaitUnit);
    }
  } else {
    set_registers_up<kEpiRegs>();
    // ---------------- epilogue: TMEM lane quarter = warp % 4; a quarter's two warps
    // take 128 features each, a lane one row
    GroupedUnits units(tables, a.G, 1, a.bn, true);
    PairUnits walk(sched, total_units, kWaitTimeoutNs, abort_flag, leader, false);
    const int q = warp & 3, col0 = (warp - 4) / 4 * 128, row = q * 32 + lane;
    const bool fp16 = a.fp16 != 0;
    const uint32_t tempty_cl = mapa_shared(smem_u32(tempty), 0);
    const uint32_t t_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(col0);
    const int64_t w_step = DGRAD ? args.w_cols : 1;
    int acc = 0, where = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u; ok && (u = walk.next()) >= 0;) {
      const GroupedUnit un = units.at(u);
      const Half z(un.n, rank);
      const int feat = un.tile * kFeatures + col0;
      const bool mine = row < z.n;
      const float* sw = feature_scales<DGRAD>(args, un.g, feat);
      const float* sx = args.x_scales + un.tok0 + z.from + row;
      float next_w[kAhead], next_x[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        next_w[k] = k < kblocks ? __ldg(sw) : 0.0f;
        next_x[k] = k < kblocks && mine ? __ldg(sx) : 0.0f;
        sw += w_step;
        sx += args.ldxs;
      }
      uint64_t sum[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) sum[i] = 0;
      for (int kb = 0; kb < kblocks; ++kb) {
        const float s = __fmul_rn(next_x[0], next_w[0]);
        uint64_t s2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(s2) : "f"(s));
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) {
          next_w[k] = next_w[k + 1];
          next_x[k] = next_x[k + 1];
        }
        if (kb + kAhead < kblocks) {
          next_w[kAhead - 1] = __ldg(sw);
          if (mine) next_x[kAhead - 1] = __ldg(sx);
          sw += w_step;
          sx += args.ldxs;
        }
        // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          where = kWaitAccFull;
          break;
        }
        tc_fence_after();
        __syncwarp();
        const uint32_t t = t_base + static_cast<uint32_t>(acc * kFeatures);
        uint32_t r[2][32];
        tmem_ld_32x32b_x32(t, r[0]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tmem_ld_wait(r[c & 1]);
          if (c < 3) {
            tmem_ld_32x32b_x32(t + 32 * (c + 1), r[(c + 1) & 1]);
          } else {  // hand the accumulator back to the MMA thread
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(tempty_cl + 8u * acc);
          }
#pragma unroll
          for (int i = 0; i < 32; i += 2) fma2(sum[16 * c + i / 2], r[c & 1][i], r[c & 1][i + 1], s2);
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) break;
      if (mine) {
        uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(un.tok0 + z.from + row) * a.ldo + feat;
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo, hi;
            asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(sum[i + k]));
            w[k] = pack16(lo, hi, fp16);
          }
          if (feat + 2 * i < a.F) *reinterpret_cast<uint4*>(out + 2 * i) = make_uint4(w[0], w[1], w[2], w[3]);  // (F: a multiple of 8)
        }
      }
      __syncwarp();
    }
    if (!walk.ok) where = kWaitUnit;
    if (!(ok && walk.ok) && lane == 0) raise_timeout(a.err, abort_flag, kKernFp8Gemm, where);
  }

  __syncthreads();
  cluster_sync();  // both CTAs keep their shared memory, barriers and TMEM until both are done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kFeatures);
  }
}

}  // namespace pair

template <bool DGRAD>
cudaError_t launch(GroupedPlan plan, const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tx32,
                   const Fp8GemmArgs& a, int num_sms, cudaStream_t stream) {
  if (plan == GroupedPlan::kLarge) {
    static PerDevice config;
    return launch_pairs(pair::fp8_pair_kernel<DGRAD>, config, pair::kThreads, pair::kSmemBytes, stream, tw, tx, tx32, a);
  }
  static PerDevice config;
  return launch_ctas(fp8_small_kernel<DGRAD>, config, num_sms < kMaxGemmCtas ? num_sms : kMaxGemmCtas, kThreads,
                     kSmemBytes, stream, tw, tx, a);
}

}  // namespace

int fp8_bn(GroupedPlan plan, int64_t, int64_t, int64_t, int) {
  return plan == GroupedPlan::kSmall ? kUnitRows : pair::kRows;
}
int fp8_tok_box(GroupedPlan plan) { return plan == GroupedPlan::kSmall ? kRowBox : 128; }

cudaError_t launch_fp8_gemm(GroupedOp op, GroupedPlan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                            const CUtensorMap& tm_x32, const Fp8GemmArgs& a, int num_sms, cudaStream_t stream) {
  return op == GroupedOp::kForward ? launch<false>(plan, tm_w, tm_x, tm_x32, a, num_sms, stream)
                                   : launch<true>(plan, tm_w, tm_x, tm_x32, a, num_sms, stream);
}

}  // namespace moe
