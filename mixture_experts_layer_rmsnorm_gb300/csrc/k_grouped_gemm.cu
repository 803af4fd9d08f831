// k_grouped_gemm.cu -- matrix products grouped by expert, ragged row counts, on
// the 5th-generation tensor cores (tcgen05, TMEM, TMA): the plan kernel of every
// grouped call, and for groups of few rows
//   forward         y[p, :]  = x[p, :] w_g^T       (p in group g)
//   input gradient  dx[p, :] = dy[p, :] w_g
// bf16 or fp16 operands, fp32 accumulation in TMEM.  (Groups of many rows:
// k_grouped_pair.cu; the weight gradient: k_grouped_wgrad.cu.)
//
// An expert holds anything from no row to thousands, and the MMA's M side is a
// fixed 128 (256 for a CTA pair) while its N side follows in steps of 16.  So
// the weights take the M side and the rows the N side: a unit is
// C^T[features, rows] = W_g[features, R] X_g[rows, R]^T.  Rows of the next group
// inside a token box feed MMA columns that are dropped: an output row depends
// on its own row alone.  The forward reads w K-major as stored.  The input
// gradient reduces over w's row index, so the same stored matrix is its MN-major
// operand (the descriptor's transpose bit): no transposed copy of the weights.
//
// Few rows per group: bound by HBM, the weights stream once.  Units of 128
// features x 32 rows on single CTAs, 10 stages of 20 KB in flight, split
// stream-K so that every SM streams the same number of weight bytes whatever
// the lists; partial sums meet in fp32 in a fixed order, so results repeat bit
// for bit.  Measured, plan included: 8 rows in 8 of 64 groups, N = 8192, K = 4096: 84.6 us
// (0.94 of the measured copy rate); 16 groups of one row, the kernel alone: 161 us.
//
// Roles in a CTA of 192 threads (persistent, one CTA per SM): warp 0 TMA
// producer, warp 1 TMEM owner and MMA issuer, warps 2..5 epilogue, one per TMEM
// lane quarter.  Every wait is bounded.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bounded_wait.cuh"
#include "grouped.cuh"
#include "launch_config.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

// ------------------------------------------------------------------ plan

// Latency alone counts here (the GEMM waits for the tables): every load first,
// what does not depend on them next, two barriers.
__global__ void __launch_bounds__(kGroupsMax, 1)
    grouped_plan_kernel(const __grid_constant__ GroupedPlanArgs a, const __grid_constant__ CUtensorMap tm_dy,
                        const __grid_constant__ CUtensorMap tm_x) {
  __shared__ int warp_sum[32];
  __shared__ int first_bad;
  pdl_wait();
  pdl_launch_dependents();  // the GEMM sets up its barriers and TMEM meanwhile
  const int g = threadIdx.x, lane = g & 31, warp = g >> 5;
  int64_t s = 0, c = 0, end = 0;  // end: where the next group may begin
  if (g < a.G) {
    if (a.offsets) {
      s = __ldg(a.offsets + g);
      end = __ldg(a.offsets + g + 1);
    } else {
      c = a.rows / a.G;
      s = g * c;
      end = s + c;
    }
    c = a.counts ? __ldg(a.counts + g) : end - s;
  }
  for (int i = g; i < a.n_flags; i += blockDim.x) a.flags[i] = 0;
  if (g == 0) first_bad = kGroupsMax;
  const bool bad = s < 0 || c < 0 || s + c > end || end > a.rows;
  const bool any_bad = __syncthreads_or(bad) != 0;
  if (any_bad) {  // (uniform) no group has rows or units then
    if (bad) atomicMin(&first_bad, g);
    __syncthreads();
    s = c = 0;
  }
  if (a.maps && g < a.G) {
    const uint32_t rows_end = s + c > 0 ? static_cast<uint32_t>(s + c) : 1u;  // (an empty group loads nothing)
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      uint4* dst = reinterpret_cast<uint4*>(a.maps + 2 * g + m);
      const uint4* src = reinterpret_cast<const uint4*>(m ? &tm_x : &tm_dy);
#pragma unroll
      for (int i = 0; i < 8; ++i) dst[i] = src[i];
      tensormap_set_dim1(dst, rows_end);
    }
    tensormap_release();
  }
  int units = 0;
  if (g < a.G && !any_bad) {
    if (a.bn > 0)
      units = static_cast<int>((c + a.bn - 1) / a.bn) * a.tiles;
    else
      units = c == 0 && a.skip_empty ? 0 : a.tiles;
  }
  int sum = units;  // inclusive scan over the block
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
    if (lane >= d) sum += v;
  }
  if (lane == 31) warp_sum[warp] = sum;
  __syncthreads();
  // the sum of the warps before this one
  int before = lane < warp ? warp_sum[lane] : 0;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) before += __shfl_xor_sync(0xFFFFFFFFu, before, d);
  sum += before;
  if (g < a.G) {
    a.start[g] = static_cast<int32_t>(s);
    a.count[g] = static_cast<int32_t>(c);
    a.unit_off[g] = sum - units;
    if (g == a.G - 1) a.unit_off[a.G] = sum;
  }
  if (g == 0) {
    a.err[0] = any_bad ? kErrDevice : 0;
    a.err[1] = any_bad ? kKernGroupedPlan : 0;
    a.err[2] = any_bad ? first_bad : 0;
    a.err[3] = 0;
  }
}

// ------------------------------------------------------------------ GEMM

constexpr int kABytes = 128 * 128;  // 128 features x 64 of the reduction, 16 bits
constexpr int kMnBox = 64 * 128;    // an MN-major box: 64 features x 64 of the reduction
constexpr int kUnitRows = 32, kRowBox = 16;
constexpr int kStageBytes = kABytes + kUnitRows * 128;
constexpr int kStages = 10;
constexpr int kThreads = 192;
constexpr uint32_t kTmemCols = 2 * kUnitRows;  // two accumulators
constexpr int kBarBytes = 256;
constexpr int kTabBytes = 3 * (kGroupsSmem[0] + 1) * 4;
constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + kBarBytes + kTabBytes;
static_assert((2 * kStages + 5) * 8 + 8 <= kBarBytes, "barrier area");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

// The waits, as recorded in the error word's detail bits.
enum : int { kWaitSlotFree = 1, kWaitAccFree = 2, kWaitSlotFull = 3, kWaitAccFull = 4, kWaitPartials = 5 };

__device__ __forceinline__ uint16_t to16(float v, bool fp16) {
  return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <bool DGRAD>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_small_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                         const __grid_constant__ GroupedGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + kStages * kStageBytes + kBarBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = static_cast<int>(blockIdx.x), workers = static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
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
  const int kblocks = (a.R + 63) / 64;
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
          if constexpr (DGRAD) {  // [64 rows of w][64 columns] boxes: the columns are the features
            tma_load_3d(sa, &tm_w, bar, feat, kb * 64, un.g, pol_w);
            tma_load_3d(sa + kMnBox, &tm_w, bar, feat + 64, kb * 64, un.g, pol_w);
          } else {
            tma_load_3d(sa, &tm_w, bar, kb * 64, feat, un.g, pol_w);
          }
          for (int r = 0; r < rows; r += kRowBox)
            tma_load_2d(sa + kABytes + r * 128, &tm_x, bar, kb * 64, un.tok0 + r, pol_keep);
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && issue) raise_timeout(a.err, abort_flag, kKernGroupedGemm, kWaitSlotFree);
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
    const uint64_t a0 = DGRAD ? sdesc_mnmajor_sw128(s0, kMnBox) : sdesc_kmajor_sw128(s0);
    const uint64_t b0 = sdesc_kmajor_sw128(s0 + kABytes);
    constexpr uint64_t kStepA = (DGRAD ? 2048 : 32) >> 4, kStepB = 32 >> 4;  // K = 16
    int stage = 0, acc = 0, where = 0;
    uint32_t phase = 0, acc_phase = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
        ok = false;
        where = kWaitAccFree;
        break;
      }
      tc_fence_after();
      const uint32_t idesc = idesc_f16_f32(128, static_cast<uint32_t>((un.n + 15) & ~15), a.fp16, DGRAD, 0);
      const uint32_t d_acc = tmem_base + static_cast<uint32_t>(acc * kUnitRows);
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          where = kWaitSlotFull;
          break;
        }
        tc_fence_after();
        const uint64_t at = static_cast<uint64_t>(stage * (kStageBytes >> 4));
        if (issue) {
          mma_bf16_ss(d_acc, a0 + at, b0 + at, idesc, kb > kb0);
#pragma unroll
          for (int k = 1; k < 4; ++k) mma_bf16_ss(d_acc, a0 + at + k * kStepA, b0 + at + k * kStepB, idesc, 1u);
          mma_commit(&empty[stage]);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (issue) mma_commit(&tfull[acc]);
      __syncwarp();
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok && issue) raise_timeout(a.err, abort_flag, kKernGroupedGemm, where);
    // all MMAs issued have finished before TMEM is released
    if (issue) mma_commit(done);
    __syncwarp();
    int dummy = 0;
    mbar_wait(done, 0, kWaitTimeoutNs, &dummy);
  } else {
    // ---------------- epilogue: warps 2..5, TMEM lane quarter = warp % 4
    const int q = warp & 3;
    const int row = q * 32 + lane;  // this thread's TMEM lane = feature of the unit's 128
    const bool fp16 = a.fp16 != 0;
    int acc = 0, where = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag))) {
        ok = false;
        where = kWaitAccFull;
        break;
      }
      tc_fence_after();
      const uint32_t t_row =
          tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * kUnitRows);
      const bool mine = un.tile * 128 + row < a.F;
      uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(un.tok0) * a.ldo + un.tile * 128 + row;
      if (kb0 > 0) {
        // a later part of a unit that an earlier CTA started: hand over the partial sums
        float* slot = a.partials + static_cast<int64_t>(worker) * kUnitRows * 128;
        for (int c0 = 0; c0 < un.n; c0 += 16) {
          uint32_t r[16];
          __syncwarp();  // tcgen05.ld is warp-aligned
          tmem_ld_32x32b_x16(t_row + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 16; ++j) __stcg(slot + (c0 + j) * 128 + row, __uint_as_float(r[j]));
        }
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
        for (int c0 = 0; c0 < un.n; c0 += 16) {
          uint32_t r[16];
          __syncwarp();  // tcgen05.ld is warp-aligned
          tmem_ld_32x32b_x16(t_row + c0, r);
          tmem_ld_wait();
          float v[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
#pragma unroll 2
          for (int c = worker + 1; c <= c_last; ++c) {
            if (rg.begin_of(c) == rg.begin_of(c + 1)) continue;  // empty range
            const float* slot = a.partials + static_cast<int64_t>(c) * kUnitRows * 128;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += __ldcg(slot + (c0 + j) * 128 + row);
          }
          if (mine) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + j < un.n) out[static_cast<int64_t>(c0 + j) * a.ldo] = to16(v[j], fp16);
          }
        }
      }
      if (!ok) break;
      // hand the accumulator back to the MMA warp
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tempty[acc]);
      if (++acc == 2) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!ok && lane == 0) raise_timeout(a.err, abort_flag, kKernGroupedGemm, where);
  }

  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

template <bool DGRAD>
cudaError_t launch_small(const CUtensorMap& tw, const CUtensorMap& tx, const GroupedGemmArgs& a, int num_sms,
                         cudaStream_t stream) {
  static PerDevice config;
  return launch_ctas(grouped_small_kernel<DGRAD>, config, num_sms < kMaxGemmCtas ? num_sms : kMaxGemmCtas, kThreads,
                     kSmemBytes, stream, tw, tx, a);
}

// rows per unit, features per unit, rows per token box of the plans
constexpr int kBn[2] = {kUnitRows, 512}, kTile[2] = {128, 256}, kTokBox[2] = {kRowBox, 128};

}  // namespace

// CTA pairs: long units win (64 groups of 520 rows, N = 8192, K = 4096: two
// units of 260 rows 1362 us, three of 174 1887 us), unless they leave pairs
// without work.  A unit of n rows takes about max(680, 2.5 n + 30) cycles a step
// (measured for 128 to 512 rows); the call, units per pair times that.
int grouped_bn(GroupedPlan plan, int64_t rows, int64_t groups, int64_t tiles, int num_sms) {
  if (plan == GroupedPlan::kSmall) return kBn[0];
  const int64_t per_group = (rows + groups - 1) / groups, pairs = num_sms / 2 > 0 ? num_sms / 2 : 1;
  int best = 512;
  int64_t least = 0;
  for (int bn = 512; bn >= 128; bn /= 2) {
    const int64_t chunks = (per_group + bn - 1) / bn, n = (per_group + chunks - 1) / chunks;
    const int64_t unit = 5 * n / 2 + 30 > 680 ? 5 * n / 2 + 30 : 680;
    const int64_t cost = (chunks * groups * tiles + pairs - 1) / pairs * unit;
    if (bn == 512 || cost < least) {
      least = cost;
      best = bn;
    }
  }
  return best;
}
int grouped_tile(GroupedPlan plan) { return kTile[static_cast<int>(plan)]; }
int grouped_tok_box(GroupedPlan plan) { return kTokBox[static_cast<int>(plan)]; }
size_t grouped_partial_bytes() { return static_cast<size_t>(kMaxGemmCtas) * kBn[0] * 128 * 4; }

cudaError_t launch_grouped_plan(const GroupedPlanArgs& a, const CUtensorMap& dy, const CUtensorMap& x,
                                cudaStream_t stream) {
  const int threads = (a.G + 31) / 32 * 32 < 256 ? 256 : (a.G + 31) / 32 * 32;
  return launch_pdl(grouped_plan_kernel, dim3(1), dim3(threads), 0, stream, a, dy, x);
}

cudaError_t launch_grouped_gemm(GroupedOp op, GroupedPlan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                                const CUtensorMap& tm_x32, const GroupedGemmArgs& a, int num_sms,
                                cudaStream_t stream) {
  if (plan == GroupedPlan::kLarge) return launch_grouped_pair(op, tm_w, tm_x, tm_x32, a, stream);
  return op == GroupedOp::kForward ? launch_small<false>(tm_w, tm_x, a, num_sms, stream)
                                   : launch_small<true>(tm_w, tm_x, a, num_sms, stream);
}

}  // namespace moe
