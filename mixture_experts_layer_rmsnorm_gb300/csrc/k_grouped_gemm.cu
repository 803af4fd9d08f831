// k_grouped_gemm.cu -- matrix products grouped by expert, ragged row counts, on
// the 5th-generation tensor cores (tcgen05, TMEM, TMA):
//   forward         y[p, :]  = x[p, :] w_g^T       (p in group g)
//   input gradient  dx[p, :] = dy[p, :] w_g
//   weight gradient dw_g     = sum_p dy[p, :]^T x[p, :]
// bf16 or fp16 operands, fp32 accumulation in TMEM.
//
// Forward and input gradient.  An expert holds anything from no row to
// thousands, and the MMA's M side is a fixed 128 (256 for a CTA pair) while its
// N side follows in steps of 16.  So the weights take the M side and the rows
// the N side: a unit is C^T[features, rows] = W_g[features, R] X_g[rows, R]^T,
// and a group of 17 rows costs 32 MMA columns, not 128.  Rows of the next group
// inside a token box feed MMA columns that are dropped: an output row depends
// on its own row alone.  The forward reads w K-major as stored.  The input
// gradient reduces over w's row index, so the same stored matrix is its MN-major
// operand (the descriptor's transpose bit): no transposed copy of the weights.
//
// Weight gradient.  The reduction runs over the group's rows, the slow index of
// both operands: both MN-major.  A group's last block of 64 rows holds rows of
// the next group, which must not enter the sum (as zeros times a NaN would): the
// plan kernel writes per group two copies of the host's tensor maps whose row
// extent ends with the group, so TMA fills the rows past it with zeros.  Output
// tiles go through shared memory and TMA stores (fp32 accumulation into dw: TMA
// add-reductions, each element added once, so the result does not depend on an
// order).
//
// Work split.  Weight gradient: whole units round-robin over CTA
// pairs (M = 256, 6 stages of 32 KB, two 256-column accumulators so that a
// unit's epilogue runs under the next unit's MMAs); forward and input gradient
// of many rows: k_grouped_pair.cu.  Small plan (few rows per
// group: the weights stream once, HBM-bound): 128 x 32-row units on single
// CTAs, split stream-K so that every SM streams the same number of weight bytes;
// partial sums meet in fp32 in a fixed order, so results repeat bit for bit.
//
// Roles in a CTA of 192 threads (persistent, one CTA per SM): warp 0 lane 0 TMA
// producer, warp 1 TMEM owner and MMA issuer (the even CTA of a pair issues for
// both), warps 2..5 epilogue, one per TMEM lane quarter.  Every wait is bounded.
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

__global__ void __launch_bounds__(kGroupsMax, 1)
    grouped_plan_kernel(const __grid_constant__ GroupedPlanArgs a, const __grid_constant__ CUtensorMap tm_dy,
                        const __grid_constant__ CUtensorMap tm_x) {
  __shared__ int warp_sum[32];
  __shared__ int bad;
  pdl_launch_dependents();  // the GEMM sets up its barriers and TMEM meanwhile
  const int g = threadIdx.x, lane = g & 31, warp = g >> 5;
  if (g == 0) bad = 0;
  for (int i = g; i < a.n_flags; i += blockDim.x) a.flags[i] = 0;
  __syncthreads();
  int64_t s = 0, c = 0;
  if (g < a.G) {
    int64_t end;  // where the next group may begin
    if (a.offsets) {
      s = a.offsets[g];
      end = a.offsets[g + 1];
      c = a.counts ? a.counts[g] : end - s;
    } else {
      c = a.rows / a.G;
      s = g * c;
      end = s + c;
      if (a.counts) c = a.counts[g];
    }
    if (s < 0 || c < 0 || s + c > end || end > a.rows) atomicMax(&bad, g + 1);
  }
  __syncthreads();
  const int bad_group = bad;
  if (bad_group) s = c = 0;
  int units = 0;
  if (g < a.G && !bad_group) {
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
  if (warp == 0) {
    int v = lane < static_cast<int>(blockDim.x >> 5) ? warp_sum[lane] : 0;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v += o;
    }
    warp_sum[lane] = v;
  }
  __syncthreads();
  if (warp > 0) sum += warp_sum[warp - 1];
  if (g < a.G) {
    a.start[g] = static_cast<int32_t>(s);
    a.count[g] = static_cast<int32_t>(c);
    a.unit_off[g] = sum - units;
    if (g == a.G - 1) a.unit_off[a.G] = sum;
    if (a.maps) {
      const uint32_t end = s + c > 0 ? static_cast<uint32_t>(s + c) : 1u;  // (an empty group loads nothing)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        uint4* dst = reinterpret_cast<uint4*>(a.maps + 2 * g + m);
        const uint4* src = reinterpret_cast<const uint4*>(m ? &tm_x : &tm_dy);
#pragma unroll
        for (int i = 0; i < 8; ++i) dst[i] = src[i];
        tensormap_set_dim1(dst, end);
      }
      tensormap_release();
    }
  }
  if (g == 0) {
    a.err[0] = bad_group ? kErrDevice : 0;
    a.err[1] = bad_group ? kKernGroupedPlan : 0;
    a.err[2] = bad_group ? bad_group - 1 : 0;
    a.err[3] = 0;
  }
}

// ------------------------------------------------------------------ GEMM

constexpr int kABytes = 128 * 128;  // 128 features x 64 of the reduction, 16 bits
constexpr int kMnBox = 64 * 128;    // an MN-major box: 64 features x 64 of the reduction

template <int OP, int BN, int STAGES, int TOKBOX, bool PAIR>
struct Cfg {
  static constexpr bool kWgrad = OP == static_cast<int>(GroupedOp::kWgrad);
  static constexpr bool kDgrad = OP == static_cast<int>(GroupedOp::kDgrad);
  static constexpr int kBRows = PAIR ? BN / 2 : BN;  // a pair splits the MMA's N side
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kThreads = 192;
  static constexpr uint32_t kTmemCols = 2 * BN <= 32 ? 32 : 2 * BN <= 64 ? 64 : 2 * BN <= 128 ? 128 : 2 * BN <= 256 ? 256 : 512;
  static constexpr int kStoreBytes = kWgrad ? 4 * 2 * 4096 : 0;  // two 32-row x 128-byte boxes per epilogue warp
  static constexpr int kBarBytes = 256;
  static constexpr int kTabGroups = kGroupsSmem[PAIR];
  static constexpr int kTabBytes = 3 * (kTabGroups + 1) * 4;
  static constexpr size_t kSmemBytes = 1024 + static_cast<size_t>(STAGES) * kStageBytes + kStoreBytes + kBarBytes + kTabBytes;
  static_assert(kBRows % TOKBOX == 0 && BN >= 32 && BN <= 256, "token tile");
  static_assert(!kWgrad || (PAIR && BN == 256), "weight gradient: 256 x 256 tiles of CTA pairs");
  static_assert((2 * STAGES + 5) * 8 + 8 <= kBarBytes, "barrier area");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

// The waits, as recorded in the error word's detail bits.
enum : int { kWaitSlotFree = 1, kWaitAccFree = 2, kWaitSlotFull = 3, kWaitAccFull = 4, kWaitPartials = 5 };

__device__ __forceinline__ uint16_t to16(float v, bool fp16) {
  return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <int OP, int BN, int STAGES, int TOKBOX, bool PAIR>
__global__ void __launch_bounds__(192, 1)
    grouped_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ GroupedGemmArgs a) {
  using C = Cfg<OP, BN, STAGES, TOKBOX, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* store_buf = smem + STAGES * C::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(store_buf + C::kStoreBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* tab = reinterpret_cast<int32_t*>(store_buf + C::kStoreBytes + C::kBarBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int worker = PAIR ? static_cast<int>(blockIdx.x >> 1) : static_cast<int>(blockIdx.x);
  const int workers = PAIR ? static_cast<int>(gridDim.x >> 1) : static_cast<int>(gridDim.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], (PAIR ? 2 : 1) * 4);  // the epilogue warps (of both CTAs of a pair)
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_w);
    if (!C::kWgrad) prefetch_tensormap(&tm_x);
  }
  if (warp == 1) {
    if (PAIR) {
      tmem_alloc_pair(tmem_slot, C::kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, C::kTmemCols);
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

  const int total_units = tables.unit_off[a.G];
  const int kblocks = C::kWgrad ? 1 : (a.R + 63) / 64;
  constexpr bool kStreamK = !PAIR;
  constexpr int kUnitBn = C::kWgrad ? 0 : BN;
  GroupedUnits units(tables, a.G, a.tiles_n, kUnitBn);  // each thread walks its role's units

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_last();
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      int map_group = -1;
      const uint32_t full_cl = PAIR ? mapa_shared(smem_u32(full), 0) : 0u;  // both CTAs signal the even one
      GroupedRange rg(total_units, kblocks, worker, workers, kStreamK);
      int u, kb0, kb1;
      while (ok && rg.next(u, kb0, kb1)) {
        const GroupedUnit un = units.at(u);
        const int feat = PAIR ? un.tile * 256 + static_cast<int>(rank) * 128 : un.tile * 128;
        if (C::kWgrad) kb1 = (un.n + 63) / 64;
        const int n_mma = PAIR ? (un.n + 31) / 32 * 32 : (un.n + 15) / 16 * 16;
        const int half = PAIR ? n_mma / 2 : n_mma;
        const int tok_first = un.tok0 + static_cast<int>(rank) * half;
        const int tok_rows = (half + TOKBOX - 1) / TOKBOX * TOKBOX;  // whole boxes
        const uint32_t bytes = C::kWgrad ? C::kStageBytes : kABytes + tok_rows * 128;
        // a weight tile read by one token chunk only is streamed; by more, kept
        const uint64_t pol_w = C::kWgrad || un.count > BN ? pol_keep : pol_stream;
        const CUtensorMap* map_dy = a.maps + 2 * un.g;
        if (C::kWgrad && un.g != map_group) {
          tensormap_acquire(map_dy);
          tensormap_acquire(map_dy + 1);
          map_group = un.g;
        }
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, kWaitTimeoutNs, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * C::kStageBytes;
          uint8_t* sb = sa + kABytes;
          uint64_t* bar = &full[stage];
          const uint32_t bar_cl = full_cl + 8u * stage;
          if (!PAIR)
            mbar_arrive_expect_tx(bar, bytes);
          else if (leader)
            mbar_arrive_expect_tx(bar, 2 * bytes);
          auto load_2d = [&](void* dst, const CUtensorMap* m, int c0, int c1, uint64_t pol) {
            if (PAIR)
              tma_load_2d_pair(dst, m, bar_cl, c0, c1, pol);
            else
              tma_load_2d(dst, m, bar, c0, c1, pol);
          };
          auto load_w = [&](void* dst, int c0, int c1) {
            if (PAIR)
              tma_load_3d_pair(dst, &tm_w, bar_cl, c0, c1, un.g, pol_w);
            else
              tma_load_3d(dst, &tm_w, bar, c0, c1, un.g, pol_w);
          };
          if constexpr (C::kWgrad) {
            const int row = un.tok0 + kb * 64;
            const int col = un.tile_n * 256 + static_cast<int>(rank) * 128;
#pragma unroll
            for (int j = 0; j < 2; ++j) load_2d(sa + j * kMnBox, map_dy, feat + 64 * j, row, pol_keep);
#pragma unroll
            for (int j = 0; j < 2; ++j) load_2d(sb + j * kMnBox, map_dy + 1, col + 64 * j, row, pol_keep);
          } else {
            if constexpr (C::kDgrad) {  // [64 rows of w][64 columns] boxes: the columns are the features
              load_w(sa, feat, kb * 64);
              load_w(sa + kMnBox, feat + 64, kb * 64);
            } else {
              load_w(sa, kb * 64, feat);
            }
            for (int r = 0; r < tok_rows; r += TOKBOX) load_2d(sb + r * 128, &tm_x, kb * 64, tok_first + r, pol_keep);
          }
          ++issued;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) raise_timeout(a.err, abort_flag, kKernGroupedGemm, kWaitSlotFree);
      // every load this thread issued has landed before the CTA exits (the odd
      // CTA of a pair sees that through the release of its stages)
      for (int s = 0; s < STAGES; ++s) {
        if (issued <= s) break;
        const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
        int dummy = 0;
        mbar_wait(PAIR && !leader ? &empty[s] : &full[s], par, kWaitTimeoutNs, &dummy);
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer: the whole warp walks the units, one lane issues
      const bool issue = elect_one();
      const uint32_t s0 = smem_u32(smem);
      const uint64_t a0 = C::kWgrad || C::kDgrad ? sdesc_mnmajor_sw128(s0, kMnBox) : sdesc_kmajor_sw128(s0);
      const uint64_t b0 = C::kWgrad ? sdesc_mnmajor_sw128(s0 + kABytes, kMnBox) : sdesc_kmajor_sw128(s0 + kABytes);
      constexpr uint64_t kStepA = (C::kWgrad || C::kDgrad ? 2048 : 32) >> 4, kStepB = (C::kWgrad ? 2048 : 32) >> 4;
      int stage = 0, acc = 0, where = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      GroupedRange rg(total_units, kblocks, worker, workers, kStreamK);
      int u, kb0, kb1;
      while (ok && rg.next(u, kb0, kb1)) {
        const GroupedUnit un = units.at(u);
        if (C::kWgrad) {
          kb1 = (un.n + 63) / 64;
          if (kb1 == 0) continue;  // an empty group: the epilogue writes zeros
        }
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          where = kWaitAccFree;
          break;
        }
        tc_fence_after();
        const int n_mma = C::kWgrad ? 256 : PAIR ? (un.n + 31) / 32 * 32 : (un.n + 15) / 16 * 16;
        const uint32_t idesc = idesc_f16_f32(PAIR ? 256 : 128, static_cast<uint32_t>(n_mma), a.fp16,
                                             C::kWgrad || C::kDgrad, C::kWgrad);
        const uint32_t d_acc = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            where = kWaitSlotFull;
            break;
          }
          tc_fence_after();
          const uint64_t at = static_cast<uint64_t>(stage * (C::kStageBytes >> 4));
          // MMAs of K = 16; a group's last block of rows ends with the group
          const int n_k = C::kWgrad ? min(4, (un.n - kb * 64 + 15) / 16) : 4;
          if (issue) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (C::kWgrad && k >= n_k) break;
              const uint32_t accum = k > 0 ? 1u : kb > kb0;
              if (PAIR)
                mma_bf16_ss_pair(d_acc, a0 + at + k * kStepA, b0 + at + k * kStepB, idesc, accum);
              else
                mma_bf16_ss(d_acc, a0 + at + k * kStepA, b0 + at + k * kStepB, idesc, accum);
            }
            if (PAIR)
              mma_commit_pair_mc(&empty[stage], 0x3);
            else
              mma_commit(&empty[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (issue) {
          if (PAIR)
            mma_commit_pair_mc(&tfull[acc], 0x3);
          else
            mma_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok && issue) raise_timeout(a.err, abort_flag, kKernGroupedGemm, where);
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
    }
  } else {
    // ---------------- epilogue: warps 2..5, TMEM lane quarter = warp % 4
    const int q = warp & 3;
    const int row = q * 32 + lane;  // this thread's TMEM lane = feature of the unit's 128
    int acc = 0, where = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    const uint32_t tempty_cl = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
    GroupedRange rg(total_units, kblocks, worker, workers, kStreamK);
    int u, kb0, kb1;
    uint8_t* my_store = store_buf + q * 8192;
    uint32_t buf = 0;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      const int feat0 = PAIR ? un.tile * 256 + static_cast<int>(rank) * 128 : un.tile * 128;
      const bool has_acc = !C::kWgrad || un.n > 0;
      if (has_acc) {
        // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
        const bool got = mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          where = kWaitAccFull;
          break;
        }
        tc_fence_after();
      }
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
      if constexpr (C::kWgrad) {
        // 32 rows x 128 bytes at a time: registers -> swizzled box -> TMA store
        const int r0 = feat0 + q * 32;
        const int span = a.out_fp32 ? 32 : 64;
        if (r0 < a.F) {
          for (int c0 = 0; c0 < 256; c0 += span) {
            const int col = un.tile_n * 256 + c0;
            if (col >= a.C) break;
            uint8_t* box = my_store + buf * 4096;
            buf ^= 1u;
            if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
            __syncwarp();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (a.out_fp32 && h == 1) break;
              uint32_t r[32];
              if (has_acc) {
                tmem_ld_32x32b_x32(t_row + c0 + 32 * h, r);
                tmem_ld_wait();
              } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = 0u;
              }
              if (a.out_fp32) {
#pragma unroll
                for (int p = 0; p < 8; ++p)
                  *reinterpret_cast<uint4*>(box + lane * 128 + ((p ^ (lane & 7)) << 4)) =
                      make_uint4(r[4 * p], r[4 * p + 1], r[4 * p + 2], r[4 * p + 3]);
              } else {
                const bool fp16 = a.fp16 != 0;
#pragma unroll
                for (int p = 0; p < 4; ++p) {
                  uint32_t w[4];
#pragma unroll
                  for (int j = 0; j < 4; ++j)
                    w[j] = static_cast<uint32_t>(to16(__uint_as_float(r[8 * p + 2 * j]), fp16)) |
                           (static_cast<uint32_t>(to16(__uint_as_float(r[8 * p + 2 * j + 1]), fp16)) << 16);
                  *reinterpret_cast<uint4*>(box + lane * 128 + (((p + 4 * h) ^ (lane & 7)) << 4)) =
                      make_uint4(w[0], w[1], w[2], w[3]);
                }
              }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (a.accumulate)
                tma_add_3d(&tm_w, box, col, r0, un.g);
              else
                tma_store_3d(&tm_w, box, col, r0, un.g);
              bulk_commit();
            }
          }
        }
      } else {
        uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(un.tok0) * a.ldo + feat0 + row;
        const bool fp16 = a.fp16 != 0, mine = feat0 + row < a.F;
        if (kStreamK && kb0 > 0) {
          // a later part of a unit that an earlier CTA started: hand over the partial sums
          float* slot = a.partials + static_cast<int64_t>(worker) * BN * 128;
          for (int c0 = 0; c0 < un.n; c0 += 16) {
            uint32_t r[16];
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
          if (kStreamK && kb1 < kblocks) {
            const int64_t unit_end = static_cast<int64_t>(u + 1) * kblocks;
            while (c_last + 1 < workers && rg.begin_of(c_last + 1) < unit_end) ++c_last;
          }
          for (int c0 = 0; c0 < un.n; c0 += 16) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(t_row + c0, r);
            tmem_ld_wait();
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(r[j]);
            bool good = true;
            for (int c = worker + 1; c <= c_last; ++c) {
              if (rg.begin_of(c) == rg.begin_of(c + 1)) continue;  // empty range
              if (c0 == 0 && !wait_flag(a.flags + c * 4 + q, abort_flag, kWaitTimeoutNs)) {
                good = false;
                break;
              }
              const float* slot = a.partials + static_cast<int64_t>(c) * BN * 128;
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] += __ldcg(slot + (c0 + j) * 128 + row);
            }
            if (!__all_sync(0xFFFFFFFFu, good)) {
              ok = false;
              where = kWaitPartials;
              break;
            }
            if (mine) {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                if (c0 + j < un.n) out[static_cast<int64_t>(c0 + j) * a.ldo] = to16(v[j], fp16);
            }
          }
        }
      }
      if (!ok) break;
      if (has_acc) {  // hand the accumulator back to the MMA thread
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote(tempty_cl + 8u * acc);
          else
            mbar_arrive(&tempty[acc]);
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
    }
    if (C::kWgrad && lane == 0) bulk_wait_all();
    if (!ok && lane == 0) raise_timeout(a.err, abort_flag, kKernGroupedGemm, where);
  }

  __syncthreads();
  // a pair keeps both CTAs (their shared memory, barriers and TMEM) until both are done
  if (PAIR) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, C::kTmemCols);
    else
      tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <int OP, int BN, int STAGES, int TOKBOX, bool PAIR>
cudaError_t launch_gemm(const CUtensorMap& tw, const CUtensorMap& tx, const GroupedGemmArgs& a, int num_sms,
                        cudaStream_t stream) {
  using C = Cfg<OP, BN, STAGES, TOKBOX, PAIR>;
  auto kernel = grouped_gemm_kernel<OP, BN, STAGES, TOKBOX, PAIR>;
  static PerDevice config;  // the smem attribute, and the CTA pairs that fit on the device at once
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = PAIR ? 2 : 1;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  int max_pairs = 0;
  const cudaError_t e = config.get(
      [&](int& pairs) -> cudaError_t {
        cudaError_t ce =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(C::kSmemBytes));
        if (ce != cudaSuccess || !PAIR) return ce;
        cudaLaunchConfig_t q = cfg;
        q.gridDim = dim3(2 * (kMaxGemmCtas / 2));
        q.attrs = attr + 1;
        q.numAttrs = 1;
        int n = 0;
        ce = cudaOccupancyMaxActiveClusters(&n, kernel, &q);
        if (ce != cudaSuccess) return ce;
        if (n <= 0) return cudaErrorInvalidConfiguration;
        pairs = n;
        return cudaSuccess;
      },
      &max_pairs);
  if (e != cudaSuccess) return e;
  const int most = PAIR ? kMaxGemmCtas / 2 : kMaxGemmCtas;
  const int workers = PAIR ? max_pairs : num_sms;
  cfg.gridDim = dim3((workers < most ? workers : most) * (PAIR ? 2 : 1));
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, tw, tx, a);
}

// rows per unit, stages, rows per token box: small (one CTA, 20 KB stages) and
// large (CTA pairs, 32 KB stages per CTA)
constexpr int kBn[2] = {32, 512}, kTile[2] = {128, 256}, kTokBox[2] = {16, 128};

}  // namespace

int grouped_bn(GroupedPlan plan) { return kBn[static_cast<int>(plan)]; }
int grouped_tile(GroupedPlan plan) { return kTile[static_cast<int>(plan)]; }
int grouped_tok_box(GroupedPlan plan) { return kTokBox[static_cast<int>(plan)]; }
size_t grouped_partial_bytes() { return static_cast<size_t>(kMaxGemmCtas) * kBn[0] * 128 * 4; }

cudaError_t launch_grouped_plan(const GroupedPlanArgs& a, const CUtensorMap& dy, const CUtensorMap& x,
                                cudaStream_t stream) {
  const int threads = (a.G + 31) / 32 * 32 < 256 ? 256 : (a.G + 31) / 32 * 32;
  grouped_plan_kernel<<<1, threads, 0, stream>>>(a, dy, x);
  return cudaGetLastError();
}

cudaError_t launch_grouped_gemm(GroupedOp op, GroupedPlan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                                const CUtensorMap& tm_x32, const GroupedGemmArgs& a, int num_sms,
                                cudaStream_t stream) {
  if (plan == GroupedPlan::kLarge) return launch_grouped_pair(op, tm_w, tm_x, tm_x32, a, stream);
  return op == GroupedOp::kForward
             ? launch_gemm<static_cast<int>(GroupedOp::kForward), kBn[0], 10, kTokBox[0], false>(tm_w, tm_x, a, num_sms,
                                                                                                  stream)
             : launch_gemm<static_cast<int>(GroupedOp::kDgrad), kBn[0], 10, kTokBox[0], false>(tm_w, tm_x, a, num_sms,
                                                                                                stream);
}

cudaError_t launch_grouped_wgrad(const CUtensorMap& tm_dw, const GroupedGemmArgs& a, cudaStream_t stream) {
  static const CUtensorMap none = {};
  return launch_gemm<static_cast<int>(GroupedOp::kWgrad), 256, 6, 128, true>(tm_dw, none, a, 0, stream);
}

}  // namespace moe
