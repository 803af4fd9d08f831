// k_grouped_wgrad.cu -- the weight gradient of the products grouped by expert,
//   dw_g = sum over the group's rows p of dy[p, :]^T x[p, :]
// on CTA pairs (tcgen05.mma cta_group::2, 256 x 256 tiles of dw_g, fp32
// accumulation in TMEM).
//
// The reduction runs over the group's rows, the slow index of both operands:
// both are MN-major (the descriptors' transpose bits), read as stored.  A
// group's last block of 64 rows holds rows of the next group, which must not
// enter the sum (as zeros times a NaN would): the plan kernel writes per group
// copies of the host's two tensor maps whose row extent ends with the group, so
// TMA fills the rows past it with zeros, and MMAs past it are not issued.
//
// Two accumulators of 256 columns: a tile's epilogue runs under the next tile's
// MMAs.  The epilogue's four warps (one per TMEM lane quarter) move 32 x 128-byte
// boxes through shared memory, two each, to TMA stores, which clip at the matrix's
// edges; fp32 accumulation into dw is a TMA add, each element added once, so no
// order changes a result.  An empty group's tile is stored as zeros, without MMAs.
// Tiles go round-robin to the CTA pairs (a group's tiles are equally long).
//
// Long groups.  The tensor core cuts each addition to its fp32 accumulator,
// towards zero: the error grows with the number of additions (relative, 2-norm,
// random signs: 4.7e-7 for 512 rows, 9.1e-6 for 8192; all signs equal: 8.0e-7 and
// 3.1e-5).  So TMEM accumulates segments of a group, and their sums are added in
// fp32, rounded to nearest, in order.
//   Into fp32: segments of 768 rows; later ones are added to dw by TMA (a warp
//   waits for its earlier stores before it adds to them).
//   Into 16 bits, which cannot hold the sum: even segments of at most 3840 rows.
//   A step of 16 rows cuts at most 17 terms by 2^-23 of the largest, so one loses
//   less than 3840 * 17 / 16 * 2^-23 = 4.9e-4 of sum |dy x|, half an fp16 step.
//   Every thread keeps the sums of its row of the tile in the workspace (128 KB per
//   CTA, in L2) and rounds once, with the last segment.  Measured, N = K = 4096: 8 groups
//   of 8192 rows 1222 us (accumulated whole 1187); 2 of 65536, N = K = 2048: 650 (625).
//
// Bound: by writing dw where groups are short (a tile of fp32 moves 128 KB per
// CTA for 64 KB of operands per 64 rows), else by the tensor cores; in between by shared memory, which
// the operands cross twice and the tile too.  Measured, fp32: 64 groups of 32768 rows in all,
// N = K = 4096: 983 to 1045 us under the power cap (0.72 to 0.68 of the bytes' time; its L1 / shared-memory pipe
// is 80% busy); 64 x 512 even rows 891 to 972 us, added to dw 1730 us (0.78 of the bytes' time: dw is read
// too), into 16 bits 700 to 762 us.
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

constexpr int kMnBox = 64 * 128;                // 64 columns x 64 rows, 16 bits
constexpr int kOperand = 2 * kMnBox;            // this CTA's 128 columns of dy, or of x
constexpr int kStageBytes = 2 * kOperand;
constexpr int kStages = 6;
// rows per accumulation: multiples of 64
constexpr int kSegment32 = 768, kSegment16 = kWgradSegment16;
static_assert(kSegment32 % 64 == 0 && kSegment16 % 64 == 0, "whole stages");
static_assert(2 * kMaxPairs <= kMaxGemmCtas, "a place of its own for each CTA's sums");
constexpr int kEpiWarps = 4;
constexpr int kBox = 32 * 128;                  // an epilogue warp has two boxes of 32 rows x 128 bytes
constexpr int kThreads = 32 * (2 + kEpiWarps);
constexpr int kBarBytes = 256;
constexpr int kTabBytes = 3 * (kGroupsSmem[1] + 1) * 4;
constexpr size_t kSmemBytes = 1024 + kStages * kStageBytes + 2 * kEpiWarps * kBox + kBarBytes + kTabBytes;
static_assert((2 * kStages + 5) * 8 + 8 <= kBarBytes, "barrier area");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

enum : int { kWaitSlotFree = 1, kWaitAccFree = 2, kWaitSlotFull = 3, kWaitAccFull = 4 };

__global__ void __launch_bounds__(kThreads, 1)
    grouped_wgrad_kernel(const __grid_constant__ CUtensorMap tm_dw, const __grid_constant__ GroupedGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* boxes = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(boxes + 2 * kEpiWarps * kBox);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* tab = reinterpret_cast<int32_t*>(boxes + 2 * kEpiWarps * kBox + kBarBytes);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int worker = static_cast<int>(blockIdx.x >> 1), workers = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * kEpiWarps);  // of both CTAs
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_dw);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  pdl_wait();  // the plan kernel's tables and maps
  const GroupedTables tables = grouped_tables(a, tab, kGroupsSmem[1], kThreads);
  tc_fence_before();
  cluster_sync();  // the peer's barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int total_units = tables.unit_off[a.G];
  GroupedUnits units(tables, a.G, a.tiles_n, 0);  // each thread walks its role's units
  // rows of a unit's segments (into 16 bits even ones: a short last one would wait for the sums' way through L2)
  auto segment_of = [&](int n) {
    if (a.out_fp32 || n <= kSegment16) return a.out_fp32 ? kSegment32 : kSegment16;
    const int parts = (n + kSegment16 - 1) / kSegment16;
    return ((n + parts - 1) / parts + 63) / 64 * 64;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer
      const uint64_t policy = policy_evict_last();  // both operands are read by every tile of their group
      const uint32_t full_cl = mapa_shared(smem_u32(full), 0);  // both CTAs signal the even one
      int stage = 0;
      uint32_t phase = 0;
      int64_t issued = 0;
      bool ok = true;
      int map_group = -1;
      for (int u = worker; ok && u < total_units; u += workers) {
        const GroupedUnit un = units.at(u);
        const int row = un.tile * 256 + static_cast<int>(rank) * 128, col = un.tile_n * 256 + static_cast<int>(rank) * 128;
        const CUtensorMap* map = a.maps + 2 * un.g;
        if (un.g != map_group) {
          tensormap_acquire(map);
          tensormap_acquire(map + 1);
          map_group = un.g;
        }
        for (int p = 0; p < un.n; p += 64) {
          if (!mbar_wait(&empty[stage], phase ^ 1u, kWaitTimeoutNs, abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* sa = smem + stage * kStageBytes;
          const uint32_t bar = full_cl + 8u * stage;
          if (leader) mbar_arrive_expect_tx(&full[stage], 2 * kStageBytes);
#pragma unroll
          for (int j = 0; j < 2; ++j) tma_load_2d_pair(sa + j * kMnBox, map, bar, row + 64 * j, un.tok0 + p, policy);
#pragma unroll
          for (int j = 0; j < 2; ++j)
            tma_load_2d_pair(sa + kOperand + j * kMnBox, map + 1, bar, col + 64 * j, un.tok0 + p, policy);
          ++issued;
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok) raise_timeout(a.err, abort_flag, kKernGroupedGemm, kWaitSlotFree);
      // every load this thread issued has landed before the CTA exits (the odd
      // CTA of a pair sees that through the release of its stages)
      for (int s = 0; s < kStages; ++s) {
        if (issued <= s) break;
        const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
        int dummy = 0;
        mbar_wait(leader ? &full[s] : &empty[s], par, kWaitTimeoutNs, &dummy);
      }
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer for both CTAs: the whole warp walks the units, one lane issues
      const bool issue = elect_one();
      const uint32_t s0 = smem_u32(smem);
      const uint64_t a0 = sdesc_mnmajor_sw128(s0, kMnBox), b0 = sdesc_mnmajor_sw128(s0 + kOperand, kMnBox);
      const uint32_t idesc = idesc_f16_f32(256, 256, a.fp16, 1, 1);
      int stage = 0, acc = 0, where = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int u = worker; ok && u < total_units; u += workers) {
        const GroupedUnit un = units.at(u);
        const int segment = segment_of(un.n);
        for (int row0 = 0; ok && row0 < un.n; row0 += segment) {  // (an empty group: the epilogue writes zeros)
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], acc_phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            where = kWaitAccFree;
            break;
          }
          tc_fence_after();
          const uint32_t d_acc = tmem_base + static_cast<uint32_t>(acc * 256);
          const int end = min(un.n, row0 + segment);
          for (int row = row0; row < end; row += 64) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, kWaitTimeoutNs, abort_flag))) {
              ok = false;
              where = kWaitSlotFull;
              break;
            }
            tc_fence_after();
            const uint64_t at = static_cast<uint64_t>(stage * (kStageBytes >> 4));
            const int n_k = min(4, (un.n - row + 15) / 16);  // MMAs of 16 rows
            if (issue) {
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (k >= n_k) break;
                mma_bf16_ss_pair(d_acc, a0 + at + k * (2048 >> 4), b0 + at + k * (2048 >> 4), idesc,
                                 k > 0 ? 1u : row > row0);
              }
              mma_commit_pair_mc(&empty[stage], 0x3);
            }
            __syncwarp();
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (issue) mma_commit_pair_mc(&tfull[acc], 0x3);
          __syncwarp();
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
      if (!ok && issue) raise_timeout(a.err, abort_flag, kKernGroupedGemm, where);
      // all MMAs issued have finished before TMEM is released
      if (issue) mma_commit_pair(done);
      __syncwarp();
      int dummy = 0;
      mbar_wait(done, 0, kWaitTimeoutNs, &dummy);
    }
  } else {
    // ---------------- epilogue: TMEM lane quarter = warp % 4
    const int q = warp & 3;
    uint8_t* my_boxes = boxes + q * 2 * kBox;
    uint32_t buf = 0;
    const uint32_t tempty_cl = mapa_shared(smem_u32(tempty), 0);
    const int span = a.out_fp32 ? 32 : 64;  // columns of a box
    const bool fp16 = a.fp16 != 0;
    // [256 columns][128 rows] of this CTA, this thread's row: read and written by this thread alone
    float* sums = a.partials + static_cast<int64_t>(blockIdx.x) * (kWgradTile * 128) + q * 32 + lane;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int u = worker; ok && u < total_units; u += workers) {
      const GroupedUnit un = units.at(u);
      const int row0 = un.tile * 256 + static_cast<int>(rank) * 128 + q * 32;
      const int segment = segment_of(un.n);
      int left = un.n;
      do {  // segments; an empty group: zeros once
        const bool has_acc = left > 0, first = left == un.n;
        if (has_acc) {
          // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        const bool add = a.out_fp32 && (a.accumulate || !first);
        const bool to_sums = !a.out_fp32 && left > segment;  // into 16 bits, and not the last segment
        if (add && !first && lane == 0) bulk_wait_all();  // the earlier segments are in dw
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * 256);
        if (to_sums) {
          for (int c0 = 0; c0 < 256 && row0 < a.F && un.tile_n * 256 + c0 < a.C; c0 += 32) {
            float* at = sums + c0 * 128;
            float before[32];  // every load ahead of the stores (one by one: 84 us a segment)
#pragma unroll
            for (int j = 0; j < 32; ++j) before[j] = first ? 0.0f : __ldcg(at + j * 128);
            uint32_t r[32];
            __syncwarp();  // tcgen05.ld is warp-aligned
            tmem_ld_32x32b_x32(t_row + c0, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) __stcg(at + j * 128, before[j] + __uint_as_float(r[j]));
          }
        }
        for (int c0 = to_sums ? 256 : 0; c0 < 256 && row0 < a.F; c0 += span) {
          const int col = un.tile_n * 256 + c0;
          if (col >= a.C) break;
          uint8_t* box = my_boxes + buf * kBox;
          buf ^= 1u;
          if (lane == 0) bulk_wait_read<1>();  // the box's last store has read it
          __syncwarp();    // (tcgen05.ld is warp-aligned: lane 0 comes from its store)
          uint32_t w[32];  // the lane's 128 bytes
          if (!has_acc) {
#pragma unroll
            for (int j = 0; j < 32; ++j) w[j] = 0u;
          } else if (a.out_fp32) {
            tmem_ld_32x32b_x32(t_row + c0, w);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t r[32];
              tmem_ld_32x32b_x32(t_row + c0 + 32 * h, r);
              tmem_ld_wait();
              if (!first) {
                const float* at = sums + (c0 + 32 * h) * 128;
#pragma unroll
                for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__ldcg(at + j * 128) + __uint_as_float(r[j]));
              }
#pragma unroll
              for (int j = 0; j < 16; ++j)
                w[16 * h + j] = pack16(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]), fp16);
            }
          }
#pragma unroll
          for (int p = 0; p < 8; ++p)  // the 128-byte swizzle of the store's map
            *reinterpret_cast<uint4*>(box + lane * 128 + ((p ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]);
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) {
            if (add)
              tma_add_3d(&tm_dw, box, col, row0, un.g);
            else
              tma_store_3d(&tm_dw, box, col, row0, un.g);
            bulk_commit();
          }
        }
        if (has_acc) {  // hand the accumulator back to the MMA warp
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(tempty_cl + 8u * acc);
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
        left -= segment;
      } while (left > 0);
    }
    if (lane == 0) bulk_wait_all();
    if (!ok && lane == 0) raise_timeout(a.err, abort_flag, kKernGroupedGemm, kWaitAccFull);
  }

  __syncthreads();
  cluster_sync();  // both CTAs keep their shared memory, barriers and TMEM until both are done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace

size_t grouped_wgrad_sum_bytes() { return static_cast<size_t>(kMaxGemmCtas) * kWgradTile * 128 * 4; }

cudaError_t launch_grouped_wgrad(const CUtensorMap& tm_dw, const GroupedGemmArgs& a, cudaStream_t stream) {
  static PerDevice config;
  return launch_pairs(grouped_wgrad_kernel, config, kThreads, kSmemBytes, stream, tm_dw, a);
}

}  // namespace moe
