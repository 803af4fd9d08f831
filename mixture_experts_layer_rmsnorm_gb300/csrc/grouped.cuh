// grouped.cuh -- what the products grouped by expert share (internal): the
// group tables a call's plan kernel writes into the workspace, the work units
// made from them, and the launchers.
//
// Rows of the token matrices belong to groups: group g holds rows
// [start_g, start_g + count_g).  Work units are numbered group by group; a
// group's units are (its token chunks or column tiles) x (its feature tiles).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "moe_kernels.cuh"
#ifdef __CUDACC__
#include "bounded_wait.cuh"
#endif

namespace moe {

enum : int32_t { kKernGroupedPlan = 9, kKernGroupedGemm = 10, kKernFp4Gemm = 11, kKernFp8Gemm = 12 };

constexpr int kGroupsMax = 1024;
// the GEMM kernels keep the tables in shared memory up to this many groups
// (single CTAs; CTA pairs, whose ring takes nearly all of it)
constexpr int kGroupsSmem[2] = {256, 128};

enum class GroupedOp : int { kForward = 0, kDgrad = 1, kWgrad = 2 };

// Plan kernel (one CTA): checks offsets / counts, writes start[G], count[G]
// and unit_off[G + 1], clears the error word and `n_flags` stream-K flags, and
// for the weight gradient writes the groups' tensor maps.
//   units of group g: ceil(count_g / bn) * tiles, or (bn = 0) `tiles`, none
//   for an empty group if skip_empty.
// A group that leaves [0, rows) or runs into the next one records
// MOE_ERR_DEVICE, and the call then has no units at all.
struct GroupedPlanArgs {
  const int32_t* offsets;  // [G + 1], or null: G equal groups of rows / G rows
  const int32_t* counts;   // [G], or null: offsets[g + 1] - offsets[g]
  int G;
  int64_t rows;
  int bn, tiles, skip_empty;
  int32_t* start;
  int32_t* count;
  int32_t* unit_off;
  int32_t* err;
  int32_t* flags;
  int n_flags;
  CUtensorMap* maps;  // weight gradient: [G][2] maps of dy and x whose rows end with the group, else null
};
cudaError_t launch_grouped_plan(const GroupedPlanArgs& a, const CUtensorMap& dy, const CUtensorMap& x,
                                cudaStream_t stream);

// One grouped 16-bit product.  F: features on the MMA's M side (N for the
// forward and the weight gradient, K for the input gradient); R: reduction
// length (forward K, input gradient N; unused by the weight gradient); C: the
// weight gradient's columns (K).
struct GroupedGemmArgs {
  const int32_t* start;
  const int32_t* count;
  const int32_t* unit_off;
  const CUtensorMap* maps;  // weight gradient: see GroupedPlanArgs
  int32_t* err;
  float* partials;  // stream-K partial sums: [kMaxGemmCtas][BN][128] fp32; weight gradient into 16 bits:
                    // sums of the segments so far, [kMaxGemmCtas][256][128]
  int32_t* flags;   // [kMaxGemmCtas * 4], zero on entry
  int32_t* next_unit;  // CTA pairs: the next unit to hand out, zero on entry
  void* out;        // forward / input gradient: rows of ldo elements of the operand type
  int64_t ldo;
  int G, F, R, C;
  int tiles;       // M tiles (of 128, or 256 for CTA pairs) per group
  int tiles_n;     // weight gradient: column tiles of 256
  int bn;          // rows per unit at most (CTA pairs; the single-CTA plan's is fixed)
  int fp16;        // operands fp16, else bf16
  int out_fp32;    // weight gradient: fp32, else the operand type
  int accumulate;  // weight gradient (fp32): add to what dw holds
};

// Tile plans of the forward and the input gradient.
enum class GroupedPlan : int { kSmall = 0, kLarge = 1 };
// token rows per unit at most: 32, or what the expected rows per group make the fastest
int grouped_bn(GroupedPlan plan, int64_t rows, int64_t groups, int64_t tiles, int num_sms);
int grouped_tile(GroupedPlan plan);       // features per unit
int grouped_tok_box(GroupedPlan plan);    // token rows per TMA box
size_t grouped_partial_bytes();           // stream-K partial sums
constexpr int kWgradTile = 256;           // rows and columns of a unit of the weight gradient
constexpr int kWgradSegment16 = 3840;     // rows whose sum the tensor core accumulates, into 16 bits
size_t grouped_wgrad_sum_bytes();         // sums of longer groups into 16 bits

// tm_x: the token rows in boxes of kTokBox[plan] rows; tm_x32: of 32 (large plan)
cudaError_t launch_grouped_gemm(GroupedOp op, GroupedPlan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                                const CUtensorMap& tm_x32, const GroupedGemmArgs& a, int num_sms,
                                cudaStream_t stream);
cudaError_t launch_grouped_pair(GroupedOp op, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                                const CUtensorMap& tm_x32, const GroupedGemmArgs& a, cudaStream_t stream);
cudaError_t launch_grouped_wgrad(const CUtensorMap& tm_dw, const GroupedGemmArgs& a, cudaStream_t stream);

#ifdef __CUDACC__

// Two fp32 values rounded to 16 bits, `lo` in the low half.
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A lane's word holds one feature (its lane's) of rows c and c + 1.  Neighbouring
// lanes trade halves: the even lane gets both features of row c, the odd
// one those of row c + 1, so that each stores 4 bytes of one row (whole warp).
__device__ __forceinline__ uint32_t trade_rows(uint32_t word) {
  const uint32_t other = __shfl_xor_sync(0xFFFFFFFFu, word, 1);
  return __byte_perm(word, other, (threadIdx.x & 1) ? 0x3276 : 0x5410);
}

struct GroupedUnit {
  int g, tile, tile_n, tok0, n, start, count;
};

// The group tables as a kernel's roles read them: copies in shared memory
// (G <= the room it has), or the workspace's, through L1.
struct GroupedTables {
  const int32_t* unit_off;
  const int32_t* start;
  const int32_t* count;
};

// Copies the tables to `smem` ([3][room + 1]) with the block's threads (visible
// after the next barrier) where they fit.
__device__ __forceinline__ GroupedTables grouped_tables(const GroupedGemmArgs& a, int32_t* smem, int room,
                                                        int threads) {
  if (a.G > room) return GroupedTables{a.unit_off, a.start, a.count};
  for (int i = threadIdx.x; i <= a.G; i += threads) {
    smem[i] = __ldcg(a.unit_off + i);
    if (i < a.G) {
      smem[room + 1 + i] = __ldcg(a.start + i);
      smem[2 * (room + 1) + i] = __ldcg(a.count + i);
    }
  }
  return GroupedTables{smem, smem + room + 1, smem + 2 * (room + 1)};
}

// Units -> groups for one role, which asks for ascending units: the group of
// the last unit is kept, and searched for (binary, in unit_off) only when a
// unit lies behind it.
// A unit's feature tile and token chunk: chunk fastest (units that read the
// same weight tile are neighbours, so the CTAs running side by side read it
// from DRAM once), or (bn = 0) its feature tile and column tile.  Chunks are
// bn rows each and a rest, or (even) as equal as rows go.
struct GroupedUnits {
  GroupedTables t;
  int G, tiles_n, bn;
  bool even;
  int g, first, last;  // the kept group and its units [first, last)
  int start, count, chunks;

  __device__ GroupedUnits(const GroupedTables& tables, int groups, int tiles_n_, int bn_, bool even_ = false)
      : t(tables), G(groups), tiles_n(tiles_n_), bn(bn_), even(even_), g(0), first(0), last(0), start(0), count(0),
        chunks(1) {}

  __device__ __forceinline__ int chunk_start(int i) const {
    return even ? static_cast<int>(static_cast<int64_t>(i) * count / chunks) : i * bn;
  }

  __device__ __forceinline__ GroupedUnit at(int u) {
    if (u >= last) {
      int lo = g, hi = G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.unit_off[mid] <= u)
          lo = mid;
        else
          hi = mid;
      }
      g = lo;
      first = t.unit_off[lo];
      last = t.unit_off[lo + 1];
      start = t.start[lo];
      count = t.count[lo];
      chunks = bn > 0 ? (count + bn - 1) / bn : tiles_n;  // >= 1: u lies in this group's range
    }
    GroupedUnit r;
    r.g = g;
    r.start = start;
    r.count = count;
    const int local = u - first;
    r.tile = local / chunks;
    const int fast = local - r.tile * chunks;
    r.tile_n = bn > 0 ? 0 : fast;
    if (bn > 0) {
      const int from = chunks > 1 ? chunk_start(fast) : 0;
      r.tok0 = start + from;
      r.n = (fast + 1 < chunks ? chunk_start(fast + 1) : count) - from;
    } else {
      r.tok0 = start;
      r.n = count;
    }
    return r;
  }
};

// A worker's share of a stream-K split, as segments: K-blocks [kb0, kb1) of
// unit u.  The (unit, K-block) iterations form one list; every worker takes a
// contiguous range of equal length.  Where there is little to do, fewer workers, since each
// part of a unit is one more to join: at least four K-blocks each, or an eighth of a unit
// where that is more, but never more than a whole unit.
//   us for parts of           1     2     4     8    16 K-blocks
//   8 rows, N 152, K 5168   50.6  33.3  18.4  13.6  12.7
//   8 x 1 row, N 512, K 128  8.1   5.8   6.6   8.6
struct GroupedRange {
  int64_t it, end, W;
  int kblocks, workers;
  __device__ GroupedRange(int units, int kb, int worker, int workers_)
      : W(static_cast<int64_t>(units) * kb), kblocks(kb), workers(workers_) {
    const int least = min(kb, max(4, kb / 8));
    if (W < static_cast<int64_t>(workers) * least) workers = max(1, static_cast<int>(W / least));
    it = begin_of(worker);
    end = begin_of(worker + 1);
  }
  // first iteration of a worker's range
  __device__ int64_t begin_of(int worker) const { return worker < workers ? W * worker / workers : W; }
  // Waits until the workers first .. last that have a range have handed over their
  // partial sums: a lane each, all flags at once (a whole warp calls; the
  // fence and the warp's barrier pass each lane's acquire on to all).  flags: 4 a worker.
  __device__ bool wait_partials(const int32_t* flags, int first, int last, const volatile int* abort_flag) const {
    bool good = true;
    for (int c = first + static_cast<int>(threadIdx.x & 31); c <= last; c += 32)
      if (begin_of(c) < begin_of(c + 1)) good = wait_flag_thread(flags + c * 4, abort_flag, kWaitTimeoutNs) && good;
    good = __all_sync(0xFFFFFFFFu, good);
    if (first <= last) __threadfence();
    __syncwarp();
    return good;
  }
  __device__ bool next(int& u, int& kb0, int& kb1) {
    if (it >= end) return false;
    u = static_cast<int>(it / kblocks);
    kb0 = static_cast<int>(it - static_cast<int64_t>(u) * kblocks);
    const int64_t stop = kb0 + (end - it);
    kb1 = stop < kblocks ? static_cast<int>(stop) : kblocks;
    it += kb1 - kb0;
    return true;
  }
};

#endif  // __CUDACC__

}  // namespace moe
