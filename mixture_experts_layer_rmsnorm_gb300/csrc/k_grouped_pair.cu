// k_grouped_pair.cu -- the forward and the input gradient of the grouped
// products for groups of many rows, on CTA pairs (tcgen05.mma cta_group::2,
// M = 256).  The mapping is k_grouped_gemm.cu's: the weights on the MMA's M
// side, a group's rows on its N side.
//
// Groups are ragged, and a weight tile has to be filled into shared memory
// once per unit whatever the unit's rows: with chunks of at most 256 rows a
// group of 520 rows costs three passes over its weights for two passes' worth
// of products (64 groups of 520 rows, N = 8192, K = 4096: 1612 us, of 512:
// 1284 us).  So a unit takes up to 512 rows, even chunks, and neither shared
// memory nor TMEM is divided into slots of the largest size:
//   - The ring in shared memory is a ring of bytes.  A stage is the 16 KB weight
//     tile plus half of the unit's rows (the pair's CTAs hold half each), so
//     units of few rows have more stages in flight.  Producer and MMA thread
//     compute the same places; the producer waits for the oldest stages until the
//     new one fits.
//   - TMEM's 512 columns are two accumulators of 256.  A unit of up to 256 rows
//     takes one, so that its epilogue runs under the next unit's MMAs; one of more takes both, with two
//     MMAs of about half its rows per step that share the stage's weight tile (an MMA of
//     few columns costs far more than its share: 256 + 32 columns 1.3 times 144 + 144).
// A group's rows are cut into units of up to bn rows, evenly (full units and a
// rest, 512 + 8 for 2 x 260 rows, measured 1.2 times as long), and units are handed out as
// pairs ask for them (pair_sched.cuh; dealt round-robin 1.14 times as long).
// Measured, 64 groups, N = 8192, K = 4096 (from card to card, as the power cap lets them): 512 rows
// 1179 to 1245 us (1.87 to 1.77 PFLOP/s, 0.96 to 0.91 of the burst rate), 520 rows 1362 to 1433 us,
// 256 rows 709 to 733 us (0.95 to 0.92 of HBM: the weights alone); one group of 8192 rows, N = K = 8192:
// 571 to 613 us (1.93 to 1.79 PFLOP/s).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bounded_wait.cuh"
#include "grouped.cuh"
#include "launch_config.cuh"
#include "pair_sched.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kABytes = 128 * 128;   // 128 features x 64 of the reduction, 16 bits
constexpr int kMnBox = 64 * 128;     // an MN-major box: 64 features x 64 of the reduction
constexpr int kRing = 224 * 1024;    // bytes: 7 stages of 256 rows, 4 of 512
constexpr int kStages = 11;          // stages in flight at most (the smallest are 20 KB)
constexpr int kAccCols = 256;
constexpr int kEpiWarps = 8;         // two per TMEM lane quarter, alternate groups of 32 columns
constexpr int kRowsWarp = 2 + kEpiWarps, kRelayWarp = kRowsWarp + 1;
constexpr int kThreads = 32 * (kRelayWarp + 1);  // + the weights' producer, the MMA warp, the rows' producer, the relay
constexpr int kBarBytes = 256;
constexpr int kTabBytes = 3 * (kGroupsSmem[1] + 1) * 4;
constexpr size_t kSmemBytes = 1024 + kRing + kBarBytes + kSchedBytes + kTabBytes;
static_assert((2 * kStages + 5) * 8 + 8 <= kBarBytes, "barrier area");
static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");

enum : int { kWaitSlotFree = 1, kWaitAccFree = 2, kWaitSlotFull = 3, kWaitAccFull = 4, kWaitUnit = 10 };

// A unit's size: MMA columns in all and of its first MMA, rows per CTA, rows
// loaded (boxes of 128 and of 32), bytes of a stage.
struct Size {
  int cols, cols0, half, rows, bytes;
  __device__ explicit Size(int n) {
    cols = (n + 15) & ~15;
    cols0 = cols <= kAccCols ? cols : (cols / 2 + 15) & ~15;
    half = cols / 2;
    const int rest = half & 127;
    rows = (half & ~127) + (rest > 96 ? 128 : (rest + 31) & ~31);
    bytes = kABytes + rows * 128;
  }
};

// Places in the byte ring, in the order of the stages: a stage lies whole, so
// the end of the ring is skipped where the next one does not fit.
struct BytePlace {
  int at = 0;
  uint32_t virt = 0;  // bytes given out so far, skipped ones included (mod 2^32)
  __device__ __forceinline__ int take(int bytes) {
    if (at + bytes > kRing) {
      virt += kRing - at;
      at = 0;
    }
    const int r = at;
    at += bytes;
    virt += bytes;
    return r;
  }
};

// A producer's walk along the ring (a whole warp): the place of the next stage,
// once the oldest stages have left room for it.  Lane s keeps the virtual end
// of stage s.
struct Producer {
  BytePlace place;
  uint64_t* empty;
  const volatile int* abort_flag;
  uint32_t freed_to = 0, my_end = 0, oldest_phase = 0;
  int stage = 0, oldest = 0, in_flight = 0;
  const int lane;
  __device__ Producer(uint64_t* e, const volatile int* f, int l) : empty(e), abort_flag(f), lane(l) {}

  __device__ __forceinline__ bool free_oldest(uint64_t timeout_ns, const volatile int* flag) {
    const bool got = __all_sync(0xFFFFFFFFu, mbar_wait(&empty[oldest], oldest_phase, timeout_ns, flag));
    freed_to = __shfl_sync(0xFFFFFFFFu, my_end, oldest);
    --in_flight;
    if (++oldest == kStages) {
      oldest = 0;
      oldest_phase ^= 1u;
    }
    return got;
  }
  // byte offset of the next stage (its index: stage, until advance()), or -1
  __device__ __forceinline__ int next(int bytes) {
    const int at = place.take(bytes);
    while (place.virt - freed_to > kRing || in_flight == kStages)
      if (!free_oldest(kWaitTimeoutNs, abort_flag)) return -1;
    if (lane == stage) my_end = place.virt;
    return at;
  }
  __device__ __forceinline__ void advance() {
    ++in_flight;
    if (++stage == kStages) stage = 0;
  }
  // every load issued has been used before the CTA exits
  __device__ __forceinline__ void drain() {
    const int never = 0;
    bool got = true;
    while (in_flight > 0 && got) got = free_oldest(kWaitTimeoutNs, &never);
  }
};

template <bool DGRAD>
__global__ void __launch_bounds__(kThreads, 1)
    grouped_pair_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                        const __grid_constant__ CUtensorMap tm_x32, const __grid_constant__ GroupedGemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kRing);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = empty + kStages;  // an accumulator's MMAs are complete
  uint64_t* tempty = tfull + 2;       // it is read, by the epilogue of both CTAs
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const PairSched sched(smem + kRing + kBarBytes);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + kRing + kBarBytes + kSchedBytes);

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
    tmem_alloc_pair(tmem_slot, 2 * kAccCols);
    tmem_relinquish_pair();
  }
  pdl_wait();  // the plan kernel's tables
  const GroupedTables tables = grouped_tables(a, tab, kGroupsSmem[1], kThreads);
  tc_fence_before();
  cluster_sync();  // the peer's barriers are initialised before any remote signal
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int total_units = tables.unit_off[a.G];
  const int kblocks = (a.R + 63) / 64;
  GroupedUnits units(tables, a.G, 1, a.bn, true);  // each warp walks its role's units
  PairUnits walk(sched, total_units, kWaitTimeoutNs, abort_flag, leader, warp == 0);

  if (warp == 0 || warp == kRowsWarp) {
    // ---------------- TMA producers: one warp for the weight tiles, one for the
    // rows (one thread that issues both, three to five copies a stage, is
    // slower than the copies); one lane issues
    const bool weights = warp == 0, issue = elect_one();
    const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_last();
    const uint32_t full_cl = mapa_shared(smem_u32(full), 0);  // both CTAs signal the even one
    Producer ring(empty, abort_flag, lane);
    bool ok = true;
    for (int u; ok && (u = walk.next()) >= 0;) {
      const GroupedUnit un = units.at(u);
      const Size z(un.n);
      const int feat = un.tile * 256 + static_cast<int>(rank) * 128;
      const int tok = un.tok0 + static_cast<int>(rank) * z.half;
      // a weight tile read by one chunk only is streamed; by more, kept
      const uint64_t pol_w = units.chunks > 1 ? pol_keep : pol_stream;
      for (int kb = 0; kb < kblocks; ++kb) {
        const int at = ring.next(z.bytes);
        if (at < 0) {
          ok = false;
          break;
        }
        if (issue) {
          uint8_t* sa = smem + at;
          const uint32_t bar = full_cl + 8u * ring.stage;
          if (weights) {
            if (leader) mbar_arrive_expect_tx(&full[ring.stage], 2 * z.bytes);
            if constexpr (DGRAD) {  // [64 rows of w][64 columns] boxes: the columns are the features
              tma_load_3d_pair(sa, &tm_w, bar, feat, kb * 64, un.g, pol_w);
              tma_load_3d_pair(sa + kMnBox, &tm_w, bar, feat + 64, kb * 64, un.g, pol_w);
            } else {
              tma_load_3d_pair(sa, &tm_w, bar, kb * 64, feat, un.g, pol_w);
            }
          } else {
            uint8_t* sb = sa + kABytes;
            int r = 0;
            for (; r + 128 <= z.rows; r += 128) tma_load_2d_pair(sb + r * 128, &tm_x, bar, kb * 64, tok + r, pol_keep);
            for (; r < z.rows; r += 32) tma_load_2d_pair(sb + r * 128, &tm_x32, bar, kb * 64, tok + r, pol_keep);
          }
        }
        __syncwarp();
        ring.advance();
      }
    }
    if (!(ok && walk.ok) && issue) raise_timeout(a.err, abort_flag, kKernGroupedGemm, walk.ok ? kWaitSlotFree : kWaitUnit);
    ring.drain();
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer for both CTAs: the whole warp walks the
      // units, one lane issues (a stage of narrow MMAs is bound by the issuing
      // thread's instructions: the descriptors advance by additions alone)
      const bool issue = elect_one();
      const uint32_t s0 = smem_u32(smem);
      const uint64_t a0 = DGRAD ? sdesc_mnmajor_sw128(s0, kMnBox) : sdesc_kmajor_sw128(s0);
      const uint64_t b0 = sdesc_kmajor_sw128(s0 + kABytes);
      constexpr uint64_t kStepA = (DGRAD ? 2048 : 32) >> 4, kStepB = 32 >> 4;  // K = 16
      bool ok = true;
      int where = 0;
      BytePlace place;
      int stage = 0;
      uint32_t phase = 0, uses = 0;  // accumulators taken so far: the next is uses & 1
      for (int u; ok && (u = walk.next()) >= 0;) {
        const GroupedUnit un = units.at(u);
        const Size z(un.n);
        const int parts = z.cols > z.cols0 ? 2 : 1;
        for (int j = 0; j < parts; ++j)
          ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&tempty[(uses + j) & 1], (((uses + j) >> 1) & 1u) ^ 1u,
                                                      kWaitTimeoutNs, abort_flag));
        if (!ok) {
          where = kWaitAccFree;
          break;
        }
        tc_fence_after();
        const uint32_t d0 = tmem_base + (uses & 1) * kAccCols, d1 = tmem_base + ((uses & 1) ^ 1) * kAccCols;
        const uint64_t b1 = static_cast<uint64_t>(z.cols0 / 2 * 128) >> 4;  // the second MMA's rows
        const uint32_t idesc0 = idesc_f16_f32(256, static_cast<uint32_t>(z.cols0), a.fp16, DGRAD, 0);
        const uint32_t idesc1 = idesc_f16_f32(256, static_cast<uint32_t>(z.cols - z.cols0), a.fp16, DGRAD, 0);
        for (int kb = 0; kb < kblocks; ++kb) {
          const int at = place.take(z.bytes);
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            where = kWaitSlotFull;
            break;
          }
          tc_fence_after();
          const uint64_t ad = a0 + static_cast<uint64_t>(at >> 4), bd = b0 + static_cast<uint64_t>(at >> 4);
          if (issue) {
            mma_bf16_ss_pair(d0, ad, bd, idesc0, kb > 0);
#pragma unroll
            for (int k = 1; k < 4; ++k) mma_bf16_ss_pair(d0, ad + k * kStepA, bd + k * kStepB, idesc0, 1u);
            if (parts == 2) {
              const uint64_t bd1 = bd + b1;
              mma_bf16_ss_pair(d1, ad, bd1, idesc1, kb > 0);
#pragma unroll
              for (int k = 1; k < 4; ++k) mma_bf16_ss_pair(d1, ad + k * kStepA, bd1 + k * kStepB, idesc1, 1u);
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
        if (issue)
          for (int j = 0; j < parts; ++j) mma_commit_pair_mc(&tfull[(uses + j) & 1], 0x3);
        __syncwarp();
        uses += parts;
      }
      if (!walk.ok) where = kWaitUnit;
      if (!(ok && walk.ok) && issue) raise_timeout(a.err, abort_flag, kKernGroupedGemm, where);
      // all MMAs issued have finished before TMEM is released
      if (issue) mma_commit_pair(done);
      __syncwarp();
      int dummy = 0;
      mbar_wait(done, 0, kWaitTimeoutNs, &dummy);
    } else if (lane == 0) {
      if (!sched.schedule(a.next_unit, total_units, kWaitTimeoutNs, abort_flag))
        raise_timeout(a.err, abort_flag, kKernGroupedGemm, kWaitUnit);
    }
  } else if (warp == kRelayWarp) {
    if (leader && lane == 0 && !sched.relay(total_units, kWaitTimeoutNs, abort_flag))
      raise_timeout(a.err, abort_flag, kKernGroupedGemm, kWaitUnit);
  } else {
    // ---------------- epilogue: TMEM lane quarter = warp % 4; a quarter's two
    // warps take alternate groups of 32 columns
    const int q = warp & 3, turn = (warp - 2) >> 2;
    const int row = q * 32 + lane;  // feature of this CTA's 128
    const bool fp16 = a.fp16 != 0;
    const int odd = lane & 1;
    const uint32_t tempty_cl = mapa_shared(smem_u32(tempty), 0);
    bool ok = true;
    uint32_t uses = 0;
    for (int u; ok && (u = walk.next()) >= 0;) {
      const GroupedUnit un = units.at(u);
      const Size z(un.n);
      const int feat = un.tile * 256 + static_cast<int>(rank) * 128 + row;
      const bool mine = feat < a.F;  // (F is even: a pair of lanes alike)
      // this lane's two features, of its row of each pair of rows
      uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(un.tok0 + odd) * a.ldo + (feat & ~1);
      const int parts = z.cols > z.cols0 ? 2 : 1;
      for (int j = 0; j < parts; ++j) {
        const uint32_t buf = uses & 1;
        // warp-uniform outcome: tcgen05.ld below is executed by all 32 lanes
        const bool got = mbar_wait(&tfull[buf], (uses >> 1) & 1u, kWaitTimeoutNs, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          ok = false;
          break;
        }
        tc_fence_after();
        ++uses;
        const int cols = j ? z.cols - z.cols0 : z.cols0, before = j ? z.cols0 / 2 : 0;
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + buf * kAccCols;
        for (int c0 = 32 * turn; c0 < cols; c0 += 64) {
          uint32_t r[32];
          __syncwarp();  // tcgen05.ld is warp-aligned: the stores before it are not
          tmem_ld_32x32b_x32(t_row + c0, r);
          tmem_ld_wait();
#pragma unroll
          for (int h = 0; h < 4; ++h) {  // 8 columns: rows of one half
            const int c = c0 + 8 * h;
            const int t = c < cols / 2 ? before + c : z.half + before + c - cols / 2;
            const int left = c < cols ? un.n - t : 0;
            uint16_t* o = out + static_cast<int64_t>(t) * a.ldo;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const uint32_t v = trade_rows(pack16(__uint_as_float(r[8 * h + i]), __uint_as_float(r[8 * h + i + 1]), fp16));
              if (mine && i + odd < left) *reinterpret_cast<uint32_t*>(o + static_cast<int64_t>(i) * a.ldo) = v;
            }
          }
        }
        // hand the accumulator back to the MMA thread
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty_cl + 8u * buf);
      }
    }
    if (!(ok && walk.ok) && lane == 0)
      raise_timeout(a.err, abort_flag, kKernGroupedGemm, walk.ok ? kWaitAccFull : kWaitUnit);
  }

  __syncthreads();
  cluster_sync();  // both CTAs keep their shared memory, barriers and TMEM until both are done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 2 * kAccCols);
  }
}

template <bool DGRAD>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const CUtensorMap& tx32, const GroupedGemmArgs& a,
                   cudaStream_t stream) {
  static PerDevice config;
  return launch_pairs(grouped_pair_kernel<DGRAD>, config, kThreads, kSmemBytes, stream, tw, tx, tx32, a);
}

}  // namespace

cudaError_t launch_grouped_pair(GroupedOp op, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                                const CUtensorMap& tm_x32, const GroupedGemmArgs& a, cudaStream_t stream) {
  return op == GroupedOp::kForward ? launch<false>(tm_w, tm_x, tm_x32, a, stream)
                                   : launch<true>(tm_w, tm_x, tm_x32, a, stream);
}

}  // namespace moe
