// pair_sched.cuh -- work units handed to CTA pairs as they ask for them.
//
// Units of ragged groups differ in length, and their order (a weight tile's
// chunks next to one another, for L2) is periodic: dealt round-robin, one
// worker would get every short last chunk and its neighbour every full one.  So
// a pair starts with the unit of its index and takes the next ones from a counter
// in global memory.  When it takes one:
//   - when its weights' producer starts on the last unit: a pair that fetches
//     further ahead takes units of a small product while others have none;
//   - one earlier where there are at least eight units a pair, which hides the
//     counter's latency.
// Measured (us): 3190 rows of 59 groups, N = 360, K = 160, NVFP4: 15.4, fetching as far
// as there are slots 19.6; the input gradient of 134 rows, N = 2192, K = 1864: 20, with two
// and four fetches under way 32 and 54; NVFP4, 64 x 512 rows, N = K = 4096: one earlier 231, else 239.
//
// The odd CTA's MMA warp, which has no MMAs to issue, is the scheduler: it
// fetches units and puts them into a ring of kSchedSlots in both CTAs' shared
// memory, where every other warp of the pair reads them in order.  Which pair
// computes a unit does not change its result.
//
// The scheduler overwrites a slot once every warp has read it, so the even CTA's
// readings have to be ordered before its remote store: a release at cluster scope.
// Given by the reading warps themselves it waits for the epilogue's stores to
// global memory (256 groups of 64 rows, N = 1536, K = 256: 66 -> 76 us).  So the
// warps of each CTA signal inside it, and a warp of the even CTA without stores of
// its own, the relay, passes its CTA's signals on (63 to 66 us).
#pragma once

#include <cstdint>

#include "tc_ptx.cuh"

namespace moe {

constexpr int kSchedSlots = 4;
constexpr int kSchedBytes = kSchedSlots * (8 + 8 + 8 + 8 + 4) + 16;

struct PairSched {
  uint64_t* full;   // a slot's unit is there (in each CTA)
  uint64_t* empty;  // the odd CTA's: its warps, and the relay, have read it
  uint64_t* taken;  // the odd CTA's: its producer of the weights has read it
  uint64_t* seen;   // the even CTA's: its warps have read it
  volatile int32_t* unit;

  __device__ explicit PairSched(uint8_t* smem)
      : full(reinterpret_cast<uint64_t*>(smem)), empty(full + kSchedSlots), taken(empty + kSchedSlots),
        seen(taken + kSchedSlots), unit(reinterpret_cast<volatile int32_t*>(seen + kSchedSlots)) {}

  // one thread of each CTA, before the pair's cluster barrier; odd_readers: warps of the odd CTA that walk
  // the units (of the even one one more, the MMA warp)
  __device__ __forceinline__ void init(int odd_readers) const {
    for (int s = 0; s < kSchedSlots; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], odd_readers + 1);
      ptx::mbar_init(&taken[s], 1);
      ptx::mbar_init(&seen[s], odd_readers + 1);
    }
  }

  // The scheduler (one thread of the odd CTA): units pair, then pairs + counter, ...
  // until one >= total, which ends the readers' walks.  False: a wait ran out.
  __device__ bool schedule(int32_t* counter, int total, uint64_t timeout_ns, const volatile int* abort) const {
    using namespace ptx;
    const int pairs = static_cast<int>(gridDim.x >> 1), early = total >= 8 * pairs ? 1 : 0;
    int u = static_cast<int>(blockIdx.x >> 1);
    for (int i = 0;; ++i) {
      const int slot = i % kSchedSlots;
      if (!mbar_wait_cluster(&empty[slot], (i / kSchedSlots & 1) ^ 1u, timeout_ns, abort)) return false;
      unit[slot] = u;
      const uint32_t theirs = mapa_shared(smem_u32(const_cast<int32_t*>(unit) + slot), 0);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(theirs), "r"(u) : "memory");
      mbar_arrive_cluster(mapa_shared(smem_u32(&full[slot]), 0));
      mbar_arrive(&full[slot]);
      if (u >= total) return true;
      const int last = i - early;
      if (last >= 0 && !mbar_wait(&taken[last % kSchedSlots], last / kSchedSlots & 1, timeout_ns, abort)) return false;
      u = pairs + atomicAdd(counter, 1);
    }
  }

  // The relay (one thread of the even CTA).  False: a wait ran out.
  __device__ bool relay(int total, uint64_t timeout_ns, const volatile int* abort) const {
    using namespace ptx;
    const uint32_t empty_odd = mapa_shared(smem_u32(empty), 1);
    for (int i = 0;; ++i) {
      const int slot = i % kSchedSlots;
      if (!mbar_wait(&seen[slot], i / kSchedSlots & 1, timeout_ns, abort)) return false;
      const int u = unit[slot];
      mbar_arrive_cluster(empty_odd + 8u * slot);
      if (u >= total) return true;
    }
  }
};

// One warp's walk along the scheduled units.
struct PairUnits {
  PairSched sched;
  const int total;
  const volatile int* abort;
  const uint64_t timeout_ns;
  uint64_t* const read;  // where this CTA's warps signal that they have read a slot
  const bool taker;      // the odd CTA's producer of the weights
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;  // false: a wait ran out

  __device__ PairUnits(const PairSched& s, int units, uint64_t timeout, const volatile int* a, bool even,
                       bool weights_producer)
      : sched(s), total(units), abort(a), timeout_ns(timeout), read(even ? s.seen : s.empty),
        taker(!even && weights_producer) {}

  // the next unit (warp-uniform; a whole warp calls), or -1
  __device__ __forceinline__ int next() {
    using namespace ptx;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&sched.full[slot], phase, timeout_ns, abort))) {
      ok = false;
      return -1;
    }
    const int u = sched.unit[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      if (taker) mbar_arrive(&sched.taken[slot]);
      mbar_arrive(&read[slot]);
    }
    if (++slot == kSchedSlots) {
      slot = 0;
      phase ^= 1u;
    }
    return u < total ? u : -1;
  }
};

}  // namespace moe
