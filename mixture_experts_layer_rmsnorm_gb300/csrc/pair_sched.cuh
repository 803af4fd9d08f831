// pair_sched.cuh -- work units handed to CTA pairs as they ask for them.
//
// Units of ragged groups differ in length, and their order (a weight tile's
// chunks next to one another, for L2) is periodic: dealt round-robin, one
// worker would get every short last chunk and its neighbour every full one.  So
// a pair takes the next unit from a counter in global memory.  The odd CTA's
// MMA warp, which has no MMAs to issue, is the scheduler: it fetches units
// ahead and puts them into a ring of kSchedSlots in both CTAs' shared memory,
// where every other warp of the pair reads them in order.  Which pair computes
// a unit does not change its result.
#pragma once

#include <cstdint>

#include "tc_ptx.cuh"

namespace moe {

constexpr int kSchedSlots = 4;
constexpr int kSchedBytes = kSchedSlots * (8 + 8 + 4) + 16;

struct PairSched {
  uint64_t* full;   // a slot's unit is there (in each CTA)
  uint64_t* empty;  // every warp of the pair has read it (the odd CTA's)
  volatile int32_t* unit;

  __device__ explicit PairSched(uint8_t* smem)
      : full(reinterpret_cast<uint64_t*>(smem)), empty(full + kSchedSlots),
        unit(reinterpret_cast<volatile int32_t*>(empty + kSchedSlots)) {}

  // one thread of each CTA, before the pair's cluster barrier; readers: warps of both CTAs that walk the units
  __device__ __forceinline__ void init(int readers) const {
    for (int s = 0; s < kSchedSlots; ++s) {
      ptx::mbar_init(&full[s], 1);
      ptx::mbar_init(&empty[s], readers);
    }
  }

  // The scheduler (one thread of the odd CTA): units counter, counter + 1, ...
  // until one >= total, which ends the readers' walks.  False: a wait ran out.
  __device__ bool schedule(int32_t* counter, int total, uint64_t timeout_ns, const volatile int* abort) const {
    using namespace ptx;
    int slot = 0;
    uint32_t phase = 0;
    while (true) {
      const int u = atomicAdd(counter, 1);
      if (!mbar_wait(&empty[slot], phase ^ 1u, timeout_ns, abort)) return false;
      unit[slot] = u;
      const uint32_t theirs = mapa_shared(smem_u32(const_cast<int32_t*>(unit) + slot), 0);
      asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(theirs), "r"(u) : "memory");
      mbar_arrive_cluster(mapa_shared(smem_u32(&full[slot]), 0));
      mbar_arrive(&full[slot]);
      if (u >= total) return true;
      if (++slot == kSchedSlots) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
};

// One warp's walk along the scheduled units.
struct PairUnits {
  PairSched sched;
  const int total;
  const volatile int* abort;
  const uint64_t timeout_ns;
  const uint32_t empty_odd;
  int slot = 0;
  uint32_t phase = 0;
  bool ok = true;  // false: a wait ran out

  __device__ PairUnits(const PairSched& s, int units, uint64_t timeout, const volatile int* a)
      : sched(s), total(units), abort(a), timeout_ns(timeout),
        empty_odd(ptx::mapa_shared(ptx::smem_u32(s.empty), 1)) {}

  // the next unit (warp-uniform; a whole warp calls), or -1
  __device__ __forceinline__ int next() {
    using namespace ptx;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&sched.full[slot], phase, timeout_ns, abort))) {
      ok = false;
      return -1;
    }
    const int u = sched.unit[slot];
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_remote(empty_odd + 8u * slot);
    if (++slot == kSchedSlots) {
      slot = 0;
      phase ^= 1u;
    }
    return u < total ? u : -1;
  }
};

}  // namespace moe
