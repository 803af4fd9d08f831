// k_fp4_gemm.cu -- the grouped product on 4-bit operands:
//   y[p, :] = x[p, :] w_g^T    (p in group g)
// with x and w as E2M1 codes under MXFP4's E8M0 scales per 32 elements
// (tcgen05.mma kind::mxf4) or NVFP4's E4M3 scales per 16 (kind::mxf4nvf4) and
// fp32 scales per row of x and per matrix, applied to the fp32 accumulators.
//
// Mapping, units and work split as in k_grouped_gemm.cu: the weights take the
// MMA's M side, a group's rows its N side.  A stage holds 256 elements of K:
// 128-byte rows of codes and, per operand, the scale tiles of its chunks (two
// for MXFP4, four for NVFP4, 512 bytes per 128 rows).  K may end inside a
// stage: TMA gives zero codes past it, the valid chunks' tiles alone are loaded
// and the valid MMAs alone issued (the quantizer writes zero scales for the
// blocks of a chunk past K, so that a last half MMA adds zeros).
//
// Scales.  The MMA reads them from TMEM: row 32 j + l of a tile in lane l of
// every lane quarter, column j, four bytes = a chunk's four blocks.  Four scale
// warps, one per lane quarter, write each stage's tiles there with tcgen05.st:
// copies by the MMA thread (tcgen05.cp, six or twelve a stage) run in the tensor
// pipe and cost the layer's NVFP4 GEMM a fifth of its rate.  In a CTA pair each
// CTA needs the scales of its own 128 features and of all the unit's rows in its
// own TMEM.  So a stage's scales are loaded on a barrier of their own in each
// CTA, each CTA's scale warps write its TMEM, and all eight signal the even CTA,
// whose thread issues the MMAs.
//
// TMEM of a pair: one accumulator of 256 columns beside 5 x 48 (NVFP4) or
// 6 x 32 (MXFP4) scale columns.  With one accumulator the MMAs of the next unit
// wait for the epilogue to read this one, so the epilogue reads all of its
// columns into registers, rounded and packed in pairs, hands the accumulator back, and
// stores after that.
//
// Few rows a group: bound by HBM (64 rows in 41 of 64 groups, N = 8192, K = 4096,
// MXFP4: 117 us with the rows' quantizer, 0.92 of the measured rate).  Many: at the FP4
// rate a pair would take a stage of 38 KB per SM every 341 cycles, 111 bytes a cycle.  The 16-bit
// kernel's loads reach 68, so the fill of shared memory bounds it, but this one takes 48: what holds it
// there is not isolated.  Ragged groups pay more: a rest unit of 20 rows fills its weight tile and
// boxes of 128 rows like a full one (64 groups of 512, 520, 540 rows, N = K = 4096, NVFP4: 230 to 255, 344 to
// 379, 379 us).  Measured,
// 64 groups of 512 rows, N = K = 4096: NVFP4 230 us (4.8 PFLOP/s), MXFP4 191 us; one group of
// 8192 rows, N = K = 8192: NVFP4 184 to 191 us (5.7 to 6.0 PFLOP/s).  In one comparison five,
// four and three stages took 224, 237 and 269 us (NVFP4; MXFP4's six and five 188 and 193).  The hand-over
// of the single accumulator is not what costs: all columns read into registers before any
// arithmetic (176 registers a thread) 229 us, MXFP4 199; nor is HBM's latency: weights prefetched into L2
// 4, 8 or 15 stages ahead 235, 237, 244 us.  The row scales' second factor (scale_parts) costs 4 us.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "bounded_wait.cuh"
#include "fp4.cuh"
#include "launch_config.cuh"
#include "pair_sched.cuh"
#include "pdl.cuh"
#include "tc_ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kABytes = 128 * 128;  // 128 features x 256 codes

template <Fp4Format F, int BN, int STAGES, int TOKBOX, bool PAIR>
struct Cfg {
  static constexpr int kChunks = F == Fp4Format::kNv ? 4 : 2;  // scale tiles per 128 rows and stage
  static constexpr int kBRows = PAIR ? BN / 2 : BN;
  static constexpr int kBBytes = kBRows * 128;
  static constexpr int kG = BN > 128 ? 2 : 1;  // 128-row scale tiles of a unit's rows
  static constexpr int kSfW = 512 * kChunks, kSfX = 512 * kChunks * kG;
  static constexpr int kStageBytes = (kABytes + kBBytes + kSfW + kSfX + 1023) / 1024 * 1024;
  static constexpr int kAccBufs = PAIR ? 1 : 2;
  static constexpr int kSfCols = 16 + (4 * kChunks * kG + 15) / 16 * 16;  // w scales from +0, x scales from +16
  static constexpr int kTmemNeed = kAccBufs * BN + STAGES * kSfCols;
  static constexpr uint32_t kTmemCols = kTmemNeed <= 128 ? 128 : kTmemNeed <= 256 ? 256 : 512;
  static constexpr int kEpiWarps = PAIR ? 8 : 4;  // two per TMEM lane quarter for the pair's single accumulator
  // the weights' producer, the MMA warp, the epilogue, 4 scale warps, the rows' producer; in pairs the relay
  static constexpr int kRowsWarp = 2 + kEpiWarps + 4, kRelayWarp = PAIR ? kRowsWarp + 1 : -1;
  static constexpr int kThreads = 32 * (kRowsWarp + (PAIR ? 2 : 1));
  static constexpr int kReaders = 2 + kEpiWarps + 4;  // warps of a pair's odd CTA that walk the units
  static constexpr int kBarBytes = 512;
  static constexpr int kTabGroups = kGroupsSmem[PAIR];
  static constexpr int kTabBytes = 3 * (kTabGroups + 1) * 4;
  static constexpr int kGxBytes = F == Fp4Format::kNv ? 2 * 4 * BN * 4 : 0;  // rows' scales and exponents, per epilogue warp
  static constexpr size_t kSmemBytes =
      1024 + static_cast<size_t>(STAGES) * kStageBytes + kBarBytes + kSchedBytes + kTabBytes + kGxBytes + 16;
  static_assert(kBRows % TOKBOX == 0 && BN >= 32 && BN <= 256, "token tile");
  static_assert(4 * kChunks <= 16 && kTmemNeed <= 512, "TMEM columns");
  static_assert((4 * STAGES + 5) * 8 + 8 <= kBarBytes, "barrier area");
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
};

enum : int {
  kWaitSlotFree = 1,
  kWaitAccFree = 2,
  kWaitSlotFull = 3,
  kWaitAccFull = 4,
  kWaitPartials = 5,
  kWaitScales = 7,
  kWaitScaleLoads = 8,
  kWaitUnit = 10
};

// A pair's walk in the form of a stream-K range: whole units.
struct PairWalk {
  PairUnits units;
  int kblocks;
  __device__ __forceinline__ bool next(int& u, int& kb0, int& kb1) {
    u = units.next();
    kb0 = 0;
    kb1 = kblocks;
    return u >= 0;
  }
};
__device__ __forceinline__ bool walk_ok(const PairWalk& w) { return w.units.ok; }
__device__ __forceinline__ bool walk_ok(const GroupedRange&) { return true; }

__device__ __forceinline__ void put4(uint32_t* d, const uint4& v) {
  d[0] = v.x, d[1] = v.y, d[2] = v.z, d[3] = v.w;
}

// gw gx = s p, s returned with p = 1, or where their product lies outside [2^-100, 2^100]
// (it might not be an fp32 value although the result is) p = 2^-120 or 2^120, taken out of the
// factor that is farther from 1: s then lies in fp32's range, or the result is zero.
__device__ __forceinline__ float scale_parts(float gw, float gx, float& p) {
  p = 1.0f;
  const float s = __fmul_rn(gw, gx), big = fmaxf(fabsf(gw), fabsf(gx)), small = fminf(fabsf(gw), fabsf(gx));
  if (fabsf(s) < 0x1p-100f) {
    p = 0x1p-120f;
    return copysignf(__fmul_rn(big, __fmul_rn(small, 0x1p120f)), s);
  }
  if (fabsf(s) > 0x1p100f) {
    p = 0x1p120f;
    return copysignf(__fmul_rn(small, __fmul_rn(big, 0x1p-120f)), s);
  }
  return s;
}

__device__ __forceinline__ uint16_t to16(float v, bool fp16) {
  return fp16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

template <Fp4Format F, int BN, int STAGES, int TOKBOX, bool PAIR>
__global__ void __launch_bounds__(Cfg<F, BN, STAGES, TOKBOX, PAIR>::kThreads, 1)
    fp4_gemm_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_x,
                    const __grid_constant__ Fp4GemmArgs args) {
  using C = Cfg<F, BN, STAGES, TOKBOX, PAIR>;
  const GroupedGemmArgs& a = args.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + STAGES * C::kStageBytes);
  uint64_t* empty = full + STAGES;
  uint64_t* sfld = empty + STAGES;   // a stage's scale tiles are in this CTA's shared memory
  uint64_t* sfull = sfld + STAGES;   // ... and in TMEM (of both CTAs of a pair; the even CTA's barrier)
  uint64_t* tfull = sfull + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const PairSched sched(smem + STAGES * C::kStageBytes + C::kBarBytes);
  int32_t* tab = reinterpret_cast<int32_t*>(smem + STAGES * C::kStageBytes + C::kBarBytes + kSchedBytes);
  float* gx_buf = reinterpret_cast<float*>(
      (reinterpret_cast<uintptr_t>(tab) + C::kTabBytes + 15) & ~uintptr_t(15));

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = PAIR ? cluster_ctarank() : 0u;
  const bool leader = rank == 0;
  const int worker = static_cast<int>(blockIdx.x), workers = static_cast<int>(gridDim.x);  // (single CTAs)

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sfld[s], 1);
      mbar_init(&sfull[s], PAIR ? 8 : 4);  // the scale warps
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], (PAIR ? 2 : 1) * C::kEpiWarps);
    }
    mbar_init(done, 1);
    if (PAIR) sched.init(C::kReaders);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm_w);
    prefetch_tensormap(&tm_x);
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
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  const int total_units = tables.unit_off[a.G];
  const int kblocks = (a.R + 255) / 256;
  const int chunks_k = (a.R + fp4_chunk(F) - 1) / fp4_chunk(F);  // scale tiles along K per tile row
  GroupedUnits units(tables, a.G, 1, BN);  // each warp walks its role's units
  // single CTAs: a stream-K range; pairs: whole units as they are handed out
  auto rg = [&] {
    if constexpr (PAIR)
      return PairWalk{PairUnits(sched, total_units, kWaitTimeoutNs, abort_flag, leader, warp == 0), kblocks};
    else
      return GroupedRange(total_units, kblocks, worker, workers);
  }();
  int u, kb0, kb1;
  auto valid_chunks = [&](int kb) { return min(C::kChunks, chunks_k - kb * C::kChunks); };
  auto n_of = [](int n) { return PAIR ? (n + 31) / 32 * 32 : (n + 15) / 16 * 16; };

  if (warp == 0 || warp == C::kRowsWarp) {
    // ---------------- TMA producers, one warp for the weights and their scales,
    // one for the rows and theirs; one lane issues
    const bool weights = warp == 0, issue = elect_one();
    const uint64_t pol_stream = policy_evict_first(), pol_keep = policy_evict_last();
    const uint32_t full_cl = PAIR ? mapa_shared(smem_u32(full), 0) : 0u;
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      const int feat = PAIR ? un.tile * 256 + static_cast<int>(rank) * 128 : un.tile * 128;
      const int n_mma = n_of(un.n);
      const int half = PAIR ? n_mma / 2 : n_mma;
      const int tok_first = un.tok0 + static_cast<int>(rank) * half;
      const int tok_rows = (half + TOKBOX - 1) / TOKBOX * TOKBOX;
      const uint64_t pol_w = units.chunks > 1 ? pol_keep : pol_stream;
      // scale tile rows: of this CTA's features (past N: a tile row of the
      // same matrix, its products are dropped), of the unit's rows
      const int64_t wt = static_cast<int64_t>(un.g) * args.w_tile_rows + min(feat / 128, args.w_tile_rows - 1);
      const int64_t xt = (args.equal ? static_cast<int64_t>(un.g) * ((args.equal + 127) / 128) : un.start / 128 + un.g) +
                         (un.tok0 - un.start) / 128;
      const int x_tiles = C::kG == 2 && un.n > 128 ? 2 : 1;
      const uint8_t* w_sf = args.w_scales + wt * chunks_k * 512;
      const uint8_t* x_sf = args.x_scales + xt * chunks_k * 512;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[stage], phase ^ 1u, kWaitTimeoutNs, abort_flag))) {
          ok = false;
          break;
        }
        if (issue) {
          uint8_t* sa = smem + stage * C::kStageBytes;
          uint8_t* sb = sa + kABytes;
          uint8_t* sf = sb + C::kBBytes;
          uint64_t* bar = &full[stage];
          const uint32_t bar_cl = full_cl + 8u * stage;
          const uint32_t sf_bytes = 512u * valid_chunks(kb);
          const int sf_at = kb * C::kChunks * 512;
          if (weights) {
            if (leader) mbar_arrive_expect_tx(bar, (PAIR ? 2 : 1) * (kABytes + tok_rows * 128));
            mbar_arrive_expect_tx(&sfld[stage], sf_bytes * (1 + x_tiles));
            bulk_load(sf, w_sf + sf_at, sf_bytes, &sfld[stage], pol_w);
            if (PAIR)
              tma_load_3d_pair(sa, &tm_w, bar_cl, kb * 128, feat, un.g, pol_w);
            else
              tma_load_3d(sa, &tm_w, bar, kb * 128, feat, un.g, pol_w);
          } else {
            for (int h = 0; h < x_tiles; ++h)
              bulk_load(sf + (1 + h) * C::kSfW, x_sf + static_cast<int64_t>(h) * chunks_k * 512 + sf_at, sf_bytes,
                        &sfld[stage], pol_keep);
            for (int r = 0; r < tok_rows; r += TOKBOX) {
              if (PAIR)
                tma_load_2d_pair(sb + r * 128, &tm_x, bar_cl, kb * 128, tok_first + r, pol_keep);
              else
                tma_load_2d(sb + r * 128, &tm_x, bar, kb * 128, tok_first + r, pol_keep);
            }
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    ok = ok && walk_ok(rg);
    if (!ok && issue) raise_timeout(a.err, abort_flag, kKernFp4Gemm, walk_ok(rg) ? kWaitSlotFree : kWaitUnit);
    // every load issued has been used before the CTA exits
    for (int s = 0; s < STAGES; ++s) {
      if (issued <= s) break;
      const uint32_t par = (s < stage) ? phase : (phase ^ 1u);
      const int never = 0;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], par, kWaitTimeoutNs, &never))) break;
    }
  } else if (warp == 1) {
    if (leader) {
      // ---------------- MMA issuer: the whole warp walks the units, one lane issues
      const bool issue = elect_one();
      const uint64_t a0 = sdesc_kmajor_sw128(smem_u32(smem));
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
        const uint32_t n_mma = static_cast<uint32_t>(n_of(un.n));
        // instruction descriptors: MXFP4's MMAs of a chunk take scale bytes 0, 1 and 2, 3
        const uint32_t id0 = F == Fp4Format::kNv ? idesc_nvf4(PAIR ? 256 : 128, n_mma) : idesc_mxf4(PAIR ? 256 : 128, n_mma, 0, 0);
        const uint32_t id2 = idesc_mxf4(PAIR ? 256 : 128, n_mma, 2, 2);
        const uint32_t d_acc = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = kb0; kb < kb1; ++kb) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], phase, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            where = kWaitSlotFull;
            break;
          }
          if (!__all_sync(0xFFFFFFFFu, mbar_wait(&sfull[stage], phase, kWaitTimeoutNs, abort_flag))) {
            ok = false;
            where = kWaitScales;
            break;
          }
          tc_fence_after();
          const uint64_t ad0 = a0 + static_cast<uint64_t>(stage * (C::kStageBytes >> 4)), bd0 = ad0 + (kABytes >> 4);
          const uint32_t sf_w = tmem_base + static_cast<uint32_t>(C::kAccBufs * BN + stage * C::kSfCols);
          const uint32_t sf_x = sf_w + 16;
          const int n_k = min(4, (a.R - kb * 256 + 63) / 64);  // MMAs of K = 64
          if (issue) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= n_k) break;
              const uint32_t accum = k > 0 ? 1u : kb > kb0;
              const uint64_t ad = ad0 + 2 * k, bd = bd0 + 2 * k;  // 32 bytes further
              if constexpr (F == Fp4Format::kNv) {
                if (PAIR)
                  mma_nvf4_ss_pair(d_acc, ad, bd, id0, sf_w + 4 * k, sf_x + 4 * C::kG * k, accum);
                else
                  mma_nvf4_ss(d_acc, ad, bd, id0, sf_w + 4 * k, sf_x + 4 * C::kG * k, accum);
              } else {
                const uint32_t c = static_cast<uint32_t>(k >> 1), id = (k & 1) ? id2 : id0;
                if (PAIR)
                  mma_mxf4_ss_pair(d_acc, ad, bd, id, sf_w + 4 * c, sf_x + 4 * C::kG * c, accum);
                else
                  mma_mxf4_ss(d_acc, ad, bd, id, sf_w + 4 * c, sf_x + 4 * C::kG * c, accum);
              }
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
        if (++acc == C::kAccBufs) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!walk_ok(rg)) where = kWaitUnit;
      ok = ok && walk_ok(rg);
      if (!ok && issue) raise_timeout(a.err, abort_flag, kKernFp4Gemm, where);
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
      if (!sched.schedule(a.next_unit, total_units, kWaitTimeoutNs, abort_flag))
        raise_timeout(a.err, abort_flag, kKernFp4Gemm, kWaitUnit);
    }
  } else if (PAIR && warp == C::kRelayWarp) {
    if (leader && lane == 0 && !sched.relay(total_units, kWaitTimeoutNs, abort_flag))
      raise_timeout(a.err, abort_flag, kKernFp4Gemm, kWaitUnit);
  } else if (warp >= 2 + C::kEpiWarps) {
    // ---------------- scale warps: lane l of a quarter takes the 16 bytes of
    // rows l, 32 + l, 64 + l, 96 + l of each tile (its four TMEM columns)
    const uint32_t quarter = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t sfull_cl = PAIR ? mapa_shared(smem_u32(sfull), 0) : 0u;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      // a unit of 32 rows may start at row 32, 64 or 96 of its tile: column j
      // of its words then belongs at column 0
      const int j0 = BN < 128 ? ((un.tok0 - un.start) & 127) >> 5 : 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        const bool got = mbar_wait(&sfld[stage], phase, kWaitTimeoutNs, abort_flag);
        if (!__all_sync(0xFFFFFFFFu, got)) {  // warp-uniform: tcgen05.st needs every lane
          ok = false;
          break;
        }
        const uint8_t* sf = smem + stage * C::kStageBytes + kABytes + C::kBBytes + lane * 16;
        const uint32_t cols = tmem_base + static_cast<uint32_t>(C::kAccBufs * BN + stage * C::kSfCols) + quarter;
        // all tiles of the stage (past K or the unit's rows: whatever the stage
        // held, which no MMA reads) with one store per operand
        uint32_t w[4 * C::kChunks], x[4 * C::kChunks * C::kG];
#pragma unroll
        for (int c = 0; c < C::kChunks; ++c) {
          put4(w + 4 * c, *reinterpret_cast<const uint4*>(sf + 512 * c));
#pragma unroll
          for (int h = 0; h < C::kG; ++h)
            put4(x + 4 * (c * C::kG + h), *reinterpret_cast<const uint4*>(sf + C::kSfW + h * C::kSfW + 512 * c));
        }
        if (BN < 128) {
#pragma unroll
          for (int c = 0; c < C::kChunks; ++c)
            x[4 * c] = j0 == 0 ? x[4 * c] : j0 == 1 ? x[4 * c + 1] : j0 == 2 ? x[4 * c + 2] : x[4 * c + 3];
        }
        tmem_st_32x32b(cols, w);
        tmem_st_32x32b(cols + 16, x);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote(sfull_cl + 8u * stage);
          else
            mbar_arrive(&sfull[stage]);
        }
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    ok = ok && walk_ok(rg);
    if (!ok && lane == 0) raise_timeout(a.err, abort_flag, kKernFp4Gemm, walk_ok(rg) ? kWaitScaleLoads : kWaitUnit);
  } else {
    // ---------------- epilogue: warps 2.., TMEM lane quarter = warp % 4; two
    // warps of a quarter take half of the columns each
    const int q = warp & 3;
    const int row = q * 32 + lane;
    int acc = 0, where = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    const uint32_t tempty_cl = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
    constexpr int kCols = BN * 4 / C::kEpiWarps;  // columns per warp
    const int col0 = (warp - 2) / 4 * kCols;
    float *gx = gx_buf + (warp - 2) * kCols, *gp = gx + 4 * BN;  // columns' scales, in two factors
    bool wide = false;  // (warp-uniform) some column's second factor is not 1
    while (ok && rg.next(u, kb0, kb1)) {
      const GroupedUnit un = units.at(u);
      const int feat0 = PAIR ? un.tile * 256 + static_cast<int>(rank) * 128 : un.tile * 128;
      const bool fp16 = a.fp16 != 0, mine = feat0 + row < a.F;
      uint16_t* out = static_cast<uint16_t*>(a.out) + static_cast<int64_t>(un.tok0) * a.ldo + feat0 + row;
      if (F == Fp4Format::kNv) {  // the rows' fp32 scales times the matrix's, read while the MMAs run
        const float gw = __ldg(args.w_gscale + un.g);
        bool other = false;
        __syncwarp();
        for (int c = lane; c < kCols; c += 32) {
          float p = 1.0f;
          gx[c] = col0 + c < un.n ? scale_parts(gw, __ldcg(args.x_gscale + un.tok0 + col0 + c), p) : 0.0f;
          gp[c] = p;
          other |= p != 1.0f;
        }
        wide = __any_sync(0xFFFFFFFFu, other);
        __syncwarp();
      }
      const bool got = mbar_wait(&tfull[acc], acc_phase, kWaitTimeoutNs, abort_flag);
      if (!__all_sync(0xFFFFFFFFu, got)) {
        ok = false;
        where = kWaitAccFull;
        break;
      }
      tc_fence_after();
      const uint32_t t_row = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc * BN);
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (PAIR)
            mbar_arrive_remote(tempty_cl + 8u * acc);
          else
            mbar_arrive(&tempty[acc]);
        }
      };
      if constexpr (PAIR) {
        const int odd = lane & 1;
        uint32_t packed[kCols / 2];
        // columns a load: NVFP4, whose scales take registers too, would spill with 32 (256 groups of 64
        // rows, N = 1536, K = 256: 132 instead of 122 us); MXFP4 is slower with 16 (102 instead of 89 us)
        constexpr int kLoad = F == Fp4Format::kNv ? 16 : 32;
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += kLoad) {
          if (col0 + c0 < un.n) {
            uint32_t r[kLoad];
            __syncwarp();  // tcgen05.ld is warp-aligned
            if constexpr (kLoad == 16)
              tmem_ld_32x32b_x16(t_row + col0 + c0, r);
            else
              tmem_ld_32x32b_x32(t_row + col0 + c0, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < kLoad; j += 4) {
              float4 v = make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]),
                                     __uint_as_float(r[j + 3]));
              if (F == Fp4Format::kNv) {
                const float4 s = *reinterpret_cast<const float4*>(gx + c0 + j);
                v = make_float4(__fmul_rn(v.x, s.x), __fmul_rn(v.y, s.y), __fmul_rn(v.z, s.z), __fmul_rn(v.w, s.w));
                if (wide) {
                  const float4 p = *reinterpret_cast<const float4*>(gp + c0 + j);
                  v = make_float4(__fmul_rn(v.x, p.x), __fmul_rn(v.y, p.y), __fmul_rn(v.z, p.z), __fmul_rn(v.w, p.w));
                }
              }
              packed[(c0 + j) / 2] = pack16(v.x, v.y, fp16);
              packed[(c0 + j) / 2 + 1] = pack16(v.z, v.w, fp16);
            }
          }
        }
        release();
        // this lane's two features, of its row of each pair of rows (F is even: a pair of lanes alike)
        uint16_t* o = out + static_cast<int64_t>(col0 + odd) * a.ldo - odd;
#pragma unroll
        for (int c = 0; c < kCols; c += 2) {
          const uint32_t v = trade_rows(packed[c / 2]);
          if (mine && col0 + c + odd < un.n) *reinterpret_cast<uint32_t*>(o + static_cast<int64_t>(c) * a.ldo) = v;
        }
      } else if (kb0 > 0) {
        // a later part of a unit that an earlier CTA started: hand over the partial sums
        float* slot = a.partials + static_cast<int64_t>(worker) * BN * 128;
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
        release();
      } else {
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
            const float* slot = a.partials + static_cast<int64_t>(c) * BN * 128;
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] += __ldcg(slot + (c0 + j) * 128 + row);
          }
          if (mine) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              if (c0 + j < un.n) {
                if (F == Fp4Format::kNv) v[j] = __fmul_rn(__fmul_rn(v[j], gx[c0 + j]), gp[c0 + j]);
                out[static_cast<int64_t>(c0 + j) * a.ldo] = to16(v[j], fp16);
              }
          }
        }
        if (ok) release();
      }
      if (!ok) break;
      if (++acc == C::kAccBufs) {
        acc = 0;
        acc_phase ^= 1u;
      }
    }
    if (!walk_ok(rg)) where = kWaitUnit;
    ok = ok && walk_ok(rg);
    if (!ok && lane == 0) raise_timeout(a.err, abort_flag, kKernFp4Gemm, where);
  }

  __syncthreads();
  if (PAIR) cluster_sync();  // a pair keeps both CTAs until both are done
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    if (PAIR)
      tmem_dealloc_pair(tmem_base, C::kTmemCols);
    else
      tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <Fp4Format F, int BN, int STAGES, int TOKBOX, bool PAIR>
cudaError_t launch_gemm(const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& a, int num_sms,
                        cudaStream_t stream) {
  using C = Cfg<F, BN, STAGES, TOKBOX, PAIR>;
  static PerDevice config;
  auto kernel = fp4_gemm_kernel<F, BN, STAGES, TOKBOX, PAIR>;
  if constexpr (PAIR) return launch_pairs(kernel, config, C::kThreads, C::kSmemBytes, stream, tw, tx, a);
  return launch_ctas(kernel, config, num_sms < kMaxGemmCtas ? num_sms : kMaxGemmCtas, C::kThreads, C::kSmemBytes, stream,
                     tw, tx, a);
}

constexpr int kBn[2] = {32, 256}, kTile[2] = {128, 256}, kTokBox[2] = {16, 128};

template <Fp4Format F>
cudaError_t launch_plan(GroupedPlan plan, const CUtensorMap& tw, const CUtensorMap& tx, const Fp4GemmArgs& a,
                        int num_sms, cudaStream_t stream) {
  constexpr int small = F == Fp4Format::kNv ? 9 : 9, large = F == Fp4Format::kNv ? 5 : 6;  // stages
  if (plan == GroupedPlan::kSmall) return launch_gemm<F, kBn[0], small, kTokBox[0], false>(tw, tx, a, num_sms, stream);
  return launch_gemm<F, kBn[1], large, kTokBox[1], true>(tw, tx, a, num_sms, stream);
}

}  // namespace

int fp4_bn(GroupedPlan plan) { return kBn[static_cast<int>(plan)]; }
int fp4_tile(GroupedPlan plan) { return kTile[static_cast<int>(plan)]; }
int fp4_tok_box(GroupedPlan plan) { return kTokBox[static_cast<int>(plan)]; }

cudaError_t launch_fp4_gemm(Fp4Format f, GroupedPlan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                            const Fp4GemmArgs& a, int num_sms, cudaStream_t stream) {
  return f == Fp4Format::kMx ? launch_plan<Fp4Format::kMx>(plan, tm_w, tm_x, a, num_sms, stream)
                             : launch_plan<Fp4Format::kNv>(plan, tm_w, tm_x, a, num_sms, stream);
}

}  // namespace moe
