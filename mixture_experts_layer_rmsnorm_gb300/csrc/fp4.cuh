// fp4.cuh -- 4-bit rows (MXFP4, NVFP4) and their grouped product: the layout
// of the scales and the launchers (internal).
//
// Codes: [rows, K / 2] bytes, element 2i in the low nibble of byte i.  Scales:
// 512-byte tiles of 128 rows x 4 blocks of K (a chunk: 128 elements for
// MXFP4's blocks of 32, 64 for NVFP4's blocks of 16), byte r * 16 + 4 * j + b
// for row 32 j + r and block b of the chunk; the tiles of one 128-row tile row
// follow one another along K.  A group's rows start a tile row of their own, so
// that the product finds the scales of its token chunks at row 0 of a tile:
//   equal groups of R rows:  tile row  g ceil(R / 128) + (p - g R) / 128
//   listed groups:           tile row  floor(offsets[g] / 128) + g + (p - offsets[g]) / 128
// (group g + 1 then starts behind the last tile row of group g: with
// offsets[g] = 128 a + r and a count of 128 b + s the last is
// a + g + b + (s > 0) - 1, the next a + b + (r + s >= 128) + g + 1 at least),
// floor(rows / 128) + groups tile rows at most in both cases.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "grouped.cuh"

namespace moe {

enum class Fp4Format : int { kMx = 0, kNv = 1 };

__host__ __device__ constexpr int fp4_block(Fp4Format f) { return f == Fp4Format::kMx ? 32 : 16; }
__host__ __device__ constexpr int fp4_chunk(Fp4Format f) { return 4 * fp4_block(f); }
inline int64_t fp4_tile_rows(int64_t rows, int64_t groups) { return rows / 128 + groups; }

struct Fp4RowsArgs {
  const int32_t* offsets;  // as in GroupedPlanArgs
  const int32_t* counts;
  int G;
  int64_t rows;
  int K;
  int64_t tile_rows;  // capacity of `scales`
  uint8_t* codes;
  uint8_t* scales;
  float* gscale;        // NVFP4: [rows], or [groups] (per_group)
  int per_group;
  const void* src;      // quantise: rows of ld elements of src_type
  void* dst;            // dequantise: rows of ld elements of dst_type
  int64_t ld;
  int type;             // 0 bf16, 1 fp16, 2 fp32
};
cudaError_t launch_fp4_quantize(Fp4Format f, const Fp4RowsArgs& a, cudaStream_t stream);
cudaError_t launch_fp4_dequantize(Fp4Format f, const Fp4RowsArgs& a, cudaStream_t stream);

// The grouped product on 4-bit operands: GroupedGemmArgs as for the 16-bit
// forward (R = K), the scales and NVFP4's fp32 scales beside it.
struct Fp4GemmArgs {
  GroupedGemmArgs g;
  const uint8_t* w_scales;
  const uint8_t* x_scales;
  const float* w_gscale;  // [G]
  const float* x_gscale;  // [rows]
  int w_tile_rows;        // ceil(N / 128)
  int equal;              // equal groups (no offsets): their tile rows
};
int fp4_bn(GroupedPlan plan);
int fp4_tile(GroupedPlan plan);
int fp4_tok_box(GroupedPlan plan);
cudaError_t launch_fp4_gemm(Fp4Format f, GroupedPlan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                            const Fp4GemmArgs& a, int num_sms, cudaStream_t stream);

}  // namespace moe
