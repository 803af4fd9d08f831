// fp8.cuh -- rows and matrices in 8 bits (E4M3 under fp32 scales of 128 elements
// or of 128 x 128) and their grouped products (internal).
//
//   rows      codes [rows, K], scales [rows][lds]: block b of row p at p * lds + b,
//             lds a multiple of 4, since the quantizer writes four at once
//   matrices  codes [G, N, K], scales [G][ceil(N / 128)][ceil(K / 128)]
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "grouped.cuh"

namespace moe {

struct Fp8Args {
  int64_t rows;      // of rows; of all matrices together
  int64_t per;       // rows of a matrix, or 0: rows
  int K;
  uint8_t* codes;
  float* scales;
  int64_t lds;       // rows: see above
  const void* src;   // quantise: rows of ld elements of `type`
  void* dst;         // dequantise
  int64_t ld;
  int type;          // 0 bf16, 1 fp16, 2 fp32
};
cudaError_t launch_fp8_quantize(const Fp8Args& a, cudaStream_t stream);
cudaError_t launch_fp8_dequantize(const Fp8Args& a, cudaStream_t stream);

// A grouped product on 8-bit operands: GroupedGemmArgs as for the 16-bit forward
// and input gradient, and the scales.
struct Fp8GemmArgs {
  GroupedGemmArgs g;
  const float* x_scales;  // of the rows, [rows][ldxs]
  int64_t ldxs;
  const float* w_scales;  // [G][w_rows][w_cols]
  int w_rows, w_cols;     // ceil(N / 128), ceil(K / 128)
};
// Tile plans: stream-K on single CTAs, units of 32 rows; units of 128 rows on single CTAs; of 256 on CTA pairs.
enum class Fp8Plan : int { kSmall, kSingle, kPairs };
int fp8_bn(Fp8Plan plan);    // rows of a unit
int fp8_tile(Fp8Plan plan);  // features of a unit
// tm_x: the rows' codes in boxes of fp8_tok_box(plan) rows; tm_x32: of 32 (unused by the small plan)
int fp8_tok_box(Fp8Plan plan);
cudaError_t launch_fp8_gemm(GroupedOp op, Fp8Plan plan, const CUtensorMap& tm_w, const CUtensorMap& tm_x,
                            const CUtensorMap& tm_x32, const Fp8GemmArgs& a, int num_sms, cudaStream_t stream);

}  // namespace moe
