// grouped_api.cu -- the C ABI of the grouped products (16-bit and 4-bit), of
// rows in 4 bits and of SwiGLU on separate rows: argument checks, workspace
// layout, tensor maps, launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstring>

#include "../../include/moe.h"
#include "fp4.cuh"
#include "grouped.cuh"
#include "grouped_elementwise.cuh"
#include "tensor_map.h"

namespace {

using moe::GroupedOp;
using moe::GroupedPlan;

constexpr int64_t kMaxDim = int64_t(1) << 20;         // N, K
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;  // 32-bit row coordinates, a token box past the end
// Weight gradient into 16 bits: the fp32 additions of a group's segments (2^26 / 3840, 2^-24 each) stay
// below a third of the half step that bf16's rounding takes.
constexpr int64_t kMaxRows16 = int64_t(1) << 26;
constexpr int64_t kMaxLd = int64_t(1) << 36;          // elements: row strides within the tensor maps' 2^40 bytes

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

struct Layout {
  size_t start, count, unit_off, flags, maps, partials, total;
};

constexpr int kFlagInts = moe::kMaxGemmCtas * 4;

// wgrad_rows: rows of a weight gradient into 16 bits, whose long groups need room for their sums; else 0
Layout make_layout(int G, int64_t wgrad_rows = 0) {
  Layout L{};
  size_t off = 64;  // the error word
  auto take = [&](size_t bytes) {
    off = align_up(off, 256);
    const size_t r = off;
    off += bytes;
    return r;
  };
  L.start = take(static_cast<size_t>(G) * 4);
  L.count = take(static_cast<size_t>(G) * 4);
  L.unit_off = take(static_cast<size_t>(G + 1) * 4);
  L.flags = take(static_cast<size_t>(kFlagInts) * 4);
  L.maps = take(static_cast<size_t>(G) * 2 * sizeof(CUtensorMap));
  L.partials = take(wgrad_rows > moe::kWgradSegment16 ? moe::grouped_wgrad_sum_bytes() : moe::grouped_partial_bytes());
  L.total = align_up(off, 256);
  return L;
}

template <typename T>
T* at(void* ws, size_t off) {
  return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
}

moe_status check_shape(const moe_grouped_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->groups <= 0 || s->N <= 0 || s->K <= 0 || s->rows < 0) return MOE_ERR_INVALID_ARG;
  if (s->type != MOE_TYPE_BF16 && s->type != MOE_TYPE_FP16) return MOE_ERR_INVALID_ARG;
  if (s->groups > moe::kGroupsMax || s->N % 8 != 0 || s->K % 8 != 0 || s->N > kMaxDim || s->K > kMaxDim ||
      s->rows > kMaxRows)
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A row matrix of `width` elements: null only without rows.
moe_status check_rows(const void* p, int64_t rows, int64_t ld, int64_t width) {
  if (ld < width) return MOE_ERR_INVALID_ARG;
  if (ld % 8 != 0 || ld > kMaxLd) return MOE_ERR_UNSUPPORTED;
  if (rows > 0 && (!p || !aligned(p, 16))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_call(const moe_grouped_shape* s, const int32_t* offsets, const int32_t* counts, void* ws,
                      size_t ws_bytes, int64_t wgrad_rows = 0) {
  if (!offsets && s->rows % s->groups != 0) return MOE_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || !aligned(counts, 4)) return MOE_ERR_INVALID_ARG;
  if (!ws || !aligned(ws, 256)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < make_layout(s->groups, wgrad_rows).total) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// Element types of the maps: 2-byte operands, or the weight gradient's output.
CUtensorMapDataType map_type(int type) {
  return type == MOE_TYPE_FP32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
         : type == MOE_TYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
}

// Rows of a token matrix: boxes of 64 columns x box_rows, 128-byte swizzle.
bool make_rows_map(CUtensorMap* m, int type, const void* base, int64_t width, int64_t rows, int64_t ld,
                   uint32_t box_rows) {
  auto fn = moe::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * 2};
  cuuint32_t box[2] = {64, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, map_type(type), 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [G, N, K] matrices: boxes of 128 bytes of K x box_rows of N.
bool make_matrix_map(CUtensorMap* m, int type, const void* base, int64_t G, int64_t N, int64_t K, uint32_t box_rows) {
  auto fn = moe::encode_fn();
  if (!fn) return false;
  const cuuint64_t size = type == MOE_TYPE_FP32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(G)};
  cuuint64_t strides[2] = {dims[0] * size, dims[0] * dims[1] * size};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(128 / size), box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, map_type(type), 3, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

moe::GroupedGemmArgs gemm_args(const moe_grouped_shape* s, const Layout& L, void* ws) {
  moe::GroupedGemmArgs a{};
  a.start = at<int32_t>(ws, L.start);
  a.count = at<int32_t>(ws, L.count);
  a.unit_off = at<int32_t>(ws, L.unit_off);
  a.err = at<int32_t>(ws, 0);
  a.partials = at<float>(ws, L.partials);
  a.flags = at<int32_t>(ws, L.flags);
  a.next_unit = a.flags;  // (a plan uses one or the other)
  a.G = s->groups;
  a.tiles_n = 1;
  a.fp16 = s->type == MOE_TYPE_FP16;
  return a;
}

moe::GroupedPlanArgs plan_args(const moe_grouped_shape* s, const Layout& L, void* ws, const int32_t* offsets,
                               const int32_t* counts) {
  moe::GroupedPlanArgs p{};
  p.offsets = offsets;
  p.counts = counts;
  p.G = s->groups;
  p.rows = s->rows;
  p.start = at<int32_t>(ws, L.start);
  p.count = at<int32_t>(ws, L.count);
  p.unit_off = at<int32_t>(ws, L.unit_off);
  p.err = at<int32_t>(ws, 0);
  p.flags = at<int32_t>(ws, L.flags);
  p.n_flags = kFlagInts;
  return p;
}

// More work units than an int counts, in the smallest ones.
bool too_many_units(const moe_grouped_shape* s, int F) {
  return (s->rows / 32 + s->groups) * ((F + 127) / 128) >= (int64_t(1) << 31);
}

// The tile plan follows the rows a group can be expected to hold, the mean: few, the product
// is bound by streaming the weights once (32-row units on single CTAs, stream-K), else by reuse
// of the weight tiles (units of up to 512 rows, 4 bits 256, on CTA pairs).
//   up to 16 rows: single CTAs, also because fewer groups than all may hold them
//   up to 24 (of ragged groups few are longer than 32 rows then): single CTAs where whole units
//   leave pairs idle for over 5% of their waves, or where a 4-bit unit is short (K <= 2048)
//   more: pairs
// The host does not see the lists: where a few of many groups hold nearly all rows, the mean
// chooses single CTAs, and groups of 64 rows and more take two to three times as long as they need.
//   us on pairs / single CTAs                       16 rows    24         64
//   16 bits, 16 groups, N = K = 4096 (3.4 waves)    91 / 83    102 / 85
//   16 bits, 64 groups, N 8192, K 4096 (26.9)       616 / 628  627 / 647  649 / 1438
//   NVFP4, 16 groups, N = K = 4096                  37 / 32    37 / 34
//   NVFP4, 64 groups, N 8192, K 4096                187 / 187  189 / 197  207 / 308
//   NVFP4, 256 groups, N 1536, K 2048               106 / 78   107 / 81   125 / 137
GroupedPlan choose_plan(const moe_grouped_shape* s, int F, int sms, bool fp4) {
  if (s->rows <= int64_t(16) * s->groups) return GroupedPlan::kSmall;
  if (s->rows > int64_t(24) * s->groups) return GroupedPlan::kLarge;
  const int tile = moe::grouped_tile(GroupedPlan::kLarge);
  const int64_t units = int64_t(s->groups) * ((F + tile - 1) / tile), pairs = sms / 2 > 0 ? sms / 2 : 1;
  const bool idle = (units + pairs - 1) / pairs * pairs * 20 > units * 21;
  return idle || (fp4 && s->K <= 2048) ? GroupedPlan::kSmall : GroupedPlan::kLarge;
}

// forward (F = N features, R = K) and input gradient (F = K, R = N)
moe_status rows_product(GroupedOp op, const moe_grouped_shape* s, const void* in, int64_t ldin, const void* w,
                        const int32_t* offsets, const int32_t* counts, void* out, int64_t ldout, void* ws,
                        size_t ws_bytes, moe_stream_t stream) {
  moe_status st = check_shape(s);
  if (st != MOE_OK) return st;
  const int F = op == GroupedOp::kForward ? s->N : s->K, R = op == GroupedOp::kForward ? s->K : s->N;
  if ((st = check_rows(in, s->rows, ldin, R)) != MOE_OK) return st;
  if ((st = check_rows(out, s->rows, ldout, F)) != MOE_OK) return st;
  if (!w || !aligned(w, 16)) return MOE_ERR_INVALID_ARG;
  if ((st = check_call(s, offsets, counts, ws, ws_bytes)) != MOE_OK) return st;
  if (too_many_units(s, F)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;
  const int sms = num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const GroupedPlan plan = choose_plan(s, F, sms, false);
  const int tile = moe::grouped_tile(plan), tiles = (F + tile - 1) / tile;
  const int bn = moe::grouped_bn(plan, s->rows, s->groups, tiles, sms);
  CUtensorMap tw, tx, tx32;
  if (!make_matrix_map(&tw, s->type, w, s->groups, s->N, s->K, op == GroupedOp::kForward ? 128 : 64) ||
      !make_rows_map(&tx, s->type, in, R, s->rows, ldin, static_cast<uint32_t>(moe::grouped_tok_box(plan))) ||
      (plan == GroupedPlan::kLarge && !make_rows_map(&tx32, s->type, in, R, s->rows, ldin, 32)))
    return MOE_ERR_CUDA;
  const Layout L = make_layout(s->groups);
  moe::GroupedPlanArgs p = plan_args(s, L, ws, offsets, counts);
  p.bn = bn;
  p.tiles = tiles;
  moe::GroupedGemmArgs a = gemm_args(s, L, ws);
  a.out = out;
  a.ldo = ldout;
  a.F = F;
  a.R = R;
  a.tiles = tiles;
  a.bn = bn;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (moe::launch_grouped_plan(p, tx, tx, cs) != cudaSuccess ||
      moe::launch_grouped_gemm(op, plan, tw, tx, plan == GroupedPlan::kLarge ? tx32 : tx, a, sms, cs) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status swiglu_check(int32_t type, int64_t rows, int32_t I) {
  if ((type != MOE_TYPE_BF16 && type != MOE_TYPE_FP16) || rows < 0 || I <= 0) return MOE_ERR_INVALID_ARG;
  if (I % 8 != 0 || I > kMaxDim || rows > kMaxRows || rows * (I / 8) >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// ---- 4 bits

moe_status check_fp4(const moe_fp4_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->format != MOE_FORMAT_MXFP4 && s->format != MOE_FORMAT_NVFP4) return MOE_ERR_INVALID_ARG;
  if (s->groups <= 0 || s->K <= 0 || s->rows < 0) return MOE_ERR_INVALID_ARG;
  // K: 16-byte rows of codes for TMA, whole blocks
  if (s->groups > moe::kGroupsMax || s->K % 32 != 0 || s->K > kMaxDim || s->rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe::Fp4Format format_of(int32_t f) { return f == MOE_FORMAT_MXFP4 ? moe::Fp4Format::kMx : moe::Fp4Format::kNv; }

size_t scale_bytes(moe::Fp4Format f, int64_t tile_rows, int64_t K) {
  return static_cast<size_t>(tile_rows) * static_cast<size_t>((K + moe::fp4_chunk(f) - 1) / moe::fp4_chunk(f)) * 512;
}

moe_status fp4_rows(const moe_fp4_shape* s, int32_t type, const void* rows, int64_t ld, const int32_t* offsets,
                    const int32_t* counts, const uint8_t* codes, const uint8_t* scales, const float* gscale,
                    int32_t gscale_per, moe::Fp4RowsArgs* out) {
  moe_status st = check_fp4(s);
  if (st != MOE_OK) return st;
  if (type != MOE_TYPE_BF16 && type != MOE_TYPE_FP16 && type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if ((st = check_rows(rows, s->rows, ld, s->K)) != MOE_OK) return st;
  if (!offsets && s->rows % s->groups != 0) return MOE_ERR_INVALID_ARG;
  if (!aligned(offsets, 4) || !aligned(counts, 4)) return MOE_ERR_INVALID_ARG;
  const bool nv = s->format == MOE_FORMAT_NVFP4;
  if (gscale_per != MOE_SCALE_PER_ROW && gscale_per != MOE_SCALE_PER_GROUP) return MOE_ERR_INVALID_ARG;
  if (s->rows > 0 && (!codes || !aligned(codes, 16) || !scales || !aligned(scales, 16))) return MOE_ERR_INVALID_ARG;
  if (s->rows > 0 && nv && (!gscale || !aligned(gscale, 4))) return MOE_ERR_INVALID_ARG;
  moe::Fp4RowsArgs a{};
  a.offsets = offsets;
  a.counts = counts;
  a.G = s->groups;
  a.rows = s->rows;
  a.K = s->K;
  a.tile_rows = moe::fp4_tile_rows(s->rows, s->groups);
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.gscale = const_cast<float*>(gscale);
  a.per_group = gscale_per == MOE_SCALE_PER_GROUP;
  a.ld = ld;
  a.type = type;
  *out = a;
  return MOE_OK;
}

// Code rows: boxes of 128 bytes x box_rows, 128-byte swizzle; matrices [G, N, K / 2] or rows (G = 0).
bool make_codes_map(CUtensorMap* m, const void* base, int64_t K, int64_t N, int64_t G, uint32_t box_rows) {
  auto fn = moe::encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(G)};
  cuuint64_t strides[2] = {dims[0], dims[0] * dims[1]};
  cuuint32_t box[3] = {128, box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, G > 0 ? 3 : 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" {

moe_status moe_grouped_workspace_size(const moe_grouped_shape* shape, size_t* bytes) {
  const moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = make_layout(shape->groups, shape->rows).total;
  return MOE_OK;
}

moe_status moe_grouped_gemm(const moe_grouped_shape* shape, const void* x, int64_t ldx, const void* w,
                            const int32_t* offsets, const int32_t* counts, void* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, moe_stream_t stream) {
  return rows_product(GroupedOp::kForward, shape, x, ldx, w, offsets, counts, y, ldy, workspace, workspace_bytes,
                      stream);
}

moe_status moe_grouped_gemm_dgrad(const moe_grouped_shape* shape, const void* dy, int64_t lddy, const void* w,
                                  const int32_t* offsets, const int32_t* counts, void* dx, int64_t lddx,
                                  void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  return rows_product(GroupedOp::kDgrad, shape, dy, lddy, w, offsets, counts, dx, lddx, workspace, workspace_bytes,
                      stream);
}

moe_status moe_grouped_gemm_wgrad(const moe_grouped_shape* shape, const void* dy, int64_t lddy, const void* x,
                                  int64_t ldx, const int32_t* offsets, const int32_t* counts, void* dw,
                                  int32_t dw_type, int32_t accumulate, void* workspace, size_t workspace_bytes,
                                  moe_stream_t stream) {
  moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  const moe_grouped_shape* s = shape;
  if ((st = check_rows(dy, s->rows, lddy, s->N)) != MOE_OK) return st;
  if ((st = check_rows(x, s->rows, ldx, s->K)) != MOE_OK) return st;
  if (!dw || !aligned(dw, 16)) return MOE_ERR_INVALID_ARG;
  if (dw_type != s->type && dw_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (accumulate && dw_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  const int64_t rows16 = dw_type != MOE_TYPE_FP32 ? s->rows : 0;
  if ((st = check_call(s, offsets, counts, workspace, workspace_bytes, rows16)) != MOE_OK) return st;
  const int tile = moe::kWgradTile;
  const int64_t tiles_m = (s->N + tile - 1) / tile, tiles_n = (s->K + tile - 1) / tile;
  if (tiles_m * tiles_n * s->groups >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (rows16 > kMaxRows16) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0 && accumulate) return MOE_OK;
  // no rows: every group is empty and dw becomes zero; nothing is loaded through the row maps
  const int64_t map_rows = s->rows > 0 ? s->rows : 1;
  CUtensorMap tdy, tx, tdw;
  if (!make_rows_map(&tdy, s->type, s->rows > 0 ? dy : dw, s->N, map_rows, lddy, 64) ||
      !make_rows_map(&tx, s->type, s->rows > 0 ? x : dw, s->K, map_rows, ldx, 64) ||
      !make_matrix_map(&tdw, dw_type, dw, s->groups, s->N, s->K, 32))
    return MOE_ERR_CUDA;
  const Layout L = make_layout(s->groups, rows16);
  moe::GroupedPlanArgs p = plan_args(s, L, workspace, offsets, counts);
  p.bn = 0;
  p.tiles = static_cast<int>(tiles_m * tiles_n);
  p.skip_empty = accumulate != 0;
  p.n_flags = 1;
  p.maps = at<CUtensorMap>(workspace, L.maps);
  moe::GroupedGemmArgs a = gemm_args(s, L, workspace);
  a.maps = p.maps;
  a.F = s->N;
  a.C = s->K;
  a.tiles = p.tiles;
  a.tiles_n = static_cast<int>(tiles_n);
  a.out_fp32 = dw_type == MOE_TYPE_FP32;
  a.accumulate = accumulate != 0;
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (moe::launch_grouped_plan(p, tdy, tx, cs) != cudaSuccess || moe::launch_grouped_wgrad(tdw, a, cs) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status moe_swiglu(int32_t type, int64_t rows, int32_t I, const void* h, int64_t ldh, void* act, int64_t ldact,
                      moe_stream_t stream) {
  moe_status st = swiglu_check(type, rows, I);
  if (st != MOE_OK) return st;
  if ((st = check_rows(h, rows, ldh, 2 * static_cast<int64_t>(I))) != MOE_OK) return st;
  if ((st = check_rows(act, rows, ldact, I)) != MOE_OK) return st;
  if (rows == 0) return MOE_OK;
  return moe::launch_swiglu(type == MOE_TYPE_FP16, h, ldh, act, ldact, rows, I,
                            reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_swiglu_grad(int32_t type, int64_t rows, int32_t I, const void* h, int64_t ldh, const void* dact,
                           int64_t lddact, void* dh, int64_t lddh, moe_stream_t stream) {
  moe_status st = swiglu_check(type, rows, I);
  if (st != MOE_OK) return st;
  if ((st = check_rows(h, rows, ldh, 2 * static_cast<int64_t>(I))) != MOE_OK) return st;
  if ((st = check_rows(dact, rows, lddact, I)) != MOE_OK) return st;
  if ((st = check_rows(dh, rows, lddh, 2 * static_cast<int64_t>(I))) != MOE_OK) return st;
  if (rows > 1 && dh == h && lddh != ldh) return MOE_ERR_INVALID_ARG;  // rows of one over rows of the other
  if (rows == 0) return MOE_OK;
  return moe::launch_swiglu_grad(type == MOE_TYPE_FP16, h, ldh, dact, lddact, dh, lddh, rows, I,
                                 reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_fp4_sizes(const moe_fp4_shape* shape, size_t* codes, size_t* scales) {
  const moe_status st = check_fp4(shape);
  if (st != MOE_OK) return st;
  if (!codes || !scales) return MOE_ERR_INVALID_ARG;
  *codes = static_cast<size_t>(shape->rows) * (shape->K / 2);
  *scales = scale_bytes(format_of(shape->format), moe::fp4_tile_rows(shape->rows, shape->groups), shape->K);
  return MOE_OK;
}

moe_status moe_fp4_quantize(const moe_fp4_shape* shape, int32_t src_type, const void* src, int64_t ldsrc,
                            const int32_t* offsets, const int32_t* counts, uint8_t* codes, uint8_t* scales,
                            float* gscale, int32_t gscale_per, moe_stream_t stream) {
  moe::Fp4RowsArgs a;
  const moe_status st =
      fp4_rows(shape, src_type, src, ldsrc, offsets, counts, codes, scales, gscale, gscale_per, &a);
  if (st != MOE_OK || shape->rows == 0) return st;
  a.src = src;
  return moe::launch_fp4_quantize(format_of(shape->format), a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_fp4_dequantize(const moe_fp4_shape* shape, const uint8_t* codes, const uint8_t* scales,
                              const float* gscale, int32_t gscale_per, const int32_t* offsets, const int32_t* counts,
                              int32_t dst_type, void* dst, int64_t lddst, moe_stream_t stream) {
  moe::Fp4RowsArgs a;
  const moe_status st =
      fp4_rows(shape, dst_type, dst, lddst, offsets, counts, codes, scales, gscale, gscale_per, &a);
  if (st != MOE_OK || shape->rows == 0) return st;
  a.dst = dst;
  return moe::launch_fp4_dequantize(format_of(shape->format), a, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_fp4_gemm(const moe_grouped_shape* shape, int32_t format, const uint8_t* x_codes,
                        const uint8_t* x_scales, const float* x_gscale, const uint8_t* w_codes,
                        const uint8_t* w_scales, const float* w_gscale, const int32_t* offsets, const int32_t* counts,
                        void* y, int64_t ldy, void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  moe_status st = check_shape(shape);
  if (st != MOE_OK) return st;
  const moe_grouped_shape* s = shape;
  if (format != MOE_FORMAT_MXFP4 && format != MOE_FORMAT_NVFP4) return MOE_ERR_INVALID_ARG;
  if (s->K % 32 != 0) return MOE_ERR_UNSUPPORTED;
  if ((st = check_rows(y, s->rows, ldy, s->N)) != MOE_OK) return st;
  const bool nv = format == MOE_FORMAT_NVFP4;
  if (s->rows > 0 && (!x_codes || !aligned(x_codes, 16) || !x_scales || !aligned(x_scales, 16)))
    return MOE_ERR_INVALID_ARG;
  if (!w_codes || !aligned(w_codes, 16) || !w_scales || !aligned(w_scales, 16)) return MOE_ERR_INVALID_ARG;
  if (nv && ((s->rows > 0 && (!x_gscale || !aligned(x_gscale, 4))) || !w_gscale || !aligned(w_gscale, 4)))
    return MOE_ERR_INVALID_ARG;
  if ((st = check_call(s, offsets, counts, workspace, workspace_bytes)) != MOE_OK) return st;
  if (too_many_units(s, s->N)) return MOE_ERR_UNSUPPORTED;
  if (s->rows == 0) return MOE_OK;
  const int sms = num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const GroupedPlan plan = choose_plan(s, s->N, sms, true);
  const int bn = moe::fp4_bn(plan), tile = moe::fp4_tile(plan);
  const int tiles = (s->N + tile - 1) / tile;
  CUtensorMap tw, tx;
  if (!make_codes_map(&tw, w_codes, s->K, s->N, s->groups, 128) ||
      !make_codes_map(&tx, x_codes, s->K, s->rows, 0, static_cast<uint32_t>(moe::fp4_tok_box(plan))))
    return MOE_ERR_CUDA;
  const Layout L = make_layout(s->groups);
  moe::GroupedPlanArgs p = plan_args(s, L, workspace, offsets, counts);
  p.bn = bn;
  p.tiles = tiles;
  moe::Fp4GemmArgs a{};
  a.g = gemm_args(s, L, workspace);
  a.g.out = y;
  a.g.ldo = ldy;
  a.g.F = s->N;
  a.g.R = s->K;
  a.g.tiles = tiles;
  a.w_scales = w_scales;
  a.x_scales = x_scales;
  a.w_gscale = w_gscale;
  a.x_gscale = x_gscale;
  a.w_tile_rows = (s->N + 127) / 128;
  a.equal = offsets ? 0 : static_cast<int>(s->rows / s->groups);
  const cudaStream_t cs = reinterpret_cast<cudaStream_t>(stream);
  if (moe::launch_grouped_plan(p, tx, tx, cs) != cudaSuccess ||
      moe::launch_fp4_gemm(format_of(format), plan, tw, tx, a, sms, cs) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

}  // extern "C"
