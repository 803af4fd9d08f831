// train_api.cu -- the C ABI of the norms of rows with their gradients, and of the
// gradients' norm and clipping: argument checks, launches.
#include <cuda_runtime.h>

#include <cmath>
#include <memory>
#include <new>

#include "../../include/moe.h"
#include "grad_clip.cuh"
#include "row_norm.cuh"

namespace {

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 512;
constexpr int64_t kMaxLd = int64_t(1) << 36;
constexpr int64_t kMaxElements = int64_t(1) << 40;  // of a tensor; chunks of a launch then fit 32 bits

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_FP16 || t == MOE_TYPE_FP32; }

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

moe_status check_norm(const moe_norm_shape* s) {
  if (!s) return MOE_ERR_INVALID_ARG;
  if (s->kind != MOE_NORM_RMS && s->kind != MOE_NORM_LAYER) return MOE_ERR_INVALID_ARG;
  if (!is_type(s->type) || (s->weight_type != s->type && s->weight_type != MOE_TYPE_FP32)) return MOE_ERR_INVALID_ARG;
  if (s->H <= 0 || s->rows < 0 || !(s->eps >= 0.0f) || !std::isfinite(s->eps)) return MOE_ERR_INVALID_ARG;
  if (s->H % 8 != 0 || s->H > moe::kNormMaxH || s->rows > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A row matrix: null only without rows.
moe_status check_rows(const void* p, const moe_norm_shape* s, int64_t ld) {
  if (ld < s->H) return MOE_ERR_INVALID_ARG;
  if (ld % 8 != 0 || ld > kMaxLd) return MOE_ERR_UNSUPPORTED;
  if (s->rows > 0 && (!p || !aligned(p, 16))) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

// In place only row by row.
bool clashes(const moe_norm_shape* s, const void* out, int64_t ldout, const void* in, int64_t ldin) {
  return s->rows > 1 && out == in && ldout != ldin;
}

moe::RowNormArgs norm_args(const moe_norm_shape* s) {
  moe::RowNormArgs a{};
  a.rows = s->rows;
  a.H = s->H;
  a.eps = s->eps;
  a.type = s->type;
  a.weight_type = s->weight_type;
  return a;
}

size_t norm_workspace(int H) { return static_cast<size_t>(moe::norm_max_ctas(H)) * 2 * H * sizeof(float); }

// The kernels' form of the tensors, empty ones left out; false: a bad one (`status`).
moe_status grad_tensors(const moe_grad_tensor* t, int32_t n, bool clip, std::unique_ptr<moe::GradTensor[]>& out,
                        int64_t& used) {
  used = 0;
  if (n < 0 || (n > 0 && !t)) return MOE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].n < 0 || !is_type(t[i].type)) return MOE_ERR_INVALID_ARG;
    if (t[i].n > kMaxElements) return MOE_ERR_UNSUPPORTED;
    const size_t size = t[i].type == MOE_TYPE_FP32 ? 4 : 2;
    if (t[i].n > 0 && (!t[i].data || !aligned(t[i].data, size))) return MOE_ERR_INVALID_ARG;
    if (!clip) continue;
    if (!is_type(t[i].out_type)) return MOE_ERR_INVALID_ARG;
    const size_t out_size = t[i].out_type == MOE_TYPE_FP32 ? 4 : 2;
    if (t[i].n > 0 && (!t[i].out || !aligned(t[i].out, out_size))) return MOE_ERR_INVALID_ARG;
    if (t[i].n > 0 && t[i].out == t[i].data && t[i].out_type != t[i].type) return MOE_ERR_INVALID_ARG;
  }
  out.reset(new (std::nothrow) moe::GradTensor[n > 0 ? n : 1]);
  if (!out) return MOE_ERR_CUDA;
  int64_t chunks = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (t[i].n == 0) continue;
    chunks += (t[i].n + moe::kGradChunk - 1) / moe::kGradChunk;
    if (chunks > (int64_t(1) << 30)) return MOE_ERR_UNSUPPORTED;
    moe::GradTensor& g = out[used++];
    g.src = t[i].data;
    g.dst = clip ? t[i].out : nullptr;
    g.n = t[i].n;
    g.type = static_cast<uint8_t>(t[i].type);
    g.dst_type = static_cast<uint8_t>(clip ? t[i].out_type : t[i].type);
    g.vec = aligned(t[i].data, 16);
    g.dst_vec = clip && aligned(t[i].out, 16);
  }
  return MOE_OK;
}

bool good_limits(const float* norm, double max_norm, double eps) {
  return norm && aligned(norm, 4) && max_norm >= 0.0 && eps >= 0.0 && std::isfinite(eps);
}

}  // namespace

extern "C" {

moe_status moe_norm(const moe_norm_shape* shape, const void* x, int64_t ldx, const void* weight, const void* bias,
                    void* y, int64_t ldy, float* mean, float* rstd, moe_stream_t stream) {
  moe_status st = check_norm(shape);
  if (st != MOE_OK) return st;
  const moe_norm_shape* s = shape;
  const bool layer = s->kind == MOE_NORM_LAYER;
  if ((st = check_rows(x, s, ldx)) != MOE_OK) return st;
  if ((st = check_rows(y, s, ldy)) != MOE_OK) return st;
  if (clashes(s, y, ldy, x, ldx)) return MOE_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || !aligned(bias, 16) || !aligned(mean, 4) || !aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
  if (!layer && (bias || mean)) return MOE_ERR_INVALID_ARG;
  if (s->rows == 0) return MOE_OK;
  moe::RowNormArgs a = norm_args(s);
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.ldy = ldy;
  a.mean = mean;
  a.rstd = rstd;
  const int sms = num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return moe::launch_row_norm(layer, a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                    : MOE_ERR_CUDA;
}

moe_status moe_norm_grad_workspace_size(const moe_norm_shape* shape, size_t* bytes) {
  const moe_status st = check_norm(shape);
  if (st != MOE_OK) return st;
  if (!bytes) return MOE_ERR_INVALID_ARG;
  *bytes = norm_workspace(shape->H);
  return MOE_OK;
}

moe_status moe_norm_grad(const moe_norm_shape* shape, const void* dy, int64_t lddy, const void* x, int64_t ldx,
                         const void* weight, const float* mean, const float* rstd, void* dx, int64_t lddx,
                         void* dweight, void* dbias, int32_t dweight_type, int32_t accumulate, void* workspace,
                         size_t workspace_bytes, moe_stream_t stream) {
  moe_status st = check_norm(shape);
  if (st != MOE_OK) return st;
  const moe_norm_shape* s = shape;
  const bool layer = s->kind == MOE_NORM_LAYER;
  if ((st = check_rows(dy, s, lddy)) != MOE_OK) return st;
  if ((st = check_rows(x, s, ldx)) != MOE_OK) return st;
  if ((st = check_rows(dx, s, lddx)) != MOE_OK) return st;
  if (clashes(s, dx, lddx, dy, lddy) || clashes(s, dx, lddx, x, ldx)) return MOE_ERR_INVALID_ARG;
  if (!aligned(weight, 16) || !aligned(mean, 4) || !aligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
  if (s->rows > 0 && (!rstd || (layer && !mean))) return MOE_ERR_INVALID_ARG;
  if (!layer && (dbias || mean)) return MOE_ERR_INVALID_ARG;
  if (dweight || dbias) {
    if (dweight_type != s->weight_type && dweight_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (accumulate && dweight_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
    if (!aligned(dweight, 16) || !aligned(dbias, 16)) return MOE_ERR_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
    if (workspace_bytes < norm_workspace(s->H)) return MOE_ERR_WORKSPACE;
  }
  if (s->rows == 0 && (accumulate || (!dweight && !dbias))) return MOE_OK;
  const int sms = num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  moe::RowNormArgs a = norm_args(s);
  a.x = x;
  a.ldx = ldx;
  a.weight = weight;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dy = dy;
  a.lddy = lddy;
  a.dx = dx;
  a.lddx = lddx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dweight_type = dweight_type;
  a.accumulate = accumulate != 0;
  a.partials = static_cast<float*>(workspace);
  return moe::launch_row_norm_grad(layer, a, sms, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK
                                                                                                         : MOE_ERR_CUDA;
}

moe_status moe_grad_norm_workspace_size(int32_t n_tensors, size_t* bytes) {
  if (n_tensors < 0 || !bytes) return MOE_ERR_INVALID_ARG;
  *bytes = moe::grad_partial_bytes(n_tensors);
  return MOE_OK;
}

moe_status moe_grad_norm(const moe_grad_tensor* tensors, int32_t n_tensors, float* norm, void* workspace,
                         size_t workspace_bytes, moe_stream_t stream) {
  std::unique_ptr<moe::GradTensor[]> t;
  int64_t n = 0;
  const moe_status st = grad_tensors(tensors, n_tensors, false, t, n);
  if (st != MOE_OK) return st;
  if (!norm || !aligned(norm, 4) || !workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe::grad_partial_bytes(n_tensors)) return MOE_ERR_WORKSPACE;
  const int sms = num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return moe::launch_grad_norm(t.get(), n, norm, static_cast<double*>(workspace), sms,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_grad_clip(const moe_grad_tensor* tensors, int32_t n_tensors, const float* norm, double max_norm,
                         double eps, moe_stream_t stream) {
  std::unique_ptr<moe::GradTensor[]> t;
  int64_t n = 0;
  const moe_status st = grad_tensors(tensors, n_tensors, true, t, n);
  if (st != MOE_OK) return st;
  if (!good_limits(norm, max_norm, eps)) return MOE_ERR_INVALID_ARG;
  if (n == 0) return MOE_OK;
  const int sms = num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  return moe::launch_grad_clip(t.get(), n, const_cast<float*>(norm), nullptr, max_norm, eps, sms,
                               reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_grad_norm_clip(const moe_grad_tensor* tensors, int32_t n_tensors, double max_norm, double eps, float* norm,
                              void* workspace, size_t workspace_bytes, moe_stream_t stream) {
  std::unique_ptr<moe::GradTensor[]> t;
  int64_t n = 0;
  const moe_status st = grad_tensors(tensors, n_tensors, true, t, n);
  if (st != MOE_OK) return st;
  if (!good_limits(norm, max_norm, eps) || !workspace || !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < moe::grad_partial_bytes(n_tensors)) return MOE_ERR_WORKSPACE;
  const int sms = num_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  double* partials = static_cast<double*>(workspace);
  const cudaError_t e = n > 0 ? moe::launch_grad_clip(t.get(), n, norm, partials, max_norm, eps, sms, s)
                              : moe::launch_grad_norm(t.get(), n, norm, partials, sms, s);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
