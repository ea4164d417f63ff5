// C ABI of the layer norm and RMS norm of rows: argument checks and launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "host_util.h"
#include "layer_norm.cuh"

using namespace flce;
using host::aligned;

namespace {

constexpr int64_t kMaxCols = 16384;

bool shape_ok(const flce_layer_norm_desc* d) {
  if (!d || d->struct_size != sizeof(flce_layer_norm_desc)) return false;
  if (d->dtype != FLCE_BF16 && d->dtype != FLCE_FP32) return false;
  if (d->rows < 0 || d->rows > (int64_t)INT_MAX - 1024) return false;
  return d->cols > 0 && d->cols % 8 == 0 && d->cols <= kMaxCols && (d->rms == 0 || d->rms == 1);
}

int elem(const flce_layer_norm_desc* d) { return d->dtype == FLCE_BF16 ? 2 : 4; }
int vectors(const flce_layer_norm_desc* d) { return (int)(d->cols * elem(d) / 16); }

// Vectors of a row that a thread holds, and the threads that share it.
struct Split {
  int c, threads;
};
Split split(const flce_layer_norm_desc* d) {
  const int v = vectors(d);
  const int c = v <= 32 ? 1 : v <= 2048 ? 2 : 4;
  return {c, (int)host::ceil_div(host::ceil_div(v, c), 32) * 32};
}

int64_t bwd_blocks(const flce_layer_norm_desc* d, int sms) {
  const int64_t per_sm = std::max(1, std::min(16, 512 / split(d).threads));
  return std::min<int64_t>(d->rows, per_sm * sms);
}

bool rows_ok(int64_t row, int64_t cols) { return row % 8 == 0 && row >= cols; }

flce_status check(const flce_layer_norm_desc* d, const void* const* ptrs, int n, const void* const* optional, int m) {
  if (!shape_ok(d)) return FLCE_ERR_ARG;
  if (!(std::isfinite(d->eps) && d->eps >= 0.f)) return FLCE_ERR_ARG;
  if (!rows_ok(d->x_row, d->cols)) return FLCE_ERR_ARG;
  for (int i = 0; i < m; ++i)
    if (!aligned(optional[i], 16)) return FLCE_ERR_ARG;
  if (d->rows == 0) return FLCE_OK;
  for (int i = 0; i < n; ++i)
    if (!ptrs[i] || !aligned(ptrs[i], 16)) return FLCE_ERR_ARG;
  return FLCE_OK;
}

LayerNormParams params(const flce_layer_norm_desc* d) {
  LayerNormParams p{};
  p.rows = d->rows;
  p.x_row = d->x_row;
  p.residual_row = d->residual_row;
  p.vectors = vectors(d);
  p.eps = d->eps;
  p.inv_cols = 1.f / (float)d->cols;
  return p;
}

template <typename T, int C>
flce_status launch_fwd(const flce_layer_norm_desc* d, const LayerNormParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)d->rows);
  const int threads = split(d).threads;
  return d->rms ? host::launch(layer_norm_fwd<T, C, false>, grid, threads, 0, st, p)
                : host::launch(layer_norm_fwd<T, C, true>, grid, threads, 0, st, p);
}

template <typename T, int C>
flce_status launch_bwd(const flce_layer_norm_desc* d, const LayerNormParams& p, int64_t blocks, cudaStream_t st) {
  const dim3 grid((unsigned)blocks);
  const int threads = split(d).threads;
  if (d->rms)
    return p.db_partial ? host::launch(layer_norm_bwd<T, C, false, true>, grid, threads, 0, st, p)
                        : host::launch(layer_norm_bwd<T, C, false, false>, grid, threads, 0, st, p);
  return p.db_partial ? host::launch(layer_norm_bwd<T, C, true, true>, grid, threads, 0, st, p)
                      : host::launch(layer_norm_bwd<T, C, true, false>, grid, threads, 0, st, p);
}

template <typename T>
flce_status run_fwd(const flce_layer_norm_desc* d, const LayerNormParams& p, cudaStream_t st) {
  const int c = split(d).c;
  return c == 1 ? launch_fwd<T, 1>(d, p, st) : c == 2 ? launch_fwd<T, 2>(d, p, st) : launch_fwd<T, 4>(d, p, st);
}
template <typename T>
flce_status run_bwd(const flce_layer_norm_desc* d, const LayerNormParams& p, int64_t blocks, cudaStream_t st) {
  const int c = split(d).c;
  return c == 1   ? launch_bwd<T, 1>(d, p, blocks, st)
         : c == 2 ? launch_bwd<T, 2>(d, p, blocks, st)
                  : launch_bwd<T, 4>(d, p, blocks, st);
}

}  // namespace

extern "C" {

size_t flce_layer_norm_workspace_size(const flce_layer_norm_desc* d) {
  if (!shape_ok(d)) return 0;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152;
  }
  return host::align_up(2 * std::max<size_t>(1, bwd_blocks(d, sms)) * d->cols * 4);
}

flce_status flce_layer_norm_forward(const flce_layer_norm_desc* d, const void* x, const void* residual,
                                    const void* weight, const void* bias, void* y, void* sum, float* mean,
                                    float* rstd, void* stream) {
  host::reset_launches();
  const void* ptrs[] = {x, y};
  const void* optional[] = {residual, weight, bias, sum};
  FLCE_HOST_TRY(check(d, ptrs, 2, optional, 4));
  if (residual && (!sum || !rows_ok(d->residual_row, d->cols))) return FLCE_ERR_ARG;
  if (!aligned(mean, 4) || !aligned(rstd, 4)) return FLCE_ERR_ARG;
  if (d->rows == 0) return FLCE_OK;
  if (!rstd || (!d->rms && !mean)) return FLCE_ERR_ARG;
  int dev, sms;
  FLCE_HOST_TRY(host::device(&dev, &sms));
  LayerNormParams p = params(d);
  p.x = x;
  p.residual = residual;
  p.w = weight;
  p.b = bias;
  p.out = y;
  p.sum = sum;
  p.mean = mean;
  p.rstd = rstd;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return d->dtype == FLCE_BF16 ? run_fwd<__nv_bfloat16>(d, p, st) : run_fwd<float>(d, p, st);
}

flce_status flce_layer_norm_backward(const flce_layer_norm_desc* d, const void* dy, const void* x, const void* weight,
                                     const float* mean, const float* rstd, const void* dsum, void* dx,
                                     float* dweight, float* dbias, void* workspace, size_t ws_bytes, void* stream) {
  host::reset_launches();
  const void* ptrs[] = {dy, x, dx};
  const void* optional[] = {weight, dsum};
  FLCE_HOST_TRY(check(d, ptrs, 3, optional, 2));
  if (!dweight || !aligned(dweight, 4) || !aligned(dbias, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return FLCE_ERR_ARG;
  if (d->rows > 0 && (!rstd || (!d->rms && !mean))) return FLCE_ERR_ARG;
  int dev, sms;
  FLCE_HOST_TRY(host::device(&dev, &sms));
  const int64_t blocks = bwd_blocks(d, sms);
  if (!workspace || !aligned(workspace, host::kAlign) ||
      ws_bytes < 2 * (size_t)std::max<int64_t>(1, blocks) * d->cols * 4)
    return FLCE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  LayerNormParams p = params(d);
  p.x = x;
  p.w = weight;
  p.dy = dy;
  p.ds = dsum;
  p.out = dx;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.dw_partial = static_cast<float*>(workspace);
  p.db_partial = dbias ? p.dw_partial + blocks * d->cols : nullptr;
  if (d->rows > 0)
    FLCE_HOST_TRY(d->dtype == FLCE_BF16 ? run_bwd<__nv_bfloat16>(d, p, blocks, st) : run_bwd<float>(d, p, blocks, st));
  return host::launch(layer_norm_dw, dim3((unsigned)host::ceil_div(d->cols, 32), dbias ? 2 : 1), 1024, 0, st,
                      static_cast<const float*>(p.dw_partial), static_cast<const float*>(p.db_partial), (int)blocks,
                      (int)d->cols, dweight, dbias);
}

}  // extern "C"
