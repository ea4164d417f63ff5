// C ABI of the layer norm and RMS norm of rows: argument checks and launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <mutex>

#include "host_util.h"
#include "layer_norm.cuh"

using namespace flce;
using host::aligned;

namespace {

constexpr int64_t kMaxCols = 16384;
constexpr int kSmemPerSm = 224 * 1024;
// Threads of an SM, as many as have room for their registers (80 and 128).
constexpr int kFwdThreads = 768, kBwdThreads = 512;

bool shape_ok(const flce_layer_norm_desc* d) {
  if (!d || d->struct_size != sizeof(flce_layer_norm_desc)) return false;
  if (d->dtype != FLCE_BF16 && d->dtype != FLCE_FP32) return false;
  if (d->rows < 0 || d->rows > (int64_t)INT_MAX - 1024) return false;
  return d->cols > 0 && d->cols % 8 == 0 && d->cols <= kMaxCols && (d->rms == 0 || d->rms == 1);
}

int elem(const flce_layer_norm_desc* d) { return d->dtype == FLCE_BF16 ? 2 : 4; }
int vectors(const flce_layer_norm_desc* d) { return (int)(d->cols * elem(d) / 16); }

// Vectors of a row that a thread holds, up to 32 values, and the threads that share it.
struct Split {
  int c, threads;
};
Split split(const flce_layer_norm_desc* d) {
  const int v = vectors(d), sixteen = elem(d);  // vectors of 16 values
  const int c = v <= 32 ? 1 : v <= sixteen * kLayerNormThreads ? sixteen : 2 * sixteen;
  return {c, (int)host::ceil_div(host::ceil_div(v, c), 32) * 32};
}

// Rows in a block's ring: four, or what shared memory has room for (three arrays of
// 16384 floats are 192 KB).
int stages(const flce_layer_norm_desc* d) {
  return vectors(d) <= 1024 ? 4 : vectors(d) <= 2048 ? 2 : 1;
}

int ring_bytes(const flce_layer_norm_desc* d, int arrays) {
  const Split s = split(d);
  return stages(d) * arrays * s.c * s.threads * 16;
}

// Blocks of a persistent launch: what an SM has room for, `most` threads at most.
int64_t blocks(const flce_layer_norm_desc* d, int arrays, int most, int sms) {
  const int per_sm = std::min(std::min(32, most / split(d).threads), kSmemPerSm / (ring_bytes(d, arrays) + 2048));
  return std::min<int64_t>(d->rows, (int64_t)std::max(1, per_sm) * sms);
}
// Forward: with a residual and sixteen rows or more for each such block, blocks of four rows
// instead, as many as that makes: the SMs take them as they come free, and reads and writes of
// four arrays mix better (16384 rows of 4096 in bf16: 88 -> 79 us, 30000 of 1024 in fp32: 80 ->
// 74; with fewer rows the blocks' own start costs more, 3001 of 2304 in fp32: 19 -> 22, and
// without a residual it does too, 8192 of 4096: 26 -> 31).
int64_t fwd_blocks(const flce_layer_norm_desc* d, bool residual, int sms) {
  const int64_t n = blocks(d, residual ? 2 : 1, kFwdThreads, sms);
  return residual && d->rows >= 16 * n ? host::ceil_div(d->rows, 4) : n;
}
// Backward: the same number whether a gradient of the sum is given or not, for its partial
// rows are the workspace.
int64_t bwd_blocks(const flce_layer_norm_desc* d, int sms) { return blocks(d, 3, kBwdThreads, sms); }

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

struct Setup {
  std::once_flag once[host::kMaxDevices];
  cudaError_t err[host::kMaxDevices] = {};
};
template <typename Kern>
flce_status run(Setup& s, Kern kern, const flce_layer_norm_desc* d, int arrays, int64_t blocks,
                const LayerNormParams& p, int dev, cudaStream_t st) {
  std::call_once(s.once[dev], [&] {
    s.err[dev] = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemPerSm);
  });
  if (s.err[dev] != cudaSuccess) return host::fail(s.err[dev], "cudaFuncSetAttribute");
  return host::launch(kern, dim3((unsigned)blocks), split(d).threads, ring_bytes(d, arrays), st, p);
}

// Rows of a barrier, backward: two where they are floats, which are read from the ring in
// twice as many loads, and there is room for four (3001 rows of 2304: 43 us, 59 with one); one
// of bf16, whose registers then leave the compiler more room (8192 rows of 4096: 67.6 us, 73.3
// with two; forward and backward both).
template <typename T, int STAGES>
constexpr int kRows = sizeof(T) == 4 && STAGES == 4 ? 2 : 1;

struct Launch {
  const flce_layer_norm_desc* d;
  const LayerNormParams& p;
  int dev, sms;
  cudaStream_t st;
  bool bwd;

  template <typename T, int C, int STAGES, bool CENTER, bool BIAS>
  flce_status backward() const {
    static Setup part;
    const int arrays = p.ds ? 3 : 2;
    const int64_t n = bwd_blocks(d, sms);
    if constexpr (sizeof(T) == 2) {
      static Setup full;
      if (split(d).threads * C == vectors(d))
        return run(full, layer_norm_bwd<T, C, STAGES, kRows<T, STAGES>, CENTER, BIAS, true>, d, arrays, n, p, dev, st);
    }
    return run(part, layer_norm_bwd<T, C, STAGES, kRows<T, STAGES>, CENTER, BIAS, false>, d, arrays, n, p, dev, st);
  }
  template <typename T, int C, int STAGES, bool CENTER>
  flce_status pick() const {
    static Setup fwd;
    if (bwd) return p.db_partial ? backward<T, C, STAGES, CENTER, true>() : backward<T, C, STAGES, CENTER, false>();
    return run(fwd, layer_norm_fwd<T, C, STAGES, CENTER>, d, p.residual ? 2 : 1, fwd_blocks(d, p.residual, sms), p,
               dev, st);
  }
  template <typename T, int C, int STAGES>
  flce_status pick() const {
    return d->rms ? pick<T, C, STAGES, false>() : pick<T, C, STAGES, true>();
  }
  template <typename T>
  flce_status pick() const {
    const int c = split(d).c;
    constexpr int kSixteen = sizeof(T);
    if (c == 1) return pick<T, 1, 4>();
    if (c == 2 * kSixteen) return pick<T, 2 * kSixteen, sizeof(T) == 2 ? 2 : 1>();
    if constexpr (sizeof(T) == 4)
      if (stages(d) == 2) return pick<T, kSixteen, 2>();
    return pick<T, kSixteen, 4>();
  }
  flce_status operator()() const { return d->dtype == FLCE_BF16 ? pick<__nv_bfloat16>() : pick<float>(); }
};

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
  return Launch{d, p, dev, sms, st, false}();
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
  const int64_t partial_rows = bwd_blocks(d, sms);
  if (!workspace || !aligned(workspace, host::kAlign) ||
      ws_bytes < 2 * (size_t)std::max<int64_t>(1, partial_rows) * d->cols * 4)
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
  p.db_partial = dbias ? p.dw_partial + partial_rows * d->cols : nullptr;
  if (d->rows > 0) FLCE_HOST_TRY((Launch{d, p, dev, sms, st, true}()));
  return host::launch(layer_norm_dw, dim3((unsigned)host::ceil_div(d->cols, 32), dbias ? 2 : 1), 1024, 0, st,
                      static_cast<const float*>(p.dw_partial), static_cast<const float*>(p.db_partial), (int)partial_rows,
                      (int)d->cols, dweight, dbias);
}

}  // extern "C"
