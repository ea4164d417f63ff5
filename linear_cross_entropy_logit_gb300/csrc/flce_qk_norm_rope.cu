// C ABI of the per-head RMS norm with rotary positions: argument checks and
// launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "host_util.h"
#include "qk_norm_rope.cuh"

using namespace flce;
using host::aligned;

namespace {

constexpr int kBlocksPerSm = 4;  // blocks of the persistent backward on each SM

bool shape_ok(const flce_qk_norm_rope_desc* d) {
  if (!d || d->struct_size != sizeof(flce_qk_norm_rope_desc)) return false;
  if (d->dtype != FLCE_BF16 && d->dtype != FLCE_FP32) return false;
  if (d->tokens < 0 || d->tokens > (int64_t)INT_MAX - 1024) return false;
  if (d->q_heads <= 0 || d->kv_heads <= 0 || d->q_heads > 65535 || d->kv_heads > 65535)
    return false;
  if (d->head_dim <= 0 || d->head_dim % 8 || d->head_dim > 256) return false;
  if (d->rot_dim < 0 || d->rot_dim % 8 || d->rot_dim > d->head_dim) return false;
  return true;
}

bool stride_ok(int64_t row, int64_t head, int64_t head_dim) {
  return row % 8 == 0 && head % 8 == 0 && row > 0 && head >= head_dim;
}

// Groups of G lanes hold a head of up to 8 G values.
int group_lanes(int64_t head_dim) { return head_dim <= 64 ? 8 : head_dim <= 128 ? 16 : 32; }

// Blocks of the backward, each of which writes one partial row: as many as
// there is work for, kBlocksPerSm for each of the device's SMs at most.
int64_t backward_blocks(const flce_qk_norm_rope_desc* d, int sms) {
  const int64_t items =
      d->tokens * host::ceil_div(d->q_heads + d->kv_heads, (int64_t)kNormHeads);
  return std::min<int64_t>(host::ceil_div(items, kNormThreads / group_lanes(d->head_dim)),
                           (int64_t)kBlocksPerSm * sms);
}

flce_status check(const flce_qk_norm_rope_desc* d, const void* const* ptrs, int n,
                  const void* const* weights, const float* cos_t, const float* sin_t,
                  const int64_t* positions, const int32_t* err_word) {
  if (!shape_ok(d)) return FLCE_ERR_ARG;
  if (!(std::isfinite(d->eps) && d->eps >= 0.f)) return FLCE_ERR_ARG;
  if (!stride_ok(d->q_row, d->q_head, d->head_dim) || !stride_ok(d->k_row, d->k_head, d->head_dim))
    return FLCE_ERR_ARG;
  if (!err_word || !aligned(err_word, 4)) return FLCE_ERR_ARG;
  for (int i = 0; i < 2; ++i)
    if (!aligned(weights[i], 16)) return FLCE_ERR_ARG;
  if (d->rot_dim > 0) {
    if (!cos_t || !sin_t || !aligned(cos_t, 16) || !aligned(sin_t, 16) || d->table_rows <= 0)
      return FLCE_ERR_ARG;
    if (!aligned(positions, 8)) return FLCE_ERR_ARG;
  }
  if (d->tokens == 0) return FLCE_OK;
  for (int i = 0; i < n; ++i)
    if (!ptrs[i] || !aligned(ptrs[i], 16)) return FLCE_ERR_ARG;
  return FLCE_OK;
}

QkNormRopeParams params(const flce_qk_norm_rope_desc* d, const void* q, const void* k,
                        const void* wq, const void* wk, const float* cos_t, const float* sin_t,
                        const int64_t* positions, void* q_out, void* k_out, int32_t* err_word) {
  QkNormRopeParams p{};
  p.q = q;
  p.k = k;
  p.wq = wq;
  p.wk = wk;
  p.cos_t = cos_t;
  p.sin_t = sin_t;
  p.positions = positions;
  p.q_out = q_out;
  p.k_out = k_out;
  p.q_row = d->q_row;
  p.q_head = d->q_head;
  p.k_row = d->k_row;
  p.k_head = d->k_head;
  p.table_rows = d->table_rows;
  p.blocks_per_token = (int)host::ceil_div(d->q_heads + d->kv_heads, (int64_t)kNormHeads);
  p.items = d->tokens * p.blocks_per_token;
  p.q_heads = (int)d->q_heads;
  p.kv_heads = (int)d->kv_heads;
  p.head_dim = (int)d->head_dim;
  p.rot_dim = (int)d->rot_dim;
  p.eps = d->eps;
  p.inv_dim = 1.f / (float)d->head_dim;
  p.err_word = err_word;
  return p;
}

template <bool BWD, typename T, int G, bool PAIRS>
void launch(const QkNormRopeParams& p, unsigned blocks, cudaStream_t st) {
  if constexpr (BWD)
    qk_norm_rope_bwd<T, G, PAIRS><<<blocks, kNormThreads, 0, st>>>(p);
  else
    qk_norm_rope_fwd<T, G, PAIRS><<<blocks, kNormThreads, 0, st>>>(p);
}

template <bool BWD, typename T>
void launch_g(const flce_qk_norm_rope_desc* d, const QkNormRopeParams& p, unsigned blocks,
              cudaStream_t st) {
  const int g = group_lanes(d->head_dim);
  if (d->interleaved) {
    if (g == 8) launch<BWD, T, 8, true>(p, blocks, st);
    else if (g == 16) launch<BWD, T, 16, true>(p, blocks, st);
    else launch<BWD, T, 32, true>(p, blocks, st);
  } else {
    if (g == 8) launch<BWD, T, 8, false>(p, blocks, st);
    else if (g == 16) launch<BWD, T, 16, false>(p, blocks, st);
    else launch<BWD, T, 32, false>(p, blocks, st);
  }
}

template <bool BWD>
flce_status launch_any(const flce_qk_norm_rope_desc* d, const QkNormRopeParams& p,
                       int64_t blocks, cudaStream_t st) {
  if (d->dtype == FLCE_BF16)
    launch_g<BWD, __nv_bfloat16>(d, p, (unsigned)blocks, st);
  else
    launch_g<BWD, float>(d, p, (unsigned)blocks, st);
  host::count_launch();
  FLCE_HOST_CUDA(cudaGetLastError());
  return FLCE_OK;
}

}  // namespace

extern "C" {

size_t flce_qk_norm_rope_workspace_size(const flce_qk_norm_rope_desc* d) {
  if (!shape_ok(d)) return 0;
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    (void)cudaGetLastError();
    sms = 152;
  }
  return host::align_up(std::max<size_t>(1, backward_blocks(d, sms)) * 2 * d->head_dim * 4);
}

flce_status flce_qk_norm_rope_forward(const flce_qk_norm_rope_desc* d, const void* q,
                                      const void* k, const void* q_weight, const void* k_weight,
                                      const float* cos_table, const float* sin_table,
                                      const int64_t* positions, void* q_out, void* k_out,
                                      int32_t* err_word, void* stream) {
  host::reset_launches();
  const void* ptrs[] = {q, k, q_out, k_out};
  const void* weights[] = {q_weight, k_weight};
  FLCE_HOST_TRY(check(d, ptrs, 4, weights, cos_table, sin_table, positions, err_word));
  if (d->tokens == 0) return FLCE_OK;
  int dev, sms;
  FLCE_HOST_TRY(host::device(&dev, &sms));
  const QkNormRopeParams p = params(d, q, k, q_weight, k_weight, cos_table, sin_table, positions,
                                    q_out, k_out, err_word);
  const int64_t blocks = host::ceil_div(p.items, kNormThreads / group_lanes(d->head_dim));
  if (blocks > INT_MAX) return FLCE_ERR_UNSUPPORTED;
  return launch_any<false>(d, p, blocks, static_cast<cudaStream_t>(stream));
}

flce_status flce_qk_norm_rope_backward(const flce_qk_norm_rope_desc* d, const void* dq_out,
                                       const void* dk_out, const void* q, const void* k,
                                       const void* q_weight, const void* k_weight,
                                       const float* cos_table, const float* sin_table,
                                       const int64_t* positions, void* dq, void* dk,
                                       float* dq_weight, float* dk_weight, void* workspace,
                                       size_t ws_bytes, int32_t* err_word, void* stream) {
  host::reset_launches();
  const void* ptrs[] = {dq_out, dk_out, q, k, dq, dk};
  const void* weights[] = {q_weight, k_weight};
  FLCE_HOST_TRY(check(d, ptrs, 6, weights, cos_table, sin_table, positions, err_word));
  if (!dq_weight || !dk_weight || !aligned(dq_weight, 4) || !aligned(dk_weight, 4))
    return FLCE_ERR_ARG;
  int dev, sms;
  FLCE_HOST_TRY(host::device(&dev, &sms));
  const int64_t blocks = backward_blocks(d, sms);
  if (!workspace || !aligned(workspace, host::kAlign) ||
      ws_bytes < (size_t)blocks * 2 * d->head_dim * 4)
    return FLCE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->tokens > 0) {
    QkNormRopeParams p = params(d, q, k, q_weight, k_weight, cos_table, sin_table, positions, dq,
                                dk, err_word);
    p.dq_out = dq_out;
    p.dk_out = dk_out;
    p.partial = static_cast<float*>(workspace);
    FLCE_HOST_TRY(launch_any<true>(d, p, blocks, st));
  }
  qk_norm_rope_dw<<<(unsigned)host::ceil_div(2 * d->head_dim, 32), 1024, 0, st>>>(
      static_cast<const float*>(workspace), (int)blocks, (int)d->head_dim, dq_weight, dk_weight);
  host::count_launch();
  FLCE_HOST_CUDA(cudaGetLastError());
  return FLCE_OK;
}

}  // extern "C"
