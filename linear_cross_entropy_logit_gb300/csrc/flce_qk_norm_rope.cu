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

// How a head is spread over lanes: 2 P values each, P = 8 where that divides what
// is turned and the whole head (each lane then loads 16 bytes at a time), else 4.
struct Spread {
  int p, log_lanes;
};
Spread spread(const flce_qk_norm_rope_desc* d) {
  const int p = d->rot_dim % 16 == 0 && d->head_dim % 16 == 0 ? 8 : 4;
  int log_lanes = 0;
  while ((2 * p << log_lanes) < d->head_dim) ++log_lanes;
  return {p, log_lanes};
}

int heads_per_item(const flce_qk_norm_rope_desc* d, bool bwd) {
  if (d->dtype == FLCE_BF16)
    return bwd ? NormHeads<__nv_bfloat16>::kBwd : NormHeads<__nv_bfloat16>::kFwd;
  return bwd ? NormHeads<float>::kBwd : NormHeads<float>::kFwd;
}

// Blocks for the items of q and of k: one lane group each forward; backward
// as many as there is work for, kNormBwdBlocks for each SM at most, in proportion.
struct Blocks {
  int64_t q, k;
};
Blocks blocks(const flce_qk_norm_rope_desc* d, bool bwd, int sms) {
  const int64_t per = kNormThreads >> spread(d).log_lanes, u = heads_per_item(d, bwd);
  const int64_t q = d->tokens * host::ceil_div(d->q_heads, u), k = d->tokens * host::ceil_div(d->kv_heads, u);
  Blocks b{host::ceil_div(q, per), host::ceil_div(k, per)};
  const int64_t most = (int64_t)kNormBwdBlocks * sms;
  if (bwd && b.q + b.k > most) {
    b.q = std::min(std::max<int64_t>(1, most * q / (q + k)), most - 1);
    b.k = most - b.q;
  }
  return b;
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
  }
  if (!aligned(positions, 8)) return FLCE_ERR_ARG;
  if (d->tokens == 0) return FLCE_OK;
  for (int i = 0; i < n; ++i)
    if (!ptrs[i] || !aligned(ptrs[i], 16)) return FLCE_ERR_ARG;
  return FLCE_OK;
}

QkNormRopeParams params(const flce_qk_norm_rope_desc* d, bool bwd, const void* q, const void* k,
                        const void* wq, const void* wk, const float* cos_t, const float* sin_t,
                        const int64_t* positions, void* q_out, void* k_out, int32_t* err_word) {
  QkNormRopeParams p{};
  const int64_t u = heads_per_item(d, bwd);
  auto side = [&](const void* x, const void* w, void* out, int64_t row, int64_t head, int64_t heads) {
    NormSide s{};
    s.x = x;
    s.w = w;
    s.out = out;
    s.row = row;
    s.head = head;
    s.heads = (int)heads;
    s.per_token = (int)host::ceil_div(heads, u);
    s.items = d->tokens * s.per_token;
    return s;
  };
  p.q = side(q, wq, q_out, d->q_row, d->q_head, d->q_heads);
  p.k = side(k, wk, k_out, d->k_row, d->k_head, d->kv_heads);
  p.cos_t = cos_t;
  p.sin_t = sin_t;
  p.positions = positions;
  p.table_rows = d->table_rows;
  p.log_lanes = spread(d).log_lanes;
  p.head_dim = (int)d->head_dim;
  p.rot_dim = (int)d->rot_dim;
  p.eps = d->eps;
  p.inv_dim = 1.f / (float)d->head_dim;
  p.err_word = err_word;
  return p;
}

template <bool BWD, typename T, int P, bool PAIRS>
flce_status launch(const QkNormRopeParams& p, unsigned n, cudaStream_t st) {
  if constexpr (BWD)
    return host::launch(qk_norm_rope_bwd<T, P, PAIRS>, n, kNormThreads, 0, st, p);
  else
    return host::launch(qk_norm_rope_fwd<T, P, PAIRS>, n, kNormThreads, 0, st, p);
}

template <bool BWD, typename T>
flce_status launch_t(const flce_qk_norm_rope_desc* d, const QkNormRopeParams& p, unsigned n,
                     cudaStream_t st) {
  const bool wide = spread(d).p == 8;
  if (d->interleaved)
    return wide ? launch<BWD, T, 8, true>(p, n, st) : launch<BWD, T, 4, true>(p, n, st);
  else
    return wide ? launch<BWD, T, 8, false>(p, n, st) : launch<BWD, T, 4, false>(p, n, st);
}

template <bool BWD>
flce_status launch_any(const flce_qk_norm_rope_desc* d, const QkNormRopeParams& p, int64_t n,
                       cudaStream_t st) {
  return d->dtype == FLCE_BF16 ? launch_t<BWD, __nv_bfloat16>(d, p, (unsigned)n, st)
                               : launch_t<BWD, float>(d, p, (unsigned)n, st);
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
  const Blocks b = blocks(d, true, sms);
  return host::align_up(std::max<size_t>(1, b.q + b.k) * d->head_dim * 4);
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
  QkNormRopeParams p = params(d, false, q, k, q_weight, k_weight, cos_table, sin_table, positions,
                              q_out, k_out, err_word);
  const Blocks n = blocks(d, false, sms);
  // items are divided as 32-bit numbers on the device
  if (n.q + n.k > INT_MAX || p.q.items > UINT_MAX || p.k.items > UINT_MAX) return FLCE_ERR_UNSUPPORTED;
  p.q_blocks = n.q;
  return launch_any<false>(d, p, n.q + n.k, static_cast<cudaStream_t>(stream));
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
  const Blocks n = blocks(d, true, sms);
  if (!workspace || !aligned(workspace, host::kAlign) ||
      ws_bytes < (size_t)(n.q + n.k) * d->head_dim * 4)
    return FLCE_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->tokens > 0) {
    QkNormRopeParams p = params(d, true, q, k, q_weight, k_weight, cos_table, sin_table, positions, dq,
                                dk, err_word);
    if (p.q.items > UINT_MAX || p.k.items > UINT_MAX) return FLCE_ERR_UNSUPPORTED;
    p.q.dy = dq_out;
    p.k.dy = dk_out;
    p.q_blocks = n.q;
    p.partial = static_cast<float*>(workspace);
    FLCE_HOST_TRY(launch_any<true>(d, p, n.q + n.k, st));
  }
  return host::launch(qk_norm_rope_dw, dim3((unsigned)host::ceil_div(d->head_dim, 32), 2), 1024, 0, st,
                      static_cast<const float*>(workspace), (int)n.q, (int)(n.q + n.k), (int)d->head_dim,
                      dq_weight, dk_weight);
}

}  // extern "C"
