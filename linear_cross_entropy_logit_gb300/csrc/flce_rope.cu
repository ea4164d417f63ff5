// C ABI of the rotary positions: argument checks and launches.
#include <algorithm>
#include <climits>
#include <cmath>

#include "host_util.h"
#include "rope.cuh"

using namespace flce;
using host::aligned;

namespace {

bool shape_ok(const flce_rope_desc* d) {
  if (!d || d->struct_size != sizeof(flce_rope_desc)) return false;
  if (d->dtype != FLCE_BF16 && d->dtype != FLCE_FP32) return false;
  if (d->tokens < 0 || d->tokens > (int64_t)INT_MAX - 1024) return false;
  if (d->q_heads <= 0 || d->kv_heads <= 0 || d->q_heads > 65535 || d->kv_heads > 65535) return false;
  if (d->head_dim <= 0 || d->head_dim % 8 || d->head_dim > 256) return false;
  return d->rot_dim > 0 && d->rot_dim % 8 == 0 && d->rot_dim <= d->head_dim;
}

bool stride_ok(int64_t row, int64_t head, int64_t head_dim) {
  return row % 8 == 0 && head % 8 == 0 && row > 0 && head >= head_dim;
}

template <typename T, int P>
flce_status launch(const flce_rope_desc* d, const RopeParams& p, dim3 grid, int threads, cudaStream_t st) {
  const size_t smem = (size_t)threads * kRopeStage<T, P> + (size_t)p.tokens_per_block * p.rot_dim * sizeof(float);
  return d->interleaved ? host::launch(rope_kernel<T, P, true>, grid, threads, smem, st, p)
                        : host::launch(rope_kernel<T, P, false>, grid, threads, smem, st, p);
}

flce_status run(const flce_rope_desc* d, const void* q, const void* k, const double* inv_freq,
                const int64_t* positions, void* q_out, void* k_out, int backward, void* stream) {
  host::reset_launches();
  if (!shape_ok(d) || !std::isfinite(d->magnitude)) return FLCE_ERR_ARG;
  if (!stride_ok(d->q_row, d->q_head, d->head_dim) || !stride_ok(d->k_row, d->k_head, d->head_dim))
    return FLCE_ERR_ARG;
  if (!inv_freq || !aligned(inv_freq, 8) || !aligned(positions, 8)) return FLCE_ERR_ARG;
  if (d->tokens == 0) return FLCE_OK;
  for (const void* ptr : {q, k, (const void*)q_out, (const void*)k_out})
    if (!ptr || !aligned(ptr, 16)) return FLCE_ERR_ARG;
  int dev, sms;
  FLCE_HOST_TRY(host::device(&dev, &sms));
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.tokens = d->tokens;
  p.q_row = d->q_row;
  p.q_head = d->q_head;
  p.k_row = d->k_row;
  p.k_head = d->k_head;
  p.q_heads = (int)d->q_heads;
  p.kv_heads = (int)d->kv_heads;
  p.head_dim = (int)d->head_dim;
  p.rot_dim = (int)d->rot_dim;
  p.magnitude = d->magnitude;
  p.backward = backward;
  const bool wide = d->rot_dim % 16 == 0 && d->head_dim % 16 == 0;
  p.units = (int)d->head_dim / (wide ? 16 : 8);
  // A thread takes kRopeHeads heads of its token, with fewer tokens a block where that would
  // leave SMs idle; the heads of a single token are then shared by as many threads as
  // there are.
  const int groups = kRopeThreads / p.units, heads = p.q_heads + p.kv_heads;
  const int in_flight = d->dtype == FLCE_BF16 ? kRopeHeads<__nv_bfloat16> : kRopeHeads<float>;
  const int fit = groups / std::min(groups, (int)host::ceil_div(heads, in_flight));
  p.tokens_per_block = (int)std::max<int64_t>(1, std::min<int64_t>(fit, d->tokens / (2 * sms)));
  p.slots = std::min(groups / p.tokens_per_block, heads);
  const int threads = p.units * p.slots * p.tokens_per_block;
  const dim3 grid((unsigned)host::ceil_div(d->tokens, p.tokens_per_block));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (d->dtype == FLCE_BF16)
    return wide ? launch<__nv_bfloat16, 8>(d, p, grid, threads, st) : launch<__nv_bfloat16, 4>(d, p, grid, threads, st);
  return wide ? launch<float, 8>(d, p, grid, threads, st) : launch<float, 4>(d, p, grid, threads, st);
}

}  // namespace

extern "C" {

flce_status flce_rope_forward(const flce_rope_desc* d, const void* q, const void* k, const double* inv_freq,
                              const int64_t* positions, void* q_out, void* k_out, void* stream) {
  return run(d, q, k, inv_freq, positions, q_out, k_out, 0, stream);
}

flce_status flce_rope_backward(const flce_rope_desc* d, const void* dq_out, const void* dk_out,
                               const double* inv_freq, const int64_t* positions, void* dq, void* dk, void* stream) {
  return run(d, dq_out, dk_out, inv_freq, positions, dq, dk, 1, stream);
}

}  // extern "C"
