// Packed causal attention straight from its formulas, one warp per row: the
// form every faster kernel is checked against.
//   s_ij = scale * q_i . k_j  for j <= i in the same sequence
//   lse_i = log sum_j exp(s_ij),  out_i = sum_j exp(s_ij - lse_i) v_j
//   delta_i = dout_i . out_i,  ds_ij = p_ij (dout_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i,  dv_j = sum_i p_ij dout_i
#pragma once
#include "attn_common.cuh"

namespace flce {

struct AttnIn : AttnParams {
  int64_t q_row, q_head, k_row, k_head;
};

// The sequence [lo, hi) holding `row`; empty when no sequence holds it.
__device__ inline void attn_sequence_of(const AttnIn& p, int row, int& lo, int& hi) {
  int a = 0, b = p.n_seqs;  // cu[a] <= row < cu[b] if both exist
  lo = hi = row;
  if (row < p.cu[0] || row >= p.cu[p.n_seqs]) return;
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (p.cu[m] <= row) a = m; else b = m;
  }
  lo = p.cu[a];
  hi = p.cu[b];
}

// Whether the offsets ascend within [0, tokens]; every thread of the block
// gets the answer.
__device__ inline bool attn_offsets_ok(const AttnIn& p) {
  bool bad = false;
  for (int s = threadIdx.x; s <= p.n_seqs; s += blockDim.x) {
    const int c = p.cu[s];
    bad |= c < 0 || c > p.tokens || (s > 0 && c < p.cu[s - 1]);
  }
  bad = __syncthreads_or(bad);
  if (bad && threadIdx.x == 0) record_error(p.err_word, kErrIndex);
  return !bad;
}

__device__ inline float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

constexpr int kSimpleE = 4;  // values of a head per lane (head_dim <= 128)

__device__ inline void load_row(float (&x)[kSimpleE], const bf16* row, int D, int lane) {
#pragma unroll
  for (int e = 0; e < kSimpleE; ++e) {
    const int d = lane + 32 * e;
    x[e] = d < D ? __bfloat162float(row[d]) : 0.f;
  }
}
__device__ inline void store_row(bf16* row, const float (&x)[kSimpleE], int D, int lane) {
#pragma unroll
  for (int e = 0; e < kSimpleE; ++e) {
    const int d = lane + 32 * e;
    if (d < D) row[d] = __float2bfloat16(x[e]);
  }
}
__device__ inline float dot_row(const float (&x)[kSimpleE], const float (&y)[kSimpleE]) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < kSimpleE; ++e) s = fmaf(x[e], y[e], s);
  return warp_sum(s);
}

__global__ void attn_simple_dq(AttnIn p, const bf16* dout, const bf16* q, const bf16* k,
                               const bf16* v, const bf16* out, const float* lse, float* delta,
                               bf16* dq) {
  const bool ok = attn_offsets_ok(p);
  const int lane = threadIdx.x & 31, h = blockIdx.y, D = p.head_dim;
  const int i = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (i >= p.tokens) return;
  int lo = i, hi = i;
  if (ok) attn_sequence_of(p, i, lo, hi);
  const int kvh = h / p.group;
  const int64_t at = ((int64_t)i * p.q_heads + h) * D;
  float qi[kSimpleE], gi[kSimpleE], x[kSimpleE], acc[kSimpleE] = {};
  load_row(qi, q + i * p.q_row + h * p.q_head, D, lane);
  load_row(gi, dout + at, D, lane);
  load_row(x, out + at, D, lane);
  const float dl = dot_row(gi, x);
  if (lane == 0) delta[(int64_t)h * p.tokens + i] = dl;
  const float li = lse[(int64_t)h * p.tokens + i];
  for (int j = lo; j < hi && j <= i; ++j) {
    load_row(x, v + j * p.v_row + kvh * p.v_head, D, lane);
    const float dp = dot_row(gi, x);
    load_row(x, k + j * p.k_row + kvh * p.k_head, D, lane);
    const float ds = expf(dot_row(qi, x) * p.scale - li) * (dp - dl);
#pragma unroll
    for (int e = 0; e < kSimpleE; ++e) acc[e] = fmaf(ds, x[e], acc[e]);
  }
#pragma unroll
  for (int e = 0; e < kSimpleE; ++e) acc[e] *= p.scale;
  store_row(dq + at, acc, D, lane);
}

__global__ void attn_simple_dkdv(AttnIn p, const bf16* dout, const bf16* q, const bf16* k,
                                 const bf16* v, const float* lse, const float* delta, bf16* dk,
                                 bf16* dv) {
  const bool ok = attn_offsets_ok(p);
  const int lane = threadIdx.x & 31, kvh = blockIdx.y, D = p.head_dim;
  const int j = blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (j >= p.tokens) return;
  int lo = j, hi = j;
  if (ok) attn_sequence_of(p, j, lo, hi);
  float kj[kSimpleE], vj[kSimpleE], x[kSimpleE], ak[kSimpleE] = {}, av[kSimpleE] = {};
  load_row(kj, k + j * p.k_row + kvh * p.k_head, D, lane);
  load_row(vj, v + j * p.v_row + kvh * p.v_head, D, lane);
  for (int g = 0; g < p.group; ++g) {
    const int h = kvh * p.group + g;
    for (int i = j; i < hi; ++i) {
      load_row(x, dout + ((int64_t)i * p.q_heads + h) * D, D, lane);
      float qi[kSimpleE];
      load_row(qi, q + i * p.q_row + h * p.q_head, D, lane);
      const float w = expf(dot_row(qi, kj) * p.scale - lse[(int64_t)h * p.tokens + i]);
      const float ds = w * (dot_row(x, vj) - delta[(int64_t)h * p.tokens + i]);
#pragma unroll
      for (int e = 0; e < kSimpleE; ++e) {
        av[e] = fmaf(w, x[e], av[e]);
        ak[e] = fmaf(ds, qi[e], ak[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kSimpleE; ++e) ak[e] *= p.scale;
  const int64_t at = ((int64_t)j * p.kv_heads + kvh) * D;
  store_row(dk + at, ak, D, lane);
  store_row(dv + at, av, D, lane);
}

}  // namespace flce
