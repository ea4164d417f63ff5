// Kernels of the linear distillation around the GEMMs: the student's logits at
// the teacher's entries, the loss, and what the entries change in dZ.
//
//   q_ik  = exp(t_ik / T - tl_i),  tl_i = log sum_k exp(t_ik / T), or the teacher's own
//   l_i   = sum_k q_ik (log q_ik - log p_ik)
//         = sum_k q_ik (t_ik - z_ik) / T + Q_i (lse_i - tl_i),   Q_i = sum_k q_ik
//   dZ_ij = c / T (Q_i exp(z_ij / T - lse_i) - sum of q_ik with id_ik = j)
//
// The GEMM core takes lse and the first term of dZ from logits that it never
// stores, with T folded into the exponentials' factor and Q_i into lse.  What is left
// is sparse, K entries a row.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "aux_kernels.cuh"
#include "ptx.cuh"

namespace flce {

struct DistillParams {
  const int64_t* ids;        // N x K; negative: no entry
  const void* teacher;       // N x K logits
  const float* teacher_lse;  // N, or null
  float* logits;             // N x K: the student's at the ids, 0 where there is none
  int N, K, H, V;
  float inv_t;               // 1 / T
  int* err_word;
};

__device__ __forceinline__ float teacher_logit(const DistillParams& p, int64_t i, const float*) {
  return static_cast<const float*>(p.teacher)[i];
}
__device__ __forceinline__ float teacher_logit(const DistillParams& p, int64_t i, const __nv_bfloat16*) {
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p.teacher)[i]);
}

// What a warp needs of a row of the teacher.
struct TeacherRow {
  bool valid;  // it has entries, and none outside the vocabulary
  bool error;  // one is
  float tl, Q;
};

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// An entry that counts: an id, and a logit that is not -infinity (NaN counts: it shows).
__device__ __forceinline__ bool entry(int64_t id, float t) { return id >= 0 && !(t == -INFINITY); }

template <typename T>
__device__ __forceinline__ TeacherRow teacher_row(const DistillParams& p, int64_t row, int lane) {
  TeacherRow r{};
  float m = -INFINITY;
  bool any = false, bad = false, nan = false;
  for (int k = lane; k < p.K; k += 32) {
    const int64_t id = p.ids[row * p.K + k];
    const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr) * p.inv_t;
    bad |= id >= p.V;
    if (entry(id, t)) {
      any = true;
      nan |= t != t;
      m = fmaxf(m, t);
    }
  }
  r.error = __any_sync(~0u, bad);
  r.valid = __any_sync(~0u, any) && !r.error;
  nan = __any_sync(~0u, nan);
  m = warp_max(m);
  float s = 0.f;
  // relative to the largest, or to the teacher's own sum
  if (p.teacher_lse) m = p.teacher_lse[row];
  for (int k = lane; k < p.K; k += 32) {
    const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr) * p.inv_t;
    if (entry(p.ids[row * p.K + k], t)) s += expf(t - m);
  }
  s = warp_sum(s);
  r.tl = p.teacher_lse ? m : m + logf(s);
  r.Q = p.teacher_lse ? s : 1.f;
  if (nan) r.tl = r.Q = __int_as_float(0x7fc00000);
  return r;
}

// The student's logits at the teacher's ids: a block a row of X, a warp four entries at a
// time, in fp32 (an exact product of two bf16 each).  Bound by the reads of the rows of W.
constexpr int kGatherThreads = 256;
__global__ void __launch_bounds__(kGatherThreads) distill_gather(const __nv_bfloat16* X, const __nv_bfloat16* W,
                                                                 const __grid_constant__ DistillParams p) {
  const int64_t row = blockIdx.x;
  const int lane = threadIdx.x & 31, vectors = p.H / 8;
  const uint4* x_row = reinterpret_cast<const uint4*>(X + row * p.H);  // in L1 after the first warp
  constexpr int U = 4;
  for (int k0 = (threadIdx.x >> 5) * U; k0 < p.K; k0 += kGatherThreads / 32 * U) {
    const uint4* w[U];
    bool live[U];
    float sum[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t id = k0 + u < p.K ? p.ids[row * p.K + k0 + u] : -1;
      live[u] = id >= 0 && id < p.V;
      w[u] = reinterpret_cast<const uint4*>(W + (live[u] ? id : 0) * p.H);
      sum[u] = 0.f;
    }
    for (int i = lane; i < vectors; i += 32) {
      const uint4 x = x_row[i];
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!live[u]) continue;
        const uint4 v = w[u][i];
        const uint32_t vs[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum[u] = fmaf(__uint_as_float(xs[j] << 16), __uint_as_float(vs[j] << 16), sum[u]);
          sum[u] = fmaf(__uint_as_float(xs[j] & 0xffff0000u), __uint_as_float(vs[j] & 0xffff0000u), sum[u]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float s = warp_sum(sum[u]);
      if (lane == 0 && k0 + u < p.K) p.logits[row * p.K + k0 + u] = live[u] ? s : 0.f;
    }
  }
}

// lse of each row from the vocabulary groups' partials (as lse_merge_kernel), then its loss
// by the entries: a block MERGE_ROWS rows, each warp four of them.  All orders are fixed.
template <typename T>
__global__ void __launch_bounds__(MERGE_THREADS)
    distill_merge(const float4* __restrict__ partials, int n_groups, int m_pad,
                  const __grid_constant__ DistillParams p, float* __restrict__ lse_out,
                  float* __restrict__ row_loss, double* __restrict__ block_loss, int* __restrict__ block_valid) {
  __shared__ float4 s_part[MERGE_SLICES][MERGE_ROWS];
  __shared__ float s_lse[MERGE_ROWS];
  __shared__ double s_loss[MERGE_ROWS];
  __shared__ int s_valid[MERGE_ROWS];
  const int r = threadIdx.x % MERGE_ROWS, slice = threadIdx.x / MERGE_ROWS;
  const int row0 = blockIdx.x * MERGE_ROWS;
  if (row0 + r < p.N) s_part[slice][r] = merge_slice(partials, n_groups, m_pad, row0 + r, slice);
  __syncthreads();
  if (slice == 0) {
    s_loss[r] = 0.0;
    s_valid[r] = 0;
    if (row0 + r < p.N) {
      const float4 t = combine_slices(s_part, r);
      s_lse[r] = (t.x + log2f(t.y)) * LN2;
      lse_out[row0 + r] = s_lse[r];
    }
  }
  __syncthreads();
  for (int i = slice; i < MERGE_ROWS && row0 + i < p.N; i += MERGE_SLICES) {
    const int64_t row = row0 + i;
    const TeacherRow tr = teacher_row<T>(p, row, r);
    if (tr.error && r == 0) record_error(p.err_word, kErrLabel);
    double l = 0.0;
    if (tr.valid) {
      for (int k = r; k < p.K; k += 32) {
        const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr) * p.inv_t;
        if (entry(p.ids[row * p.K + k], t)) {
          const float q = expf(t - tr.tl);
          if (!(q == 0.f)) l += (double)q * (double)(t - p.logits[row * p.K + k] * p.inv_t);
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(~0u, l, o);
      if (!(tr.Q == 0.f)) l += (double)tr.Q * (double)(s_lse[i] - tr.tl);
    }
    if (r == 0) {
      s_loss[i] = l;
      s_valid[i] = tr.valid;
      if (row_loss) row_loss[row] = (float)l;
    }
  }
  __syncthreads();
  if (slice) return;
  double loss = s_loss[r];
  int valid = s_valid[r];
#pragma unroll
  for (int o = MERGE_ROWS / 2; o > 0; o >>= 1) {
    loss += __shfl_xor_sync(~0u, loss, o);
    valid += __shfl_xor_sync(~0u, valid, o);
  }
  if (r == 0) {
    block_loss[blockIdx.x] = loss;
    block_valid[blockIdx.x] = valid;
  }
}

// Backward, a warp a row: what the GEMM core needs of it (the mark V of a row that counts, -1
// of one that does not, and lse - log Q, so that its softmax term is Q p), and dZ at each
// entry, c / T (Q p - sum of q of the same id), formed in fp32 from the forward's logit and
// rounded once: the difference of nearly equal p and q keeps its digits.
constexpr int kPrepareThreads = 128;
template <typename T>
__global__ void __launch_bounds__(kPrepareThreads)
    distill_prepare(const __grid_constant__ DistillParams p, const float* __restrict__ lse,
                    const int* __restrict__ valid_count, const float* __restrict__ grad_loss, int reduction_sum,
                    float* __restrict__ scale, int64_t* __restrict__ marks, float* __restrict__ lse_q,
                    int* __restrict__ ids32, uint16_t* __restrict__ dz) {
  extern __shared__ int shared[];  // each warp: K ids, K probabilities
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* id_of = shared + warp * 2 * p.K;
  float* q_of = reinterpret_cast<float*>(id_of + p.K);
  const float g = grad_loss ? *grad_loss : 1.f;
  const int nv = reduction_sum ? 1 : *valid_count;
  const float c = nv > 0 ? (float)((double)g * (double)p.inv_t / (double)nv) : 0.f;
  if (blockIdx.x == 0 && threadIdx.x == 0) *scale = c;
  const int64_t row = (int64_t)blockIdx.x * (kPrepareThreads / 32) + warp;
  if (row >= p.N) return;
  const TeacherRow tr = teacher_row<T>(p, row, lane);
  for (int k = lane; k < p.K; k += 32) {
    const int64_t id = p.ids[row * p.K + k];
    const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr) * p.inv_t;
    const bool in = tr.valid && entry(id, t);
    id_of[k] = in ? (int)id : -1;
    q_of[k] = in ? expf(t - tr.tl) : 0.f;
  }
  __syncwarp();
  const float l = lse[row];
  if (lane == 0) {
    marks[row] = tr.valid ? p.V : -1;
    lse_q[row] = tr.valid ? l - logf(tr.Q) : 0.f;
  }
  for (int k = lane; k < p.K; k += 32) {
    const int id = id_of[k];
    float same = 0.f;
    for (int j = 0; j < p.K; ++j) same += id_of[j] == id ? q_of[j] : 0.f;
    const float d = fmaf(tr.Q, expf(p.logits[row * p.K + k] * p.inv_t - l), -same);
    ids32[row * p.K + k] = id;
    dz[row * p.K + k] = __bfloat16_as_ushort(__float2bfloat16_rn(c * d));
  }
}

// The entries of a vocabulary chunk put into its dZ, which holds the softmax term there.
__global__ void __launch_bounds__(256) distill_scatter(const int* __restrict__ ids32, const uint16_t* __restrict__ dz,
                                                       int64_t entries, int K, int v0, int width, int64_t pitch,
                                                       uint16_t* __restrict__ chunk) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries; i += (int64_t)gridDim.x * 256) {
    const int at = ids32[i] - v0;
    if (ids32[i] >= 0 && at >= 0 && at < width) chunk[i / K * pitch + at] = dz[i];
  }
}

}  // namespace flce
