// Kernels of the linear distillation around the GEMMs: the student's logits at
// the teacher's entries, the loss, and what the entries change in dZ.
//
//   q_ik  = exp(t_ik / T - tl_i),  tl_i = log sum_k exp(t_ik / T), or the teacher's own
//   l_i   = sum_k q_ik (log q_ik - log p_ik)
//         = sum_k q_ik (t_ik - z_ik) / T + Q_i (lse_i - tl_i),   Q_i = sum_k q_ik
// (t and tl may both be taken relative to the row's largest t: they are, without the teacher's
// own tl, so that its logits may lie anywhere and reach to the ends of their type)
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
  float* logits;             // N x K: the student's at the ids, 0 where the id is none of V
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
  float top;   // what t and tl are relative to: the largest t of the entries, or 0
  float tl, Q;
  // t / T relative to top; -infinity where the difference is more than a float holds
  __device__ __forceinline__ float scaled(float t, float inv_t) const { return (t - top) * inv_t; }
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
    const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr);
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
  r.top = p.teacher_lse ? 0.f : m;
  r.tl = p.teacher_lse ? p.teacher_lse[row] : 0.f;
  float s = 0.f;
  for (int k = lane; k < p.K; k += 32) {
    const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr);
    if (entry(p.ids[row * p.K + k], t)) s += expf(r.scaled(t, p.inv_t) - r.tl);
  }
  s = warp_sum(s);
  r.Q = 1.f;
  if (p.teacher_lse)
    r.Q = s;
  else
    r.tl = logf(s);
  if (nan) r.tl = r.Q = __int_as_float(0x7fc00000);
  return r;
}

// What a row's loss needs beside lse: l = rest + Q (lse - tl) for a row that counts.
struct DistillRow {
  float rest;  // sum of q (t - z) / T, t as tl relative to the row's top
  float tl, Q;
  int valid;
};

// Forward, a block a row at a time: the student's logits at the teacher's ids, in fp32 (products
// of two bf16 are exact; the tensor cores' sums are off by up to 4e-6 at H = 4096, these by
// 1e-7), and the row's part of the loss.  A warp takes four entries at a time, so that eight
// loads of 512 bytes are in flight; the row of X stays in L1.
// Bound by the reads of the rows of W, 4.3 GB for 8192 tokens of 64 entries at H = 4096: 680 us
// alone.  So it is launched ahead of the forward GEMM, which does not read its results, and
// lets it start at once: two small blocks a SM find room beside the GEMM's and read
// while that computes (V = 128256, forward and backward: 20.77 -> 20.06 ms).
constexpr int kRowsThreads = 256, kRowsBlocks = 2;  // blocks of an SM
template <typename T>
__global__ void __launch_bounds__(kRowsThreads, 4) distill_rows(const __nv_bfloat16* X, const __nv_bfloat16* W,
                                                             const __grid_constant__ DistillParams p,
                                                             DistillRow* rows, unsigned* merged) {
  extern __shared__ float z_of[];  // two rows of K logits
  launch_dependents();
  if (blockIdx.x == 0 && threadIdx.x == 0) *merged = 0;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vectors = p.H / 8;
  constexpr int U = 4, kWarps = kRowsThreads / 32;
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x, ++turn) {
    const uint4* x_row = reinterpret_cast<const uint4*>(X + row * p.H);
    float* z = z_of + (turn & 1) * p.K;
    for (int k0 = warp * U; k0 < p.K; k0 += kWarps * U) {
      const uint4* w[U];
      bool live[U];
      uint64_t sum[U];
      int64_t any = -1;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t id = k0 + u < p.K ? p.ids[row * p.K + k0 + u] : -1;
        live[u] = id >= 0 && id < p.V;
        if (live[u]) any = id;
        w[u] = reinterpret_cast<const uint4*>(W + (live[u] ? id : 0) * p.H);
        sum[u] = 0;
      }
      // loads without branches between them: what is no entry reads another's row (2001 tokens, 6%
      // without entries and others with few: 213 -> 211 us; all read row 0 before)
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (!live[u]) w[u] = reinterpret_cast<const uint4*>(W + any * p.H);
      auto step = [&](int i) {
        const uint4 x = x_row[i];
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] = ld_stream_v4(w[u] + i);
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t vs[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sum[u] = fma_f32x2(pack_u32x2(xs[j] << 16, xs[j] & 0xffff0000u),
                               pack_u32x2(vs[j] << 16, vs[j] & 0xffff0000u), sum[u]);
        }
      };
      if (any >= 0)
#pragma unroll 2
        for (int i = lane; i < vectors; i += 32) step(i);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float a, b;
        unpack_f32x2(sum[u], a, b);
        const float s = live[u] ? warp_sum(a + b) : 0.f;
        if (lane == 0 && k0 + u < p.K) {
          p.logits[row * p.K + k0 + u] = s;
          z[k0 + u] = s;
        }
      }
    }
    __syncthreads();
    // one warp has the rest of the row; the others go on to the next, whose logits lie elsewhere
    if (turn % kWarps != warp) continue;
    const TeacherRow tr = teacher_row<T>(p, row, lane);
    if (tr.error && lane == 0) record_error(p.err_word, kErrLabel);
    float rest = 0.f;
    for (int k = lane; k < p.K; k += 32) {
      const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr);
      if (tr.valid && entry(p.ids[row * p.K + k], t)) {
        const float u = tr.scaled(t, p.inv_t), q = expf(u - tr.tl);
        if (!(q == 0.f)) rest = fmaf(q, u - z[k] * p.inv_t, rest);
      }
    }
    rest = warp_sum(rest);
    if (lane == 0) rows[row] = DistillRow{rest, tr.tl, tr.Q, tr.valid};
  }
}

// lse of each row from the vocabulary groups' partials, and its loss: a block MERGE_ROWS rows,
// as lse_merge_kernel, but a warp for every 32nd group: with few tokens there are few
// blocks, and each waits for its reads (64 tokens, 501 groups: 30 -> 10 us).  The block that
// ends last adds the blocks' sums.  All orders are fixed, whichever that is.
constexpr int kMergeWarps = 32;
__global__ void __launch_bounds__(32 * kMergeWarps)
    distill_merge(const float4* __restrict__ partials, int n_groups, int m_pad, int N,
                  const DistillRow* __restrict__ rows, float* __restrict__ lse_out, float* __restrict__ row_loss,
                  double* block_loss, int* block_valid, unsigned* merged, int reduction_sum,
                  float* __restrict__ loss_out, int* __restrict__ valid_out) {
  __shared__ float2 part[kMergeWarps][MERGE_ROWS];
  __shared__ double loss_of[kMergeWarps];
  __shared__ int valid_of[kMergeWarps];
  __shared__ bool last;
  const int r = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int row = blockIdx.x * MERGE_ROWS + r;
  grid_wait();
  float m = -INFINITY, sum = 0.f;
  if (row < N)
#pragma unroll 4
    for (int g = warp; g < n_groups; g += kMergeWarps) {
      const float4 q = partials[(size_t)g * m_pad + row];
      const float top = fmaxf(m, q.x);  // above -infinity, as every group's maximum is
      sum = sum * ex2_approx(m - top) + q.y * ex2_approx(q.x - top);
      m = top;
    }
  part[warp][r] = make_float2(m, sum);
  __syncthreads();
  double loss = 0.0;
  int valid = 0;
  auto warp_total = [&] {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      loss += __shfl_xor_sync(~0u, loss, o);
      valid += __shfl_xor_sync(~0u, valid, o);
    }
  };
  if (warp == 0) {
    if (row < N) {
      float top = -INFINITY, total = 0.f;
#pragma unroll
      for (int k = 0; k < kMergeWarps; ++k) top = fmaxf(top, part[k][r].x);
#pragma unroll
      for (int k = 0; k < kMergeWarps; ++k)
        total += part[k][r].y * ex2_approx(part[k][r].x - top);  // a warp without groups has 0 at -infinity
      const float lse = (top + log2f(total)) * LN2;
      lse_out[row] = lse;
      const DistillRow d = rows[row];
      valid = d.valid;
      if (valid) {
        loss = d.rest;
        if (!(d.Q == 0.f)) loss += (double)d.Q * (double)(lse - d.tl);
      }
      if (row_loss) row_loss[row] = (float)loss;
    }
    warp_total();
    if (r == 0) {
      block_loss[blockIdx.x] = loss;
      block_valid[blockIdx.x] = valid;
      __threadfence();
      last = atomicAdd(merged, 1u) == gridDim.x - 1;
    }
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  loss = 0.0;
  valid = 0;
  for (int b = threadIdx.x; b < gridDim.x; b += 32 * kMergeWarps) {
    loss += __ldcg(block_loss + b);
    valid += __ldcg(block_valid + b);
  }
  warp_total();
  if (r == 0) loss_of[warp] = loss, valid_of[warp] = valid;
  __syncthreads();
  if (warp) return;
  loss = loss_of[r];
  valid = valid_of[r];
  warp_total();
  if (r == 0) {
    *loss_out = (float)(reduction_sum ? loss : valid > 0 ? loss / (double)valid : 0.0);
    *valid_out = valid;
  }
}

// Which rows count, as bits of groups of 64: a block a group, a warp eight rows.
constexpr int kGroup = 64;
template <typename T>
__global__ void __launch_bounds__(256) distill_flags(const __grid_constant__ DistillParams p,
                                                     unsigned long long* __restrict__ masks) {
  __shared__ unsigned char bits[kGroup / 8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_wait();
  unsigned mine = 0;
  for (int i = 0; i < 8; ++i) {
    const int64_t row = (int64_t)blockIdx.x * kGroup + warp * 8 + i;
    bool any = false, bad = false;
    if (row < p.N)
      for (int k = lane; k < p.K; k += 32) {
        const int64_t id = p.ids[row * p.K + k];
        bad |= id >= p.V;
        any |= entry(id, teacher_logit(p, row * p.K + k, (const T*)nullptr));
      }
    if (__any_sync(~0u, any) && !__any_sync(~0u, bad)) mine |= 1u << i;
  }
  if (lane == 0) bits[warp] = (unsigned char)mine;
  __syncthreads();
  if (threadIdx.x) return;
  unsigned long long m = 0;
#pragma unroll
  for (int w = 0; w < kGroup / 8; ++w) m |= (unsigned long long)bits[w] << (8 * w);
  masks[blockIdx.x] = m;
}

// Backward, a warp a row.  The rows that count come first, in their order, the others behind
// them: the GEMMs then walk the former alone (their number is live[0]), and 10% of tokens
// without entries are 10% less work, wherever they lie.  For a row's place, what the GEMM core
// needs: its X, the mark V of a row with a softmax term or -1, and lse - log Q, so that this
// term is Q p; and dZ at each entry, c / T (Q p - sum of q of the same id), formed in fp32
// from the forward's logit and rounded once: the difference of nearly equal p and q keeps its
// digits.  8192 tokens, H = 4096, 64 entries: 30 us, 134 MB of X in and out and chains of reads.
constexpr int kPrepareThreads = 128;
struct DistillPlaces {
  const unsigned long long* masks;
  int* live;      // rows that count
  int* place;     // N: of each row, or -1 - place of one that does not count
  uint4* X;       // by place
  int64_t* marks;
  float* lse_q;
  int* ids;       // N x K; -1: no entry
  uint16_t* dz;
  float* scale;   // c / T
};
template <typename T>
__global__ void __launch_bounds__(kPrepareThreads)
    distill_prepare(const __nv_bfloat16* __restrict__ X, const __grid_constant__ DistillParams p,
                    const float* __restrict__ lse, const int* __restrict__ valid_count,
                    const float* __restrict__ grad_loss, int reduction_sum, const DistillPlaces out) {
  extern __shared__ int shared[];  // each warp: K ids, K probabilities
  __shared__ int counts[2][kPrepareThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int* id_of = shared + warp * 2 * p.K;
  float* q_of = reinterpret_cast<float*>(id_of + p.K);
  grid_wait();
  const float g = grad_loss ? *grad_loss : 1.f;
  const int nv = reduction_sum ? 1 : *valid_count;
  const float c = nv > 0 ? (float)((double)g * (double)p.inv_t / (double)nv) : 0.f;
  // rows that count: in the groups before this block's, and in all
  const int64_t row0 = (int64_t)blockIdx.x * (kPrepareThreads / 32);
  const int groups = (p.N + kGroup - 1) / kGroup, group = (int)(row0 / kGroup);
  int before = 0, all = 0;
  for (int i = threadIdx.x; i < groups; i += kPrepareThreads) {
    const int n = __popcll(out.masks[i]);
    all += n;
    before += i < group ? n : 0;
  }
  before = __reduce_add_sync(~0u, before);
  all = __reduce_add_sync(~0u, all);
  if (lane == 0) counts[0][warp] = before, counts[1][warp] = all;
  __syncthreads();
  before = all = 0;
#pragma unroll
  for (int i = 0; i < kPrepareThreads / 32; ++i) before += counts[0][i], all += counts[1][i];
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *out.scale = c;
    *out.live = all;
  }
  const int64_t row = row0 + warp;
  if (row >= p.N) return;
  const unsigned long long mask = out.masks[group];
  const int in_group = (int)(row % kGroup);
  const bool counts_here = mask >> in_group & 1;
  const int rank = before + __popcll(mask & ((1ull << in_group) - 1));
  int64_t place = counts_here ? rank : all + ((int)row - rank);
  if (!dbg_ok(place >= 0 && place < p.N, p.err_word)) place = 0;
  const uint4* from = reinterpret_cast<const uint4*>(X + row * p.H);
  uint4* to = out.X + place * (p.H / 8);
#pragma unroll 8
  for (int i = lane; i < p.H / 8; i += 32) to[i] = from[i];
  const TeacherRow tr = teacher_row<T>(p, row, lane);
  for (int k = lane; k < p.K; k += 32) {
    const int64_t id = p.ids[row * p.K + k];
    const float t = teacher_logit(p, row * p.K + k, (const T*)nullptr);
    const bool in = counts_here && entry(id, t);
    id_of[k] = in ? (int)id : -1;
    q_of[k] = in ? expf(tr.scaled(t, p.inv_t) - tr.tl) : 0.f;
  }
  __syncwarp();
  const float l = lse[row];
  // a row whose entries all have probability 0 counts, but has no softmax term (its log Q is none)
  const bool weighs = counts_here && !(tr.Q == 0.f);
  if (lane == 0) {
    out.place[row] = counts_here ? (int)place : -1 - (int)place;
    out.marks[place] = weighs ? p.V : -1;
    // without a term, lse itself: its exponentials are taken all the same where the scale is
    // negative, and have to be finite before they are multiplied by 0
    out.lse_q[place] = weighs ? l - logf(tr.Q) : l;
  }
  for (int k = lane; k < p.K; k += 32) {
    const int id = id_of[k];
    float same = 0.f;
    for (int j = 0; j < p.K; ++j) same += id_of[j] == id ? q_of[j] : 0.f;
    const float d = fmaf(tr.Q, expf(p.logits[row * p.K + k] * p.inv_t - l), -same);
    out.ids[place * p.K + k] = id;
    out.dz[place * p.K + k] = __bfloat16_as_ushort(__float2bfloat16_rn(c * d));
  }
}

// dX of each row from its place in the fp32 sums, of k_parts parts `pitch` values apart, added
// in their order; zero for a row that does not count.  A block a row: 201 MB of 8192 rows of 4096
// in 26 us, HBM.
__global__ void __launch_bounds__(256) distill_dx(const float4* __restrict__ sums, int k_parts, int64_t pitch4,
                                                  const int* __restrict__ place, int vectors,
                                                  uint2* __restrict__ dX) {
  grid_wait();
  const int at = place[blockIdx.x];
  const float4* from = sums + (int64_t)at * vectors;
  uint2* to = dX + (int64_t)blockIdx.x * vectors;
  for (int i = threadIdx.x; i < vectors; i += 256) {
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    if (at >= 0) {
      t = from[i];
#pragma unroll 4
      for (int k = 1; k < k_parts; ++k) {
        const float4 v = from[k * pitch4 + i];
        t.x += v.x, t.y += v.y, t.z += v.z, t.w += v.w;
      }
    }
    to[i] = make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
  }
}

// The entries of a vocabulary chunk put into its dZ, which holds the softmax term there: reads
// of all ids from L2 and a few scattered writes, 5 us for 8192 tokens of 64.
__global__ void __launch_bounds__(256) distill_scatter(const int* __restrict__ ids32, const uint16_t* __restrict__ dz,
                                                       int64_t entries, int K, int v0, int width, int64_t pitch,
                                                       uint16_t* __restrict__ chunk) {
  grid_wait();
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < entries; i += (int64_t)gridDim.x * 256) {
    const int at = ids32[i] - v0;
    if (ids32[i] >= 0 && at >= 0 && at < width) chunk[i / K * pitch + at] = dz[i];
  }
}

}  // namespace flce
