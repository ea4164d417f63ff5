// RMS norm of each query and key head with the rotary position rotation in
// the same pass, and its backward.
//   forward   n = x r,  r = 1 / sqrt(mean(x^2) + eps),  y = R (w n)
//   backward  g = R^T dy,  dw = sum over tokens and heads of g n,
//             dx = r (g w - n mean(g w n))
// R turns pair j of the first `rot_dim` values by the angle whose cosine and
// sine are row `position` of the tables: pair (j, j + rot/2), or (2j, 2j+1)
// when interleaved; the other values pass through.
//
// About 10 flops per element against 4 bytes moved (bf16): bound by HBM.  A
// group of G lanes holds one head in registers, 8 values a lane, so every
// input is read once and the norm needs log2(G) shuffles and no shared
// memory.  A lane's 8 values are both halves of 4 pairs, so the rotation is
// lane-local.  A group takes kHeads heads of one token: that many independent
// loads are in flight, and the angles and the position are read once for them.
// All arithmetic is fp32; outputs are rounded once.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace flce {

struct QkNormRopeParams {
  const void *q, *k;            // inputs; row / head strides below
  const void *wq, *wk;          // head_dim weights, or null (ones)
  const float *cos_t, *sin_t;   // table_rows x rot/2
  const int64_t* positions;     // one per token, or null (0, 1, 2, ...)
  void *q_out, *k_out;          // contiguous; backward: dq, dk
  const void *dq_out, *dk_out;  // backward: contiguous output gradients
  float* partial;               // backward: gridDim.x x 2 x head_dim
  int64_t q_row, q_head, k_row, k_head;
  int64_t table_rows;
  int64_t items;                // tokens x blocks_per_token
  int blocks_per_token;         // blocks of kHeads heads
  int q_heads, kv_heads, head_dim, rot_dim;
  float eps, inv_dim;
  int* err_word;
};

constexpr int kNormThreads = 256;
constexpr int kNormHeads = 4;  // heads of a token a group takes at once

struct Vec8 {
  float x[8];
};

__device__ __forceinline__ void load4(float* x, const float* p) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load4(float* x, const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  x[0] = __uint_as_float(v.x << 16), x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16), x[3] = __uint_as_float(v.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]));
}

// Turns the lane's four pairs by +angle (forward) or -angle (backward).
template <bool PAIRS>
__device__ __forceinline__ void turn(Vec8& v, const float (&c)[4], const float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float& a = v.x[PAIRS ? 2 * i : i];
    float& b = v.x[PAIRS ? 2 * i + 1 : i + 4];
    const float u = a * c[i] - b * s[i];
    b = b * c[i] + a * s[i];
    a = u;
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// A lane's place in its head and its angles.
struct NormLane {
  int a0, a1;    // offsets of its two groups of four values
  bool in_head;  // head_dim covers this lane
  bool turns;    // its values are rotated
  int j;         // its first pair
};
template <bool PAIRS>
__device__ __forceinline__ NormLane norm_lane(const QkNormRopeParams& p, int l) {
  NormLane n;
  n.in_head = l * 8 < p.head_dim;
  n.turns = l * 8 < p.rot_dim;
  n.j = 4 * l;
  n.a0 = !PAIRS && n.turns ? 4 * l : 8 * l;
  n.a1 = !PAIRS && n.turns ? p.rot_dim / 2 + 4 * l : 8 * l + 4;
  return n;
}

__device__ __forceinline__ void norm_angles(const QkNormRopeParams& p, const NormLane& n,
                                            int64_t token, float (&c)[4], float (&s)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = 1.f, s[i] = 0.f;
  if (!n.turns) return;
  const int64_t pos = p.positions ? p.positions[token] : token;
  if (pos < 0 || pos >= p.table_rows) {  // left unrotated and reported
    record_error(p.err_word, kErrIndex);
    return;
  }
  load4(c, p.cos_t + pos * (p.rot_dim / 2) + n.j);
  load4(s, p.sin_t + pos * (p.rot_dim / 2) + n.j);
}

template <typename T>
__device__ __forceinline__ Vec8 norm_weight(const void* w, const NormLane& n) {
  Vec8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v.x[i] = 1.f;
  if (w && n.in_head) {
    load4(v.x, static_cast<const T*>(w) + n.a0);
    load4(v.x + 4, static_cast<const T*>(w) + n.a1);
  }
  return v;
}

template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_fwd(QkNormRopeParams p) {
  const NormLane n = norm_lane<PAIRS>(p, threadIdx.x % G);
  const int64_t item = (int64_t)blockIdx.x * (kNormThreads / G) + threadIdx.x / G;
  const bool live = item < p.items;
  const int64_t token = live ? item / p.blocks_per_token : 0;
  const int h0 = live ? (int)(item - token * p.blocks_per_token) * kNormHeads : 0;
  const int heads = live ? p.q_heads + p.kv_heads : 0;
  Vec8 x[kNormHeads];
#pragma unroll
  for (int u = 0; u < kNormHeads; ++u) {
    const int h = h0 + u;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u].x[i] = 0.f;
    if (h < heads && n.in_head) {
      const T* row = h < p.q_heads
                         ? static_cast<const T*>(p.q) + token * p.q_row + h * p.q_head
                         : static_cast<const T*>(p.k) + token * p.k_row +
                               (h - p.q_heads) * p.k_head;
      load4(x[u].x, row + n.a0);
      load4(x[u].x + 4, row + n.a1);
    }
  }
  float c[4], s[4];
  if (live) norm_angles(p, n, token, c, s);
  const Vec8 wq = norm_weight<T>(p.wq, n), wk = norm_weight<T>(p.wk, n);
#pragma unroll
  for (int u = 0; u < kNormHeads; ++u) {
    const int h = h0 + u;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[u].x[i], x[u].x[i], ss);
    const float r = rsqrtf(group_sum<G>(ss) * p.inv_dim + p.eps);
    if (h >= heads || !n.in_head) continue;
    const bool isq = h < p.q_heads;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[u].x[i] *= r * (isq ? wq.x[i] : wk.x[i]);
    if (n.turns) turn<PAIRS>(x[u], c, s);
    T* row = isq ? static_cast<T*>(p.q_out) + (token * p.q_heads + h) * p.head_dim
                 : static_cast<T*>(p.k_out) +
                       (token * p.kv_heads + (h - p.q_heads)) * p.head_dim;
    store4(row + n.a0, x[u].x);
    store4(row + n.a1, x[u].x + 4);
  }
}

// Persistent over items: each lane keeps the sums of its 8 weight gradients
// (query and key) in registers; the block adds its groups' sums in a fixed
// order and writes one partial row, so results do not change run to run.
template <typename T, int G, bool PAIRS>
__global__ void __launch_bounds__(kNormThreads) qk_norm_rope_bwd(QkNormRopeParams p) {
  constexpr int kGroups = kNormThreads / G;
  const int l = threadIdx.x % G;
  const NormLane n = norm_lane<PAIRS>(p, l);
  const Vec8 wq = norm_weight<T>(p.wq, n), wk = norm_weight<T>(p.wk, n);
  const int heads = p.q_heads + p.kv_heads;
  float dwq[8] = {}, dwk[8] = {};
  const int64_t stride = (int64_t)gridDim.x * kGroups;
  // every group of a warp runs the same number of rounds (the shuffles below
  // need the whole warp)
  for (int64_t base = (int64_t)blockIdx.x * kGroups; base < p.items; base += stride) {
    const int64_t item = base + threadIdx.x / G;
    const bool live = item < p.items;
    const int64_t token = live ? item / p.blocks_per_token : 0;
    const int h0 = live ? (int)(item - token * p.blocks_per_token) * kNormHeads : 0;
    Vec8 x[kNormHeads], g[kNormHeads];
#pragma unroll
    for (int u = 0; u < kNormHeads; ++u) {
      const int h = h0 + u;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[u].x[i] = g[u].x[i] = 0.f;
      if (live && h < heads && n.in_head) {
        const bool isq = h < p.q_heads;
        const T* row = isq ? static_cast<const T*>(p.q) + token * p.q_row + h * p.q_head
                           : static_cast<const T*>(p.k) + token * p.k_row +
                                 (h - p.q_heads) * p.k_head;
        const T* grow = isq ? static_cast<const T*>(p.dq_out) +
                                  (token * p.q_heads + h) * p.head_dim
                            : static_cast<const T*>(p.dk_out) +
                                  (token * p.kv_heads + (h - p.q_heads)) * p.head_dim;
        load4(x[u].x, row + n.a0);
        load4(x[u].x + 4, row + n.a1);
        load4(g[u].x, grow + n.a0);
        load4(g[u].x + 4, grow + n.a1);
      }
    }
    float c[4], s[4];
    norm_angles(p, n, token, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = -s[i];
#pragma unroll
    for (int u = 0; u < kNormHeads; ++u) {
      const int h = h0 + u;
      const bool isq = h < p.q_heads;
      if (n.turns) turn<PAIRS>(g[u], c, s);
      float ss = 0.f, gx = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        ss = fmaf(x[u].x[i], x[u].x[i], ss);
        gx = fmaf(g[u].x[i] * (isq ? wq.x[i] : wk.x[i]), x[u].x[i], gx);
      }
      const float r = rsqrtf(group_sum<G>(ss) * p.inv_dim + p.eps);
      const float mean = group_sum<G>(gx) * r * p.inv_dim;  // mean of g w n
      if (!live || h >= heads || !n.in_head) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float nx = x[u].x[i] * r;
        const float gn = g[u].x[i] * nx;
        dwq[i] += isq ? gn : 0.f;
        dwk[i] += isq ? 0.f : gn;
        x[u].x[i] = r * (g[u].x[i] * (isq ? wq.x[i] : wk.x[i]) - nx * mean);
      }
      T* row = isq ? static_cast<T*>(p.q_out) + (token * p.q_heads + h) * p.head_dim
                   : static_cast<T*>(p.k_out) +
                         (token * p.kv_heads + (h - p.q_heads)) * p.head_dim;
      store4(row + n.a0, x[u].x);
      store4(row + n.a1, x[u].x + 4);
    }
  }
  __shared__ float sums[kGroups][16 * G];
  float* mine = sums[threadIdx.x / G];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    mine[i * G + l] = dwq[i];
    mine[(8 + i) * G + l] = dwk[i];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 16 * G; e += kNormThreads) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kGroups; ++w) t += sums[w][e];
    const int which = e / (8 * G), i = e / G % 8, lane = e % G;
    const NormLane m = norm_lane<PAIRS>(p, lane);
    if (m.in_head)
      p.partial[((int64_t)blockIdx.x * 2 + which) * p.head_dim + (i < 4 ? m.a0 + i : m.a1 + i - 4)] = t;
  }
}

// dw = sum of the blocks' partial rows, 32 columns per block, 32 rows at a
// time, added in a fixed order.
__global__ void __launch_bounds__(1024) qk_norm_rope_dw(const float* partial, int rows,
                                                        int head_dim, float* dwq, float* dwk) {
  const int cols = 2 * head_dim;
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  float t = 0.f;
  if (c < cols)
#pragma unroll 4
    for (int r = w; r < rows; r += 32) t += partial[(int64_t)r * cols + c];
  __shared__ float sums[32][33];
  sums[w][threadIdx.x & 31] = t;
  __syncthreads();
  if (w || c >= cols) return;
  t = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
  (c < head_dim ? dwq[c] : dwk[c - head_dim]) = t;
}

}  // namespace flce
