// Layer norm and RMS norm of rows, with the residual sum in front of it, and
// its backward.
//   forward   s = x + residual (rounded to the type and stored: what is normed)
//             n = (s - mu) r,  mu = mean(s) or 0 (RMS),
//             r = 1 / sqrt(mean((s - mu)^2) + eps),  y = w n + b
//   backward  dx = r (g w - mean(g w) - n mean(g w n)) + ds   (RMS: without mean(g w)),
//             dw = sum over rows of g n,  db = sum over rows of g
//
// A few flops per value: bound by HBM.  A row is held in the registers of the
// threads that share it, so that it is read once and the variance is summed from
// differences to the mean.  All arithmetic is fp32; outputs are rounded once.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace flce {

struct LayerNormParams {
  const void *x, *residual;  // backward: x is the sum that was normed
  const void *w, *b;         // null: ones, zeros
  const void *dy, *ds;       // backward; ds may be null
  void *out, *sum;           // y or dx; the stored sum
  float *mean, *rstd;
  float *dw_partial, *db_partial;  // backward: a row of sums per block
  int64_t rows, x_row, residual_row;
  int vectors;               // 16-byte vectors of a row
  float eps, inv_cols;
};

// 16 bytes as floats.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T);
  float f[N];
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4 v = static_cast<const uint4*>(p)[i];
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (sizeof(T) == 4) {
        f[j] = __uint_as_float(u[j]);
      } else {
        f[2 * j] = __uint_as_float(u[j] << 16);
        f[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = x;
  }
  __device__ __forceinline__ uint4 packed() const {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      u[j] = sizeof(T) == 4 ? __float_as_uint(f[j]) : pack_bf16x2(f[2 * j], f[2 * j + 1]);
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const { static_cast<uint4*>(p)[i] = packed(); }
  // To the type and back.
  __device__ __forceinline__ void round() {
    if constexpr (sizeof(T) == 2) {
      const uint4 v = packed();
      load(&v, 0);
    }
  }
};

// Sum over the block, the same in every thread.  `shared` holds 32 floats that no
// thread still reads.
__device__ __forceinline__ float block_sum(float x, float* shared) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  if (blockDim.x == 32) return x;
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = x;
  __syncthreads();
  x = (threadIdx.x & 31) < blockDim.x >> 5 ? shared[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// A block a row, C vectors a thread.
template <typename T, int C, bool CENTER>
__global__ void __launch_bounds__(1024) layer_norm_fwd(const __grid_constant__ LayerNormParams p) {
  __shared__ float shared[2][32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(p.x) + row * p.x_row;
  grid_wait();
  Vec<T> v[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + threadIdx.x;
    if (i < p.vectors)
      v[c].load(x, i);
    else
      v[c].fill(0.f);
  }
  if (p.residual) {
    const T* r = static_cast<const T*>(p.residual) + row * p.residual_row;
    Vec<T> e[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i < p.vectors) e[c].load(r, i);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i < p.vectors) {
#pragma unroll
        for (int j = 0; j < Vec<T>::N; ++j) v[c].f[j] += e[c].f[j];
        v[c].round();
        v[c].store(p.sum, row * p.vectors + i);
      }
    }
  }
  float mean = 0.f;
  if constexpr (CENTER) {
    float t = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < Vec<T>::N; ++j) t += v[c].f[j];
    mean = block_sum(t, shared[0]) * p.inv_cols;
  }
  float t = 0.f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const bool in = c * blockDim.x + threadIdx.x < p.vectors;
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) {
      v[c].f[j] -= mean;
      if (in) t = fmaf(v[c].f[j], v[c].f[j], t);
    }
  }
  const float r = rsqrtf(block_sum(t, shared[1]) * p.inv_cols + p.eps);
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + threadIdx.x;
    if (i >= p.vectors) continue;
    Vec<T> w, b;
    if (p.w)
      w.load(p.w, i);
    else
      w.fill(1.f);
    if (p.b)
      b.load(p.b, i);
    else
      b.fill(0.f);
#pragma unroll
    for (int j = 0; j < Vec<T>::N; ++j) v[c].f[j] = fmaf(v[c].f[j] * r, w.f[j], b.f[j]);
    v[c].store(p.out, row * p.vectors + i);
  }
  if (threadIdx.x == 0) {
    if (CENTER) p.mean[row] = mean;
    p.rstd[row] = r;
  }
}

// Persistent over rows: a thread has the same columns of each, so that the weights'
// gradients are summed in its registers, in the order of the rows; one partial row per
// block goes to the workspace.  No atomics: results do not change run to run.
template <typename T, int C, bool CENTER, bool BIAS>
__global__ void __launch_bounds__(1024) layer_norm_bwd(const __grid_constant__ LayerNormParams p) {
  __shared__ float shared[2][2][32];
  constexpr int N = Vec<T>::N;
  float dw[C][N] = {}, db[BIAS ? C : 1][N] = {};
  grid_wait();
  int turn = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(p.x) + row * p.x_row;
    const float mean = CENTER ? p.mean[row] : 0.f, r = p.rstd[row];
    Vec<T> v[C], g[C];
    float gw = 0.f, gwn = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) continue;
      v[c].load(x, i);
      g[c].load(p.dy, row * p.vectors + i);
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) continue;
      Vec<T> w;
      if (p.w)
        w.load(p.w, i);
      else
        w.fill(1.f);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float n = (v[c].f[j] - mean) * r;
        dw[c][j] = fmaf(g[c].f[j], n, dw[c][j]);
        if (BIAS) db[c][j] += g[c].f[j];
        v[c].f[j] = n;
        g[c].f[j] *= w.f[j];
        if (CENTER) gw += g[c].f[j];
        gwn = fmaf(g[c].f[j], n, gwn);
      }
    }
    gwn = block_sum(gwn, shared[turn][0]) * p.inv_cols;
    if (CENTER) gw = block_sum(gw, shared[turn][1]) * p.inv_cols;
    turn ^= 1;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) continue;
      Vec<T> d;
      if (p.ds)
        d.load(p.ds, row * p.vectors + i);
      else
        d.fill(0.f);
#pragma unroll
      for (int j = 0; j < N; ++j) d.f[j] = fmaf(r, g[c].f[j] - gw * (CENTER ? 1.f : 0.f) - v[c].f[j] * gwn, d.f[j]);
      d.store(p.out, row * p.vectors + i);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + threadIdx.x;
    if (i >= p.vectors) continue;
    const int64_t at = ((int64_t)blockIdx.x * p.vectors + i) * N;
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      *reinterpret_cast<float4*>(p.dw_partial + at + j) = make_float4(dw[c][j], dw[c][j + 1], dw[c][j + 2], dw[c][j + 3]);
      if (BIAS)
        *reinterpret_cast<float4*>(p.db_partial + at + j) =
            make_float4(db[c][j], db[c][j + 1], db[c][j + 2], db[c][j + 3]);
    }
  }
}

// dw, db = sums of the blocks' partial rows: 32 columns a block, 32 rows at a time,
// added in a fixed order.
__global__ void __launch_bounds__(1024) layer_norm_dw(const float* dw_partial, const float* db_partial, int rows,
                                                      int cols, float* dw, float* db) {
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  const float* partial = blockIdx.y ? db_partial : dw_partial;
  float t = 0.f;
  grid_wait();
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
  (blockIdx.y ? db : dw)[c] = t;
}

}  // namespace flce
