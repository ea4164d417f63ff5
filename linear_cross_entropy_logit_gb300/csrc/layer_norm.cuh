// Layer norm and RMS norm of rows, with the residual sum in front of it, and
// its backward.
//   forward   s = x + residual (rounded to the type and stored: what is normed)
//             n = (s - mu) r,  mu = mean(s) or 0 (RMS),
//             r = 1 / sqrt(mean((s - mu)^2) + eps),  y = w n + b
//   backward  dx = r (g w - mean(g w) - n mean(g w n)) + ds   (RMS: without mean(g w)),
//             dw = sum over rows of g n,  db = sum over rows of g
//
// A few flops per value: bound by HBM.  Persistent blocks, a row at a time shared by a
// block's threads, the next rows on their way to shared memory.  The variance is summed from
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

constexpr int kLayerNormThreads = 512;  // at most

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
};

// Sums over the block of K values, the same in every thread.  `shared` holds 32 K floats
// that no thread still reads.
template <int K>
__device__ __forceinline__ void block_sum(float (&x)[K], float (*shared)[K]) {
  auto warp = [&] {
#pragma unroll
    for (int o = 16; o; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(~0u, x[k], o);
  };
  warp();
  if (blockDim.x == 32) return;
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (lane == 0) shared[threadIdx.x >> 5][k] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) x[k] = lane < blockDim.x >> 5 ? shared[lane][k] : 0.f;
  warp();
}

// The rows of a persistent block that are on their way, each of `arrays` arrays, in shared
// memory.  A thread copies the vectors that it reads itself, so that nothing waits for
// another thread, and no registers are held for them.
template <int C>
struct RowRing {
  uint4* mine;
  int vectors, arrays;
  __device__ __forceinline__ RowRing(uint4* ring, int vectors, int arrays)
      : mine(ring + threadIdx.x), vectors(vectors), arrays(arrays) {}
  __device__ __forceinline__ uint4* at(int s, int array, int c) const {
    return mine + ((s * arrays + array) * C + c) * blockDim.x;
  }
  __device__ __forceinline__ void fetch(int s, int array, const void* row) const {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i < vectors) cp_async<16>(at(s, array, c), static_cast<const uint4*>(row) + i);
    }
  }
};

// Persistent over rows, C vectors of a row a thread, STAGES rows in the ring.
template <typename T, int C, int STAGES, bool CENTER>
__global__ void __launch_bounds__(kLayerNormThreads) layer_norm_fwd(const __grid_constant__ LayerNormParams p) {
  extern __shared__ uint4 ring_space[];
  __shared__ float shared[2][2][32][1];
  constexpr int N = Vec<T>::N;
  RowRing<C> ring(ring_space, p.vectors, p.residual ? 2 : 1);
  auto fetch = [&](int s, int64_t row) {
    if (row < p.rows) {
      ring.fetch(s, 0, static_cast<const T*>(p.x) + row * p.x_row);
      if (p.residual) ring.fetch(s, 1, static_cast<const T*>(p.residual) + row * p.residual_row);
    }
    cp_async_commit();
  };
  grid_wait();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s, blockIdx.x + (int64_t)s * gridDim.x);
  int stage = 0, parity = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    fetch((stage + STAGES - 1) % STAGES, row + (STAGES - 1) * (int64_t)gridDim.x);
    cp_async_wait<STAGES - 1>();
    Vec<T> v[C];
    float sum[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) {
        v[c].fill(0.f);
        continue;
      }
      v[c].load(ring.at(stage, 0, c), 0);
      if (p.residual) {
        Vec<T> e;
        e.load(ring.at(stage, 1, c), 0);
#pragma unroll
        for (int j = 0; j < N; ++j) v[c].f[j] += e.f[j];
        const uint4 stored = v[c].packed();
        static_cast<uint4*>(p.sum)[row * p.vectors + i] = stored;
        v[c].load(&stored, 0);
      }
      if (CENTER)
#pragma unroll
        for (int j = 0; j < N; ++j) sum[0] += v[c].f[j];
    }
    float mean = 0.f;
    if constexpr (CENTER) {
      block_sum(sum, shared[parity][0]);
      mean = sum[0] * p.inv_cols;
    }
    float square[1] = {0.f};
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const bool in = c * blockDim.x + threadIdx.x < p.vectors;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        v[c].f[j] -= mean;
        if (in) square[0] = fmaf(v[c].f[j], v[c].f[j], square[0]);
      }
    }
    block_sum(square, shared[parity][1]);
    const float r = rsqrtf(square[0] * p.inv_cols + p.eps);
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
      for (int j = 0; j < N; ++j) v[c].f[j] = fmaf(v[c].f[j] * r, w.f[j], b.f[j]);
      v[c].store(p.out, row * p.vectors + i);
    }
    if (threadIdx.x == 0) {
      if (CENTER) p.mean[row] = mean;
      p.rstd[row] = r;
    }
    stage = (stage + 1) % STAGES;
    parity ^= 1;
  }
}

// Persistent over rows: a thread has the same columns of each, so that the weights'
// gradients are summed in its registers, in the order of the rows; one partial row per
// block goes to the workspace.  No atomics: results do not change run to run.  The row is
// read from the ring twice, before and after its sums, instead of being held.
template <typename T, int C, int STAGES, bool CENTER, bool BIAS>
__global__ void __launch_bounds__(kLayerNormThreads) layer_norm_bwd(const __grid_constant__ LayerNormParams p) {
  extern __shared__ uint4 ring_space[];
  constexpr int K = CENTER ? 2 : 1, N = Vec<T>::N;
  __shared__ float shared[2][32][K];
  RowRing<C> ring(ring_space, p.vectors, p.ds ? 3 : 2);
  auto fetch = [&](int s, int64_t row) {
    if (row < p.rows) {
      ring.fetch(s, 0, static_cast<const T*>(p.x) + row * p.x_row);
      ring.fetch(s, 1, static_cast<const uint4*>(p.dy) + row * p.vectors);
      if (p.ds) ring.fetch(s, 2, static_cast<const uint4*>(p.ds) + row * p.vectors);
    }
    cp_async_commit();
  };
  float dw[C][N] = {}, db[BIAS ? C : 1][N] = {};
  grid_wait();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s, blockIdx.x + (int64_t)s * gridDim.x);
  int stage = 0, parity = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    fetch((stage + STAGES - 1) % STAGES, row + (STAGES - 1) * (int64_t)gridDim.x);
    const float mean = CENTER ? p.mean[row] : 0.f, r = p.rstd[row];
    cp_async_wait<STAGES - 1>();
    float sum[K] = {};  // of g w n, and of g w
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) continue;
      Vec<T> x, g, w;
      x.load(ring.at(stage, 0, c), 0);
      g.load(ring.at(stage, 1, c), 0);
      if (p.w)
        w.load(p.w, i);
      else
        w.fill(1.f);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float n = (x.f[j] - mean) * r, gw = g.f[j] * w.f[j];
        dw[c][j] = fmaf(g.f[j], n, dw[c][j]);
        if (BIAS) db[c][j] += g.f[j];
        sum[0] = fmaf(gw, n, sum[0]);
        if (CENTER) sum[K - 1] += gw;
      }
    }
    block_sum(sum, shared[parity]);
    const float along = sum[0] * p.inv_cols, level = CENTER ? sum[K - 1] * p.inv_cols : 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) continue;
      Vec<T> x, g, w, d;
      x.load(ring.at(stage, 0, c), 0);
      g.load(ring.at(stage, 1, c), 0);
      if (p.w)
        w.load(p.w, i);
      else
        w.fill(1.f);
      if (p.ds)
        d.load(ring.at(stage, 2, c), 0);
      else
        d.fill(0.f);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float n = (x.f[j] - mean) * r;
        d.f[j] = fmaf(r, fmaf(g.f[j], w.f[j], -level) - n * along, d.f[j]);
      }
      d.store(p.out, row * p.vectors + i);
    }
    stage = (stage + 1) % STAGES;
    parity ^= 1;
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
