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

// 16 bytes as floats, packed in twos.
template <typename T>
struct Vec {
  static constexpr int N = 16 / sizeof(T), H = N / 2;
  uint64_t f[H];
  __device__ __forceinline__ void unpack(const uint4& v) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < H; ++j)
      f[j] = sizeof(T) == 4 ? pack_u32x2(u[2 * j], u[2 * j + 1]) : pack_u32x2(u[j] << 16, u[j] & 0xffff0000u);
  }
  __device__ __forceinline__ void load(const void* p, int64_t i) { unpack(static_cast<const uint4*>(p)[i]); }
  __device__ __forceinline__ void fill(float x) {
#pragma unroll
    for (int j = 0; j < H; ++j) f[j] = pack_f32x2(x, x);
  }
  __device__ __forceinline__ uint4 packed() const {
    uint32_t u[4];
#pragma unroll
    for (int j = 0; j < H; ++j) {
      float a, b;
      unpack_f32x2(f[j], a, b);
      if constexpr (sizeof(T) == 4)
        u[2 * j] = __float_as_uint(a), u[2 * j + 1] = __float_as_uint(b);
      else
        u[j] = pack_bf16x2(a, b);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
};
__device__ __forceinline__ float halves(uint64_t x) {
  float a, b;
  unpack_f32x2(x, a, b);
  return a + b;
}
__device__ __forceinline__ float lanes(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Two values of each warp, those of warp i in lane i of every warp, zeros in the other
// lanes.  Two calls in a row use different `shared`; the barrier of the second tells that
// the first has been read.
constexpr int kLayerNormWarps = kLayerNormThreads / 32;
__device__ __forceinline__ float2 warp_pairs(float a, float b, float2* shared) {
  const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (warps == 1) return lane ? make_float2(0.f, 0.f) : make_float2(a, b);
  if (lane == 0) shared[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
  return lane < warps ? shared[lane] : make_float2(0.f, 0.f);
}
// Their sums, of ROWS rows.  Every lane reads them, two warps at a time, and adds: shorter than
// the tree of shuffles that the forward's weighted sums take (backward of 8192 rows of 4096,
// bf16: 48 -> 43 us).  `shared` has zeros behind an odd last warp.
template <int ROWS>
__device__ __forceinline__ void warp_pairs_sum(float2 (&x)[ROWS], float2 (*shared)[kLayerNormWarps]) {
  const int warps = blockDim.x >> 5;
  if (warps == 1) return;
#pragma unroll
  for (int k = 0; k < ROWS; ++k)
    if ((threadIdx.x & 31) == 0) shared[k][threadIdx.x >> 5] = x[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < ROWS; ++k) x[k] = make_float2(0.f, 0.f);
  for (int i = 0; i < warps; i += 2)
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const float4 q = *reinterpret_cast<const float4*>(&shared[k][i]);
      x[k].x += q.x + q.z;
      x[k].y += q.y + q.w;
    }
}

// The rows of a persistent block that are on their way, A arrays of each (the last if it is
// there), in shared memory.  A thread copies the vectors that it reads itself, so that
// nothing waits for another thread, and no registers are held for them.  Neighbouring
// threads' vectors are neighbours there too: with a thread's own vectors together the
// copies are three times slower.
template <int C, int STAGES, int A, bool FULL = false>
struct RowRing {
  uint4* mine;        // this thread's first vector
  int in = 0, out = 0, stage;  // vectors: the stage to fill and to read next, and from one to the next
  const uint4* from[A];
  int64_t step[A];    // from a row of this block to the next
  int left;           // rows not yet fetched
  int vectors;
  bool last;          // the last array is there
  __device__ __forceinline__ RowRing(uint4* ring, const LayerNormParams& p, bool last)
      : mine(ring + threadIdx.x), stage((last ? A : A - 1) * C * blockDim.x), vectors(p.vectors), last(last) {
    left = p.rows > blockIdx.x ? (int)((p.rows - blockIdx.x + gridDim.x - 1) / gridDim.x) : 0;
  }
  // row_vectors: from a row of the array to the next, in vectors
  __device__ __forceinline__ void source(int a, const void* p, int64_t row_vectors) {
    from[a] = static_cast<const uint4*>(p) + blockIdx.x * row_vectors + threadIdx.x;
    step[a] = gridDim.x * row_vectors;
  }
  __device__ __forceinline__ void fetch() {
    if (left > 0) {
#pragma unroll
      for (int a = 0; a < A; ++a) {
        if (a + 1 == A && !last) continue;
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (FULL || c * blockDim.x + threadIdx.x < vectors)
            cp_async<16>(mine + in + (a * C + c) * blockDim.x, from[a] + c * blockDim.x);
        from[a] += step[a];
      }
      --left;
    }
    cp_async_commit();
    in = in + stage == STAGES * stage ? 0 : in + stage;
  }
  __device__ __forceinline__ const uint4& at(int a, int c, int row = 0) const {
    return mine[out + row * stage + (a * C + c) * blockDim.x];
  }
  __device__ __forceinline__ void next(int rows = 1) {
    out = out + rows * stage == STAGES * stage ? 0 : out + rows * stage;
  }
};

// A thread's columns of the weight or the bias: held in registers where there are few, else
// read again for each row.
template <typename T, int C>
struct Columns {
  static constexpr bool kHeld = C * Vec<T>::N <= 16;
  const void* p;
  float missing;
  Vec<T> held[kHeld ? C : 1];
  __device__ __forceinline__ void take(Vec<T>& v, int c, int vectors) const {
    const int i = c * blockDim.x + threadIdx.x;
    if (p && i < vectors)
      v.load(p, i);
    else
      v.fill(missing);
  }
  __device__ __forceinline__ Columns(const void* p, float missing, int vectors) : p(p), missing(missing) {
    if constexpr (kHeld) {
#pragma unroll
      for (int c = 0; c < C; ++c) take(held[c], c, vectors);
    }
  }
  __device__ __forceinline__ Vec<T> at(int c, int vectors) const {
    if constexpr (kHeld) return held[c];
    Vec<T> v;
    take(v, c, vectors);
    return v;
  }
};

// Persistent over rows, C vectors of a row a thread, STAGES rows in the ring.  Each warp takes
// its own part's mean m_w and sum of squares s_w around it; the row's are
//   mean = sum n_w m_w / n,   sum s_w + sum n_w (m_w - mean)^2:
// one barrier a row, and nothing cancels.  16384 rows of 4096 in bf16, RMS with a residual: 537 MB
// in 79.4 us, 6760 GB/s; 8192 rows, layer norm: 134 MB in 25.5, 5260, where barriers and issue
// (54%) of three rows a SM count too.
template <typename T, int C, int STAGES, bool CENTER>
__global__ void __maxnreg__(80) layer_norm_fwd(const __grid_constant__ LayerNormParams p) {
  extern __shared__ uint4 ring_space[];
  __shared__ float2 shared[2][kLayerNormWarps];
  __shared__ float share[kLayerNormWarps];  // n_w / n
  constexpr int H = Vec<T>::H;
  RowRing<C, STAGES, 2> ring(ring_space, p, p.residual != nullptr);
  ring.source(0, p.x, p.x_row / Vec<T>::N);
  ring.source(1, p.residual, p.residual_row / Vec<T>::N);
  float count = 0.f;  // values of this warp
#pragma unroll
  for (int c = 0; c < C; ++c)
    count += Vec<T>::N * min(32, max(0, p.vectors - (c * (int)blockDim.x + ((int)threadIdx.x & ~31))));
  const float inv_count = count > 0.f ? 1.f / count : 0.f;
  if ((threadIdx.x & 31) == 0) share[threadIdx.x >> 5] = count * p.inv_cols;
  __syncthreads();
  const float share_of_lane = (threadIdx.x & 31) < blockDim.x >> 5 ? share[threadIdx.x & 31] : 0.f;
  grid_wait();
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) ring.fetch();
  const Columns<T, C> weight(p.w, 1.f, p.vectors), bias(p.b, 0.f, p.vectors);
  const int64_t out_step = (int64_t)gridDim.x * p.vectors;
  uint4* out = static_cast<uint4*>(p.out) + (int64_t)blockIdx.x * p.vectors + threadIdx.x;
  uint4* sum_out = static_cast<uint4*>(p.sum) + (int64_t)blockIdx.x * p.vectors + threadIdx.x;
  int parity = 0;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    ring.fetch();
    cp_async_wait<STAGES - 1>();
    Vec<T> v[C];
    uint64_t sum = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) {
        v[c].fill(0.f);
        continue;
      }
      v[c].unpack(ring.at(0, c));
      if (p.residual) {
        Vec<T> e;
        e.unpack(ring.at(1, c));
#pragma unroll
        for (int j = 0; j < H; ++j) v[c].f[j] = add_f32x2(v[c].f[j], e.f[j]);
        const uint4 stored = v[c].packed();
        sum_out[c * blockDim.x] = stored;
        v[c].unpack(stored);
      }
      if (CENTER)
#pragma unroll
        for (int j = 0; j < H; ++j) sum = add_f32x2(sum, v[c].f[j]);
    }
    const float part = CENTER ? lanes(halves(sum)) * inv_count : 0.f;
    const uint64_t minus = pack_f32x2(-part, -part);
    uint64_t square = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      if (c * blockDim.x + threadIdx.x >= p.vectors) continue;
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const uint64_t d = CENTER ? add_f32x2(v[c].f[j], minus) : v[c].f[j];
        square = fma_f32x2(d, d, square);
      }
    }
    const float2 w = warp_pairs(part, lanes(halves(square)), shared[parity]);
    const float mean = CENTER ? lanes(share_of_lane * w.x) : 0.f, off = w.x - mean;
    const float total = lanes(CENTER ? fmaf(share_of_lane * off, off, w.y * p.inv_cols) : w.y * p.inv_cols);
    const float r = rsqrtf(total + p.eps);
    const uint64_t r2 = pack_f32x2(r, r), m2 = pack_f32x2(-mean, -mean);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int i = c * blockDim.x + threadIdx.x;
      if (i >= p.vectors) continue;
      const Vec<T> wc = weight.at(c, p.vectors), bc = bias.at(c, p.vectors);
#pragma unroll
      for (int j = 0; j < H; ++j) {
        const uint64_t d = CENTER ? add_f32x2(v[c].f[j], m2) : v[c].f[j];
        v[c].f[j] = fma_f32x2(mul_f32x2(d, r2), wc.f[j], bc.f[j]);
      }
      out[c * blockDim.x] = v[c].packed();
    }
    if (threadIdx.x == 0) {
      if (CENTER) p.mean[row] = mean;
      p.rstd[row] = r;
    }
    ring.next();
    out += out_step;
    sum_out += out_step;
    parity ^= 1;
  }
}

// Persistent over rows: a thread has the same columns of each, so that the weights'
// gradients are summed in its registers, in the order of the rows; one partial row per
// block goes to the workspace.  No atomics: results do not change run to run.  8192 rows of
// 4096 in bf16: 201 MB, and 10 of partial rows, in 37 us, 5700 GB/s: two rows at once a SM, as
// many as the sums' registers leave room for.  ROWS rows share
// a barrier: what one waits for, the other computes.  n and g w are made a second time, from
// the ring, instead of being held over it.  FULL: the row fills C vectors of every thread, none is
// asked whether it is there (16384 rows of 4096 in bf16, RMS: 75 -> 69 us; not taken for floats,
// 30000 rows of 1024: 75 -> 79).
template <typename T, int C, int STAGES, int ROWS, bool CENTER, bool BIAS, bool FULL>
__global__ void __launch_bounds__(kLayerNormThreads) layer_norm_bwd(const __grid_constant__ LayerNormParams p) {
  extern __shared__ uint4 ring_space[];
  __shared__ __align__(16) float2 shared[2][ROWS][kLayerNormWarps];
  constexpr int H = Vec<T>::H;
  static_assert(STAGES % ROWS == 0, "the rows of a turn lie together");
  RowRing<C, STAGES, 3, FULL> ring(ring_space, p, p.ds != nullptr);
  ring.source(0, p.x, p.x_row / Vec<T>::N);
  ring.source(1, p.dy, p.vectors);
  ring.source(2, p.ds, p.vectors);
  uint64_t dw[C][H] = {}, db[BIAS ? C : 1][H] = {};
  if (blockDim.x & 32 && threadIdx.x < 2 * ROWS)  // an odd number of warps: behind the last
    shared[threadIdx.x & 1][threadIdx.x >> 1][blockDim.x >> 5] = make_float2(0.f, 0.f);
  grid_wait();
  const int rows = ring.left;
#pragma unroll
  for (int s = 0; s < STAGES - ROWS; ++s) ring.fetch();
  const Columns<T, C> weight(p.w, 1.f, p.vectors);
  const int64_t step = (int64_t)gridDim.x * p.vectors;
  uint4* out = static_cast<uint4*>(p.out) + (int64_t)blockIdx.x * p.vectors + threadIdx.x;
  const float *mean = p.mean + blockIdx.x, *rstd = p.rstd + blockIdx.x;
  float mean_next[ROWS], r_next[ROWS];  // of the rows after these, on their way
  auto next_stats = [&](int row) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const bool in = row + i < rows;
      mean_next[i] = CENTER && in ? mean[(int64_t)(row + i) * gridDim.x] : 0.f;
      r_next[i] = in ? rstd[(int64_t)(row + i) * gridDim.x] : 0.f;
    }
  };
  next_stats(0);
  int parity = 0;
  for (int row = 0; row < rows; row += ROWS) {
    uint64_t r2[ROWS], m2[ROWS], sn[ROWS] = {}, sg[ROWS] = {};  // sums of g w n, and of g w
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      ring.fetch();
      r2[i] = pack_f32x2(r_next[i], r_next[i]);
      m2[i] = pack_f32x2(-mean_next[i], -mean_next[i]);
    }
    next_stats(row + ROWS);
    cp_async_wait<STAGES - ROWS>();
    auto read = [&](int i, int c, Vec<T>& n, Vec<T>& g) {
      n.unpack(ring.at(0, c, i));
      g.unpack(ring.at(1, c, i));
#pragma unroll
      for (int j = 0; j < H; ++j) n.f[j] = mul_f32x2(CENTER ? add_f32x2(n.f[j], m2[i]) : n.f[j], r2[i]);
    };
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (i && row + i >= rows) break;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!FULL && c * blockDim.x + threadIdx.x >= p.vectors) continue;
        Vec<T> n, g;
        read(i, c, n, g);
        const Vec<T> w = weight.at(c, p.vectors);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          dw[c][j] = fma_f32x2(g.f[j], n.f[j], dw[c][j]);
          if (BIAS) db[c][j] = add_f32x2(db[c][j], g.f[j]);
          const uint64_t gw = mul_f32x2(g.f[j], w.f[j]);
          sn[i] = fma_f32x2(gw, n.f[j], sn[i]);
          if (CENTER) sg[i] = add_f32x2(sg[i], gw);
        }
      }
    }
    float2 sum[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
      sum[i] = make_float2(lanes(halves(sn[i])), CENTER ? lanes(halves(sg[i])) : 0.f);
    warp_pairs_sum(sum, shared[parity]);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (i && row + i >= rows) break;
      const float along = -sum[i].x * p.inv_cols, level = -sum[i].y * p.inv_cols;
      const uint64_t a2 = pack_f32x2(along, along), l2 = pack_f32x2(level, level);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (!FULL && c * blockDim.x + threadIdx.x >= p.vectors) continue;
        Vec<T> n, g, d;
        read(i, c, n, g);
        const Vec<T> w = weight.at(c, p.vectors);
        if (p.ds)
          d.unpack(ring.at(2, c, i));
        else
          d.fill(0.f);
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const uint64_t gw = CENTER ? fma_f32x2(g.f[j], w.f[j], l2) : mul_f32x2(g.f[j], w.f[j]);
          d.f[j] = fma_f32x2(r2[i], fma_f32x2(n.f[j], a2, gw), d.f[j]);
        }
        out[i * step + c * blockDim.x] = d.packed();
      }
    }
    ring.next(ROWS);
    out += ROWS * step;
    parity ^= 1;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int i = c * blockDim.x + threadIdx.x;
    if (i >= p.vectors) continue;
    const int64_t at = ((int64_t)blockIdx.x * p.vectors + i) * H;
#pragma unroll
    for (int j = 0; j < H; j += 2) {
      reinterpret_cast<ulonglong2*>(p.dw_partial)[(at + j) / 2] = make_ulonglong2(dw[c][j], dw[c][j + 1]);
      if (BIAS) reinterpret_cast<ulonglong2*>(p.db_partial)[(at + j) / 2] = make_ulonglong2(db[c][j], db[c][j + 1]);
    }
  }
}

// dw, db = sums of the blocks' partial rows: 32 columns a block, 32 rows at a time,
// added in a fixed order.  304 rows of 4096, twice: 10 MB from L2 in 5 us, mostly latency.
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
