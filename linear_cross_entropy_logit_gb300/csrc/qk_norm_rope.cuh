// RMS norm of each query and key head with the rotary position rotation in
// the same pass, and its backward.
//   forward   n = x r,  r = 1 / sqrt(mean(x^2) + eps),  y = R (w n)
//   backward  g = R^T dy,  dw = sum over tokens and heads of g n,
//             dx = r (g w - n mean(g w n))
// R turns pair j of the first `rot_dim` values by the angle whose cosine and
// sine are row `position` of the tables: pair (j, j + rot/2), or (2j, 2j+1)
// when interleaved; the other values pass through.
//
// About 10 flops per element against 4 bytes moved (bf16): bound by HBM, next by
// instruction issue.  A group of lanes holds one head, 2 P values a lane, so every
// input is read once and the norm needs a few shuffles and no shared memory.  A
// lane's values are both halves of P pairs, so the rotation is lane-local.  An
// item is a block of heads of one token, all queries or all keys: its loads are
// independent, and the position, the angles and the weight are read once for
// it.  All arithmetic is fp32; outputs are rounded once.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace flce {

// One of q, k: `heads` heads of every token in `per_token` items.
struct NormSide {
  const void* x;       // input
  const void* w;       // head_dim weights, or null (ones)
  const void* dy;      // backward: output gradient, contiguous
  void* out;           // contiguous; backward: dx
  int64_t row, head;   // strides of x
  int64_t items;
  int heads, per_token;
};

struct QkNormRopeParams {
  NormSide q, k;
  const float *cos_t, *sin_t;   // table_rows x rot/2
  const int64_t* positions;     // one per token, or null (0, 1, 2, ...)
  float* partial;               // backward: one row of head_dim sums per block
  int64_t table_rows;
  int64_t q_blocks;             // blocks that take q's items; the others take k's
  int log_lanes;                // a head is held by 1 << log_lanes lanes
  int head_dim, rot_dim;
  float eps, inv_dim;
  int* err_word;
};

constexpr int kNormThreads = 128;
constexpr int kNormBwdBlocks = 4;  // blocks of the persistent backward on each SM
// Heads of an item, whose loads are in flight together (forward, backward).
template <typename T>
struct NormHeads {
  static constexpr int kFwd = sizeof(T) == 2 ? 4 : 2, kBwd = sizeof(T) == 2 ? 2 : 1;
};

// N consecutive values as they lie in memory.
template <typename T, int N>
struct Raw {
  static constexpr int kWords = N * sizeof(T) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0;
  }
  // Values 2 i and 2 i + 1, packed.
  __device__ __forceinline__ uint64_t pair(int i) const {
    if constexpr (sizeof(T) == 4)
      return pack_u32x2(w[2 * i], w[2 * i + 1]);
    else
      return pack_u32x2(w[i] << 16, w[i] & 0xffff0000u);
  }
};
// N values, packed in twos.
template <typename T, int N>
__device__ __forceinline__ void store_values(T* p, const uint64_t* x) {
  constexpr int kWords = N * sizeof(T) / 4;
  uint32_t w[kWords];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    float a, b;
    unpack_f32x2(x[i], a, b);
    if constexpr (sizeof(T) == 4) {
      w[2 * i] = __float_as_uint(a);
      w[2 * i + 1] = __float_as_uint(b);
    } else {
      w[i] = pack_bf16x2(a, b);
    }
  }
  if constexpr (kWords == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < kWords; i += 4)
      reinterpret_cast<uint4*>(p)[i / 4] = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  }
}

// A lane's place in its head.
template <int P, bool PAIRS>
struct NormLane {
  int a0, a1;    // offsets of its two runs of P values
  bool in_head;  // head_dim covers this lane
  bool turns;    // its values are rotated
  int j;         // its first pair
  __device__ __forceinline__ NormLane(const QkNormRopeParams& p, int l) {
    in_head = l * 2 * P < p.head_dim;
    turns = l * 2 * P < p.rot_dim;
    j = P * l;
    a0 = !PAIRS && turns ? P * l : 2 * P * l;
    a1 = !PAIRS && turns ? p.rot_dim / 2 + P * l : 2 * P * l + P;
  }
};

// The cosines and sines of a lane's pairs for one token; 1 and 0 where nothing is
// turned.
template <int P>
struct Angles {
  float c[P], s[P];
  template <bool PAIRS>
  __device__ __forceinline__ void load(const QkNormRopeParams& p, const NormLane<P, PAIRS>& n,
                                       int64_t pos) {
#pragma unroll
    for (int i = 0; i < P; ++i) c[i] = 1.f, s[i] = 0.f;
    if (!n.turns) return;
    if (pos < 0 || pos >= p.table_rows) {  // left unrotated and reported
      record_error(p.err_word, kErrIndex);
      return;
    }
    const int64_t at = pos * (p.rot_dim / 2) + n.j;
#pragma unroll
    for (int i = 0; i < P; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(p.cos_t + at + i);
      const float4 b = *reinterpret_cast<const float4*>(p.sin_t + at + i);
      c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
      s[i] = b.x, s[i + 1] = b.y, s[i + 2] = b.z, s[i + 3] = b.w;
    }
  }
};
__device__ __forceinline__ int64_t position(const QkNormRopeParams& p, int64_t token) {
  return p.positions ? p.positions[token] : token;
}
// Turns the lane's pairs by +angle (SIGN = 1) or -angle (-1); v packs its values in
// twos.
template <int P, bool PAIRS, int SIGN>
__device__ __forceinline__ void turn(uint64_t (&v)[P], const Angles<P>& t) {
  if constexpr (PAIRS) {  // (a, b) (c, c) + (b, a) (-s, s)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float a, b;
      unpack_f32x2(v[i], a, b);
      v[i] = fma_f32x2(pack_f32x2(b, a), pack_f32x2(-SIGN * t.s[i], SIGN * t.s[i]),
                       mul_f32x2(v[i], pack_f32x2(t.c[i], t.c[i])));
    }
  } else {  // two pairs at a time
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      uint64_t &a = v[i], &b = v[i + P / 2];
      const uint64_t c = pack_f32x2(t.c[2 * i], t.c[2 * i + 1]);
      const uint64_t s = pack_f32x2(SIGN * t.s[2 * i], SIGN * t.s[2 * i + 1]);
      const uint64_t m = pack_f32x2(-SIGN * t.s[2 * i], -SIGN * t.s[2 * i + 1]);
      const uint64_t u = fma_f32x2(b, m, mul_f32x2(a, c));
      b = fma_f32x2(a, s, mul_f32x2(b, c));
      a = u;
    }
  }
}

__device__ __forceinline__ float both(uint64_t x) {
  float a, b;
  unpack_f32x2(x, a, b);
  return a + b;
}
__device__ __forceinline__ float lanes_sum(float x, int log_lanes) {
  for (int o = 1 << log_lanes >> 1; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// One item a lane group.  Bound by HBM: 8192 tokens, 32 / 8 heads of 128 in bf16 move
// 172 MB in 30.4 us back to back, 5650 GB/s.
template <typename T, int P, bool PAIRS>
__global__ void __launch_bounds__(kNormThreads, 6)
qk_norm_rope_fwd(const __grid_constant__ QkNormRopeParams p) {
  constexpr int U = NormHeads<T>::kFwd;
  const bool is_q = blockIdx.x < p.q_blocks;
  const NormSide& side = is_q ? p.q : p.k;
  const int64_t item = (((int64_t)blockIdx.x - (is_q ? 0 : p.q_blocks)) * kNormThreads + threadIdx.x) >>
                       p.log_lanes;
  const NormLane<P, PAIRS> n(p, threadIdx.x & ((1 << p.log_lanes) - 1));
  const bool live = item < side.items && n.in_head;
  const uint32_t token = item < side.items ? (uint32_t)item / (uint32_t)side.per_token : 0;
  const int h0 = ((uint32_t)item - token * side.per_token) * U;
  const int heads = live ? side.heads - h0 : 0;
  const T* in = static_cast<const T*>(side.x) + token * side.row + h0 * side.head;
  grid_wait();
  // first, for the angles wait for the position (55.6 -> 48.5 us at 16384 tokens, 28 + 4
  // heads of 128)
  Angles<P> t;
  if (live) t.load(p, n, position(p, token));
  Raw<T, P> x[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    x[u][0].zero();
    x[u][1].zero();
    if (u < heads) {
      x[u][0].load(in + u * side.head + n.a0);
      x[u][1].load(in + u * side.head + n.a1);
    }
  }
  Raw<T, P> w[2];
  const bool weighted = side.w != nullptr;
  if (live && weighted) {
    w[0].load(static_cast<const T*>(side.w) + n.a0);
    w[1].load(static_cast<const T*>(side.w) + n.a1);
  }
  T* out = static_cast<T*>(side.out) + ((int64_t)token * side.heads + h0) * p.head_dim;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    uint64_t v[P], sq = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i] = x[u][i / (P / 2)].pair(i % (P / 2));
      sq = fma_f32x2(v[i], v[i], sq);
    }
    const float r = rsqrtf(lanes_sum(both(sq), p.log_lanes) * p.inv_dim + p.eps);
    if (u >= heads) continue;
    const uint64_t r2 = pack_f32x2(r, r);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      v[i] = mul_f32x2(v[i], r2);
      if (weighted) v[i] = mul_f32x2(v[i], w[i / (P / 2)].pair(i % (P / 2)));
    }
    if (n.turns) turn<P, PAIRS, 1>(v, t);
    store_values<T, P>(out + u * p.head_dim + n.a0, v);
    store_values<T, P>(out + u * p.head_dim + n.a1, v + P / 2);
  }
}

// Persistent over the items of q or of k: each lane keeps the sums of its 2 P
// weight gradients in registers; the block adds its groups' sums in a fixed
// order and writes one partial row, so results do not change run to run.
// The next item's heads are copied to shared memory while this one's are used, each
// thread its own pieces, so that loads are always in flight without registers to
// hold them.  Bound by HBM and instruction issue (66%): 16384 tokens, 28 / 4 heads of 128
// in bf16, 403 MB in 69 us.
template <typename T, int P, bool PAIRS>
__global__ void __launch_bounds__(kNormThreads, kNormBwdBlocks)
qk_norm_rope_bwd(const __grid_constant__ QkNormRopeParams p) {
  constexpr int U = NormHeads<T>::kBwd;
  constexpr int kBytes = P * sizeof(T), kCopy = kBytes < 16 ? kBytes : 16, kCopies = kBytes / kCopy;
  // by stage, head, run (x's two, dy's two), 16 or 8 byte copy and thread
  __shared__ __align__(16) uint8_t stage[2][U][4][kCopies][kNormThreads * kCopy];
  const bool is_q = blockIdx.x < p.q_blocks;
  const NormSide& side = is_q ? p.q : p.k;
  const int64_t block = (int64_t)blockIdx.x - (is_q ? 0 : p.q_blocks);
  const int64_t blocks = is_q ? p.q_blocks : gridDim.x - p.q_blocks;
  const int lanes = 1 << p.log_lanes, l = threadIdx.x & (lanes - 1);
  const NormLane<P, PAIRS> n(p, l);
  const bool weighted = side.w != nullptr;
  grid_wait();
  Raw<T, P> w[2];
  w[0].zero();
  w[1].zero();
  if (weighted && n.in_head) {
    w[0].load(static_cast<const T*>(side.w) + n.a0);
    w[1].load(static_cast<const T*>(side.w) + n.a1);
  }
  uint64_t dw[P] = {};
  const int64_t stride = (blocks * kNormThreads) >> p.log_lanes;
  struct At {
    uint32_t token;
    int h0, heads;  // heads: how many there are for this lane
  };
  auto at = [&](int64_t item) {
    At a;
    const bool live = item < side.items;
    a.token = live ? (uint32_t)item / (uint32_t)side.per_token : 0;
    a.h0 = live ? ((uint32_t)item - a.token * side.per_token) * U : 0;
    a.heads = live && n.in_head ? side.heads - a.h0 : 0;
    return a;
  };
  auto fetch = [&](const At& a, int buf) {
    const T* in = static_cast<const T*>(side.x) + a.token * side.row + a.h0 * side.head;
    const T* dy = static_cast<const T*>(side.dy) + ((int64_t)a.token * side.heads + a.h0) * p.head_dim;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (u < a.heads)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const T* from = (e < 2 ? in + u * side.head : dy + u * p.head_dim) + (e & 1 ? n.a1 : n.a0);
#pragma unroll
          for (int c = 0; c < kCopies; ++c)
            cp_async<kCopy>(&stage[buf][u][e][c][threadIdx.x * kCopy],
                            reinterpret_cast<const uint8_t*>(from) + c * kCopy);
        }
    cp_async_commit();
  };
  auto fetched = [&](Raw<T, P>& r, int buf, int u, int e) {
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      if constexpr (kCopy == 16) {
        const uint4 v = *reinterpret_cast<const uint4*>(&stage[buf][u][e][c][threadIdx.x * kCopy]);
        r.w[4 * c] = v.x, r.w[4 * c + 1] = v.y, r.w[4 * c + 2] = v.z, r.w[4 * c + 3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(&stage[buf][u][e][c][threadIdx.x * kCopy]);
        r.w[0] = v.x, r.w[1] = v.y;
      }
    }
  };
  int64_t item = ((block * kNormThreads) >> p.log_lanes) + (threadIdx.x >> p.log_lanes);
  At a = at(item);
  fetch(a, 0);
  Angles<P> t, t_next;
  t.load(p, n, n.turns ? position(p, a.token) : 0);
  int64_t pos = n.turns ? position(p, at(item + stride).token) : 0;
  int buf = 0;
  // every group of a warp runs the same number of rounds (the shuffles below
  // need the whole warp)
  for (int64_t base = (block * kNormThreads) >> p.log_lanes; base < side.items; base += stride) {
    const At next = at(item + stride);
    fetch(next, buf ^ 1);
    t_next.load(p, n, pos);
    if (n.turns) pos = position(p, at(item + 2 * stride).token);
    cp_async_wait<1>();
    T* out = static_cast<T*>(side.out) + ((int64_t)a.token * side.heads + a.h0) * p.head_dim;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint64_t v[P], y[P], sq = 0, gx = 0;
      Raw<T, P> x[2], g[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[e].zero();
        g[e].zero();
        if (u < a.heads) {
          fetched(x[e], buf, u, e);
          fetched(g[e], buf, u, 2 + e);
        }
      }
#pragma unroll
      for (int i = 0; i < P; ++i) {
        v[i] = x[i / (P / 2)].pair(i % (P / 2));
        y[i] = g[i / (P / 2)].pair(i % (P / 2));
        sq = fma_f32x2(v[i], v[i], sq);
      }
      if (n.turns) turn<P, PAIRS, -1>(y, t);
#pragma unroll
      for (int i = 0; i < P; ++i)
        gx = fma_f32x2(weighted ? mul_f32x2(y[i], w[i / (P / 2)].pair(i % (P / 2))) : y[i], v[i], gx);
      const float r = rsqrtf(lanes_sum(both(sq), p.log_lanes) * p.inv_dim + p.eps);
      // -mean(g w n) r^2, the factor of x in dx
      const float c = -lanes_sum(both(gx), p.log_lanes) * r * r * r * p.inv_dim;
      if (u >= a.heads) continue;
      const uint64_t r2 = pack_f32x2(r, r), c2 = pack_f32x2(c, c);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint64_t yr = mul_f32x2(y[i], r2);
        dw[i] = fma_f32x2(yr, v[i], dw[i]);
        v[i] = fma_f32x2(v[i], c2, weighted ? mul_f32x2(yr, w[i / (P / 2)].pair(i % (P / 2))) : yr);
      }
      store_values<T, P>(out + u * p.head_dim + n.a0, v);
      store_values<T, P>(out + u * p.head_dim + n.a1, v + P / 2);
    }
    a = next;
    t = t_next;
    item += stride;
    buf ^= 1;
  }
  cp_async_wait<0>();
  // sums of the groups: value i of lane l, by thread i * lanes + l
  static_assert(sizeof(stage) >= 2 * P * kNormThreads * sizeof(float), "the sums reuse the stages");
  float(*sums)[kNormThreads] = reinterpret_cast<float(*)[kNormThreads]>(&stage[0][0][0][0][0]);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < P; ++i) unpack_f32x2(dw[i], sums[2 * i][threadIdx.x], sums[2 * i + 1][threadIdx.x]);
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * P * lanes; e += kNormThreads) {
    const int i = e >> p.log_lanes, lane = e & (lanes - 1);
    const NormLane<P, PAIRS> m(p, lane);
    float s = 0.f;
    for (int g = lane; g < kNormThreads; g += lanes) s += sums[i][g];
    if (m.in_head) p.partial[(int64_t)blockIdx.x * p.head_dim + (i < P ? m.a0 + i : m.a1 + i - P)] = s;
  }
}

// dw = sum of the blocks' partial rows: q's are the first q_rows.  32 columns per
// block, 32 rows at a time, added in a fixed order.  300 KB at most: latency, 6 us.
__global__ void __launch_bounds__(1024) qk_norm_rope_dw(const float* partial, int q_rows, int rows,
                                                        int head_dim, float* dwq, float* dwk) {
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), w = threadIdx.x >> 5;
  const int end = blockIdx.y ? rows : q_rows;
  float t = 0.f;
  grid_wait();
  if (c < head_dim)
#pragma unroll 4
    for (int r = (blockIdx.y ? q_rows : 0) + w; r < end; r += 32) t += partial[(int64_t)r * head_dim + c];
  __shared__ float sums[32][33];
  sums[w][threadIdx.x & 31] = t;
  __syncthreads();
  if (w || c >= head_dim) return;
  t = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) t += sums[i][threadIdx.x];
  (blockIdx.y ? dwk : dwq)[c] = t;
}

}  // namespace flce
