// Rotary positions of query and key heads.
//   y = m R(position) x on the first rot values of a head, y = x on the others;
// R turns pair j by position * inv_freq[j]: pair (j, j + rot/2), or (2j, 2j + 1) when
// interleaved.  The backward is the same with the negative angle.
//
// Angles are taken in turns, as 64-bit fractions of one: position * (2^64 f), f = inv_freq / 2 pi,
// wraps around as the angle does.  2^64 f is cut off to an integer (for inv_freq from 4 on, to as
// many bits of it as 64 bits of f leave), so that the angle is off by less than |position| *
// 2^-64 * max(1, inv_freq / 2) turns: nothing for a position of a million, 2e-7 radians at 2^39,
// 2e-4 at 2^49.  Integers take f from inv_freq's bits, the fp64 pipe is slow here.  Cosine and
// sine take the angle as a float of half turns, off by 2^-25 at most.
//
// About 4 flops a value: bound by HBM.  A block computes the cosines and sines of its
// tokens once, in shared memory, while the heads are on their way there: each thread
// copies what it turns itself.  It has both halves of P pairs of a head, so that every value is
// read once, 16 bytes at a time, and turns the same pairs of several heads of one token with
// angles that stay in its registers.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "heads.cuh"
#include "ptx.cuh"

namespace flce {

struct RopeParams {
  const void *q, *k;
  void *q_out, *k_out;       // contiguous
  const double* inv_freq;    // rot / 2
  const int64_t* positions;  // one per token, or null (0, 1, 2, ...)
  int64_t tokens, q_row, q_head, k_row, k_head;
  int q_heads, kv_heads, head_dim, rot_dim;
  int units;             // threads that share a head, 2 P values each
  int tokens_per_block;
  int slots;             // groups of units threads that share a token's heads
  float magnitude;
  int backward;
};

constexpr int kRopeThreads = 256;  // at most: slots x tokens x units of them work
// Heads whose loads a thread has in flight.
template <typename T>
constexpr int kRopeHeads = sizeof(T) == 2 ? 4 : 2;

// inv_freq / 2 pi in turns, modulo one, as a 64-bit fraction, cut off: its 53 bits times
// 2^66 / 2 pi, shifted by its exponent.
__device__ __forceinline__ uint64_t rope_step(double inv_freq) {
  const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq);
  const int e = (int)(bits >> 52 & 2047);
  const uint64_t mantissa = (bits << 11) | 0x8000000000000000ull;
  const uint64_t f = e ? __umul64hi(mantissa, 0xa2f9836e4e44152aull) : 0;
  const int left = e - 1024;
  const uint64_t step = left >= 0 ? (left < 64 ? f << left : 0) : (left > -64 ? f >> -left : 0);
  return bits >> 63 ? 0 - step : step;
}
// Cosine and sine of the position's angle; NaN for a frequency that is not finite.
__device__ __forceinline__ float2 rope_angle(int64_t position, double inv_freq) {
  const int64_t phase = (int64_t)((uint64_t)position * rope_step(inv_freq));
  float s, c;
  sincospif(__ll2float_rn(phase) * 1.0842021724855044e-19f, &s, &c);  // 2^-63
  const float bad = isfinite(inv_freq) ? 0.f : __int_as_float(0x7fc00000);
  return make_float2(c + bad, s + bad);
}

// Turns the values of a unit, in twos: those of its first run, then of its second.
template <int P, bool PAIRS>
__device__ __forceinline__ void rope_turn(uint64_t (&v)[P], const uint64_t (&c)[P / 2], const uint64_t (&s)[P / 2]) {
  if constexpr (PAIRS) {  // (a, b) (c, c) + (b, a) (-s, s)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      float a, b, ci[2], si[2];
      unpack_f32x2(v[i], a, b);
      unpack_f32x2(c[i / 2], ci[0], ci[1]);
      unpack_f32x2(s[i / 2], si[0], si[1]);
      v[i] = fma_f32x2(pack_f32x2(b, a), pack_f32x2(-si[i & 1], si[i & 1]),
                       mul_f32x2(v[i], pack_f32x2(ci[i & 1], ci[i & 1])));
    }
  } else {  // two pairs at a time
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const uint64_t a = v[i], b = v[i + P / 2], m = mul_f32x2(s[i], pack_f32x2(-1.f, -1.f));
      v[i] = fma_f32x2(b, m, mul_f32x2(a, c[i]));
      v[i + P / 2] = fma_f32x2(a, s[i], mul_f32x2(b, c[i]));
    }
  }
}

// Shared memory of a block: its threads' heads, then the angles.
template <typename T, int P>
constexpr int kRopeStage = kRopeHeads<T> * 2 * P * (int)sizeof(T);  // bytes a thread

// 32768 tokens, 28 / 4 heads of 128 in bf16: 537 MB in 78.3 us, 6860 GB/s; loads into registers
// behind the angles took 92.  8192 tokens, 32 / 8 heads: 168 MB in 25.
template <typename T, int P, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ __align__(16) uint8_t rope_space[];
  // angles by token: rot / 2 cosines, rot / 2 sines
  float* angles = reinterpret_cast<float*>(rope_space + blockDim.x * kRopeStage<T, P>);
  const int64_t token0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.tokens - token0), half = p.rot_dim / 2;
  const int group = threadIdx.x / p.units, u = threadIdx.x - group * p.units;
  const int t = group / p.slots, slot = group - t * p.slots, heads = p.q_heads + p.kv_heads;
  const bool turns = u * 2 * P < p.rot_dim;
  const int a0 = !PAIRS && turns ? P * u : 2 * P * u;
  const int a1 = !PAIRS && turns ? half + P * u : 2 * P * u + P;
  const int64_t token = token0 + t;
  const T* q = static_cast<const T*>(p.q) + token * p.q_row;
  const T* k = static_cast<const T*>(p.k) + token * p.k_row;
  T* q_out = static_cast<T*>(p.q_out) + token * p.q_heads * p.head_dim;
  T* k_out = static_cast<T*>(p.k_out) + token * p.kv_heads * p.head_dim;
  auto in = [&](int h) { return h < p.q_heads ? q + h * p.q_head : k + (h - p.q_heads) * p.k_head; };
  constexpr int U = kRopeHeads<T>, kBytes = P * sizeof(T), kCopy = kBytes < 16 ? kBytes : 16;
  // by head, run, 16 or 8 byte copy and thread
  auto piece = [&](int i, int run, int copy) {
    return rope_space + (((i * 2 + run) * (kBytes / kCopy) + copy) * blockDim.x + threadIdx.x) * kCopy;
  };
  auto fetch = [&](int h0) {
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (t < tokens && h0 + i * p.slots < heads) {
        const T* from = in(h0 + i * p.slots);
#pragma unroll
        for (int c = 0; c < kBytes / kCopy; ++c) {
          cp_async<kCopy>(piece(i, 0, c), reinterpret_cast<const uint8_t*>(from + a0) + c * kCopy);
          cp_async<kCopy>(piece(i, 1, c), reinterpret_cast<const uint8_t*>(from + a1) + c * kCopy);
        }
      }
    cp_async_commit();
  };
  grid_wait();
  fetch(slot);
  for (int i = threadIdx.x; i < tokens * half; i += blockDim.x) {
    const int at = i / half, j = i - at * half;
    const float2 w = rope_angle(p.positions ? p.positions[token0 + at] : token0 + at, p.inv_freq[j]);
    angles[at * p.rot_dim + j] = w.x * p.magnitude;
    angles[at * p.rot_dim + half + j] = (p.backward ? -w.y : w.y) * p.magnitude;
  }
  __syncthreads();
  if (t >= tokens) return;
  uint64_t c[P / 2] = {}, s[P / 2] = {};
  if (turns) {
#pragma unroll
    for (int i = 0; i < P; i += 4) {
      const float4 a = *reinterpret_cast<const float4*>(angles + t * p.rot_dim + P * u + i);
      const float4 b = *reinterpret_cast<const float4*>(angles + t * p.rot_dim + half + P * u + i);
      c[i / 2] = pack_f32x2(a.x, a.y), c[i / 2 + 1] = pack_f32x2(a.z, a.w);
      s[i / 2] = pack_f32x2(b.x, b.y), s[i / 2 + 1] = pack_f32x2(b.z, b.w);
    }
  }
  for (int h0 = slot; h0 < heads; h0 += U * p.slots) {
    cp_async_wait<0>();
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int h = h0 + i * p.slots;
      if (h >= heads) break;
      Raw<T, P> r[2];
#pragma unroll
      for (int run = 0; run < 2; ++run)
#pragma unroll
        for (int c = 0; c < kBytes / kCopy; ++c) {
          if constexpr (kCopy == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(piece(i, run, c));
            r[run].w[4 * c] = v.x, r[run].w[4 * c + 1] = v.y, r[run].w[4 * c + 2] = v.z, r[run].w[4 * c + 3] = v.w;
          } else {
            const uint2 v = *reinterpret_cast<const uint2*>(piece(i, run, c));
            r[run].w[0] = v.x, r[run].w[1] = v.y;
          }
        }
      uint64_t v[P];
#pragma unroll
      for (int j = 0; j < P; ++j) v[j] = r[j / (P / 2)].pair(j % (P / 2));
      if (turns) rope_turn<P, PAIRS>(v, c, s);
      T* out = h < p.q_heads ? q_out + h * p.head_dim : k_out + (h - p.q_heads) * p.head_dim;
      store_values<T, P>(out + a0, v);
      store_values<T, P>(out + a1, v + P / 2);
    }
    if (h0 + U * p.slots < heads) fetch(h0 + U * p.slots);
  }
}

}  // namespace flce
