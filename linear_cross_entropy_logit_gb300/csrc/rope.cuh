// Rotary positions of query and key heads.
//   y = m R(position) x on the first rot values of a head, y = x on the others;
// R turns pair j by position * inv_freq[j]: pair (j, j + rot/2), or (2j, 2j + 1) when
// interleaved.  The backward is the same with the negative angle.
//
// Angles are taken in turns, as 64-bit fractions of one: position * round(2^64 f),
// f = inv_freq / 2 pi, wraps around as the angle does, so that only f's own rounding
// (2^-53) grows with the position, and a position of a million is as exact as one of
// ten.  Its upper 24 bits go to cosine and sine of pi x.
//
// About 4 flops a value: bound by HBM.  A block computes the cosines and sines of its
// tokens once, in shared memory, and turns all their heads with them; a thread holds
// both halves of P pairs, so that every value is read once, 16 bytes at a time.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace flce {

struct RopeParams {
  const void *q, *k;
  void *q_out, *k_out;       // contiguous
  const double* inv_freq;    // rot / 2
  const int64_t* positions;  // one per token, or null (0, 1, 2, ...)
  int64_t tokens, q_row, q_head, k_row, k_head;
  int q_heads, kv_heads, head_dim, rot_dim;
  int units;      // pieces of 2 P values of a head
  int tokens_per_block, heads_per_block;
  float magnitude;
  int backward;
};

constexpr int kRopeThreads = 256;  // at most; a multiple of the units

// The position's angle in turns, in [-1/2, 1/2), times two: the argument of sincospi.
__device__ __forceinline__ float rope_half_turns(int64_t position, double inv_freq) {
  const double f = inv_freq * 0.15915494309189533577;  // 1 / 2 pi
  const uint64_t step = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
  const int64_t phase = (int64_t)((uint64_t)position * step);
  return __ll2float_rn(phase) * 1.0842021724855044e-19f;  // 2^-63
}

template <typename T, int P, bool PAIRS>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  extern __shared__ float2 angles[];  // tokens_per_block x rot / 2
  const int64_t token0 = (int64_t)blockIdx.x * p.tokens_per_block;
  const int tokens = (int)min((int64_t)p.tokens_per_block, p.tokens - token0), half = p.rot_dim / 2;
  const int head0 = blockIdx.y * p.heads_per_block;
  const int heads = min(p.heads_per_block, p.q_heads + p.kv_heads - head0);
  grid_wait();
  for (int i = threadIdx.x; i < tokens * half; i += blockDim.x) {
    const int t = i / half;
    const int64_t position = p.positions ? p.positions[token0 + t] : token0 + t;
    float s, c;
    sincospif(rope_half_turns(position, p.inv_freq[i - t * half]), &s, &c);
    angles[i] = make_float2(c * p.magnitude, (p.backward ? -s : s) * p.magnitude);
  }
  __syncthreads();
  const int u = threadIdx.x % p.units, groups = blockDim.x / p.units;
  const bool turns = u * 2 * P < p.rot_dim;
  const int a0 = !PAIRS && turns ? P * u : 2 * P * u;
  const int a1 = !PAIRS && turns ? half + P * u : 2 * P * u + P;
  for (int i = threadIdx.x / p.units; i < tokens * heads; i += groups) {
    const int t = i / heads, h = head0 + i - t * heads;
    const int64_t token = token0 + t;
    const bool is_q = h < p.q_heads;
    const T* in = is_q ? static_cast<const T*>(p.q) + token * p.q_row + h * p.q_head
                       : static_cast<const T*>(p.k) + token * p.k_row + (h - p.q_heads) * p.k_head;
    T* out = is_q ? static_cast<T*>(p.q_out) + (token * p.q_heads + h) * p.head_dim
                  : static_cast<T*>(p.k_out) + (token * p.kv_heads + h - p.q_heads) * p.head_dim;
    float x[2 * P];
#pragma unroll
    for (int j = 0; j < P; ++j) x[j] = (float)in[a0 + j], x[P + j] = (float)in[a1 + j];
    if (turns) {
      const float2* w = angles + t * half + P * u;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        float &a = PAIRS ? x[2 * j] : x[j], &b = PAIRS ? x[2 * j + 1] : x[P + j];
        const float c = w[j].x, s = w[j].y, y = a * c - b * s;
        b = b * c + a * s;
        a = y;
      }
    }
#pragma unroll
    for (int j = 0; j < P; ++j) out[a0 + j] = (T)x[j], out[a1 + j] = (T)x[P + j];
  }
}

}  // namespace flce
