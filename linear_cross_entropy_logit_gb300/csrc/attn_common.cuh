// Shared by the packed attention kernels: the call's parameters, the walk over
// the work units of the packed sequences, and shared-memory helpers.
#pragma once
#include <cuda_bf16.h>
#include <cstdint>
#include "ptx.cuh"

namespace flce {

using bf16 = __nv_bfloat16;

constexpr int kTile = 128;             // rows of a query or key tile (TMEM lanes)
constexpr int kBoxBytes = kTile * 128; // one 64-column box of a tile, 128-byte rows
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct AttnParams {
  const int32_t* cu;   // n_seqs + 1 offsets of the packed sequences
  int n_seqs;
  int tokens;
  int q_heads, kv_heads, group;  // group = q_heads / kv_heads
  int head_dim;
  float scale;
  bf16* out;           // tokens x q_heads x head_dim
  float* lse;          // q_heads x tokens
  const bf16 *k, *v;   // read directly where they hold non-finite values
  int64_t k_row, k_head, v_row, v_head;
  int* err_word;
  unsigned long long timeout_ns;
};

// One work unit: rows [q0, q0 + unit rows) of the sequence [start, start +
// len), or, with len = 0, `rows` rows from `start` that belong to no sequence.
struct AttnUnit {
  int start, len, q0, rows;
  int head;
};

__device__ __forceinline__ int warp_add(int x) { return __reduce_add_sync(~0u, x); }
__device__ __forceinline__ int warp_max(int x) { return __reduce_max_sync(~0u, x); }

// Whether [begin, end) may be a sequence among `tokens` rows.  By comparisons alone: the
// difference of offsets that may be anything passes 32 bits.
__host__ __device__ constexpr bool sequence_ok(int begin, int end, int tokens) {
  return 0 <= begin && begin <= end && end <= tokens;
}

// The sequences of a pack cut into units of ROWS rows, numbered so that the
// longest come first: dealt out in this order, the CTAs end together.  Unit i of a
// sequence sees i + 1 units' worth of keys and stands in class i; of two query tiles
// (ROWS = 256) the last unit of a sequence may have rows in one only, which takes
// about 5/8 of the time and stands in class 5/8 i (151 -> 145 us for 37 ragged
// sequences).  Every unit number is mapped by one warp on its own from the offsets,
// so no list of units is written and no launch goes before the attention.  A CTA's
// numbers ascend, so that the search goes on from where the last one ended: one pass
// over the offsets for all its units of a class, and log2(classes) passes to find
// the next class.
template <int ROWS>
struct UnitWalk {
  const int32_t* cu;
  int n, tokens;
  int classes;    // every unit's class is below this
  int units;      // units of all sequences
  int lead, gaps; // rows before the first sequence; units of all rows in none
  int tail_start;
  // The last unit's class, whose units are numbers [first, end); whether it was part of a
  // unit; its block of 32 sequences, and the units of the class before that block.
  int cls, first, end;
  int part, block, seen;

  static __device__ __forceinline__ int cut(int rows) { return (rows + ROWS - 1) / ROWS; }
  // Whole units of a sequence: with rows in every query tile.
  static __device__ __forceinline__ int whole(int len) { return (len + kTile - 1) / ROWS; }
  // The class of the unit after those; -1 if there is none.
  static __device__ __forceinline__ int part_class(int len) {
    return cut(len) > whole(len) ? whole(len) * 5 >> 3 : -1;
  }
  // Units of class c and above.
  static __device__ __forceinline__ int above(int len, int c) {
    return max(0, whole(len) - c) + (part_class(len) >= c);
  }
  __device__ __forceinline__ int length(int s) const { return s < n ? cu[s + 1] - cu[s] : 0; }
  __device__ __forceinline__ int from(int c) const {
    int t = 0;
#pragma unroll 4
    for (int s = threadIdx.x & 31; s < n; s += 32) t += above(length(s), c);
    return warp_add(t);
  }
  // Executed by one whole warp.  Offsets that do not ascend within [0,
  // tokens] leave every row in no sequence.
  __device__ __forceinline__ void init(const AttnParams& p) {
    cu = p.cu;
    n = p.n_seqs;
    tokens = p.tokens;
    lead = cu[0];
    tail_start = cu[n];
    int bad = !sequence_ok(lead, tail_start, tokens), most = 0, sum = 0;
#pragma unroll 4
    for (int s = threadIdx.x & 31; s < n; s += 32) {
      const int begin = cu[s], end = cu[s + 1];
      const bool ok = sequence_ok(begin, end, tokens);
      const int rows = ok ? end - begin : 0;
      bad |= !ok;
      most = max(most, max(whole(rows), part_class(rows) + 1));
      sum += cut(rows);
    }
    classes = warp_max(most);
    units = warp_add(sum);
    if (__any_sync(~0u, bad)) {
      if (blockIdx.x == 0 && (threadIdx.x & 31) == 0) record_error(p.err_word, kErrIndex);
      n = classes = units = lead = tail_start = 0;
    }
    gaps = cut(lead) + cut(tokens - tail_start);
    first = end = 0;
  }
  __device__ __forceinline__ int total() const { return units + gaps; }

  // Unit `rank` in [0, total()).  Executed by one whole warp, for ascending ranks.
  __device__ __forceinline__ AttnUnit at(int rank) {
    AttnUnit u{};
    if (rank >= units) {
      const int g = rank - units, before = cut(lead);
      u.start = g < before ? g * ROWS : tail_start + (g - before) * ROWS;
      u.rows = min(ROWS, (g < before ? lead : tokens) - u.start);
      return u;
    }
    if (rank >= end) {  // another class: from(lo) > rank >= from(hi)
      int lo = 0, hi = classes;
      first = 0;
      end = units;
#pragma unroll 1
      while (hi - lo > 1) {
        const int m = (lo + hi) >> 1, f = from(m);
        if (f > rank) lo = m, end = f; else hi = m, first = f;
      }
      cls = lo;
      part = block = seen = 0;
    }
    // The unit is the nth of its class: the whole units come first, then the parts.
    const int nth = rank - first;
#pragma unroll 1
    for (; part < 2; ++part, block = 0)
#pragma unroll 1
      for (; 32 * block < n; ++block) {
        const int s = 32 * block + (threadIdx.x & 31), len = length(s);
        const unsigned has = __ballot_sync(~0u, part ? part_class(len) == cls : whole(len) > cls);
        const int before = __popc(has & ((1u << (threadIdx.x & 31)) - 1));
        const unsigned here = __ballot_sync(~0u, ((has >> (threadIdx.x & 31)) & 1) && seen + before == nth);
        if (here) {
          const int q = 32 * block + __ffs(here) - 1;
          u.start = cu[q];
          u.len = cu[q + 1] - u.start;
          u.q0 = (part ? whole(u.len) : cls) * ROWS;
          return u;
        }
        seen += __popc(has);
      }
    return u;  // not reached
  }
};

// Debug build: a mapped unit lies within the tokens (else it is reported and ends the
// CTA's walk).
__device__ __forceinline__ bool unit_ok(const AttnUnit& u, const AttnParams& p) {
  const int end = u.len > 0 ? u.len : u.rows;
  return dbg_ok(u.start >= 0 && end > 0 && u.start + (int64_t)end <= p.tokens && u.q0 >= 0 &&
                    (u.len == 0 || u.q0 < u.len),
                p.err_word);
}

// Unit number of round r of CTA c of g: every other round runs backwards, so
// that a CTA with a long unit in one round gets a short one in the next.
__device__ __forceinline__ int64_t dealt_unit(uint32_t r, int c, int g) {
  return (int64_t)r * g + ((r & 1) ? g - 1 - c : c);
}

// Bounded waits like mbar_wait, with the time limit in a function of its own:
// these kernels wait in some thirty places, and what a warp does between two
// waits is short enough for fetching its instructions to count.
// Returns ~0 to give up, else the time of the first call for this wait.
__device__ __noinline__ uint64_t wait_limit(uint64_t since, const WaitCtx ctx) {
  if (*ctx.abort) return ~0ull;
  const uint64_t now = global_timer_ns();
  if (since == 0) return now;
  if (now - since <= ctx.timeout_ns) return since;
  *ctx.abort = 1;
  record_error(ctx.err_word, kErrTimeout);
  return ~0ull;
}
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, const WaitCtx& ctx) {
  const uint32_t a = smem_u32(bar);
  uint64_t since = 0;
  for (uint32_t n = 1; !mbar_try_wait(a, parity); ++n)
    if ((n & 63u) == 0u && (since = wait_limit(since, ctx)) == ~0ull) return false;
  return true;
}
// By a whole warp: all its lanes get the same answer, so that they leave a loop
// together.
__device__ __forceinline__ bool wait_bar_warp(uint64_t* bar, uint32_t parity, const WaitCtx& ctx) {
  return __all_sync(~0u, wait_bar(bar, parity, ctx));
}

// Products of whole tiles, issued by the elected lane of a converged warp.  The
// whole warp keeps the issuing loop's state, in uniform registers: an
// instruction takes 64 tensor cycles at N = 128, and with the state in one
// lane's registers issuing one took longer than that (1.4x slower kernels).
//
// d (+)= A B^T over DP head values; A and B are 128-row tiles in shared memory.
template <int DP>
__device__ __forceinline__ void mma_tiles(uint32_t el, uint32_t d, uint32_t a_tile, uint32_t b_tile) {
  constexpr uint32_t idesc = make_idesc(false, false, kTile, kTile);
  const uint32_t a = desc_lo(a_tile, 16), b = desc_lo(b_tile, 16);
#pragma unroll
  for (int kk = 0; kk < DP / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kBoxBytes + (kk & 3) * 32) >> 4;
    mma_issue_lo(el, d, a + off, b + off, idesc, kk != 0);
  }
}
// One thread's 64 columns.
__device__ __forceinline__ void load64(uint32_t (&r)[2][32], uint32_t at) {
  tmem_ld_32x32b_x32(at, r[0]);
  tmem_ld_32x32b_x32(at + 32, r[1]);
  tmem_ld_wait();
}

// d (+)= A B over 128 rows of the tile B (128 x DP); A is packed bf16 in TMEM,
// `gap` columns from one run of 64 k to the next (32 when they are adjacent).
// R0, R1: which runs.
template <int DP, int R0 = 0, int R1 = 2>
__device__ __forceinline__ void mma_tmem_tile(uint32_t el, uint32_t d, uint32_t a, int gap,
                                              uint32_t b_tile, bool accumulate) {
  constexpr uint32_t idesc = make_idesc(false, true, kTile, DP);
  const uint32_t b = desc_lo(b_tile, kBoxBytes);
#pragma unroll
  for (int kk = 4 * R0; kk < 4 * R1; ++kk)
    mma_issue_ts(el, d, a + (kk >> 2) * gap + (kk & 3) * 8, b + ((kk * 2048) >> 4), idesc,
                 kk != 4 * R0 || accumulate);
}

// Stores `cols` columns of a warp's 32 TMEM lanes (one row each) times `scale`, in
// bf16 or fp32, through 4 KB of shared memory: eight lanes then write 128 bytes of
// one row.  (Written by each lane for itself, a warp's store touches 32 lines and
// takes as many cycles.)  `to`: the first row's first column; `rows`, `cols`: how
// many are written, cols a multiple of 8.  The pieces of a row are permuted by the
// row number, so that both sides are free of bank conflicts.  Once per unit, so its
// instructions come from L2, eight to a line: unrolled it took 4000 cycles, rolled
// loops a quarter of that.
template <typename T>
__device__ __forceinline__ void store_rows(uint8_t* stage, uint32_t taddr, float scale, T* to,
                                           int64_t row_stride, int rows, int cols) {
  constexpr int kCols = 128 / sizeof(T);  // columns in 128 bytes
  const int lane = threadIdx.x & 31, p = lane & 7;
  const uint32_t mine = smem_u32(stage) + lane * 128;
#pragma unroll 1
  for (int c = 0; c < cols; c += kCols) {
    __syncwarp();  // the last round's reads
#pragma unroll 1
    for (int i = 0; i < 8; i += 16 * sizeof(T) / 16) {  // 16 columns: two or four pieces
      uint32_t r[16];
      tmem_ld_32x32b_x16(taddr + c + i * (16 / sizeof(T)), r);
      tmem_ld_wait();
#pragma unroll
      for (int e = 0; e < (int)sizeof(T); ++e) {
        uint32_t w[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if constexpr (sizeof(T) == 2)
            w[g] = pack_bf16x2(__uint_as_float(r[8 * e + 2 * g]) * scale,
                               __uint_as_float(r[8 * e + 2 * g + 1]) * scale);
          else
            w[g] = __float_as_uint(__uint_as_float(r[4 * e + g]) * scale);
        }
        st_shared_v4(mine + (((i + e) ^ p) << 4), w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
    T* at = to + (lane >> 3) * row_stride + c + p * (16 / sizeof(T));
    const bool in = c + p * (int)(16 / sizeof(T)) < cols;
#pragma unroll 2
    for (int r = lane >> 3; r < 32; r += 4, at += 4 * row_stride) {
      const uint4 x = *reinterpret_cast<const uint4*>(stage + r * 128 + ((p ^ (r & 7)) << 4));
      if (in && r < rows) *reinterpret_cast<uint4*>(at) = x;
    }
  }
}
// Adds the non-finite ones among the `cols` values of x, times `weight`, to a row just
// stored.
template <typename T>
__device__ __noinline__ void add_nonfinite(T* row, const bf16* x, int cols, float weight) {
#pragma unroll 1
  for (int d = 0; d < cols; ++d) {
    const float v = __bfloat162float(x[d]);
    if (!isfinite(v)) row[d] = static_cast<T>(static_cast<float>(row[d]) + v * weight);
  }
}

// A unit read from shared memory by a whole warp, the same in all its lanes.
__device__ __forceinline__ AttnUnit uniform(const AttnUnit& from) {
  AttnUnit u;
  u.start = __shfl_sync(~0u, from.start, 0);
  u.len = __shfl_sync(~0u, from.len, 0);
  u.q0 = __shfl_sync(~0u, from.q0, 0);
  u.rows = __shfl_sync(~0u, from.rows, 0);
  u.head = __shfl_sync(~0u, from.head, 0);
  return u;
}

// Bits 15 and 31 set where a packed bf16 half is infinite or NaN.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t x) {
  return ((x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// The part of clean_tile that zeroes the rows from `valid` on.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int boxes, int valid, int w, int warps) {
#pragma unroll 1
  for (int i = w * 32 + (threadIdx.x & 31); i < boxes * kTile * 8; i += warps * 32)
    if (((i >> 3) & (kTile - 1)) >= valid)
      reinterpret_cast<uint4*>(tile)[i] = make_uint4(0, 0, 0, 0);
}

// Fills the rows from `valid` on with row valid - 1 (16-byte pieces are swizzled by the
// row number).  Before clean_tile: whether another warp has cleaned that row by then does not
// matter, as each cleans its copies.
__device__ __forceinline__ void repeat_row(uint8_t* tile, int boxes, int valid, int w, int warps) {
#pragma unroll 1
  for (int i = w * 32 + (threadIdx.x & 31); i < boxes * kTile * 8; i += warps * 32) {
    const int row = (i >> 3) & (kTile - 1), from = valid - 1;
    if (row >= valid)
      reinterpret_cast<uint4*>(tile)[i] =
          reinterpret_cast<const uint4*>(tile)[(i & ~(kTile * 8 - 1)) + from * 8 + ((i ^ row ^ from) & 7)];
  }
}

// Whether a warp's share of a tile (the pieces that it cleans) holds a non-finite value.
__device__ __forceinline__ bool has_nonfinite(const uint8_t* tile, int boxes, int w, int warps) {
  constexpr int kAhead = 8;  // loads in flight
  uint32_t top = 0;  // the largest magnitude, NaN above all; its sign says nothing
#pragma unroll 1
  for (int i = w * 32 + (threadIdx.x & 31); i < boxes * kTile * 8; i += kAhead * warps * 32) {
    uint4 x[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      x[e] = reinterpret_cast<const uint4*>(tile)[i + e * warps * 32];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      top = bf16x2_max_abs(bf16x2_max_abs(bf16x2_max_abs(bf16x2_max_abs(top, x[e].x), x[e].y), x[e].z), x[e].w);
  }
  return __any_sync(~0u, nonfinite2(top) != 0);
}

// Makes a tile fit to be multiplied by zeros: rows from `valid` on (another
// sequence's, or none's) become zero; non-finite values become zero and their
// row's bit is set in flags[4], for the caller to add them back where they are
// visible.  Called by each of `warps` warps (w = 0 ..) with flags of its own.
__device__ __forceinline__ void clean_tile(uint8_t* tile, int boxes, int valid, int w, int warps,
                                           uint32_t* flags) {
  const int lane = threadIdx.x & 31;
  if (lane < 4) flags[lane] = 0;
  if (valid < kTile) zero_rows(tile, boxes, valid, w, warps);
  __syncwarp();
  constexpr int kAhead = 8;  // loads in flight
#pragma unroll 1
  for (int i = w * 32 + lane; i < boxes * kTile * 8; i += kAhead * warps * 32) {
    uint4 x[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      x[e] = reinterpret_cast<const uint4*>(tile)[i + e * warps * 32];
    // the largest magnitude, NaN above all; its sign says nothing
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
      top = bf16x2_max_abs(bf16x2_max_abs(bf16x2_max_abs(bf16x2_max_abs(top, x[e].x), x[e].y), x[e].z), x[e].w);
    if (nonfinite2(top) == 0) continue;
#pragma unroll 1
    for (int e = 0; e < kAhead; ++e) {
      uint4* at = reinterpret_cast<uint4*>(tile) + i + e * warps * 32;
      uint4 y = *at;
      if ((nonfinite2(y.x) | nonfinite2(y.y) | nonfinite2(y.z) | nonfinite2(y.w)) == 0) continue;
      uint32_t* h = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const uint32_t b = nonfinite2(h[g]);
        h[g] &= (b & 0x8000u ? 0u : 0xffffu) | (b & 0x80000000u ? 0u : 0xffff0000u);
      }
      *at = y;
      const int row = ((i + e * warps * 32) >> 3) & (kTile - 1);
      atomicOr(&flags[row >> 5], 1u << (row & 31));
    }
  }
  __syncwarp();
}

}  // namespace flce
