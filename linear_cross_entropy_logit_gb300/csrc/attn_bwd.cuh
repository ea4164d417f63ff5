// Backward of packed causal attention on the tensor cores.
//
//   p_ij = exp(s_ij - lse_i),  delta_i = dout_i . out_i   attn_delta
//   ds_ij = p_ij (dout_i . v_j - delta_i)
//   dq_i = scale sum_j ds_ij k_j          attn_dq: a CTA owns 128 query rows
//   dv_j = sum_i p_ij dout_i              attn_dkdv: a CTA owns 128 key rows and
//   dk_j = scale sum_i ds_ij q_i          sums over the query heads that read them
//
// The last two recompute S and dP = dout V^T, so that every sum stays in the
// TMEM of the CTA that owns its rows: no fp32 gradient goes through memory, no
// atomics, the same bits every run.  Seven products where one kernel for all
// three gradients would take five, but that one has to add dq up in memory
// across CTAs.  At 8192 tokens, 32 / 8 heads of 128, each launch by itself: delta 25 us, dq
// 498 us and dkdv 643 us, the two at 1660 and 1710 TFLOP/s of their three and four products
// over the visible pairs: bound by the tensor cores.  61 ragged sequences of 9999 tokens, 16
// heads of 64: 11, 50 and 67 us, bound by each unit's latency.
//
// Both: warps 0-7 compute (a thread owns one TMEM lane and 64 of the 128
// columns), warp 8 issues MMAs, warp 9 maps units and loads, warps 12-15 clean
// tiles.  P and dS are rounded to bf16 for the products (their operands' type);
// everything else is fp32.  A masked entry is set to zero after the
// multiplication, so that what it held does not matter; its partner in the
// product (a row of another sequence, or a non-finite value) is zeroed in shared
// memory, as in the forward.
#pragma once
#include "attn_common.cuh"

namespace flce {

constexpr int kBwdThreads = 512;
constexpr int kBwdComputeRegs = 184, kBwdOtherRegs = 72;
static_assert(2 * (kBwdComputeRegs + kBwdOtherRegs) == 4 * (65536 / kBwdThreads),
              "shares add up to what the block is launched with");

struct AttnBwdParams : AttnParams {
  const bf16* dout;    // tokens x q_heads x head_dim
  bf16 *dq, *dk, *dv;  // contiguous
  float *nlse, *delta; // q_heads x tokens: -lse log2 e, delta (by attn_delta, then attn_dq)
  float* partial;      // splits > 1: dk, dv partial sums, 2 x splits x tokens x kv_heads x head_dim
  int splits;          // CTAs that share the query heads of a key / value head
  // Where the partial sums of dk, or dv, of a split begin.
  __host__ __device__ int64_t partial_at(bool dv_sum, int split) const {
    return (int64_t)((dv_sum ? splits : 0) + split) * tokens * kv_heads * head_dim;
  }
};

__device__ __forceinline__ float as_f(uint32_t x) { return __uint_as_float(x); }

// Zeroes a diagonal tile's entries on the far side of the diagonal in this thread's 64
// columns: those below (columns < row) or above it.  A warp's 32 rows meet the
// diagonal in one run of 32 columns; other runs are kept or dropped whole.
template <bool BELOW>
__device__ __forceinline__ void mask_diagonal(uint32_t (&v)[2][32], int half) {
  const int w = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int run = 2 * half + k;
    if (run == w) {
      asm volatile("");  // kept a branch, as selects it would cost every run
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (BELOW ? e < lane : e > lane) v[k][e] = 0;
    } else if (BELOW ? run < w : run > w) {
      asm volatile("");
#pragma unroll
      for (int e = 0; e < 32; ++e) v[k][e] = 0;
    }
  }
}

// dS of a sequence's first query and key, in its first diagonal tile.  That query sees one
// key, its p is 1 and its dS nothing but the rounding of lse and delta (1e-7 of dP): with it
// a sequence of one token would have gradients where there are none.  A dS that is not
// finite stays so.
__device__ __forceinline__ void zero_first(uint32_t (&v)[2][32]) {
  if (threadIdx.x == 0) v[0][0] = __float_as_uint(as_f(v[0][0]) * 0.f);
}

// ----------------------------------------------------------------------------
// delta
// ----------------------------------------------------------------------------
// Bound by reading out and dout once: 136 MB in 22 to 25 us at 8192 tokens, 32 heads of 128
// (5.4 to 6.1 TB/s).  Eight lanes hold a row, 8 or 16 values each, and eight or four rows: 16
// loads in flight a lane.  Blocks of all heads of the same tokens run together (one head's
// tokens after another's: 27 us).  A kernel of its own rather than attn_dq's work:
// there its loads stood before every unit, 3-4 us each (145 us against 10 + 48 for 61 ragged
// sequences of 9999 tokens, 16 heads of 64).
constexpr int kDeltaRows = 128;  // tokens of one head per block
template <int DP>
__global__ void __launch_bounds__(DP == 128 ? 256 : 128) attn_delta(const AttnBwdParams p) {
  constexpr int kPieces = DP / 64, kRows = 8 / kPieces, kStep = kDeltaRows / kRows;
  const int lane = threadIdx.x & 7, slot = threadIdx.x >> 3;
  const int64_t h = blockIdx.x % p.q_heads, t0 = (int64_t)(blockIdx.x / p.q_heads) * kDeltaRows + slot;
  uint4 a[kRows][kPieces], b[kRows][kPieces];
  float lse = 0.f;  // of row `lane`
  grid_wait();
#pragma unroll
  for (int i = 0; i < kRows; ++i)
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const int64_t t = t0 + kStep * i;
      const int d = lane * 8 + 64 * e;
      a[i][e] = b[i][e] = make_uint4(0, 0, 0, 0);
      if (t < p.tokens && d < p.head_dim) {
        const int64_t at = (t * p.q_heads + h) * p.head_dim + d;
        a[i][e] = *reinterpret_cast<const uint4*>(p.out + at);
        b[i][e] = *reinterpret_cast<const uint4*>(p.dout + at);
      }
    }
  const int64_t t = t0 + kStep * lane, at = h * p.tokens + t;
  const bool mine = lane < kRows && t < p.tokens;  // lane i writes row i
  if (mine) lse = p.lse[at];
  float delta = 0.f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
      const uint32_t x[4] = {a[i][e].x, a[i][e].y, a[i][e].z, a[i][e].w};
      const uint32_t y[4] = {b[i][e].x, b[i][e].y, b[i][e].z, b[i][e].w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        sum = fmaf(as_f(x[w] << 16), as_f(y[w] << 16), sum);
        sum = fmaf(as_f(x[w] & 0xffff0000u), as_f(y[w] & 0xffff0000u), sum);
      }
    }
#pragma unroll
    for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
    if (lane == i) delta = sum;
  }
  if (mine) {
    // A row whose scores are all -infinity has no softmax: + nl 0 makes its +infinity NaN, which
    // would make p infinite where the score is made of a cleaned query.
    const float nl = -lse * kLog2e;
    p.nlse[at] = fmaf(nl, 0.f, nl);
    p.delta[at] = delta;
  }
}

// ----------------------------------------------------------------------------
// dq
// ----------------------------------------------------------------------------
// TMEM: S, two dP buffers (dS overwrites its own), dQ.  S of the next key tile
// follows as soon as this one's is in registers, and its dP goes to the other
// buffer, so the tensor cores never wait for a dS other than dQ's own.  Three K
// tiles are held: of this step (for dQ += dS K), the next (S) and one in flight.
//
// S is made of the keys as they are, also on the diagonal, whose tile, if it holds a
// non-finite value, is cleaned between that product and dQ's: a key with an infinite value may have a score of -infinity, which
// leaves the row's softmax to its other keys (of the cleaned key it would be some finite
// score instead).  Its part of dq is then 0 x infinity, so that value of dq is NaN in every
// row that sees the key; the tile's non-finite values are all made up for in this way, for
// the rows where they give another score have a NaN lse.
template <int DP>
struct DqCfg {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  static constexpr int kK = DP == 128 ? 3 : 5, kV = DP == 128 ? 2 : 4;  // ring sizes
  static constexpr int kRingK = 2 * kTileBytes;                        // after Q and dout
  static constexpr int kRingV = kRingK + kK * kTileBytes;
  // 4 KB for each storing warp: dout's tile, or beside the rings where there is room
  static constexpr bool kThroughG = DP == 128;
  static constexpr int kStage = kThroughG ? kTileBytes : kRingV + kV * kTileBytes;
  static constexpr int kBars = kRingV + kV * kTileBytes + (kThroughG ? 0 : 4 * 4096);
  static constexpr int kSums = kBars + 512;  // by half and row: sums of p dP
  static constexpr int kSmem = kSums + 2 * kTile * 4;
};

struct DqShared {
  uint64_t kfull[5], kempty[5], vfull[4], vempty[4];
  uint64_t qfull, qempty, gfull, gempty;  // Q and dout tiles
  uint64_t sfull, sread, dpfull[2], dsfull, accfull, exchange;
  uint64_t diagonal;                      // S of a unit's diagonal tile is made
  uint64_t clean[2];
  uint64_t ufull[2], uempty[2];
  uint64_t mma_done;
  AttnUnit unit[2];
  uint32_t flags[2][4][4];  // by unit parity and cleaning warp: keys that are not finite
  uint32_t dirty[2][4];     // whether flags[..][warp] has any set
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(DqShared) <= 512, "barrier area");

// Makes `cols` values of a row of dq NaN where one of the diagonal keys it sees is not finite:
// keys 0 to `row` of a tile at k with a bit in flags[4][4].
__device__ __noinline__ void dq_nonfinite(bf16* dq, const bf16* k, int64_t k_row, const uint32_t* flags,
                                          int row, int cols) {
#pragma unroll 1
  for (int i = 0; i <= row; ++i) {
    const uint32_t* fl = flags + (i >> 5);
    if (((fl[0] | fl[4] | fl[8] | fl[12]) >> (i & 31)) & 1) add_nonfinite(dq, k + i * k_row, cols, 0.f);
  }
}

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dq(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
        const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
        const AttnBwdParams p) {
  using C = DqCfg<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  DqShared& sh = *reinterpret_cast<DqShared*>(smem + C::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx ctx{&sh.abort, p.err_word, p.timeout_ns};

  if (threadIdx.x == 0) {
    // a K slot is given back by the MMAs and by the cleaning warps, which so see
    // every K tile pass
    for (int i = 0; i < C::kK; ++i) mbar_init(&sh.kfull[i], 1), mbar_init(&sh.kempty[i], 5);
    for (int i = 0; i < C::kV; ++i) mbar_init(&sh.vfull[i], 1), mbar_init(&sh.vempty[i], 1);
    mbar_init(&sh.qfull, 1);
    mbar_init(&sh.qempty, 1);
    mbar_init(&sh.gfull, 1);
    mbar_init(&sh.gempty, C::kThroughG ? 9 : 1);  // the MMAs; the 8 compute warps if they store through it
    mbar_init(&sh.sfull, 1);
    mbar_init(&sh.sread, 8);
    mbar_init(&sh.dsfull, 8);
    mbar_init(&sh.accfull, 1);
    mbar_init(&sh.exchange, 8);
    mbar_init(&sh.diagonal, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.dpfull[i], 1);
      mbar_init(&sh.clean[i], 4);
      mbar_init(&sh.ufull[i], 1);
      mbar_init(&sh.uempty[i], 13);  // 8 compute warps, the MMA lane, 4 cleaning warps
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  grid_wait();
  const uint32_t t_acc = tmem + 3 * kTile;

  if (warp >= 8) regs_down<kBwdOtherRegs>();
  if (warp < 8) {
    // ------------------------------------------------------------ compute
    regs_up<kBwdComputeRegs>();
    const int half = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const float c = p.scale * kLog2e;
    const uint64_t c2 = pack_f32x2(c, c);
    float* sums = reinterpret_cast<float*>(smem + C::kSums);
    uint32_t step = 0, units = 0, singles = 0;
    for (uint32_t it = 0;; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = sh.unit[it & 1];
      if (u.head < 0) break;
      bool ok = true;
      if (u.len == 0) {  // rows of no sequence
        if (half == 0 && row < u.rows) {
          uint4* o = reinterpret_cast<uint4*>(
              p.dq + ((int64_t)(u.start + row) * p.q_heads + u.head) * p.head_dim);
#pragma unroll 1
          for (int d = 0; d < p.head_dim / 8; ++d) o[d] = make_uint4(0, 0, 0, 0);
        }
      } else {
        const bool live = u.q0 + row < u.len;
        const int64_t at = (int64_t)u.head * p.tokens + u.start + u.q0 + row;
        const float nl = live ? p.nlse[at] : 0.f, dl = live ? -p.delta[at] : 0.f;
        const uint64_t nl2 = pack_f32x2(nl, nl);
        uint64_t dl2 = pack_f32x2(dl, dl);
        const int n = u.q0 / kTile + 1;
        for (int j = n - 1; j >= 0; --j, ++step) {
          const uint32_t t_dp = tmem + (1 + (step & 1)) * kTile + lanes + half * 64;
          if (!(ok = wait_bar_warp(&sh.sfull, step & 1, ctx))) break;
          tc_fence_after();
          uint32_t s[2][32], g[2][32];
          load64(s, tmem + lanes + half * 64);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.sread);
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            float a, b;
            unpack_f32x2(fma_f32x2(pack_u32x2(s[i >> 5][i & 31], s[i >> 5][(i & 31) + 1]), c2, nl2), a, b);
            s[i >> 5][i & 31] = __float_as_uint(ex2_approx(a));
            s[i >> 5][(i & 31) + 1] = __float_as_uint(ex2_approx(b));
          }
          if (!(ok = wait_bar_warp(&sh.dpfull[step & 1], (step >> 1) & 1, ctx))) break;
          tc_fence_after();
          load64(g, t_dp);
          if (n == 1) {
            // A sequence's first rows see few keys, each with a large p, so that the rounding
            // of out in delta shows in their gradients.  All their keys are here: delta =
            // sum_j p_ij dP_ij in fp32 (dq and dk 3.6e-3 -> 2.4e-3 off for short sequences).
            mask_diagonal<false>(s, half);
            uint64_t sum = 0;
#pragma unroll
            for (int i = 0; i < 64; i += 2) {
              // a masked dP may be anything
              const uint32_t x = half * 64 + i <= row ? g[i >> 5][i & 31] : 0;
              const uint32_t y = half * 64 + i < row ? g[i >> 5][(i & 31) + 1] : 0;
              sum = fma_f32x2(pack_u32x2(s[i >> 5][i & 31], s[i >> 5][(i & 31) + 1]), pack_u32x2(x, y), sum);
            }
            float a, b;
            unpack_f32x2(sum, a, b);
            sums[half * kTile + row] = a + b;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.exchange);
            if (!(ok = wait_bar_warp(&sh.exchange, singles & 1, ctx))) break;
            ++singles;
            const float d = sums[row] + sums[kTile + row];
            dl2 = pack_f32x2(-d, -d);
            if (half == 0 && live) p.delta[at] = d;  // for attn_dkdv
          }
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            float a, b;
            unpack_f32x2(add_f32x2(pack_u32x2(g[i >> 5][i & 31], g[i >> 5][(i & 31) + 1]), dl2), a, b);
            s[i >> 5][i & 31] = __float_as_uint(a * as_f(s[i >> 5][i & 31]));
            s[i >> 5][(i & 31) + 1] = __float_as_uint(b * as_f(s[i >> 5][(i & 31) + 1]));
          }
          if (j == n - 1) {
            // dQ's product, which follows, reads the cleaned keys (the issuing warp waiting for
            // them: 501 us at 8192 tokens, 32 / 8 heads of 128, these: 490)
            if (!(ok = wait_bar_warp(&sh.clean[it & 1], (it >> 1) & 1, ctx))) break;
            mask_diagonal<false>(s, half);  // keys after the row
            if (u.q0 == 0) zero_first(s);
          }
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i)
            pk[i] = pack_bf16x2(as_f(s[i >> 4][2 * (i & 15)]), as_f(s[i >> 4][2 * (i & 15) + 1]));
          tmem_st_32x32b_x32(t_dp, pk);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.dsfull);
        }
        if (!ok || !wait_bar_warp(&sh.accfull, units & 1, ctx)) break;
        ++units;
        tc_fence_after();
        // each half of the warps writes half of the columns
        const int first = u.q0 + (warp & 3) * 32;
        if (DP == 128 || half == 0)
          store_rows(smem + C::kStage + warp * 4096, t_acc + lanes + half * 64, p.scale,
                     p.dq + ((int64_t)(u.start + first) * p.q_heads + u.head) * p.head_dim + half * 64,
                     (int64_t)p.q_heads * p.head_dim, u.len - first, min(64, p.head_dim - half * 64));
        const uint32_t* dw = sh.dirty[it & 1];
        if ((DP == 128 || half == 0) && (dw[0] | dw[1] | dw[2] | dw[3])) {
          __syncwarp();
          if (u.q0 + row < u.len)
            dq_nonfinite(p.dq + ((int64_t)(u.start + u.q0 + row) * p.q_heads + u.head) * p.head_dim + half * 64,
                         p.k + (int64_t)(u.start + u.q0) * p.k_row + (u.head / p.group) * p.k_head + half * 64,
                         p.k_row, sh.flags[it & 1][0], row, min(64, p.head_dim - half * 64));
          __syncwarp();
        }
        if (C::kThroughG) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.gempty);
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t tm = __shfl_sync(~0u, tmem, 0), el = elect_one();
    const uint32_t acc = tm + 3 * kTile;
    auto dp = [&](uint32_t t) { return tm + (1 + (t & 1)) * kTile; };
    const uint32_t q0 = smem_u32(smem), do0 = q0 + C::kTileBytes;
    const uint32_t kr = smem_u32(smem + C::kRingK), vr = smem_u32(smem + C::kRingV);
    uint32_t base = 0, units = 0;  // steps before this unit
    bool ok = true;
    auto issue_s = [&](uint32_t t) {
      if (!(ok = ok && wait_bar_warp(&sh.kfull[t % C::kK], (t / C::kK) & 1, ctx))) return;
      mma_tiles<DP>(el, tm, q0, kr + (t % C::kK) * C::kTileBytes);
      mma_commit_if(el, &sh.sfull);
    };
    auto issue_dp = [&](uint32_t t) {
      if (!(ok = ok && wait_bar_warp(&sh.vfull[t % C::kV], (t / C::kV) & 1, ctx))) return;
      mma_tiles<DP>(el, dp(t), do0, vr + (t % C::kV) * C::kTileBytes);
      mma_commit_if(el, &sh.dpfull[t & 1]);
      mma_commit_if(el, &sh.vempty[t % C::kV]);
    };
    for (uint32_t it = 0; ok; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = uniform(sh.unit[it & 1]);
      if (u.head < 0) break;
      if (u.len > 0) {
        const int n = u.q0 / kTile + 1;
        if (!wait_bar_warp(&sh.qfull, units & 1, ctx)) break;
        issue_s(base);
        mma_commit_if(el, &sh.diagonal);
        if (!(ok = ok && wait_bar_warp(&sh.gfull, units & 1, ctx))) break;
        issue_dp(base);
        if (n == 1) {
          mma_commit_if(el, &sh.qempty);
          mma_commit_if(el, &sh.gempty);
        }
        for (int i = 0; i < n && ok; ++i) {
          const uint32_t t = base + i;
          if (!(ok = wait_bar_warp(&sh.sread, t & 1, ctx))) break;
          tc_fence_after();
          if (i + 1 < n) {
            issue_s(t + 1);
            issue_dp(t + 1);
          }
          // Q and dout are free once the last S and dP are done
          if (i + 2 == n) {
            mma_commit_if(el, &sh.qempty);
            mma_commit_if(el, &sh.gempty);
          }
          if (!(ok = ok && wait_bar_warp(&sh.dsfull, t & 1, ctx))) break;
          tc_fence_after();
          mma_tmem_tile<DP>(el, acc, dp(t), 64, kr + (t % C::kK) * C::kTileBytes, i != 0);
          mma_commit_if(el, &sh.kempty[t % C::kK]);
        }
        if (!ok) break;
        mma_commit_if(el, &sh.accfull);
        base += n;
        ++units;
      }
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
      __syncwarp();
    }
    mma_commit_if(el, &sh.mma_done);
    if (el) {
      mbar_wait_drain(&sh.mma_done, 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ units, loads
    if (lane == 0) {
      prefetch_tensormap(&tq);
      prefetch_tensormap(&tk);
      prefetch_tensormap(&tv);
      prefetch_tensormap(&tdo);
    }
    UnitWalk<kTile> walk;
    walk.init(p);
    const int64_t total = (int64_t)walk.total() * p.q_heads;
    uint32_t t = 0, units = 0, nq = 0;
    uint32_t loaded_k = 0, loaded_v = 0;
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int64_t id = dealt_unit(it, blockIdx.x, gridDim.x);
      AttnUnit u{};
      u.head = -1;
      if (id < total) {
        u = walk.at((int)(id / p.q_heads));
        u.head = unit_ok(u, p) ? (int)(id % p.q_heads) : -1;
      }
      if (lane == 0) {
        ok = wait_bar(&sh.uempty[it & 1], ((it >> 1) & 1) ^ 1, ctx);
        if (ok) {
          sh.unit[it & 1] = u;
          mbar_arrive(&sh.ufull[it & 1]);
        }
        if (ok && u.len > 0) {
          const int kvh = u.head / p.group;
          if ((ok = wait_bar(&sh.qempty, (nq & 1) ^ 1, ctx))) {
            ++nq;
            mbar_arrive_expect_tx(&sh.qfull, C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_3d(smem + b * kBoxBytes, &tq, &sh.qfull, b * 64, u.head, u.start + u.q0);
          }
          for (int j = u.q0 / kTile; j >= 0 && ok; --j, ++t) {
            const int ks = t % C::kK, vs = t % C::kV, r = u.start + j * kTile;
            if (!(ok = wait_bar(&sh.kempty[ks], ((t / C::kK) & 1) ^ 1, ctx))) break;
            mbar_arrive_expect_tx(&sh.kfull[ks], C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_3d(smem + C::kRingK + ks * C::kTileBytes + b * kBoxBytes, &tk, &sh.kfull[ks],
                          b * 64, kvh, r);
            ++loaded_k;
            if (j == u.q0 / kTile) {  // dout only now: its tile is free after the last unit's store
              if (!(ok = wait_bar(&sh.gempty, (units & 1) ^ 1, ctx))) break;
              mbar_arrive_expect_tx(&sh.gfull, C::kTileBytes);
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_3d(smem + C::kTileBytes + b * kBoxBytes, &tdo, &sh.gfull, b * 64, u.head,
                            u.start + u.q0);
              ++units;
            }
            if (!(ok = wait_bar(&sh.vempty[vs], ((t / C::kV) & 1) ^ 1, ctx))) break;
            mbar_arrive_expect_tx(&sh.vfull[vs], C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_3d(smem + C::kRingV + vs * C::kTileBytes + b * kBoxBytes, &tv, &sh.vfull[vs],
                          b * 64, kvh, r);
            ++loaded_v;
          }
        }
      }
      ok = __shfl_sync(~0u, ok, 0);
      if (u.head < 0) break;
    }
    if (!ok && lane == 0) {
      if (nq) mbar_wait_drain(&sh.qfull, (nq - 1) & 1, p.timeout_ns);
      if (units) mbar_wait_drain(&sh.gfull, (units - 1) & 1, p.timeout_ns);
      for (uint32_t i = loaded_k > C::kK ? loaded_k - C::kK : 0; i < loaded_k; ++i)
        mbar_wait_drain(&sh.kfull[i % C::kK], (i / C::kK) & 1, p.timeout_ns);
      for (uint32_t i = loaded_v > C::kV ? loaded_v - C::kV : 0; i < loaded_v; ++i)
        mbar_wait_drain(&sh.vfull[i % C::kV], (i / C::kV) & 1, p.timeout_ns);
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ diagonal key tiles
    const int w = warp - 12;
    uint32_t t = 0, units = 0;
    for (uint32_t it = 0;; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = sh.unit[it & 1];
      if (u.head < 0) break;
      if (u.len > 0) {
        bool ok = true;
        for (int j = u.q0 / kTile; j >= 0; --j, ++t) {
          const uint32_t s = t % C::kK;
          if (!(ok = wait_bar_warp(&sh.kfull[s], (t / C::kK) & 1, ctx))) break;
          if (j == u.q0 / kTile) {
            // rows of another sequence are masked in S, so they are zeroed at any time
            uint8_t* tile = smem + C::kRingK + s * C::kTileBytes;
            if (u.len - u.q0 < kTile) zero_rows(tile, C::kBoxes, u.len - u.q0, w, 4);
            uint32_t* fl = sh.flags[it & 1][w];
            const bool dirty = has_nonfinite(tile, C::kBoxes, w, 4);
            if (dirty) {
              if (!(ok = wait_bar_warp(&sh.diagonal, units & 1, ctx))) break;
              clean_tile(tile, C::kBoxes, kTile, w, 4, fl);
            } else if (lane < 4) {
              fl[lane] = 0;
            }
            ++units;
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              sh.dirty[it & 1][w] = dirty;
              mbar_arrive(&sh.clean[it & 1]);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.kempty[s]);
        }
        if (!ok) break;
      } else if (lane == 0) {
        mbar_arrive(&sh.clean[it & 1]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ----------------------------------------------------------------------------
// dk, dv
// ----------------------------------------------------------------------------
// Products with keys as rows: S^T = K Q^T, dP^T = V dout^T (128 keys x 128
// queries), dV += P^T dout, dK += dS^T Q with P^T and dS^T read from TMEM, where
// they overwrite S^T and dP^T.  While the threads make P of a step, the tensor
// cores run the last step's dK and this one's dP; while they make dS, this
// step's dV and the next S.
//
// A ragged last tile of queries is filled up with copies of the last query, whose lse counts
// as +infinity: p is 0, and so are they in the sums.  (Of zeros a key with an infinite value
// would make 0 x infinity.)  The last query sees every key, so where a copy's score is such that
// its p is NaN, the query's own p and with it the key's dv and dk are NaN.  Its dout is zero:
// dP of a copy is NaN only for a value that is not finite, whose key's dk is NaN anyhow.
template <int DP>
struct DkvCfg {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  // Q tiles (read by S and, last of a step, by dK) and dout tiles (dP, dV)
  static constexpr int kQ = DP == 128 ? 3 : 4, kG = DP == 128 ? 2 : 4;
  static constexpr int kRingQ = 2 * kTileBytes;      // after K and V
  static constexpr int kRingG = kRingQ + kQ * kTileBytes;
  // 4 KB for each compute warp's stores: V's tile, or beside the rings where there is
  // room
  static constexpr bool kThroughV = DP == 128;
  static constexpr int kStage = kThroughV ? kTileBytes : kRingG + kG * kTileBytes;
  static constexpr int kBars = kRingG + kG * kTileBytes + (kThroughV ? 0 : 8 * 4096);
  static constexpr int kStatStages = 2;              // -lse and delta of 128 queries
  static constexpr int kSmem = kBars + kStatStages * 1024 + 1024;  // 227 KB at 128
};

struct DkvShared {
  uint64_t qfull[4], qempty[4], gfull[4], gempty[4];  // Q and dout tiles
  uint64_t tfull[4], tempty[4];                       // statistics
  uint64_t kfull, kempty, vfull, vempty;
  uint64_t sfull, dpfull, pfull, dsfull, accfull;
  uint64_t clean[4];                                  // by stage
  uint64_t ufull[2], uempty[2];
  uint64_t mma_done;
  AttnUnit unit[2];
  uint32_t flags[4][4];  // by cleaning warp: non-finite rows of the tile it is at
  uint32_t dirty[2][4];  // by unit parity and cleaning warp: non-finite dout on the diagonal
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(DkvShared) <= 1024, "barrier area");

// Whether the query tile `i` of a unit whose diagonal tile is `first` has to be
// cleaned: the diagonal one, and a ragged last one.
__device__ __forceinline__ bool dkv_cleaned(const AttnUnit& u, int i, int first) {
  return i == first || u.len - i * kTile < kTile;
}

template <int DP>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_dkdv(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
          const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tdo,
          const AttnBwdParams p) {
  using C = DkvCfg<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  DkvShared& sh = *reinterpret_cast<DkvShared*>(smem + C::kBars + C::kStatStages * 1024);
  float* stat = reinterpret_cast<float*>(smem + C::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx ctx{&sh.abort, p.err_word, p.timeout_ns};
  const int heads = p.kv_heads * p.splits, per_split = p.group / p.splits;

  if (threadIdx.x == 0) {
    // slots are given back by the MMAs and by the cleaning warps, which so see
    // every tile pass
    for (int i = 0; i < C::kQ; ++i) {
      mbar_init(&sh.qfull[i], 1), mbar_init(&sh.qempty[i], 5);
      mbar_init(&sh.clean[i], 4);
    }
    for (int i = 0; i < C::kG; ++i) mbar_init(&sh.gfull[i], 1), mbar_init(&sh.gempty[i], 5);
    for (int i = 0; i < C::kStatStages; ++i) mbar_init(&sh.tfull[i], 1), mbar_init(&sh.tempty[i], 8);
    mbar_init(&sh.kfull, 1);
    mbar_init(&sh.kempty, 1);
    mbar_init(&sh.vfull, 1);
    mbar_init(&sh.vempty, C::kThroughV ? 9 : 1);  // the MMAs; the 8 compute warps if they store through it
    mbar_init(&sh.sfull, 1);
    mbar_init(&sh.dpfull, 1);
    mbar_init(&sh.pfull, 8);
    mbar_init(&sh.dsfull, 8);
    mbar_init(&sh.accfull, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.ufull[i], 1);
      mbar_init(&sh.uempty[i], 14);  // 8 compute, the MMA lane, statistics, 4 cleaning warps
    }
    mbar_init(&sh.mma_done, 1);
    sh.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  grid_wait();
  const uint32_t t_s = tmem, t_dp = tmem + kTile, t_dv = tmem + 2 * kTile, t_dk = tmem + 3 * kTile;

  if (warp >= 8) regs_down<kBwdOtherRegs>();
  if (warp < 8) {
    // ------------------------------------------------------------ compute
    regs_up<kBwdComputeRegs>();
    const int half = warp >> 2, row = threadIdx.x & 127;  // 64 queries; a key
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;
    const float c = p.scale * kLog2e;
    const uint64_t c2 = pack_f32x2(c, c);
    uint32_t step = 0, units = 0;
    for (uint32_t it = 0;; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = sh.unit[it & 1];
      if (u.head < 0) break;
      const int kvh = u.head / p.splits, split = u.head % p.splits;
      bool ok = true;
      if (u.len == 0) {  // rows of no sequence
        if (row < u.rows) {
          const int64_t at = ((int64_t)(u.start + row) * p.kv_heads + kvh) * p.head_dim;
          uint4* o = p.splits == 1 ? reinterpret_cast<uint4*>((half ? p.dk : p.dv) + at)
                                   : reinterpret_cast<uint4*>(p.partial + p.partial_at(!half, split) + at);
#pragma unroll 1
          for (int d = 0; d < p.head_dim / (p.splits == 1 ? 8 : 4); ++d) o[d] = make_uint4(0, 0, 0, 0);
        }
      } else {
        const int first = u.q0 / kTile, end = (u.len + kTile - 1) / kTile;
        for (int h = 0; h < per_split && ok; ++h)
          for (int i = first; i < end; ++i, ++step) {
            const uint32_t ts = step % C::kStatStages;
            if (!(ok = wait_bar_warp(&sh.tfull[ts], (step / C::kStatStages) & 1, ctx))) break;
            const float* nl = stat + ts * 256 + half * 64;
            if (!(ok = wait_bar_warp(&sh.sfull, step & 1, ctx))) break;
            tc_fence_after();
            uint32_t s[2][32];
            load64(s, t_s + lanes + half * 64);
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const float4 b = *reinterpret_cast<const float4*>(nl + e);
              uint32_t(&r)[32] = s[e >> 5];
              const int i0 = e & 31;
              float x, y;
              unpack_f32x2(fma_f32x2(pack_u32x2(r[i0], r[i0 + 1]), c2, pack_f32x2(b.x, b.y)), x, y);
              r[i0] = __float_as_uint(ex2_approx(x));
              r[i0 + 1] = __float_as_uint(ex2_approx(y));
              unpack_f32x2(fma_f32x2(pack_u32x2(r[i0 + 2], r[i0 + 3]), c2, pack_f32x2(b.z, b.w)), x, y);
              r[i0 + 2] = __float_as_uint(ex2_approx(x));
              r[i0 + 3] = __float_as_uint(ex2_approx(y));
            }
            if (i == first) mask_diagonal<true>(s, half);  // queries before the key
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 32; ++e)
              pk[e] = pack_bf16x2(as_f(s[e >> 4][2 * (e & 15)]), as_f(s[e >> 4][2 * (e & 15) + 1]));
            tmem_st_32x32b_x32(t_s + lanes + half * 64, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.pfull);
            if (!(ok = wait_bar_warp(&sh.dpfull, step & 1, ctx))) break;
            tc_fence_after();
            uint32_t g[2][32];
            load64(g, t_dp + lanes + half * 64);
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              const float4 b = *reinterpret_cast<const float4*>(nl + 128 + e);
              uint32_t(&r)[32] = g[e >> 5];
              const uint32_t(&q)[32] = s[e >> 5];
              const int i0 = e & 31;
              r[i0] = __float_as_uint((as_f(r[i0]) - b.x) * as_f(q[i0]));
              r[i0 + 1] = __float_as_uint((as_f(r[i0 + 1]) - b.y) * as_f(q[i0 + 1]));
              r[i0 + 2] = __float_as_uint((as_f(r[i0 + 2]) - b.z) * as_f(q[i0 + 2]));
              r[i0 + 3] = __float_as_uint((as_f(r[i0 + 3]) - b.w) * as_f(q[i0 + 3]));
            }
            if (i == first) {
              mask_diagonal<true>(g, half);
              if (u.q0 == 0) zero_first(g);
            }
#pragma unroll
            for (int e = 0; e < 32; ++e)
              pk[e] = pack_bf16x2(as_f(g[e >> 4][2 * (e & 15)]), as_f(g[e >> 4][2 * (e & 15) + 1]));
            tmem_st_32x32b_x32(t_dp + lanes + half * 64, pk);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&sh.dsfull);
              mbar_arrive(&sh.tempty[ts]);
            }
          }
        if (!ok || !wait_bar_warp(&sh.accfull, units & 1, ctx)) break;
        ++units;
        tc_fence_after();
        // warps 0-3 write dV, warps 4-7 dK
        const int row0 = u.q0 + (warp & 3) * 32, r = row0 + lane;  // the warp's first; this lane's
        const float scale = half ? p.scale : 1.f;
        const int64_t stride = (int64_t)p.kv_heads * p.head_dim;
        const int64_t at = (int64_t)(u.start + row0) * stride + kvh * p.head_dim;
        const uint32_t* dw = sh.dirty[it & 1];
        const bool dirty = half == 0 && (dw[0] | dw[1] | dw[2] | dw[3]);
        uint8_t* stage = smem + C::kStage + warp * 4096;
        const uint32_t from = (half ? t_dk : t_dv) + lanes;
        if (p.splits == 1)
          store_rows(stage, from, scale, (half ? p.dk : p.dv) + at, stride, u.len - row0, p.head_dim);
        else
          store_rows(stage, from, scale, p.partial + p.partial_at(!half, split) + at, stride,
                     u.len - row0, p.head_dim);
        if (dirty) {  // add back the non-finite values of dout that each key sees
          __syncwarp();
#pragma unroll 1
          for (int i = row; r < u.len && i < kTile * per_split; ++i) {
            const int q = i % kTile;  // query of the diagonal tile
            if (q < row || u.q0 + q >= u.len) continue;
            const bf16* g = p.dout + ((int64_t)(u.start + u.q0 + q) * p.q_heads + kvh * p.group +
                                      split * per_split + i / kTile) * p.head_dim;
            if (p.splits == 1) add_nonfinite(p.dv + at + lane * stride, g, p.head_dim, 1.f);
            else add_nonfinite(p.partial + p.partial_at(true, split) + at + lane * stride, g, p.head_dim, 1.f);
          }
          __syncwarp();
        }
        if (C::kThroughV) {
          fence_proxy_async_shared();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.vempty);
        }
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t tm = __shfl_sync(~0u, tmem, 0), el = elect_one();
    const uint32_t a_s = tm, a_dp = tm + kTile, a_dv = tm + 2 * kTile, a_dk = tm + 3 * kTile;
    const uint32_t k0 = smem_u32(smem), v0 = k0 + C::kTileBytes;
    const uint32_t ring_q = smem_u32(smem + C::kRingQ), ring_g = smem_u32(smem + C::kRingG);
    uint32_t base = 0, units = 0, nclean = 0;  // nclean: next phase of each Q slot's barrier
    bool ok = true;
    auto q_tile = [&](uint32_t t) { return ring_q + (t % C::kQ) * C::kTileBytes; };
    auto g_tile = [&](uint32_t t) { return ring_g + (t % C::kG) * C::kTileBytes; };
    // waits for step t's Q (S and later dK read it) and, if it is cleaned, for that
    auto issue_s = [&](uint32_t t, bool cleaned) {
      const uint32_t s = t % C::kQ;
      if (!(ok = ok && wait_bar_warp(&sh.qfull[s], (t / C::kQ) & 1, ctx))) return;
      if (cleaned) {
        if (!(ok = wait_bar_warp(&sh.clean[s], (nclean >> s) & 1, ctx))) return;
        nclean ^= 1u << s;
      }
      mma_tiles<DP>(el, a_s, k0, q_tile(t));
      mma_commit_if(el, &sh.sfull);
    };
    auto issue_dp = [&](uint32_t t) {
      if (!(ok = ok && wait_bar_warp(&sh.gfull[t % C::kG], (t / C::kG) & 1, ctx))) return;
      mma_tiles<DP>(el, a_dp, v0, g_tile(t));
      mma_commit_if(el, &sh.dpfull);
    };
    for (uint32_t it = 0; ok; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = uniform(sh.unit[it & 1]);
      if (u.head < 0) break;
      if (u.len > 0) {
        const int first = u.q0 / kTile, tiles = (u.len + kTile - 1) / kTile - first;
        const int n = tiles * per_split;
        if (!wait_bar_warp(&sh.kfull, units & 1, ctx)) break;
        issue_s(base, true);
        if (!(ok = ok && wait_bar_warp(&sh.vfull, units & 1, ctx))) break;
        issue_dp(base);
        if (n == 1) {
          mma_commit_if(el, &sh.kempty);
          mma_commit_if(el, &sh.vempty);
        }
        int i = 0;  // query tile of step x within its head
        for (int x = 0; x < n && ok; ++x) {
          const uint32_t t = base + x;
          if (!(ok = wait_bar_warp(&sh.pfull, t & 1, ctx))) break;
          tc_fence_after();
          mma_tmem_tile<DP>(el, a_dv, a_s, 64, g_tile(t), x != 0);
          mma_commit_if(el, &sh.gempty[t % C::kG]);
          if (++i == tiles) i = 0;
          if (x + 1 < n) issue_s(t + 1, dkv_cleaned(u, first + i, first));
          if (!(ok = ok && wait_bar_warp(&sh.dsfull, t & 1, ctx))) break;
          tc_fence_after();
          mma_tmem_tile<DP>(el, a_dk, a_dp, 64, q_tile(t), x != 0);
          mma_commit_if(el, &sh.qempty[t % C::kQ]);
          if (x + 1 < n) issue_dp(t + 1);
          if (x + 2 == n) {
            mma_commit_if(el, &sh.kempty);
            mma_commit_if(el, &sh.vempty);
          }
        }
        if (!ok) break;
        mma_commit_if(el, &sh.accfull);
        base += n;
        ++units;
      }
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
      __syncwarp();
    }
    mma_commit_if(el, &sh.mma_done);
    if (el) {
      mbar_wait_drain(&sh.mma_done, 0, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ units, loads
    if (lane == 0) {
      prefetch_tensormap(&tq);
      prefetch_tensormap(&tk);
      prefetch_tensormap(&tv);
      prefetch_tensormap(&tdo);
    }
    UnitWalk<kTile> walk;
    walk.init(p);
    const int64_t total = (int64_t)walk.total() * heads;
    uint32_t nq = 0, ng = 0, nk = 0, nv = 0;
    bool ok = true;
    for (uint32_t it = 0; ok; ++it) {
      const int64_t id = dealt_unit(it, blockIdx.x, gridDim.x);
      AttnUnit u{};
      u.head = -1;
      if (id < total) {
        u = walk.at((int)(id / heads));
        u.head = unit_ok(u, p) ? (int)(id % heads) : -1;
        // the walk counts from the sequence's start, key tiles have the most
        // queries there: mirrored
        if (u.len > 0) u.q0 = ((u.len + kTile - 1) / kTile - 1) * kTile - u.q0;
      }
      if (lane == 0) {
        ok = wait_bar(&sh.uempty[it & 1], ((it >> 1) & 1) ^ 1, ctx);
        if (ok) {
          sh.unit[it & 1] = u;
          mbar_arrive(&sh.ufull[it & 1]);
        }
        if (ok && u.len > 0) {
          const int kvh = u.head / p.splits;
          const int h0 = kvh * p.group + (u.head % p.splits) * per_split;
          if ((ok = wait_bar(&sh.kempty, (nk & 1) ^ 1, ctx))) {
            mbar_arrive_expect_tx(&sh.kfull, C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b)
              tma_load_3d(smem + b * kBoxBytes, &tk, &sh.kfull, b * 64, kvh, u.start + u.q0);
            ++nk;
          }
          for (int h = h0; h < h0 + per_split && ok; ++h)
            for (int i = u.q0; i < u.len; i += kTile) {
              const int qs = nq % C::kQ, gs = ng % C::kG;
              if (!(ok = wait_bar(&sh.qempty[qs], ((nq / C::kQ) & 1) ^ 1, ctx))) break;
              mbar_arrive_expect_tx(&sh.qfull[qs], C::kTileBytes);
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_3d(smem + C::kRingQ + qs * C::kTileBytes + b * kBoxBytes, &tq, &sh.qfull[qs],
                            b * 64, h, u.start + i);
              ++nq;
              if (h == h0 && i == u.q0) {  // V only now: its tile is free after the last unit's store
                if (!(ok = wait_bar(&sh.vempty, (nv & 1) ^ 1, ctx))) break;
                mbar_arrive_expect_tx(&sh.vfull, C::kTileBytes);
                for (int b = 0; b < C::kBoxes; ++b)
                  tma_load_3d(smem + C::kTileBytes + b * kBoxBytes, &tv, &sh.vfull, b * 64, kvh,
                              u.start + u.q0);
                ++nv;
              }
              if (!(ok = wait_bar(&sh.gempty[gs], ((ng / C::kG) & 1) ^ 1, ctx))) break;
              mbar_arrive_expect_tx(&sh.gfull[gs], C::kTileBytes);
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_3d(smem + C::kRingG + gs * C::kTileBytes + b * kBoxBytes, &tdo, &sh.gfull[gs],
                            b * 64, h, u.start + i);
              ++ng;
            }
        }
      }
      ok = __shfl_sync(~0u, ok, 0);
      if (u.head < 0) break;
    }
    if (!ok && lane == 0) {
      if (nk) mbar_wait_drain(&sh.kfull, (nk - 1) & 1, p.timeout_ns);
      if (nv) mbar_wait_drain(&sh.vfull, (nv - 1) & 1, p.timeout_ns);
      for (uint32_t i = nq > C::kQ ? nq - C::kQ : 0; i < nq; ++i)
        mbar_wait_drain(&sh.qfull[i % C::kQ], (i / C::kQ) & 1, p.timeout_ns);
      for (uint32_t i = ng > C::kG ? ng - C::kG : 0; i < ng; ++i)
        mbar_wait_drain(&sh.gfull[i % C::kG], (i / C::kG) & 1, p.timeout_ns);
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ statistics of the queries
    uint32_t step = 0;
    for (uint32_t it = 0;; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = sh.unit[it & 1];
      if (u.head < 0) break;
      const int kvh = u.head / p.splits;
      const int h0 = kvh * p.group + (u.head % p.splits) * per_split;
      bool ok = true;
      if (u.len > 0)
        for (int h = h0; h < h0 + per_split && ok; ++h)
          for (int i = u.q0; i < u.len; i += kTile, ++step) {
            const uint32_t ts = step % C::kStatStages;
            const int64_t at = (int64_t)h * p.tokens + u.start + i;
            float nl[4], dl[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = e * 32 + lane;
              const bool in = i + r < u.len;
              nl[e] = in ? p.nlse[at + r] : -INFINITY;  // beyond the sequence: p = 0
              dl[e] = in ? p.delta[at + r] : 0.f;
            }
            if (!(ok = wait_bar_warp(&sh.tempty[ts], ((step / C::kStatStages) & 1) ^ 1, ctx))) break;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              stat[ts * 256 + e * 32 + lane] = nl[e];
              stat[ts * 256 + 128 + e * 32 + lane] = dl[e];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.tfull[ts]);
          }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
    }
  } else if (warp >= 12) {
    // ------------------------------------------------------------ cleaned tiles
    const int w = warp - 12;
    uint32_t step = 0;
    for (uint32_t it = 0;; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = sh.unit[it & 1];
      if (u.head < 0) break;
      bool ok = true;
      if (lane == 0) sh.dirty[it & 1][w] = 0;
      if (u.len > 0) {
        const int first = u.q0 / kTile, end = (u.len + kTile - 1) / kTile;
        for (int h = 0; h < per_split && ok; ++h)
          for (int i = first; i < end; ++i, ++step) {
            const uint32_t qs = step % C::kQ, gs = step % C::kG;
            uint8_t* q = smem + C::kRingQ + qs * C::kTileBytes;
            uint8_t* g = smem + C::kRingG + gs * C::kTileBytes;
            const int valid = u.len - i * kTile;
            if (!(ok = wait_bar_warp(&sh.qfull[qs], (step / C::kQ) & 1, ctx))) break;
            if (valid < kTile) repeat_row(q, C::kBoxes, valid, w, 4);
            // a query that is not finite has no finite lse: nothing to add back
            if (i == first) clean_tile(q, C::kBoxes, kTile, w, 4, sh.flags[w]);
            if (!(ok = wait_bar_warp(&sh.gfull[gs], (step / C::kG) & 1, ctx))) break;
            if (i == first) {
              uint32_t* fl = sh.flags[w];
              clean_tile(g, C::kBoxes, valid, w, 4, fl);
              __syncwarp();
              if (lane == 0 && (fl[0] | fl[1] | fl[2] | fl[3])) sh.dirty[it & 1][w] = 1;
            } else if (valid < kTile) {
              zero_rows(g, C::kBoxes, valid, w, 4);
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
              if (dkv_cleaned(u, i, first)) mbar_arrive(&sh.clean[qs]);
              mbar_arrive(&sh.qempty[qs]);
              mbar_arrive(&sh.gempty[gs]);
            }
          }
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dk, dv = sums of the splits' partial ones, in a fixed order.  Bound by reading them
// once, 16 bytes a lane; only with more than one split.
__global__ void __launch_bounds__(256) attn_sum_splits(const AttnBwdParams p) {
  const int64_t size = (int64_t)p.tokens * p.kv_heads * p.head_dim;
  const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  grid_wait();
  if (i >= size) return;
  const float* from = p.partial + (int64_t)blockIdx.y * p.splits * size + i;
  float4 t = *reinterpret_cast<const float4*>(from);
  for (int s = 1; s < p.splits; ++s) {
    const float4 x = *reinterpret_cast<const float4*>(from + s * size);
    t.x += x.x, t.y += x.y, t.z += x.z, t.w += x.w;
  }
  *reinterpret_cast<uint2*>((blockIdx.y ? p.dv : p.dk) + i) =
      make_uint2(pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w));
}

}  // namespace flce
