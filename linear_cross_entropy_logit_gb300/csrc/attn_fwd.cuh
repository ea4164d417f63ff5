// Forward of packed causal attention on the tensor cores.
//
//   s_ij = scale q_i . k_j,  m_i a moving reference,  p_ij = 2^((s_ij - m_i) log2 e)
//   l_i = sum_j p_ij,  out_i = sum_j p_ij v_j / l_i,  lse_i = m_i + log l_i
//
// A persistent CTA takes units of 256 query rows of one sequence and head: two
// tiles of 128, so that one tile's softmax runs beside the other's products.
//   warps 0-3, 4-7  softmax of tile 0 / 1: a thread owns one row (TMEM lane)
//   warp 8          issues the MMAs (one lane)
//   warp 9          maps the units and loads Q, K and V by TMA
//   warps 10-11     clean the value tile on the diagonal (see below)
// TMEM: S of each tile (128 columns; P overwrites it as packed bf16) and O of
// each tile.  S = Q K^T reads both operands from shared memory, O += P V reads
// P from TMEM.  MMAs complete in order, so S of the next key tile may follow
// the product that reads P out of the same columns, and a softmax that sees its
// S also knows that every earlier product into its O is done.
//
// Key tiles run from the diagonal down: only the first tile of a query tile
// needs a mask (key <= row).  The rest of a ragged last tile belongs to the
// next sequence: its keys are masked by the same comparison, its values are
// zeroed in shared memory, since 0 x NaN is NaN.  Non-finite values inside the
// sequence that only some rows see are zeroed too and added back in the
// epilogue to the rows that see them.
//
// Exponentials are relative to a reference, the diagonal tile's maximum at first.  It is
// only moved when they would pass 2^kMoveLog2, and O and l with it: until then O is left alone. So
// half of a tile's exponentials are made at once, and made again in the rare case that it
// moves; their sum tells whether it has to for them, and the other half's maximum for those
// (the maximum of both halves: 142 / 136 us for 37 ragged sequences of 16384 tokens, 985 / 954
// at 32768 tokens, 8 / 2 heads of 64; both halves by their sums, the second's reference
// moved by itself: 140 and 1013).  P is handed over in halves, the first to be multiplied
// while the second is made.  An exponential is 2^-kShiftLog2 at the reference, so that none
// passes 2^-16 and no sum over 65536 keys of them times finite values leaves fp32's range (at
// 1, values above 5e33 did); l carries the same factor.  l is fp32; P is rounded to bf16
// (the type of V, at most 2^-8 of it), and l sums it before that rounding.
//
// What bounds it (times of calls one after the other).  Heads of 128: a tile's chain of S,
// softmax, P V and the next S, as TMEM holds one S and one O a tile (all 512 columns): 361 us
// at 8192 tokens, 32 / 8 heads, 1520 TFLOP/s of the visible pairs, tensor pipe 67% active
// (a launch by itself takes 339 to 348).  Heads of 64: the same chain with half the products
// in it, no pipe above 50%: 953 us at 32768 tokens, 8 / 2 heads, 1154 TFLOP/s.  Short
// sequences: each unit's latency of some 6000 cycles and the empty part of its tiles: 136 us
// for 37 ragged sequences of 16384 tokens, 28 / 4 heads of 128, 620 TFLOP/s.  Tried and slower: a third or fourth softmax warpgroup, the
// epilogue in warps of its own, S ahead of P in more buffers, two issuing warps.
#pragma once
#include "attn_common.cuh"

namespace flce {

constexpr int kFwdThreads = 384;
constexpr int kFwdRows = 2 * kTile;
constexpr float kMoveLog2 = 16.f, kShiftLog2 = 32.f;
static_assert(kShiftLog2 - kMoveLog2 == 16.f, "0x1p16f where the reference moves");
// Registers per thread of the two softmax warpgroups and of the third: a
// softmax thread holds a row of 128 scores.
constexpr int kFwdSoftmaxRegs = 216, kFwdOtherRegs = 72;
static_assert(2 * kFwdSoftmaxRegs + kFwdOtherRegs == 3 * (65536 / kFwdThreads / 8 * 8),
              "shares add up to what the block is launched with");

template <int DP>
struct FwdCfg {
  static constexpr int kBoxes = DP / 64;
  static constexpr int kTileBytes = kBoxes * kBoxBytes;
  // A stage of the ring holds what one step needs: V of a key tile and K of the next (the
  // first of a unit only K, the last only V).  One wait and one release a step: each costs
  // the issuing warp some 150 to 250 cycles beside the softmax.  A ring of single tiles /
  // this: 355 / 340 us at 8192 tokens, 32 / 8 heads of 128; 1020 / 976 us at 32768 tokens,
  // 8 / 2 heads of 64.
  static constexpr int kStages = DP == 128 ? 2 : 4;
  static constexpr int kRing = 2 * kTileBytes;      // after the two Q tiles
  static constexpr int kStage = kRing + kStages * 2 * kTileBytes;  // 4 KB for each softmax warp
  static constexpr int kBars = kStage + 8 * 4096;
  static constexpr int kSmem = kBars + 512;
};

struct FwdShared {
  uint64_t full[4], empty[4];  // ring of K and V tiles
  uint64_t qfull, qempty;
  uint64_t sfull[2], phalf[2], pfull[2], ofull[2];
  uint64_t clean[2][2];        // by unit parity and query tile: its diagonal value tile is fit for use
  uint64_t ufull[2], uempty[2];
  uint64_t mma_done;
  AttnUnit unit[2];
  uint32_t flags[2][2][2][4];  // by unit parity, diagonal tile and cleaning warp: non-finite rows
  alignas(16) uint32_t any[2][4];  // by unit parity: whether flags[..][tile][warp] has any set
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(FwdShared) <= 512, "barrier area");

// Tiles of a unit: key tiles of query tile 0 and 1 (0: it has no rows).
__device__ __forceinline__ void unit_tiles(const AttnUnit& u, int& n0, int& n1) {
  n0 = u.len > 0 ? u.q0 / kTile + 1 : 0;
  n1 = u.q0 + kTile < u.len ? n0 + 1 : 0;
}

template <int DP>
__global__ void __launch_bounds__(kFwdThreads, 1)
attn_fwd(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
         const __grid_constant__ CUtensorMap tv, const AttnParams p) {
  using C = FwdCfg<DP>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* ring = smem + C::kRing;
  FwdShared& sh = *reinterpret_cast<FwdShared*>(smem + C::kBars);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const WaitCtx ctx{&sh.abort, p.err_word, p.timeout_ns};

  if (threadIdx.x == 0) {
    // a stage is given back by the MMAs and by both cleaning warps, which so see every
    // stage pass
    for (int i = 0; i < C::kStages; ++i) mbar_init(&sh.full[i], 1), mbar_init(&sh.empty[i], 3);
    mbar_init(&sh.qfull, 1);
    mbar_init(&sh.qempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.sfull[i], 1);
      mbar_init(&sh.phalf[i], 4);
      mbar_init(&sh.pfull[i], 4);
      mbar_init(&sh.ofull[i], 1);
      mbar_init(&sh.ufull[i], 1);
      mbar_init(&sh.uempty[i], 11);  // 8 softmax warps, the MMA lane, 2 cleaning warps
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.clean[i >> 1][i & 1], 2);
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

  if (warp >= 8) regs_down<kFwdOtherRegs>();
  if (warp < 8) {
    // ------------------------------------------------------------ softmax
    regs_up<kFwdSoftmaxRegs>();
    const int x = warp >> 2;           // query tile
    const int row = threadIdx.x & 127; // row of the tile = TMEM lane
    const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // (32 * warp) << 16
    const uint32_t ts = tmem + lanes + x * kTile;
    const uint32_t to = tmem + lanes + 2 * kTile + x * DP;
    const float c = p.scale * kLog2e;
    uint32_t ns = 0, no = 0;  // tiles and units of this query tile so far
    for (uint32_t it = 0;; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = sh.unit[it & 1];
      if (u.head < 0) break;
      int n0, n1;
      unit_tiles(u, n0, n1);
      const int n = x ? n1 : n0;
      if (u.len == 0) {  // rows of no sequence
        const int r = x * kTile + row;
        if (r < u.rows) {
          const int64_t t = u.start + r;
          p.lse[(int64_t)u.head * p.tokens + t] = -INFINITY;
          uint4* o = reinterpret_cast<uint4*>(p.out + (t * p.q_heads + u.head) * p.head_dim);
#pragma unroll 1
          for (int d = 0; d < p.head_dim / 8; ++d) o[d] = make_uint4(0, 0, 0, 0);
        }
      }
      if (n == 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
        continue;
      }
      float b = 0.f, l = 0.f;  // p = 2^(s c + b), l their sum; 2^-kShiftLog2 of what they stand for
      bool ok = true;
      for (int j = n - 1; j >= 0; --j, ++ns) {
        if (!(ok = wait_bar_warp(&sh.sfull[x], ns & 1, ctx))) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(ts + 32 * i, s[i]);
        tmem_ld_wait();
        auto row_max = [&](int i0) {  // of runs i0 to 3
          float mx[4];
#pragma unroll
          for (int i = i0; i < 4; ++i) {
            mx[i] = __uint_as_float(s[i][0]);
#pragma unroll
            for (int e = 1; e < 31; e += 2)
              mx[i] = fmax3(mx[i], __uint_as_float(s[i][e]), __uint_as_float(s[i][e + 1]));
            mx[i] = fmaxf(mx[i], __uint_as_float(s[i][31]));
          }
          return i0 ? fmaxf(mx[2], mx[3]) : fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        };
        uint64_t sum[4];
        // P of half of the row's keys; returns its sum
        auto half = [&](int i0) {
          const uint64_t c2 = pack_f32x2(c, c), b2 = pack_f32x2(b, b);
#pragma unroll
          for (int i = i0; i < i0 + 2; ++i) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float p0, p1;
              unpack_f32x2(fma_f32x2(pack_u32x2(s[i][e], s[i][e + 1]), c2, b2), p0, p1);
              p0 = ex2_approx(p0);
              p1 = ex2_approx(p1);
              const uint64_t both = pack_f32x2(p0, p1);
              sum[(e >> 1) & 3] = i == i0 && e < 8 ? both : add_f32x2(sum[(e >> 1) & 3], both);
              pk[e >> 1] = pack_bf16x2(p0, p1);
            }
            tmem_st_32x32b_x16(ts + 16 * i, pk);
          }
          float l0, l1;
          unpack_f32x2(add_f32x2(add_f32x2(sum[0], sum[1]), add_f32x2(sum[2], sum[3])), l0, l1);
          return l0 + l1;
        };
        auto ready = [&](uint64_t* bar) {
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar);
        };
        if (j == n - 1) {  // the diagonal
          // a warp's 32 rows meet the diagonal in one run of 32 keys; those after it are masked
          // whole.  Branches: as selects these would cost every tile.
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (i == (warp & 3)) {
              asm volatile("");
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (e > lane) s[i][e] = 0xff800000u;  // -infinity
            } else if (i > (warp & 3)) {
              asm volatile("");
#pragma unroll
              for (int e = 0; e < 32; ++e) s[i][e] = 0xff800000u;
            }
          }
          const float top = row_max(0);
          b = top == -INFINITY ? 0.f : fmaf(-top, c, -kShiftLog2);  // no key so far: l stays 0
        }
        // The first half goes by the reference so far: its sum, and the second half's
        // maximum, tell whether it has to move.
        float s0;
        for (bool again = false;; again = true) {
          s0 = half(0);
          const bool empty = l == 0.f && j < n - 1;
          const bool move =
              fmaxf(s0 * 0x1p16f, fmaf(row_max(2), c, b) + (kShiftLog2 - kMoveLog2 + 1.f)) > 1.f || empty;
          if (again || !__any_sync(~0u, move)) break;
          // b moves, O and l are rescaled, and the half is done again
          float f = 1.f;
          if (move) {
            const float top = row_max(0), to_b = top == -INFINITY ? 0.f : fmaf(-top, c, -kShiftLog2);
            if (!empty) f = ex2_approx(to_b - b);
            b = to_b;
          }
          l *= f;
#pragma unroll 1
          for (int d = 0; d < DP; d += 32) {
            uint32_t o[32];
            tmem_ld_32x32b_x32(to + d, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st_32x32b_x32(to + d, o);
          }
        }
        ready(&sh.phalf[x]);
        const float s1 = half(2);
        ready(&sh.pfull[x]);
        l += s0 + s1;
      }
      if (!ok || !wait_bar_warp(&sh.ofull[x], no & 1, ctx)) break;
      ++no;
      tc_fence_after();
      const uint4 found = *reinterpret_cast<const uint4*>(sh.any[it & 1]);
      const bool any = found.x | found.y | (x ? found.z | found.w : 0);
      const int r = u.q0 + x * kTile + row;  // row within the sequence
      const int first = u.q0 + x * kTile + (warp & 3) * 32;  // the warp's first
      store_rows(smem + C::kStage + warp * 4096, to, rcp_approx(l),
                 p.out + ((int64_t)(u.start + first) * p.q_heads + u.head) * p.head_dim,
                 (int64_t)p.q_heads * p.head_dim, u.len - first, p.head_dim);
      if (any) {  // add back the non-finite values each row sees
        __syncwarp();
#pragma unroll 1
        for (int i = 0; i < kTile * (x + 1) && u.q0 + i <= r && r < u.len; ++i) {
          const int f = i / kTile, w = (i / 32) & 3;
          if (((sh.flags[it & 1][f][0][w] | sh.flags[it & 1][f][1][w]) >> (i & 31)) & 1)
            add_nonfinite(p.out + ((int64_t)(u.start + r) * p.q_heads + u.head) * p.head_dim,
                          p.v + (int64_t)(u.start + u.q0 + i) * p.v_row + (u.head / p.group) * p.v_head,
                          p.head_dim, 1.f);
        }
        __syncwarp();
      }
      tc_fence_before();  // O is read before the next unit's first product into it
      if (r < u.len)
        p.lse[(int64_t)u.head * p.tokens + u.start + r] = (lg2_approx(l * 0x1p32f) - (b + kShiftLog2)) * kLn2;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.uempty[it & 1]);
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t tm = __shfl_sync(~0u, tmem, 0), el = elect_one();
    const uint32_t q0 = smem_u32(smem);
    uint32_t base = 0;  // the unit's first stage
    uint32_t np[2] = {0, 0}, nq = 0, nclean = 0;  // bit 2 parity + tile of nclean: next phase
    bool ok = true;
    auto k_tile = [&](uint32_t t) { return smem_u32(ring) + (t % C::kStages) * 2 * C::kTileBytes; };
    auto v_tile = [&](uint32_t t) { return k_tile(t) + C::kTileBytes; };
    auto wait_stage = [&](uint32_t t) {
      return ok = ok && wait_bar_warp(&sh.full[t % C::kStages], (t / C::kStages) & 1, ctx);
    };
    for (uint32_t it = 0; ok; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = uniform(sh.unit[it & 1]);
      if (u.head < 0) break;
      if (u.len > 0) {
        int n0, n1;
        unit_tiles(u, n0, n1);
        const int last = max(n0, n1) - 1;  // step j takes V_j and K_j-1 from stage base + last - j + 1
        if (!wait_bar_warp(&sh.qfull, nq & 1, ctx)) break;
        ++nq;
        if (!wait_stage(base)) break;
        const int x = n1 ? 1 : 0;
        mma_tiles<DP>(el, tm + x * kTile, q0 + x * C::kTileBytes, k_tile(base));
        mma_commit_if(el, &sh.sfull[x]);
        mma_commit_if(el, &sh.empty[base % C::kStages]);
        if (last == 0) mma_commit_if(el, &sh.qempty);
        if (n1) {  // tile 0 starts one key tile lower
          if (!wait_stage(base + 1)) break;
          mma_tiles<DP>(el, tm, q0, k_tile(base + 1));
          mma_commit_if(el, &sh.sfull[0]);
        }
        for (int j = last; j >= 0 && ok; --j) {
          const uint32_t t = base + last - j + 1;
          if (!wait_stage(t)) break;
          if (j >= n0 - 1) {
            const uint32_t f = j - (n0 - 1), bit = 2 * (it & 1) + f;
            if (!(ok = wait_bar_warp(&sh.clean[it & 1][f], (nclean >> bit) & 1, ctx))) break;
            nclean ^= 1u << bit;
          }
#pragma unroll
          for (int x = 1; x >= 0; --x) {
            const int n = x ? n1 : n0;
            if (j >= n) continue;
            // the product with the first half of P runs while the second is made
            if (!(ok = wait_bar_warp(&sh.phalf[x], np[x] & 1, ctx))) break;
            tc_fence_after();
            mma_tmem_tile<DP, 0, 1>(el, tm + 2 * kTile + x * DP, tm + x * kTile, 32, v_tile(t), j < n - 1);
            if (!(ok = wait_bar_warp(&sh.pfull[x], np[x] & 1, ctx))) break;
            ++np[x];
            tc_fence_after();
            mma_tmem_tile<DP, 1, 2>(el, tm + 2 * kTile + x * DP, tm + x * kTile, 32, v_tile(t), true);
            if (j > 0) {
              mma_tiles<DP>(el, tm + x * kTile, q0 + x * C::kTileBytes, k_tile(t));
              mma_commit_if(el, &sh.sfull[x]);
            } else {
              mma_commit_if(el, &sh.ofull[x]);
            }
            if (x == 0 || j >= n0) mma_commit_if(el, &sh.empty[t % C::kStages]);
            // the last product that reads Q is issued
            if (j == 1 && (x == 0 || n0 == 1)) mma_commit_if(el, &sh.qempty);
          }
        }
        if (!ok) break;
        base += last + 2;
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
    }
    UnitWalk<kFwdRows> walk;
    walk.init(p);
    const int64_t total = (int64_t)walk.total() * p.q_heads;
    uint32_t t = 0, nq = 0;
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
          int n0, n1;
          unit_tiles(u, n0, n1);
          const int last = max(n0, n1) - 1, kvh = u.head / p.group;
          if ((ok = wait_bar(&sh.qempty, (nq & 1) ^ 1, ctx))) {
            mbar_arrive_expect_tx(&sh.qfull, (n1 ? 2 : 1) * C::kTileBytes);
            for (int x = 0; x <= (n1 ? 1 : 0); ++x)
              for (int b = 0; b < C::kBoxes; ++b)
                tma_load_3d(smem + x * C::kTileBytes + b * kBoxBytes, &tq, &sh.qfull, b * 64, u.head,
                            u.start + u.q0 + x * kTile);
            ++nq;
          }
          for (int j = last; j >= -1 && ok; --j, ++t) {  // K_j and V_j+1
            const int st = t % C::kStages;
            uint8_t* at = ring + st * 2 * C::kTileBytes;
            if (!(ok = wait_bar(&sh.empty[st], ((t / C::kStages) & 1) ^ 1, ctx))) break;
            mbar_arrive_expect_tx(&sh.full[st], (j == last || j < 0 ? 1 : 2) * C::kTileBytes);
            for (int b = 0; b < C::kBoxes; ++b) {
              if (j < last)
                tma_load_3d(at + C::kTileBytes + b * kBoxBytes, &tv, &sh.full[st], b * 64, kvh,
                            u.start + (j + 1) * kTile);
              if (j >= 0)
                tma_load_3d(at + b * kBoxBytes, &tk, &sh.full[st], b * 64, kvh, u.start + j * kTile);
            }
          }
        }
      }
      ok = __shfl_sync(~0u, ok, 0);
      if (u.head < 0) break;
    }
    if (!ok && lane == 0) {
      // copies in flight must land before the CTA's shared memory is given up
      if (nq) mbar_wait_drain(&sh.qfull, (nq - 1) & 1, p.timeout_ns);
      for (uint32_t i = t > C::kStages ? t - C::kStages : 0; i < t; ++i)
        mbar_wait_drain(&sh.full[i % C::kStages], (i / C::kStages) & 1, p.timeout_ns);
    }
  } else {
    // ------------------------------------------------------------ diagonal value tiles
    const int w = warp - 10;
    uint32_t t = 0;
    for (uint32_t it = 0;; ++it) {
      if (!wait_bar_warp(&sh.ufull[it & 1], (it >> 1) & 1, ctx)) break;
      const AttnUnit u = sh.unit[it & 1];
      if (u.head < 0) break;
      bool ok = true;
      if (u.len > 0) {
        int n0, n1;
        unit_tiles(u, n0, n1);
        const int last = max(n0, n1) - 1;
        for (int j = last + 1; j >= 0; --j, ++t) {  // the stage of V_j, if there is one
          const int f = j <= last ? j - (n0 - 1) : -1;
          if (!(ok = wait_bar_warp(&sh.full[t % C::kStages], (t / C::kStages) & 1, ctx))) break;
          if (f >= 0) {
            clean_tile(ring + (t % C::kStages * 2 + 1) * C::kTileBytes, C::kBoxes, u.len - j * kTile, w, 2,
                       sh.flags[it & 1][f][w]);
            fence_proxy_async_shared();
          }
          __syncwarp();
          if (lane == 0) {
            if (f >= 0) {
              const uint32_t* fl = sh.flags[it & 1][f][w];
              sh.any[it & 1][2 * f + w] = fl[0] | fl[1] | fl[2] | fl[3];
              mbar_arrive(&sh.clean[it & 1][f]);
            }
            mbar_arrive(&sh.empty[t % C::kStages]);
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

}  // namespace flce
