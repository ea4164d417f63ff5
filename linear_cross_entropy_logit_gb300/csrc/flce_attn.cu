// C ABI of causal attention over packed sequences: argument checks, the
// workspace plan and the launches.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdio>
#include <mutex>

#include "attn_bwd.cuh"
#include "attn_fwd.cuh"
#include "host_util.h"

using namespace flce;
using host::aligned;

namespace {

bool shape_ok(const flce_attention_desc* d) {
  if (!d || d->struct_size != sizeof(flce_attention_desc)) return false;
  if (d->tokens < 0 || d->tokens > (int64_t)INT_MAX - 1024) return false;
  if (d->sequences < 0 || d->sequences > (int64_t)INT_MAX - 1024) return false;
  if (d->kv_heads <= 0 || d->q_heads <= 0 || d->q_heads % d->kv_heads) return false;
  if (d->q_heads > 65535) return false;
  if (d->head_dim <= 0 || d->head_dim % 8 || d->head_dim > 128) return false;
  return true;
}

bool stride_ok(int64_t row, int64_t head, int64_t head_dim) {
  return row % 8 == 0 && head % 8 == 0 && row > 0 && head >= head_dim && row < (1ll << 38) &&
         head < (1ll << 38);
}

flce_status check(const flce_attention_desc* d, const void* const* ptrs, int n, const void* cu,
                  const float* lse, const int32_t* err_word) {
  if (!shape_ok(d)) return FLCE_ERR_ARG;
  if (d->dtype != FLCE_BF16) return d->dtype == FLCE_FP32 ? FLCE_ERR_UNSUPPORTED : FLCE_ERR_ARG;
  if (!(std::isfinite(d->scale) && d->scale > 0.f)) return FLCE_ERR_ARG;
  if (!stride_ok(d->q_row, d->q_head, d->head_dim) ||
      !stride_ok(d->k_row, d->k_head, d->head_dim) ||
      !stride_ok(d->v_row, d->v_head, d->head_dim))
    return FLCE_ERR_ARG;
  if (!err_word || !aligned(err_word, 4) || !cu || !aligned(cu, 4)) return FLCE_ERR_ARG;
  if (d->tokens == 0) return FLCE_OK;
  if (!lse || !aligned(lse, 4)) return FLCE_ERR_ARG;
  for (int i = 0; i < n; ++i)
    if (!ptrs[i] || !aligned(ptrs[i], 16)) return FLCE_ERR_ARG;
  return FLCE_OK;
}

void fill(AttnParams& p, const flce_attention_desc* d, const int32_t* cu, int32_t* err_word) {
  p.cu = cu;
  p.n_seqs = (int)d->sequences;
  p.tokens = (int)d->tokens;
  p.q_heads = (int)d->q_heads;
  p.kv_heads = (int)d->kv_heads;
  p.group = p.q_heads / p.kv_heads;
  p.head_dim = (int)d->head_dim;
  p.scale = d->scale;
  p.k_row = d->k_row;
  p.k_head = d->k_head;
  p.v_row = d->v_row;
  p.v_head = d->v_head;
  p.err_word = err_word;
  p.timeout_ns = host::kTimeoutNs;
}

// Work units of `rows` rows at most: every sequence's last and the gaps before
// and after the sequences may be partial.
int64_t most_units(const flce_attention_desc* d, int rows) {
  return d->tokens / rows + d->sequences + 2;
}

// 3-D map (head value, head, token) with boxes of 64 values x 1 head x 128
// tokens, 128-byte swizzle; values and tokens outside read as zero.
flce_status map_heads(CUtensorMap* m, const void* base, const flce_attention_desc* d,
                      int64_t heads, int64_t row, int64_t head) {
  auto fn = host::encode_fn();
  if (!fn) return host::fail_text("cuTensorMapEncodeTiled entry point unavailable");
  cuuint64_t dims[3] = {(cuuint64_t)d->head_dim, (cuuint64_t)heads, (cuuint64_t)d->tokens};
  cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)row * 2};
  cuuint32_t box[3] = {64, 1, kTile};
  cuuint32_t es[3] = {1, 1, 1};
  CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
                  box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r == CUDA_SUCCESS) return FLCE_OK;
  char buf[160];
  snprintf(buf, sizeof buf, "cuTensorMapEncodeTiled failed (%d): heads=%lld strides %lld, %lld",
           (int)r, (long long)heads, (long long)row, (long long)head);
  return host::fail_text(buf);
}

// A kernel's shared-memory limit, set once per device.
struct Setup {
  std::once_flag once;
  cudaError_t err = cudaSuccess;
};
template <typename Kern>
flce_status set_smem(Setup& s, Kern kern, int smem) {
  std::call_once(s.once, [&] {
    s.err = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  return s.err == cudaSuccess ? FLCE_OK : host::fail(s.err, "cudaFuncSetAttribute");
}

// CTAs that share the query heads of one key / value head in attn_dkdv, each
// summing its own (a divisor of their number): the fewest that give every SM a unit, counted
// as if the tokens filled whole tiles (short sequences have more units than that).
// Without (backward, us): 8192 tokens, 8 / 1 heads of 128 792, with 329; 2048 tokens,
// 32 / 8 heads 152, with 123.  More splits cost the partial sums' traffic: 2 units a
// SM 135, 8192 tokens, 32 / 8 heads 1170 unsplit and 1297 fully split.
int choose_splits(const flce_attention_desc* d, int sms) {
  const int group = (int)(d->q_heads / d->kv_heads);
  const int64_t units = std::max<int64_t>(1, d->tokens / kTile) * d->kv_heads;
  for (int s = 1; s < group; ++s)
    if (group % s == 0 && units * s >= sms) return s;
  return group;
}

struct BwdPlan {
  int splits;
  size_t off_delta, off_partial, total;
};
BwdPlan plan_backward(const flce_attention_desc* d, int sms) {
  BwdPlan b;
  const size_t rows = host::align_up((size_t)d->tokens * d->q_heads * sizeof(float));
  b.splits = choose_splits(d, sms);
  b.off_delta = rows;
  b.off_partial = 2 * rows;
  b.total = b.off_partial;
  if (b.splits > 1)
    b.total += host::align_up((size_t)2 * b.splits * d->tokens * d->kv_heads * d->head_dim * 4);
  b.total = std::max(b.total, host::kAlign);
  return b;
}

// SMs of the current device (152 when there is none to ask).
int device_sms() {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) == cudaSuccess &&
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess)
    return sms;
  (void)cudaGetLastError();
  return 152;
}

template <int DP>
flce_status launch_backward(const flce_attention_desc* d, const CUtensorMap (&m)[4],
                            const AttnBwdParams& p, int dev, int sms, cudaStream_t st) {
  static Setup setup[2][host::kMaxDevices];
  FLCE_HOST_TRY(set_smem(setup[0][dev], attn_dq<DP>, DqCfg<DP>::kSmem));
  FLCE_HOST_TRY(set_smem(setup[1][dev], attn_dkdv<DP>, DkvCfg<DP>::kSmem));
  const int64_t units = most_units(d, kTile);
  FLCE_HOST_TRY(host::launch(
      attn_delta<DP>, dim3((unsigned)(host::ceil_div(d->tokens, kDeltaRows) * d->q_heads)),
      DP == 128 ? 256 : 128, 0, st, p));
  FLCE_HOST_TRY(host::launch(attn_dq<DP>, dim3((unsigned)std::min<int64_t>(units * d->q_heads, sms)),
                             kBwdThreads, DqCfg<DP>::kSmem, st, m[0], m[1], m[2], m[3], p));
  return host::launch(attn_dkdv<DP>, dim3((unsigned)std::min<int64_t>(units * d->kv_heads * p.splits, sms)),
                      kBwdThreads, DkvCfg<DP>::kSmem, st, m[0], m[1], m[2], m[3], p);
}

}  // namespace

extern "C" {

size_t flce_attention_workspace_size(const flce_attention_desc* d) {
  if (!shape_ok(d) || d->dtype != FLCE_BF16) return 0;
  return plan_backward(d, device_sms()).total;
}

flce_status flce_attention_forward(const flce_attention_desc* d, const void* q, const void* k,
                                   const void* v, const int32_t* cu_seqlens, void* out,
                                   float* lse, int32_t* err_word, void* stream) {
  host::reset_launches();
  const void* ptrs[] = {q, k, v, out};
  FLCE_HOST_TRY(check(d, ptrs, 4, cu_seqlens, lse, err_word));
  if (d->tokens == 0) return FLCE_OK;
  int dev, sms;
  FLCE_HOST_TRY(host::device(&dev, &sms));
  AttnParams p{};
  fill(p, d, cu_seqlens, err_word);
  p.out = static_cast<bf16*>(out);
  p.lse = lse;
  p.v = static_cast<const bf16*>(v);
  CUtensorMap tq, tk, tv;
  FLCE_HOST_TRY(map_heads(&tq, q, d, d->q_heads, d->q_row, d->q_head));
  FLCE_HOST_TRY(map_heads(&tk, k, d, d->kv_heads, d->k_row, d->k_head));
  FLCE_HOST_TRY(map_heads(&tv, v, d, d->kv_heads, d->v_row, d->v_head));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int grid = (int)std::min<int64_t>(most_units(d, kFwdRows) * d->q_heads, sms);
  static Setup setup[2][host::kMaxDevices];
  if (d->head_dim <= 64) {
    FLCE_HOST_TRY(set_smem(setup[0][dev], attn_fwd<64>, FwdCfg<64>::kSmem));
    return host::launch(attn_fwd<64>, grid, kFwdThreads, FwdCfg<64>::kSmem, st, tq, tk, tv, p);
  } else {
    FLCE_HOST_TRY(set_smem(setup[1][dev], attn_fwd<128>, FwdCfg<128>::kSmem));
    return host::launch(attn_fwd<128>, grid, kFwdThreads, FwdCfg<128>::kSmem, st, tq, tk, tv, p);
  }
}

flce_status flce_attention_backward(const flce_attention_desc* d, const void* dout, const void* q,
                                    const void* k, const void* v, const void* out,
                                    const float* lse, const int32_t* cu_seqlens, void* dq,
                                    void* dk, void* dv, void* workspace, size_t ws_bytes,
                                    int32_t* err_word, void* stream) {
  host::reset_launches();
  const void* ptrs[] = {dout, q, k, v, out, dq, dk, dv};
  FLCE_HOST_TRY(check(d, ptrs, 8, cu_seqlens, lse, err_word));
  if (!workspace || !aligned(workspace, host::kAlign) ||
      ws_bytes < flce_attention_workspace_size(d))
    return FLCE_ERR_WORKSPACE;
  if (d->tokens == 0) return FLCE_OK;
  int dev, sms;
  FLCE_HOST_TRY(host::device(&dev, &sms));
  const BwdPlan plan = plan_backward(d, sms);
  char* ws = static_cast<char*>(workspace);
  AttnBwdParams p{};
  fill(p, d, cu_seqlens, err_word);
  p.out = const_cast<bf16*>(static_cast<const bf16*>(out));
  p.lse = const_cast<float*>(lse);
  p.dout = static_cast<const bf16*>(dout);
  p.k = static_cast<const bf16*>(k);
  p.dq = static_cast<bf16*>(dq);
  p.dk = static_cast<bf16*>(dk);
  p.dv = static_cast<bf16*>(dv);
  p.nlse = reinterpret_cast<float*>(ws);
  p.delta = reinterpret_cast<float*>(ws + plan.off_delta);
  p.partial = reinterpret_cast<float*>(ws + plan.off_partial);
  p.splits = plan.splits;
  CUtensorMap m[4];
  FLCE_HOST_TRY(map_heads(&m[0], q, d, d->q_heads, d->q_row, d->q_head));
  FLCE_HOST_TRY(map_heads(&m[1], k, d, d->kv_heads, d->k_row, d->k_head));
  FLCE_HOST_TRY(map_heads(&m[2], v, d, d->kv_heads, d->v_row, d->v_head));
  FLCE_HOST_TRY(map_heads(&m[3], dout, d, d->q_heads, d->q_heads * d->head_dim, d->head_dim));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  FLCE_HOST_TRY(d->head_dim <= 64 ? launch_backward<64>(d, m, p, dev, sms, st)
                                  : launch_backward<128>(d, m, p, dev, sms, st));
  if (p.splits > 1) {
    const int64_t values = d->tokens * d->kv_heads * d->head_dim;
    return host::launch(attn_sum_splits, dim3((unsigned)host::ceil_div(values, 1024), 2), 256, 0, st, p);
  }
  return FLCE_OK;
}

}  // extern "C"
