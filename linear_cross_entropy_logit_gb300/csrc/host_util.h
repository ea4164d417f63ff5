// Host-side helpers shared by the library's translation units; defined in
// flce_api.cu.
#pragma once
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstddef>
#include <cstdint>

#include "flce.h"

namespace flce {
namespace host {

constexpr int kMaxDevices = 64;
constexpr size_t kAlign = 256;                           // workspace regions
constexpr unsigned long long kTimeoutNs = 2000000000ull;  // bounded device waits

// Current device, with its context on this thread, and its SM count;
// FLCE_ERR_UNSUPPORTED off sm_103.
flce_status device(int* dev, int* sms);
// Keeps the error's text for flce_last_cuda_error and returns FLCE_ERR_CUDA.
flce_status fail(cudaError_t e, const char* what);
flce_status fail_text(const char* what);
PFN_cuTensorMapEncodeTiled_v12000 encode_fn();
// flce_last_launch_count of the calling thread.
void reset_launches();
void count_launch();

inline bool aligned(const void* p, size_t a) {
  return (reinterpret_cast<uintptr_t>(p) % a) == 0;
}
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Launches a kernel that calls grid_wait: its launch and set-up overlap the end of the
// kernel ahead of it in the stream (head norm and its backward over 16384 tokens, 28 / 4
// heads of 128: 125 -> 116.5 us; attention backward of 61 ragged sequences of 9999 tokens,
// 16 heads of 64: 131 -> 123.5).  It may start as blocks of that one end, not before:
// with launch_dependents at the kernels' start the attention passes are up to 7% slower.
template <typename... P, typename... A>
flce_status launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st,
                   const A&... args) {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &a;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, kernel, args...);
  count_launch();
  if (e == cudaSuccess) return FLCE_OK;
  (void)cudaGetLastError();
  return fail(e, "cudaLaunchKernelEx");
}

}  // namespace host
}  // namespace flce

#define FLCE_HOST_TRY(expr)              \
  do {                                   \
    flce_status s_ = (expr);             \
    if (s_ != FLCE_OK) return s_;        \
  } while (0)
