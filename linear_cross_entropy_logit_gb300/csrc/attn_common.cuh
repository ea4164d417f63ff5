// Shared by the packed attention kernels: the call's parameters and the map
// from rows to packed sequences.
#pragma once
#include <cstdint>
#include "ptx.cuh"

namespace flce {

struct AttnParams {
  const int32_t* cu;   // n_seqs + 1 offsets of the packed sequences
  int n_seqs;
  int tokens;
  int q_heads, kv_heads, group;  // group = q_heads / kv_heads
  int head_dim;
  float scale;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head;  // strides in elements
  int* err_word;
  unsigned long long timeout_ns;
};

}  // namespace flce
