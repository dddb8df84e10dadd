// Launch of prefill over quantised caches (arguments already validated).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace pkv {

struct PrefillQuantParams {
  void* out;
  const void* q;
  const void *k_cache, *v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  float scale, k_scale, v_scale;  // softmax scale; fp8 pools: what a code is multiplied by (1 for q4_0)
  int num_seqs, num_heads, num_kv_heads, group, block_size, max_blocks_per_seq, num_blocks, max_query_len;
  void* workspace;
  int32_t* dev_err;
  uint64_t wait_limit_ns;
};

size_t prefill_quant_workspace_bytes(int head_dim);
// nullptr where the combination is not built
using PrefillQuantLauncher = cudaError_t (*)(const PrefillQuantParams&, cudaStream_t);
PrefillQuantLauncher prefill_quant_launcher(bool q4, bool bf16, int head_dim);

}  // namespace pkv
