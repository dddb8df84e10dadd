// Host launcher of the cache eviction kernels (arguments already validated).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace pkv {

struct EvictParams {
  void* k_cache;
  void* v_cache;
  const float* scores;  // [num_seqs][num_kv_heads][score_stride]
  float* scores_out;    // [num_seqs][num_kv_heads][out_stride]
  int64_t score_stride, out_stride;
  const int32_t* block_tables;      // [num_seqs][max_blocks_per_seq]
  const int32_t* dst_block_tables;  // likewise
  const int32_t* context_lens;
  int32_t* new_context_lens;
  int32_t* kept;  // [num_seqs][num_kv_heads][budget]
  int budget, sinks, recent;
  int num_seqs, num_kv_heads, block_size, max_blocks_per_seq, num_blocks;
  int cap;        // upper bound of a context length
  int row_bytes;  // of a cache row
  int32_t* dev_err;
};

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream);

}  // namespace pkv
