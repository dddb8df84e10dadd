// Launch of the rotating cache write (arguments already validated).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "pkv.h"

namespace pkv {

struct RopeParams {
  void* q_out;
  const void *q, *k, *v;
  int64_t q_out_stride, q_stride, k_stride, v_stride;  // from token to token, in 16-byte chunks
  void *k_cache, *v_cache;
  const int64_t* slot_mapping;
  const int32_t* positions;  // [num_axes][num_tokens]
  const float* cos_sin;      // [max_position][rotary_dim]: cosines, then sines
  int max_position, rotary_dim, num_axes, interleaved;
  uint32_t pair_axis[16];    // axis of each pair, a byte each
  int num_tokens, num_heads, num_kv_heads, block_size;
  int64_t num_slots;
  float k_scale, v_scale;    // fp8 caches
  int32_t* dev_err;
};

// What a cache row holds: the values as they are, e4m3 codes, or q4_0 blocks.
enum class RopeCache { kSame, kFp8, kQ4 };

// nullptr where the combination is not built
using RopeLauncher = cudaError_t (*)(const RopeParams&, cudaStream_t);
RopeLauncher rope_launcher(RopeCache cache, pkv_dtype dtype, int head_dim);

}  // namespace pkv
