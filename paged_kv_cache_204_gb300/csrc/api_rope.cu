// C ABI of the rotating cache writes: argument checks and dispatch. Owns no
// memory, keeps no state, never synchronises.
#include <cmath>
#include <cstdint>
#include <cstring>

#include "pkv.h"
#include "rope_cache.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_scale(float s) { return std::isfinite(s) && s > 0.f; }

// A step's rows in bytes, one to a token, no two of which overlap; begin, end: the first byte and behind the last.
struct Rows {
  uintptr_t begin, end;
  int64_t stride, row;
  int tokens;
  Rows(const void* p, int64_t stride_, int64_t row_, int tokens_)
      : begin(reinterpret_cast<uintptr_t>(p)), end(begin + (uintptr_t)((tokens_ - 1) * stride_ + row_)), stride(stride_),
        row(row_), tokens(tokens_) {}
  bool range_meets(const Rows& o) const { return begin < o.end && o.begin < end; }
  // A row here has a byte in common with one of o's: parts of one projection lie between one another without that.
  bool meets(const Rows& o) const {
    if (!range_meets(o)) return false;
    if (stride == o.stride) {  // o's row i + d begins x + d * stride behind row i here: is that above -o.row and below row?
      const int64_t x = (int64_t)(o.begin - begin), low = -o.row - x;
      int64_t d = low >= 0 ? low / stride + 1 : -(-low / stride) + (-low % stride == 0 ? 1 : 0);  // the first above
      if (d < 1 - tokens) d = 1 - tokens;
      return d < tokens && d * stride < row - x;
    }
    for (int i = 0, j = 0; i < tokens && j < o.tokens;) {
      const uintptr_t a = begin + (uintptr_t)(i * stride), b = o.begin + (uintptr_t)(j * o.stride);
      if (a + (uintptr_t)row <= b)
        ++i;
      else if (b + (uintptr_t)o.row <= a)
        ++j;
      else
        return true;
    }
    return false;
  }
};

pkv_status rope(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                const void* v, int64_t v_stride, void* k_cache, void* v_cache, const int64_t* slot_mapping,
                const int32_t* positions, const float* cos_sin, int max_position, int rotary_dim,
                const uint8_t* pair_axis, int num_axes, int interleaved, int num_tokens, int num_heads,
                int num_kv_heads, int head_dim, int block_size, int num_blocks, pkv_dtype dtype, pkv::RopeCache cache,
                float k_scale, float v_scale, int32_t* dev_err, pkv_stream_t stream) {
  if (num_tokens < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
      max_position <= 0 || rotary_dim <= 0 || num_axes <= 0 || num_heads % num_kv_heads != 0)
    return PKV_ERR_INVALID_ARG;
  if (!valid_scale(k_scale) || !valid_scale(v_scale)) return PKV_ERR_INVALID_ARG;
  const pkv::RopeLauncher launch = pkv::rope_launcher(cache, dtype, head_dim);
  if (launch == nullptr || (block_size != 8 && block_size != 16 && block_size != 32) || num_axes > 4 ||
      num_heads > 65535 || num_kv_heads > 65535)
    return PKV_ERR_UNSUPPORTED;
  if (rotary_dim % 16 != 0 || rotary_dim > head_dim) return PKV_ERR_UNSUPPORTED;
  if (num_axes > 1 && pair_axis == nullptr) return PKV_ERR_INVALID_ARG;
  pkv::RopeParams p{};
  for (int i = 0; pair_axis != nullptr && i < rotary_dim / 2; ++i) {
    if (pair_axis[i] >= num_axes) return PKV_ERR_INVALID_ARG;
    p.pair_axis[i / 4] |= (uint32_t)pair_axis[i] << (8 * (i % 4));
  }
  if (num_tokens == 0) return PKV_OK;
  if (!q_out || !q || !k || !v || !k_cache || !v_cache || !slot_mapping || !positions || !cos_sin)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(slot_mapping, 8) || !aligned(positions, 4) || !aligned(cos_sin, 16) ||
      (dev_err && !aligned(dev_err, 4)))
    return PKV_ERR_INVALID_ARG;
  const int es = dtype == PKV_F32 ? 4 : 2, chunk = 16 / es;
  const int64_t q_row = (int64_t)num_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  if (num_tokens > 1) {
    if (q_out_stride < q_row || q_stride < q_row || k_stride < kv_row || v_stride < kv_row) return PKV_ERR_INVALID_ARG;
    if (q_out_stride % chunk || q_stride % chunk || k_stride % chunk || v_stride % chunk) return PKV_ERR_INVALID_ARG;
    const int64_t most = INT64_MAX / 16 / num_tokens;
    if (q_out_stride > most || q_stride > most || k_stride > most || v_stride > most) return PKV_ERR_INVALID_ARG;
  } else {
    q_out_stride = q_stride = q_row;
    k_stride = v_stride = kv_row;
  }
  // in place (the very rows), or no byte in common
  const bool in_place = q_out == q && q_out_stride == q_stride;
  const Rows out(q_out, q_out_stride * es, q_row * es, num_tokens);
  if (!in_place && out.range_meets(Rows(q, q_stride * es, q_row * es, num_tokens))) return PKV_ERR_INVALID_ARG;
  if (out.meets(Rows(k, k_stride * es, kv_row * es, num_tokens)) ||
      out.meets(Rows(v, v_stride * es, kv_row * es, num_tokens)))
    return PKV_ERR_INVALID_ARG;
  const int64_t cache_row = cache == pkv::RopeCache::kSame ? head_dim * es
                                                           : (cache == pkv::RopeCache::kFp8 ? head_dim : head_dim / 16 * 9);
  for (const void* pool : {k_cache, v_cache}) {
    const Rows whole(pool, 0, (int64_t)num_blocks * num_kv_heads * block_size * cache_row, 1);
    if (out.range_meets(whole)) return PKV_ERR_INVALID_ARG;
  }
  p.q_out = q_out;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_out_stride = q_out_stride / chunk;
  p.q_stride = q_stride / chunk;
  p.k_stride = k_stride / chunk;
  p.v_stride = v_stride / chunk;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_position = max_position;
  p.rotary_dim = rotary_dim;
  p.num_axes = num_axes;
  p.interleaved = interleaved != 0;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.num_slots = (int64_t)num_blocks * block_size;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.dev_err = dev_err;
  const cudaError_t e = launch(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : (e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA);
}

}  // namespace

extern "C" {

pkv_status pkv_rope_and_cache(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride, void* k_cache, void* v_cache,
                              const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
                              int max_position, int rotary_dim, const uint8_t* pair_axis, int num_axes,
                              int interleaved, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                              int block_size, int num_blocks, pkv_dtype dtype, int32_t* dev_err,
                              pkv_stream_t stream) {
  return rope(q_out, q_out_stride, q, q_stride, k, k_stride, v, v_stride, k_cache, v_cache, slot_mapping, positions,
              cos_sin, max_position, rotary_dim, pair_axis, num_axes, interleaved, num_tokens, num_heads,
              num_kv_heads, head_dim, block_size, num_blocks, dtype, pkv::RopeCache::kSame, 1.f, 1.f, dev_err,
              stream);
}

pkv_status pkv_rope_and_cache_fp8(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride, void* k_cache, void* v_cache,
                                  const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
                                  int max_position, int rotary_dim, const uint8_t* pair_axis, int num_axes,
                                  int interleaved, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                  int block_size, int num_blocks, pkv_dtype src_dtype, float k_scale, float v_scale,
                                  int32_t* dev_err, pkv_stream_t stream) {
  return rope(q_out, q_out_stride, q, q_stride, k, k_stride, v, v_stride, k_cache, v_cache, slot_mapping, positions,
              cos_sin, max_position, rotary_dim, pair_axis, num_axes, interleaved, num_tokens, num_heads,
              num_kv_heads, head_dim, block_size, num_blocks, src_dtype, pkv::RopeCache::kFp8, k_scale, v_scale,
              dev_err, stream);
}

pkv_status pkv_rope_and_cache_q4_0(void* q_out, int64_t q_out_stride, const void* q, int64_t q_stride, const void* k,
                                   int64_t k_stride, const void* v, int64_t v_stride, void* k_cache, void* v_cache,
                                   const int64_t* slot_mapping, const int32_t* positions, const float* cos_sin,
                                   int max_position, int rotary_dim, const uint8_t* pair_axis, int num_axes,
                                   int interleaved, int num_tokens, int num_heads, int num_kv_heads, int head_dim,
                                   int block_size, int num_blocks, pkv_dtype src_dtype, int32_t* dev_err,
                                   pkv_stream_t stream) {
  return rope(q_out, q_out_stride, q, q_stride, k, k_stride, v, v_stride, k_cache, v_cache, slot_mapping, positions,
              cos_sin, max_position, rotary_dim, pair_axis, num_axes, interleaved, num_tokens, num_heads,
              num_kv_heads, head_dim, block_size, num_blocks, src_dtype, pkv::RopeCache::kQ4, 1.f, 1.f, dev_err,
              stream);
}

}  // extern "C"
