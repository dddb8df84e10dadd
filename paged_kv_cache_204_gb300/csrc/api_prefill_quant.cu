// C ABI of prefill over quantised caches: argument checks and dispatch. Owns no
// memory, keeps no state, never synchronises.
#include <cmath>
#include <cstdint>

#include "pkv.h"
#include "prefill_quant.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool valid_scale(float s) { return std::isfinite(s) && s > 0.f; }

pkv_status prefill(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                   const int32_t* context_lens, const int32_t* query_start, float scale, float k_scale, float v_scale,
                   int num_heads, int num_kv_heads, int head_dim, int block_size, int num_seqs, int max_blocks_per_seq,
                   int num_blocks, int max_query_len, pkv_dtype dtype, bool q4, void* workspace,
                   size_t workspace_bytes, int32_t* dev_err, pkv_stream_t stream) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || num_blocks <= 0 || max_query_len < 0 || !std::isfinite(scale) ||
      !valid_scale(k_scale) || !valid_scale(v_scale) || !std::isfinite(scale * k_scale * 1.4426950408889634f))
    return PKV_ERR_INVALID_ARG;
  if (num_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  if ((dtype != PKV_F16 && dtype != PKV_BF16) || (block_size != 8 && block_size != 16 && block_size != 32))
    return PKV_ERR_UNSUPPORTED;
  const pkv::PrefillQuantLauncher launch = pkv::prefill_quant_launcher(q4, dtype == PKV_BF16, head_dim);
  // token positions are kept in 32 bits, with a tile to spare
  if (launch == nullptr || num_seqs > 65535 || (int64_t)max_blocks_per_seq * block_size > 0x7fff0000LL)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0 || max_query_len == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start) return PKV_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start, 4) ||
      (dev_err && !aligned(dev_err, 4)))
    return PKV_ERR_INVALID_ARG;
  if (!workspace || workspace_bytes < pkv::prefill_quant_workspace_bytes(head_dim)) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return PKV_ERR_INVALID_ARG;
  if (out == q) return PKV_ERR_INVALID_ARG;  // parts of a pair read its queries when others may have written outputs
  pkv::PrefillQuantParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.scale = scale;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.max_query_len = max_query_len;
  p.workspace = workspace;
  p.dev_err = dev_err;
  p.wait_limit_ns = pkv_get_wait_timeout_ns();
  const cudaError_t e = launch(p, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? PKV_OK : (e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA);
}

}  // namespace

extern "C" {

size_t pkv_prefill_workspace_bytes(int head_dim) { return pkv::prefill_quant_workspace_bytes(head_dim); }

pkv_status pkv_paged_attention_prefill_fp8(void* out, const void* q, const void* k_cache, const void* v_cache,
                                           const int32_t* block_tables, const int32_t* context_lens,
                                           const int32_t* query_start, float scale, float k_scale, float v_scale,
                                           int num_heads, int num_kv_heads, int head_dim, int block_size,
                                           int num_seqs, int max_blocks_per_seq, int num_blocks, int max_query_len,
                                           pkv_dtype dtype, void* workspace, size_t workspace_bytes,
                                           int32_t* dev_err, pkv_stream_t stream) {
  return prefill(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, k_scale, v_scale, num_heads,
                 num_kv_heads, head_dim, block_size, num_seqs, max_blocks_per_seq, num_blocks, max_query_len, dtype,
                 false, workspace, workspace_bytes, dev_err, stream);
}

pkv_status pkv_paged_attention_prefill_q4_0(void* out, const void* q, const void* k_cache, const void* v_cache,
                                            const int32_t* block_tables, const int32_t* context_lens,
                                            const int32_t* query_start, float scale, int num_heads, int num_kv_heads,
                                            int head_dim, int block_size, int num_seqs, int max_blocks_per_seq,
                                            int num_blocks, int max_query_len, pkv_dtype dtype, void* workspace,
                                            size_t workspace_bytes, int32_t* dev_err, pkv_stream_t stream) {
  return prefill(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, 1.f, 1.f, num_heads,
                 num_kv_heads, head_dim, block_size, num_seqs, max_blocks_per_seq, num_blocks, max_query_len, dtype,
                 true, workspace, workspace_bytes, dev_err, stream);
}

}  // extern "C"
