// C ABI of the bounded-cache operators (sliding window with first tokens,
// score-accumulating decode, eviction): argument checks, launch-shape choice
// and dispatch. Owns no memory, keeps no state, never synchronises.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "decode_window.cuh"
#include "evict.h"
#include "pkv.h"
#include "prefill_window.cuh"

namespace {

// Pieces of a segment: long enough that its start and join do not count, many
// enough that the last wave of CTAs is a small part of all (kWaveCtas: CTAs that
// are resident at a time). 64 sequences, window 4096 / 8 sequences of up to 32768
// with scores: 171 / 141 us with 4 waves, 2 more or 1 less with 3, 4 and 2 more with 5, 11
// and 5 more with 6.
// At least kMinTiles on average: one sequence, window 1024: 7.5 us, 10.5 with 16. At most kMaxTiles,
// for the one long sequence of a batch that is sized by its length (131072 tokens beside
// 127 x 100: 227 us with 16 pieces, 1295 with the 2 that an equal share of tiles gives).
constexpr int64_t kWaveCtas = 152 * 3, kWaves = 4;
constexpr int kMinTiles = 4, kMaxTiles = 96;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool supported_shape(int head_dim, int block_size) {
  return (head_dim == 64 || head_dim == 128) && (block_size == 8 || block_size == 16 || block_size == 32);
}
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
pkv_status launch_status(cudaError_t e) {
  return e == cudaSuccess ? PKV_OK : (e == cudaErrorNotSupported ? PKV_ERR_UNSUPPORTED : PKV_ERR_CUDA);
}

// Query heads of a kv head that one CTA takes, and how many such parts there are.
struct HeadParts {
  int parts, heads;
};
HeadParts head_parts(int group, bool f32) {
  const int most = f32 ? 4 : 8;
  HeadParts h;
  h.parts = (group + most - 1) / most;
  h.heads = (group + h.parts - 1) / h.parts;
  return h;
}

struct WindowLayout {
  size_t counter = 0, ml = 0, o = 0, row_ml = 0, logits = 0, total = 0;
  int64_t logit_stride = 0, pieces = 0;
};

// Counters of the segments, the pieces' partial results, and (scores) the
// final maximum and sum of every row and its logits. The counters' place is the same in
// every call, whatever its sizes, and nothing else is ever written there: they have to
// be zero from one call to the next, also where a call of other sizes (or of the other operator)
// lies between. A split segment has two pieces at least, so that there are never more of
// them than kWinPiecesMost / 2.
constexpr int64_t kCounterBytes = PKV_WINDOW_COUNTER_BYTES;
static_assert(kCounterBytes == pkv::kWinPiecesMost / 2 * (int64_t)sizeof(int32_t), "a counter to a split segment");
WindowLayout window_layout(int num_seqs, int num_heads, int num_kv_heads, int head_dim, bool scores,
                           int max_context_len) {
  WindowLayout w;
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_heads % num_kv_heads != 0 ||
      max_context_len < 0)
    return w;
  const size_t rows = (size_t)num_seqs * num_heads;  // at least as many as segments
  const int64_t most = std::min(std::max(pkv::kWinRowPieces * (int64_t)rows, pkv::kWinPiecesLeast), pkv::kWinPiecesMost);
  const size_t piece = sizeof(float2) + (size_t)head_dim * sizeof(float);
  size_t off = align_up(rows * sizeof(int32_t), 256) + align_up((size_t)most * sizeof(float2), 256) +
               (size_t)most * head_dim * sizeof(float);
  // what the counters leave of that (a segment of one piece has no partial results)
  w.pieces = std::min(most, std::max<int64_t>(((int64_t)off - kCounterBytes - 256) / (int64_t)piece, 0));
  w.ml = kCounterBytes;
  w.o = w.ml + align_up((size_t)w.pieces * sizeof(float2), 256);
  if (scores) {
    w.row_ml = off;
    off += align_up(rows * sizeof(float2), 256);
    w.logits = off;
    w.logit_stride = ((int64_t)max_context_len + 7) / 8 * 8;
    off += rows * (size_t)w.logit_stride * sizeof(float);
  }
  w.total = off;
  return w;
}

pkv_status check_args(const void* out, const void* q, const void* k_cache, const void* v_cache,
                      const int32_t* block_tables, const int32_t* context_lens, float scale, int num_heads,
                      int num_kv_heads, int head_dim, int block_size, int num_seqs, int max_blocks_per_seq,
                      int num_blocks, int max_context_len, pkv_dtype dtype, const int32_t* dev_err) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      max_blocks_per_seq <= 0 || num_blocks <= 0 || max_context_len < 0 || !std::isfinite(scale))
    return PKV_ERR_INVALID_ARG;
  if (num_heads % num_kv_heads != 0) return PKV_ERR_INVALID_ARG;
  if ((int64_t)max_context_len > (int64_t)max_blocks_per_seq * block_size) return PKV_ERR_INVALID_ARG;
  if ((dtype != PKV_F32 && dtype != PKV_F16 && dtype != PKV_BF16) || !supported_shape(head_dim, block_size))
    return PKV_ERR_UNSUPPORTED;
  // token positions are kept in 32 bits, with a tile to spare
  if (num_seqs > 65535 || (int64_t)max_blocks_per_seq * block_size > 0x7fff0000LL) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!out || !q || !k_cache || !v_cache || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || (dev_err && !aligned(dev_err, 4)))
    return PKV_ERR_INVALID_ARG;
  return PKV_OK;
}

// Everything of a window / score decode launch but the operands' addresses.
pkv_status launch_decode(pkv::WindowParams& p, float scale, int head_dim, pkv_dtype dtype, char* ws,
                         const WindowLayout& lay, bool scores, cudaStream_t stream) {
  const HeadParts hp = head_parts(p.group, dtype == PKV_F32);
  p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
  p.parts = hp.parts;
  p.part_heads = hp.heads;
  const int64_t segments = (int64_t)p.num_seqs * p.num_kv_heads * hp.parts;
  const int64_t seen = std::min<int64_t>(p.max_context_len, (int64_t)p.window + p.sinks);
  const int64_t tiles = (seen + 15) / 16 + 2;
  const int64_t per = std::min<int64_t>(std::max<int64_t>(segments * tiles / (kWaves * kWaveCtas), kMinTiles), kMaxTiles);
  const int64_t splits = std::min((tiles + per - 1) / per, lay.pieces / hp.heads / segments);
  p.splits = (int)std::max<int64_t>(splits, 1);
  p.min_tiles = (int)per;
  p.counter = reinterpret_cast<int32_t*>(ws + lay.counter);
  p.piece_ml = reinterpret_cast<float2*>(ws + lay.ml);
  p.piece_o = reinterpret_cast<float*>(ws + lay.o);
  if (scores) {
    p.row_ml = reinterpret_cast<float2*>(ws + lay.row_ml);
    p.logits = reinterpret_cast<float*>(ws + lay.logits);
    p.logit_stride = lay.logit_stride;
  }
  const pkv::WindowLauncher launch = dtype == PKV_F32
                                         ? pkv::window_launcher_f32(head_dim, hp.heads, scores)
                                         : pkv::window_launcher_16(dtype == PKV_BF16, head_dim, hp.heads, scores);
  if (!launch) return PKV_ERR_UNSUPPORTED;
  return launch_status(launch(p, stream));
}

pkv::WindowParams operands(void* out, const void* q, const void* k_cache, const void* v_cache,
                           const int32_t* block_tables, const int32_t* context_lens, int num_heads,
                           int num_kv_heads, int block_size, int num_seqs, int max_blocks_per_seq, int num_blocks,
                           int max_context_len, int32_t* dev_err) {
  pkv::WindowParams p{};
  p.out = out;
  p.q = q;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.block_size = block_size;
  p.block_bits = block_size == 8 ? 3 : (block_size == 16 ? 4 : 5);
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.max_context_len = max_context_len;
  p.dev_err = dev_err;
  return p;
}

bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

// Two sets of score rows that are the same rows (same address and stride) or
// share no byte.
bool same_or_apart(const float* a, int64_t stride_a, int64_t used_a, const float* b, int64_t stride_b,
                   int64_t used_b, int64_t rows) {
  if (a == b) return stride_a == stride_b;
  return !overlap(a, sizeof(float) * (size_t)((rows - 1) * stride_a + used_a), b,
                  sizeof(float) * (size_t)((rows - 1) * stride_b + used_b));
}

}  // namespace

extern "C" {

size_t pkv_decode_window_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim) {
  return window_layout(num_seqs, num_heads, num_kv_heads, head_dim, false, 0).total;
}

size_t pkv_decode_scores_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                         int max_context_len) {
  return window_layout(num_seqs, num_heads, num_kv_heads, head_dim, true, max_context_len).total;
}

pkv_status pkv_paged_attention_decode_window(void* out, const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, const int32_t* context_lens, float scale,
                                             int window, int num_sinks, int num_heads, int num_kv_heads,
                                             int head_dim, int block_size, int num_seqs, int max_blocks_per_seq,
                                             int num_blocks, int max_context_len, pkv_dtype dtype, void* workspace,
                                             size_t workspace_bytes, int32_t* dev_err, pkv_stream_t stream) {
  if (window < 1 || num_sinks < 0) return PKV_ERR_INVALID_ARG;
  const pkv_status st =
      check_args(out, q, k_cache, v_cache, block_tables, context_lens, scale, num_heads, num_kv_heads, head_dim,
                 block_size, num_seqs, max_blocks_per_seq, num_blocks, max_context_len, dtype, dev_err);
  if (st != PKV_OK || num_seqs == 0) return st;
  const WindowLayout lay = window_layout(num_seqs, num_heads, num_kv_heads, head_dim, false, 0);
  if (!workspace || workspace_bytes < lay.total) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return PKV_ERR_INVALID_ARG;
  pkv::WindowParams p = operands(out, q, k_cache, v_cache, block_tables, context_lens, num_heads, num_kv_heads,
                                 block_size, num_seqs, max_blocks_per_seq, num_blocks, max_context_len, dev_err);
  p.window = std::min(window, std::max(max_context_len, 1));
  p.sinks = std::min(num_sinks, max_context_len);
  return launch_decode(p, scale, head_dim, dtype, static_cast<char*>(workspace), lay, false,
                       reinterpret_cast<cudaStream_t>(stream));
}

pkv_status pkv_paged_attention_decode_scores(void* out, float* scores_out, const float* scores, int64_t score_stride,
                                             const void* q, const void* k_cache, const void* v_cache,
                                             const int32_t* block_tables, const int32_t* context_lens, float scale,
                                             int num_heads, int num_kv_heads, int head_dim, int block_size,
                                             int num_seqs, int max_blocks_per_seq, int num_blocks,
                                             int max_context_len, pkv_dtype dtype, void* workspace,
                                             size_t workspace_bytes, int32_t* dev_err, pkv_stream_t stream) {
  const pkv_status st =
      check_args(out, q, k_cache, v_cache, block_tables, context_lens, scale, num_heads, num_kv_heads, head_dim,
                 block_size, num_seqs, max_blocks_per_seq, num_blocks, max_context_len, dtype, dev_err);
  if (st != PKV_OK) return st;
  if (score_stride < max_context_len) return PKV_ERR_INVALID_ARG;
  if (num_kv_heads > 65535) return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return st;
  if (!scores_out || !aligned(scores_out, 4) || !aligned(scores, 4)) return PKV_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)num_seqs * num_kv_heads;
  if (scores && !same_or_apart(scores, score_stride, max_context_len, scores_out, score_stride, max_context_len, rows))
    return PKV_ERR_INVALID_ARG;
  const WindowLayout lay = window_layout(num_seqs, num_heads, num_kv_heads, head_dim, true, max_context_len);
  if (!workspace || workspace_bytes < lay.total) return PKV_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return PKV_ERR_INVALID_ARG;
  pkv::WindowParams p = operands(out, q, k_cache, v_cache, block_tables, context_lens, num_heads, num_kv_heads,
                                 block_size, num_seqs, max_blocks_per_seq, num_blocks, max_context_len, dev_err);
  p.window = std::max(max_context_len, 1);
  p.sinks = 0;
  const pkv_status run = launch_decode(p, scale, head_dim, dtype, static_cast<char*>(workspace), lay, true,
                                       reinterpret_cast<cudaStream_t>(stream));
  if (run != PKV_OK) return run;
  pkv::ScoreParams sp{};
  sp.logits = p.logits;
  sp.logit_stride = p.logit_stride;
  sp.row_ml = p.row_ml;
  sp.scores = scores;
  sp.scores_out = scores_out;
  sp.score_stride = score_stride;
  sp.context_lens = context_lens;
  sp.num_heads = num_heads;
  sp.num_kv_heads = num_kv_heads;
  sp.group = p.group;
  sp.cap = max_context_len;
  return launch_status(
      pkv::launch_add_scores(sp, num_seqs, max_context_len, reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status pkv_paged_attention_prefill_window(void* out, const void* q, const void* k_cache, const void* v_cache,
                                              const int32_t* block_tables, const int32_t* context_lens,
                                              const int32_t* query_start, float scale, int window, int num_sinks,
                                              int num_heads, int num_kv_heads, int head_dim, int block_size,
                                              int num_seqs, int max_blocks_per_seq, int num_blocks,
                                              int max_query_len, pkv_dtype dtype, int32_t* dev_err,
                                              pkv_stream_t stream) {
  if (window < 1 || num_sinks < 0 || max_query_len < 0) return PKV_ERR_INVALID_ARG;
  if (dtype == PKV_F32) return PKV_ERR_UNSUPPORTED;
  const pkv_status st =
      check_args(out, q, k_cache, v_cache, block_tables, context_lens, scale, num_heads, num_kv_heads, head_dim,
                 block_size, num_seqs, max_blocks_per_seq, num_blocks, 0, dtype, dev_err);
  if (st != PKV_OK || num_seqs == 0 || max_query_len == 0) return st;
  if (!query_start || !aligned(query_start, 4)) return PKV_ERR_INVALID_ARG;
  const pkv::PrefillWindowLauncher launch = pkv::prefill_window_launcher(dtype == PKV_BF16 ? 1 : 0, head_dim);
  if (!launch) return PKV_ERR_UNSUPPORTED;
  const int longest = max_blocks_per_seq * block_size;  // fits: checked above
  pkv::PrefillWindowParams p{};
  p.out = out;
  p.q = q;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start = query_start;
  p.scale_log2 = scale * 1.4426950408889634f;  // log2(e)
  p.window = std::min(window, longest);
  p.sinks = std::min(num_sinks, longest);
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = num_heads / num_kv_heads;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.dev_err = dev_err;
  p.wait_limit_ns = pkv_get_wait_timeout_ns();
  return launch_status(launch(p, k_cache, v_cache, max_query_len, reinterpret_cast<cudaStream_t>(stream)));
}

pkv_status pkv_evict_tokens(void* k_cache, void* v_cache, const float* scores, int64_t score_stride,
                            float* scores_out, int64_t out_stride, const int32_t* block_tables,
                            const int32_t* dst_block_tables, const int32_t* context_lens,
                            int32_t* new_context_lens, int32_t* kept, int budget, int num_sinks, int num_recent,
                            int num_kv_heads, int head_dim, int block_size, int num_seqs, int max_blocks_per_seq,
                            int num_blocks, int max_context_len, pkv_dtype dtype, int32_t* dev_err,
                            pkv_stream_t stream) {
  if (budget < 1 || num_sinks < 0 || num_recent < 0 || (int64_t)num_sinks + num_recent > budget || num_seqs < 0 ||
      num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || max_blocks_per_seq <= 0 || num_blocks <= 0 ||
      max_context_len < 0)
    return PKV_ERR_INVALID_ARG;
  if ((int64_t)max_context_len > (int64_t)max_blocks_per_seq * block_size) return PKV_ERR_INVALID_ARG;
  const int64_t most = std::min(budget, max_context_len);  // tokens kept of a sequence
  if (score_stride < max_context_len || out_stride < most) return PKV_ERR_INVALID_ARG;
  if ((dtype != PKV_F32 && dtype != PKV_F16 && dtype != PKV_BF16 && dtype != PKV_FP8_E4M3 && dtype != PKV_Q4_0) ||
      !supported_shape(head_dim, block_size))
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs > 65535 || num_kv_heads > 65535 || (int64_t)max_blocks_per_seq * block_size > 0x7fff0000LL)
    return PKV_ERR_UNSUPPORTED;
  if (num_seqs == 0) return PKV_OK;
  if (!k_cache || !v_cache || !scores || !scores_out || !block_tables || !dst_block_tables || !context_lens ||
      !new_context_lens || !kept)
    return PKV_ERR_INVALID_ARG;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(scores, 4) || !aligned(scores_out, 4) ||
      !aligned(block_tables, 4) || !aligned(dst_block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(new_context_lens, 4) || !aligned(kept, 4) || (dev_err && !aligned(dev_err, 4)))
    return PKV_ERR_INVALID_ARG;
  if (!same_or_apart(scores, score_stride, max_context_len, scores_out, out_stride, most,
                     (int64_t)num_seqs * num_kv_heads))
    return PKV_ERR_INVALID_ARG;
  pkv::EvictParams p{};
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.scores = scores;
  p.scores_out = scores_out;
  p.score_stride = score_stride;
  p.out_stride = out_stride;
  p.block_tables = block_tables;
  p.dst_block_tables = dst_block_tables;
  p.context_lens = context_lens;
  p.new_context_lens = new_context_lens;
  p.kept = kept;
  p.budget = budget;
  p.sinks = num_sinks;
  p.recent = num_recent;
  p.num_seqs = num_seqs;
  p.num_kv_heads = num_kv_heads;
  p.block_size = block_size;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.num_blocks = num_blocks;
  p.cap = max_context_len;
  p.row_bytes = dtype == PKV_Q4_0 ? head_dim / 16 * 9
                                  : head_dim * (dtype == PKV_F32 ? 4 : (dtype == PKV_FP8_E4M3 ? 1 : 2));
  p.dev_err = dev_err;
  return launch_status(pkv::launch_evict(p, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
