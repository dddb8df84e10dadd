// Eviction from a paged cache by accumulated attention weight (sm_103a).
//
// Sequence s of L tokens, kv head g, is cut to n = min(L, budget) tokens: its
// first `sinks`, its last `recent`, and of those between the budget - sinks -
// recent with the largest scores (equal scores: the lower position; NaN below
// every number). The kept rows of K, V and the scores move to positions
// 0 .. n - 1 in their order.
//
// Two launches: evict_select_kernel, one CTA per (sequence, kv head), finds the
// kept positions and moves the scores; evict_move_kernel moves the rows.
#include "evict.h"

#include "common.cuh"

namespace pkv {

namespace {

constexpr int kSelThreads = 512;
constexpr int kSelPer = 4;  // scores per thread of an ordered pass
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;  // vectors per thread in flight

__device__ __forceinline__ int evict_len(const EvictParams& p, int s) {
  int L = p.context_lens[s];
  if (L < 0 || L > p.cap) {
    if (threadIdx.x == 0) set_err(p.dev_err, PKV_DEV_ERR_CONTEXT_LEN);
    L = L < 0 ? 0 : p.cap;
  }
  return L;
}

// Order-preserving map of a binary32 to uint32: NaN 0, then -inf .. +inf, with
// -0 and +0 alike.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

// Exclusive sum over the block of one value per thread; total gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* scratch, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFullMask, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // scratch free again
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kSelThreads / 32; ++i) {
    const uint32_t t = scratch[i];
    if (i < warp) before += t;
    total += t;
  }
  return before + x - v;
}

// The k-th largest key by radix selection, 11 + 11 + 10 bits, then one ordered
// pass over the positions: with G keys above the k-th and r = k - G of those
// equal to it wanted, a kept position's place is (kept above before it) +
// min(equal before it, r).
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[2048];
  __shared__ uint32_t scratch[kSelThreads / 32];
  __shared__ uint32_t sh_bin, sh_left;
  const int g = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
  const int L = evict_len(p, s);
  const size_t rowi = (size_t)s * p.num_kv_heads + g;
  const float* row = p.scores + rowi * p.score_stride;
  float* out = p.scores_out + rowi * p.out_stride;
  int32_t* kept = p.kept + rowi * p.budget;

  if (L <= p.budget) {
    for (int t = tid; t < L; t += kSelThreads) {
      kept[t] = t;
      if (out != row) out[t] = row[t];
    }
    return;
  }
  const int lo = p.sinks, hi = L - p.recent;
  uint32_t left = (uint32_t)(p.budget - p.sinks - p.recent);  // still to choose, of `prefix`'s keys
  uint32_t prefix = 0xffffffffu;                              // no key is above or equal to it
  if (left > 0) {
    prefix = 0;
    uint32_t mask = 0;
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < 2048; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int t = lo + tid; t < hi; t += kSelThreads) {
        const uint32_t k = score_key(row[t]);
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & digit], 1u);
      }
      __syncthreads();
      // thread i owns bins 2047 - 4 i .. 2044 - 4 i: from the largest down
      uint32_t c[4], sum = 0, total;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        c[j] = hist[2047 - 4 * tid - j];
        sum += c[j];
      }
      uint32_t above = block_scan(sum, scratch, total);
      if (above < left && left <= above + sum) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (above < left && left <= above + c[j]) {
            sh_bin = 2047u - 4u * tid - j;
            sh_left = left - above;
          }
          above += c[j];
        }
      }
      __syncthreads();
      prefix |= sh_bin << shift;
      mask |= digit << shift;
      left = sh_left;
      __syncthreads();
    }
  }

  uint32_t base_g = 0, base_e = 0;
  for (int64_t c0 = 0; c0 < L; c0 += kSelThreads * kSelPer) {
    float v[kSelPer];
    uint32_t above[kSelPer], equal[kSelPer], cnt = 0;
    const int64_t t0 = c0 + tid * kSelPer;
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) {
      const int64_t t = t0 + j;
      above[j] = equal[j] = 0;
      if (t < L) {
        v[j] = row[t];
        const bool mid = t >= lo && t < hi;
        const uint32_t k = score_key(v[j]);
        above[j] = !mid || k > prefix;
        equal[j] = mid && k == prefix;
        cnt += above[j] + (equal[j] << 16);
      }
    }
    uint32_t total;
    const uint32_t before = block_scan(cnt, scratch, total);  // every score of the chunk has been read
    uint32_t ng = base_g + (before & 0xffffu), ne = base_e + (before >> 16);
#pragma unroll
    for (int j = 0; j < kSelPer; ++j) {
      if (above[j] || (equal[j] && ne < left)) {
        const uint32_t at = ng + min(ne, left);
        kept[at] = (int)(t0 + j);
        out[at] = v[j];
      }
      ng += above[j];
      ne += equal[j];
    }
    base_g += total & 0xffffu;
    base_e += total >> 16;
  }
}

// grid = (K or V and column slice, kv head, sequence). A CTA moves its columns
// of the kept rows in ascending order, a chunk at a time: a row's new place is
// never behind its old one, so a chunk's stores, made once its loads and all
// earlier ones are done, overwrite nothing that is still to be read, and rows
// may move within the blocks they lie in.
template <typename V>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int slices) {
  const int g = blockIdx.y, s = blockIdx.z;
  const int slice = blockIdx.x >> 1;
  char* pool = static_cast<char*>((blockIdx.x & 1) ? p.v_cache : p.k_cache);
  const int n = min(evict_len(p, s), p.budget);
  const int vecs = p.row_bytes / (int)sizeof(V) / slices;  // of a row in this slice
  const int32_t* kept = p.kept + ((size_t)s * p.num_kv_heads + g) * p.budget;
  const int32_t* src_row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
  const int32_t* dst_row = p.dst_block_tables + (size_t)s * p.max_blocks_per_seq;
  const int64_t items = (int64_t)n * vecs;
  for (int64_t c0 = 0; c0 < items; c0 += kMoveThreads * kMoveUnroll) {
    V v[kMoveUnroll];
    char* to[kMoveUnroll];
#pragma unroll
    for (int j = 0; j < kMoveUnroll; ++j) {
      const int64_t i = c0 + j * kMoveThreads + threadIdx.x;
      to[j] = nullptr;
      if (i < items) {
        const int r = (int)(i / vecs);
        const int col = (int)(i - (int64_t)r * vecs) + slice * vecs;
        const int t = kept[r];
        const int a = src_row[t / p.block_size], b = dst_row[r / p.block_size];
        if (a < 0 || a >= p.num_blocks || b < 0 || b >= p.num_blocks) {
          set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
        } else {
          char* from = pool + (((size_t)a * p.num_kv_heads + g) * p.block_size + t % p.block_size) * p.row_bytes +
                       col * sizeof(V);
          char* dst = pool + (((size_t)b * p.num_kv_heads + g) * p.block_size + r % p.block_size) * p.row_bytes +
                      col * sizeof(V);
          if (from != dst) {
            v[j] = *reinterpret_cast<const V*>(from);
            to[j] = dst;
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kMoveUnroll; ++j)
      if (to[j] != nullptr) *reinterpret_cast<V*>(to[j]) = v[j];
  }
  if (blockIdx.x == 0 && g == 0 && threadIdx.x == 0) p.new_context_lens[s] = n;
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  evict_select_kernel<<<dim3(p.num_kv_heads, p.num_seqs), kSelThreads, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // few (sequence, head) pairs: the columns of a row are cut into slices of at
  // least 64 bytes
  int slices = 1;
  const int64_t ctas = (int64_t)p.num_seqs * p.num_kv_heads * 2;
  while (ctas * slices < 304 && p.row_bytes % (slices * 2) == 0 && p.row_bytes / (slices * 2) >= 64) slices *= 2;
  const dim3 grid(2 * slices, p.num_kv_heads, p.num_seqs);
  if (p.row_bytes % 16 == 0)
    evict_move_kernel<uint4><<<grid, kMoveThreads, 0, stream>>>(p, slices);
  else if (p.row_bytes % 8 == 0)
    evict_move_kernel<uint2><<<grid, kMoveThreads, 0, stream>>>(p, slices);
  else
    evict_move_kernel<uint32_t><<<grid, kMoveThreads, 0, stream>>>(p, slices);
  return cudaGetLastError();
}

}  // namespace pkv
