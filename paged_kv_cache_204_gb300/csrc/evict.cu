// Eviction from a paged cache by accumulated attention weight (sm_103a).
//
// Sequence s of L tokens, kv head g, is cut to n = min(L, budget) tokens: its
// first `sinks`, its last `recent`, and of those between the budget - sinks -
// recent with the largest scores (equal scores: the lower position; NaN below
// every number). The kept rows of K, V and the scores move to positions
// 0 .. n - 1 in their order.
//
// Bound by memory: every score is read once and a kept one written, a kept row read and
// written. GPU times (a call by itself takes 2 us more), with head_dim 128 in 16 bits: 64 sequences of 700 to 4000 tokens to 1001, 8 kv
// heads: 106 us, 5.0 TB/s (8-token blocks: a row's neighbours in its block are 2 KB); 8 of
// 16385 to 32768 to 8192, 32 kv heads: 390 us, 5.6 TB/s; of these the selection takes 16
// and 41 us. One sequence of 2001 tokens to 1024: 8.3 us, the latency of two dependent
// kernels.
//
// Two launches: evict_select_kernel, one CTA per (sequence, kv head), finds the
// kept positions and moves the scores; evict_move_kernel moves the rows. The
// second is a programmatic dependent of the first: it is set up while the
// first runs and waits for it.
#include "evict.h"

#include <type_traits>

#include "tc.cuh"

namespace pkv {

namespace {

constexpr int kBins = 2048;
constexpr int kListMost = 128;          // candidates that are ranked one against all
constexpr int kScoresInSmem = 32768;    // scores of a row that are kept in shared memory
constexpr int kFewScores = 8192;         // rows up to this long: kSelectFew threads, else kSelectMost
constexpr int kSelectFew = 512, kSelectMost = 1024;
constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 8;          // vectors per thread and chunk

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

// A token's rank among the candidates as one number, larger first: its score's
// key, then the lower position. No two tokens have the same.
__device__ __forceinline__ uint64_t rank_of(uint32_t key, int t) {
  return ((uint64_t)key << 32) | (uint32_t)~(uint32_t)t;
}

// Selection: the k-th largest rank. The interval that holds it is cut into 2048
// bins of equal width (a power of two), the candidates are counted into them and
// the bin that holds the k-th is the next interval; the width of the first comes
// from the smallest and the largest score, so that the counts spread over the
// bins whatever the scores' scale is (leading digits of the scores' bits put most
// scores of one magnitude into a few counters, whose atomics then queue). Once at most kListMost candidates
// are left each is compared with all others (64 to 512: no difference). The pass that lists
// them also notes what lies above, a bit per token; a warp counts the bits of its
// stretch, and the counts of the warps before it give its first place.
template <int NT>
__global__ void __launch_bounds__(NT) evict_select_kernel(const EvictParams p, int smem_scores) {
  constexpr int NW = NT / 32;
  extern __shared__ __align__(16) float smem[];  // smem_scores (a multiple of 32) scores and 4 more, then a bit for each
  __shared__ uint32_t hist[kBins];
  __shared__ uint64_t list[kListMost];
  __shared__ uint32_t warp_sum[NW];
  __shared__ uint32_t sh_min, sh_max, sh_bin, sh_left, sh_count, sh_n;
  __shared__ uint64_t sh_rank;
  grid_launch_dependents();
  const int g = blockIdx.x, s = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int L = evict_len(p, s);
  const size_t rowi = (size_t)s * p.num_kv_heads + g;
  const float* row = p.scores + rowi * p.score_stride;
  float* out = p.scores_out + rowi * p.out_stride;
  int32_t* kept = p.kept + rowi * p.budget;

  if (L <= p.budget) {
    for (int t = tid; t < L; t += NT) {
      kept[t] = t;
      if (out != row) out[t] = row[t];
    }
    return;
  }
  const int first = p.sinks, last = L - p.recent;  // candidates are [first, last)
  uint32_t left = (uint32_t)(p.budget - p.sinks - p.recent);
  const bool whole = L <= smem_scores;
  if (tid == 0) {
    sh_min = 0xffffffffu;
    sh_max = 0u;
    sh_n = 0u;
  }
  for (int i = tid; i < kBins; i += NT) hist[i] = 0u;
  // the row in 16-byte loads, `head` scores before them; in shared memory as aligned as there
  const int head = min((int)((16u - (uint32_t)(reinterpret_cast<uintptr_t>(row) & 15u)) & 15u) >> 2, L);
  float* sm = smem + ((4 - head) & 3);
  const int quads = (L - head) >> 2;
  __syncthreads();
  uint32_t kmin = 0xffffffffu, kmax = 0u;
  auto look = [&](float x, int t) {
    if (t >= first && t < last) {
      const uint32_t k = score_key(x);
      kmin = min(kmin, k);
      kmax = max(kmax, k);
    }
  };
#pragma unroll 4
  for (int i = tid; i < quads; i += NT) {
    const int t = head + 4 * i;
    const float4 x = *reinterpret_cast<const float4*>(row + t);
    if (whole) *reinterpret_cast<float4*>(sm + t) = x;
    look(x.x, t);
    look(x.y, t + 1);
    look(x.z, t + 2);
    look(x.w, t + 3);
  }
  for (int i = tid; i < L - 4 * quads; i += NT) {  // at most 6: before the 16-byte loads and behind
    const int t = i < head ? i : i + 4 * quads;
    const float x = row[t];
    if (whole) sm[t] = x;
    look(x, t);
  }
  const float* from = whole ? sm : row;
  uint64_t threshold = ~0ull;  // above every rank: no candidate is kept
  uint64_t lo = ~0ull, hi = ~0ull;
  uint32_t* kept_bits = reinterpret_cast<uint32_t*>(smem + smem_scores + 4);  // of a stretch, a bit per token
  // a warp's tokens of a stretch of m: [w0, w1)
  auto mine = [&](int m, int& w0, int& w1) {
    const int per = (m + NT - 1) / NT * 32;
    w0 = min(warp * per, m);
    w1 = min(w0 + per, m);
  };
  if (left > 0) {
    kmin = __reduce_min_sync(kFullMask, kmin);
    kmax = __reduce_max_sync(kFullMask, kmax);
    if (lane == 0) {
      atomicMin(&sh_min, kmin);
      atomicMax(&sh_max, kmax);
    }
    __syncthreads();
    lo = (uint64_t)sh_min << 32, hi = ((uint64_t)sh_max << 32) | 0xffffffffu;
    for (bool every = true;; every = false) {  // every: [lo, hi] holds all candidates
      const int width = 64 - __clzll((long long)(hi - lo));
      const int shift = width > 11 ? width - 11 : 0;
      if (every && shift >= 32) {  // the positions do not count yet
        const uint32_t klo = (uint32_t)(lo >> 32);
#pragma unroll 8
        for (int t = first + tid; t < last; t += NT)
          atomicAdd(&hist[(score_key(from[t]) - klo) >> (shift - 32)], 1u);
      } else {
#pragma unroll 4
        for (int t = first + tid; t < last; t += NT) {
          const uint64_t r = rank_of(score_key(from[t]), t);
          if (r >= lo && r <= hi) atomicAdd(&hist[(uint32_t)((r - lo) >> shift)], 1u);
        }
      }
      __syncthreads();
      // a thread sums the bins kBins - 1 - (tid * P + j), from the largest down
      constexpr int P = kBins / NT;
      uint32_t c[P], sum = 0;
#pragma unroll
      for (int j = 0; j < P; ++j) {
        c[j] = hist[kBins - 1 - (tid * P + j)];
        sum += c[j];
      }
      uint32_t above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kFullMask, above, o);
        if (lane >= o) above += y;
      }
      if (lane == 31) warp_sum[warp] = above;
      __syncthreads();
      above -= sum;
#pragma unroll
      for (int i = 0; i < NW; ++i)
        if (i < warp) above += warp_sum[i];
      if (above < left && left <= above + sum) {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          if (above < left && left <= above + c[j]) {
            sh_bin = (uint32_t)(kBins - 1 - (tid * P + j));
            sh_left = left - above;
            sh_count = c[j];
          }
          above += c[j];
        }
      }
      __syncthreads();
      left = sh_left;
      lo += (uint64_t)sh_bin << shift;
      const uint64_t top = lo + (((uint64_t)1 << shift) - 1);
      hi = top < hi ? top : hi;
      if (sh_count <= kListMost) break;
      for (int i = tid; i < kBins; i += NT) hist[i] = 0u;
      __syncthreads();
    }
  } else {
    __syncthreads();  // the scores are in place
  }
  const uint32_t klo = (uint32_t)(lo >> 32), khi = (uint32_t)(hi >> 32);
  if (whole) {
    int w0, w1;
    mine(L, w0, w1);
#pragma unroll 4
    for (int i = w0; i < w1; i += 32) {
      const int t = i + lane;
      bool above = false;
      if (t < w1) {
        above = true;
        if (t >= first && t < last) {
          const uint32_t k = score_key(from[t]);
          above = k > khi;
          if (k >= klo && k <= khi) {
            const uint64_t r = rank_of(k, t);
            above = r > hi;
            if (r >= lo && r <= hi) list[atomicAdd(&sh_n, 1u)] = r;
          }
        }
      }
      const uint32_t b = __ballot_sync(kFullMask, above);
      if (lane == 0) kept_bits[i >> 5] = b;
    }
  } else if (left > 0) {
#pragma unroll 8
    for (int t = first + tid; t < last; t += NT) {
      const uint32_t k = score_key(from[t]);
      if (k >= klo && k <= khi) {
        const uint64_t r = rank_of(k, t);
        if (r >= lo && r <= hi) list[atomicAdd(&sh_n, 1u)] = r;
      }
    }
  }
  __syncthreads();
  const int n = (int)sh_n;
  for (int i = tid; i < n; i += NT) {
    const uint64_t r = list[i];
    uint32_t larger = 0;
    for (int j = 0; j < n; ++j) larger += list[j] > r;
    if (larger == left - 1) sh_rank = r;
    if (whole && larger < left) {
      const uint32_t t = ~(uint32_t)r;
      atomicOr(&kept_bits[t >> 5], 1u << (t & 31));
    }
  }
  __syncthreads();
  if (left > 0) threshold = sh_rank;

  // Ordered pass, a stretch of smem_scores tokens at a time: its scores are all
  // in shared memory before a place in it may be overwritten (scores in place).
  int base = 0;
  for (int64_t c0 = 0; c0 < L; c0 += smem_scores) {
    const int m = (int)min((int64_t)smem_scores, L - c0);
    int w0, w1;
    mine(m, w0, w1);
    if (!whole) {
#pragma unroll 8
      for (int t = tid; t < m; t += NT) sm[t] = row[c0 + t];
      __syncthreads();
      const uint32_t tkey = (uint32_t)(threshold >> 32), tpos = ~(uint32_t)threshold;
#pragma unroll 4
      for (int i = w0; i < w1; i += 32) {
        const int t = (int)c0 + i + lane;
        bool k = false;
        if (i + lane < w1) {
          const uint32_t key = score_key(sm[i + lane]);
          k = t < first || t >= last || key > tkey || (key == tkey && (uint32_t)t <= tpos);
        }
        const uint32_t b = __ballot_sync(kFullMask, k);
        if (lane == 0) kept_bits[i >> 5] = b;
      }
      __syncwarp();
    }
    // a lane's words of 32 tokens: their counts, and those of the lanes before it
    static_assert((NT == kSelectMost ? kScoresInSmem : kFewScores) <= 32 * NT, "a word to a lane");
    const bool has = w0 + 32 * lane < w1;
    const uint32_t bits = has ? kept_bits[(w0 >> 5) + lane] : 0u;
    int before = __popc(bits);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFullMask, before, o);
      if (lane >= o) before += y;
    }
    if (lane == 31) warp_sum[warp] = (uint32_t)before;
    before -= __popc(bits);
    __syncthreads();
    int at = base;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int v = (int)warp_sum[i];
      if (i < warp) at += v;
      base += v;
    }
#pragma unroll 4
    for (int i = w0; i < w1; i += 32) {
      const uint32_t b = __shfl_sync(kFullMask, bits, (i - w0) >> 5);
      const int to = at + __shfl_sync(kFullMask, before, (i - w0) >> 5) + __popc(b & ((1u << lane) - 1u));
      if (b >> lane & 1u) {
        kept[to] = (int)c0 + i + lane;
        out[to] = sm[i + lane];
      }
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// grid.x = (K or V, CTA of the cluster), y = kv head, z = sequence. The cluster
// (one CTA where there are many (sequence, head) pairs) moves the kept rows of its
// pool in ascending order, a chunk per CTA at a time. A row's new place is never
// behind its old one, so the stores of a step, made once the loads of it and of all
// steps before are done, overwrite nothing that is still to be read: rows may move
// within the blocks they lie in. The loads of the next step are asked for before
// the stores of this one (its rows lie behind every place written now), the
// addresses of the step after it before that.
//   V: vector of a row, VPR: vectors per row
template <typename V, int VPR>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictParams p, int cluster) {
  constexpr int NT = kMoveThreads, U = kMoveUnroll;
  constexpr int RC = NT * U / VPR;  // rows of a chunk
  __shared__ int64_t from[4][RC], to[4][RC];
  const int g = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
  const int rank = blockIdx.x % cluster;
  V* pool = static_cast<V*>(blockIdx.x / cluster ? p.v_cache : p.k_cache);
  const int n = min(evict_len(p, s), p.budget);
  const int32_t* kept = p.kept + ((size_t)s * p.num_kv_heads + g) * p.budget;
  const int32_t* src_row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
  const int32_t* dst_row = p.dst_block_tables + (size_t)s * p.max_blocks_per_seq;
  const int bits = __ffs(p.block_size) - 1, mask = p.block_size - 1;
  const int steps = ((n + RC - 1) / RC + cluster - 1) / cluster;

  auto find = [&](int step) {  // where the rows of a step's chunk are and go: -1 for none to move
    const int64_t r0 = ((int64_t)step * cluster + rank) * RC;
    for (int i = tid; i < RC; i += NT) {
      const int64_t r = r0 + i;
      int64_t a = -1, b = -1;
      if (r < n) {
        const int t = kept[r];
        const int x = __ldg(src_row + (t >> bits)), y = __ldg(dst_row + (r >> bits));
        if (x < 0 || x >= p.num_blocks || y < 0 || y >= p.num_blocks) {
          set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
        } else {
          a = ((int64_t)x * p.num_kv_heads + g) * p.block_size + (t & mask);
          b = ((int64_t)y * p.num_kv_heads + g) * p.block_size + ((int)r & mask);
          if (a == b) a = b = -1;
        }
      }
      from[step & 3][i] = a;
      to[step & 3][i] = b;
    }
  };
  V v[2][U];
  auto load = [&](int step, V (&x)[U]) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = j * NT + tid, r = i / VPR;
      const int64_t a = r < RC ? from[step & 3][r] : -1;
      if (a >= 0) x[j] = pool[a * VPR + (i - r * VPR)];
    }
  };
  auto store = [&](int step, const V (&x)[U]) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = j * NT + tid, r = i / VPR;
      const int64_t b = r < RC ? to[step & 3][r] : -1;
      if (b >= 0) pool[b * VPR + (i - r * VPR)] = x[j];
    }
  };
  auto one = [&](int k, V (&now)[U], V (&next)[U]) {
    if (k + 1 < steps) load(k + 1, next);
    if (k + 2 < steps) find(k + 2);
    if (cluster > 1)
      cluster_barrier();
    else
      __syncthreads();
    store(k, now);
  };

  grid_dependency_wait();  // the kept positions
  if (steps > 0) {
    find(0);
    if (steps > 1) find(1);
    __syncthreads();
    load(0, v[0]);
    for (int k = 0; k < steps; k += 2) {
      one(k, v[0], v[1]);
      if (k + 1 < steps) one(k + 1, v[1], v[0]);
    }
  }
  if (blockIdx.x == 0 && g == 0 && tid == 0) p.new_context_lens[s] = n;
}

template <typename K, typename... Args>
cudaError_t launch_with(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, int cluster, bool dependent,
                        Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  cfg.attrs = attr;
  if (cluster > 1) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (dependent) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int NT>
cudaError_t launch_select(const EvictParams& p, cudaStream_t stream) {
  const int scores = p.cap < kScoresInSmem ? (p.cap / 32 + 1) * 32 : kScoresInSmem;
  const size_t smem = ((size_t)scores * 33 / 32 + 4) * sizeof(float);
  static int configured[64] = {0};  // per device ordinal
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(evict_select_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (kScoresInSmem / 32 * 33 + 4) * (int)sizeof(float));
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
  }
  return launch_with(evict_select_kernel<NT>, dim3(p.num_kv_heads, p.num_seqs), NT, smem, stream, 1, false, p, scores);
}

template <typename V, int VPR>
cudaError_t launch_move(const EvictParams& p, cudaStream_t stream) {
  constexpr int64_t rows = kMoveThreads * kMoveUnroll / VPR;
  const int64_t chains = (int64_t)p.num_seqs * p.num_kv_heads * 2;
  const int64_t chunks = ((p.budget < p.cap ? p.budget : p.cap) + rows - 1) / rows;
  // few (sequence, head, pool) triples: clusters of up to 8 CTAs share one, while
  // that gives each SM no more than two CTAs and each CTA a chunk (one sequence of
  // 8 kv heads: 8.3 us, 9.6 with clusters of 4, 15.7 with none)
  int cluster = 1;
  while (cluster < 8 && chains * cluster * 2 <= 304 && cluster < chunks) cluster *= 2;
  return launch_with(evict_move_kernel<V, VPR>, dim3(2 * cluster, p.num_kv_heads, p.num_seqs), kMoveThreads, 0, stream,
                     cluster, true, p, cluster);
}

}  // namespace

cudaError_t launch_evict(const EvictParams& p, cudaStream_t stream) {
  // threads for a row's selection: 1024 for rows of up to kFewScores instead of 512 take 10.0
  // us instead of 8.3 (one sequence of 2001) and 116 instead of 106 (64 of up to 4000); longer
  // rows need them, a word of bits to a lane
  const cudaError_t e = p.cap > kFewScores ? launch_select<kSelectMost>(p, stream) : launch_select<kSelectFew>(p, stream);
  if (e != cudaSuccess) return e;
  switch (p.row_bytes) {
    case 36: return launch_move<uint32_t, 9>(p, stream);
    case 64: return launch_move<uint4, 4>(p, stream);
    case 72: return launch_move<uint2, 9>(p, stream);
    case 128: return launch_move<uint4, 8>(p, stream);
    case 256: return launch_move<uint4, 16>(p, stream);
    case 512: return launch_move<uint4, 32>(p, stream);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace pkv
