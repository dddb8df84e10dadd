// Paged prefill over the first tokens and a sliding window (sm_103a): the query at
// position P of its sequence sees the tokens t <= P with t < sinks or
// t > P - window.
//
// Work: the queries of a sequence against one kv head are n x group rows, row
// m = i * group + j for new token i and the kv head's j-th query head, so that a
// tile of 128 rows holds few tokens and K/V are read once for a whole group. One
// CTA takes two such tiles, A and B, and walks the K/V tiles of 128 tokens that one
// of their queries sees: those of the sinks, then those from the first query's
// window on. On the fifth-generation tensor cores S = Q K^T and O += P V accumulate
// in fp32 in tensor memory; a softmax warpgroup of its own serves each of A and B, a
// row to a thread, so that one tile's exponentials run under the other's MMAs. A CTA
// stays on its SM and takes one pair of query tiles after another; every role runs
// ahead into the next pair as far as the barriers let it, so that the start of one
// pair lies under the end of another.
// Where there are few pairs, a cluster shares one: each of its CTAs walks a part
// of the K/V tiles, and the parts are joined through the cluster's shared memory
// (log-sum-exp).
// P enters its product as a 16-bit high part and a 16-bit remainder, two MMAs for one: 16
// significant bits or more. One part, 2^-8 (bfloat16) or 2^-11 of each weight, would put an error
// of its own beside the output's rounding (each is that fraction of the output, rms, whatever
// the values' signs): 1.4 times the rounding's alone; it would take 214 us instead of 260 for
// the 8192 queries below.
// Bound by the MMAs for long walks: 8192 queries over a window of 2048 (32 query and 8 kv heads,
// bfloat16, head_dim 128) take 260 us of GPU time (as all times here), 930 TFLOP/s over the visible
// tokens and 1400 with the remainders' MMAs (1956 are the library product's); the tensor pipe is
// active for 71 %. A step of 128 tokens for both A and B takes
// about 3500 cycles, 87 % of them MMAs; what lies between is the way from S over the softmax and
// the waits to the next MMA. Tiles that a row sees in part take longer, the start and the end
// of a pair some 8000 cycles: of short walks they are most (8 sequences of up to
// 1500 tokens, window 500, head_dim 64, 40 heads: 114 us). One chunk of 100 queries, window
// 1024: 18 us.
#pragma once

#include <type_traits>

#include "tc.cuh"

namespace pkv {

constexpr int kPwRows = 128;     // rows of a query tile = tensor-memory lanes
constexpr int kPwTokens = 128;   // tokens of a K/V tile
constexpr int kPwStages = 4;     // tiles in shared memory: two links of a V and a K tile
constexpr int kPwSoft = 256;     // 2 softmax warpgroups
constexpr int kPwThreads = kPwSoft + 128;  // + MMA warp of A, TMA warp, clearing warp, MMA warp of B
constexpr uint32_t kPwTmemCols = 512;     // S of A and B (128 columns each), O of A and B
constexpr float kPwFar = 8388608.f;       // 2^23
// CTAs to a cluster at most. One chunk of 100 queries, window 1024: 29 us with 1, 23 with 2,
// 18 with 4; of clusters of 8 no more than 15 are resident at a time, so that 16 items
// would take two rounds.
constexpr int kPwMaxCluster = 4;

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31 as a product and a shift: with
// 2^(s-1) < d <= 2^s and m = ceil(2^(31+s) / d), n / d = n m >> (31 + s). (An integer
// division takes some hundred cycles in a warp that comes by seldom, and the start of
// a pair has several.)
struct PwDivisor {
  uint32_t d, m, s;
  void set(uint32_t divisor) {
    d = divisor;
    s = 0;
    while ((1ull << s) < d) ++s;
    m = (uint32_t)(((1ull << (31 + s)) + d - 1) / d);
  }
  __device__ __forceinline__ int of(int n) const { return (int)(((uint64_t)(uint32_t)n * m) >> (31 + s)); }
};

struct PrefillWindowParams {
  void* out;
  const void* q;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  float scale_log2;   // |scale| * log2(e), above 0
  uint32_t flip;      // sign bits of a pair of query elements for a negative scale, else 0
  int window, sinks;  // window >= 1, sinks >= 0, no larger than the longest table
  int num_seqs, num_heads, num_kv_heads, group, block_size, max_blocks_per_seq, num_blocks;
  int pairs;    // of the longest sequence, per kv head
  PwDivisor by_columns, by_heads, by_group;  // num_seqs * num_kv_heads, num_kv_heads, group
  int cluster;  // CTAs that share a pair of query tiles
  int32_t* dev_err;
  uint64_t wait_limit_ns;  // limit of every wait on another role's progress
};

// The base of a row's running maximum moves only when that grows by more than
// kRescaleLog2, and it lies kTopLog2 - kRescaleLog2 below the maximum that it was taken
// from, so that every weight stays below 2^kTopLog2. In bfloat16 the base is that maximum and
// moves by 8 (with 0: 9 % slower). Binary16 has a short range: its weights reach up to 2^15, so that
// they keep 22 bits down to 2^-16 of the largest and have an error of 2^-38 of it below that (with
// 2^8, 2^-32: 2^17 tokens that far below one other lose 2^-15 of the output). The base moves by 2; by 8, 4
// or 1 the time is the same (8 sequences of up to 1500 tokens, 40 heads of 64).
template <typename T>
struct PwPack;
template <>
struct PwPack<__half> {
  static constexpr float kRescaleLog2 = 2.f, kTopLog2 = 15.f;
  __device__ __forceinline__ static uint32_t pack(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
  }
  // the high part of a pair of weights, packed, and what it stands for
  __device__ __forceinline__ static uint32_t high(float2 e, float2& h) {
    const __half2 r = __floats2half2_rn(e.x, e.y);
    h = __half22float2(r);
    uint32_t u;
    memcpy(&u, &r, 4);
    return u;
  }
};
template <>
struct PwPack<__nv_bfloat16> {
  static constexpr float kRescaleLog2 = 8.f, kTopLog2 = 8.f;
  __device__ __forceinline__ static uint32_t pack(float x, float y) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    uint32_t u;
    memcpy(&u, &h, 4);
    return u;
  }
  // (cut off, which takes fewer instructions than rounding: the remainder is at most
  // 2^-7 of the weight, its own rounding 2^-16)
  __device__ __forceinline__ static uint32_t high(float2 e, float2& h) {
    const uint32_t x = __float_as_uint(e.x), y = __float_as_uint(e.y);
    h = make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u));
    return __byte_perm(x, y, 0x7632);
  }
};

// 2^x by the hardware's approximate exponential (relative error about 2^-22, -inf
// -> +0); what it gives is rounded to 16 bits afterwards.
__device__ __forceinline__ float pw_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared memory of a CTA, from a 1024-byte aligned base: Q of A and B
// ([D / 64 column blocks][128 rows][128 bytes] each), then the K/V stages (the same
// with tokens as rows), barriers, tensor-memory address. The join of a cluster
// reuses it from the start: O [2][128][D] in fp32, then (m, l).
template <int D>
struct PwShape {
  static constexpr int kCB = D / 64;
  static constexpr int kColBlock = 128 * 128;
  static constexpr int kTile = kCB * kColBlock;  // a Q, K or V tile
  static constexpr int kStageOff = 2 * kTile;
  static constexpr int kBarOff = kStageOff + kPwStages * kTile;
  static constexpr int kSlotOff = kBarOff + 24 * 8;
  static constexpr int kOutOff = kSlotOff + 64;           // 4 KB per softmax warp: output rows on their way out
  static constexpr int kUsed = kOutOff + 8 * 4096 + 1024;  // + alignment slack
  // more than half of an SM's, so that one CTA has its tensor memory to itself
  static constexpr int kSmemBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static constexpr int kJoinMl = 2 * kPwRows * D * 4;
  static_assert(kJoinMl + 2 * kPwRows * 8 <= kBarOff, "room for the join");
};

// mbar_wait_bounded with the clock left alone until the hardware's own wait has run out once
// (two readings of the global timer before it made every wait that had to wait late).
__device__ __forceinline__ bool pw_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_test_wait(bar, parity)) return true;
  if (limit_ns == 0) return false;
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  do {
    if (mbar_try_wait(bar, parity)) return true;
  } while (globaltimer_ns() - t0 < limit_ns);
  return false;
}

__device__ __forceinline__ uint32_t pw_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void pw_cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of `saddr` in the shared memory of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t pw_remote(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 pw_remote_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a)
               : "memory");
  return v;
}
__device__ __forceinline__ float2 pw_remote_f2(uint32_t a) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// What a CTA walks: K/V tiles [0, first) hold the sinks, [from, end) the windows; its
// part is the j-th of these for j in [j0, j1).
struct PwWalk {
  int first, from, j0, j1;
  __device__ __forceinline__ int tile(int j) const { return j < first ? j : j - first + from; }
};

// The tokens that the queries of one query tile see: [0, min(sinks, end)) and [lo, end).
struct PwSpan {
  int lo, end;
  __device__ __forceinline__ bool sees(int k0, int sinks) const {  // one of [k0, k0 + kPwTokens)
    return k0 < end && (k0 < sinks || k0 + kPwTokens > lo);
  }
};

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pw_pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 pw_unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t pw_fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t pw_add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// The MMAs of kind::f16 with a descriptor's words apart (see mma_ss, mma_ts).
__device__ __forceinline__ void pw_mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tmov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void pw_mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\ttcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(hi), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The lowest n bits set (none for n <= 0, all for n >= 32).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

__device__ __forceinline__ float pw_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// A warp's walk over the items `item`, `item` + step, .. < items that have query rows.
// The grid is laid out for the longest sequence, so that in a ragged batch most may have
// none: 32 are looked at together, one by a lane (8192 queries beside 63 sequences of one
// query each, window 1024: 240 us, 169 for the 8192 alone; 70 us more with a look at one item
// after another).
struct PwScan {
  int base;       // item of lane 0
  uint32_t mask;  // lanes whose items are still to come
  __device__ __forceinline__ void look(const PrefillWindowParams& p, int item, int step, int items, bool report) {
    base = item;
    const int i = item + (int)(threadIdx.x & 31) * step;
    bool some = false;
    if (i < items) {
      const int row = p.by_columns.of(i), s = p.by_heads.of(i - row * (int)p.by_columns.d);
      const int L = __ldg(p.context_lens + s), n = __ldg(p.query_start + s + 1) - __ldg(p.query_start + s);
      if (L < 0 || L > p.max_blocks_per_seq * p.block_size || n < 0 || n > L) {
        if (report) set_err(p.dev_err, PKV_DEV_ERR_CONTEXT_LEN);
      } else {
        some = (p.pairs - 1 - row) * 2 * kPwRows < (int64_t)n * p.group;
      }
    }
    mask = __ballot_sync(kFullMask, some);
  }
  __device__ __forceinline__ int ahead(int step) const { return base + (__ffs(mask) - 1) * step; }
  // Moves `item` on to the next with rows; false past the last.
  __device__ __forceinline__ bool next(const PrefillWindowParams& p, int step, int items, int& item) {
    while (mask == 0u) {
      if (items - base <= 32 * step) return false;
      look(p, base + 32 * step, step, items, false);
    }
    item = ahead(step);
    mask &= mask - 1;
    return true;
  }
};

// A pair of query tiles of one sequence and kv head, and the K/V tiles this CTA
// walks for it.
struct PwItem {
  int s, kvh, L, q0, n, row0, rows;  // rows: query rows of the kv head
  int active_a, active_b;            // rows of A and B
  PwSpan span_a, span_b;
  int kv_end, wlo;  // past the last token that a query sees; first token in the first query's window
  PwWalk walk;

  // The item with index `item`, which has rows (its lengths come from the first-level
  // cache, where the scan left them, and in registers that a warp shares).
  __device__ __forceinline__ void load(const PrefillWindowParams& p, int item, uint32_t rank) {
    const int row = p.by_columns.of(item), column = item - row * (int)p.by_columns.d;
    const int pair = p.pairs - 1 - row;  // later queries first: theirs are the longest walks
    s = p.by_heads.of(column);
    kvh = column - s * p.num_kv_heads;
    L = __ldg(p.context_lens + s);
    q0 = __ldg(p.query_start + s);
    n = __ldg(p.query_start + s + 1) - q0;
    rows = (int)min((int64_t)n * p.group, (int64_t)p.pairs * 2 * kPwRows);  // the launch covers no more
    row0 = pair * 2 * kPwRows;
    auto place = [&](int a, int& active, PwSpan& span) {
      active = max(min(rows - a, kPwRows), 0);
      const int t0 = p.by_group.of(a), t1 = p.by_group.of(a + max(active, 1) - 1);
      const int p0 = L - n + t0;
      span.lo = p0 >= p.window ? p0 - p.window + 1 : 0;
      span.end = active > 0 ? L - n + t1 + 1 : 0;
    };
    place(row0, active_a, span_a);
    place(row0 + kPwRows, active_b, span_b);
    kv_end = max(span_a.end, span_b.end);
    wlo = span_a.lo;
    const int tend = (kv_end + kPwTokens - 1) / kPwTokens;
    walk.first = (min(p.sinks, kv_end) + kPwTokens - 1) / kPwTokens;
    walk.from = max(wlo / kPwTokens, walk.first);
    const int all = walk.first + tend - walk.from;
    walk.j0 = p.cluster == 1 ? 0 : (int)((int64_t)all * rank / p.cluster);
    walk.j1 = p.cluster == 1 ? all : (int)((int64_t)all * (rank + 1) / p.cluster);
  }
  __device__ __forceinline__ PwSpan span(int x) const { return x ? span_b : span_a; }
  // Rows [hide0, hide1) and from `tail` on of the K/V tile at k0 are seen by no query.
  __device__ __forceinline__ bool hidden(const PrefillWindowParams& p, int k0, int& hide0, int& hide1,
                                         int& tail) const {
    hide0 = max(p.sinks - k0, 0);
    hide1 = min(wlo - k0, kPwTokens);
    tail = min(kv_end - k0, kPwTokens);
    return hide0 < hide1 || tail < kPwTokens;
  }
};

template <typename T, int D>
__global__ void __launch_bounds__(kPwThreads, 1)
    pa_prefill_window_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                             const __grid_constant__ PrefillWindowParams p) {
  using S = PwShape<D>;
  using P16 = PwPack<T>;
  constexpr int kBf16 = std::is_same<T, __nv_bfloat16>::value ? 1 : 0;
  constexpr int CB = S::kCB;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // Every barrier's phases follow one another in the order of the work (K/V tiles, or
  // pairs of query tiles), and nobody who waits for a phase can fall two behind.
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBarOff);
  // K and V tiles come as links of a chain: the V of one tile with the K of the next,
  // which the MMAs of one step need together (a pair of query tiles of n K/V tiles
  // has n + 1 links: the first without V, the last without K). Link c is in stages
  // 2 (c % 2) (K) and 2 (c % 2) + 1 (V).
  uint64_t* full = bars;         // [2] the link landed
  uint64_t* ready = bars + 2;    // [2] and rows of its V that no query sees are cleared
  uint64_t* empty = bars + 4;    // [2] the MMAs are done with it (A's and B's: two arrivals)
  uint64_t* s_full = bars + 6;   // [A, B] S computed
  uint64_t* p_full = bars + 8;   // [A, B] P written (one arrival per softmax warp)
  uint64_t* q_full = bars + 10;  // [A, B] query rows in place (one arrival per softmax warp)
  uint64_t* o_full = bars + 12;  // [A, B] the pair's last O computed
  uint64_t* drained = bars + 14; // every MMA of the CTA done (two arrivals)
  uint64_t* turn = bars + 15;    // [A, B] the other's MMAs of a link are issued
  uint32_t* slot = reinterpret_cast<uint32_t*>(sm + S::kSlotOff);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = p.cluster;
  const uint32_t rank = cluster > 1 ? pw_cluster_rank() : 0u;
  const int items = p.pairs * p.num_seqs * p.num_kv_heads;
  const int item0 = blockIdx.x / cluster, step = gridDim.x / cluster;

  // ---- set-up: barriers, tensor memory ----------------------------------------
  if (tid == 0) {
    for (int i = 0; i < 17; ++i) mbar_init(&bars[i], i == 4 || i == 5 || i == 14 ? 2 : (i >= 8 && i < 12 ? 4 : 1));
    mbar_init_fence();
  }
  if (warp == 8) tmem_alloc(slot, kPwTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *slot;
  bool bad = false;  // a wait ran out

  if (warp == 9) {
    // ---- TMA: K and V tiles, box by box (one box: 64 head dims of one cache block of
    // the kv head); lane b holds the row of block b of the next tile in the pool
    PwItem it;
    PwScan scan;
    scan.look(p, item0, step, items, false);
    const int per_tile = kPwTokens / p.block_size;  // <= 16 blocks
    const int bs = p.block_size, bits = __ffs(bs) - 1;
    const int zero_row = p.num_blocks * p.num_kv_heads * bs;  // first row past the pool: reads zeros
    const uint32_t box_bytes = (uint32_t)bs * 128u;
    uint32_t link = 0;  // links so far
    for (int item; !bad && scan.next(p, step, items, item);) {
      it.load(p, item, rank);
      const int32_t* bt = p.block_tables + (size_t)it.s * p.max_blocks_per_seq;
      auto blocks_of = [&](int k0) { return min(per_tile, (it.kv_end - k0 + bs - 1) >> bits); };
      auto seen = [&](int k) { return k < p.sinks || k + bs > it.wlo; };  // the block at token k, by a query
      auto fetch = [&](int j) {  // issues the load only
        if (j >= it.walk.j1) return -1;
        const int k0 = it.walk.tile(j) * kPwTokens, k = k0 + lane * bs;
        return lane < blocks_of(k0) && seen(k) ? __ldg(bt + (k >> bits)) : -1;
      };
      int id = fetch(it.walk.j0);
      int y = zero_row, nblk = 0;  // of the tile whose V is next
      for (int j = it.walk.j0; j <= it.walk.j1 && it.walk.j0 < it.walk.j1; ++j, ++link) {  // K of tile j, V of tile j - 1
        const uint32_t c = link & 1;
        const int k0 = j < it.walk.j1 ? it.walk.tile(j) * kPwTokens : 0;
        const int nk = j < it.walk.j1 ? blocks_of(k0) : 0;
        int yk = zero_row;
        if (lane < nk && seen(k0 + lane * bs)) {
          if (id >= 0 && id < p.num_blocks)
            yk = (id * p.num_kv_heads + it.kvh) * bs;
          else
            set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
        }
        id = fetch(j + 1);
        if (link >= 2 &&
            !__all_sync(kFullMask, pw_wait(&empty[c], ((link >> 1) + 1) & 1, p.wait_limit_ns))) {
          bad = true;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(&full[c], (uint32_t)((nk + nblk) * CB) * box_bytes);
        __syncwarp();
        const int b = lane / CB, cb = lane % CB;
        const int row_k = __shfl_sync(kFullMask, yk, b), row_v = __shfl_sync(kFullMask, y, b);
        unsigned char* at = sm + S::kStageOff + 2 * c * S::kTile + cb * S::kColBlock + b * bs * 128;
        if (lane < nblk * CB) tma_load_2d(at + S::kTile, &vmap, cb * 64, row_v, &full[c]);
        if (lane < nk * CB) tma_load_2d(at, &kmap, cb * 64, row_k, &full[c]);
        y = yk;
        nblk = nk;
      }
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    // the last links must land and come back before the CTA can leave (earlier ones are
    // known to have)
    if (lane == 0)
      for (uint32_t c = link >= 2 ? link - 2 : 0; c < link; ++c) {
        mbar_wait_bounded(&full[c & 1], (c >> 1) & 1, kDrainLimitNs);
        if (!bad) pw_wait(&empty[c & 1], (c >> 1) & 1, p.wait_limit_ns);
      }
    __syncwarp();
  } else if (warp == 8 || warp == 11) {
    // ---- MMA issue, a warp for each of A and B ------------------------------------------
    // Per link: O += P V of one tile, S of the next. At head_dim 128 the two take turns, A
    // first, so that A's softmax runs under B's MMAs and the other way round: without turns
    // both fall into step and the tensor pipe idles under both softmaxes. The pipe holds no
    // more than an MMA or two ahead, so that what comes between one's MMAs and the other's
    // leaves it idle: each makes its waits, and works out its next step, under the other's
    // MMAs (without turns 4 % slower for 8192 queries, window 2048, 32 query and 8 kv heads; one warp
    // for both 5 %, when P had one part). At head_dim 64 the MMAs are shorter than the softmax, and both
    // may go as they are ready (114 us, 119 with turns, for 8 sequences of 40 heads).
    // MMAs of one thread complete in order, so S may take the place of a P that the MMA
    // before it reads, and "S done" says that O holds every earlier tile.
    // The whole warp walks and waits, one elected lane issues; what a step needs to know is
    // worked out before its wait.
    const int x = warp == 8 ? 0 : 1;
    constexpr bool kTurns = D == 128;
    constexpr uint32_t id_s = mma_idesc_f16(kPwRows, kPwTokens, kBf16, 0);
    constexpr uint32_t id_o = mma_idesc_f16(kPwRows, D, kBf16, 1);
    const uint32_t tb = __shfl_sync(kFullMask, tbase, 0);
    const uint32_t sb = __shfl_sync(kFullMask, smem_u32(sm), 0);
    // of a descriptor only the start address in its low word moves (shared addresses stay
    // below 256 KB, so the sums never carry out of the field)
    const uint32_t qd = (uint32_t)smem_desc_sw128(sb + x * S::kTile, 16, 1024);
    const uint32_t kd = (uint32_t)smem_desc_sw128(sb + S::kStageOff, 16, 1024);
    const uint32_t vd = (uint32_t)smem_desc_sw128(sb + S::kStageOff + S::kTile, S::kColBlock, 1024);
    const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);  // K-major and MN-major alike
    uint32_t link = 0, nth = 0, done = 0;  // links, pairs and P's so far
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool ok = __all_sync(kFullMask, pw_wait(bar, parity, p.wait_limit_ns));
      tc_fence_after();
      return ok;
    };
    // within one elected region: S into the place of the scores ...
    auto mmas_s = [&](uint32_t c) {
      const uint32_t kb = kd + (c * (2 * S::kTile) >> 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t off = ((ks >> 2) * S::kColBlock + (ks & 3) * 32) >> 4;
        pw_mma_ss(tb + 128 * x, qd + off, kb + off, hi, id_s, ks > 0);
      }
      mma_commit(&s_full[x]);
    };
    // ... and O += P V
    auto mmas_o = [&](uint32_t c, bool first) {
      const uint32_t vb = vd + (c * (2 * S::kTile) >> 4);
#pragma unroll
      for (int part = 0; part < 2; ++part)  // the high parts of P, then the remainders
#pragma unroll
        for (int ks = 0; ks < kPwTokens / 16; ++ks)
          pw_mma_ts(tb + 256 + 128 * x, tb + 128 * x + 64 * part + 8 * ks, vb + (ks * 2048 >> 4), hi, id_o,
                    (part > 0 || ks > 0 || !first) ? 1u : 0u);
    };
    PwItem it;
    PwScan scan;
    scan.look(p, item0, step, items, false);
    for (int item; !bad && scan.next(p, step, items, item);) {
      it.load(p, item, rank);
      const int tiles = it.walk.j1 - it.walk.j0;
      const PwSpan span = it.span(x);
      bool sees = false, opened = false;                   // the tile at hand is seen, O holds something
      // rows that no S of this part needs are in place before the pair ends all the same
      bad = !wait(&q_full[x], nth & 1);
      int k1 = 0;  // the tile whose S is next
      bool next = false;
      auto look = [&](int i) {
        k1 = i < tiles ? it.walk.tile(it.walk.j0 + i) * kPwTokens : 0;
        next = i < tiles && span.sees(k1, p.sinks);
      };
      look(0);
      for (int i = tiles > 0 ? 0 : 1; i <= tiles && !bad; ++i, ++link) {  // O of tile i - 1, S of tile i
        const uint32_t c = link & 1;
        bad = !wait(&ready[c], (link >> 1) & 1);
        if (kTurns && !bad && (x == 1 || link > 0)) bad = !wait(&turn[x], (link + (x ^ 1)) & 1);
        // (a pair's first P comes from warps that have read the O of the pair before)
        if (!bad && sees) bad = !wait(&p_full[x], done++ & 1);
        if (!bad && elect_one()) {
          if (sees) mmas_o(c, !opened);
          if (next)
            mmas_s(c);
          else
            mma_commit(&empty[c]);  // (with an S the softmax sees to that)
          if (kTurns) mbar_arrive(&turn[x ^ 1]);
        }
        __syncwarp();
        opened |= sees;
        sees = next;
        look(i + 1);
      }
      if (!bad && elect_one()) {
        mma_commit(&o_full[x]);
      }
      __syncwarp();
      ++nth;
    }
    // nothing may be torn down before the last MMA, after a timeout neither
    if (elect_one()) mma_commit(drained);
    __syncwarp();
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    mbar_wait_bounded(drained, 0, kDrainLimitNs);
    __syncwarp();
  } else if (warp == 10) {
    // ---- the links: rows of a V tile that no query sees may hold anything (a NaN would
    // survive a zero weight), they become zeros
    PwItem it;
    PwScan scan;
    scan.look(p, item0, step, items, false);
    const T* q = static_cast<const T*>(p.q);
    uint32_t link = 0;  // links so far
    for (int item; !bad && scan.next(p, step, items, item);) {
      it.load(p, item, rank);
      for (int j = it.walk.j0; j <= it.walk.j1 && it.walk.j0 < it.walk.j1; ++j, ++link) {
        const uint32_t c = link & 1;
        if (!__all_sync(kFullMask, pw_wait(&full[c], (link >> 1) & 1, p.wait_limit_ns))) {
          bad = true;
          break;
        }
        int h0, h1, tail;
        if (j > it.walk.j0 && it.hidden(p, it.walk.tile(j - 1) * kPwTokens, h0, h1, tail)) {
          unsigned char* v = sm + S::kStageOff + (2 * c + 1) * S::kTile;
          const int before = max(h1 - h0, 0), count = before + kPwTokens - tail;  // hidden rows
          for (int e = lane; e < count * CB * 8; e += 32) {
            const int i2 = e / (CB * 8), ch = e % (CB * 8), r = i2 < before ? h0 + i2 : tail + i2 - before;
            *reinterpret_cast<uint4*>(v + (ch >> 3) * S::kColBlock + r * 128 + (ch & 7) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ready[c]);
        // in passing, the next pair's query rows into L2 (a hint only)
        if (j == it.walk.j0 + 1 && scan.mask != 0u) {
          const int next = scan.ahead(step);
          const int row = p.by_columns.of(next), column = next - row * (int)p.by_columns.d;
          const int of = p.by_heads.of(column), head = (column - of * p.num_kv_heads) * p.group;
          const int q0 = __ldg(p.query_start + of), n = __ldg(p.query_start + of + 1) - q0;
          const int g0 = (p.pairs - 1 - row) * 2 * kPwRows;
          const int rows = (int)min((int64_t)n * p.group - g0, (int64_t)2 * kPwRows);
#pragma unroll 4
          for (int e = lane; e < rows * CB; e += 32) {
            const int g = g0 + e / CB, t = p.by_group.of(g);
            asm volatile("prefetch.global.L2 [%0];" ::"l"(
                q + ((size_t)(q0 + t) * p.num_heads + head + g - t * p.group) * D + e % CB * 64));
          }
        }
      }
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
  } else {
    // ---- softmax: warpgroup x serves query tile x, a row to a thread --------------------
    PwItem it;
    const int x = warp >> 2, r = tid & 127;
    const uint32_t ts = tbase + ((uint32_t)(32 * (warp & 3)) << 16) + 128 * x;  // S of this warp's lanes
    const uint32_t to = ts + 256;                                              // and O
    const float sc = p.scale_log2;  // > 0
    uint32_t done = 0, nth = 0, link = 0;  // tiles, pairs and links so far
    int item = item0;
    auto find = [&]() {  // the pair at `item` or the next that has rows
      for (; item < items; item += 32 * step) {
        PwScan scan;  // (no registers to spare for one that is kept)
        scan.look(p, item, step, items, warp == 0);
        if (scan.mask == 0u) continue;
        item = scan.ahead(step);
        it.load(p, item, rank);
        return true;
      }
      return false;
    };
    // The pair's query rows, 16 bytes a copy, 128 bytes of a row by 8 lanes. S of the pair before
    // is over, so their place is free.
    const uint32_t q_at = smem_u32(sm + x * S::kTile), q_row = 32 * (warp & 3) + (lane >> 3), ch = lane & 7;
    auto copy_q = [&]() {
      const T* q = static_cast<const T*>(p.q);
      const int active = x ? it.active_b : it.active_a;
#pragma unroll 4
      for (int rr = q_row; rr < 32 * (warp & 3) + 32; rr += 4) {
        const bool in = rr < active;
        const int g = it.row0 + x * kPwRows + rr, t = in ? p.by_group.of(g) : 0, j = in ? g - t * p.group : 0;
        const T* src = q + ((size_t)(it.q0 + t) * p.num_heads + it.kvh * p.group + j) * D + 8 * ch;
        const uint32_t to = q_at + rr * 128 + ((ch ^ (rr & 7)) << 4), bytes = in ? 16 : 0;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + cb * S::kColBlock),
                       "l"(src + cb * 64), "r"(bytes)
                       : "memory");
      }
    };
    auto copied_q = [&]() {
      asm volatile("cp.async.wait_all;" ::: "memory");
      if (p.flip != 0u) {  // a negative scale: the queries change their sign instead
        for (int e = 0; e < 8 * CB; ++e) {
          const int rr = q_row + 4 * (e / CB);
          uint4* at = reinterpret_cast<uint4*>(sm + x * S::kTile + (e % CB) * S::kColBlock + rr * 128 +
                                               ((ch ^ (rr & 7)) << 4));
          const uint4 f = *at;
          *at = make_uint4(f.x ^ p.flip, f.y ^ p.flip, f.z ^ p.flip, f.w ^ p.flip);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&q_full[x]);
    };
    bool have = find();
    if (have) {
      copy_q();
      copied_q();
    }
    while (have) {
      const int active = x ? it.active_b : it.active_a;
      const PwSpan span = it.span(x);
      const int g = it.row0 + x * kPwRows + min(r, max(active - 1, 0));  // past the last row: any finite result
      const int tok = p.by_group.of(g);
      const int pos = it.L - it.n + tok;
      float m_use = -INFINITY, l = 0.f;
      bool first = true;
      for (int j = it.walk.j0; j < it.walk.j1; ++j) {
        const int k0 = it.walk.tile(j) * kPwTokens;
        if (!span.sees(k0, p.sinks)) continue;
        const int vis = pos - k0 + 1;                // tokens of the tile up to the row's own
        const int before = pos - p.window + 1 - k0;  // tokens of the tile before its window
        const bool cut = __any_sync(kFullMask, vis < kPwTokens || before > 0);
        // every wait is made warp-uniform before the warp-collective loads and stores
        if (!__all_sync(kFullMask, pw_wait(&s_full[x], done & 1, p.wait_limit_ns))) {
          bad = true;
          break;
        }
        tc_fence_after();
        // S is the query tile's last MMA that reads its link
        if ((warp & 3) == 0 && lane == 0) mbar_arrive(&empty[(link + (j - it.walk.j0)) & 1]);
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, u[c]);
        tmem_wait_ld();
        float* v = reinterpret_cast<float*>(&u[0][0]);
        // (raw scores: their maximum is the scaled scores', the scale being positive)
        if (cut) {
          const int kept = p.sinks - k0;  // of those before the window, the sinks stay
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // the row's visible tokens of 32 as bits: [0, vis) without [kept, before)
            const uint32_t hide = low_bits(before - 32 * c) & ~low_bits(kept - 32 * c);
            const uint32_t see = low_bits(vis - 32 * c) & ~hide;
            if (__any_sync(kFullMask, see != 0xffffffffu)) {
#pragma unroll
              for (int i = 0; i < 32; ++i) v[32 * c + i] = (see >> i) & 1u ? v[32 * c + i] : -INFINITY;
            }
          }
        }
        float m4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) m4[i] = fmaxf(v[i], v[i + 4]);
#pragma unroll
        for (int i = 8; i < 128; i += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) m4[e] = pw_max3(m4[e], v[i + e], v[i + e + 4]);
        const float mt = sc * fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
        // the base moves only when the maximum grows by more than kRescaleLog2: every
        // P stays below 2^kTopLog2, and O and the row sum have the same base. (Logits from kPwFar on
        // are whole numbers, and a base may be off by half their distance: there it is the maximum
        // and moves whenever that does.)
        const bool grow = mt - m_use > (fabsf(m_use) < kPwFar ? P16::kTopLog2 : 0.f);  // (no for -inf - -inf)
        float alpha = 1.f;
        if (grow) {
          const float base = mt - (fabsf(mt) < kPwFar ? P16::kTopLog2 - P16::kRescaleLog2 : 0.f);
          alpha = exp2f(m_use - base);  // 0 while nothing was visible
          m_use = base;
        }
        if (!first && __any_sync(kFullMask, grow)) {
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t w[16];
            tmem_ld16(to + 16 * c, w);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
            tmem_st16(to + 16 * c, w);
          }
        }
        first = false;
        const float nbase = m_use == -INFINITY ? 0.f : -m_use;
        const uint64_t sc2 = pw_pair(sc, sc), nb2 = pw_pair(nbase, nbase);
        const uint64_t minus1 = pw_pair(-1.f, -1.f);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16], rest[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 e = pw_unpair(pw_fma2(pw_pair(v[32 * c + 2 * i], v[32 * c + 2 * i + 1]), sc2, nb2));
            e.x = pw_exp2(e.x);
            e.y = pw_exp2(e.y);
            sum[i & 1] = pw_add2(sum[i & 1], pw_pair(e.x, e.y));
            float2 h;
            w[i] = P16::high(e, h);
            h = pw_unpair(pw_fma2(pw_pair(h.x, h.y), minus1, pw_pair(e.x, e.y)));
            rest[i] = P16::pack(h.x, h.y);
          }
          tmem_st16(ts + 16 * c, w);
          tmem_st16(ts + 64 + 16 * c, rest);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        const float2 total = pw_unpair(pw_add2(sum[0], sum[1]));
        l = l * alpha + (total.x + total.y);
        ++done;
      }
      // what the output needs of this pair, then the next pair's place, then the wait
      link += it.walk.j0 < it.walk.j1 ? it.walk.j1 - it.walk.j0 + 1 : 0;
      T* og = static_cast<T*>(p.out) +
              ((size_t)(it.q0 + tok) * p.num_heads + it.kvh * p.group + (g - tok * p.group)) * D;
      item += step;
      have = find();
      if (have && !bad) copy_q();
      if (!bad && !__all_sync(kFullMask, pw_wait(&o_full[x], nth & 1, p.wait_limit_ns))) bad = true;
      if (bad) break;
      tc_fence_after();
      // (the issuing warp has had the rows of this pair)
      if (have) copied_q();
      if (cluster == 1) {
        if (active > 0) {
          const float inv = 1.f / l;  // a row whose every logit is -inf: 0 / 0, as the formula has it
          // 64 dims at a time through the warp's 4 KB (16-byte chunk k of row r at k ^ (r & 7)),
          // so that a store covers whole lines: a row to a lane, each store touched 32
          // lines and the pair's stores kept the memory pipe for 4000 cycles
          unsigned char* stage = sm + S::kOutOff + warp * 4096;
          const uint64_t mine = reinterpret_cast<uint64_t>(og);
#pragma unroll 1
          for (int half = 0; half < CB; ++half) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t w[32];
              tmem_ld32(to + 64 * half + 32 * c, w);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 4; ++i)
                *reinterpret_cast<uint4*>(stage + lane * 128 + (((4 * c + i) ^ (lane & 7)) << 4)) =
                    make_uint4(P16::pack(__uint_as_float(w[8 * i]) * inv, __uint_as_float(w[8 * i + 1]) * inv),
                               P16::pack(__uint_as_float(w[8 * i + 2]) * inv, __uint_as_float(w[8 * i + 3]) * inv),
                               P16::pack(__uint_as_float(w[8 * i + 4]) * inv, __uint_as_float(w[8 * i + 5]) * inv),
                               P16::pack(__uint_as_float(w[8 * i + 6]) * inv, __uint_as_float(w[8 * i + 7]) * inv));
            }
            __syncwarp();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int rr = 4 * k + (lane >> 3), ch = lane & 7;
              const uint64_t row = __shfl_sync(kFullMask, mine, rr);
              if (32 * (warp & 3) + rr < active)
                reinterpret_cast<uint4*>(row)[8 * half + ch] =
                    *reinterpret_cast<const uint4*>(stage + rr * 128 + ((ch ^ (rr & 7)) << 4));
            }
            __syncwarp();
          }
        }
        tc_fence_before();
      } else {
        // A cluster has one pair only. This part's O and (m, l) go into shared memory, in
        // place of Q, K and V, once every MMA of both A and B, and so every copy that one
        // reads, is over.
        if (!__all_sync(kFullMask, pw_wait(&o_full[x ^ 1], nth & 1, p.wait_limit_ns))) {
          bad = true;
          break;
        }
        float* so = reinterpret_cast<float*>(sm) + (size_t)(x * kPwRows + r) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[32];
          if (!first) {
            tmem_ld32(to + 32 * c, w);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = 0u;
          }
          // 16-byte chunk k of the row at k ^ (r & 7): neighbouring rows' chunks fall into different banks
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(so + 4 * ((8 * c + i) ^ (r & 7))) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        }
        reinterpret_cast<float2*>(sm + S::kJoinMl)[x * kPwRows + r] = make_float2(m_use, l);
      }
      ++nth;
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }

  // ---- a cluster joins its parts: each CTA its share of the rows --------------------------
  if (cluster > 1) {
    pw_cluster_barrier();
    PwScan scan;
    scan.look(p, item0, step, items, false);
    if (scan.mask != 0u) {
      PwItem it;
      it.load(p, item0, rank);
      const int share = 2 * kPwRows / cluster;
      const uint32_t base = smem_u32(sm);
      for (int e = tid; e < share * (D / 4); e += kPwThreads) {
        const int rr = (int)rank * share + e / (D / 4), k = e % (D / 4);
        const int g = it.row0 + rr;
        if (g >= it.rows) continue;
        float2 ml[kPwMaxCluster];
        float4 a[kPwMaxCluster];
#pragma unroll
        for (int c = 0; c < kPwMaxCluster; ++c) {
          ml[c] = make_float2(-INFINITY, 0.f);
          a[c] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c < cluster) {
            ml[c] = pw_remote_f2(pw_remote(base + S::kJoinMl + rr * 8, c));
            a[c] = pw_remote_f4(pw_remote(base + (uint32_t)rr * D * 4 + 16 * (k ^ (rr & 7)), c));
          }
        }
        float M = ml[0].x;
#pragma unroll
        for (int c = 1; c < kPwMaxCluster; ++c) M = fmaxf(M, ml[c].x);
        const float nb = M == -INFINITY ? 0.f : M;
        float lt = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < kPwMaxCluster; ++c) {
          const float f = exp2f(ml[c].x - nb);
          lt += ml[c].y * f;
          o[0] = fmaf(a[c].x, f, o[0]), o[1] = fmaf(a[c].y, f, o[1]);
          o[2] = fmaf(a[c].z, f, o[2]), o[3] = fmaf(a[c].w, f, o[3]);
        }
        const float inv = 1.f / lt;
        const int t = p.by_group.of(g), j = g - t * p.group;
        T* og = static_cast<T*>(p.out) + ((size_t)(it.q0 + t) * p.num_heads + it.kvh * p.group + j) * D + 4 * k;
        *reinterpret_cast<uint2*>(og) =
            make_uint2(P16::pack(o[0] * inv, o[1] * inv), P16::pack(o[2] * inv, o[3] * inv));
      }
    }
    pw_cluster_barrier();  // no CTA leaves while another reads its shared memory
  }

  // ---- tear-down: boxes have landed, MMAs have completed (bounded drains above) ------------
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, kPwTmemCols);
  }
}

using PrefillWindowLauncher = cudaError_t (*)(const PrefillWindowParams&, const void*, const void*, int, cudaStream_t);
PrefillWindowLauncher prefill_window_launcher(int is_bf16, int head_dim);  // prefill_window.cu

}  // namespace pkv
