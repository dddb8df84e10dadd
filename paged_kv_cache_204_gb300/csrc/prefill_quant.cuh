// Prefill over quantised paged caches (sm_103a): causal attention of each sequence's newest
// tokens over e4m3 or q4_0 pools.
//
// Work: the queries of a sequence against one kv head are n x group rows, row m = i * group + j
// for new token i and the kv head's j-th query head, taken in pairs of tiles (A, B) of 128 rows.
// A pair walks the K/V tiles of 128 tokens up to its last query's. On the fifth-generation tensor
// cores S = Q K^T and O += P V accumulate in fp32 in tensor memory; a softmax warpgroup of its own
// serves each of A and B, a row to a thread. The operands are binary16 whatever the queries' type
// (11 significant bits for 8, and bfloat16 queries are exact in it once a power of two of their
// row's own is taken out): a copying warp brings a tile's bytes into shared memory, block by block,
// and four warps turn them, a row to a thread, into the operand's values: e4m3 codes exactly (the
// pool's scale multiplies 32-bit sums), q4_0 values d (q - 8) with one rounding. A tile's V and
// the next one's K, which the MMAs of one step need together, are a link of a chain of two buffers.
//
// Where a pair has one tile only, B takes every other K/V tile of A's rows, so that one tile's
// softmax runs under the other's MMAs there too, and A's warps join the two.
//
// Split: the pairs of all sequences and kv heads are laid end to end, each as long as its walk and
// a start, and every CTA takes an equal stretch (the grid has one to an SM, fewer where the whole
// is short). A pair that a border cuts leaves partial results in the workspace, and the last of its
// CTAs to get there joins them (log-sum-exp).
#pragma once

#include <type_traits>

#include "prefill_quant.h"
#include "prefill_window.cuh"

namespace pkv {

constexpr int kPqThreads = 512;   // 2 softmax warpgroups; MMA warps of A and B, copying warp; 4 converting warps
constexpr int kPqMaxCtas = 152;
// Registers of a thread after the split, which the launch's 128 add up to: softmax, MMA and copy, conversion.
constexpr int kPqSoftRegs = 176, kPqIssueRegs = 64, kPqConvertRegs = 96;
static_assert(2 * kPqSoftRegs + kPqIssueRegs + kPqConvertRegs == 4 * 128, "no more than the launch has");
constexpr int kPqStart = 256;     // a pair's start and end, as tokens of its walk
constexpr int kPqMinTokens = 512; // a CTA's stretch is no shorter

// Cost of what a CTA does, in tokens x group.
using PqCost = long long;

struct PqParams {
  void* out;
  const void* q;
  const unsigned char *k_cache, *v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* query_start;
  float scale_log2;  // |scale| k_scale log2(e), above 0
  float v_scale;
  uint32_t flip;     // sign bits of a pair of query elements for a negative scale, else 0
  int zero_scale;    // scale 0: rows have equal weights, their exponents left alone
  int num_seqs, num_heads, num_kv_heads, group, block_size, block_bits, max_blocks_per_seq, num_blocks, max_query_len;
  PwDivisor by_group;
  int32_t* counter;  // [kPqMaxCtas]
  float2* part_ml;   // [2 kPqMaxCtas][256]
  float4* part_o;    // [2 kPqMaxCtas][D / 4][256]
  int32_t* dev_err;
  uint64_t wait_limit_ns;
};

enum class PqFormat { kQ4, kFp8 };

template <PqFormat F, int D>
struct PqShape {
  static constexpr int kCB = D / 64;
  static constexpr int kColBlock = 128 * 128;
  static constexpr int kTile = kCB * kColBlock;                      // a Q, K or V operand tile
  static constexpr int kRow = F == PqFormat::kQ4 ? D / 16 * 9 : D;   // bytes of a cache row
  static constexpr int kRaw = 128 * kRow;
  static constexpr int kRawStages = D == 64 ? 6 : (F == PqFormat::kQ4 ? 3 : 2);
  static constexpr int kStageOff = 2 * kTile;                        // links: K, V, K, V
  static constexpr int kRawOff = kStageOff + 4 * kTile;
  static constexpr int kBarOff = kRawOff + kRawStages * kRaw;
  static constexpr int kMiscOff = kBarOff + 32 * 8;
  static constexpr int kUsed = kMiscOff + 256 + 512 + 1024;          // + alignment slack
  // more than half of an SM's, so that one CTA has its tensor memory to itself
  static constexpr int kSmemBytes = kUsed > 120 * 1024 ? kUsed : 120 * 1024;
  static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
  static_assert(kRaw % 16 == 0 && kTile % 1024 == 0, "alignment of copies and operands");
};

// A sequence's place in the batch; live: it has queries, and its lengths are in range.
struct PqSeq {
  int L, n, q0;
  bool valid, live;
  __device__ __forceinline__ void load(const PqParams& p, int s) {
    L = __ldg(p.context_lens + s);
    q0 = __ldg(p.query_start + s);
    n = __ldg(p.query_start + s + 1) - q0;
    valid = L >= 0 && L <= p.max_blocks_per_seq * p.block_size && n >= 0 && n <= L && n <= p.max_query_len;
    live = valid && n > 0;
  }
  __device__ __forceinline__ int pairs(int group) const { return (int)(((int64_t)n * group + 255) / 256); }
  // cost of the first k of its pairs (per kv head)
  __device__ __forceinline__ PqCost before(int k, int group) const {
    const PqCost each = (PqCost)group * (kPqStart + L - n), rows = (PqCost)n * group;
    return k * each + (256 * (PqCost)k < rows ? 128 * (PqCost)k * (k + 1) : 128 * (PqCost)k * (k - 1) + rows);
  }
};

// The whole batch's cost and how CTAs share it.
struct PqShare {
  PqCost whole;
  int ctas;
  __device__ __forceinline__ PqCost begin(int c) const { return whole / ctas * c + whole % ctas * c / ctas; }
  __device__ __forceinline__ int of(PqCost y) const {
    int c = min(ctas - 1, (int)(y / (whole / ctas + 1)));
    while (begin(c + 1) <= y) ++c;
    return c;
  }
};

// A CTA's walk over the pairs (or parts of them) in its stretch; every role makes it for itself.
struct PqItem {
  PqSeq seq;
  int s, kvh, pair, np;
  PqCost at, cost, lo, hi;  // of the pair: its place and length; the CTA's stretch
  int row0, rows;           // first row; rows of the kv head's queries
  int active;               // of the pair
  int end_a, end_b;         // tokens that the last queries of A and B see
  int j0, j1;               // K/V tiles of this part
  bool dual;                // one tile of rows: A and B take K/V tiles in turn

  __device__ __forceinline__ bool done() const { return at >= hi; }
  __device__ __forceinline__ bool whole() const { return lo <= at && at + cost <= hi; }
  __device__ __forceinline__ int end() const { return dual ? end_a : end_b; }
  __device__ __forceinline__ int active_of(int x) const {
    return dual ? active : max(min(active - 128 * x, 128), 0);
  }
  // Queries of tile x (A: 0, B: 1) take part in K/V tile j.
  __device__ __forceinline__ bool sees(int x, int j) const {
    if (dual) return ((j - j0) & 1) == x;
    return x ? j * 128 < end_b : j * 128 < end_a;
  }
  __device__ __forceinline__ void shape(const PqParams& p) {
    const PqCost c0 = seq.before(pair, p.group);
    cost = seq.before(pair + 1, p.group) - c0;
    rows = seq.n * p.group;
    row0 = pair * 256;
    active = min(rows - row0, 256);
    dual = active <= 128;
    const int base = seq.L - seq.n + 1;
    end_a = base + p.by_group.of(row0 + min(active, 128) - 1);
    end_b = dual ? 0 : base + p.by_group.of(row0 + active - 1);
    const int tiles = (end() + 127) / 128;
    const PqCost a = max(lo - at, (PqCost)0), b = min(hi - at, cost);
    j0 = a == 0 ? 0 : (int)(tiles * a / cost);
    j1 = b == cost ? tiles : (int)(tiles * b / cost);
  }
  __device__ __forceinline__ void next(const PqParams& p) {
    at += cost;
    if (at >= hi) return;
    if (++pair == np) {
      pair = 0;
      if (++kvh == p.num_kv_heads) {
        kvh = 0;
        // the next sequence with queries: there is one, the stretch not being at its end
        for (++s; s < p.num_seqs; s += 32) {
          PqSeq q;
          q.live = false;
          const int mine = s + (int)(threadIdx.x & 31);
          if (mine < p.num_seqs) q.load(p, mine);
          const uint32_t some = __ballot_sync(kFullMask, q.live);
          if (some != 0u) {
            s += __ffs(some) - 1;
            break;
          }
        }
        if (s >= p.num_seqs) {
          at = hi;
          return;
        }
        seq.load(p, s);
        np = seq.pairs(p.group);
      }
    }
    shape(p);
  }
};

// Where a CTA's stretch begins, worked out once by the whole CTA.
struct PqBegin {
  PqShare share;
  PqCost at, lo, hi;
  int s, kvh, pair;
};

__device__ __forceinline__ PqCost pq_warp_scan(PqCost v) {  // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const PqCost u = __shfl_up_sync(kFullMask, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// 8 bytes of codes as 16 values d (q - 8): low halves to lo, high halves to hi. A code placed
// under the exponent of 1024 (low halves, last place 1) or of 64 (high halves, last place 1/16)
// is a binary16 number that exceeds it by that constant.
__device__ __forceinline__ void pq_from_q4(uint32_t w0, uint32_t w1, __half2 d, uint4& lo, uint4& hi) {
  const __half2 k1032 = __half2half2(__ushort_as_half(0x6408)), k72 = __half2half2(__ushort_as_half(0x5480));
  auto part = [&](uint32_t w, uint32_t exponent, uint32_t sel, __half2 minus) {
    const uint32_t u = __byte_perm(w, exponent, sel);
    __half2 h;
    memcpy(&h, &u, 4);
    h = __hmul2(__hsub2(h, minus), d);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
  };
  const uint32_t l0 = w0 & 0x0f0f0f0fu, l1 = w1 & 0x0f0f0f0fu, h0 = w0 & 0xf0f0f0f0u, h1 = w1 & 0xf0f0f0f0u;
  lo = make_uint4(part(l0, 0x64646464u, 0x4140, k1032), part(l0, 0x64646464u, 0x4342, k1032),
                  part(l1, 0x64646464u, 0x4140, k1032), part(l1, 0x64646464u, 0x4342, k1032));
  hi = make_uint4(part(h0, 0x54545454u, 0x4140, k72), part(h0, 0x54545454u, 0x4342, k72),
                  part(h1, 0x54545454u, 0x4140, k72), part(h1, 0x54545454u, 0x4342, k72));
}

__device__ __forceinline__ uint32_t pq_from_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}

// Row r of a tile: its bytes at `row` become the operand's values (zeros where !held) in the
// swizzled tile at `tile`.
template <PqFormat F, int D>
__device__ __forceinline__ void pq_convert_row(const unsigned char* row, unsigned char* tile, int r, bool held) {
  unsigned char* at = tile + r * 128;
  const uint32_t swz = (r & 7) << 4;
  // values 8 c .. 8 c + 7 of the row
  auto put = [&](int c, uint4 v) {
    *reinterpret_cast<uint4*>(at + (c >> 3) * (128 * 128) + ((((uint32_t)c & 7) << 4) ^ swz)) = v;
  };
  if (!held) {
#pragma unroll
    for (int c = 0; c < D / 8; ++c) put(c, make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  if constexpr (F == PqFormat::kQ4) {
    // (rows start on 8 bytes at head_dim 128, on 4 at 64)
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      const __half2 d = __half2half2(*reinterpret_cast<const __half*>(row + 2 * b));
      uint32_t w[4];
      const unsigned char* codes = row + D / 16 + 16 * b;
      if constexpr (D == 128) {
        const uint2 x = *reinterpret_cast<const uint2*>(codes), y = *reinterpret_cast<const uint2*>(codes + 8);
        w[0] = x.x, w[1] = x.y, w[2] = y.x, w[3] = y.y;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const uint32_t*>(codes)[i];
      }
      uint4 lo, hi;
      pq_from_q4(w[0], w[1], d, lo, hi);
      put(4 * b, lo);
      put(4 * b + 2, hi);
      pq_from_q4(w[2], w[3], d, lo, hi);
      put(4 * b + 1, lo);
      put(4 * b + 3, hi);
    }
  } else {
    // lanes take a row's 16-byte chunks in orders of their own, so that eight lanes' chunks fall
    // into different banks
    const int turn = D == 128 ? r & 7 : (r >> 1) & 3;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int c = i ^ turn;
      const uint4 x = *reinterpret_cast<const uint4*>(row + 16 * c);
      put(2 * c, make_uint4(pq_from_e4m3x2(x.x & 0xffffu), pq_from_e4m3x2(x.x >> 16), pq_from_e4m3x2(x.y & 0xffffu),
                            pq_from_e4m3x2(x.y >> 16)));
      put(2 * c + 1, make_uint4(pq_from_e4m3x2(x.z & 0xffffu), pq_from_e4m3x2(x.z >> 16),
                                pq_from_e4m3x2(x.w & 0xffffu), pq_from_e4m3x2(x.w >> 16)));
    }
  }
}

__device__ __forceinline__ void pq_barrier(int id, int threads) {
  asm volatile("barrier.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Four lanes hand round 16-byte pieces: v[i] of lane l becomes v[l % 4] of lane (l & ~3) + i.
__device__ __forceinline__ void pq_transpose(uint4 (&v)[4]) {
  const int lane = threadIdx.x & 31;
  auto swap = [&](uint4& a, uint4& b, int bit) {  // a: index bit clear, b: set
    const bool up = lane & bit;
    uint4 send = up ? a : b;
    send.x = __shfl_xor_sync(kFullMask, send.x, bit);
    send.y = __shfl_xor_sync(kFullMask, send.y, bit);
    send.z = __shfl_xor_sync(kFullMask, send.z, bit);
    send.w = __shfl_xor_sync(kFullMask, send.w, bit);
    if (up)
      a = send;
    else
      b = send;
  };
  swap(v[0], v[1], 1);
  swap(v[2], v[3], 1);
  swap(v[0], v[2], 2);
  swap(v[1], v[3], 2);
}

template <typename T, PqFormat F, int D>
__global__ void __launch_bounds__(kPqThreads, 1) pa_prefill_quant_kernel(const __grid_constant__ PqParams p) {
  using S = PqShape<F, D>;
  using Out = PwPack<T>;
  using P16 = PwPack<__half>;
  constexpr int CB = S::kCB, NR = S::kRawStages;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  // Every barrier's phases follow one another in the order of the work, and nobody who waits for
  // a phase can fall two behind.
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBarOff);
  uint64_t* raw_full = bars;                // [NR] a tile's bytes landed
  uint64_t* raw_empty = bars + NR;          // [NR] and were converted (an arrival per converting warp)
  uint64_t* ready = bars + 2 * NR;          // [2] a link's operands are in place (likewise)
  uint64_t* empty = ready + 2;              // [2] the MMAs are done with it (A's and B's: two arrivals)
  uint64_t* s_full = ready + 4;             // [A, B] S computed
  uint64_t* p_full = ready + 6;             // [A, B] P written (one arrival per softmax warp)
  uint64_t* q_full = ready + 8;             // [A, B] query rows in place (likewise)
  uint64_t* o_full = ready + 10;            // [A, B] the part's last O computed
  uint64_t* turn = ready + 12;              // [A, B] the other's MMAs of a link are issued
  uint64_t* shared_q = ready + 14;          // A's query rows in place for B too (an arrival per warp of A)
  uint64_t* drained = ready + 15;           // every MMA of the CTA done (two arrivals)
  unsigned char* misc = sm + S::kMiscOff;
  uint32_t* slot = reinterpret_cast<uint32_t*>(misc);           // tensor-memory address
  volatile int* last_flag = reinterpret_cast<int*>(misc + 4);
  uint32_t* held_blocks = reinterpret_cast<uint32_t*>(misc + 8);  // [NR] blocks of a raw tile that were copied
  PqBegin* begin = reinterpret_cast<PqBegin*>(misc + 64);
  float* shared_sc = reinterpret_cast<float*>(misc + 256);        // [128] factors of A's rows for B
  static_assert(sizeof(PqBegin) <= 128 && 8 + 4 * NR <= 64 && (2 * NR + 16) * 8 <= 32 * 8, "room");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group;

  // ---- the CTA's stretch of the whole -----------------------------------------
  {
    PqCost* sums = reinterpret_cast<PqCost*>(sm);  // [16], before anything else is there
    auto cost_of = [&](int s) {
      if (s >= p.num_seqs) return (PqCost)0;
      PqSeq q;
      q.load(p, s);
      if (!q.valid && blockIdx.x == 0) set_err(p.dev_err, PKV_DEV_ERR_CONTEXT_LEN);
      return q.live ? q.before(q.pairs(G), G) * p.num_kv_heads : (PqCost)0;
    };
    PqCost mine = 0;
    for (int s = tid; s < p.num_seqs; s += kPqThreads) mine += cost_of(s);
    const PqCost w = pq_warp_scan(mine);
    if (lane == 31) sums[warp] = w;
    __syncthreads();
    PqShare share;
    share.whole = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) share.whole += sums[i];
    const PqCost most = share.whole / ((PqCost)G * kPqMinTokens);
    share.ctas = (int)max(min(most, (PqCost)gridDim.x), (PqCost)1);
    if (share.whole == 0 || (int)blockIdx.x >= share.ctas) return;
    const PqCost lo = share.begin(blockIdx.x);
    PqCost base = 0;
    for (int s0 = 0; s0 < p.num_seqs; s0 += kPqThreads) {
      __syncthreads();
      const PqCost own = p.num_seqs <= kPqThreads ? mine : cost_of(s0 + tid);
      const PqCost upto = pq_warp_scan(own);
      if (lane == 31) sums[warp] = upto;
      __syncthreads();
      PqCost before = base;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if (i < warp) before += sums[i];
        base += sums[i];
      }
      before += upto - own;
      if (own > 0 && before <= lo && lo < before + own) {
        PqSeq q;
        q.load(p, s0 + tid);
        const int np = q.pairs(G);
        const PqCost head = q.before(np, G);
        begin->s = s0 + tid;
        begin->kvh = (int)((lo - before) / head);
        const PqCost y = (lo - before) % head;
        int a = 0, b = np;  // the pair that holds y: before(a) <= y < before(b)
        while (b - a > 1) {
          const int mid = (a + b) / 2;
          if (q.before(mid, G) <= y)
            a = mid;
          else
            b = mid;
        }
        begin->pair = a;
        begin->at = lo - y + q.before(a, G);
        begin->lo = lo;
        begin->hi = share.begin(blockIdx.x + 1);
        begin->share = share;
      }
      if (base > lo) break;  // (uniform)
    }
  }

  // ---- set-up: barriers, tensor memory ----------------------------------------
  if (tid == 0) {
    for (int i = 0; i < NR; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ready[i], 4);
      mbar_init(&empty[i], 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&q_full[i], 4);
      mbar_init(&o_full[i], 1);
      mbar_init(&turn[i], 1);
    }
    mbar_init(shared_q, 4);
    mbar_init(drained, 2);
    mbar_init_fence();
  }
  if (warp == 8) tmem_alloc(slot, kPwTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *slot;
  bool bad = false;  // a wait ran out
  PqItem it;
  it.s = begin->s, it.kvh = begin->kvh, it.pair = begin->pair;
  it.at = begin->at, it.lo = begin->lo, it.hi = begin->hi;
  it.seq.load(p, it.s);
  it.np = it.seq.pairs(G);
  it.shape(p);

  // (the registers of a warpgroup change hands for all its warps at once)
  if (warp >= 12) {
    // ---- conversion: V of one tile, K of the next, into the link's operands -----------------
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPqConvertRegs));
    const int r = tid & 127, block = r >> p.block_bits;
    uint32_t link = 0, raw = 0;  // links and tiles so far
    int stage = 0;
    uint32_t phase = 0;
    for (; !bad && !it.done(); it.next(p)) {
      const int end = it.end();
      for (int j = it.j0; j <= it.j1 && it.j0 < it.j1 && !bad; ++j, ++link) {
        const uint32_t c = link & 1;
        if (link >= 2 && !__all_sync(kFullMask, pw_wait(&empty[c], ((link >> 1) + 1) & 1, p.wait_limit_ns))) {
          bad = true;
          break;
        }
#pragma unroll 1
        for (int which = 1; which >= 0; --which) {  // V of tile j - 1, K of tile j
          const int t = j - which;
          if (t < it.j0 || t >= it.j1) continue;
          if (!__all_sync(kFullMask, pw_wait(&raw_full[stage], phase, p.wait_limit_ns))) {
            bad = true;
            break;
          }
          const bool held = t * 128 + r < end && ((held_blocks[stage] >> block) & 1u);
          pq_convert_row<F, D>(sm + S::kRawOff + stage * S::kRaw + r * S::kRow,
                               sm + S::kStageOff + (2 * c + which) * S::kTile, r, held);
          __syncwarp();
          if (lane == 0) mbar_arrive(&raw_empty[stage]);
          ++raw;
          if (++stage == NR) stage = 0, phase ^= 1;
        }
        fence_async_smem();
        __syncwarp();
        if (!bad && lane == 0) mbar_arrive(&ready[c]);
      }
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPqIssueRegs));
    if (warp == 9) {
    // ---- copies: a tile's cache blocks, one to a lane -----------------------------------------
    const int per_tile = 128 >> p.block_bits;  // <= 16 blocks
    const uint32_t bytes = (uint32_t)p.block_size * S::kRow;
    uint32_t raw = 0;
    int stage = 0;
    uint32_t phase = 1;  // of raw_empty, from the second round on
    for (; !bad && !it.done(); it.next(p)) {
      const int32_t* bt = p.block_tables + (size_t)it.s * p.max_blocks_per_seq;
      const int blocks = (it.end() + p.block_size - 1) >> p.block_bits;
      auto fetch = [&](int j) {
        const int b = j * per_tile + lane;
        return j < it.j1 && lane < per_tile && b < blocks ? __ldg(bt + b) : -2;  // -2: none there
      };
      int id = fetch(it.j0), id_v = -2;
      for (int j = it.j0; j <= it.j1 && it.j0 < it.j1 && !bad; ++j) {
        if (id != -2 && (id < 0 || id >= p.num_blocks)) {
          set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
          id = -2;
        }
        const int id_next = fetch(j + 1);
#pragma unroll
        for (int which = 1; which >= 0; --which) {  // V of tile j - 1, K of tile j
          const int t = j - which;
          if (t < it.j0 || t >= it.j1 || bad) continue;
          if (raw >= NR && !__all_sync(kFullMask, pw_wait(&raw_empty[stage], phase, p.wait_limit_ns))) {
            bad = true;
            break;
          }
          const int b = which ? id_v : id;
          const uint32_t some = __ballot_sync(kFullMask, b != -2);
          if (lane == 0) {
            held_blocks[stage] = some;
            mbar_arrive_expect_tx(&raw_full[stage], __popc(some) * bytes);
          }
          __syncwarp();
          if (b != -2)
            bulk_copy_g2s(sm + S::kRawOff + stage * S::kRaw + lane * bytes,
                          (which ? p.v_cache : p.k_cache) + ((size_t)b * p.num_kv_heads + it.kvh) * bytes, bytes,
                          &raw_full[stage]);
          ++raw;
          if (++stage == NR) stage = 0, phase ^= 1;
        }
        id_v = id;
        id = id_next;
      }
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    // the last copies must land before the CTA can leave
    if (lane == 0)
      for (uint32_t c = raw >= NR ? raw - NR : 0; c < raw; ++c)
        mbar_wait_bounded(&raw_full[c % NR], (c / NR) & 1, kDrainLimitNs);
    __syncwarp();
    } else if (warp != 10) {
    // ---- MMA issue, a warp for each of A and B ------------------------------------------
    // Per link: O += P V of one tile, S of the next. With two tiles of rows at head_dim 128 A and B
    // take turns, so that one's softmax runs under the other's MMAs. MMAs of one thread complete
    // in order, so S may take the place of a P that the MMA before it reads, and "S done" says
    // that O holds every earlier tile.
    const int x = warp == 8 ? 0 : 1;
    constexpr uint32_t id_s = mma_idesc_f16(128, 128, 0, 0);
    constexpr uint32_t id_o = mma_idesc_f16(128, D, 0, 1);
    const uint32_t tb = __shfl_sync(kFullMask, tbase, 0);
    const uint32_t sb = __shfl_sync(kFullMask, smem_u32(sm), 0);
    // of a descriptor only the start address in its low word moves
    const uint32_t kd = (uint32_t)smem_desc_sw128(sb + S::kStageOff, 16, 1024);
    const uint32_t vd = (uint32_t)smem_desc_sw128(sb + S::kStageOff + S::kTile, S::kColBlock, 1024);
    const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);  // K-major and MN-major alike
    uint32_t link = 0, nth = 0, done = 0, turns = 0;  // links, parts, P's and links in turn so far
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      const bool ok = __all_sync(kFullMask, pw_wait(bar, parity, p.wait_limit_ns));
      tc_fence_after();
      return ok;
    };
    for (; !bad && !it.done(); it.next(p)) {
      const int tiles = it.j1 - it.j0;
      const bool in_turn = D == 128 && !it.dual;
      const uint32_t qd = (uint32_t)smem_desc_sw128(sb + (it.dual ? 0 : x) * S::kTile, 16, 1024);
      bool seen = false, opened = false;  // the tile at hand is seen, O holds something
      bad = !wait(&q_full[x], nth & 1);
      for (int i = tiles > 0 ? 0 : 1; i <= tiles && !bad; ++i, ++link) {  // O of tile i - 1, S of tile i
        const uint32_t c = link & 1;
        const bool next = i < tiles && it.sees(x, it.j0 + i);
        bad = !wait(&ready[c], (link >> 1) & 1);
        if (in_turn && !bad && (x == 1 || turns > 0)) bad = !wait(&turn[x], (turns + (x ^ 1)) & 1);
        // (a part's first P comes from warps that have read the O of the part before)
        if (!bad && seen) bad = !wait(&p_full[x], done++ & 1);
        if (!bad && elect_one()) {
          if (seen) {
            const uint32_t vb = vd + (c * (2 * S::kTile) >> 4);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              pw_mma_ts(tb + 256 + 128 * x, tb + 128 * x + 8 * ks, vb + (ks * 2048 >> 4), hi, id_o,
                        (ks > 0 || opened) ? 1u : 0u);
          }
          if (next) {
            const uint32_t kb = kd + (c * (2 * S::kTile) >> 4);
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
              const uint32_t off = ((ks >> 2) * S::kColBlock + (ks & 3) * 32) >> 4;
              pw_mma_ss(tb + 128 * x, qd + off, kb + off, hi, id_s, ks > 0);
            }
            mma_commit(&s_full[x]);
          } else {
            mma_commit(&empty[c]);  // (with an S the softmax sees to that)
          }
          if (in_turn) mbar_arrive(&turn[x ^ 1]);
        }
        __syncwarp();
        turns += in_turn;
        opened |= seen;
        seen = next;
      }
      if (!bad && elect_one()) mma_commit(&o_full[x]);
      __syncwarp();
      ++nth;
    }
    // nothing may be torn down before the last MMA, after a timeout neither
    if (elect_one()) mma_commit(drained);
    __syncwarp();
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    mbar_wait_bounded(drained, 0, kDrainLimitNs);
    __syncwarp();
    }
  } else {
    // ---- softmax: warpgroup x serves query tile x, a row to a thread --------------------
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPqSoftRegs));
    const int x = warp >> 2, w4 = warp & 3, r = tid & 127;
    const uint32_t ts = tbase + ((uint32_t)(32 * w4) << 16) + 128 * x;  // S of this warp's lanes
    const uint32_t to = ts + 256;                                      // and O
    uint32_t done = 0, nth = 0, link = 0, duals = 0;  // tiles, parts, links and parts of one tile so far
    constexpr int kLoads = 8 * CB;         // 16-byte loads of a lane for its warp's query rows
    uint4 qv[kLoads];
    float sc = 0.f;                        // this row's factor from S to logits in powers of two

    // The part's query rows: 8 lanes to a row, 4 rows at a time (a row of 256 bytes in two).
    auto load_q = [&]() {
      const T* q = static_cast<const T*>(p.q);
      const int active = it.active_of(x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = 32 * w4 + 4 * i + (lane >> 3);
        const bool in = rr < active;
        const int g = it.row0 + (it.dual ? 0 : x * 128) + rr, t = in ? p.by_group.of(g) : 0, j = in ? g - t * G : 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            q + ((size_t)(it.seq.q0 + t) * p.num_heads + it.kvh * G + j) * D) + (lane & 7);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) qv[i * CB + cb] = in ? __ldg(src + 8 * cb) : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    // The next part's query rows on their way to L2 while this one's last MMAs run (a hint only).
    auto prefetch_q = [&]() {
      if (it.dual && x == 1) return;
      const int rr = 32 * w4 + lane;
      if (rr >= it.active_of(x)) return;
      const int g = it.row0 + (it.dual ? 0 : x * 128) + rr, t = p.by_group.of(g);
      const T* src = static_cast<const T*>(p.q) +
                     ((size_t)(it.seq.q0 + t) * p.num_heads + it.kvh * G + g - t * G) * D;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64 * cb));
    };
    // Into shared memory as binary16. A bfloat16 row is divided by 2^e so that its largest value lies in
    // [2^14, 2^15): what exceeds 2^-28 of that keeps its 8 bits.
    auto store_q = [&]() {
      float mine = p.scale_log2;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int rr = 32 * w4 + 4 * i + (lane >> 3);
        if constexpr (kBf16) {
          uint32_t top = 0u;  // largest exponent bits of the row
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            const uint4 v = qv[i * CB + cb];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7f80u, (w[k] >> 16) & 0x7f80u));
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(kFullMask, top, o));
          // 2^(14 - k) for an exponent of k, at most 2^126
          const int k = max((int)(top >> 7) - 127, -112);
          const float by = top == 0u ? 1.f : __uint_as_float((uint32_t)(14 - k + 127) << 23);
          const float back = top == 0u ? 1.f : __uint_as_float((uint32_t)(k - 14 + 127) << 23);
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            float f[8];
            Chunk<__nv_bfloat16>::widen(qv[i * CB + cb], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= by;
            qv[i * CB + cb] = Chunk<__half>::narrow(f);
          }
          const float theirs = __shfl_sync(kFullMask, back, (lane & 3) * 8);
          if (!p.zero_scale && i == lane >> 2) mine = fmaxf(p.scale_log2 * theirs, 1.401298464e-45f);
        }
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          const uint4 v = qv[i * CB + cb];
          *reinterpret_cast<uint4*>(sm + x * S::kTile + cb * S::kColBlock + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4)) =
              make_uint4(v.x ^ p.flip, v.y ^ p.flip, v.z ^ p.flip, v.w ^ p.flip);
        }
      }
      sc = mine;
    };
    auto place_q = [&]() {
      if (it.dual && x == 1) return;  // A's rows serve both
      load_q();
      store_q();
      if (it.dual) shared_sc[r] = sc;
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&q_full[x]);
        if (it.dual) mbar_arrive(shared_q);
      }
    };
    place_q();
    while (!it.done()) {
      const bool dual = it.dual, whole = it.whole();
      if (dual && x == 1) {
        // (A's warps put the next rows in place behind this part's join only, so that the phase
        // waited for is never more than one away)
        if (!bad && !__all_sync(kFullMask, pw_wait(shared_q, duals & 1, p.wait_limit_ns))) bad = true;
        sc = shared_sc[r];
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[1]);
        ++duals;
      }
      const int active = it.active_of(x);
      const bool idle = 32 * w4 >= active;  // no row of this warp is a query's
      const int g = it.row0 + (dual ? 0 : x * 128) + min(r, max(active - 1, 0));
      const int tok = p.by_group.of(g);
      const int pos = it.seq.L - it.seq.n + tok;
      const int j0 = it.j0, j1 = it.j1;
      float m_use = -INFINITY, l = 0.f;
      bool first = true;
      for (int j = j0; j < j1 && !bad; ++j) {
        if (!it.sees(x, j)) continue;
        const int vis = pos - j * 128 + 1;  // tokens of the tile up to the row's own
        if (!__all_sync(kFullMask, pw_wait(&s_full[x], done & 1, p.wait_limit_ns))) {
          bad = true;
          break;
        }
        tc_fence_after();
        // S is the query tile's last MMA that reads its link
        if (w4 == 0 && lane == 0) mbar_arrive(&empty[(link + (j - j0)) & 1]);
        ++done;
        if (idle) {  // (its rows of P, and so of O, may hold anything)
          if (lane == 0) mbar_arrive(&p_full[x]);
          continue;
        }
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, u[c]);
        tmem_wait_ld();
        float* v = reinterpret_cast<float*>(&u[0][0]);
        if (__any_sync(kFullMask, vis < 128)) {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const uint32_t see = low_bits(vis - 32 * c);
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
        // the base moves only when the maximum grows by more than kTopLog2: every P stays below 2^kTopLog2,
        // and O and the row sum have the same base. (Logits from kPwFar on are whole numbers, and
        // a base may be off by half their distance: there it is the maximum and moves whenever that does.)
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
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float2 e = pw_unpair(pw_fma2(pw_pair(v[32 * c + 2 * i], v[32 * c + 2 * i + 1]), sc2, nb2));
            e.x = pw_exp2(e.x);
            e.y = pw_exp2(e.y);
            sum[i & 1] = pw_add2(sum[i & 1], pw_pair(e.x, e.y));
            w[i] = P16::pack(e.x, e.y);
          }
          tmem_st16(ts + 16 * c, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        const float2 total = pw_unpair(pw_add2(sum[0], sum[1]));
        l = l * alpha + (total.x + total.y);
      }
      // what the output needs of this part, then the next one's place and loads, then the wait
      link += j0 < j1 ? j1 - j0 + 1 : 0;
      T* og = static_cast<T*>(p.out) +
              ((size_t)(it.seq.q0 + tok) * p.num_heads + it.kvh * G + (g - tok * G)) * D;
      const PqCost part_at = it.at, part_end = it.at + it.cost;
      const bool head = it.lo <= it.at;
      it.next(p);
      const bool more = !it.done();
      if (more) prefetch_q();
      if (!bad && !__all_sync(kFullMask, pw_wait(&o_full[x], nth & 1, p.wait_limit_ns))) bad = true;
      tc_fence_after();
      ++nth;
      if (more && !bad && !dual) place_q();

      // 32 dims of this row at a time: O as it is
      auto load_o = [&](int c, uint32_t (&w)[32]) {
        if (first || idle) {
#pragma unroll
          for (int i = 0; i < 32; ++i) w[i] = 0u;
        } else {
          tmem_ld32(to + 32 * c, w);
          tmem_wait_ld();
        }
      };
      // Output of 32 dims (chunk c) of the warp's rows: w holds fp32 values of this row, `inv` its factor.
      uint64_t row_at[4];
      auto rows_of = [&]() {
        const uint64_t mine = reinterpret_cast<uint64_t>(og);
#pragma unroll
        for (int k = 0; k < 4; ++k) row_at[k] = __shfl_sync(kFullMask, mine, (lane & ~3) + k);
      };
      auto put = [&](int c, const uint32_t (&w)[32], float inv) {
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = make_uint4(Out::pack(__uint_as_float(w[8 * i]) * inv, __uint_as_float(w[8 * i + 1]) * inv),
                            Out::pack(__uint_as_float(w[8 * i + 2]) * inv, __uint_as_float(w[8 * i + 3]) * inv),
                            Out::pack(__uint_as_float(w[8 * i + 4]) * inv, __uint_as_float(w[8 * i + 5]) * inv),
                            Out::pack(__uint_as_float(w[8 * i + 6]) * inv, __uint_as_float(w[8 * i + 7]) * inv));
        pq_transpose(v);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (32 * w4 + (lane & ~3) + k < active) reinterpret_cast<uint4*>(row_at[k])[4 * c + (lane & 3)] = v[k];
      };
      // a part of a pair: into the workspace, 16 bytes of 32 rows side by side
      const int my_slot = 2 * blockIdx.x + (head ? 1 : 0);
      auto leave = [&](int c, const uint32_t (&w)[32]) {
        float4* dst = p.part_o + (size_t)my_slot * (D / 4) * 256 + (dual ? 0 : 128 * x) + r;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          dst[(size_t)(8 * c + i) * 256] = make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]),
                                                       __uint_as_float(w[4 * i + 2]), __uint_as_float(w[4 * i + 3]));
      };
      auto leave_ml = [&](float m, float sum) {
        p.part_ml[(size_t)my_slot * 256 + (dual ? 0 : 128 * x) + r] = make_float2(m, sum);
      };
      rows_of();
      if (dual) {
        // B's part of the rows goes to A's warps through the place of B's query rows, 32 dims at a
        // time (16-byte chunk k of row r at k ^ (r & 7)), warp by warp: 4 KB each
        float4* box = reinterpret_cast<float4*>(sm + S::kTile + w4 * 4096) + lane * 8;
        const int bar = 2 + w4;
        if (x == 1) {
          box[0] = make_float4(m_use, l, 0.f, 0.f);
          pq_barrier(bar, 64);
          pq_barrier(bar, 64);
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t w[32];
            load_o(c, w);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              *reinterpret_cast<uint4*>(box + (k ^ (lane & 7))) = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            pq_barrier(bar, 64);
            pq_barrier(bar, 64);
          }
        } else {
          pq_barrier(bar, 64);
          const float4 b = box[0];
          pq_barrier(bar, 64);
          const float M = fmaxf(m_use, b.x), nb = M == -INFINITY ? 0.f : M;
          const float fa = exp2f(m_use - nb), fb = exp2f(b.x - nb);
          const float sum = l * fa + b.y * fb;
          const float inv = p.v_scale / sum;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t w[32];
            load_o(c, w);
            pq_barrier(bar, 64);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float4 o = box[k ^ (lane & 7)];
              w[4 * k] = __float_as_uint(fmaf(o.x, fb, __uint_as_float(w[4 * k]) * fa));
              w[4 * k + 1] = __float_as_uint(fmaf(o.y, fb, __uint_as_float(w[4 * k + 1]) * fa));
              w[4 * k + 2] = __float_as_uint(fmaf(o.z, fb, __uint_as_float(w[4 * k + 2]) * fa));
              w[4 * k + 3] = __float_as_uint(fmaf(o.w, fb, __uint_as_float(w[4 * k + 3]) * fa));
            }
            pq_barrier(bar, 64);
            if (bad || idle) continue;
            if (whole)
              put(c, w, inv);
            else
              leave(c, w);
          }
          if (!whole && !bad && !idle) leave_ml(M, sum);
        }
      } else if (!idle && !bad) {
        const float inv = p.v_scale / l;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[32];
          load_o(c, w);
          if (whole)
            put(c, w, inv);
          else
            leave(c, w);
        }
        if (!whole) leave_ml(m_use, l);
      }
      tc_fence_before();
      if (!whole) {
        // the last of the pair's CTAs joins the parts
        __threadfence();
        const bool lost = barrier_or(1, 256, bad);  // (every warp comes by here, also after a timeout)
        const PqShare share = begin->share;
        const int c0 = share.of(part_at), c1 = share.of(part_end - 1);
        if (tid == 0) {
          int last = 0;
          if (!lost && atomic_add_acq_rel_gpu(p.counter + c0, 1) == c1 - c0) {
            p.counter[c0] = 0;
            last = 1;
          }
          *last_flag = last;
        }
        pq_barrier(1, 256);
        const bool last = *last_flag != 0;
        pq_barrier(1, 256);  // (the flag's next value may come at once)
        if (last && !idle) {
          __threadfence();
          const int row = (dual ? 0 : 128 * x) + r;
          const size_t slot0 = 2 * (size_t)c0 + 1;
          auto slot_of = [&](int c) { return c == c0 ? slot0 : 2 * (size_t)c; };
          float M = -INFINITY;
          for (int c = c0; c <= c1; ++c) M = fmaxf(M, __ldcg(p.part_ml + slot_of(c) * 256 + row).x);
          const float nb = M == -INFINITY ? 0.f : M;
          float sum = 0.f;
          for (int c = c0; c <= c1; ++c) {
            const float2 ml = __ldcg(p.part_ml + slot_of(c) * 256 + row);
            sum += ml.y * exp2f(ml.x - nb);
          }
          const float inv = p.v_scale / sum;
          // (of a single tile's rows A's warps take one half of the dims, B's the other)
          const int from = dual ? x * (D / 64) : 0, upto = dual ? (x + 1) * (D / 64) : D / 32;
#pragma unroll 1
          for (int k = from; k < upto; ++k) {
            float o[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.f;
            for (int c = c0; c <= c1; ++c) {
              const float2 ml = __ldcg(p.part_ml + slot_of(c) * 256 + row);
              if (ml.y == 0.f) continue;  // nothing of the part is visible to the row
              const float f = exp2f(ml.x - nb);
              const float4* src = p.part_o + (slot_of(c) * (D / 4) + 8 * k) * 256 + row;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 a = __ldcg(src + (size_t)i * 256);
                o[4 * i] = fmaf(a.x, f, o[4 * i]), o[4 * i + 1] = fmaf(a.y, f, o[4 * i + 1]);
                o[4 * i + 2] = fmaf(a.z, f, o[4 * i + 2]), o[4 * i + 3] = fmaf(a.w, f, o[4 * i + 3]);
              }
            }
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(o[i]);
            put(k, w, inv);
          }
        }
      }
      if (more && !bad && dual) place_q();
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    __syncwarp();
  }

  // ---- tear-down: copies have landed, MMAs have completed (bounded drains above) ------------
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, kPwTmemCols);
  }
}

}  // namespace pkv
