// Prefill over quantised paged caches (sm_103a): causal attention of each sequence's newest
// tokens over e4m3 or q4_0 pools.
//
// Work: the queries of a sequence against one kv head are n x group rows, row m = i * group + j
// for new token i and the kv head's j-th query head, taken in pairs of tiles (A, B) of 128 rows.
// A pair walks the K/V tiles of 128 tokens up to its last query's. On the fifth-generation tensor
// cores S = Q K^T and O += P V accumulate in fp32 in tensor memory; two softmax warpgroups serve
// each of A and B, half a row to a thread. The operands are binary16 whatever the queries' type
// (11 significant bits for 8, and bfloat16 queries are exact in it once a power of two of their
// row's own is taken out): a copying warp brings a tile's bytes into shared memory, block by block,
// and four warps turn them, a row to a thread, into the operand's values: e4m3 codes exactly (the
// pool's scale multiplies 32-bit sums), q4_0 values d (q - 8) with one rounding, or, K beside binary16 queries, in two
// parts. Doing it once for
// 256 rows costs a sixth of a tile's instructions; the scales of q4_0 differ by token and by 32 dims,
// so that they cannot be left to the sums of one MMA.
// Where a pair has one tile only, B takes every other K/V tile of A's rows, so that one tile's
// softmax runs under the other's MMAs there too, and A's warps join the two.
//
// Split: the pairs of all sequences and kv heads are laid end to end, each as long as its walk and
// a start, and every CTA takes an equal stretch (the grid has one to an SM, fewer where the whole
// is short). A pair that a border cuts leaves partial results in the workspace, which a second kernel
// joins (log-sum-exp), 32 rows to a CTA. (The last CTA of a pair as the joiner took 13 us of 51 for the
// chunk below: one SM read 1.3 MB.)
//
// Bound by the way from S over the softmax back to the MMAs: at head_dim 128 a K/V tile takes A and B about 4300 cycles,
// of which the MMAs are 2048; A's S, softmax (about 1900) and O follow one another, and B's only half hide
// them, tensor memory having no room for a second S of either (at 64 it has 128 columns that are not used). 8192 queries
// over q4_0 (32 query, 8 kv heads, head_dim 128, bfloat16): 482 us, 1140 TFLOP/s over the visible tokens, where the same
// heads over 16-bit pools take the window prefill 513 us; 1024 queries of 4 sequences of up to 6001 tokens over e4m3 (64
// query heads): 298 us; 8 prompts of up to 1500 tokens over q4_0 (40 heads of 64, binary16): 121 us; one chunk of 100
// queries behind 2677 tokens: 31 us; 5 drafted tokens for 16 sequences of up to 32768: 176 us over q4_0, 2.0 TB/s, 221
// over e4m3, there bound by the copying and the converting warps (about 1100 and 1500 cycles each for a tile's K or V).
// Tried and slower there and elsewhere, when the 8192 queries took 516 us and the drafted tokens 173 to 186: copies by the
// converting warps (bulk: 586 us for the 8192 queries; 16 bytes a lane: 513), three times the converting warps where few
// have rows (200 us for the drafted tokens), twice as many with half a row to a thread (180, and 186 with a copying warp
// each for K and V), S in halves of 64 tokens, two of each A and B under way (560 us).
#pragma once

#include <type_traits>

#include "prefill_quant.h"
#include "prefill_window.cuh"

namespace pkv {

// 4 softmax warpgroups; MMA warps of A and B, copying warp, walking warp; a converting warpgroup. (With one softmax
// warpgroup to A and B: 522 us instead of 516 for the 8192 queries, 154 instead of 113 for the 8 prompts.)
constexpr int kPqThreads = 768;
constexpr int kPqSoft = 16;       // softmax warps: A's first and second halves of the columns, B's
constexpr int kPqConvert = 4;     // converting warps
constexpr int kPqMaxCtas = 152;
// Registers of a thread after the split, which the launch's 80 add up to: softmax, MMA and copy, conversion.
constexpr int kPqLaunchRegs = 80, kPqSoftRegs = 88, kPqIssueRegs = 56, kPqConvertRegs = 72;
static_assert(4 * kPqSoftRegs + kPqIssueRegs + kPqConvertRegs <= kPqThreads / 128 * kPqLaunchRegs, "no more than the launch has");
// A pair's start and end, as tokens of its walk. Head_dim 128: 522 us with 256, 466 with 512, 484 with 1024 (8192
// queries over q4_0, 32 query and 8 kv heads, which took 16 us less before rows were read whole); head_dim 64, where a tile
// takes less: 109 with 256, 108 with 384, 116 with 512 (8 prompts of up to 1500 tokens, 40 heads, K in one part). Not
// swept over e4m3.
constexpr int pq_start(int head_dim) { return head_dim == 64 ? 384 : 512; }
// A CTA's stretch is no shorter: one chunk of 100 queries behind 2677 tokens takes 31 us (35 with 1024, 50 with 2048; 128
// to 384 give the same).
constexpr int kPqMinTokens = 512;
constexpr int kPqRing = 4;        // parts that the walking warp may be ahead

// pw_wait for a kernel of many warps that wait much of their time: sixty-four attempts between two looks at the
// clock. (Polls take issue slots from the warps that work; a look at the clock is four times a poll.)
__device__ __forceinline__ bool pq_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_test_wait(bar, parity)) return true;
  if (limit_ns == 0) return false;
  const uint32_t at = smem_u32(bar);
  auto attempts = [&]() {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
        "mov.u32 n, 64;\n\t"
        "AGAIN_%=:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra OUT_%=;\n\t"
        "sub.u32 n, n, 1;\n\t"
        "setp.ne.u32 q, n, 0;\n\t"
        "@q bra AGAIN_%=;\n\t"
        "OUT_%=:\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(at), "r"(parity)
        : "memory");
    return done != 0;
  };
  if (attempts()) return true;
  const uint64_t t0 = globaltimer_ns();
  do {
    if (attempts()) return true;
  } while (globaltimer_ns() - t0 < limit_ns);
  return false;
}

// What a stretch is measured in: tokens x group, halved until the whole fits in 30 bits.
using PqCost = int;

// What a CTA tells the joining kernel: the pair that starts in it and goes on in others, and whether it has met rows
// that it cannot do.
struct alignas(16) PqCut {
  int last;  // CTA of its last part; below 0: no such pair
  int q0, kvh, row0, active;
  int wide;  // of the CTA: it has met a scale whose values exceed binary16's range
  int pad[2];
};

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
  int start;         // pq_start()
  PwDivisor by_group;
  PqCut* cuts;       // [kPqMaxCtas]
  float2* part_ml;   // [2 kPqMaxCtas][256]
  float4* part_o;    // [2 kPqMaxCtas][D / 4][256]
  int32_t* dev_err;
  uint64_t wait_limit_ns;
};

enum class PqFormat { kQ4, kFp8 };

// Binary16 queries over q4_0: P and K enter in two 16-bit parts, a value rounded and what that leaves, since one
// rounding of either is as much as an output's own. K's second part costs 3 to 17 % at head_dim 64 (the 8 prompts: 123 us
// instead of 106). At 128 there is room for one tile of K only, and both second parts together cost 63 to 103 % (16
// sequences of 40 queries behind 300 to 2600 tokens, 64 heads: 111 us instead of 68; the 8192 queries: 915 instead of 470;
// the drafted tokens: 350 instead of 173). Error against 64 bits over that of the output's rounding alone,
// standard normal rows: 1.6 to 1.9 with one part of both, 1.5 to 1.6 with one of K (2.0 with logits of twice the
// spread, since K's roundings grow with them), 1.3 with two of both. e4m3 values are exact (1.4 with one part of P), and a
// bfloat16 output's rounding is 8 times as large.
template <typename T, PqFormat F>
constexpr bool kPqTwoParts = std::is_same<T, __half>::value && F == PqFormat::kQ4;

template <typename T, PqFormat F, int D>
struct PqShape {
  static constexpr int kCB = D / 64;
  static constexpr int kColBlock = 128 * 128;
  static constexpr int kTile = kCB * kColBlock;                      // a Q, K or V operand tile
  static constexpr int kRow = F == PqFormat::kQ4 ? D / 16 * 9 : D;   // bytes of a cache row
  static constexpr int kRaw = 128 * kRow;
  static constexpr int kRawStages = D == 64 ? 6 : (F == PqFormat::kQ4 ? 3 : 2);
  static constexpr int kParts = kPqTwoParts<T, F> ? 2 : 1;           // of K and P
  static constexpr int kKStages = kParts == 2 && D == 128 ? 1 : 2;   // (there is no room for two tiles of two parts)
  static constexpr int kKOff = 2 * kTile;
  static constexpr int kVOff = kKOff + kKStages * kParts * kTile;    // two V tiles
  static constexpr int kRawOff = kVOff + 2 * kTile;
  static constexpr int kBarOff = kRawOff + kRawStages * kRaw;
  static constexpr int kBars = 2 * kRawStages + 18 + 2 * kPqRing + 16 + 2;
  static constexpr int kRingOff = (kBarOff + 8 * kBars + 15) / 16 * 16;
  static constexpr int kSwapOff = kRingOff + 64 * kPqRing;
  static constexpr int kExpOff = kSwapOff + 2 * 2 * 128 * 4;
  static constexpr int kMiscOff = kExpOff + 2 * 128;
  static constexpr int kUsed = kMiscOff + 64;
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
    n = (int)((uint32_t)__ldg(p.query_start + s + 1) - (uint32_t)q0);
    // (rows outside q and out, which have query_start[num_seqs] of them, are never touched)
    const bool inside = q0 >= 0 && (uint32_t)q0 + (uint32_t)n <= (uint32_t)max(__ldg(p.query_start + p.num_seqs), 0);
    valid = L >= 0 && L <= p.max_blocks_per_seq * p.block_size && n >= 0 && n <= L && n <= p.max_query_len && inside;
    live = valid && n > 0;
  }
  __device__ __forceinline__ int pairs(int group) const { return (int)(((int64_t)n * group + 255) / 256); }
  // tokens x group of the first k of its pairs (per kv head) ...
  __device__ __forceinline__ long long tokens(int k, int group, int start) const {
    const long long each = (long long)group * (start + L - n), rows = (long long)n * group;
    return k * each + (256LL * k < rows ? 128LL * k * (k + 1) : 128LL * k * (k - 1) + rows);
  }
  // ... and their cost: no pair without any
  __device__ __forceinline__ PqCost before(int k, int group, int start, int shift) const {
    return (PqCost)(tokens(k, group, start) >> shift) + k;
  }
};

// The whole batch's cost and how CTAs share it.
struct PqShare {
  PqCost whole;
  int ctas, shift;
  __device__ __forceinline__ PqCost begin(int c) const { return whole / ctas * c + whole % ctas * c / ctas; }
  __device__ __forceinline__ int of(PqCost y) const {
    int c = min(ctas - 1, y / (whole / ctas + 1));
    while (begin(c + 1) <= y) ++c;
    return c;
  }
};

// A pair of query tiles, or the part of one that lies in the CTA's stretch.
struct alignas(16) PqPart {
  int s, kvh, q0, base;      // sequence; kv head; its first query; tokens before it
  int row0, active;          // first row; rows of the pair
  int end_a, end_b;          // tokens that the last queries of A and B see (0: B has none)
  int j0, j1;                // K/V tiles of this part
  int kind;                  // bits below
  int last;                  // CTA of the pair's last part
  int pad[4];
  static constexpr int kStop = 1;   // no part: the walk is over
  static constexpr int kDual = 2;   // one tile of rows: A and B take K/V tiles in turn
  static constexpr int kHead = 4;   // the pair starts here
  static constexpr int kWhole = 8;  // and ends here
  __device__ __forceinline__ bool stop() const { return kind & kStop; }
  __device__ __forceinline__ bool dual() const { return kind & kDual; }
  __device__ __forceinline__ bool whole() const { return kind & kWhole; }
  __device__ __forceinline__ int end() const { return max(end_a, end_b); }
  __device__ __forceinline__ int active_of(int x) const { return dual() ? active : max(min(active - 128 * x, 128), 0); }
  // Queries of tile x (A: 0, B: 1) take part in K/V tile j.
  __device__ __forceinline__ bool sees(int x, int j) const {
    return dual() ? ((j - j0) & 1) == x : j * 128 < (x ? end_b : end_a);
  }
};
static_assert(sizeof(PqPart) == 64, "a slot of the ring");

// A CTA's walk over the pairs in its stretch.
struct PqWalk {
  PqShare share;
  PqSeq seq;
  int s, kvh, pair, np;
  PqCost at, cost, lo, hi;  // the pair's place and length; the CTA's stretch

  __device__ __forceinline__ bool done() const { return at >= hi; }
  // The pair at hand, or what of it lies here; false where that is nothing.
  __device__ __forceinline__ bool part(const PqParams& p, PqPart& t) {
    cost = seq.before(pair + 1, p.group, p.start, share.shift) - seq.before(pair, p.group, p.start, share.shift);
    t.s = s, t.kvh = kvh, t.q0 = seq.q0, t.base = seq.L - seq.n;
    t.row0 = pair * 256;
    t.active = min(seq.n * p.group - t.row0, 256);
    const bool one = t.active <= 128;
    t.end_a = t.base + 1 + p.by_group.of(t.row0 + min(t.active, 128) - 1);
    t.end_b = one ? 0 : t.base + 1 + p.by_group.of(t.row0 + t.active - 1);
    const int tiles = (t.end() + 127) / 128;
    // (the same place gives the same tile to the CTA before it and to the one behind)
    const float scale = (float)tiles / (float)cost;
    auto tile_at = [&](PqCost y) { return y <= 0 ? 0 : (y >= cost ? tiles : min((int)((float)y * scale), tiles)); };
    t.j0 = tile_at(lo - at);
    t.j1 = tile_at(hi - at);
    t.kind = (lo <= at ? PqPart::kHead : 0) | (t.j0 == 0 && t.j1 == tiles ? PqPart::kWhole : 0);
    t.last = blockIdx.x;
    if (!t.whole()) {
      // one CTA may have every tile, although borders lie in the pair: the others have nothing to do then
      int c = lo <= at ? (int)blockIdx.x : share.of(at);
      while (tile_at(share.begin(c + 1) - at) == 0) ++c;
      if (tile_at(share.begin(c + 1) - at) == tiles) return false;
      t.last = share.of(at + cost - 1);
    }
    if (one && t.j1 - t.j0 > 1) t.kind |= PqPart::kDual;
    return true;
  }
  __device__ __forceinline__ void next(const PqParams& p) {
    at += cost;
    if (at >= hi || ++pair < np) return;
    pair = 0;
    if (++kvh < p.num_kv_heads) return;
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
};

// Sum over a warp's lanes of those up to this one.
template <typename I>
__device__ __forceinline__ I pq_warp_scan(I v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const I u = __shfl_up_sync(kFullMask, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// The walk at the beginning of the CTA's stretch; false where it has none. By one warp (a lane to a
// sequence): the others have their barriers and tensor memory to see to.
__device__ __forceinline__ bool pq_begin(const PqParams& p, PqWalk& walk) {
  const int lane = threadIdx.x & 31, G = p.group;
  long long tokens = 0;
  PqSeq first;  // of sequence `lane`
  first.live = false;
#pragma unroll 1
  for (int s = lane; s < p.num_seqs; s += 32) {
    PqSeq q;
    q.load(p, s);
    if (q.live) tokens += q.tokens(q.pairs(G), G, p.start) * p.num_kv_heads;
    if (!q.valid && blockIdx.x == 0) set_err(p.dev_err, PKV_DEV_ERR_CONTEXT_LEN);
    if (s == lane) first = q;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) tokens += __shfl_xor_sync(kFullMask, tokens, o);
  PqShare& share = walk.share;
  share.ctas = min(max((int)fminf((float)tokens / (float)(G * kPqMinTokens), 1e6f), 1), (int)gridDim.x);
  if (tokens == 0 || (int)blockIdx.x >= share.ctas) return false;
  share.shift = max(34 - __clzll(tokens), 0);  // tokens >> shift < 2^30
  auto cost_of = [&](int s, PqSeq& q) {
    if (s < 32)
      q = first;
    else if (s < p.num_seqs)
      q.load(p, s);
    return s < p.num_seqs && q.live ? q.before(q.pairs(G), G, p.start, share.shift) * p.num_kv_heads : 0;
  };
  share.whole = 0;
#pragma unroll 1
  for (int s = lane; s < p.num_seqs; s += 32) {
    PqSeq q;
    share.whole += cost_of(s, q);
  }
  share.whole = __reduce_add_sync(kFullMask, share.whole);
  const PqCost lo = share.begin(blockIdx.x);
  PqCost base = 0;
#pragma unroll 1
  for (int s0 = 0; s0 < p.num_seqs; s0 += 32) {
    PqSeq q;
    const PqCost own = cost_of(s0 + lane, q), upto = base + pq_warp_scan(own);
    const uint32_t here = __ballot_sync(kFullMask, lo < upto);
    if (here != 0u) {
      const int src = __ffs(here) - 1;
      walk.s = s0 + src;
      const PqCost at = __shfl_sync(kFullMask, upto - own, src);
      q.load(p, walk.s);
      walk.seq = q;
      walk.np = q.pairs(G);
      const PqCost head = q.before(walk.np, G, p.start, share.shift);
      walk.kvh = (lo - at) / head;
      const PqCost y = (lo - at) - walk.kvh * head;
      int a = 0, b = walk.np;  // the pair that holds y: before(a) <= y < before(b)
      while (b - a > 1) {
        const int mid = (a + b) / 2;
        if (q.before(mid, G, p.start, share.shift) <= y)
          a = mid;
        else
          b = mid;
      }
      walk.pair = a;
      walk.at = lo - y + q.before(a, G, p.start, share.shift);
      walk.lo = lo;
      walk.hi = share.begin(blockIdx.x + 1);
      return true;
    }
    base = __shfl_sync(kFullMask, upto, 31);
  }
  return false;
}

// q4_0 values d (q - 8) go up to 8 * 65504, eight times what binary16 holds: bfloat16 rows have them, and keys of
// binary16 once they were turned. The kernel goes on as if there were none; the converting warps note a scale of 8192 or
// more in magnitude, and the joining kernel does these pairs again in 32 bits. (That note and the joining kernel's look at
// it take 3 of the drafted tokens' 176 us. With a vote and a flag for each 32 rows, and MMAs that run eight times over
// eighths of the values, it was 184; with such parts walked a second time in here, the 8 prompts took 131 to 142 us instead
// of 124: longer code in all the roles.)

// 8 bytes of codes as 16 values d (q - 8): low halves to lo, high halves to hi. A code placed
// under the exponent of 1024 (low halves, last place 1) or of 64 (high halves, last place 1/16)
// is a binary16 number that exceeds it by that constant. kRest: not the values, but what their rounding
// leaves, which is exact: a multiple of 2^-24, as d is, of at most 11 bits (at most 16, and no matter what beside an
// infinite value).
template <bool kRest>
__device__ __forceinline__ void pq_from_q4(uint32_t w0, uint32_t w1, __half2 d, uint4& lo, uint4& hi) {
  const __half2 k1032 = __half2half2(__ushort_as_half(0x6408)), k72 = __half2half2(__ushort_as_half(0x5480));
  auto part = [&](uint32_t w, uint32_t exponent, uint32_t sel, __half2 minus) {
    const uint32_t u = __byte_perm(w, exponent, sel);
    __half2 h;
    memcpy(&h, &u, 4);
    h = __hsub2(h, minus);
    if constexpr (kRest) {
      const __half2 most = __half2half2(__ushort_as_half(0x4c00));
      h = __hmax2(__hmin2(__hfma2(h, d, __hneg2(__hmul2(h, d))), most), __hneg2(most));
    } else {
      h = __hmul2(h, d);
    }
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

// Row r of a tile: its bytes at `row` become the operand's values (zeros where !held) in the swizzled tile
// at `tile`. kRest: what the values' rounding leaves as well, in the tile behind it. large: the
// largest magnitudes of the scales so far.
template <PqFormat F, int D, bool kRest>
__device__ __forceinline__ void pq_convert(const unsigned char* row, unsigned char* tile, int r, bool held, __half2& large) {
  unsigned char* at = tile + r * 128;
  const uint32_t swz = (r & 7) << 4;
  // values 8 c .. 8 c + 7 of the row
  auto put = [&](int c, uint4 v) {
    *reinterpret_cast<uint4*>(at + (c >> 3) * (128 * 128) + ((((uint32_t)c & 7) << 4) ^ swz)) = v;
  };
  if (!held) {
#pragma unroll
    for (int c = 0; c < (kRest ? 2 : 1) * D / 8; ++c) put(c, make_uint4(0u, 0u, 0u, 0u));
    return;
  }
  // all is read before anything is written, so that the reads need not wait for one another
  if constexpr (F == PqFormat::kQ4) {
    constexpr int kWords = D / 64 * 9;
    uint32_t w[kWords];
    if constexpr (D == 128) {  // (rows start on 8 bytes at head_dim 128, on 4 at 64)
#pragma unroll
      for (int i = 0; i < kWords / 2; ++i) {
        const uint2 x = reinterpret_cast<const uint2*>(row)[i];
        w[2 * i] = x.x, w[2 * i + 1] = x.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint32_t*>(row)[i];
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      __half2 d;
      memcpy(&d, &w[i], 4);
      large = __hmax2(large, __habs2(d));
    }
#pragma unroll
    for (int b = 0; b < D / 32; ++b) {
      const __half2 d = __half2half2(__ushort_as_half((unsigned short)(w[b / 2] >> (16 * (b & 1)))));
      const uint32_t* codes = w + D / 64 + 4 * b;
      uint4 lo, hi;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        pq_from_q4<false>(codes[2 * i], codes[2 * i + 1], d, lo, hi);
        put(4 * b + i, lo);
        put(4 * b + 2 + i, hi);
        if constexpr (kRest) {
          pq_from_q4<true>(codes[2 * i], codes[2 * i + 1], d, lo, hi);
          put(D / 8 + 4 * b + i, lo);
          put(D / 8 + 4 * b + 2 + i, hi);
        }
      }
    }
  } else {
    // lanes take a row's 16-byte chunks in orders of their own, so that eight lanes' chunks fall
    // into different banks
    const int turn = D == 128 ? r & 7 : (r >> 1) & 3;
    uint4 x[D / 16];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) x[i] = *reinterpret_cast<const uint4*>(row + 16 * (i ^ turn));
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const int c = i ^ turn;
      put(2 * c, make_uint4(pq_from_e4m3x2(x[i].x & 0xffffu), pq_from_e4m3x2(x[i].x >> 16),
                            pq_from_e4m3x2(x[i].y & 0xffffu), pq_from_e4m3x2(x[i].y >> 16)));
      put(2 * c + 1, make_uint4(pq_from_e4m3x2(x[i].z & 0xffffu), pq_from_e4m3x2(x[i].z >> 16),
                                pq_from_e4m3x2(x[i].w & 0xffffu), pq_from_e4m3x2(x[i].w >> 16)));
    }
  }
}

template <typename T, PqFormat F, int D>
__global__ void __launch_bounds__(kPqThreads, 1) pa_prefill_quant_kernel(const __grid_constant__ PqParams p) {
  using S = PqShape<T, F, D>;
  using Out = PwPack<T>;
  using P16 = PwPack<__half>;
  // The base of a row's running maximum moves only when that grows by more than kRescaleLog2, and it lies kTopLog2 -
  // kRescaleLog2 below the maximum that it was taken from: every weight stays below 2^kTopLog2, binary16's range, and
  // the largest at or above 2^7, so that a weight keeps its bits down to 2^-21 of it and has an error of 2^-32 of it
  // below that (131072 tokens that far below one other lose 2^-15 of the output). Moved by 2, some row of a
  // warp's 32 moves it in every third tile: 560 us instead of 516 for the 8192 queries.
  constexpr float kTopLog2 = 15.f, kRescaleLog2 = 8.f;
  constexpr int CB = S::kCB, NR = S::kRawStages;
  constexpr bool kBf16 = std::is_same<T, __nv_bfloat16>::value;
  constexpr int kParts = S::kParts, KS = S::kKStages;
  extern __shared__ __align__(1024) unsigned char sm[];
  // Every barrier's phases follow one another in the order of the work, and nobody who waits for
  // a phase can fall two behind. K and V tiles are counted through all parts of the CTA: tile m is in
  // buffers m % KS and m % 2.
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S::kBarOff);
  uint64_t* raw_full = bars;             // [NR] a tile's bytes landed
  uint64_t* raw_empty = raw_full + NR;   // [NR] and were converted (an arrival per converting warp)
  uint64_t* k_ready = raw_empty + NR;    // [KS] a K tile is in place (likewise)
  uint64_t* v_ready = k_ready + 2;       // [2] a V tile is
  uint64_t* k_empty = k_ready + 4;       // [KS] the MMAs are done with it (A's and B's: two arrivals)
  uint64_t* v_empty = k_ready + 6;       // [2] likewise
  uint64_t* s_full = k_ready + 8;        // [A, B] S computed
  uint64_t* p_full = k_ready + 10;       // [A, B] P written (one arrival per softmax warp)
  uint64_t* q_full = k_ready + 12;       // [A, B] query rows in place (likewise)
  uint64_t* o_full = k_ready + 14;       // [A, B] the part's last O computed
  uint64_t* turn = k_ready + 16;         // [A, B] the other's MMAs of a step are issued
  uint64_t* part_full = k_ready + 18;    // [kPqRing] the walk's next part is there
  uint64_t* part_empty = part_full + kPqRing;  // [kPqRing] and was read (by every warp but the walking one)
  uint64_t* box_full = part_empty + kPqRing;   // [8] B's partial results for A's warp are there
  uint64_t* box_empty = box_full + 8;    // [8] and were read
  uint64_t* shared_q = box_empty + 8;    // A's query rows in place for B too (an arrival per warp of A)
  uint64_t* drained = shared_q + 1;      // every MMA of the CTA done (two arrivals)
  PqPart* ring = reinterpret_cast<PqPart*>(sm + S::kRingOff);     // [kPqRing]
  float* swap = reinterpret_cast<float*>(sm + S::kSwapOff);       // [half][A, B][128] from one half's warp to the other's
  unsigned char* exps = sm + S::kExpOff;                          // [A, B][128] exponents taken out of the query rows
  unsigned char* misc = sm + S::kMiscOff;
  uint32_t* slot = reinterpret_cast<uint32_t*>(misc);             // tensor-memory address
  uint32_t* held_blocks = reinterpret_cast<uint32_t*>(misc + 16); // [NR] blocks of a raw tile that were copied
  static_assert(16 + 4 * NR <= 64, "room");

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = p.group;

  grid_launch_dependents();  // (the joining kernel waits for all of this one's memory all the same)

  // ---- set-up: barriers, tensor memory ----------------------------------------
  if (tid == kPqThreads - 1) {
    for (int i = 0; i < NR; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kPqConvert);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_ready[i], kPqConvert);
      mbar_init(&v_ready[i], kPqConvert);
      mbar_init(&k_empty[i], 2);
      mbar_init(&v_empty[i], 2);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 8);
      mbar_init(&q_full[i], 8);
      mbar_init(&o_full[i], 1);
      mbar_init(&turn[i], 1);
    }
    for (int i = 0; i < kPqRing; ++i) {
      mbar_init(&part_full[i], 1);
      mbar_init(&part_empty[i], kPqSoft + 3 + kPqConvert);
    }
    for (int i = 0; i < 8; ++i) {
      mbar_init(&box_full[i], 1);
      mbar_init(&box_empty[i], 1);
    }
    mbar_init(shared_q, 8);
    mbar_init(drained, 2);
    mbar_init_fence();
  }
  if (warp == 16) tmem_alloc(slot, kPwTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *slot;
  bool bad = false;  // a wait ran out
  auto wait = [&](uint64_t* bar, uint32_t parity) {  // the same answer in the whole warp
    return __all_sync(kFullMask, pq_wait(bar, parity, p.wait_limit_ns));
  };
  // The n-th part of the walk; false where there is none.
  auto take = [&](uint32_t n, PqPart& part) {
    if (!bad && !wait(&part_full[n % kPqRing], (n / kPqRing) & 1)) bad = true;
    if (bad) return false;
    part = ring[n % kPqRing];
    __syncwarp();
    if (lane == 0) mbar_arrive(&part_empty[n % kPqRing]);
    return !part.stop();
  };

  // (the registers of a warpgroup change hands for all its warps at once)
  if (warp >= 20) {
    // ---- conversion: K of one tile, V of the one before, into the operands' buffers; a thread to a row
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPqConvertRegs));
    const int r = tid & 127, block = r >> p.block_bits;
    uint32_t tiles = 0;  // of earlier parts
    int stage = 0;
    uint32_t phase = 0;
    __half2 large = __half2half2(__ushort_as_half(0));
    PqPart part;
    for (uint32_t n = 0; take(n, part); ++n) {
      const int end = part.end(), j0 = part.j0, j1 = part.j1;
      for (int i = 0; i < 2 * (j1 - j0) && !bad; ++i) {
        // K0, K1, V0, K2, V1, ...; with one buffer for K, where K1 must wait for S of K0, K0, V0, K1, V1, ...
        const bool is_v = KS == 1 ? i & 1 : i == 2 * (j1 - j0) - 1 || (i > 0 && (i & 1) == 0);
        const int j = j0 + (KS == 1 ? i / 2 : is_v ? (i - 1) / 2 : (i + 1) / 2);
        const uint32_t m = tiles + (j - j0), ks = is_v ? 2 : KS, c = m % ks;
        if (m >= ks && !wait((is_v ? v_empty : k_empty) + c, (m / ks + 1) & 1)) {
          bad = true;
          break;
        }
        if (!wait(&raw_full[stage], phase)) {
          bad = true;
          break;
        }
        const bool held = j * 128 + r < end && ((held_blocks[stage] >> block) & 1u);
        const unsigned char* row = sm + S::kRawOff + stage * S::kRaw + r * S::kRow;
        if (kParts == 2 && !is_v)
          pq_convert<F, D, kParts == 2>(row, sm + S::kKOff + c * (kParts * S::kTile), r, held, large);
        else
          pq_convert<F, D, false>(row, sm + (is_v ? S::kVOff : S::kKOff) + c * S::kTile, r, held, large);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&raw_empty[stage]);
          mbar_arrive((is_v ? v_ready : k_ready) + c);
        }
        if (++stage == NR) stage = 0, phase ^= 1;
      }
      tiles += j1 - j0;
    }
    if (F == PqFormat::kQ4 && __any_sync(kFullMask, fmaxf(__low2float(large), __high2float(large)) >= 8192.f) && lane == 0)
      p.cuts[blockIdx.x].wide = 1;
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
  } else if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kPqIssueRegs));
    if (warp == 18) {
      // ---- the walk
      PqWalk walk;
      if (lane == 0) p.cuts[blockIdx.x].last = -1, p.cuts[blockIdx.x].wide = 0;  // (before any part is told)
      const bool any = pq_begin(p, walk);
      for (uint32_t n = 0;; ++n) {
        if (n >= kPqRing && !wait(&part_empty[n % kPqRing], (n / kPqRing + 1) & 1)) {
          bad = true;
          break;
        }
        PqPart part;
        while (any && !walk.done() && !walk.part(p, part)) walk.next(p);
        const bool stop = !any || walk.done();
        if (lane == 0) {
          if (!stop && (part.kind & PqPart::kHead) && !part.whole()) {
            PqCut& told = p.cuts[blockIdx.x];
            told.last = part.last;
            told.q0 = part.q0, told.kvh = part.kvh, told.row0 = part.row0, told.active = part.active;
          }
          if (stop)
            ring[n % kPqRing].kind = PqPart::kStop;
          else
            ring[n % kPqRing] = part;
          mbar_arrive(&part_full[n % kPqRing]);
        }
        __syncwarp();
        if (stop) break;
        walk.next(p);
      }
    } else if (warp == 17) {
      // ---- copies: a tile's cache blocks, one to a lane
      const int per_tile = 128 >> p.block_bits;  // <= 16 blocks
      const uint32_t bytes = (uint32_t)p.block_size * S::kRow;
      uint32_t raw = 0;  // tiles so far
      int stage = 0;
      uint32_t phase = 1;  // of raw_empty, from the second round on
      PqPart part;
      for (uint32_t n = 0; take(n, part); ++n) {
        const int32_t* bt = p.block_tables + (size_t)part.s * p.max_blocks_per_seq;
        const int blocks = (part.end() + p.block_size - 1) >> p.block_bits, j0 = part.j0, j1 = part.j1;
        // whether this lane has a block of tile j; what the table says there is checked when it has come
        auto has = [&](int j) { return j < j1 && lane < per_tile && j * per_tile + lane < blocks; };
        auto fetch = [&](int j) { return has(j) ? __ldg(bt + j * per_tile + lane) : -1; };
        auto copy = [&](int b, const unsigned char* pool) {  // b: a block of the pool, below 0: none
          if (raw >= NR && !wait(&raw_empty[stage], phase)) {
            bad = true;
            return;
          }
          const uint32_t some = __ballot_sync(kFullMask, b >= 0);
          if (lane == 0) {
            held_blocks[stage] = some;
            mbar_arrive_expect_tx(&raw_full[stage], __popc(some) * bytes);
          }
          __syncwarp();
          if (b >= 0)
            bulk_copy_g2s(sm + S::kRawOff + stage * S::kRaw + lane * bytes,
                          pool + ((size_t)b * p.num_kv_heads + part.kvh) * bytes, bytes, &raw_full[stage]);
          ++raw;
          if (++stage == NR) stage = 0, phase ^= 1;
        };
        int id = fetch(j0), id_v = -1;
        for (int j = j0; j <= j1 && j0 < j1 && !bad; ++j) {  // K of tile j, V of the one before (KS == 1: V too)
          if (id < 0 || id >= p.num_blocks) {
            if (has(j)) set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
            id = -1;
          }
          const int id_next = fetch(j + 1);
          if (j < j1) copy(id, p.k_cache);
          if (KS == 1) id_v = id;
          if ((KS == 1 ? j < j1 : j > j0) && !bad) copy(id_v, p.v_cache);
          id_v = id;
          id = id_next;
        }
      }
      // the last copies must land before the CTA can leave
      if (lane == 0)
        for (uint32_t c = raw >= NR ? raw - NR : 0; c < raw; ++c)
          mbar_wait_bounded(&raw_full[c % NR], (c / NR) & 1, kDrainLimitNs);
      __syncwarp();
    } else {
      // ---- MMA issue, a warp for each of A and B ------------------------------------------
      // A step: O += P V of one tile, S of the next. With two tiles of rows at head_dim 128 A and B
      // take turns, so that one's softmax runs under the other's MMAs. MMAs of one thread complete
      // in order, so S may take the place of a P that the MMA before it reads, and "S done" says
      // that O holds every earlier tile.
      const int x = warp == 16 ? 0 : 1;
      constexpr uint32_t id_s = mma_idesc_f16(128, 128, 0, 0);
      constexpr uint32_t id_o = mma_idesc_f16(128, D, 0, 1);
      // The whole warp waits, one elected lane issues; operands handed round from one lane are known to the
      // compiler to be the same in all, and stay where the MMAs take them from.
      const uint32_t tb = __shfl_sync(kFullMask, tbase, 0);
      const uint32_t sb = __shfl_sync(kFullMask, smem_u32(sm), 0);
      // of a descriptor only the start address in its low word moves
      const uint32_t kd = (uint32_t)smem_desc_sw128(sb + S::kKOff, 16, 1024);
      const uint32_t vd = (uint32_t)smem_desc_sw128(sb + S::kVOff, S::kColBlock, 1024);
      const uint32_t hi = (uint32_t)(smem_desc_sw128(0, 16, 1024) >> 32);  // K-major and MN-major alike
      uint32_t tiles = 0, done = 0, turns = 0;  // tiles of earlier parts; P's and steps in turn so far
      PqPart part;
      for (uint32_t n = 0; take(n, part); ++n) {
        const int count = part.j1 - part.j0;
        const bool in_turn = D == 128 && !part.dual();
        const uint32_t qd =
            __shfl_sync(kFullMask, (uint32_t)smem_desc_sw128(sb + (part.dual() ? 0 : x) * S::kTile, 16, 1024), 0);
        bool seen = false, opened = false;  // the tile before is seen, O holds something
        bad = !wait(&q_full[x], n & 1);
        for (int i = 0; i <= count && count > 0 && !bad; ++i) {  // O of tile i - 1, S of tile i
          const uint32_t mk = tiles + i, mv = mk - 1;
          const bool next = i < count && part.sees(x, part.j0 + i);
          const uint32_t kb = __shfl_sync(kFullMask, kd + (mk % KS * (kParts * S::kTile) >> 4), 0);
          const uint32_t vb = __shfl_sync(kFullMask, vd + ((mv & 1) * S::kTile >> 4), 0);
          // (the turn comes last, so that nothing but the issue lies between it and the other's)
          if (i < count) bad = !wait(&k_ready[mk % KS], (mk / KS) & 1);
          // (a part's first P comes from warps that have read the O of the part before)
          if (!bad && seen) bad = !wait(&v_ready[mv & 1], (mv >> 1) & 1) || !wait(&p_full[x], done++ & 1);
          if (!bad && in_turn && (x == 1 || turns > 0)) bad = !wait(&turn[x], (turns + (x ^ 1)) & 1);
          tc_fence_after();
          if (!bad && elect_one()) {
            if (seen) {
#pragma unroll
              for (int part16 = 0; part16 < kParts; ++part16)  // the high parts of P, then the remainders
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                  pw_mma_ts(tb + 256 + 128 * x, tb + 128 * x + 32 * (ks >> 1) + 16 * part16 + 8 * (ks & 1),
                            vb + (ks * 2048 >> 4), hi, id_o, (part16 > 0 || ks > 0 || opened) ? 1u : 0u);
              mma_commit(&v_empty[mv & 1]);
            }
            if (next) {
#pragma unroll
              for (int part16 = 0; part16 < kParts; ++part16)
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks) {
                  const uint32_t off = ((ks >> 2) * S::kColBlock + (ks & 3) * 32) >> 4;
                  pw_mma_ss(tb + 128 * x, qd + off, kb + (part16 * S::kTile >> 4) + off, hi, id_s, part16 > 0 || ks > 0);
                }
              mma_commit(&s_full[x]);  // (the softmax gives K back)
            } else if (i < count) {
              mbar_arrive(&k_empty[mk % KS]);
            }
            if (in_turn) mbar_arrive(&turn[x ^ 1]);
          }
          __syncwarp();
          // (a tile that is not seen is given back when it is there, not before: an arrival ahead of its
          // time would stand for the other query tile's)
          if (!bad && i > 0 && !seen) {
            bad = !wait(&v_ready[mv & 1], (mv >> 1) & 1);
            if (!bad && lane == 0) mbar_arrive(&v_empty[mv & 1]);
          }
          turns += in_turn;
          opened |= seen;
          seen = next;
        }
        if (!bad && elect_one()) mma_commit(&o_full[x]);
        __syncwarp();
        tiles += count;
      }
      // nothing may be torn down before the last MMA, after a timeout neither
      if (elect_one()) mma_commit(drained);
      __syncwarp();
      mbar_wait_bounded(drained, 0, kDrainLimitNs);
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    __syncwarp();
  } else {
    // ---- softmax: two warpgroups to a query tile, half the columns of a row (64 of S, D / 2 of O) to a
    // thread. The two warps of a row's halves have a named barrier, which both pass whatever happens to
    // either, and agree there whether a wait ran out.
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kPqSoftRegs));
    const int x = warp >> 3, h = (warp >> 2) & 1, w4 = warp & 3, r = tid & 127;
    const int pair_id = 1 + 4 * x + w4;
    const uint32_t ts = tbase + ((uint32_t)(32 * w4) << 16) + 128 * x;  // S of this warp's lanes
    const uint32_t to = ts + 256 + h * (D / 2);                        // and its half of O
    float* const mine_at = swap + 256 * h + 128 * x + r;
    const float* const other_at = swap + 256 * (h ^ 1) + 128 * x + r;
    uint32_t done = 0, tiles = 0;             // P's, tiles of earlier parts
    uint32_t duals = 0, boxes = 0;            // parts of one tile, boxes between A and B

    // A part's place in the ring is read from there whenever it is needed (no registers to spare) and
    // given back at the part's end.
    auto look = [&](uint32_t n) {
      if (!bad && !wait(&part_full[n % kPqRing], (n / kPqRing) & 1)) bad = true;
      return !bad && !ring[n % kPqRing].stop();
    };
    auto first_row = [&](const PqPart& part) { return part.row0 + (part.dual() ? 0 : x * 128); };
    // The part's query rows into shared memory as binary16: 16 rows to a warp, 8 lanes to a row, 4 rows at a
    // time. A bfloat16 row is divided by 2^e so that its largest value lies in [2^14, 2^15): what exceeds
    // 2^-28 of that keeps its 8 bits.
    auto place_q = [&](const PqPart& part) {
      if (part.dual() && x == 1) return;  // A's rows serve both
      const T* q = static_cast<const T*>(p.q);
      const int active = part.active_of(x);
      uint4 all[4][CB];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = 32 * w4 + 16 * h + 4 * i + (lane >> 3);
        const bool in = rr < active;
        const int g = first_row(part) + rr, t = in ? p.by_group.of(g) : 0, j = in ? g - t * G : 0;
        const uint4* src = reinterpret_cast<const uint4*>(
            q + ((size_t)(part.q0 + t) * p.num_heads + part.kvh * G + j) * D) + (lane & 7);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) all[i][cb] = in ? __ldg(src + 8 * cb) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int rr = 32 * w4 + 16 * h + 4 * i + (lane >> 3);
        uint4(&v)[CB] = all[i];
        if constexpr (kBf16) {
          uint32_t top = 0u;  // largest exponent bits of the row
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            const uint32_t w[4] = {v[cb].x, v[cb].y, v[cb].z, v[cb].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) top = max(top, max(w[k] & 0x7f80u, (w[k] >> 16) & 0x7f80u));
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(kFullMask, top, o));
          // times 2^(14 - k) for an exponent of k, at most 2^126
          const int k = top == 0u ? 14 : max((int)(top >> 7) - 127, -112);
          const float by = __uint_as_float((uint32_t)(14 - k + 127) << 23);
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) {
            float f[8];
            Chunk<__nv_bfloat16>::widen(v[cb], f);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= by;
            v[cb] = Chunk<__half>::narrow(f);
          }
          if ((lane & 7) == 0) exps[128 * x + rr] = (unsigned char)(k + 112);
        }
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          *reinterpret_cast<uint4*>(sm + x * S::kTile + cb * S::kColBlock + rr * 128 + (((lane & 7) ^ (rr & 7)) << 4)) =
              make_uint4(v[cb].x ^ p.flip, v[cb].y ^ p.flip, v[cb].z ^ p.flip, v[cb].w ^ p.flip);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&q_full[x]);
        if (part.dual()) mbar_arrive(shared_q);
      }
    };
    // The part's query rows on their way to L2 while earlier MMAs run (a hint only).
    auto prefetch_q = [&](const PqPart& part) {
      const int rr = 32 * w4 + lane;
      if ((part.dual() && x == 1) || rr >= part.active_of(x)) return;
      const int g = first_row(part) + rr, t = p.by_group.of(g);
      const T* src = static_cast<const T*>(p.q) +
                     ((size_t)(part.q0 + t) * p.num_heads + part.kvh * G + g - t * G) * D;
      if (D == 128 || h == 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(src + 64 * h));
    };
    bool more = look(0);
    if (more) place_q(ring[0]);
    for (uint32_t n = 0;; ++n) {
      // (also: the other half's warp has put its query rows' exponents in place, and done with `swap`)
      if (barrier_or(pair_id, 64, bad)) bad = true;
      if (bad || !more) break;
      const PqPart& part = ring[n % kPqRing];
      const bool dual = part.dual();
      if (dual && x == 1) {
        // (A's warps put the next rows in place when they have B's results of this part only, so
        // that the phase waited for is never more than one away)
        if (!wait(shared_q, duals & 1)) bad = true;
        if (lane == 0) mbar_arrive(&q_full[1]);
        ++duals;
      }
      const int active = part.active_of(x);
      const bool idle = 32 * w4 >= active;  // no row of this warp is a query's
      float sc = p.scale_log2;              // this row's factor from S to logits in powers of two
      if (kBf16 && !p.zero_scale)
        sc = fmaxf(sc * __uint_as_float((uint32_t)(exps[(dual ? 0 : 128 * x) + r] + 1) << 23), 1.401298464e-45f);
      float m_use = -INFINITY, l = 0.f;
      bool first = true;
      {
        const int g = first_row(part) + min(r, max(active - 1, 0));  // past the last row: any result
        const int pos = part.base + p.by_group.of(g) - 64 * h;
        const int j0 = part.j0, step = dual ? 2 : 1;
        const int j1 = dual ? part.j1 : min(part.j1, ((x ? part.end_b : part.end_a) + 127) / 128);  // that x sees
#pragma unroll 1
        for (int j = j0 + (dual ? x : 0); j < j1; j += step) {
          if (!bad && !wait(&s_full[x], done & 1)) bad = true;
          tc_fence_after();
          if ((warp & 7) == 0 && lane == 0) mbar_arrive(&k_empty[(tiles + (j - j0)) % KS]);
          ++done;
          if (idle) {  // (its rows of P, and so of O, may hold anything)
            if (bad) break;
            if (lane == 0) mbar_arrive(&p_full[x]);
            continue;
          }
          const int vis = pos - j * 128 + 1;  // columns of this half up to the row's own
          const bool cut = __any_sync(kFullMask, vis < 64);
          auto hide = [&](int c, uint32_t (&w)[32]) {  // of columns 32 c .. those that the row does not see
            const uint32_t see = low_bits(vis - 32 * c);
#pragma unroll
            for (int i = 0; i < 32; ++i) w[i] = (see >> i) & 1u ? w[i] : 0xff800000u;
          };
          uint32_t u[32];  // (the first 32 columns are read again for the weights: no registers for all 64)
          float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            tmem_ld32(ts + 64 * h + 32 * c, u);
            tmem_wait_ld();
            if (cut) hide(c, u);
#pragma unroll
            for (int i = 0; i < 32; i += 2)
              m4[i / 2 & 3] = pw_max3(m4[i / 2 & 3], __uint_as_float(u[i]), __uint_as_float(u[i + 1]));
          }
          float mt = sc * fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
          // the base moves only when the maximum exceeds it by more than kTopLog2, that is, has grown by more than
          // kRescaleLog2 since: every P stays below 2^kTopLog2, and O and the row sum have the same base. (Logits
          // from kPwFar on are whole numbers, and a base may be off by half their distance: there it is the
          // maximum and moves whenever that does.)
          const float most = fabsf(m_use) < kPwFar ? kTopLog2 : 0.f;
          // (the difference is not a number, and no growth, for -inf - -inf)
          float alpha = 1.f;
          if (barrier_or(pair_id, 64, bad || mt - m_use > most)) {
            *mine_at = bad ? __uint_as_float(0x7fffffffu) : mt;
            if (barrier_or(pair_id, 64, bad)) {
              bad = true;
              break;
            }
            mt = fmaxf(mt, *other_at);
            const bool grow = mt - m_use > most;
            if (grow) {
              const float base = mt - (fabsf(mt) < kPwFar ? kTopLog2 - kRescaleLog2 : 0.f);
              alpha = exp2f(m_use - base);  // 0 while nothing was visible
              m_use = base;
            }
            if (!first && __any_sync(kFullMask, grow)) {
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t w[16];
                tmem_ld16(to + 16 * c, w);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(__uint_as_float(w[i]) * alpha);
                tmem_st16(to + 16 * c, w);
              }
            }
          }
          first = false;
          const float nbase = m_use == -INFINITY ? 0.f : -m_use;
          const uint64_t sc2 = pw_pair(sc, sc), nb2 = pw_pair(nbase, nbase);
          uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 1; c >= 0; --c) {
            if (c == 0) {
              tmem_ld32(ts + 64 * h, u);
              tmem_wait_ld();
              if (cut) hide(0, u);
            }
            uint32_t w[16], rest[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float2 e = pw_unpair(
                  pw_fma2(pw_pair(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), sc2, nb2));
              e.x = pw_exp2(e.x);
              e.y = pw_exp2(e.y);
              sum[i & 1] = pw_add2(sum[i & 1], pw_pair(e.x, e.y));
              if constexpr (kParts == 2) {
                float2 hp;
                w[i] = P16::high(e, hp);
                hp = pw_unpair(pw_fma2(pw_pair(hp.x, hp.y), pw_pair(-1.f, -1.f), pw_pair(e.x, e.y)));
                rest[i] = P16::pack(hp.x, hp.y);
              } else {
                w[i] = P16::pack(e.x, e.y);
              }
            }
            // the weights of 32 tokens take the first half of their scores' place, remainders the second
            tmem_st16(ts + 64 * h + 32 * c, w);
            if constexpr (kParts == 2) tmem_st16(ts + 64 * h + 32 * c + 16, rest);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&p_full[x]);
          const float2 total = pw_unpair(pw_add2(sum[0], sum[1]));
          l = l * alpha + (total.x + total.y);
        }
      }
      // what the output needs of this part, then the next one's place, then the wait
      tiles += part.j1 - part.j0;
      const bool whole = part.whole();
      const int row0 = first_row(part);
      const int my_slot = 2 * blockIdx.x + ((part.kind & PqPart::kHead) ? 1 : 0);
      T* const rows_out = static_cast<T*>(p.out) + ((size_t)part.q0 * p.num_heads + part.kvh * G) * D;
      auto row_out = [&](int g) {  // row g of the kv head
        const int t = p.by_group.of(g);
        return rows_out + ((size_t)t * p.num_heads + (g - t * G)) * D;
      };
      more = look(n + 1);
      const PqPart& after = ring[(n + 1) % kPqRing];
      if (more) prefetch_q(after);
      // the row's sum over both halves
      barrier_or(pair_id, 64, false);
      *mine_at = l;
      barrier_or(pair_id, 64, false);
      l += *other_at;
      if (!bad && !wait(&o_full[x], n & 1)) bad = true;
      tc_fence_after();
      if (more && !bad && !dual) place_q(after);
      __syncwarp();
      if (lane == 0) mbar_arrive(&part_empty[n % kPqRing]);

      // 16 dims (chunk c of this half) of this row's O as it is
      auto load_o = [&](int c, uint32_t (&w)[16]) {
        if (first || idle) {
#pragma unroll
          for (int i = 0; i < 16; ++i) w[i] = 0u;
        } else {
          tmem_ld16(to + 16 * c, w);
          tmem_wait_ld();
        }
      };
      // Output: w holds 16 dims of this thread's row, `inv` their factor
      T* const to_row = row_out(row0 + min(r, max(active - 1, 0))) + h * (D / 2);
      auto put = [&](int c, const uint32_t (&w)[16], float inv) {
        uint32_t v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          v[i] = Out::pack(__uint_as_float(w[2 * i]) * inv, __uint_as_float(w[2 * i + 1]) * inv);
        if (r < active) {
          reinterpret_cast<uint4*>(to_row)[2 * c] = make_uint4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<uint4*>(to_row)[2 * c + 1] = make_uint4(v[4], v[5], v[6], v[7]);
        }
      };
      // a part of a pair: into the workspace, 16 bytes of 32 rows side by side
      auto leave = [&](int c, const uint32_t (&w)[16]) {
        float4* dst = p.part_o + ((size_t)my_slot * (D / 4) + h * (D / 8) + 4 * c) * 256 + (dual ? 0 : 128 * x) + r;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          dst[(size_t)i * 256] = make_float4(__uint_as_float(w[4 * i]), __uint_as_float(w[4 * i + 1]),
                                             __uint_as_float(w[4 * i + 2]), __uint_as_float(w[4 * i + 3]));
      };
      auto leave_ml = [&](float m, float sum) {
        if (h == 0) p.part_ml[(size_t)my_slot * 256 + (dual ? 0 : 128 * x) + r] = make_float2(m, sum);
      };
      if (dual) {
        // B's part of the rows goes to A's warps through the place of B's query rows, warp by warp (2 KB
        // each, where that warp's own query rows come next): maxima and sums, then 16 dims at a time (16-byte chunk k of row r at k ^ (r / 2 & 3))
        float4* box = reinterpret_cast<float4*>(sm + S::kTile + (2 * w4 + h) * 2048) + lane * 4;
        uint64_t *full = &box_full[4 * h + w4], *empty = &box_empty[4 * h + w4];
        const int most = idle ? 0 : D / 32;
        float fa = 0.f, fb = 0.f, M = 0.f, total = 0.f;
#pragma unroll 1
        for (int c = -1; c < most; ++c, ++boxes) {
          uint32_t w[16];
          if (c >= 0) load_o(c, w);
          if (x == 1) {
            if (boxes > 0 && !bad && !wait(empty, (boxes + 1) & 1)) bad = true;
            if (c < 0) {
              box[0] = make_float4(m_use, l, 0.f, 0.f);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                *reinterpret_cast<uint4*>(box + (k ^ (lane >> 1 & 3))) =
                    make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(full);
            continue;
          }
          if (!bad && !wait(full, boxes & 1)) bad = true;
          if (c < 0) {
            const float4 b = box[0];
            M = fmaxf(m_use, b.x);
            const float nb = M == -INFINITY ? 0.f : M;
            fa = exp2f(m_use - nb), fb = exp2f(b.x - nb);
            total = l * fa + b.y * fb;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float4 o = box[k ^ (lane >> 1 & 3)];
              w[4 * k] = __float_as_uint(fmaf(o.x, fb, __uint_as_float(w[4 * k]) * fa));
              w[4 * k + 1] = __float_as_uint(fmaf(o.y, fb, __uint_as_float(w[4 * k + 1]) * fa));
              w[4 * k + 2] = __float_as_uint(fmaf(o.z, fb, __uint_as_float(w[4 * k + 2]) * fa));
              w[4 * k + 3] = __float_as_uint(fmaf(o.w, fb, __uint_as_float(w[4 * k + 3]) * fa));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(empty);
          if (c < 0 || bad) continue;
          if (whole)
            put(c, w, p.v_scale / total);
          else
            leave(c, w);
        }
        if (x == 1 && !bad && !wait(empty, (boxes + 1) & 1)) bad = true;  // the place is B's again
        if (x == 0 && !whole && !bad && !idle) leave_ml(M, total);
      } else if (!idle && !bad) {
        const float inv = p.v_scale / l;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          uint32_t w[16];
          load_o(c, w);
          if (whole)
            put(c, w, inv);
          else
            leave(c, w);
        }
        if (!whole) leave_ml(m_use, l);
      }
      tc_fence_before();
      if (more && !bad && dual) place_q(after);
    }
    if (bad && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_TIMEOUT);
    __syncwarp();
  }

  // ---- tear-down: copies have landed, MMAs have completed (bounded drains above) ------------
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tbase, kPwTmemCols);
  }
}

// Row `row` of a pair over q4_0 in 32 bits, by a warp: a token to a lane for the scores, D / 32 dims to a lane for
// the output. qs: room for the query row.
template <typename T, int D>
__device__ __forceinline__ void pq_wide_row(const PqParams& p, const PqPart& part, int row, float* qs) {
  constexpr int E = D / 32, kHalf = 16 / E, kRow = D / 16 * 9;  // values to a lane, lanes to a block's halves
  const int lane = threadIdx.x & 31, G = p.group;
  const int g = part.row0 + row, t = p.by_group.of(g), pos = part.base + t;
  const size_t at = ((size_t)(part.q0 + t) * p.num_heads + part.kvh * G + (g - t * G)) * D;
  const float factor = p.zero_scale ? 0.f : (p.flip != 0u ? -p.scale_log2 : p.scale_log2);
  for (int i = lane; i < D; i += 32) qs[i] = factor * static_cast<float>(static_cast<const T*>(p.q)[at + i]);
  __syncwarp();
  const int32_t* bt = p.block_tables + (size_t)part.s * p.max_blocks_per_seq;
  const int block = lane / (2 * kHalf), upper = lane / kHalf & 1;  // this lane's dims: E of half a block
  const int byte0 = D / 16 + 16 * block + E * (lane % kHalf);
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
#pragma unroll 1
  for (int t0 = 0; t0 <= pos; t0 += 32) {
    const int tok = t0 + lane;
    long long from = -1;  // this lane's row; a bad block's rows are zeros
    if (tok <= pos) {
      const int b = __ldg(bt + (tok >> p.block_bits));
      if (b >= 0 && b < p.num_blocks)
        from = (((long long)b * p.num_kv_heads + part.kvh) * p.block_size + (tok & (p.block_size - 1))) * kRow;
    }
    float x = tok <= pos ? 0.f : -INFINITY;
    if (from >= 0) {
      const unsigned char* k = p.k_cache + from;
#pragma unroll 1
      for (int b = 0; b < D / 32; ++b) {
        float sum = 0.f;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int code = k[D / 16 + 16 * b + i];
          sum = fmaf(qs[32 * b + i], (float)((code & 15) - 8), sum);
          sum = fmaf(qs[32 * b + 16 + i], (float)((code >> 4) - 8), sum);
        }
        x = fmaf(sum, __half2float(reinterpret_cast<const __half*>(k)[b]), x);
      }
    }
    float top = x;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, i));
    top = fmaxf(top, m);
    const float base = top == -INFINITY ? 0.f : top, keep = exp2f(m - base), w = exp2f(x - base);
    m = top;
    float total = w;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) total += __shfl_xor_sync(kFullMask, total, i);
    l = fmaf(l, keep, total);
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= keep;
    const int count = min(32, pos - t0 + 1);
#pragma unroll 1
    for (int i = 0; i < count; ++i) {
      const long long row_at = __shfl_sync(kFullMask, from, i);
      const float wi = __shfl_sync(kFullMask, w, i);
      if (row_at < 0) continue;
      const unsigned char* v = p.v_cache + row_at;
      const float wd = wi * __half2float(reinterpret_cast<const __half*>(v)[block]);
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] = fmaf(wd, (float)((v[byte0 + e] >> (4 * upper) & 15) - 8), o[e]);
    }
  }
  const float inv = p.v_scale / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + at + 32 * block + 16 * upper + E * (lane % kHalf));
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = PwPack<T>::pack(o[e] * inv, o[e + 1] * inv);
  __syncwarp();
}

// The pairs that start in this CTA's stretch and meet rows with values beyond binary16, whole or cut: all of their
// rows again, 32 to a CTA of the join. (8192 queries of 32 heads with such keys throughout: 184 ms instead of 0.48; a
// prompt of 1500 tokens, 10 heads of 64: 3.2 ms instead of 0.03.)
template <typename T, int D>
__device__ __noinline__ void pq_wide(const PqParams& p, float* qs) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  PqWalk walk;
  if (!pq_begin(p, walk)) return;
  for (; !walk.done(); walk.next(p)) {
    PqPart part;
    if (!walk.part(p, part) || !(part.whole() || (part.kind & PqPart::kHead))) continue;
    bool wide = false;
    for (int c = blockIdx.x + lane; c <= part.last; c += 32) wide |= __ldcg(&p.cuts[c].wide) != 0;
    if (!__any_sync(kFullMask, wide)) continue;
#pragma unroll 1
    for (int row = blockIdx.y * 32 + warp; row < min(blockIdx.y * 32 + 32, part.active); row += 2 * D / 32)
      pq_wide_row<T, D>(p, part, row, qs + warp * D);
  }
}

// The cut pairs' parts joined: grid = (CTA that a pair starts in, 32 rows of it), 16 head dims to a warp, a row to
// a lane; the parts come four at a time, so that their loads are under way together.
template <typename T, PqFormat F, int D>
__global__ void __launch_bounds__(2 * D) pa_prefill_quant_join_kernel(const __grid_constant__ PqParams p) {
  grid_dependency_wait();
  const int c0 = blockIdx.x;
  const int4 told = __ldcg(reinterpret_cast<const int4*>(p.cuts + c0));  // last, q0, kvh, row0
  const int active = __ldcg(&p.cuts[c0].active);
  const int c1 = told.x;
  if constexpr (F == PqFormat::kQ4) {
    __shared__ float qs[2 * D / 32 * D];
    bool wide = false;
    for (int c = c0 + (threadIdx.x & 31); c <= max(c0, c1); c += 32) wide |= __ldcg(&p.cuts[c].wide) != 0;
    if (__any_sync(kFullMask, wide)) {
      pq_wide<T, D>(p, qs);
      return;
    }
  }
  if (c1 < 0) return;
  const int row = blockIdx.y * 32 + (threadIdx.x & 31), k0 = threadIdx.x >> 5;
  if (row >= active) return;
  float M = -INFINITY, o[16], total = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
#pragma unroll 1
  for (int c = c0; c <= c1; c += 4) {
    float2 ml[4];
    float4 a[4][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e > c1) break;
      const size_t slot = (size_t)(c + e == c0 ? 2 * c0 + 1 : 2 * (c + e)) * 256;
      ml[e] = __ldcg(p.part_ml + slot + row);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[e][i] = __ldcg(p.part_o + slot * (D / 4) + (size_t)(4 * k0 + i) * 256 + row);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (c + e > c1 || ml[e].y == 0.f) continue;  // (0: nothing of the part is visible to the row)
      const float top = fmaxf(M, ml[e].x), nb = top == -INFINITY ? 0.f : top;
      const float keep = exp2f(M - nb), f = exp2f(ml[e].x - nb);
      M = top;
      total = fmaf(total, keep, ml[e].y * f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        o[4 * i] = fmaf(o[4 * i], keep, a[e][i].x * f), o[4 * i + 1] = fmaf(o[4 * i + 1], keep, a[e][i].y * f);
        o[4 * i + 2] = fmaf(o[4 * i + 2], keep, a[e][i].z * f), o[4 * i + 3] = fmaf(o[4 * i + 3], keep, a[e][i].w * f);
      }
    }
  }
  const float inv = p.v_scale / total;
  const int g = told.w + row, t = p.by_group.of(g);
  T* out = static_cast<T*>(p.out) +
           ((size_t)(told.y + t) * p.num_heads + told.z * p.group + (g - t * p.group)) * D + 16 * k0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    reinterpret_cast<uint4*>(out)[i] =
        make_uint4(PwPack<T>::pack(o[8 * i] * inv, o[8 * i + 1] * inv), PwPack<T>::pack(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                   PwPack<T>::pack(o[8 * i + 4] * inv, o[8 * i + 5] * inv),
                   PwPack<T>::pack(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
}

}  // namespace pkv
