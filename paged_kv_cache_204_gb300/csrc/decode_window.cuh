// Single-token attention over part of a paged context (sliding window and
// first tokens), or over all of it with every token's attention weight added
// to a score (sm_103a).
//
// Operations. For sequence s of L tokens, query head h and kv head g:
//   window   visible tokens t < L with t < sinks or t >= L - window;
//            out = sum over visible t of softmax(scale q . k_t) v_t
//   scores   every t < L is visible, the same output, and
//            score[s][g][t] += sum over the heads h of g of softmax(x_h)_t
//
// Work: one CTA per piece of a (sequence, kv head, head part) segment; a head
// part is up to 8 query heads of one kv head (16-bit caches) or up to 4 (32-bit
// caches), so a K/V row is read once for all of them. A segment's visible
// tokens are cut into aligned tiles of 16: first those of the sinks, then those
// of the window. A piece is a contiguous run of its tiles; warp w of the CTA
// takes the tiles w, w + 4, ... of the run. Each warp keeps its own running
// maximum, exponential sum and output (online softmax, base 2); the CTA joins its
// warps in shared memory, and the last CTA of a segment to finish joins the
// pieces in their order (log-sum-exp), all in one launch.
//
// Bound by memory: K and V of the visible tokens are read once, 4 to 32 operations to an
// element. What keeps the reads coming (GPU times of 128 sequences of up to 2048 tokens, 40
// heads, window 1000 / 64 sequences of up to 32768, 64 query and 8 kv heads, window
// 4096; bfloat16, head_dim 128):
//  - asynchronous copies into shared-memory rings, 16 KB a warp, two tiles deep, three CTAs
//    on an SM: 280 / 173 us. Three tiles and two CTAs: 288 / 180; rows from registers
//    straight into the MMAs: 290 / 185.
//  - pieces handed to the SMs as they come free, rather than one equal run of tiles per
//    resident CTA across the segments' borders (307 / 175, and 10.3 instead of 7.4 us for one
//    sequence): SMs differ in speed, and the start and the join of one CTA lie
//    under the loads of the two beside it.
//  - first pieces first and longest, so that the last ones to start are short: 173 -> 171,
//    and 8 sequences of up to 32768 with scores 4 us less of 147.
// 280 us are 7.1 TB/s and 171 us 6.4 (a plain copy runs at 6.8). One sequence of 7001
// tokens, window 1024: 7.4 us, the latency of table, rows, join and launch. 32-bit caches (16
// sequences of up to 32768, window 4096): 40 heads 384 us, 7.1 TB/s; 32 query and 8 kv heads 114 us,
// 4.8 TB/s, the queries and outputs of four heads in registers leaving two CTAs on an SM.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "tc.cuh"

namespace pkv {

constexpr int kWinWarps = 4;
constexpr int kWinThreads = kWinWarps * 32;
constexpr float kWinFirst = 1.7f;     // length of a segment's first piece over the mean
// Partial results (pieces x heads) that a workspace holds: kWinRowPieces for every query
// head, within these bounds (16 to 128 MB at head_dim 128). Where one sequence is far longer
// than the others it alone has to fill the GPU: 131072 tokens beside 127 sequences of
// 100 take 141 us with 32 pieces, 227 with 16, 406 with 8 (124 on their own).
constexpr int64_t kWinRowPieces = 32, kWinPiecesLeast = 32768, kWinPiecesMost = 262144;

struct WindowParams {
  void* out;
  const void* q;
  const void* k_cache;
  const void* v_cache;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float scale_log2;  // scale * log2(e)
  int window;        // >= 1; at least max_context_len: no window
  int sinks;         // >= 0
  int num_seqs, num_heads, num_kv_heads, group;
  int parts;       // head parts of one kv head
  int part_heads;  // query heads of a part (the last part may have fewer)
  int block_size, block_bits, max_blocks_per_seq, num_blocks, max_context_len;  // block_size = 2^block_bits
  int splits;        // pieces a segment may be cut into
  int min_tiles;     // tiles of a piece on average, at least (where the segment has as many)
  int32_t* counter;  // [segments], zero between calls (used where splits > 1)
  float2* piece_ml;  // [segments * splits][part_heads] (m, l)
  float* piece_o;    // [segments * splits][part_heads][D]
  float* logits;     // scores: [num_seqs][num_heads][logit_stride], base-2 logits
  int64_t logit_stride;
  float2* row_ml;    // scores: [num_seqs][num_heads] final (m, l)
  int32_t* dev_err;
};

struct ScoreParams {
  const float* logits;
  int64_t logit_stride;
  const float2* row_ml;
  const float* scores;  // may be null: zeros
  float* scores_out;
  int64_t score_stride;
  const int32_t* context_lens;
  int num_heads, num_kv_heads, group, cap;
};

// The tiles of a segment: [0, first) hold the sinks, then [from, end).
struct TileRange {
  int first, from, n;
  __device__ __forceinline__ int tile(int i) const { return i < first ? i : i - first + from; }
};

template <int TT>
__device__ __forceinline__ TileRange tiles_visible(int L, int window, int sinks) {
  TileRange r;
  const int end = (int)(((int64_t)L + TT - 1) / TT);
  const int lo = L > window ? L - window : 0;
  const int s = min(sinks, L);
  r.first = min((int)(((int64_t)s + TT - 1) / TT), end);
  r.from = max(lo / TT, r.first);
  r.n = r.first + (end - r.from);
  return r;
}

__device__ __forceinline__ int checked_len(const WindowParams& p, int s) {
  const int cap = (int)min((int64_t)p.max_context_len, (int64_t)p.max_blocks_per_seq * p.block_size);
  int L = __ldg(p.context_lens + s);
  if (L < 0 || L > cap) {
    if (threadIdx.x == 0) set_err(p.dev_err, PKV_DEV_ERR_CONTEXT_LEN);
    L = L < 0 ? 0 : cap;
  }
  return L;
}

// 16-byte asynchronous copy to shared memory, past L1.
__device__ __forceinline__ void copy16(uint32_t smem, const void* gmem) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem), "l"(gmem) : "memory");
}
// The same with `bytes` 16, or zeros (and nothing read) with 0.
__device__ __forceinline__ void copy16_or_zeros(uint32_t smem, const void* gmem, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the newest N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
  const __half2 h = __floats2half2_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __half) {
  __half2 h;
  memcpy(&h, &u, 4);
  return __half22float2(h);
}
__device__ __forceinline__ float2 unpack2(uint32_t u, __nv_bfloat16) {
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}

// 2^(x - m) where m may still be -inf (nothing but -inf seen so far): 0 then.
__device__ __forceinline__ float exp2_from(float x, float m) { return exp2f(x - (m == -INFINITY ? 0.f : m)); }

__device__ __forceinline__ bool token_seen(const WindowParams& p, int64_t tok, int L) {
  return tok < L && (tok < p.sinks || tok >= (int64_t)L - p.window);
}

// A warp's tiles of TT tokens, one after another, through a ring of kStages slots
// in shared memory (K rows, then V rows), filled by 16-byte asynchronous copies
// kStages - 1 tiles ahead. Nothing is waited for but the warp's own copies. A row
// of a tile in which a token is not visible reads as zeros, so that whatever its
// place holds never meets a product. 16-byte chunk c of row r lies at chunk
// position c ^ (r & 7) of its 128 bytes: eight rows' chunks c fall into
// eight different bank groups.
//
// The table entries of the tiles come 32 tiles at a time: lane i holds the blocks
// of the warp's tile 32 b + i, one for each 8 tokens. Blocks without a visible token are neither
// read nor checked: their entries may name blocks that were given back.
template <int TT, int ROW, int kStages>
struct TileRing {
  static constexpr int kIds = TT / 8;           // 8-token runs of a tile
  static constexpr int kTileBytes = TT * ROW;   // K or V
  static constexpr int kSlotBytes = 2 * kTileBytes;
  static constexpr int kBytes = kStages * kSlotBytes;
  static constexpr int CPR = ROW / 16;          // chunks of a row
  static constexpr int kPerRun = 8 * CPR / 32;  // copies of a lane for one run of K (or V)
  static_assert(CPR % 8 == 0 && 8 * CPR % 32 == 0, "rows of whole 128-byte lines");

  unsigned char* base;
  const int32_t* row;
  int id[kIds], next[kIds];
  int L, kvh, lane, step, end;   // end: of the tile indexes of the piece
  int issue_at, issued;          // next tile to copy, tiles copied so far
  TileRange r;

  __device__ __forceinline__ void fetch(const WindowParams& p, int i) {
#pragma unroll
    for (int k = 0; k < kIds; ++k) {
      next[k] = 0;
      if (i < end) {
        const int64_t t = (int64_t)r.tile(i) * TT + 8 * k;
        if (t < L && (t < p.sinks || t + 8 > (int64_t)L - p.window)) {
          int b = __ldg(row + (t >> p.block_bits));
          if (b < 0 || b >= p.num_blocks) {
            set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
            b = 0;
          }
          next[k] = b;
        }
      }
    }
  }

  // Tile issue_at into its slot; always commits a group.
  __device__ __forceinline__ void issue(const WindowParams& p) {
    if (issue_at < end) {
      if ((issued & 31) == 0) {
#pragma unroll
        for (int k = 0; k < kIds; ++k) id[k] = next[k];
        fetch(p, issue_at + (32 + lane) * step);
      }
      const int64_t t0 = (int64_t)r.tile(issue_at) * TT;
      const uint32_t slot = smem_u32(base) + (issued % kStages) * kSlotBytes;
      // the tile's tokens are all visible, or it is looked at row by row
      const bool full = t0 + TT <= L && (t0 + TT <= p.sinks || t0 >= (int64_t)L - p.window);
#pragma unroll
      for (int k = 0; k < kIds; ++k) {
        const int b = __shfl_sync(kFullMask, id[k], issued & 31);
        const int64_t t = t0 + 8 * k;
        const size_t at =
            (((size_t)b * p.num_kv_heads + kvh) * p.block_size + (size_t)(t & (p.block_size - 1))) * ROW + lane * 16;
        const char* kg = static_cast<const char*>(p.k_cache) + at;
        const char* vg = static_cast<const char*>(p.v_cache) + at;
#pragma unroll
        for (int j = 0; j < kPerRun; ++j) {
          const int e = j * 32 + lane, rr = e / CPR, c = e % CPR;
          const uint32_t to = slot + (8 * k + rr) * ROW + (c ^ (rr & 7)) * 16;
          if (full) {
            copy16(to, kg + j * 512);
            copy16(to + kTileBytes, vg + j * 512);
          } else {
            const int bytes = token_seen(p, t + rr, L) ? 16 : 0;
            copy16_or_zeros(to, kg + j * 512, bytes);
            copy16_or_zeros(to + kTileBytes, vg + j * 512, bytes);
          }
        }
      }
      issue_at += step;
      ++issued;
    }
    copies_commit();
  }

  __device__ __forceinline__ void start(const WindowParams& p, unsigned char* ring, int s, int kv_head, int length,
                                        const TileRange& range, int begin, int stop, int warp, int warps, int ln) {
    base = ring;
    row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    L = length;
    kvh = kv_head;
    r = range;
    lane = ln;
    step = warps;
    end = stop;
    issue_at = begin + warp;
    issued = 0;
    fetch(p, issue_at + lane * step);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(p);
  }
};

// ---- 16-bit caches: tensor-core tiles ----------------------------------------
// Tiles of 16 tokens through m16n8k16 MMAs (binary16 or bfloat16 operands, fp32
// accumulation): with at most 8 queries to a K/V row the work is bound by memory,
// and these take the rows as the cache holds them.
//
// Scores, S^T = K q^T: tokens are M, head dims K, query heads N. Output,
// O^T += V^T P^T: head dims are M, tokens K, query heads N; V^T comes from V rows by
// transposing matrix loads, P^T from the score layout by 8 x 8 transposes. Lane
// (g, t) = (lane / 4, lane % 4) ends with head dims 16 m + g and 16 m + g + 8 of
// the heads 2t, 2t + 1.
// P enters as a 16-bit high part and a 16-bit remainder, so that its rounding stays
// below the output's: 16 significant bits or more in bfloat16, 22 in binary16. That type's
// range is short, so its weights enter times 2^15 (the largest is 1): a weight
// above 2^-18 keeps all bits, and below that the error is 2^-40 of the largest weight, so that
// 2^20 tokens far below it lose no more than 2^-20 of the output. (As they are, weights below 2^-25
// would be 0 in both parts and full in the sum that divides.) With at most 4 heads the high parts fill columns 0-3 and the remainders columns 4-7 of
// one MMA (kWide false); with 5-8 heads they take two.
template <typename T, int D, bool kWide, bool kLogits>
struct MmaTile {
  static constexpr int TT = 16;
  static constexpr int kHeads = kWide ? 8 : 4;
  static constexpr int KS = D / 16;  // k-steps of the scores, m-tiles of the output
  static constexpr int ROW = D * 2;
  static constexpr int kStages = D == 128 ? 2 : 4;  // 16 KB of ring per warp, three CTAs on an SM
  static constexpr bool kTwoParts = true;  // weights in 16-bit parts
  static constexpr bool kScaled = std::is_same<T, __half>::value;
  static constexpr float kWeight = kScaled ? 32768.f : 1.f;  // factor of the weights in l and o until finish()
  using Ring = TileRing<TT, ROW, kStages>;

  uint32_t qf[KS][2];
  float m[2], l[2];  // heads 2t, 2t + 1 (of the lane's columns); l: this lane's tokens
  float o[KS][4];
  int heads, g, t;

  __device__ __forceinline__ void init(const WindowParams& p, int s, int h0, int nheads, int lane) {
    heads = nheads;
    g = lane >> 2;
    t = lane & 3;
    const int h = kWide ? g : (g & 3);
    const bool ok = h < nheads;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(static_cast<const char*>(p.q) +
                                                          ((size_t)s * p.num_heads + h0 + (ok ? h : 0)) * ROW);
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      qf[k][0] = ok ? __ldg(q + 8 * k + t) : 0u;
      qf[k][1] = ok ? __ldg(q + 8 * k + 4 + t) : 0u;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  // kExact: V in products with the 32-bit weights (see the kernel)
  template <bool kExact>
  __device__ __forceinline__ void consume(const WindowParams& p, int s, int h0, const unsigned char* slot, int64_t t0,
                                          int L, int lane) {
    const uint32_t ks = smem_u32(slot);
    // K fragments: lane i gives row i % 16, chunk 2 k + i / 16
    const uint32_t r = lane & 15, half = lane >> 4;
    float a[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      uint32_t f[4];
      ldsm_x4(ks + r * ROW + ((2 * k + half) ^ (r & 7)) * 16, f);
      mma_16816<T>(a[k & 1], f[0], f[1], f[2], f[3], qf[k][0], qf[k][1]);
    }
    float x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = token_seen(p, t0 + g + 8 * (i >> 1), L) ? (a[0][i] + a[1][i]) * p.scale_log2 : -INFINITY;
    if constexpr (kLogits) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = 2 * t + (i & 1);
        const int64_t tok = t0 + g + 8 * (i >> 1);
        if (h < heads && (kWide || t < 2) && tok < L)
          p.logits[((size_t)s * p.num_heads + h0 + h) * p.logit_stride + tok] = x[i];
      }
    }
    // running maximum and sums, then the P operand
    float pr[4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float mx = fmaxf(x[c], x[c + 2]);
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, off));
      const float mn = fmaxf(m[c], mx);
      const float alpha = exp2_from(m[c], mn);
      m[c] = mn;
      pr[c] = exp2_from(x[c], mn);
      pr[c + 2] = exp2_from(x[c + 2], mn);
      if constexpr (kScaled) {
        pr[c] *= kWeight;
        pr[c + 2] *= kWeight;
      }
      l[c] = l[c] * alpha + (pr[c] + pr[c + 2]);
      if (__any_sync(kFullMask, alpha != 1.f)) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          o[i][c] *= alpha;
          o[i][c + 2] *= alpha;
        }
      }
    }
    if constexpr (kExact) {
      const bool mine = kWide || t < 2;  // else the lane's columns are those of remainders
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll 1
        for (int r8 = 0; r8 < 8; ++r8) {
          const float p0 = __shfl_sync(kFullMask, pr[2 * half], 4 * r8 + t);
          const float p1 = __shfl_sync(kFullMask, pr[2 * half + 1], 4 * r8 + t);
          const unsigned char* row = slot + Ring::kTileBytes + (8 * half + r8) * ROW;
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // dims 16 i + g and 16 i + g + 8
              const float v =
                  static_cast<float>(reinterpret_cast<const T*>(row + (((2 * i + e) ^ r8) * 16))[g]);
              if (mine) {
                o[i][2 * e] = fmaf(p0, v, o[i][2 * e]);
                o[i][2 * e + 1] = fmaf(p1, v, o[i][2 * e + 1]);
              }
            }
        }
    } else {
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int v = 0; v < 2; ++v) {
        const uint32_t h = pack2(pr[2 * v], pr[2 * v + 1], T());
        const float2 f = unpack2(h, T());
        const uint32_t rest = pack2(pr[2 * v] - f.x, pr[2 * v + 1] - f.y, T());
        if constexpr (kWide) {
          hi[v] = transpose8x8(h);
          lo[v] = transpose8x8(rest);
        } else {
          hi[v] = transpose8x8(t < 2 ? h : rest);
        }
      }
      // V^T fragments: matrices (dims 0-7, tokens 0-7), (dims 8-15, tokens 0-7), then
      // tokens 8-15; lane i gives token row i % 8 + 8 (i / 16), chunk 2 m + (i / 8) % 2
      const uint32_t vr = (lane & 7) + 8 * (lane >> 4), vc = (lane >> 3) & 1;
      const uint32_t vs = ks + Ring::kTileBytes + vr * ROW;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) {
        uint32_t f[4];
        ldsm_x4_trans(vs + ((2 * mt + vc) ^ (vr & 7)) * 16, f);
        mma_16816<T>(o[mt], f[0], f[1], f[2], f[3], hi[0], hi[1]);
        if constexpr (kWide) mma_16816<T>(o[mt], f[0], f[1], f[2], f[3], lo[0], lo[1]);
      }
    }
  }

  // This warp's result to shared memory: sm_o [kHeads][D], sm_ml [kHeads].
  __device__ __forceinline__ void finish(float* sm_o, float2* sm_ml) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) l[c] += __shfl_xor_sync(kFullMask, l[c], off);
    }
    if constexpr (!kWide) {  // high part plus remainder: columns 2t and 2t + 4
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += __shfl_xor_sync(kFullMask, o[i][e], 2);
    }
    if constexpr (kScaled) {  // a power of two: exact
      l[0] *= 1.f / kWeight, l[1] *= 1.f / kWeight;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= 1.f / kWeight;
    }
    if (kWide || t < 2) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 2 * t + c;
        if (g == 0) sm_ml[h] = make_float2(m[c], l[c]);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          sm_o[h * D + 16 * i + g] = o[i][c];
          sm_o[h * D + 16 * i + g + 8] = o[i][c + 2];
        }
      }
    }
  }
};

// ---- 32-bit caches: fp32 FMAs -------------------------------------------------
// Lanes form 4 groups of 8; a group takes every fourth row of the tile and lane
// `sub` of it the 16-byte chunks sub, sub + 8, ... of the row. q . k is summed
// over the group with shuffles.
template <int D, int kPart, bool kLogits>
struct FmaTile {
  static constexpr int TT = D == 128 ? 8 : 16;  // 8 KB of K and V rows
  static constexpr int RPG = TT / 4;            // rows of a tile per group
  static constexpr int kHeads = kPart;
  static constexpr bool kTwoParts = false;
  static constexpr int NC = D / 32;  // chunks of a row per lane
  static constexpr int ROW = D * 4;
  static constexpr int kStages = 2;
  using Ring = TileRing<TT, ROW, kStages>;

  float qf[kPart][NC * 4], o[kPart][NC * 4];
  float m[kPart], l[kPart];
  int heads, grp, sub;

  __device__ __forceinline__ void init(const WindowParams& p, int s, int h0, int nheads, int lane) {
    heads = nheads;
    grp = lane >> 3;
    sub = lane & 7;
#pragma unroll
    for (int h = 0; h < kPart; ++h) {
      const bool ok = h < nheads;
      const float4* q =
          reinterpret_cast<const float4*>(p.q) + ((size_t)s * p.num_heads + h0 + (ok ? h : 0)) * (D / 4);
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 u = ok ? __ldg(q + sub + 8 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
        qf[h][4 * c] = u.x, qf[h][4 * c + 1] = u.y, qf[h][4 * c + 2] = u.z, qf[h][4 * c + 3] = u.w;
      }
      m[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int e = 0; e < NC * 4; ++e) o[h][e] = 0.f;
    }
  }

  __device__ __forceinline__ float4 chunk(const unsigned char* rows, int r, int c) const {
    return *reinterpret_cast<const float4*>(rows + r * ROW + ((sub + 8 * c) ^ (r & 7)) * 16);
  }

  template <bool>
  __device__ __forceinline__ void consume(const WindowParams& p, int s, int h0, const unsigned char* slot, int64_t t0,
                                          int L, int) {
    bool ok[RPG];
    float x[kPart][RPG];
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
      const int r = 4 * j + grp;
      ok[j] = token_seen(p, t0 + r, L);
      float4 k[NC];
#pragma unroll
      for (int c = 0; c < NC; ++c) k[c] = chunk(slot, r, c);
#pragma unroll
      for (int h = 0; h < kPart; ++h) {
        float a = 0.f;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          a = fmaf(qf[h][4 * c], k[c].x, a);
          a = fmaf(qf[h][4 * c + 1], k[c].y, a);
          a = fmaf(qf[h][4 * c + 2], k[c].z, a);
          a = fmaf(qf[h][4 * c + 3], k[c].w, a);
        }
        a += __shfl_xor_sync(kFullMask, a, 1);
        a += __shfl_xor_sync(kFullMask, a, 2);
        a += __shfl_xor_sync(kFullMask, a, 4);
        x[h][j] = ok[j] ? a * p.scale_log2 : -INFINITY;
        if constexpr (kLogits) {
          if (sub == 0 && h < heads && t0 + r < L)
            p.logits[((size_t)s * p.num_heads + h0 + h) * p.logit_stride + t0 + r] = x[h][j];
        }
      }
    }
#pragma unroll
    for (int h = 0; h < kPart; ++h) {
      float mx = x[h][0];
#pragma unroll
      for (int j = 1; j < RPG; ++j) mx = fmaxf(mx, x[h][j]);
      mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, 16));
      const float mn = fmaxf(m[h], mx);
      const float alpha = exp2_from(m[h], mn);
      m[h] = mn;
      l[h] *= alpha;
#pragma unroll
      for (int e = 0; e < NC * 4; ++e) o[h][e] *= alpha;
#pragma unroll
      for (int j = 0; j < RPG; ++j) {
        x[h][j] = exp2_from(x[h][j], mn);
        l[h] += x[h][j];
      }
    }
#pragma unroll
    for (int j = 0; j < RPG; ++j) {
      const int r = 4 * j + grp;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 v = chunk(slot + Ring::kTileBytes, r, c);
#pragma unroll
        for (int h = 0; h < kPart; ++h) {
          o[h][4 * c] = fmaf(x[h][j], v.x, o[h][4 * c]);
          o[h][4 * c + 1] = fmaf(x[h][j], v.y, o[h][4 * c + 1]);
          o[h][4 * c + 2] = fmaf(x[h][j], v.z, o[h][4 * c + 2]);
          o[h][4 * c + 3] = fmaf(x[h][j], v.w, o[h][4 * c + 3]);
        }
      }
    }
  }

  __device__ __forceinline__ void finish(float* sm_o, float2* sm_ml) {
#pragma unroll
    for (int h = 0; h < kPart; ++h) {
      l[h] += __shfl_xor_sync(kFullMask, l[h], 8);
      l[h] += __shfl_xor_sync(kFullMask, l[h], 16);
#pragma unroll
      for (int e = 0; e < NC * 4; ++e) {
        o[h][e] += __shfl_xor_sync(kFullMask, o[h][e], 8);
        o[h][e] += __shfl_xor_sync(kFullMask, o[h][e], 16);
      }
      if (grp == 0) {
        if (sub == 0) sm_ml[h] = make_float2(m[h], l[h]);
#pragma unroll
        for (int c = 0; c < NC; ++c)
          *reinterpret_cast<float4*>(sm_o + h * D + 4 * (sub + 8 * c)) =
              make_float4(o[h][4 * c], o[h][4 * c + 1], o[h][4 * c + 2], o[h][4 * c + 3]);
      }
    }
  }
};

template <typename T>
__device__ __forceinline__ void store4(T* p, float a, float b, float c, float d) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(a, b, T()), pack2(c, d, T()));
  }
}

// Join of partial results (m_j, l_j, o_j): M = max m_j, l = sum l_j 2^(m_j - M),
// o = sum o_j 2^(m_j - M); an empty part has m_j = -inf, l_j = 0 and o_j = 0.
struct Join {
  float l, a[4];
  __device__ __forceinline__ void clear() { l = a[0] = a[1] = a[2] = a[3] = 0.f; }
  __device__ __forceinline__ void add(float2 ml, float4 o, float M) {
    const float f = exp2_from(ml.x, M);
    l += ml.y * f;
    a[0] = fmaf(o.x, f, a[0]), a[1] = fmaf(o.y, f, a[1]), a[2] = fmaf(o.z, f, a[2]), a[3] = fmaf(o.w, f, a[3]);
  }
};

template <typename T, int D, typename Tile, bool kLogits>
__global__ void __launch_bounds__(kWinThreads) pa_window_kernel(const WindowParams p) {
  constexpr int HP = Tile::kHeads;
  using Ring = typename Tile::Ring;
  extern __shared__ __align__(128) unsigned char rings[];  // one per warp; its result replaces it at the end
  __shared__ float2 sm_ml[kWinWarps][HP];
  __shared__ int sm_last;
  static_assert(Ring::kBytes >= HP * D * (int)sizeof(float), "room for a warp's result");
  if constexpr (kLogits) grid_launch_dependents();

  const int segments = p.num_seqs * p.num_kv_heads * p.parts;
  const int piece = blockIdx.x / segments;
  const int seg = blockIdx.x - piece * segments;
  const int part = seg % p.parts;
  const int kvh = (seg / p.parts) % p.num_kv_heads;
  const int s = seg / p.parts / p.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = kvh * p.group + part * p.part_heads;
  const int heads = min(p.part_heads, p.group - part * p.part_heads);
  const int L = checked_len(p, s);
  const TileRange r = tiles_visible<Tile::TT>(L, p.window, p.sinks);
  // pieces of this segment: min_tiles or more on average (the last are shorter, and may have no
  // tile at all: then m = -inf and nothing is added)
  const int pieces = max(1, min(p.splits, r.n / p.min_tiles));
  if (piece >= pieces) return;
  // in whole rounds of the warps
  const int rounds = (r.n + kWinWarps - 1) / kWinWarps;
  // The lengths fall linearly, from kWinFirst to 2 - kWinFirst of their mean. One CTA's end
  // has to be the next one's begin, so no operation may be fused into another.
  auto cut = [&](int j) {
    const float x = __fdiv_rn((float)j, (float)pieces);
    const float part = __fmul_rn(x, __fsub_rn(kWinFirst, __fmul_rn(kWinFirst - 1.f, x)));
    return j == pieces ? rounds : (int)__fmul_rn((float)rounds, part);
  };
  const int begin = cut(piece) * kWinWarps, end = min(cut(piece + 1) * kWinWarps, r.n);

  unsigned char* mine = rings + warp * Ring::kBytes;
  Tile tile;
  auto walk = [&](auto exact) {
    Ring ring;
    ring.start(p, mine, s, kvh, L, r, begin, end, warp, kWinWarps, lane);
    tile.init(p, s, h0, heads, lane);
    for (int i = begin + warp, n = 0; i < end; i += kWinWarps, ++n) {
      copies_wait<Tile::kStages - 2>();
      __syncwarp();  // tile n has landed for all lanes, and all are done with the slot refilled now
      ring.issue(p);
      tile.template consume<decltype(exact)::value>(p, s, h0, mine + (n % Tile::kStages) * Ring::kSlotBytes,
                                                    (int64_t)r.tile(i) * Tile::TT, L, lane);
    }
    __syncwarp();
    tile.finish(reinterpret_cast<float*>(mine), sm_ml[warp]);
    __syncthreads();
  };

  // join the warps: a thread takes 4 dims of a head. True where an output is a NaN and its weights are not.
  T* out = static_cast<T*>(p.out) + ((size_t)s * p.num_heads + h0) * D;
  const size_t first = (size_t)seg * p.splits * p.part_heads;
  const size_t slot = first + (size_t)piece * p.part_heads;
  auto join = [&]() {
    bool nan = false;
    for (int i = threadIdx.x; i < heads * (D / 4); i += kWinThreads) {
      const int h = i / (D / 4), d = 4 * (i % (D / 4));
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWinWarps; ++w) M = fmaxf(M, sm_ml[w][h].x);
      Join t;
      t.clear();
#pragma unroll
      for (int w = 0; w < kWinWarps; ++w)
        t.add(sm_ml[w][h], reinterpret_cast<const float4*>(rings + w * Ring::kBytes)[(h * D + d) / 4], M);
      const float all = (t.a[0] + t.a[1]) + (t.a[2] + t.a[3]);
      nan |= all != all && t.l == t.l;
      if (pieces == 1) {
        // no token: zeros; a row whose every logit is -inf: 0 / 0, as the formula has it
        const float inv = L > 0 ? 1.f / t.l : 0.f;
        store4(out + h * D + d, t.a[0] * inv, t.a[1] * inv, t.a[2] * inv, t.a[3] * inv);
        if (kLogits && d == 0) p.row_ml[(size_t)s * p.num_heads + h0 + h] = make_float2(M, t.l);
      } else {
        __stcg(reinterpret_cast<float4*>(p.piece_o + (slot + h) * D + d), make_float4(t.a[0], t.a[1], t.a[2], t.a[3]));
        if (d == 0) __stcg(p.piece_ml + slot + h, make_float2(M, t.l));
      }
    }
    return nan;
  };
  walk(std::false_type());
  const bool nan = join();
  if constexpr (Tile::kTwoParts) {
    if (__syncthreads_or(nan)) {
      // A remainder of 0, or below 0, times an infinity in V is a NaN where the weight itself gives
      // infinity: the tiles once more with the weights as they are, slowly.
      walk(std::true_type());
      join();
    }
  }
  if (pieces == 1) return;

  // the last piece of the segment joins them all
  __syncthreads();  // the partial's writes precede the release below
  if (threadIdx.x == 0) {
    const int prev = atomic_add_acq_rel_gpu(p.counter + seg, 1);
    sm_last = prev == pieces - 1;
    if (prev == pieces - 1) p.counter[seg] = 0;  // all have counted: zero for the next call
  }
  __syncthreads();
  if (!sm_last) return;
  for (int i = threadIdx.x; i < heads * (D / 4); i += kWinThreads) {
    const int h = i / (D / 4), d = 4 * (i % (D / 4));
    float M = -INFINITY;
#pragma unroll 8
    for (int j = 0; j < pieces; ++j) M = fmaxf(M, __ldcg(p.piece_ml + first + (size_t)j * p.part_heads + h).x);
    Join t;
    t.clear();
#pragma unroll 8
    for (int j = 0; j < pieces; ++j) {
      const size_t at = first + (size_t)j * p.part_heads + h;
      t.add(__ldcg(p.piece_ml + at), __ldcg(reinterpret_cast<const float4*>(p.piece_o + at * D + d)), M);
    }
    const float inv = 1.f / t.l;
    store4(out + h * D + d, t.a[0] * inv, t.a[1] * inv, t.a[2] * inv, t.a[3] * inv);
    if (kLogits && d == 0) p.row_ml[(size_t)s * p.num_heads + h0 + h] = make_float2(M, t.l);
  }
}

using WindowLauncher = cudaError_t (*)(const WindowParams&, cudaStream_t);

// 16-bit (is_bf16) and 32-bit caches; part_heads picks the variant.
WindowLauncher window_launcher_16(int is_bf16, int head_dim, int part_heads, bool logits);
WindowLauncher window_launcher_f32(int head_dim, int part_heads, bool logits);
cudaError_t launch_add_scores(const ScoreParams& p, int num_seqs, int max_context_len, cudaStream_t stream);

}  // namespace pkv
