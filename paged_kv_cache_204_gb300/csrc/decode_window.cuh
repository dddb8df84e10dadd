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
// tokens are cut into aligned tiles of kTile tokens: first those of the sinks,
// then those of the window. A piece is a contiguous run of its tiles; warp w
// of the CTA takes the tiles w, w + 4, ... of the run. Each warp keeps its own
// running maximum, exponential sum and output (online softmax, base 2); the
// CTA joins its warps in shared memory, and the last CTA of a segment to
// finish joins the pieces (log-sum-exp), all in one launch.
#pragma once

#include <type_traits>

#include "common.cuh"
#include "tc.cuh"

namespace pkv {

constexpr int kWinWarps = 4;
constexpr int kWinThreads = kWinWarps * 32;
constexpr int kWinMaxPieces = 2048;  // pieces of split segments that a workspace holds

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
  int block_size, max_blocks_per_seq, num_blocks, max_context_len;
  int splits;        // pieces a segment may be cut into
  int min_tiles;     // tiles a piece has at least (where the segment has as many)
  int32_t* counter;  // [segments], zero between calls (splits > 1)
  float2* piece_ml;  // [segments * splits][8] (m, l)
  float* piece_o;    // [segments * splits][8][D], o / l
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

// A streaming 16-byte read: used once, so it takes no room in L1.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
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

// Physical blocks of a warp's tiles, fetched 32 tiles at a time: lane i holds
// those of the warp's tile 32 b + i, one block for each 8 tokens of the tile's
// first 16 (a tile lies in one block when the block is as long as the tile).
// Blocks without a visible token are neither read nor checked: their table
// entries may name blocks that were given back.
template <int TT>
struct TileBlocks {
  static constexpr int kIds = TT / 8;  // 8-token runs of a tile
  int id[kIds], next[kIds];

  __device__ __forceinline__ void fetch(const WindowParams& p, const int32_t* row, const TileRange& r, int L, int i,
                                        int end) {
#pragma unroll
    for (int k = 0; k < kIds; ++k) {
      next[k] = 0;
      if (i < end) {
        const int64_t t = (int64_t)r.tile(i) * TT + 8 * k;
        if (t < L && (t < p.sinks || t + 8 > (int64_t)L - p.window)) {
          int b = __ldg(row + t / p.block_size);
          if (b < 0 || b >= p.num_blocks) {
            set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
            b = 0;
          }
          next[k] = b;
        }
      }
    }
  }
  __device__ __forceinline__ void advance() {
#pragma unroll
    for (int k = 0; k < kIds; ++k) id[k] = next[k];
  }
};

// ---- 16-bit caches: tensor-core tiles ----------------------------------------
// Tiles of 16 tokens, read from global memory straight into the registers that
// feed m16n8k16 MMAs (binary16 or bfloat16 operands, fp32 accumulation): a row
// is used by one warp only, so shared memory would only add a copy.
//
// Scores, S^T = K q^T: tokens are M, head dims K, query heads N. The head dims
// are permuted alike in K and q, which leaves the product as it is: lane
// (g, t) = (lane / 4, lane % 4) takes 16-byte chunks t, t + 4, ... of token
// rows g and g + 8, so the four lanes of a row read 64 contiguous bytes, and of
// the row of head g. Words 0, 1 of a chunk make one k-step, words 2, 3 the next.
// Output, O^T += V^T P^T: head dims are M, tokens K, query heads N. Lane (g, t)
// reads chunks g, g + 8 of token rows 2t, 2t + 1, 2t + 8, 2t + 9; word w of a
// chunk makes one m-tile, its low half row g and its high half row g + 8.
// P^T comes from the score layout by 8 x 8 transposes.
// P enters as a 16-bit high part and a 16-bit remainder (16 significant bits or
// more with either type), so that its rounding stays below the output's. With at most 4
// heads the high parts fill columns 0-3 and the remainders columns 4-7 of one
// MMA (kWide false); with 5-8 heads they take two.
template <typename T, int D, bool kWide, bool kLogits>
struct MmaTile {
  static constexpr int TT = 16;
  static constexpr int kHeads = kWide ? 8 : 4;
  static constexpr int NC = D / 32;  // chunks of a K row per lane
  static constexpr int NV = D / 64;  // chunks of a V row per lane
  static constexpr int ROW = D * 2;

  uint32_t qf[NC][4];
  float m[2], l[2];       // heads 2t, 2t + 1 (of the lane's columns); l: this lane's tokens
  float o[NV * 4][4];
  uint4 kr[2][NC], vr[4][NV];
  int heads, g, t;

  __device__ __forceinline__ void init(const WindowParams& p, int s, int h0, int nheads, int lane) {
    heads = nheads;
    g = lane >> 2;
    t = lane & 3;
    const int h = kWide ? g : (g & 3);
    const bool ok = h < nheads;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p.q) +
                                                    ((size_t)s * p.num_heads + h0 + (ok ? h : 0)) * ROW);
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const uint4 u = ok ? __ldg(q + t + 4 * c) : make_uint4(0u, 0u, 0u, 0u);
      qf[c][0] = u.x, qf[c][1] = u.y, qf[c][2] = u.z, qf[c][3] = u.w;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int i = 0; i < NV * 4; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  }

  static __device__ __forceinline__ bool seen(const WindowParams& p, int64_t tok, int L) {
    return tok < L && (tok < p.sinks || tok >= (int64_t)L - p.window);
  }

  __device__ __forceinline__ void load_k(const WindowParams& p, int kvh, int64_t t0, int L, int b0, int b1) {
    const char* base = static_cast<const char*>(p.k_cache);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t tok = t0 + g + 8 * i;
      const bool ok = seen(p, tok, L);
      const char* row = base + (((size_t)(i ? b1 : b0) * p.num_kv_heads + kvh) * p.block_size +
                                (int)(tok & (p.block_size - 1))) * ROW;
#pragma unroll
      for (int c = 0; c < NC; ++c) kr[i][c] = ok ? ld_stream(row + 16 * (t + 4 * c)) : make_uint4(0u, 0u, 0u, 0u);
    }
  }
  __device__ __forceinline__ void load_v(const WindowParams& p, int kvh, int64_t t0, int L, int b0, int b1) {
    const char* base = static_cast<const char*>(p.v_cache);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t tok = t0 + 2 * t + (i & 1) + 8 * (i >> 1);
      const bool ok = seen(p, tok, L);
      const char* row = base + (((size_t)(i >> 1 ? b1 : b0) * p.num_kv_heads + kvh) * p.block_size +
                                (int)(tok & (p.block_size - 1))) * ROW;
#pragma unroll
      for (int c = 0; c < NV; ++c) vr[i][c] = ok ? ld_stream(row + 16 * (g + 8 * c)) : make_uint4(0u, 0u, 0u, 0u);
    }
  }

  // Scores of the tile in kr, as base-2 logits; masked tokens -inf.
  __device__ __forceinline__ void scores(const WindowParams& p, int64_t t0, int L, float (&x)[4]) {
    float a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      mma_16816<T>(a, kr[0][c].x, kr[1][c].x, kr[0][c].y, kr[1][c].y, qf[c][0], qf[c][1]);
      mma_16816<T>(a, kr[0][c].z, kr[1][c].z, kr[0][c].w, kr[1][c].w, qf[c][2], qf[c][3]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = seen(p, t0 + g + 8 * (i >> 1), L) ? a[i] * p.scale_log2 : -INFINITY;
  }

  __device__ __forceinline__ void store_logits(const WindowParams& p, int s, int h0, int64_t t0, int L,
                                               const float (&x)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int h = 2 * t + (i & 1);
      const int64_t tok = t0 + g + 8 * (i >> 1);
      if (h < heads && (kWide || t < 2) && tok < L)
        p.logits[((size_t)s * p.num_heads + h0 + h) * p.logit_stride + tok] = x[i];
    }
  }

  // Running maximum and sums, then the P operand of the tile.
  __device__ __forceinline__ void softmax(const float (&x)[4], uint32_t (&hi)[2], uint32_t (&lo)[2]) {
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
      l[c] = l[c] * alpha + (pr[c] + pr[c + 2]);
#pragma unroll
      for (int i = 0; i < NV * 4; ++i) {
        o[i][c] *= alpha;
        o[i][c + 2] *= alpha;
      }
    }
#pragma unroll
    for (int v = 0; v < 2; ++v) {
      const uint32_t h = pack2(pr[2 * v], pr[2 * v + 1], T());
      const float2 f = unpack2(h, T());
      const uint32_t r = pack2(pr[2 * v] - f.x, pr[2 * v + 1] - f.y, T());
      if constexpr (kWide) {
        hi[v] = transpose8x8(h);
        lo[v] = transpose8x8(r);
      } else {
        hi[v] = transpose8x8(t < 2 ? h : r);
      }
    }
  }

  __device__ __forceinline__ void accumulate(const uint32_t (&hi)[2], const uint32_t (&lo)[2]) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const uint32_t* r0 = reinterpret_cast<const uint32_t*>(&vr[0][c]);
      const uint32_t* r1 = reinterpret_cast<const uint32_t*>(&vr[1][c]);
      const uint32_t* r2 = reinterpret_cast<const uint32_t*>(&vr[2][c]);
      const uint32_t* r3 = reinterpret_cast<const uint32_t*>(&vr[3][c]);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t a0 = __byte_perm(r0[w], r1[w], 0x5410), a1 = __byte_perm(r0[w], r1[w], 0x7632);
        const uint32_t a2 = __byte_perm(r2[w], r3[w], 0x5410), a3 = __byte_perm(r2[w], r3[w], 0x7632);
        mma_16816<T>(o[4 * c + w], a0, a1, a2, a3, hi[0], hi[1]);
        if constexpr (kWide) mma_16816<T>(o[4 * c + w], a0, a1, a2, a3, lo[0], lo[1]);
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
      for (int i = 0; i < NV * 4; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] += __shfl_xor_sync(kFullMask, o[i][e], 2);
    }
    if (kWide || t < 2) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int h = 2 * t + c;
        if (g == 0) sm_ml[h] = make_float2(m[c], l[c]);
#pragma unroll
        for (int n = 0; n < NV; ++n)
#pragma unroll
          for (int w = 0; w < 4; ++w)
            *reinterpret_cast<float2*>(sm_o + h * D + (g + 8 * n) * 8 + 2 * w) =
                make_float2(o[4 * n + w][c], o[4 * n + w][c + 2]);
      }
    }
  }

  // One tile after another; the next tile's K rows are asked for as soon as
  // this tile's have been used, the V rows likewise.
  __device__ __forceinline__ void walk(const WindowParams& p, int s, int kvh, int h0, int L, const TileRange& r,
                                       int begin, int end, int warp, int lane) {
    const int32_t* row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    TileBlocks<TT> tb;
    int i = begin + warp;
    if (i >= end) return;
    tb.fetch(p, row, r, L, i + lane * kWinWarps, end);
    tb.advance();
    tb.fetch(p, row, r, L, i + (32 + lane) * kWinWarps, end);
    int64_t t0 = (int64_t)r.tile(i) * TT;
    int b0 = __shfl_sync(kFullMask, tb.id[0], 0), b1 = __shfl_sync(kFullMask, tb.id[1], 0);
    load_k(p, kvh, t0, L, b0, b1);
    load_v(p, kvh, t0, L, b0, b1);
    for (int n = 1;; ++n) {
      const int in = i + kWinWarps;
      const bool more = in < end;
      int64_t t1 = t0;
      if (more) {
        if ((n & 31) == 0) {
          tb.advance();
          tb.fetch(p, row, r, L, in + (32 + lane) * kWinWarps, end);
        }
        t1 = (int64_t)r.tile(in) * TT;
        b0 = __shfl_sync(kFullMask, tb.id[0], n & 31);
        b1 = __shfl_sync(kFullMask, tb.id[1], n & 31);
      }
      float x[4];
      scores(p, t0, L, x);
      if (more) load_k(p, kvh, t1, L, b0, b1);
      if constexpr (kLogits) store_logits(p, s, h0, t0, L, x);
      uint32_t hi[2], lo[2];
      softmax(x, hi, lo);
      accumulate(hi, lo);
      if (!more) break;
      load_v(p, kvh, t1, L, b0, b1);
      i = in;
      t0 = t1;
    }
  }
};

// ---- 32-bit caches: fp32 FMAs -------------------------------------------------
// Lanes form 4 groups of 8; a group takes every fourth row of the tile and lane
// `sub` of it the 16-byte chunks sub, sub + 8, ... of the row. q . k is summed
// over the group with shuffles.
template <int D, int kPart, bool kLogits>
struct FmaTile {
  static constexpr int RPG = D == 128 ? 2 : 4;  // rows of a tile per group
  static constexpr int TT = 16;                 // two steps of 8 tokens at head_dim 128
  static constexpr int kSteps = TT / (4 * RPG);
  static constexpr int kHeads = kPart;
  static constexpr int NC = D / 32;  // chunks of a row per lane
  static constexpr int ROW = D * 4;

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

  __device__ __forceinline__ void walk(const WindowParams& p, int s, int kvh, int h0, int L, const TileRange& r,
                                       int begin, int end, int warp, int lane) {
    const int32_t* row = p.block_tables + (size_t)s * p.max_blocks_per_seq;
    TileBlocks<TT> tb;
    if (begin + warp >= end) return;
    tb.fetch(p, row, r, L, begin + warp + lane * kWinWarps, end);
    for (int i = begin + warp, n = 0; i < end; i += kWinWarps, ++n) {
      if ((n & 31) == 0) {
        tb.advance();
        tb.fetch(p, row, r, L, i + (32 + lane) * kWinWarps, end);
      }
      const int b0 = __shfl_sync(kFullMask, tb.id[0], n & 31), b1 = __shfl_sync(kFullMask, tb.id[1], n & 31);
#pragma unroll
      for (int st = 0; st < kSteps; ++st) {
        const int64_t t0 = (int64_t)r.tile(i) * TT + st * 4 * RPG;
        float4 kr[RPG][NC], vr[RPG][NC];
        bool ok[RPG];
#pragma unroll
        for (int j = 0; j < RPG; ++j) {
          const int64_t tok = t0 + 4 * j + grp;
          ok[j] = tok < L && (tok < p.sinks || tok >= (int64_t)L - p.window);
          const int b = (tok & 8) ? b1 : b0;
          const size_t at =
              (((size_t)b * p.num_kv_heads + kvh) * p.block_size + (int)(tok & (p.block_size - 1))) * ROW;
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            uint4 u = make_uint4(0u, 0u, 0u, 0u), v = u;
            if (ok[j]) {
              u = ld_stream(static_cast<const char*>(p.k_cache) + at + 16 * (sub + 8 * c));
              v = ld_stream(static_cast<const char*>(p.v_cache) + at + 16 * (sub + 8 * c));
            }
            memcpy(&kr[j][c], &u, 16);
            memcpy(&vr[j][c], &v, 16);
          }
        }
#pragma unroll
        for (int h = 0; h < kPart; ++h) {
          float x[RPG], mx = -INFINITY;
#pragma unroll
          for (int j = 0; j < RPG; ++j) {
            float a = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              a = fmaf(qf[h][4 * c], kr[j][c].x, a);
              a = fmaf(qf[h][4 * c + 1], kr[j][c].y, a);
              a = fmaf(qf[h][4 * c + 2], kr[j][c].z, a);
              a = fmaf(qf[h][4 * c + 3], kr[j][c].w, a);
            }
            a += __shfl_xor_sync(kFullMask, a, 1);
            a += __shfl_xor_sync(kFullMask, a, 2);
            a += __shfl_xor_sync(kFullMask, a, 4);
            x[j] = ok[j] ? a * p.scale_log2 : -INFINITY;
            mx = fmaxf(mx, x[j]);
            if constexpr (kLogits) {
              const int64_t tok = t0 + 4 * j + grp;
              if (sub == 0 && h < heads && tok < L)
                p.logits[((size_t)s * p.num_heads + h0 + h) * p.logit_stride + tok] = x[j];
            }
          }
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
            const float w = exp2_from(x[j], mn);
            l[h] += w;
#pragma unroll
            for (int c = 0; c < NC; ++c) {
              o[h][4 * c] = fmaf(w, vr[j][c].x, o[h][4 * c]);
              o[h][4 * c + 1] = fmaf(w, vr[j][c].y, o[h][4 * c + 1]);
              o[h][4 * c + 2] = fmaf(w, vr[j][c].z, o[h][4 * c + 2]);
              o[h][4 * c + 3] = fmaf(w, vr[j][c].w, o[h][4 * c + 3]);
            }
          }
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

// Join of n partial results (m_j, l_j, o_j): M = max m_j, l = sum l_j 2^(m_j - M),
// o = sum o_j w_j; an empty part has m_j = -inf and l_j = 0.
template <typename T, int D, typename Tile, bool kLogits>
__global__ void __launch_bounds__(kWinThreads) pa_window_kernel(const WindowParams p) {
  constexpr int HP = Tile::kHeads;
  __shared__ __align__(16) float sm_o[kWinWarps][HP * D];
  __shared__ float2 sm_ml[kWinWarps][HP];
  __shared__ int sm_last;

  const int piece = blockIdx.x % p.splits;
  const int seg = blockIdx.x / p.splits;
  const int part = seg % p.parts;
  const int kvh = (seg / p.parts) % p.num_kv_heads;
  const int s = seg / p.parts / p.num_kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = kvh * p.group + part * p.part_heads;
  const int heads = min(p.part_heads, p.group - part * p.part_heads);
  const int L = checked_len(p, s);
  const TileRange r = tiles_visible<Tile::TT>(L, p.window, p.sinks);
  // pieces of this segment: none is shorter than min_tiles where that can be
  const int pieces = max(1, min(p.splits, r.n / p.min_tiles));
  if (piece >= pieces) return;
  const int begin = (int)((int64_t)r.n * piece / pieces), end = (int)((int64_t)r.n * (piece + 1) / pieces);

  Tile tile;
  tile.init(p, s, h0, heads, lane);
  tile.walk(p, s, kvh, h0, L, r, begin, end, warp, lane);
  tile.finish(sm_o[warp], sm_ml[warp]);
  __syncthreads();

  // join the warps: a thread takes 4 dims of a head
  T* out = static_cast<T*>(p.out) + ((size_t)s * p.num_heads + h0) * D;
  const size_t slot = ((size_t)seg * p.splits + piece) * HP;
  for (int i = threadIdx.x; i < heads * (D / 4); i += kWinThreads) {
    const int h = i / (D / 4), d = 4 * (i % (D / 4));
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWinWarps; ++w) M = fmaxf(M, sm_ml[w][h].x);
    float l = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kWinWarps; ++w) {
      const float2 ml = sm_ml[w][h];
      const float f = exp2_from(ml.x, M);
      const float4 v = *reinterpret_cast<const float4*>(&sm_o[w][h * D + d]);
      l += ml.y * f;
      a[0] = fmaf(v.x, f, a[0]), a[1] = fmaf(v.y, f, a[1]), a[2] = fmaf(v.z, f, a[2]), a[3] = fmaf(v.w, f, a[3]);
    }
    if (pieces == 1) {
      // no token: zeros; a row whose every logit is -inf: 0 / 0, as the formula has it
      const float inv = L > 0 ? 1.f / l : 0.f;
      store4(out + h * D + d, a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
      if (kLogits && d == 0) p.row_ml[(size_t)s * p.num_heads + h0 + h] = make_float2(M, l);
    } else {
      __stcg(reinterpret_cast<float4*>(p.piece_o + (slot + h) * D + d), make_float4(a[0], a[1], a[2], a[3]));
      if (d == 0) __stcg(p.piece_ml + slot + h, make_float2(M, l));
    }
  }
  if (pieces == 1) return;

  // the last piece of the segment joins them all
  __syncthreads();  // the partial's writes precede the release below
  if (threadIdx.x == 0) {
    __threadfence();
    const int prev = atomic_add_acq_rel_gpu(p.counter + seg, 1);
    sm_last = prev == pieces - 1;
    if (prev == pieces - 1) p.counter[seg] = 0;  // all have counted: zero for the next call
  }
  __syncthreads();
  if (!sm_last) return;
  __threadfence();
  const size_t first = (size_t)seg * p.splits * HP;
  for (int i = threadIdx.x; i < heads * (D / 4); i += kWinThreads) {
    const int h = i / (D / 4), d = 4 * (i % (D / 4));
    float M = -INFINITY;
    for (int j = 0; j < pieces; ++j) M = fmaxf(M, __ldcg(p.piece_ml + first + (size_t)j * HP + h).x);
    float l = 0.f, a[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int j = 0; j < pieces; ++j) {
      const float2 ml = __ldcg(p.piece_ml + first + (size_t)j * HP + h);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(p.piece_o + (first + (size_t)j * HP + h) * D + d));
      const float f = exp2_from(ml.x, M);
      l += ml.y * f;
      a[0] = fmaf(v.x, f, a[0]), a[1] = fmaf(v.y, f, a[1]), a[2] = fmaf(v.z, f, a[2]), a[3] = fmaf(v.w, f, a[3]);
    }
    const float inv = 1.f / l;
    store4(out + h * D + d, a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
    if (kLogits && d == 0) p.row_ml[(size_t)s * p.num_heads + h0 + h] = make_float2(M, l);
  }
}

using WindowLauncher = cudaError_t (*)(const WindowParams&, cudaStream_t);

// 16-bit (is_bf16) and 32-bit caches; part_heads picks the variant (see WindowShape).
WindowLauncher window_launcher_16(int is_bf16, int head_dim, int part_heads, bool logits);
WindowLauncher window_launcher_f32(int head_dim, int part_heads, bool logits);
cudaError_t launch_add_scores(const ScoreParams& p, int num_seqs, int max_context_len, cudaStream_t stream);

}  // namespace pkv
