// Rotating cache write: a step's queries and keys turned by their positions, keys and values
// stored in the slots of a paged cache, in one pass over the step's rows.
//
// A pair (a, b) of a row becomes (a c - b s, b c + a s), c and s the cosine and sine of the
// pair's angle, read from a table: angles of far positions are the caller's to work out in as
// many bits as they need. Every product and the sum of two are rounded to binary32 by themselves,
// so that the bytes written do not depend on how a compiler fuses them; then the one rounding to
// the row's type, to e4m3 or to a q4_0 block.
//
// A thread takes two 16-byte chunks of a row, which hold a run of whole pairs in either pairing
// (a chunk of the first half and its partner, or two neighbours), so that a pair never leaves a
// thread and the run's cosines and sines stay in registers for every row that the thread takes.
//
// Bound by HBM: every row is read once and written once. 8192 tokens of 32 heads (8 kv, head_dim 128, bfloat16)
// take 32.6 us, 6.30 TB/s; into e4m3 35.7 us (the divisions: 1.3 times the instructions), into q4_0 37.2 us (the blocks'
// maxima and codes: 1.5 times, issue slots 62 % busy); 4099 tokens of 40 heads of 64 21.5 us, 5.92 TB/s, and 24.7 us with
// three axes (a CTA waits for a position, then for its table row, and has one short token to do it for); 128 tokens of 40
// heads 2.7 us, one token 1.8 us: a launch.
#include "common.cuh"
#include "rope_cache.h"

namespace pkv {

namespace {

constexpr int kThreads = 128;

// The thread's run of cosines and sines: pairs [first, first + N) of the token. False where a
// position is outside the table.
template <int N>
__device__ __forceinline__ bool load_turn(const RopeParams& p, int t, int first, float (&c)[N], float (&s)[N]) {
  const int half = p.rotary_dim / 2;
  if (p.num_axes == 1) {
    const int pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_position) return false;
    const float4* row = reinterpret_cast<const float4*>(p.cos_sin + (size_t)pos * p.rotary_dim + first);
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 x = __ldg(row + i), y = __ldg(row + half / 4 + i);
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
    }
    return true;
  }
  bool ok = true;
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const uint32_t axes = p.pair_axis[(first >> 2) + i];
    if (axes == (axes & 0xffu) * 0x01010101u) {  // four pairs of one axis, as sections mostly have them
      const int pos = __ldg(p.positions + (size_t)(axes & 0xffu) * p.num_tokens + t);
      ok &= pos >= 0 && pos < p.max_position;
      const float4* at =
          reinterpret_cast<const float4*>(p.cos_sin + (size_t)(ok ? pos : 0) * p.rotary_dim + first + 4 * i);
      const float4 x = __ldg(at), y = __ldg(at + half / 4);
      c[4 * i] = x.x, c[4 * i + 1] = x.y, c[4 * i + 2] = x.z, c[4 * i + 3] = x.w;
      s[4 * i] = y.x, s[4 * i + 1] = y.y, s[4 * i + 2] = y.z, s[4 * i + 3] = y.w;
      continue;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int pos = __ldg(p.positions + (size_t)((axes >> (8 * e)) & 0xffu) * p.num_tokens + t);
      ok &= pos >= 0 && pos < p.max_position;
      const float* at = p.cos_sin + (size_t)(ok ? pos : 0) * p.rotary_dim + first + 4 * i + e;
      c[4 * i + e] = __ldg(at);
      s[4 * i + e] = __ldg(at + half);
    }
  }
  return ok;
}

// The pairs of two chunks turned: (a[i], b[i]), or with `interleaved` neighbours within a, then b.
template <int N>
__device__ __forceinline__ void turn(float (&a)[N], float (&b)[N], const float (&c)[N], const float (&s)[N],
                                     bool interleaved) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = a[i], y = b[i];
      a[i] = __fsub_rn(__fmul_rn(x, c[i]), __fmul_rn(y, s[i]));
      b[i] = __fadd_rn(__fmul_rn(y, c[i]), __fmul_rn(x, s[i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float& x = i < N / 2 ? a[2 * i] : b[2 * i - N];
      float& y = i < N / 2 ? a[2 * i + 1] : b[2 * i + 1 - N];
      const float u = x, w = y;
      x = __fsub_rn(__fmul_rn(u, c[i]), __fmul_rn(w, s[i]));
      y = __fadd_rn(__fmul_rn(w, c[i]), __fmul_rn(u, s[i]));
    }
  }
}

__device__ __forceinline__ uint2 to_e4m3(const float (&f)[8], float scale) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = narrow_e4m3x2(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale));
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// A q4_0 block by two neighbouring lanes of 16 values each (lane parity `upper`): m the block's
// first value of largest magnitude, d = m / -8, code = min(15, trunc(x / d + 8.5)), every step in
// binary32. Each lane ends with 8 of the 16 code bytes (low halves: values 0 .. 15) and d.
__device__ __forceinline__ uint2 to_q4(const float (&x)[16], bool upper, float& d) {
  float amax = 0.f, m = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float a = fabsf(x[i]);
    if (a > amax) amax = a, m = x[i];
  }
  const float amax2 = __shfl_xor_sync(kFullMask, amax, 1), m2 = __shfl_xor_sync(kFullMask, m, 1);
  if (upper ? amax2 >= amax : amax2 > amax) m = m2;  // of equal magnitudes the first
  d = __fdiv_rn(m, -8.f);
  const float inv = d != 0.f ? __fdiv_rn(1.f, d) : 0.f;
  // trunc(y) for y in [0, 15] is the last byte of y + 2^23 rounded down (a NaN gives 0 by the first maximum)
  uint32_t code[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float y = fminf(fmaxf(__fadd_rn(__fmul_rn(x[i], inv), 8.5f), 0.f), 15.f);
    code[i] = __float_as_uint(__fadd_rd(y, 8388608.f));
  }
  uint32_t lo[2], hi[2];  // codes 0 .. 7 and 8 .. 15 of this lane, a byte each
#pragma unroll
  for (int i = 0; i < 4; ++i)
    (i < 2 ? lo : hi)[i & 1] = __byte_perm(__byte_perm(code[4 * i], code[4 * i + 1], 0x0040),
                                           __byte_perm(code[4 * i + 2], code[4 * i + 3], 0x0040), 0x5410);
  // the lower lane makes bytes 0 .. 7, the upper one 8 .. 15
  const uint32_t g0 = __shfl_xor_sync(kFullMask, upper ? lo[0] : hi[0], 1);
  const uint32_t g1 = __shfl_xor_sync(kFullMask, upper ? lo[1] : hi[1], 1);
  return upper ? make_uint2(g0 | (hi[0] << 4), g1 | (hi[1] << 4)) : make_uint2(lo[0] | (g0 << 4), lo[1] | (g1 << 4));
}

// grid = (token, part of its rows); kUnits pairs of chunks to a thread, all loads first. A token
// with a negative position is an idle row of a fixed batch: nothing of it is read or written.
template <typename T, int D, RopeCache C, int kUnits>
__global__ void __launch_bounds__(kThreads) rope_and_cache_kernel(const __grid_constant__ RopeParams p) {
  constexpr int N = Chunk<T>::kElems;      // values of a chunk
  constexpr int kRowChunks = D / N;        // chunks of a row
  constexpr int kRowUnits = kRowChunks / 2;
  constexpr int kRowBytes = C == RopeCache::kSame ? D * (int)sizeof(T) : (C == RopeCache::kFp8 ? D : D / 16 * 9);
  static_assert(kThreads % kRowUnits == 0, "a thread's place in its rows is the same for all of them");
  const int t = blockIdx.x, H = p.num_heads, G = p.num_kv_heads;
  const int rows = H + 2 * G;
  const int j = threadIdx.x % kRowUnits;
  const int row0 = (blockIdx.y * kThreads * kUnits + threadIdx.x) / kRowUnits;
  constexpr int kStep = kThreads / kRowUnits;
  // a unit below rotary_dim / (2 N) is turned
  const int turned_units = p.rotary_dim / (2 * N);
  const bool turned = j < turned_units;
  const int ca = turned && !p.interleaved ? j : 2 * j;
  const int cb = turned && !p.interleaved ? j + turned_units : 2 * j + 1;

  const int first_pos = __ldg(p.positions + t);
  const int64_t slot = __ldg(p.slot_mapping + t);
  uint4 xa[kUnits], xb[kUnits];
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int r = row0 + i * kStep;
    const uint4* src = nullptr;
    if (r < H)
      src = static_cast<const uint4*>(p.q) + t * p.q_stride + (int64_t)r * kRowChunks;
    else if (r < H + G)
      src = static_cast<const uint4*>(p.k) + t * p.k_stride + (int64_t)(r - H) * kRowChunks;
    else if (r < rows)
      src = static_cast<const uint4*>(p.v) + t * p.v_stride + (int64_t)(r - H - G) * kRowChunks;
    xa[i] = xb[i] = make_uint4(0, 0, 0, 0);
    if (src != nullptr && first_pos >= 0) xa[i] = src[ca], xb[i] = src[cb];
  }
  if (first_pos < 0) return;
  float c[N], s[N];
  const bool inside = load_turn<N>(p, t, turned ? N * j : 0, c, s);
  // one axis beside the pairs of this thread may be outside: the whole token is left out then
  bool known = inside;
  if (p.num_axes > 1)
    for (int a = 0; a < p.num_axes; ++a) {
      const int pos = __ldg(p.positions + (size_t)a * p.num_tokens + t);
      known &= pos >= 0 && pos < p.max_position;
    }
  const bool stored = slot >= 0 && slot < p.num_slots;
  if (threadIdx.x == 0 && blockIdx.y == 0) {
    if (!known) set_err(p.dev_err, PKV_DEV_ERR_POSITION);
    if (slot >= p.num_slots) set_err(p.dev_err, PKV_DEV_ERR_SLOT);
  }
  if (!known) return;
  const int64_t blk = stored ? slot / p.block_size : 0;
  const int off = stored ? static_cast<int>(slot - blk * p.block_size) : 0;

#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const int r = row0 + i * kStep;
    const bool is_q = r < H, is_v = r >= H + G;
    float a[N], b[N];
    if constexpr (C == RopeCache::kSame) {  // V rows and what is not turned move as they are
      if (r >= rows || (!is_q && !stored)) continue;
      if (turned && !is_v) {
        Chunk<T>::widen(xa[i], a);
        Chunk<T>::widen(xb[i], b);
        turn<N>(a, b, c, s, p.interleaved != 0);
        xa[i] = Chunk<T>::narrow(a);
        xb[i] = Chunk<T>::narrow(b);
      }
      uint4* dst;
      if (is_q) {
        dst = static_cast<uint4*>(p.q_out) + t * p.q_out_stride + (int64_t)r * kRowChunks;
      } else {
        const int h = r - H - (is_v ? G : 0);
        dst = static_cast<uint4*>(is_v ? p.v_cache : p.k_cache) +
              ((blk * G + h) * p.block_size + off) * (int64_t)kRowChunks;
      }
      dst[ca] = xa[i];
      dst[cb] = xb[i];
    } else {
      Chunk<T>::widen(xa[i], a);
      Chunk<T>::widen(xb[i], b);
      if (turned && !is_v) turn<N>(a, b, c, s, p.interleaved != 0);
      if (is_q) {
        uint4* dst = static_cast<uint4*>(p.q_out) + t * p.q_out_stride + (int64_t)r * kRowChunks;
        dst[ca] = turned ? Chunk<T>::narrow(a) : xa[i];
        dst[cb] = turned ? Chunk<T>::narrow(b) : xb[i];
      }
      const int h = is_v ? r - H - G : max(r - H, 0);
      unsigned char* dst = static_cast<unsigned char*>(is_v ? p.v_cache : p.k_cache) +
                           ((blk * G + h) * p.block_size + off) * (int64_t)kRowBytes;
      const bool store = !is_q && r < rows && stored;
      if constexpr (C == RopeCache::kFp8) {
        if (store) {
          const float scale = is_v ? p.v_scale : p.k_scale;
          reinterpret_cast<uint2*>(dst)[ca] = to_e4m3(a, scale);
          reinterpret_cast<uint2*>(dst)[cb] = to_e4m3(b, scale);
        }
      } else if (__any_sync(kFullMask, store)) {
        // 16 neighbouring values to a lane, two lanes to a block: where a lane holds a chunk and
        // its partner half a row away, the warp's rows change hands in shared memory
        __shared__ float4 turnover[kThreads / 32][32 * 4];
        float x[16];
        if (__any_sync(kFullMask, cb != ca + 1)) {
          float4* mine = turnover[threadIdx.x >> 5] + (threadIdx.x & 31) / kRowUnits * (D / 4);
          mine[2 * ca] = make_float4(a[0], a[1], a[2], a[3]);
          mine[2 * ca + 1] = make_float4(a[4], a[5], a[6], a[7]);
          mine[2 * cb] = make_float4(b[0], b[1], b[2], b[3]);
          mine[2 * cb + 1] = make_float4(b[4], b[5], b[6], b[7]);
          __syncwarp();
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 f = mine[4 * j + e];
            x[4 * e] = f.x, x[4 * e + 1] = f.y, x[4 * e + 2] = f.z, x[4 * e + 3] = f.w;
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = a[e], x[8 + e] = b[e];
        }
        float d;
        const uint2 codes = to_q4(x, j & 1, d);
        if (store) {
          // a row of 9 D / 16 bytes starts on 4 bytes (head_dim 64) or 8 (128)
          unsigned char* to = dst + D / 16 + 8 * j;
          if constexpr (D == 128) {
            *reinterpret_cast<uint2*>(to) = codes;
          } else {
            reinterpret_cast<uint32_t*>(to)[0] = codes.x;
            reinterpret_cast<uint32_t*>(to)[1] = codes.y;
          }
          if ((j & 1) == 0) reinterpret_cast<unsigned short*>(dst)[j >> 1] = __half_as_ushort(__float2half_rn(d));
        }
      }
    }
  }
}

// One unit to a thread where that fills no more than the threads that are resident together. Else
// 2 to 4, as the fewest threads of a token's last CTA stay idle: 384 units (8192 tokens, 32 heads, 8 kv,
// bfloat16) take 33.0 us with 3, 34.7 with 4, 38.4 with 2; 480 (4099 tokens of three axes, 40 heads of 64) 25.2 with 4,
// 26.0 with 2, 29.2 with 3; 192 (8192 tokens, 32 heads of 64, 8 kv) 21.3 with 2, 23.5 with 3, 25.8 with 4.
constexpr int64_t kResident = 152 * 2048;

template <typename T, int D, RopeCache C>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  constexpr int kRowUnits = D / Chunk<T>::kElems / 2;
  const int64_t units = (int64_t)(p.num_heads + 2 * p.num_kv_heads) * kRowUnits;
  auto parts_of = [&](int each) { return (units + kThreads * each - 1) / (kThreads * each); };
  int each = 4;
  for (int e = 3; e > 1; --e)
    if (parts_of(e) * e < parts_of(each) * each) each = e;
  if (p.num_tokens * units <= kResident) each = 1;
  if (parts_of(each) > 65535) return cudaErrorNotSupported;
  const dim3 grid(p.num_tokens, (unsigned)parts_of(each));
  const auto kernel = each == 1   ? rope_and_cache_kernel<T, D, C, 1>
                      : each == 2 ? rope_and_cache_kernel<T, D, C, 2>
                      : each == 3 ? rope_and_cache_kernel<T, D, C, 3>
                                  : rope_and_cache_kernel<T, D, C, 4>;
  kernel<<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

template <RopeCache C>
RopeLauncher of_16(pkv_dtype dtype, int head_dim) {
  if (dtype == PKV_F16) return head_dim == 64 ? launch<__half, 64, C> : launch<__half, 128, C>;
  if (dtype == PKV_BF16) return head_dim == 64 ? launch<__nv_bfloat16, 64, C> : launch<__nv_bfloat16, 128, C>;
  return nullptr;
}

}  // namespace

RopeLauncher rope_launcher(RopeCache cache, pkv_dtype dtype, int head_dim) {
  if (head_dim != 64 && head_dim != 128) return nullptr;
  switch (cache) {
    case RopeCache::kSame:
      if (dtype == PKV_F32)
        return head_dim == 64 ? launch<float, 64, RopeCache::kSame> : launch<float, 128, RopeCache::kSame>;
      return of_16<RopeCache::kSame>(dtype, head_dim);
    case RopeCache::kFp8: return of_16<RopeCache::kFp8>(dtype, head_dim);
    case RopeCache::kQ4: return of_16<RopeCache::kQ4>(dtype, head_dim);
  }
  return nullptr;
}

}  // namespace pkv
