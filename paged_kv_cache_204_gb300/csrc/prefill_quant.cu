// Prefill over quantised caches: a warp to a query row, lanes over the head dims.
#include "common.cuh"
#include "prefill_quant.h"

namespace pkv {

namespace {

// Values 4 l .. 4 l + 3 (head_dim 128) or 2 l, 2 l + 1 (64) of a cache row.
template <bool Q4, int D>
__device__ __forceinline__ void row_values(const unsigned char* row, int lane, float (&x)[D / 32]) {
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const int d = lane * (D / 32) + i;
    if constexpr (Q4) {
      const float s = __half2float(__ushort_as_half(reinterpret_cast<const unsigned short*>(row)[d / 32]));
      const int byte = row[D / 16 + d / 32 * 16 + d % 16];
      x[i] = s * (float)((d % 32 < 16 ? byte & 15 : byte >> 4) - 8);
    } else {
      __nv_fp8_e4m3 v;
      v.__x = row[d];
      x[i] = (float)v;
    }
  }
}

template <typename T, bool Q4, int D>
__global__ void __launch_bounds__(128) prefill_quant_kernel(const __grid_constant__ PrefillQuantParams p) {
  constexpr int N = D / 32, kRow = Q4 ? D / 16 * 9 : D;
  const int lane = threadIdx.x & 31, s = blockIdx.z, h = blockIdx.y;
  const int L = p.context_lens[s], q0 = p.query_start[s], n = p.query_start[s + 1] - q0;
  const int i = blockIdx.x * 4 + (threadIdx.x >> 5);
  if (L < 0 || L > p.max_blocks_per_seq * p.block_size || n < 0 || n > L || n > p.max_query_len) {
    if (i == 0 && lane == 0) set_err(p.dev_err, PKV_DEV_ERR_CONTEXT_LEN);
    return;
  }
  if (i >= n) return;
  const int g = h / p.group;
  const size_t at = ((size_t)(q0 + i) * p.num_heads + h) * D + lane * N;
  float q[N], o[N] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < N; ++e) q[e] = to_float(static_cast<const T*>(p.q)[at + e]);
  for (int t = 0; t <= L - n + i; ++t) {
    const int b = p.block_tables[(size_t)s * p.max_blocks_per_seq + t / p.block_size];
    float k[N] = {}, v[N] = {}, x = 0.f;
    if (b >= 0 && b < p.num_blocks) {
      const size_t row = (((size_t)b * p.num_kv_heads + g) * p.block_size + t % p.block_size) * kRow;
      row_values<Q4, D>(static_cast<const unsigned char*>(p.k_cache) + row, lane, k);
      row_values<Q4, D>(static_cast<const unsigned char*>(p.v_cache) + row, lane, v);
    } else if (lane == 0) {
      set_err(p.dev_err, PKV_DEV_ERR_BLOCK_ID);
    }
    for (int e = 0; e < N; ++e) x += q[e] * k[e];
    for (int e = 16; e > 0; e >>= 1) x += __shfl_xor_sync(kFullMask, x, e);
    x *= p.scale * p.k_scale;
    const float top = fmaxf(m, x), keep = expf(m - top), w = expf(x - top);
    l = l * keep + w;
    for (int e = 0; e < N; ++e) o[e] = o[e] * keep + w * v[e];
    m = top;
  }
  for (int e = 0; e < N; ++e) store_elem(static_cast<T*>(p.out) + at + e, o[e] * p.v_scale / l);
}

template <typename T, bool Q4, int D>
cudaError_t launch(const PrefillQuantParams& p, cudaStream_t stream) {
  if (p.num_heads > 65535) return cudaErrorNotSupported;
  const int64_t longest = (int64_t)p.max_blocks_per_seq * p.block_size;
  const int64_t queries = p.max_query_len < longest ? p.max_query_len : longest;
  prefill_quant_kernel<T, Q4, D><<<dim3((unsigned)((queries + 3) / 4), p.num_heads, p.num_seqs), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

template <bool Q4>
PrefillQuantLauncher of(bool bf16, int head_dim) {
  if (head_dim == 64) return bf16 ? launch<__nv_bfloat16, Q4, 64> : launch<__half, Q4, 64>;
  if (head_dim == 128) return bf16 ? launch<__nv_bfloat16, Q4, 128> : launch<__half, Q4, 128>;
  return nullptr;
}

}  // namespace

size_t prefill_quant_workspace_bytes(int head_dim) { return head_dim == 64 || head_dim == 128 ? 4096 : 0; }

PrefillQuantLauncher prefill_quant_launcher(bool q4, bool bf16, int head_dim) {
  return q4 ? of<true>(bf16, head_dim) : of<false>(bf16, head_dim);
}

}  // namespace pkv
