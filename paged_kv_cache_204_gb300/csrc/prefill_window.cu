// Launch of the windowed prefill kernel (binary16 and bfloat16).
#include "prefill_window.cuh"

#include <limits>

namespace pkv {

namespace {

template <typename T, int D>
cudaError_t launch_prefill_window(const PrefillWindowParams& params, const void* k_cache, const void* v_cache,
                                  int max_query_len, cudaStream_t stream) {
  using S = PwShape<D>;
  auto kernel = pa_prefill_window_kernel<T, D>;
  PrefillWindowParams p = params;
  // the TMA row coordinate (and one box past the pool) must fit in int32
  const long long pool_rows = (long long)p.num_blocks * p.num_kv_heads * p.block_size;
  if (pool_rows + kPwTokens > 0x7fffffffLL) return cudaErrorNotSupported;
  static int sms_of_device[64] = {0};  // SMs per device ordinal (0 = not yet known)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = (dev >= 0 && dev < 64) ? __atomic_load_n(&sms_of_device[dev], __ATOMIC_ACQUIRE) : 0;
  if (sms == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) __atomic_store_n(&sms_of_device[dev], sms, __ATOMIC_RELEASE);
  }
  // scores are taken raw, so the scale has to be positive: a negative one's sign goes
  // into the queries, and 0 becomes the smallest number: any finite score's product with it is
  // 2^-21 at most
  p.flip = p.scale_log2 < 0.f ? 0x80008000u : 0u;
  p.scale_log2 = p.scale_log2 == 0.f ? std::numeric_limits<float>::denorm_min() : fabsf(p.scale_log2);
  CUtensorMap kmap, vmap;
  constexpr bool bf16 = std::is_same<T, __nv_bfloat16>::value;
  e = encode_pool_rows_map(&kmap, k_cache, (uint64_t)pool_rows, D, p.block_size, bf16);
  if (e != cudaSuccess) return e;
  e = encode_pool_rows_map(&vmap, v_cache, (uint64_t)pool_rows, D, p.block_size, bf16);
  if (e != cudaSuccess) return e;
  const int64_t longest = (int64_t)p.max_blocks_per_seq * p.block_size;  // no sequence has more queries either
  const int64_t queries = max_query_len < longest ? max_query_len : longest;
  const int64_t pairs = (queries * p.group + 2 * kPwRows - 1) / (2 * kPwRows);
  const int64_t items = pairs * p.num_seqs * p.num_kv_heads;
  if (items > 0x3fffffff || pairs * 2 * kPwRows > 0x7fffffffLL) return cudaErrorNotSupported;
  p.pairs = (int)pairs;
  p.by_columns.set((uint32_t)(p.num_seqs * p.num_kv_heads));
  p.by_heads.set((uint32_t)p.num_kv_heads);
  p.by_group.set((uint32_t)p.group);
  // K/V tiles of a walk, at most
  const int64_t seen = (int64_t)p.window + p.sinks + 2 * kPwRows;
  const int64_t tiles = ((seen < longest ? seen : longest) + kPwTokens - 1) / kPwTokens;
  p.cluster = 1;
  while (p.cluster < kPwMaxCluster && items * p.cluster * 2 <= sms && p.cluster * 2 <= tiles) p.cluster *= 2;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.cluster > 1 ? items * p.cluster : (items < sms ? items : sms)));
  cfg.blockDim = dim3(kPwThreads);
  cfg.dynamicSmemBytes = S::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, kmap, vmap, p);
}

}  // namespace

PrefillWindowLauncher prefill_window_launcher(int is_bf16, int head_dim) {
  if (head_dim == 64) return is_bf16 ? launch_prefill_window<__nv_bfloat16, 64> : launch_prefill_window<__half, 64>;
  if (head_dim == 128) return is_bf16 ? launch_prefill_window<__nv_bfloat16, 128> : launch_prefill_window<__half, 128>;
  return nullptr;
}

}  // namespace pkv
