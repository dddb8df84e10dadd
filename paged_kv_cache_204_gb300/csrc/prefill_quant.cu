// Launch of prefill over quantised caches (binary16 and bfloat16 queries; q4_0 and e4m3 pools).
#include "prefill_quant.cuh"

#include <limits>

namespace pkv {

namespace {

size_t cut_bytes() { return sizeof(PqCut) * kPqMaxCtas; }
size_t ml_bytes() { return sizeof(float2) * 2 * kPqMaxCtas * 256; }

template <typename T, PqFormat F, int D>
cudaError_t launch(const PrefillQuantParams& a, cudaStream_t stream) {
  using S = PqShape<T, F, D>;
  auto kernel = pa_prefill_quant_kernel<T, F, D>;
  static int sms_of_device[64] = {0};  // SMs per device ordinal (0 = not yet known)
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int sms = (dev >= 0 && dev < 64) ? __atomic_load_n(&sms_of_device[dev], __ATOMIC_ACQUIRE) : 0;
  if (sms == 0) {
    // the warpgroups' shares of registers are taken from what the launch has: a kernel that was
    // given fewer would wait for them without end
    cudaFuncAttributes attr;
    e = cudaFuncGetAttributes(&attr, kernel);
    if (e != cudaSuccess) return e;
    if (attr.numRegs < kPqLaunchRegs) return cudaErrorNotSupported;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemBytes);
    if (e != cudaSuccess) return e;
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) __atomic_store_n(&sms_of_device[dev], sms, __ATOMIC_RELEASE);
  }
  PqParams p{};
  p.out = a.out;
  p.q = a.q;
  p.k_cache = static_cast<const unsigned char*>(a.k_cache);
  p.v_cache = static_cast<const unsigned char*>(a.v_cache);
  p.block_tables = a.block_tables;
  p.context_lens = a.context_lens;
  p.query_start = a.query_start;
  // scores are taken raw, so the factor has to be positive: a negative one's sign goes into the
  // queries, and 0 becomes the smallest number: any finite score's product with it is next to nothing
  const float factor = a.scale * a.k_scale * 1.4426950408889634f;
  p.flip = factor < 0.f ? 0x80008000u : 0u;
  p.zero_scale = factor == 0.f;
  p.scale_log2 = factor == 0.f ? std::numeric_limits<float>::denorm_min() : fabsf(factor);
  p.v_scale = a.v_scale;
  p.num_seqs = a.num_seqs;
  p.num_heads = a.num_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.group;
  p.block_size = a.block_size;
  p.block_bits = a.block_size == 8 ? 3 : (a.block_size == 16 ? 4 : 5);
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_blocks = a.num_blocks;
  // rows of a kv head's queries are counted in 32 bits
  const int64_t longest = (int64_t)a.max_blocks_per_seq * a.block_size;
  const int64_t queries = a.max_query_len < longest ? a.max_query_len : longest;
  if (queries * a.group > 0x7fffffffLL - 256) return cudaErrorNotSupported;
  p.max_query_len = a.max_query_len;
  p.start = pq_start(D);
  p.by_group.set((uint32_t)a.group);
  char* ws = static_cast<char*>(a.workspace);
  p.cuts = reinterpret_cast<PqCut*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + cut_bytes());
  p.part_o = reinterpret_cast<float4*>(ws + cut_bytes() + ml_bytes());
  p.dev_err = a.dev_err;
  p.wait_limit_ns = a.wait_limit_ns;
  const unsigned ctas = sms < kPqMaxCtas ? sms : kPqMaxCtas;
  kernel<<<ctas, kPqThreads, S::kSmemBytes, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  // the join, launched under the first kernel's end (8 blocks of 32 rows to a pair)
  cudaLaunchConfig_t cfg{};
  const int64_t rows = queries * a.group < 256 ? queries * a.group : 256;
  cfg.gridDim = dim3(ctas, (unsigned)((rows + 31) / 32));
  cfg.blockDim = dim3(2 * D);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pa_prefill_quant_join_kernel<T, F, D>, p);
}

template <PqFormat F>
PrefillQuantLauncher of(bool bf16, int head_dim) {
  if (head_dim == 64) return bf16 ? launch<__nv_bfloat16, F, 64> : launch<__half, F, 64>;
  if (head_dim == 128) return bf16 ? launch<__nv_bfloat16, F, 128> : launch<__half, F, 128>;
  return nullptr;
}

}  // namespace

size_t prefill_quant_workspace_bytes(int head_dim) {
  if (head_dim != 64 && head_dim != 128) return 0;
  return cut_bytes() + ml_bytes() + sizeof(float) * 2 * kPqMaxCtas * 256 * (size_t)head_dim;
}

PrefillQuantLauncher prefill_quant_launcher(bool q4, bool bf16, int head_dim) {
  return q4 ? of<PqFormat::kQ4>(bf16, head_dim) : of<PqFormat::kFp8>(bf16, head_dim);
}

}  // namespace pkv
