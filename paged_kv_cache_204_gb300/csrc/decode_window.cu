// Instantiations of the window / score decode kernel, and the kernel that adds
// the attention weights to the scores.
#include "decode_window.cuh"

namespace pkv {

namespace {

template <typename T, int D, typename Tile, bool kLogits>
cudaError_t launch_window(const WindowParams& p, cudaStream_t stream) {
  const int64_t grid = (int64_t)p.num_seqs * p.num_kv_heads * p.parts * p.splits;
  if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
  constexpr int kSmem = kWinWarps * Tile::Ring::kBytes;
  static int configured[64] = {0};  // per device ordinal
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !__atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE)) {
    e = cudaFuncSetAttribute(pa_window_kernel<T, D, Tile, kLogits>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) __atomic_store_n(&configured[dev], 1, __ATOMIC_RELEASE);
  }
  pa_window_kernel<T, D, Tile, kLogits><<<(unsigned)grid, kWinThreads, kSmem, stream>>>(p);
  return cudaGetLastError();
}

template <typename T, int D, bool kLogits>
WindowLauncher pick_16(int part_heads) {
  return part_heads > 4 ? launch_window<T, D, MmaTile<T, D, true, kLogits>, kLogits>
                        : launch_window<T, D, MmaTile<T, D, false, kLogits>, kLogits>;
}

template <int D, bool kLogits>
WindowLauncher pick_f32(int part_heads) {
  return part_heads > 2   ? launch_window<float, D, FmaTile<D, 4, kLogits>, kLogits>
         : part_heads > 1 ? launch_window<float, D, FmaTile<D, 2, kLogits>, kLogits>
                          : launch_window<float, D, FmaTile<D, 1, kLogits>, kLogits>;
}

// scores_out[s][g][t] = (t < L - 1 ? scores[s][g][t] : 0) + sum over the heads h of
// g of 2^(x_h[t] - m_h) / l_h, the heads in order. A thread takes kAddTokens tokens.
constexpr int kAddThreads = 256;
constexpr int kAddTokens = 4;
__global__ void __launch_bounds__(kAddThreads) add_scores_kernel(const ScoreParams p) {
  const int s = blockIdx.z, g = blockIdx.y;
  const int L = min(max(__ldg(p.context_lens + s), 0), p.cap);
  const int64_t t0 = (int64_t)blockIdx.x * (kAddThreads * kAddTokens) + threadIdx.x;
  if ((int64_t)blockIdx.x * (kAddThreads * kAddTokens) >= L) {
    grid_dependency_wait();  // what follows in the stream waits for this grid only
    return;
  }
  const size_t row = (size_t)s * p.num_kv_heads + g;
  float sum[kAddTokens], old[kAddTokens];
#pragma unroll
  for (int k = 0; k < kAddTokens; ++k) {
    const int64_t t = t0 + k * kAddThreads;
    sum[k] = 0.f;
    old[k] = p.scores != nullptr && t < L - 1 ? p.scores[row * p.score_stride + t] : 0.f;
  }
  grid_dependency_wait();  // the logits, maxima and sums
  for (int j = 0; j < p.group; ++j) {
    const size_t h = (size_t)s * p.num_heads + (size_t)g * p.group + j;
    const float2 ml = p.row_ml[h];
    const float inv = 1.f / ml.y;
#pragma unroll
    for (int k = 0; k < kAddTokens; ++k) {
      const int64_t t = t0 + k * kAddThreads;
      if (t < L) sum[k] = fmaf(exp2_from(p.logits[h * p.logit_stride + t], ml.x), inv, sum[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < kAddTokens; ++k) {
    const int64_t t = t0 + k * kAddThreads;
    if (t < L) p.scores_out[row * p.score_stride + t] = old[k] + sum[k];
  }
}

}  // namespace

WindowLauncher window_launcher_16(int is_bf16, int head_dim, int part_heads, bool logits) {
  using H = __half;
  using B = __nv_bfloat16;
  if (head_dim == 64) {
    if (logits) return is_bf16 ? pick_16<B, 64, true>(part_heads) : pick_16<H, 64, true>(part_heads);
    return is_bf16 ? pick_16<B, 64, false>(part_heads) : pick_16<H, 64, false>(part_heads);
  }
  if (head_dim == 128) {
    if (logits) return is_bf16 ? pick_16<B, 128, true>(part_heads) : pick_16<H, 128, true>(part_heads);
    return is_bf16 ? pick_16<B, 128, false>(part_heads) : pick_16<H, 128, false>(part_heads);
  }
  return nullptr;
}

WindowLauncher window_launcher_f32(int head_dim, int part_heads, bool logits) {
  if (head_dim == 64) return logits ? pick_f32<64, true>(part_heads) : pick_f32<64, false>(part_heads);
  if (head_dim == 128) return logits ? pick_f32<128, true>(part_heads) : pick_f32<128, false>(part_heads);
  return nullptr;
}

cudaError_t launch_add_scores(const ScoreParams& p, int num_seqs, int max_context_len, cudaStream_t stream) {
  if (p.num_kv_heads > 65535 || num_seqs > 65535) return cudaErrorNotSupported;
  constexpr int kTokens = kAddThreads * kAddTokens;
  const dim3 grid((unsigned)(((int64_t)max_context_len + kTokens - 1) / kTokens), p.num_kv_heads, num_seqs);
  if (grid.x == 0) return cudaSuccess;
  // a programmatic dependent of the decode: set up while that runs, waits for it
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kAddThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, add_scores_kernel, p);
}

}  // namespace pkv
