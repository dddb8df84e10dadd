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
// g of 2^(x_h[t] - m_h) / l_h, the heads in order. A thread takes 4 neighbouring tokens;
// `quads`: the scores' rows are aligned for 16-byte accesses (128 sequences x 40 heads: 16 us
// behind the decode's 395, 21 with single floats; added by the CTA that finishes a
// row instead, 50).
constexpr int kAddThreads = 256;
constexpr int kAddTokens = kAddThreads * 4;  // of a CTA
__global__ void __launch_bounds__(kAddThreads) add_scores_kernel(const ScoreParams p, bool quads) {
  const int s = blockIdx.z, g = blockIdx.y;
  const int L = min(max(__ldg(p.context_lens + s), 0), p.cap);
  const int64_t t = (int64_t)blockIdx.x * kAddTokens + 4 * threadIdx.x;
  const size_t row = ((size_t)s * p.num_kv_heads + g) * p.score_stride;
  float old[4] = {0.f, 0.f, 0.f, 0.f}, sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.scores != nullptr) {
    if (quads && t + 4 < L) {
      const float4 x = *reinterpret_cast<const float4*>(p.scores + row + t);
      old[0] = x.x, old[1] = x.y, old[2] = x.z, old[3] = x.w;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (t + k < L - 1) old[k] = p.scores[row + t + k];
    }
  }
  // the logits, maxima and sums; by idle CTAs too: what follows in the stream waits for this grid only
  grid_dependency_wait();
  if (t >= L) return;
  for (int j = 0; j < p.group; ++j) {
    const size_t h = (size_t)s * p.num_heads + (size_t)g * p.group + j;
    const float2 ml = p.row_ml[h];
    const float inv = 1.f / ml.y;
    // (rows of logits are whole 8s: the last 16 bytes may hold what no token has)
    const float4 x = *reinterpret_cast<const float4*>(p.logits + h * p.logit_stride + t);
    sum[0] = fmaf(exp2_from(x.x, ml.x), inv, sum[0]);
    sum[1] = fmaf(exp2_from(x.y, ml.x), inv, sum[1]);
    sum[2] = fmaf(exp2_from(x.z, ml.x), inv, sum[2]);
    sum[3] = fmaf(exp2_from(x.w, ml.x), inv, sum[3]);
  }
  if (quads && t + 4 <= L) {
    *reinterpret_cast<float4*>(p.scores_out + row + t) =
        make_float4(old[0] + sum[0], old[1] + sum[1], old[2] + sum[2], old[3] + sum[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (t + k < L) p.scores_out[row + t + k] = old[k] + sum[k];
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
  const dim3 grid((unsigned)(((int64_t)max_context_len + kAddTokens - 1) / kAddTokens), p.num_kv_heads, num_seqs);
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
  const uintptr_t at = reinterpret_cast<uintptr_t>(p.scores) | reinterpret_cast<uintptr_t>(p.scores_out);
  const bool quads = (at & 15u) == 0 && p.score_stride % 4 == 0;
  return cudaLaunchKernelEx(&cfg, add_scores_kernel, p, quads);
}

}  // namespace pkv
