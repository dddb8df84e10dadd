// Instantiations of the window / score decode kernel, and the kernel that adds
// the attention weights to the scores.
#include "decode_window.cuh"

namespace pkv {

namespace {

template <typename T, int D, typename Tile, bool kLogits>
cudaError_t launch_window(const WindowParams& p, cudaStream_t stream) {
  const int64_t grid = (int64_t)p.num_seqs * p.num_kv_heads * p.parts * p.splits;
  if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
  pa_window_kernel<T, D, Tile, kLogits><<<(unsigned)grid, kWinThreads, 0, stream>>>(p);
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
// g of 2^(x_h[t] - m_h) / l_h, the heads in order. One thread per token.
constexpr int kAddThreads = 256;
__global__ void __launch_bounds__(kAddThreads) add_scores_kernel(const ScoreParams p) {
  const int s = blockIdx.z, g = blockIdx.y;
  const int L = min(max(__ldg(p.context_lens + s), 0), p.cap);
  const int64_t t = (int64_t)blockIdx.x * kAddThreads + threadIdx.x;
  if (t >= L) return;
  const size_t row = (size_t)s * p.num_kv_heads + g;
  float sum = 0.f;
  for (int j = 0; j < p.group; ++j) {
    const size_t h = (size_t)s * p.num_heads + (size_t)g * p.group + j;
    const float2 ml = __ldg(p.row_ml + h);
    sum += exp2_from(__ldg(p.logits + h * p.logit_stride + t), ml.x) / ml.y;
  }
  const float old = p.scores != nullptr && t < L - 1 ? p.scores[row * p.score_stride + t] : 0.f;
  p.scores_out[row * p.score_stride + t] = old + sum;
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
  const dim3 grid((unsigned)(((int64_t)max_context_len + kAddThreads - 1) / kAddThreads), p.num_kv_heads, num_seqs);
  if (grid.x == 0) return cudaSuccess;
  add_scores_kernel<<<grid, kAddThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace pkv
