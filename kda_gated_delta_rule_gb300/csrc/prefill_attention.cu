// Attention over packed prompts: choice of form, workspace layout, and the row statistics that the gradients share.
#include "device.h"
#include "prefill_attention.cuh"

namespace kda {

namespace {

// Per query row: its log-sum-exp in powers of two, and D = <d_out, out> = sum_j p_j (d_out . v_j), the softmax gradient's
// mean.  A row of `d` channels takes d / 8 lanes.  Written as [Hq][T] so that a block of rows of one head is contiguous.
template <typename In, typename Out, int D>
__global__ void __launch_bounds__(256)
    pf_stats_kernel(const PromptAttnArgs a, const PromptGradArgs g, float2* __restrict__ stats) {
  pdl_begin();
  constexpr int L = D / 8;
  const int64_t row = ((int64_t)blockIdx.x * 256 + threadIdx.x) / L;
  const int c = (threadIdx.x % L) * 8;
  if (row >= a.T * a.Hq) return;  // whole rows: the lanes of one leave together
  const int64_t t = row / a.Hq;
  const int h = (int)(row - t * a.Hq);
  const In* x = static_cast<const In*>(g.d_out) + t * g.d_out_stride + h * D + c;
  const Out* y = static_cast<const Out*>(a.out) + t * a.out_stride + h * D + c;
  In xs[8];
  Out ys[8];
#pragma unroll
  for (int i = 0; i < (int)sizeof(xs) / 16; ++i) reinterpret_cast<uint4*>(xs)[i] = __ldg(reinterpret_cast<const uint4*>(x) + i);
#pragma unroll
  for (int i = 0; i < (int)sizeof(ys) / 16; ++i) reinterpret_cast<uint4*>(ys)[i] = __ldg(reinterpret_cast<const uint4*>(y) + i);
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum = fmaf(to_f32(xs[i]), to_f32(ys[i]), sum);
  const unsigned lanes = __activemask();
#pragma unroll
  for (int i = 1; i < L; i <<= 1) sum += __shfl_xor_sync(lanes, sum, i);
  if (c == 0) stats[h * a.T + t] = make_float2(__ldg(a.lse + row) * PA_LOG2E, sum);
}

template <typename In, typename Out>
cudaError_t stats_launch(const PromptAttnArgs& a, const PromptGradArgs& g, float2* stats, cudaStream_t s) {
  const int64_t threads = a.T * a.Hq * (a.d / 8);
  const dim3 grid((unsigned)((threads + 255) / 256));
  switch (a.d) {
    case 16: return launch_pdl(pf_stats_kernel<In, Out, 16>, grid, dim3(256), 0, s, a, g, stats);
    case 32: return launch_pdl(pf_stats_kernel<In, Out, 32>, grid, dim3(256), 0, s, a, g, stats);
    case 64: return launch_pdl(pf_stats_kernel<In, Out, 64>, grid, dim3(256), 0, s, a, g, stats);
    default: return launch_pdl(pf_stats_kernel<In, Out, 128>, grid, dim3(256), 0, s, a, g, stats);
  }
}

}  // namespace

cudaError_t launch_prefill_attention(const PromptAttnArgs& a, cudaStream_t s) {
  return a.in_bf16 ? pf_tc(a, s) : pf_f32(a, s);
}

namespace {
size_t stats_bytes(int64_t T, int Hq) { return ((size_t)T * Hq * sizeof(float2) + 255) & ~size_t(255); }
}  // namespace

size_t prefill_attention_grad_ws_bytes(int64_t T, int N, int Hq, int Hkv, int d) {
  const int parts = pg_parts(T, Hq, Hkv);
  return stats_bytes(T, Hq) + (parts > 1 ? (size_t)parts * 2 * T * Hkv * d * 4 : 0);
}

cudaError_t launch_prefill_attention_backward(const PromptAttnArgs& a, const PromptGradArgs& g, cudaStream_t s) {
  float2* stats = static_cast<float2*>(g.ws);
  cudaError_t e = a.in_bf16 ? (a.out_bf16 ? stats_launch<bf16, bf16>(a, g, stats, s) : stats_launch<bf16, float>(a, g, stats, s))
                            : (a.out_bf16 ? stats_launch<float, bf16>(a, g, stats, s) : stats_launch<float, float>(a, g, stats, s));
  if (e != cudaSuccess) return e;
  if (!a.in_bf16) return pf_f32_grad(a, g, stats, s);
  return pf_tc_grad(a, g, stats, reinterpret_cast<float*>(static_cast<char*>(g.ws) + stats_bytes(a.T, a.Hq)), s);
}

}  // namespace kda
