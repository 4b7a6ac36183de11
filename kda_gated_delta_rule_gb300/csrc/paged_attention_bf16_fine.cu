// Attention over the paged cache: bf16 cache, fp32 queries or outputs.
#include "paged_attention.cuh"

namespace kda {

cudaError_t pa_bf16_fine(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  return pa_heads<false, true>(a, p, sms, s);
}

}  // namespace kda
