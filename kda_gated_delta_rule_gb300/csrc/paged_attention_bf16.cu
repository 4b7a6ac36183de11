// Attention over the paged cache: bf16 cache, bf16 queries and outputs.
#include "paged_attention.cuh"

namespace kda {

cudaError_t pa_bf16(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  return pa_heads<false, false>(a, p, sms, s);
}

}  // namespace kda
