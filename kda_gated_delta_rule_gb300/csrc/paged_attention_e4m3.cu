// Attention over the paged cache: e4m3 cache, bf16 queries and outputs.
#include "paged_attention.cuh"

namespace kda {

cudaError_t pa_e4m3(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  return pa_heads<true, false>(a, p, sms, s);
}

}  // namespace kda
