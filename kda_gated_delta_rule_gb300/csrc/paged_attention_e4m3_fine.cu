// Attention over the paged cache: e4m3 cache, fp32 queries or outputs.
#include "paged_attention.cuh"

namespace kda {

cudaError_t pa_e4m3_fine(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  return pa_heads<true, true>(a, p, sms, s);
}

}  // namespace kda
