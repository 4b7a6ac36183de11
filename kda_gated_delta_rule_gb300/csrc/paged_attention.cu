// Attention over the paged cache: workspace layout and choice of kernel (kernels in paged_attention.cuh).
#include "device.h"
#include "paged_attention.cuh"

namespace kda {

namespace {
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
}  // namespace

size_t paged_attention_ws_bytes(int W, int Hq, int Hkv, int d) {
  const size_t rb = 8 * (size_t)pa_nt(W * (Hq / Hkv));
  return up256(PA_MAX_CTAS * 2 * rb * d * 4) + up256(PA_MAX_CTAS * 2 * rb * 8) + up256(PA_MAX_CTAS * sizeof(PaMeta));
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  PaPlan p;
  p.G = a.Hq / a.c.Hkv;
  p.rows = a.W * p.G;
  const int rb = 8 * pa_nt(p.rows);
  p.blocks = (p.rows + rb - 1) / rb;
  char* w = reinterpret_cast<char*>(a.ws);
  p.part_o = reinterpret_cast<float*>(w);
  w += up256((size_t)PA_MAX_CTAS * 2 * rb * a.c.d * 4);
  p.part_ml = reinterpret_cast<float*>(w);
  w += up256((size_t)PA_MAX_CTAS * 2 * rb * 8);
  p.meta = reinterpret_cast<PaMeta*>(w);
  const bool fine = !a.q_bf16 || !a.out_bf16;
  if (a.c.e4m3) return fine ? pa_e4m3_fine(a, p, sms, s) : pa_e4m3(a, p, sms, s);
  return fine ? pa_bf16_fine(a, p, sms, s) : pa_bf16(a, p, sms, s);
}

}  // namespace kda
