// Attention over the paged cache: workspace layout and choice of kernel (kernels in paged_attention.cuh).
#include "device.h"
#include "paged_attention.cuh"

namespace kda {

namespace {
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
}  // namespace

size_t paged_attention_ws_bytes(int W, int Hq, int Hkv, int d) {
  // the larger of the forms that a call's types may choose
  size_t most = 0;
  for (int fine = 0; fine < 2; ++fine) {
    const int nt = pa_nt(W * (Hq / Hkv), fine != 0);
    const size_t parts = (size_t)PA_SMS * pa_resident(nt) * PA_WARPS * 2 * 8 * nt;
    const size_t n = up256(parts * d * 4) + up256(parts * 8) + up256(parts / (16 * nt) * sizeof(PaMeta));
    most = n > most ? n : most;
  }
  return most;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, cudaStream_t s) {
  const int sms = sm_count();
  if (sms <= 0) return cudaErrorNoDevice;
  const bool fine = !a.q_bf16 || !a.out_bf16;
  PaPlan p;
  p.G = a.Hq / a.c.Hkv;
  p.rows = a.W * p.G;
  const int nt = pa_nt(p.rows, fine), rb = 8 * nt;
  p.blocks = (p.rows + rb - 1) / rb;
  const size_t parts = (size_t)PA_SMS * pa_resident(nt) * PA_WARPS * 2 * rb;
  char* w = reinterpret_cast<char*>(a.ws);
  p.part_o = reinterpret_cast<float*>(w);
  w += up256(parts * a.c.d * 4);
  p.part_ml = reinterpret_cast<float*>(w);
  w += up256(parts * 8);
  p.meta = reinterpret_cast<PaMeta*>(w);
  if (a.c.e4m3) return fine ? pa_e4m3_fine(a, p, sms, s) : pa_e4m3(a, p, sms, s);
  return fine ? pa_bf16_fine(a, p, sms, s) : pa_bf16(a, p, sms, s);
}

}  // namespace kda
