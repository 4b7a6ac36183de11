// Attention over the paged cache: workspace layout and choice of kernel (kernels in paged_attention.cuh).
#include "device.h"
#include "paged_attention.cuh"

namespace kda {

namespace {
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
}  // namespace

namespace {

// The workspace's places for `workers` warps or CTAs with row blocks of rb.
size_t lay_out(PaPlan& p, char* w, int workers, int rb, int d) {
  const size_t parts = (size_t)workers * 2 * rb;
  p.part_o = reinterpret_cast<float*>(w);
  w += up256(parts * d * 4);
  p.part_ml = reinterpret_cast<float*>(w);
  w += up256(parts * 8);
  p.meta = reinterpret_cast<PaMeta*>(w);
  return up256(parts * d * 4) + up256(parts * 8) + up256(workers * sizeof(PaMeta));
}

}  // namespace

size_t paged_attention_ws_bytes(int W, int Hq, int Hkv, int d) {
  // the largest of the forms that a call's types may choose
  const int rows = W * (Hq / Hkv);
  PaPlan p;
  size_t most = lay_out(p, nullptr, PA_SMS, pa_tc_row_block(rows), d);
  for (int fine = 0; fine < 2; ++fine) {
    const int nt = pa_nt(rows, fine != 0);
    const size_t n = lay_out(p, nullptr, PA_SMS * pa_resident(nt) * PA_WARPS, 8 * nt, d);
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
  const int tc_rb = pa_tc_row_block(p.rows), tc_blocks = (p.rows + tc_rb - 1) / tc_rb;
  // The tensor-memory form is ahead with many query rows per cached row (96 rows: 88 against 119 us; 24: 43 against 57), and
  // with fewer units than CTAs, where its larger and so fewer parts join faster (one request of 4096 tokens and 8 heads: 15
  // against 26 us, of 262144: 167 against 175); with many units of few rows their starts and ends cost it more (16 requests
  // of 4096 tokens, 128 units: 64 against 56 us).
  if (pa_tc_supported(a) && (p.rows > 16 || (int64_t)a.B * a.c.Hkv * tc_blocks <= 64)) {
    const int rb = tc_rb;
    p.blocks = tc_blocks;
    lay_out(p, reinterpret_cast<char*>(a.ws), PA_SMS, rb, a.c.d);
    return pa_tc(a, p, sms, s);
  }
  const int nt = pa_nt(p.rows, fine), rb = 8 * nt;
  p.blocks = (p.rows + rb - 1) / rb;
  lay_out(p, reinterpret_cast<char*>(a.ws), PA_SMS * pa_resident(nt) * PA_WARPS, rb, a.c.d);
  if (a.c.e4m3) return fine ? pa_e4m3_fine(a, p, sms, s) : pa_e4m3(a, p, sms, s);
  return fine ? pa_bf16_fine(a, p, sms, s) : pa_bf16(a, p, sms, s);
}

}  // namespace kda
