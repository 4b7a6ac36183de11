// Attention over the paged cache: workspace layout and choice of kernel (kernels in paged_attention.cuh).
#include "device.h"
#include "paged_attention.cuh"

namespace kda {

namespace {
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }
}  // namespace

namespace {

// More query rows per cached row than this take the many-rows form: its time hardly grows up to 128 (64 requests of 500 to 6000
// tokens, 24 rows and 96: 29 and 33 us with bf16, 39 and 44 with e4m3), where the register form's grows with the rows (52
// and 94; 48 and 78).  At 12 and 16 rows that one is as fast with bf16 (31 and 32 against 29; 90 requests of 2227 to 8908 tokens:
// 57 and 58 against 57) and faster with e4m3 (28 and 29 against 38; 46 and 47 against 88).  Units of a tile or less are the
// many-rows form's worst case (239 requests of 4 tokens, 8 drafts, 32 heads over 8: 80 against 48 us with bf16, 89 against 45 with e4m3; of
// 64 tokens 78 against 87, 87 against 76): the host knows no lengths, and a table wide enough for long ones says nothing.
constexpr int PA_ROWS_FROM = 16;

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
  if (rows > PA_ROWS_FROM) {
    const size_t n = lay_out(p, nullptr, PA_SMS, PA_ROWS_BLOCK, d);
    most = n > most ? n : most;
  }
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
  p.stall = a.test_stall;
  if (p.rows > PA_ROWS_FROM && pa_rows_supported(a)) {
    p.blocks = (p.rows + PA_ROWS_BLOCK - 1) / PA_ROWS_BLOCK;
    lay_out(p, reinterpret_cast<char*>(a.ws), PA_SMS, PA_ROWS_BLOCK, a.c.d);
    return pa_rows(a, p, sms, s);
  }
  // With few units the tensor-memory form's larger and so fewer parts join faster (one request with 8 heads, of 1000 tokens: 10.5
  // against 12.2 us, of 4096: 13.3 against 15.7, of 262144: 164 against 167; 64 units of 100 to 30000 tokens: 43.6 against
  // 44.0); with many units of few rows their starts and ends cost it more (64 units of 4096 tokens: 35 against 33 us, 128: 56
  // against 53).
  if (pa_tc_supported(a) && p.rows <= 16 && (int64_t)a.B * a.c.Hkv <= 64) {
    const int rb = pa_tc_row_block(p.rows);
    p.blocks = 1;
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
