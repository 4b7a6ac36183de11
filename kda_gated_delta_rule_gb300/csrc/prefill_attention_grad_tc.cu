// Gradients of the attention over packed prompts on the 5th-generation tensor cores: bf16 inputs, any head size.
//
//   p_ij = exp(x_ij - lse_i),  dv_j = sum_i p_ij do_i,  dx_ij = p_ij (do_i . v_j - D_i) (cap's slope),
//   dk_j = scale sum_i dx_ij q_i,  dq_i = scale sum_j dx_ij k_j
//
// Two kernels, so that every sum has one owner and a fixed order; the price is that scores and do . v are formed twice, seven
// products where one kernel that adds dq up with atomics would need five.
//   keys:    128 keys of a key/value head against the blocks of 128 queries that see them, of all query heads of its group.  Scores are
//            formed as S^T = K Q^T and dO V^T as V dO^T: keys are rows, so that P^T and dX^T are row operands in tensor memory
//            (over the S^T and V dO^T they come from) of dV += P^T dO and dK += dX^T Q.
//   queries: 128 queries of a head against the tiles of 128 keys that they see: S = Q K^T, dO V^T, dQ += dX K, with two buffers for
//            dO V^T (dX in its place), so that the next tile's products run under a tile's arithmetic.
// Where keys' blocks are too few for the SMs (one key/value head for all queries), the group's heads are dealt to several CTAs, whose
// fp32 parts a third kernel adds up in order.
// A CTA has 12 warps: 0 to 7 the arithmetic, thread = row and half of the tile's columns; 8 the products; 9 the loads (TMA);
// 10 and 11 clear what lies behind the sequence in tiles that are column operands (0 * NaN), and bring the queries' statistics.
// p and dx are rounded to bf16 (2^-8) for their products; everything else is fp32.
#include "device.h"
#include "prefill_attention_tc.cuh"

namespace kda {

namespace {

constexpr int PG_MOST_PARTS = 16;

template <int D>
struct PgCfg {
  static constexpr int SLOT = D / 64 * PT_HALF;
  static constexpr int QR = D == 128 ? 2 : 3, OR = D == 128 ? 2 : 3;  // keys' kernel: slots of Q, of dO
  static constexpr int KR = 3, VR = D == 128 ? 2 : 3;                 // queries' kernel: slots of K, of V
};

struct PgMaps {
  CUtensorMap q, k, v, d_out;
};

struct PgKeysShared {
  // every barrier is waited on only by roles that see each of its rounds
  uint64_t kv_full, q_full[3], q_ready[3], q_empty[3], o_full[3], o_ready[3], o_empty[3], st_full[2], st_empty[2];
  uint64_t s_full, p_full, dp_full, ds_full, out_full, drain;
  alignas(16) float minus_lse[2][PT_B], minus_d[2][PT_B];  // of a block's queries: log-sum-exp in powers of two, D
  uint32_t tmem;
  int dead;
};
struct PgQueriesShared {
  uint64_t q_full, k_full[3], k_ready[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full, s_read, dp_full[2], ds_full[2], out_full, drain;
  uint32_t tmem;
  int dead;
};
template <int D>
constexpr int pg_keys_smem() {
  using C = PgCfg<D>;
  return 1024 + (2 + C::QR + C::OR) * C::SLOT + (int)sizeof(PgKeysShared);
}
template <int D>
constexpr int pg_queries_smem() {
  using C = PgCfg<D>;
  return 1024 + (2 + C::KR + C::VR) * C::SLOT + (int)sizeof(PgQueriesShared);
}
static_assert(pg_keys_smem<128>() <= 227 * 1024 && pg_queries_smem<128>() <= 227 * 1024, "shared memory of one SM");

// Rows from `rows` on of a tile of D / 64 halves become zeros; two warps, t = 0 .. 63.
template <int D>
__device__ __forceinline__ void clear_behind(unsigned char* tile, int rows, int t) {
  const int first = max(0, rows) * 8, n = PT_B * 8 - first;  // pieces of 16 bytes in a half
  for (int i = t; i < n * (D / 64); i += 64) {
    const int half = i / n;
    *reinterpret_cast<uint4*>(tile + half * PT_HALF + (first + i - half * n) * 16) = make_uint4(0, 0, 0, 0);
  }
  tc::fence_proxy_async();
}

// Products of 128 x 128 scores: rows a, columns b, both K-major.
template <int D>
__device__ __forceinline__ void scores_mma(uint32_t to, uint64_t a, uint64_t b) {
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {  // 16 channels per step
    const uint32_t at = (kk / 4 * PT_HALF + kk % 4 * 32) / 16;
    tc::mma_ss(to, a + at, b + at, pt_idesc(PT_B), kk > 0);
  }
}
// to (128 x D) += the 128 x 128 bf16 in tensor memory at `a` (each half of the columns over its own scores) times rows of b
template <int D>
__device__ __forceinline__ void rows_mma(uint32_t to, uint32_t a, uint64_t b, bool first) {
#pragma unroll
  for (int kk = 0; kk < PT_B / 16; ++kk)  // 16 rows per step
    tc::mma_ts(to, a + kk / 4 * 64 + kk % 4 * 8, b + kk * (2048 / 16), pt_idesc(D) | tc::IDESC_B_MN, !(first && kk == 0));
}

// Half a row of a block's result, 128 x D in tensor memory, times `by`.
template <int D>
__device__ __forceinline__ void store_rows(void* base, bool is_bf16, int64_t at, uint32_t from, float by, int d, bool mine) {
#pragma unroll 1
  for (int c = 0; c < D; c += 16) {
    float o[16];
    tc::tmem_ld16(from + c, o);
    if (mine && c < d) {
#pragma unroll
      for (int i = 0; i < 16; ++i) o[i] *= by;
      pt_store16(base, is_bf16, at + c, o);
    }
    __syncwarp();  // the next load is the whole warp's
  }
}

template <int D, bool CAP>
__global__ void __launch_bounds__(PT_NT, 1)
    prefill_attention_grad_keys_kernel(const __grid_constant__ PgMaps maps, const PromptAttnArgs a, const PromptGradArgs g,
                                       const float2* __restrict__ stats, float* __restrict__ parts, const int nparts) {
  using C = PgCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* kbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *vbuf = kbuf + C::SLOT, *qslots = vbuf + C::SLOT, *oslots = qslots + C::QR * C::SLOT;
  PgKeysShared& sh = *reinterpret_cast<PgKeysShared*>(oslots + C::OR * C::SLOT);
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int window = a.window > 0 ? a.window : 0x7fffffff;
  if (blockIdx.x == 0 && warp == 0) pf_check_offsets(a);
  // the first keys first: most queries see them
  const int unit = blockIdx.x % (a.Hkv * nparts), kh = unit / nparts, part = unit - kh * nparts;
  const PfBlock b = pf_block<7>(a, blockIdx.x / (a.Hkv * nparts));
  if (b.len == 0) return;
  const int group = a.Hq / a.Hkv, h0 = kh * group + part * group / nparts, h1 = kh * group + (part + 1) * group / nparts;
  const int k0 = b.row0, keys = min(PT_B, b.len - k0), tile = k0 / PT_B;
  const int last = (int)min((int64_t)b.len - 1, (int64_t)k0 + keys - 2 + window);  // the last query that sees one of the keys
  const int blocks = last / PT_B - tile + 1, n = blocks * (h1 - h0);              // a round: a block of one head

  if (tid == 0) {
    tc::bar_init(&sh.kv_full, 1);
    for (int i = 0; i < C::QR; ++i) tc::bar_init(&sh.q_full[i], 1), tc::bar_init(&sh.q_ready[i], 2), tc::bar_init(&sh.q_empty[i], 1);
    for (int i = 0; i < C::OR; ++i) tc::bar_init(&sh.o_full[i], 1), tc::bar_init(&sh.o_ready[i], 2), tc::bar_init(&sh.o_empty[i], 1);
    for (int i = 0; i < 2; ++i) tc::bar_init(&sh.st_full[i], 2), tc::bar_init(&sh.st_empty[i], 8);
    tc::bar_init(&sh.s_full, 1), tc::bar_init(&sh.p_full, 8), tc::bar_init(&sh.dp_full, 1), tc::bar_init(&sh.ds_full, 8);
    tc::bar_init(&sh.out_full, 1), tc::bar_init(&sh.drain, 1);
    tc::bar_fence_init();
    sh.dead = 0;
  }
  if (warp == 8) tc::tmem_alloc(&sh.tmem, PT_TMEM);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem, t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;

  if (warp == 9) {
    // ---- loads
    if (lane == 0) {
      bool ok = true;
      int sent_q = 0, sent_o = 0;
      tc::bar_arrive_expect_tx(&sh.kv_full, 2 * C::SLOT);
      pt_load<D>(kbuf, &maps.k, kh, b.t0 + k0, &sh.kv_full);
      pt_load<D>(vbuf, &maps.v, kh, b.t0 + k0, &sh.kv_full);
      TcRing<C::QR> qr;
      TcRing<C::OR> orr;
      int h = h0, block = tile;
      for (int i = 0; i < n; ++i) {
        const int tok = b.t0 + block * PT_B;
        ok = tc_wait(&sh.q_empty[qr.at], qr.parity ^ 1, &sh.dead);
        if (!ok) break;
        tc::bar_arrive_expect_tx(&sh.q_full[qr.at], C::SLOT);
        pt_load<D>(qslots + qr.at * C::SLOT, &maps.q, h, tok, &sh.q_full[qr.at]);
        ++sent_q;
        qr.step();
        if (a.test_stall && i == PT_STALL_AT) ok = tc_give_up(&sh.dead);
        ok = ok && tc_wait(&sh.o_empty[orr.at], orr.parity ^ 1, &sh.dead);
        if (!ok) break;
        tc::bar_arrive_expect_tx(&sh.o_full[orr.at], C::SLOT);
        pt_load<D>(oslots + orr.at * C::SLOT, &maps.d_out, h, tok, &sh.o_full[orr.at]);
        ++sent_o;
        orr.step();
        if (++block == tile + blocks) block = tile, ++h;
      }
      if (!ok) {
        // let what is on its way arrive before the CTA ends: the last round of every slot
        flag_status(a.status, KDA_DEV_TIMEOUT);
        tc::bar_wait(&sh.kv_full, 0, 1u << 16);
        for (int i = max(0, sent_q - C::QR); i < sent_q; ++i) tc::bar_wait(&sh.q_full[i % C::QR], i / C::QR & 1, 1u << 16);
        for (int i = max(0, sent_o - C::OR); i < sent_o; ++i) tc::bar_wait(&sh.o_full[i % C::OR], i / C::OR & 1, 1u << 16);
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---- products
    if (lane == 0) {
      bool ok = tc_wait(&sh.kv_full, 0, &sh.dead);
      const uint64_t kd = tc::sdesc(tc::smem_u32(kbuf)), vd = tc::sdesc(tc::smem_u32(vbuf));
      const uint64_t q_s = tc::sdesc(tc::smem_u32(qslots)), o_s = tc::sdesc(tc::smem_u32(oslots));
      const uint64_t q_r = tc::sdesc_mn(tc::smem_u32(qslots), PT_HALF), o_r = tc::sdesc_mn(tc::smem_u32(oslots), PT_HALF);
      constexpr int STEP = C::SLOT / 16;
      TcRing<C::QR> q_next, q_now;   // of the scores to form next, and of the gradients'
      TcRing<C::OR> o_next, o_now;
      auto form_s = [&]() {
        ok = ok && tc_wait(&sh.q_ready[q_next.at], q_next.parity, &sh.dead);
        if (!ok) return;
        tc::fence_after_sync();
        scores_mma<D>(t_s, kd, q_s + q_next.at * STEP);
        tc::commit(&sh.s_full);
        q_next.step();
      };
      auto form_dp = [&]() {
        ok = ok && tc_wait(&sh.o_ready[o_next.at], o_next.parity, &sh.dead);
        if (!ok) return;
        tc::fence_after_sync();
        scores_mma<D>(t_dp, vd, o_s + o_next.at * STEP);
        tc::commit(&sh.dp_full);
        o_next.step();
      };
      form_s();
      form_dp();
      for (int i = 0; ok && i < n; ++i) {
        ok = tc_wait(&sh.p_full, i & 1, &sh.dead);
        if (!ok) break;
        tc::fence_after_sync();
        rows_mma<D>(t_dv, t_s, o_r + o_now.at * STEP, i == 0);
        tc::commit(&sh.o_empty[o_now.at]);
        o_now.step();
        // the next scores go where these probabilities lie: products run in the order of their issue
        if (i + 1 < n) form_s();
        ok = ok && tc_wait(&sh.ds_full, i & 1, &sh.dead);
        if (!ok) break;
        tc::fence_after_sync();
        rows_mma<D>(t_dk, t_dp, q_r + q_now.at * STEP, i == 0);
        tc::commit(&sh.q_empty[q_now.at]);
        q_now.step();
        if (i + 1 < n) form_dp();
      }
      // nothing of this thread's is on its way when the CTA ends
      if (ok) tc::commit(&sh.out_full);
      else flag_status(a.status, KDA_DEV_TIMEOUT);
      tc::commit(&sh.drain);
      tc::bar_wait(&sh.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ---- statistics, and rows behind the sequence
    const int t = tid - 320;
    TcRing<C::QR> qr;
    TcRing<C::OR> orr;
    TcRing<2> st;
    bool ok = true;
    int h = h0, block = tile;
    float2 next[2];
    auto fetch = [&]() {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = block * PT_B + t + 64 * r;
        next[r] = row < b.len ? __ldg(stats + (int64_t)h * a.T + b.t0 + row) : make_float2(0.f, 0.f);
      }
    };
    fetch();
    for (int i = 0; i < n; ++i) {
      const int rows = b.len - block * PT_B;  // of the sequence, from the block on
      ok = ok && tc_wait(&sh.st_empty[st.at], st.parity ^ 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
#pragma unroll
      for (int r = 0; r < 2; ++r) sh.minus_lse[st.at][t + 64 * r] = -next[r].x, sh.minus_d[st.at][t + 64 * r] = -next[r].y;
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.st_full[st.at]);
      st.step();
      if (++block == tile + blocks) block = tile, ++h;
      if (i + 1 < n) fetch();
      ok = tc_wait(&sh.q_full[qr.at], qr.parity, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (rows < PT_B) clear_behind<D>(qslots + qr.at * C::SLOT, rows, t);
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.q_ready[qr.at]);
      qr.step();
      ok = tc_wait(&sh.o_full[orr.at], orr.parity, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (rows < PT_B) clear_behind<D>(oslots + orr.at * C::SLOT, rows, t);
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.o_ready[orr.at]);
      orr.step();
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  } else {
    // ---- arithmetic: thread = key, and 64 of a block's queries
    const int half = warp >> 2, key = k0 + (tid & 127);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, own_s = t_s + half * 64 + lanes, own_dp = t_dp + half * 64 + lanes;
    const float cap2 = a.softcap * PA_LOG2E, factor = a.scale * (CAP ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E);
    bool ok = true;
    TcRing<2> st;
    int block = tile;
    for (int i = 0; i < n; ++i) {
      const int row0 = block * PT_B + half * 64;
      const bool masked = block == tile || (block + 1) * PT_B > b.len || (block + 1) * PT_B - k0 > window;
      if (++block == tile + blocks) block = tile;
      ok = ok && tc_wait(&sh.st_full[st.at], st.parity, &sh.dead) && tc_wait(&sh.s_full, i & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      float2 x[32];
      tc::tmem_ld64(own_s, reinterpret_cast<float*>(x));
      if constexpr (CAP) pt_cap(x, factor, cap2);
      const float4* lse = reinterpret_cast<const float4*>(sh.minus_lse[st.at] + half * 64);
      const float4* dd = reinterpret_cast<const float4*>(sh.minus_d[st.at] + half * 64);
      // the key is seen by queries from .. to - 1 of the 64
      const int from = masked ? key - row0 : 0, to = masked ? (int)min((int64_t)b.len, (int64_t)key + window) - row0 : 64;
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float4 minus = lse[(16 * c + j) / 2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = 16 * c + j + e;
            const float2 ml = e == 0 ? make_float2(minus.x, minus.y) : make_float2(minus.z, minus.w);
            float2 p = CAP ? add2(x[at], ml) : fma2(x[at], both(factor), ml);
            p = make_float2(ex2(p.x), ex2(p.y));
            if (masked) {
              if (2 * at < from || 2 * at >= to) p.x = 0.f;
              if (2 * at + 1 < from || 2 * at + 1 >= to) p.y = 0.f;
            }
            w[j + e] = pack_bf16(p.x, p.y);
            if constexpr (CAP) {  // times the cap's slope from here on
              const float2 y = mul2(x[at], both(1.f / cap2));
              p = mul2(p, fma2(mul2(y, both(-1.f)), y, both(1.f)));
              if (masked) {
                if (2 * at < from || 2 * at >= to) p.x = 0.f;
                if (2 * at + 1 < from || 2 * at + 1 >= to) p.y = 0.f;
              }
            }
            x[at] = p;
          }
        }
        tc::tmem_st16(own_s + 16 * c, w);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.p_full);
      ok = tc_wait(&sh.dp_full, i & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      float2 dp[32];
      tc::tmem_ld64(own_dp, reinterpret_cast<float*>(dp));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float4 minus = dd[(16 * c + j) / 2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int at = 16 * c + j + e;
            const float2 md = e == 0 ? make_float2(minus.x, minus.y) : make_float2(minus.z, minus.w);
            float2 ds = mul2(x[at], add2(dp[at], md));
            if (masked) {
              if (2 * at < from || 2 * at >= to) ds.x = 0.f;
              if (2 * at + 1 < from || 2 * at + 1 >= to) ds.y = 0.f;
            }
            w[j + e] = pack_bf16(ds.x, ds.y);
          }
        }
        tc::tmem_st16(own_dp + 16 * c, w);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.ds_full), tc::bar_arrive(&sh.st_empty[st.at]);
      st.step();
    }
    ok = ok && tc_wait(&sh.out_full, 0, &sh.dead);
    ok = __all_sync(0xffffffffu, ok);
    tc::fence_after_sync();
    if (ok) {
      // the first half of the warps has dv, the second dk
      const bool mine = key - k0 < keys;
      const int64_t t = b.t0 + key;
      const uint32_t from = (half ? t_dk : t_dv) + lanes;
      const float by = half ? a.scale : 1.f;
      if (nparts > 1) {
        float* to = parts + (int64_t)(part * 2 + half) * a.T * a.Hkv * a.d;
        store_rows<D>(to, false, (t * a.Hkv + kh) * a.d, from, by, a.d, mine);
      } else {
        store_rows<D>(half ? g.dk : g.dv, g.bf16, t * (half ? g.dk_stride : g.dv_stride) + (int64_t)kh * a.d, from, by, a.d, mine);
      }
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 8) tc::tmem_dealloc(tmem, PT_TMEM);
}

template <int D, bool CAP>
__global__ void __launch_bounds__(PT_NT, 1)
    prefill_attention_grad_queries_kernel(const __grid_constant__ PgMaps maps, const PromptAttnArgs a, const PromptGradArgs g,
                                          const float2* __restrict__ stats, const int64_t places) {
  using C = PgCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* qbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *obuf = qbuf + C::SLOT, *kslots = obuf + C::SLOT, *vslots = kslots + C::KR * C::SLOT;
  PgQueriesShared& sh = *reinterpret_cast<PgQueriesShared*>(vslots + C::VR * C::SLOT);
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int window = a.window > 0 ? a.window : 0x7fffffff;
  const int h = blockIdx.x % a.Hq, kh = h / (a.Hq / a.Hkv);
  const PfBlock b = pf_block<7>(a, places - 1 - blockIdx.x / a.Hq);  // the longest rows first
  if (b.len == 0) return;
  const int rows = min(PT_B, b.len - b.row0);
  const int lo = max(0, b.row0 - window + 1) / PT_B, n = b.row0 / PT_B - lo + 1;

  if (tid == 0) {
    tc::bar_init(&sh.q_full, 1);
    for (int i = 0; i < C::KR; ++i) tc::bar_init(&sh.k_full[i], 1), tc::bar_init(&sh.k_ready[i], 2), tc::bar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < C::VR; ++i) tc::bar_init(&sh.v_full[i], 1), tc::bar_init(&sh.v_empty[i], 1);
    tc::bar_init(&sh.s_full, 1), tc::bar_init(&sh.s_read, 8);
    for (int i = 0; i < 2; ++i) tc::bar_init(&sh.dp_full[i], 1), tc::bar_init(&sh.ds_full[i], 8);
    tc::bar_init(&sh.out_full, 1), tc::bar_init(&sh.drain, 1);
    tc::bar_fence_init();
    sh.dead = 0;
  }
  if (warp == 8) tc::tmem_alloc(&sh.tmem, PT_TMEM);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem, t_s = tmem, t_dp = tmem + 128, t_dq = tmem + 384;  // two buffers of dp

  if (warp == 9) {
    // ---- loads
    if (lane == 0) {
      bool ok = true;
      int sent_k = 0, sent_v = 0;
      tc::bar_arrive_expect_tx(&sh.q_full, 2 * C::SLOT);
      pt_load<D>(qbuf, &maps.q, h, b.t0 + b.row0, &sh.q_full);
      pt_load<D>(obuf, &maps.d_out, h, b.t0 + b.row0, &sh.q_full);
      TcRing<C::KR> kr;
      TcRing<C::VR> vr;
      for (int i = 0; i < n; ++i) {
        const int tok = b.t0 + (lo + i) * PT_B;
        ok = tc_wait(&sh.k_empty[kr.at], kr.parity ^ 1, &sh.dead);
        if (!ok) break;
        tc::bar_arrive_expect_tx(&sh.k_full[kr.at], C::SLOT);
        pt_load<D>(kslots + kr.at * C::SLOT, &maps.k, kh, tok, &sh.k_full[kr.at]);
        ++sent_k;
        kr.step();
        if (a.test_stall && i == PT_STALL_AT) ok = tc_give_up(&sh.dead);
        ok = ok && tc_wait(&sh.v_empty[vr.at], vr.parity ^ 1, &sh.dead);
        if (!ok) break;
        tc::bar_arrive_expect_tx(&sh.v_full[vr.at], C::SLOT);
        pt_load<D>(vslots + vr.at * C::SLOT, &maps.v, kh, tok, &sh.v_full[vr.at]);
        ++sent_v;
        vr.step();
      }
      if (!ok) {
        flag_status(a.status, KDA_DEV_TIMEOUT);
        tc::bar_wait(&sh.q_full, 0, 1u << 16);
        for (int i = max(0, sent_k - C::KR); i < sent_k; ++i) tc::bar_wait(&sh.k_full[i % C::KR], i / C::KR & 1, 1u << 16);
        for (int i = max(0, sent_v - C::VR); i < sent_v; ++i) tc::bar_wait(&sh.v_full[i % C::VR], i / C::VR & 1, 1u << 16);
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ---- products
    if (lane == 0) {
      bool ok = tc_wait(&sh.q_full, 0, &sh.dead);
      const uint64_t qd = tc::sdesc(tc::smem_u32(qbuf)), od = tc::sdesc(tc::smem_u32(obuf));
      const uint64_t k_s = tc::sdesc(tc::smem_u32(kslots)), v_s = tc::sdesc(tc::smem_u32(vslots));
      const uint64_t k_r = tc::sdesc_mn(tc::smem_u32(kslots), PT_HALF);
      constexpr int STEP = C::SLOT / 16;
      TcRing<C::KR> k_next, k_now;
      TcRing<C::VR> vr;
      TcRing<2> dp_next, dp_now;
      auto form = [&]() {  // scores and dp of the next tile
        ok = ok && tc_wait(&sh.k_ready[k_next.at], k_next.parity, &sh.dead);
        if (!ok) return;
        tc::fence_after_sync();
        scores_mma<D>(t_s, qd, k_s + k_next.at * STEP);
        tc::commit(&sh.s_full);
        k_next.step();
        ok = tc_wait(&sh.v_full[vr.at], vr.parity, &sh.dead);
        if (!ok) return;
        tc::fence_after_sync();
        scores_mma<D>(t_dp + dp_next.at * 128, od, v_s + vr.at * STEP);
        tc::commit(&sh.dp_full[dp_next.at]);
        tc::commit(&sh.v_empty[vr.at]);
        vr.step();
        dp_next.step();
      };
      form();
      for (int i = 0; ok && i < n; ++i) {
        if (i + 1 < n) {
          ok = tc_wait(&sh.s_read, i & 1, &sh.dead);
          if (ok) form();
        }
        ok = ok && tc_wait(&sh.ds_full[dp_now.at], dp_now.parity, &sh.dead);
        if (!ok) break;
        tc::fence_after_sync();
        rows_mma<D>(t_dq, t_dp + dp_now.at * 128, k_r + k_now.at * STEP, i == 0);
        tc::commit(&sh.k_empty[k_now.at]);
        k_now.step();
        dp_now.step();
      }
      if (ok) tc::commit(&sh.out_full);
      else flag_status(a.status, KDA_DEV_TIMEOUT);
      tc::commit(&sh.drain);
      tc::bar_wait(&sh.drain, 0);
    }
    __syncwarp();
  } else if (warp >= 10) {
    // ---- keys behind the sequence
    TcRing<C::KR> kr;
    bool ok = true;
    for (int i = 0; i < n; ++i, kr.step()) {
      ok = tc_wait(&sh.k_full[kr.at], kr.parity, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const int left = b.len - (lo + i) * PT_B;
      if (left < PT_B) clear_behind<D>(kslots + kr.at * C::SLOT, left, tid - 320);
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.k_ready[kr.at]);
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  } else {
    // ---- arithmetic: thread = query, and 64 of a tile's keys
    const int half = warp >> 2, row = b.row0 + (tid & 127);
    const bool mine = row - b.row0 < rows;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, own_s = t_s + half * 64 + lanes;
    const float cap2 = a.softcap * PA_LOG2E, factor = a.scale * (CAP ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E);
    const float2 stat = mine ? __ldg(stats + (int64_t)h * a.T + b.t0 + row) : make_float2(0.f, 0.f);
    const float2 minus_lse = both(-stat.x), minus_d = both(-stat.y);
    bool ok = true;
    TcRing<2> buf;
    for (int i = 0; i < n; ++i, buf.step()) {
      const int k0 = (lo + i) * PT_B, first = k0 + half * 64;
      const bool masked = k0 + PT_B - 1 > b.row0 || k0 <= b.row0 + PT_B - 1 - window;
      // of the 64 the row sees keys from .. to - 1; a row behind the sequence none
      const int to = !masked ? 64 : mine ? row + 1 - first : 0, from = masked && row - first >= window ? row - first - window + 1 : 0;
      ok = ok && tc_wait(&sh.s_full, i & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      float2 x[32];
      tc::tmem_ld64(own_s, reinterpret_cast<float*>(x));
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.s_read);
      if constexpr (CAP) pt_cap(x, factor, cap2);
#pragma unroll
      for (int at = 0; at < 32; ++at) {
        float2 p = CAP ? add2(x[at], minus_lse) : fma2(x[at], both(factor), minus_lse);
        p = make_float2(ex2(p.x), ex2(p.y));
        if constexpr (CAP) {
          const float2 y = mul2(x[at], both(1.f / cap2));
          p = mul2(p, fma2(mul2(y, both(-1.f)), y, both(1.f)));
        }
        x[at] = p;
      }
      ok = tc_wait(&sh.dp_full[buf.at], buf.parity, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      const uint32_t own_dp = t_dp + buf.at * 128 + half * 64 + lanes;
      float2 dp[32];
      tc::tmem_ld64(own_dp, reinterpret_cast<float*>(dp));
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int at = 16 * c + j;
          float2 ds = mul2(x[at], add2(dp[at], minus_d));
          if (masked) {
            if (2 * at < from || 2 * at >= to) ds.x = 0.f;
            if (2 * at + 1 < from || 2 * at + 1 >= to) ds.y = 0.f;
          }
          w[j] = pack_bf16(ds.x, ds.y);
        }
        tc::tmem_st16(own_dp + 16 * c, w);
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.ds_full[buf.at]);
    }
    ok = ok && tc_wait(&sh.out_full, 0, &sh.dead);
    ok = __all_sync(0xffffffffu, ok);
    tc::fence_after_sync();
    if (ok && half == 0) {
      store_rows<D>(g.dq, g.bf16, (b.t0 + (int64_t)row) * g.dq_stride + (int64_t)h * a.d, t_dq + lanes, a.scale, a.d, mine);
      if (tid == 0) add_work(a.status, rows);
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 8) tc::tmem_dealloc(tmem, PT_TMEM);
}

// dv and dk of a block's keys: the parts' sum, in order.  A thread has 4 channels of a row.
__global__ void __launch_bounds__(256) pg_join_kernel(const PromptAttnArgs a, const PromptGradArgs g, const float* __restrict__ parts,
                                                      const int nparts) {
  pdl_begin();
  const PfBlock b = pf_block<7>(a, blockIdx.x);
  if (b.len == 0) return;
  const int per_row = a.d / 4, rows = min(PT_B, b.len - b.row0), kh = blockIdx.y >> 1, which = blockIdx.y & 1;
  const int64_t step = 2 * a.T * a.Hkv * a.d;
  for (int i = threadIdx.x; i < rows * per_row; i += 256) {
    const int r = i / per_row, c = (i - r * per_row) * 4;
    const int64_t t = b.t0 + b.row0 + r;
    const float* p = parts + which * (step / 2) + (t * a.Hkv + kh) * a.d + c;
    float4 sum = __ldg(reinterpret_cast<const float4*>(p));
    for (int n = 1; n < nparts; ++n) {
      const float4 x = __ldg(reinterpret_cast<const float4*>(p + n * step));
      sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
    }
    const int64_t at = t * (which ? g.dk_stride : g.dv_stride) + (int64_t)kh * a.d + c;
    void* to = which ? g.dk : g.dv;
    if (g.bf16) *reinterpret_cast<uint2*>(static_cast<bf16*>(to) + at) = make_uint2(pack_bf16(sum.x, sum.y), pack_bf16(sum.z, sum.w));
    else *reinterpret_cast<float4*>(static_cast<float*>(to) + at) = sum;
  }
}

template <int D, bool CAP>
cudaError_t grad_launch(const PromptAttnArgs& a, const PromptGradArgs& g, const float2* stats, float* parts, int nparts, cudaStream_t s) {
  auto keys = prefill_attention_grad_keys_kernel<D, CAP>;
  auto queries = prefill_attention_grad_queries_kernel<D, CAP>;
  cudaError_t e = cudaFuncSetAttribute(keys, cudaFuncAttributeMaxDynamicSharedMemorySize, pg_keys_smem<D>());
  if (e == cudaSuccess) e = cudaFuncSetAttribute(queries, cudaFuncAttributeMaxDynamicSharedMemorySize, pg_queries_smem<D>());
  if (e != cudaSuccess) return e;
  PgMaps maps;
  if (!encode_rows_map_sw128(&maps.q, a.q, a.T, a.Hq, a.d, a.q_stride, PT_B) ||
      !encode_rows_map_sw128(&maps.k, a.k, a.T, a.Hkv, a.d, a.k_stride, PT_B) ||
      !encode_rows_map_sw128(&maps.v, a.v, a.T, a.Hkv, a.d, a.v_stride, PT_B) ||
      !encode_rows_map_sw128(&maps.d_out, g.d_out, a.T, a.Hq, a.d, g.d_out_stride, PT_B))
    return cudaErrorInvalidValue;
  const int64_t places = pf_places(a.T, a.N, PT_B);
  if (places * a.Hq > 0x7fffffff) return cudaErrorInvalidValue;
  e = launch_pdl(keys, dim3((unsigned)(places * a.Hkv * nparts)), dim3(PT_NT), pg_keys_smem<D>(), s, maps, a, g, stats, parts, nparts);
  if (e != cudaSuccess) return e;
  if (nparts > 1) {
    e = launch_pdl(pg_join_kernel, dim3((unsigned)places, 2 * a.Hkv), dim3(256), 0, s, a, g, parts, nparts);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(queries, dim3((unsigned)(places * a.Hq)), dim3(PT_NT), pg_queries_smem<D>(), s, maps, a, g, stats, places);
}

}  // namespace

// How many CTAs share the query heads of a block of keys: enough for two blocks per SM, by the tokens alone (the host knows no
// lengths).
int pg_parts(int64_t T, int Hq, int Hkv) {
  const int64_t blocks = (T + PT_B - 1) / PT_B * Hkv;
  const int64_t want = blocks > 0 ? 2 * 152 / blocks : 1;
  const int64_t most = Hq / Hkv < PG_MOST_PARTS ? Hq / Hkv : PG_MOST_PARTS;
  return (int)(want < 1 ? 1 : want > most ? most : want);
}

cudaError_t pf_tc_grad(const PromptAttnArgs& a, const PromptGradArgs& g, const float2* stats, float* parts, cudaStream_t s) {
  const bool cap = a.softcap > 0.f;
  const int n = pg_parts(a.T, a.Hq, a.Hkv);
  if (a.d == 128) return cap ? grad_launch<128, true>(a, g, stats, parts, n, s) : grad_launch<128, false>(a, g, stats, parts, n, s);
  return cap ? grad_launch<64, true>(a, g, stats, parts, n, s) : grad_launch<64, false>(a, g, stats, parts, n, s);
}

}  // namespace kda
