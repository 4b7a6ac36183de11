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
// A query that sees one key has p = 1 and dx = 0 exactly, whatever p (from the rounded log-sum-exp) and D come out as: the keys' kernel takes
// it as a row of zeros with a log-sum-exp of 0, the queries' as one that sees nothing.
// D_i from the forward's output carries that output's rounding, d_out . (o rounded - o): against dx's own size it matters in rows that see
// few keys (over many, o and its rounding shrink with the mean, and what is wrong in D meets the keys' mean).  So before both,
//   means:   in blocks of queries that walk up to PG_FEW tiles, D_i = sum_j p_ij (do_i . v_j) in fp32, by the queries' kernel without
//            its third product.
// Where keys' blocks are too few for the SMs (one key/value head for all queries), the group's heads are dealt to several CTAs, whose
// fp32 parts a third kernel adds up in order.
// As in the forward, one CTA per SM walks units and takes over those that have not started, the most work first.  Its warps: the
// arithmetic's, thread = row and one of PG_GROUPS parts of the tile's columns; one for the products; one for units and loads (TMA);
// and two that clear what lies behind the sequence in tiles that are column operands (0 * NaN), and bring the queries' statistics.
// p and dx are rounded to bf16 (2^-8) for their products, as the results are, but dx for dq, where that rounding left 1.5 times the
// results' own error: it goes in as two bf16, as both do in sequences of one block.  Everything else is fp32.
//
// Measured (backward alone): 8 documents of 8192 tokens, 32 / 8 heads of 128: 522 to 542 us, keys some 262, queries 238, means 25, statistics 37 (their
// starts and ends overlap); 8192 tokens, 12 heads: 591 us and, when it goes on, up to 626, 820 to 870 TFLOP/s of the five products, 1310 to 1390
// with those formed twice.  Bound by
// the chain of products and arithmetic, and by shared memory's bandwidth: 61 % of the products' pipe, in the keys' kernel 79 % of
// shared memory's, half of that the queries' statistics that all threads read.  Handing those to the products instead, as
// six more channels, came out the same (522 -> 520 us), so they stay here.
#include "device.h"
#include "prefill_attention_tc.cuh"

namespace kda {

namespace {

constexpr int PG_MOST_PARTS = 16;
constexpr int PG_FEW = 3;  // tiles
constexpr int PG_GROUPS = 4;               // (2 with twice the columns: backward of 8192 tokens, 12 heads of 128, 566 us against 548)
constexpr int PG_COLS = PT_B / PG_GROUPS;  // columns of a thread
constexpr int PG_SOFT = 128 * PG_GROUPS, PG_NT = PG_SOFT + 128, PG_W = PG_SOFT / 32;

template <int D>
struct PgCfg {
  static constexpr int SLOT = D / 64 * PT_HALF;
  static constexpr int QR = D == 128 ? 2 : 3, OR = D == 128 ? 2 : 3;  // keys' kernel: slots of Q, of dO
  static constexpr int KR = 3, VR = D == 128 ? 2 : 3;                 // queries' kernel: slots of K, of V
};

struct PgMaps {
  CUtensorMap q, k, v, d_out;
};

// A block of keys with query heads h0 .. h1 - 1: a round is a block of one head's queries, `blocks` of them from number `tile` on.
struct PgKeysUnit {
  int t0, len, k0, tile, blocks, kh, part, h0, h1;  // len = 0: no more units
};
// A block of a head's queries: n tiles of keys from number lo on.
struct PgQueriesUnit {
  int t0, len, row0, h, lo, n;
};

struct PgKeysShared {
  // every barrier is waited on only by roles that see each of its rounds
  PtFeed feed;
  uint64_t kv_full, kv_empty, q_full[3], q_ready[3], q_empty[3], o_full[3], o_ready[3], o_empty[3], st_full[2], st_empty[2];
  uint64_t s_full, p_full, dp_full, ds_full, out_full, drain;
  alignas(16) float minus_lse[2][PT_B], minus_d[2][PT_B];  // of a block's queries: log-sum-exp in powers of two, D
  PgKeysUnit unit[2];
  uint32_t tmem;
  int dead;
};
struct PgQueriesShared {
  PtFeed feed;
  uint64_t q_full, q_empty, k_full[3], k_ready[3], k_empty[3], v_full[3], v_empty[3];
  uint64_t s_full, s_read, dp_full[2], ds_full[2], out_full, drain;
  PgQueriesUnit unit[2];
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

// Registers of a thread: 640 threads with 96 each were launched; 512 x 104 + 128 x 64 is as many.
__device__ __forceinline__ void more_registers() {
  if constexpr (PG_GROUPS == 4) asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
}
__device__ __forceinline__ void fewer_registers() {
  if constexpr (PG_GROUPS == 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
}

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

// The first `rows` rows become zeros.
template <int D>
__device__ __forceinline__ void clear_first(unsigned char* tile, int rows, int t) {
  for (int i = t; i < rows * 8 * (D / 64); i += 64) {
    const int half = i / (rows * 8);
    *reinterpret_cast<uint4*>(tile + half * PT_HALF + (i - half * rows * 8) * 16) = make_uint4(0, 0, 0, 0);
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
// to (128 x D) += the 128 x 128 bf16 in tensor memory at `a` (each thread's columns over its own scores; TWO: with what that rounding
// left beside them) times rows of b
template <int D, bool TWO = false>
__device__ __forceinline__ void rows_mma(uint32_t to, uint32_t a, uint64_t b, bool first) {
#pragma unroll
  for (int kk = 0; kk < PT_B / 16; ++kk) {  // 16 rows per step
    const uint32_t at = a + kk * 16 / PG_COLS * PG_COLS + kk * 16 % PG_COLS / 2;
    tc::mma_ts(to, at, b + kk * (2048 / 16), pt_idesc(D) | tc::IDESC_B_MN, !(first && kk == 0));
    if (TWO) tc::mma_ts(to, at + PG_COLS / 2, b + kk * (2048 / 16), pt_idesc(D) | tc::IDESC_B_MN, 1);
  }
}

// Channels c0 .. c0 + N - 1 of a warp's 32 rows of a block's result in tensor memory, times `by`; `at`: the first row's first channel.
template <int N>
__device__ __forceinline__ void store_rows(void* base, bool is_bf16, int64_t at, int64_t stride, int rows, uint32_t from, int c0, float by, int d) {
  static_assert(N % 32 == 0, "32 at a time");
#pragma unroll 1
  for (int c = c0; c < min(c0 + N, d); c += 32) {
    float o[32];
    tc::tmem_ld32(from + c, o);
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] *= by;
    pt_store32(base, is_bf16, at + c, stride, rows, d - c, o);
  }
}

__device__ __forceinline__ void ld_columns(uint32_t at, float2 (&x)[PG_COLS / 2]) {
  if constexpr (PG_COLS == 64) tc::tmem_ld64(at, reinterpret_cast<float*>(x));
  else tc::tmem_ld32(at, reinterpret_cast<float*>(x));
}
// bf16 pairs over the columns that they come from
__device__ __forceinline__ void st_columns(uint32_t at, const uint32_t (&w)[PG_COLS / 2]) {
#pragma unroll
  for (int c = 0; c < PG_COLS / 2; c += 16) tc::tmem_st16(at + c, w + c);
  tc::tmem_wait_st();
}
__device__ __forceinline__ float2 only(float2 x, int i, int from, int to) {  // of columns i and i + 1 those from .. to - 1
  return make_float2(i < from || i >= to ? 0.f : x.x, i + 1 < from || i + 1 >= to ? 0.f : x.y);
}
// The cap's slope at a score in powers of two.
__device__ __forceinline__ float2 cap_slope(float2 x, float over_cap2) {
  const float2 y = mul2(x, both(over_cap2));
  return fma2(mul2(y, both(-1.f)), y, both(1.f));
}

struct Yes {
  static constexpr bool value = true;
};
struct No {
  static constexpr bool value = false;
};

// Whether p and dx go into dv's and dk's products as two bf16: in sequences of one block.  Few terms average little of a rounding out: dk's
// error against 64 bits, relative to its size, was 0.0023 to 0.0034 for two tokens, up to twice that of the formula in fp32 rounded once, and
// 0.0025 for 39, 1.5 times; now it is 0.0017 to 0.0019 in both, as the formula's.  Longer sequences keep 1.4 times, and four
// products instead of six.  The roles take such units in loops of their own: where both kinds shared one, its instructions cost the others
// (forward and gradients, 8 documents: 658 us without, 673 in one loop, 661 so).
__device__ __forceinline__ bool pg_twice(int len) { return len <= PT_B; }

// Block id % PG_FEW of sequence id / PG_FEW.
__device__ __forceinline__ PfBlock pg_first_block(const PromptAttnArgs& a, int id) {
  PfBlock b{0, 0, 0};
  const int i = id / PG_FEW, row0 = (id - i * PG_FEW) * PT_B;
  if (i >= a.N) return b;
  const int c0 = __ldcg(a.cu + i), c1 = __ldcg(a.cu + i + 1);
  if (c0 < 0 || c1 < c0 || c1 > a.T || c1 - c0 > a.max_seqlen || row0 >= c1 - c0) return b;
  b.t0 = c0, b.len = c1 - c0, b.row0 = row0;
  return b;
}

template <int D, bool CAP>
__global__ void __launch_bounds__(PG_NT, 1)
    prefill_attention_grad_keys_kernel(const __grid_constant__ PgMaps maps, const PromptAttnArgs a, const PromptGradArgs g,
                                       const float2* __restrict__ stats, float* __restrict__ parts, const int nparts, const int64_t places) {
  using C = PgCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* kbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *vbuf = kbuf + C::SLOT, *qslots = vbuf + C::SLOT, *oslots = qslots + C::QR * C::SLOT;
  PgKeysShared& sh = *reinterpret_cast<PgKeysShared*>(oslots + C::OR * C::SLOT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int window = a.window > 0 ? a.window : 0x7fffffff;

  if (tid == 0) {
    sh.feed.init(PG_W + 1 + 2);
    tc::bar_init(&sh.kv_full, 1), tc::bar_init(&sh.kv_empty, 1);
    for (int i = 0; i < C::QR; ++i) tc::bar_init(&sh.q_full[i], 1), tc::bar_init(&sh.q_ready[i], 2), tc::bar_init(&sh.q_empty[i], 1);
    for (int i = 0; i < C::OR; ++i) tc::bar_init(&sh.o_full[i], 1), tc::bar_init(&sh.o_ready[i], 2), tc::bar_init(&sh.o_empty[i], 1);
    for (int i = 0; i < 2; ++i) tc::bar_init(&sh.st_full[i], 2), tc::bar_init(&sh.st_empty[i], PG_W);
    tc::bar_init(&sh.s_full, 1), tc::bar_init(&sh.p_full, PG_W), tc::bar_init(&sh.dp_full, 1), tc::bar_init(&sh.ds_full, PG_W);
    tc::bar_init(&sh.out_full, 1), tc::bar_init(&sh.drain, 1);
    tc::bar_fence_init();
    sh.dead = 0;
  }
  if (tid == PG_SOFT + 32)
    tc::prefetch_map(&maps.q), tc::prefetch_map(&maps.k), tc::prefetch_map(&maps.v), tc::prefetch_map(&maps.d_out);
  if (warp == PG_W) tc::tmem_alloc(&sh.tmem, PT_TMEM);
  pdl_begin();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  if (warp == PG_W + 1) {
    // ---- units, and their loads
    fewer_registers();
    PfRanks<7> ranks(a);
    bool ok = true, more = true;
    int sent_q = 0, sent_o = 0, units = 0, id = blockIdx.x;
    TcRing<2> un;
    TcRing<C::QR> qr;
    TcRing<C::OR> orr;
    const int group = a.Hq / a.Hkv;
    while (more) {
      const int col = id % (a.Hkv * nparts);
      // the first keys first: most queries see them
      const PfBlock b = pf_ranked(a, ranks, id / (a.Hkv * nparts), places, true);
      if (b.len > 0) {
        PgKeysUnit u;
        u.t0 = b.t0, u.len = b.len, u.k0 = b.row0, u.tile = b.row0 / PT_B;
        u.kh = col / nparts, u.part = col - u.kh * nparts;
        u.h0 = u.kh * group + u.part * group / nparts, u.h1 = u.kh * group + (u.part + 1) * group / nparts;
        const int keys = min(PT_B, b.len - b.row0);
        const int last = (int)min((int64_t)b.len - 1, (int64_t)b.row0 + keys - 2 + window);  // the last query that sees one of the keys
        u.blocks = last / PT_B - u.tile + 1;
        ok = tc_wait_warp(&sh.feed.empty[un.at], un.parity ^ 1, &sh.dead);
        if (!ok) break;
        if (lane == 0) {
          sh.unit[un.at] = u;
          tc::bar_arrive(&sh.feed.full[un.at]);
          ok = tc_wait(&sh.kv_empty, (units & 1) ^ 1, &sh.dead);
          if (ok) {
            tc::bar_arrive_expect_tx(&sh.kv_full, 2 * C::SLOT);
            pt_load<D>(kbuf, &maps.k, u.kh, u.t0 + u.k0, &sh.kv_full);
            pt_load<D>(vbuf, &maps.v, u.kh, u.t0 + u.k0, &sh.kv_full);
            ++units;
          }
          const int n = u.blocks * (u.h1 - u.h0);
          int h = u.h0, block = u.tile;
          for (int i = 0; ok && i < n; ++i) {
            const int tok = u.t0 + block * PT_B;
            ok = tc_wait(&sh.q_empty[qr.at], qr.parity ^ 1, &sh.dead);
            if (!ok) break;
            tc::bar_arrive_expect_tx(&sh.q_full[qr.at], C::SLOT);
            pt_load<D>(qslots + qr.at * C::SLOT, &maps.q, h, tok, &sh.q_full[qr.at]);
            ++sent_q;
            qr.step();
            if (i + 1 == n) sh.feed.ask();
            if (a.test_stall && i == PT_STALL_AT) ok = tc_give_up(&sh.dead);
            ok = ok && tc_wait(&sh.o_empty[orr.at], orr.parity ^ 1, &sh.dead);
            if (!ok) break;
            tc::bar_arrive_expect_tx(&sh.o_full[orr.at], C::SLOT);
            pt_load<D>(oslots + orr.at * C::SLOT, &maps.d_out, h, tok, &sh.o_full[orr.at]);
            ++sent_o;
            orr.step();
            if (++block == u.tile + u.blocks) block = u.tile, ++h;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        un.step();
      } else if (lane == 0) {
        sh.feed.ask();
      }
      if (id == 0) pf_check_offsets(a);  // once in a call: whichever CTA walks the unit
      ok = sh.feed.answered(&sh.dead, id);
      if (!ok) break;
      more = id >= 0;
    }
    if (ok) {
      ok = tc_wait_warp(&sh.feed.empty[un.at], un.parity ^ 1, &sh.dead);
      if (lane == 0 && ok) {
        sh.unit[un.at].len = 0;
        tc::bar_arrive(&sh.feed.full[un.at]);
      }
    }
    if (!ok && lane == 0) {
      // let what is on its way arrive before the CTA ends: the last round of every slot
      flag_status(a.status, KDA_DEV_TIMEOUT);
      sh.feed.drain();
      if (units > 0) tc::bar_wait(&sh.kv_full, (units - 1) & 1, 1u << 16);
      for (int i = max(0, sent_q - C::QR); i < sent_q; ++i) tc::bar_wait(&sh.q_full[i % C::QR], i / C::QR & 1, 1u << 16);
      for (int i = max(0, sent_o - C::OR); i < sent_o; ++i) tc::bar_wait(&sh.o_full[i % C::OR], i / C::OR & 1, 1u << 16);
    }
    __syncwarp();
  } else if (warp == PG_W) {
    // ---- products: the warp waits and counts as one, one lane issues
    fewer_registers();
    bool ok = true;
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem), t_s = tm, t_dp = tm + 128, t_dv = tm + 256, t_dk = tm + 384;
    const uint64_t kd = tc::sdesc(tc::smem_u32(kbuf)), vd = tc::sdesc(tc::smem_u32(vbuf));
    const uint64_t q_s = tc::sdesc(tc::smem_u32(qslots)), o_s = tc::sdesc(tc::smem_u32(oslots));
    const uint64_t q_r = tc::sdesc_mn(tc::smem_u32(qslots), PT_HALF), o_r = tc::sdesc_mn(tc::smem_u32(oslots), PT_HALF);
    constexpr int STEP = C::SLOT / 16;
    TcRing<2> un;
    TcRing<C::QR> q_next, q_now;  // of the scores to form next, and of the gradients'
    TcRing<C::OR> o_next, o_now;
    uint32_t p_parity = 0, ds_parity = 0;
    auto form_s = [&]() {
      ok = ok && tc_wait_warp(&sh.q_ready[q_next.at], q_next.parity, &sh.dead);
      if (!ok) return;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        scores_mma<D>(t_s, kd, q_s + q_next.at * STEP);
        tc::commit(&sh.s_full);
      }
      q_next.step();
    };
    auto form_dp = [&](bool last) {
      ok = ok && tc_wait_warp(&sh.o_ready[o_next.at], o_next.parity, &sh.dead);
      if (!ok) return;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        scores_mma<D>(t_dp, vd, o_s + o_next.at * STEP);
        tc::commit(&sh.dp_full);
        if (last) tc::commit(&sh.kv_empty);
      }
      o_next.step();
    };
    for (uint32_t kv_parity = 0;; kv_parity ^= 1, un.step()) {
      ok = tc_wait_warp(&sh.feed.full[un.at], un.parity, &sh.dead);
      if (!ok) break;
      const PgKeysUnit& u = sh.unit[un.at];
      // numbers that are known to be the same for all lanes
      const int end = __reduce_max_sync(0xffffffffu, u.len), n = __reduce_max_sync(0xffffffffu, u.blocks * (u.h1 - u.h0));
      if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
      __syncwarp();
      if (end == 0) break;
      ok = tc_wait_warp(&sh.kv_full, kv_parity, &sh.dead);
      form_s();
      form_dp(n == 1);
      auto walk = [&](auto two) {
        for (int i = 0; ok && i < n; ++i) {
          ok = tc_wait_warp(&sh.p_full, p_parity, &sh.dead);
          if (!ok) break;
          p_parity ^= 1;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            rows_mma<D, decltype(two)::value>(t_dv, t_s, o_r + o_now.at * STEP, i == 0);
            tc::commit(&sh.o_empty[o_now.at]);
          }
          o_now.step();
          // the next scores go where these probabilities lie: products run in the order of their issue
          if (i + 1 < n) form_s();
          ok = ok && tc_wait_warp(&sh.ds_full, ds_parity, &sh.dead);
          if (!ok) break;
          ds_parity ^= 1;
          tc::fence_after_sync();
          if (tc::elect_one()) {
            rows_mma<D, decltype(two)::value>(t_dk, t_dp, q_r + q_now.at * STEP, i == 0);
            tc::commit(&sh.q_empty[q_now.at]);
            if (i + 1 == n) tc::commit(&sh.out_full);
          }
          q_now.step();
          if (i + 1 < n) form_dp(i + 2 == n);
        }
      };
      if (pg_twice(end)) walk(Yes());
      else walk(No());
      if (!ok) break;
    }
    // nothing of this warp's is on its way when the CTA ends
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    __syncwarp();
    if (tc::elect_one()) tc::commit(&sh.drain);
    tc::bar_wait(&sh.drain, 0);
    __syncwarp();
  } else if (warp >= PG_W + 2) {
    // ---- statistics, and rows behind the sequence
    fewer_registers();
    const int t = tid - PG_SOFT - 64;
    TcRing<C::QR> qr;
    TcRing<C::OR> orr;
    TcRing<2> st, un;
    bool ok = true;
    for (;; un.step()) {
      ok = tc_wait_warp(&sh.feed.full[un.at], un.parity, &sh.dead);
      if (!ok) break;
      const PgKeysUnit u = sh.unit[un.at];
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
      if (u.len == 0) break;
      const int n = u.blocks * (u.h1 - u.h0);
      int h = u.h0, block = u.tile;
      const int single = window == 1 ? 0x7fffffff : 1;  // queries at positions below see one key
      float2 next[2];
      auto fetch = [&]() {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = block * PT_B + t + 64 * r;
          next[r] = row < u.len ? __ldg(stats + (int64_t)h * a.T + u.t0 + row) : make_float2(0.f, 0.f);
          if (row < single) next[r].x = 0.f;
        }
      };
      fetch();
      for (int i = 0; i < n; ++i) {
        const int rows = u.len - block * PT_B, alone = min(PT_B, single - block * PT_B);  // of the sequence, from the block on; that see one key
        ok = tc_wait_warp(&sh.st_empty[st.at], st.parity ^ 1, &sh.dead);
        if (!ok) break;
#pragma unroll
        for (int r = 0; r < 2; ++r) sh.minus_lse[st.at][t + 64 * r] = -next[r].x, sh.minus_d[st.at][t + 64 * r] = -next[r].y;
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.st_full[st.at]);
        st.step();
        if (++block == u.tile + u.blocks) block = u.tile, ++h;
        if (i + 1 < n) fetch();
        ok = tc_wait_warp(&sh.q_full[qr.at], qr.parity, &sh.dead);
        if (!ok) break;
        if (rows < PT_B) clear_behind<D>(qslots + qr.at * C::SLOT, rows, t);
        if (alone > 0) clear_first<D>(qslots + qr.at * C::SLOT, alone, t);
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.q_ready[qr.at]);
        qr.step();
        ok = tc_wait_warp(&sh.o_full[orr.at], orr.parity, &sh.dead);
        if (!ok) break;
        if (rows < PT_B) clear_behind<D>(oslots + orr.at * C::SLOT, rows, t);
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.o_ready[orr.at]);
        orr.step();
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  } else {
    // ---- arithmetic: thread = key, and PG_COLS of a block's queries
    more_registers();
    const int part = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, t_s = tmem, t_dp = tmem + 128, t_dv = tmem + 256, t_dk = tmem + 384;
    const uint32_t own_s = t_s + part * PG_COLS + lanes, own_dp = t_dp + part * PG_COLS + lanes;
    const float cap2 = a.softcap * PA_LOG2E, factor = pt_factor(a.scale, CAP ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E), over_cap2 = 1.f / cap2;
    bool ok = true;
    TcRing<2> st, un;
    uint32_t s_parity = 0, dp_parity = 0, out_parity = 0;
    for (;; un.step()) {
      ok = tc_wait_warp(&sh.feed.full[un.at], un.parity, &sh.dead);
      if (!ok) break;
      const PgKeysUnit u = sh.unit[un.at];
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
      if (u.len == 0) break;
      const int key = u.k0 + (tid & 127), n = u.blocks * (u.h1 - u.h0);
      int block = u.tile;
      auto rounds = [&](auto two) {
        for (int i = 0; i < n; ++i) {
          const int row0 = block * PT_B + part * PG_COLS;
          const bool masked = block == u.tile || (block + 1) * PT_B > u.len || (block + 1) * PT_B - u.k0 > window;
          // of the thread's queries the key is seen by from .. to - 1
          const int from = key - row0, to = (int)min((int64_t)u.len, (int64_t)key + window) - row0;
          if (++block == u.tile + u.blocks) block = u.tile;
          ok = tc_wait(&sh.st_full[st.at], st.parity, &sh.dead) && tc_wait(&sh.s_full, s_parity, &sh.dead);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          s_parity ^= 1;
          tc::fence_after_sync();
          float2 x[PG_COLS / 2];
          const float4* lse = reinterpret_cast<const float4*>(sh.minus_lse[st.at] + part * PG_COLS);
          const float4* dd = reinterpret_cast<const float4*>(sh.minus_d[st.at] + part * PG_COLS);
          ld_columns(own_s, x);
          if constexpr (CAP) pt_cap(x, factor, cap2);
          // x becomes the probabilities, times the cap's slope
          auto probabilities = [&](auto some) {
            uint32_t w[PG_COLS / 2], rest[PG_COLS / 2];
#pragma unroll
            for (int j = 0; j < PG_COLS / 2; j += 2) {
              const float4 minus = lse[j / 2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float2 ml = e == 0 ? make_float2(minus.x, minus.y) : make_float2(minus.z, minus.w);
                float2 p = CAP ? add2(x[j + e], ml) : fma2(x[j + e], both(factor), ml);
                p = make_float2(ex2(p.x), ex2(p.y));
                if (decltype(some)::value) p = only(p, 2 * (j + e), from, to);
                if (decltype(two)::value) tc::split_pair(p.x, p.y, w[j + e], rest[j + e]);
                else w[j + e] = pack_bf16(p.x, p.y);
                x[j + e] = CAP ? mul2(p, cap_slope(x[j + e], over_cap2)) : p;
              }
            }
            if (decltype(two)::value) tc::tmem_st16(own_s + PG_COLS / 2, rest);
            st_columns(own_s, w);
          };
          if (decltype(two)::value || masked) probabilities(Yes());
          else probabilities(No());
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(&sh.p_full);
          ok = tc_wait_warp(&sh.dp_full, dp_parity, &sh.dead);
          if (!ok) break;
          dp_parity ^= 1;
          tc::fence_after_sync();
          float2 dp[PG_COLS / 2];
          ld_columns(own_dp, dp);
          auto slopes = [&](auto some) {
            uint32_t w[PG_COLS / 2], rest[PG_COLS / 2];
#pragma unroll
            for (int j = 0; j < PG_COLS / 2; j += 2) {
              const float4 minus = dd[j / 2];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const float2 md = e == 0 ? make_float2(minus.x, minus.y) : make_float2(minus.z, minus.w);
                float2 ds = mul2(x[j + e], add2(dp[j + e], md));
                if (decltype(some)::value) ds = only(ds, 2 * (j + e), from, to);
                if (decltype(two)::value) tc::split_pair(ds.x, ds.y, w[j + e], rest[j + e]);
                else w[j + e] = pack_bf16(ds.x, ds.y);
              }
            }
            if (decltype(two)::value) tc::tmem_st16(own_dp + PG_COLS / 2, rest);
            st_columns(own_dp, w);
          };
          if (decltype(two)::value || masked) slopes(Yes());
          else slopes(No());
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) tc::bar_arrive(&sh.ds_full), tc::bar_arrive(&sh.st_empty[st.at]);
          st.step();
        }
      };
      if (pg_twice(u.len)) rounds(Yes());
      else rounds(No());
      if (!ok) break;
      ok = tc_wait_warp(&sh.out_full, out_parity, &sh.dead);
      if (!ok) break;
      out_parity ^= 1;
      tc::fence_after_sync();
      // the first half of the parts has dv, the second dk, each its channels
      constexpr int N = D * 2 / PG_GROUPS;
      const int of_k = part / (PG_GROUPS / 2), c0 = part % (PG_GROUPS / 2) * N;
      const int warp_row = (warp & 3) * 32, rows = u.len - u.k0 - warp_row;  // of the sequence, from the warp's first on
      const int64_t t = u.t0 + u.k0 + warp_row;
      const uint32_t from = (of_k ? t_dk : t_dv) + lanes;
      const float by = of_k ? a.scale : 1.f;
      if (nparts > 1) {
        float* to = parts + (int64_t)(u.part * 2 + of_k) * a.T * a.Hkv * a.d;
        store_rows<N>(to, false, (t * a.Hkv + u.kh) * a.d, (int64_t)a.Hkv * a.d, rows, from, c0, by, a.d);
      } else {
        const int64_t stride = of_k ? g.dk_stride : g.dv_stride;
        store_rows<N>(of_k ? g.dk : g.dv, g.bf16, t * stride + (int64_t)u.kh * a.d, stride, rows, from, c0, by, a.d);
      }
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == PG_W) tc::tmem_dealloc(tmem, PT_TMEM);
}

template <int D, bool CAP, bool MEANS>
__global__ void __launch_bounds__(PG_NT, 1)
    prefill_attention_grad_queries_kernel(const __grid_constant__ PgMaps maps, const PromptAttnArgs a, const PromptGradArgs g,
                                          float2* __restrict__ stats, const int64_t places, const bool firsts) {
  using C = PgCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* qbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char *obuf = qbuf + C::SLOT, *kslots = obuf + C::SLOT, *vslots = kslots + C::KR * C::SLOT;
  PgQueriesShared& sh = *reinterpret_cast<PgQueriesShared*>(vslots + C::VR * C::SLOT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int window = a.window > 0 ? a.window : 0x7fffffff;

  if (tid == 0) {
    sh.feed.init(PG_W + 1 + 2);
    tc::bar_init(&sh.q_full, 1), tc::bar_init(&sh.q_empty, 1);
    for (int i = 0; i < C::KR; ++i) tc::bar_init(&sh.k_full[i], 1), tc::bar_init(&sh.k_ready[i], 2), tc::bar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < C::VR; ++i) tc::bar_init(&sh.v_full[i], 1), tc::bar_init(&sh.v_empty[i], 1);
    tc::bar_init(&sh.s_full, 1), tc::bar_init(&sh.s_read, PG_W);
    for (int i = 0; i < 2; ++i) tc::bar_init(&sh.dp_full[i], 1), tc::bar_init(&sh.ds_full[i], PG_W);
    tc::bar_init(&sh.out_full, 1), tc::bar_init(&sh.drain, 1);
    tc::bar_fence_init();
    sh.dead = 0;
  }
  if (tid == PG_SOFT + 32)
    tc::prefetch_map(&maps.q), tc::prefetch_map(&maps.k), tc::prefetch_map(&maps.v), tc::prefetch_map(&maps.d_out);
  if (warp == PG_W) tc::tmem_alloc(&sh.tmem, PT_TMEM);
  if constexpr (MEANS) {
    pdl_begin();
  } else {
    // No wait for the kernel before, the keys': nothing of it is read here.  That one's blocks let this start only when each had
    // waited for the statistics itself, and the statistics are read past L1.
    tc::pdl_launch_dependents();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  if (warp == PG_W + 1) {
    // ---- units, and their loads
    fewer_registers();
    PfRanks<7> ranks(a);
    bool ok = true, more = true;
    int sent_k = 0, sent_v = 0, units = 0, id = blockIdx.x;
    TcRing<2> un;
    TcRing<C::KR> kr;
    TcRing<C::VR> vr;
    while (more) {
      // the longest rows first; of the sequences' first blocks in their own order
      const PfBlock b = MEANS && firsts ? pg_first_block(a, id / a.Hq) : pf_ranked(a, ranks, id / a.Hq, places, false);
      PgQueriesUnit u;
      u.t0 = b.t0, u.len = b.len, u.row0 = b.row0, u.h = id % a.Hq;
      u.lo = max(0, b.row0 - window + 1) / PT_B, u.n = b.row0 / PT_B - u.lo + 1;
      if (b.len > 0 && (!MEANS || u.n <= PG_FEW)) {
        ok = tc_wait_warp(&sh.feed.empty[un.at], un.parity ^ 1, &sh.dead);
        if (!ok) break;
        if (lane == 0) {
          sh.unit[un.at] = u;
          tc::bar_arrive(&sh.feed.full[un.at]);
          const int kh = u.h / (a.Hq / a.Hkv);
          for (int i = 0; i < u.n; ++i) {
            const int tok = u.t0 + (u.lo + i) * PT_B;
            ok = tc_wait(&sh.k_empty[kr.at], kr.parity ^ 1, &sh.dead);
            if (!ok) break;
            tc::bar_arrive_expect_tx(&sh.k_full[kr.at], C::SLOT);
            pt_load<D>(kslots + kr.at * C::SLOT, &maps.k, kh, tok, &sh.k_full[kr.at]);
            ++sent_k;
            kr.step();
            if (i == 0) {
              ok = tc_wait(&sh.q_empty, (units & 1) ^ 1, &sh.dead);
              if (!ok) break;
              tc::bar_arrive_expect_tx(&sh.q_full, 2 * C::SLOT);
              pt_load<D>(qbuf, &maps.q, u.h, u.t0 + u.row0, &sh.q_full);
              pt_load<D>(obuf, &maps.d_out, u.h, u.t0 + u.row0, &sh.q_full);
              ++units;
            }
            if (i + 1 == u.n) sh.feed.ask();
            if (a.test_stall && i == PT_STALL_AT) ok = tc_give_up(&sh.dead);
            ok = ok && tc_wait(&sh.v_empty[vr.at], vr.parity ^ 1, &sh.dead);
            if (!ok) break;
            tc::bar_arrive_expect_tx(&sh.v_full[vr.at], C::SLOT);
            pt_load<D>(vslots + vr.at * C::SLOT, &maps.v, kh, tok, &sh.v_full[vr.at]);
            ++sent_v;
            vr.step();
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        un.step();
      } else if (lane == 0) {
        sh.feed.ask();
      }
      ok = sh.feed.answered(&sh.dead, id);
      if (!ok) break;
      more = id >= 0;
    }
    if (ok) {
      ok = tc_wait_warp(&sh.feed.empty[un.at], un.parity ^ 1, &sh.dead);
      if (lane == 0 && ok) {
        sh.unit[un.at].len = 0;
        tc::bar_arrive(&sh.feed.full[un.at]);
      }
    }
    if (!ok && lane == 0) {
      flag_status(a.status, KDA_DEV_TIMEOUT);
      sh.feed.drain();
      if (units > 0) tc::bar_wait(&sh.q_full, (units - 1) & 1, 1u << 16);
      for (int i = max(0, sent_k - C::KR); i < sent_k; ++i) tc::bar_wait(&sh.k_full[i % C::KR], i / C::KR & 1, 1u << 16);
      for (int i = max(0, sent_v - C::VR); i < sent_v; ++i) tc::bar_wait(&sh.v_full[i % C::VR], i / C::VR & 1, 1u << 16);
    }
    __syncwarp();
  } else if (warp == PG_W) {
    // ---- products: the warp waits and counts as one, one lane issues
    fewer_registers();
    bool ok = true;
    const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem), t_s = tm, t_dp = tm + 128, t_dq = tm + 384;  // two buffers of dp
    const uint64_t qd = tc::sdesc(tc::smem_u32(qbuf)), od = tc::sdesc(tc::smem_u32(obuf));
    const uint64_t k_s = tc::sdesc(tc::smem_u32(kslots)), v_s = tc::sdesc(tc::smem_u32(vslots));
    const uint64_t k_r = tc::sdesc_mn(tc::smem_u32(kslots), PT_HALF);
    constexpr int STEP = C::SLOT / 16;
    TcRing<2> un, dp_next, dp_now;
    TcRing<C::KR> k_next, k_now;
    TcRing<C::VR> vr;
    uint32_t read_parity = 0;
    auto form = [&](bool last) {  // scores and dp of the next tile
      ok = ok && tc_wait_warp(&sh.k_ready[k_next.at], k_next.parity, &sh.dead);
      if (!ok) return;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        scores_mma<D>(t_s, qd, k_s + k_next.at * STEP);
        tc::commit(&sh.s_full);
      }
      k_next.step();
      ok = tc_wait_warp(&sh.v_full[vr.at], vr.parity, &sh.dead);
      if (!ok) return;
      tc::fence_after_sync();
      if (tc::elect_one()) {
        scores_mma<D>(t_dp + dp_next.at * 128, od, v_s + vr.at * STEP);
        tc::commit(&sh.dp_full[dp_next.at]);
        tc::commit(&sh.v_empty[vr.at]);
        if (last) tc::commit(&sh.q_empty);
      }
      vr.step();
      dp_next.step();
    };
    for (uint32_t q_parity = 0;; q_parity ^= 1, un.step()) {
      ok = tc_wait_warp(&sh.feed.full[un.at], un.parity, &sh.dead);
      if (!ok) break;
      const int end = __reduce_max_sync(0xffffffffu, sh.unit[un.at].len), n = __reduce_max_sync(0xffffffffu, sh.unit[un.at].n);
      if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
      __syncwarp();
      if (end == 0) break;
      ok = tc_wait_warp(&sh.q_full, q_parity, &sh.dead);
      form(n == 1);
      for (int i = 0; ok && i < n; ++i) {
        ok = tc_wait_warp(&sh.s_read, read_parity, &sh.dead);
        read_parity ^= 1;
        if (ok && i + 1 < n) form(i + 2 == n);
        ok = ok && tc_wait_warp(&sh.ds_full[dp_now.at], dp_now.parity, &sh.dead);
        if (!ok) break;
        tc::fence_after_sync();
        if (tc::elect_one()) {
          if (!MEANS) rows_mma<D, true>(t_dq, t_dp + dp_now.at * 128, k_r + k_now.at * STEP, i == 0);
          tc::commit(&sh.k_empty[k_now.at]);
          if (!MEANS && i + 1 == n) tc::commit(&sh.out_full);
        }
        k_now.step();
        dp_now.step();
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    __syncwarp();
    if (tc::elect_one()) tc::commit(&sh.drain);
    tc::bar_wait(&sh.drain, 0);
    __syncwarp();
  } else if (warp >= PG_W + 2) {
    // ---- keys behind the sequence
    fewer_registers();
    TcRing<2> un;
    TcRing<C::KR> kr;
    bool ok = true;
    for (;; un.step()) {
      ok = tc_wait_warp(&sh.feed.full[un.at], un.parity, &sh.dead);
      if (!ok) break;
      const PgQueriesUnit u = sh.unit[un.at];
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
      if (u.len == 0) break;
      for (int i = 0; i < u.n; ++i, kr.step()) {
        ok = tc_wait_warp(&sh.k_full[kr.at], kr.parity, &sh.dead);
        if (!ok) break;
        const int left = u.len - (u.lo + i) * PT_B;
        if (left < PT_B) clear_behind<D>(kslots + kr.at * C::SLOT, left, tid - PG_SOFT - 64);
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.k_ready[kr.at]);
      }
      if (!ok) break;
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  } else {
    // ---- arithmetic: thread = query, and PG_COLS of a tile's keys
    more_registers();
    const int part = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, t_s = tmem, t_dp = tmem + 128, t_dq = tmem + 384;
    const uint32_t own_s = t_s + part * PG_COLS + lanes;
    const float cap2 = a.softcap * PA_LOG2E, factor = pt_factor(a.scale, CAP ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E), over_cap2 = 1.f / cap2;
    bool ok = true;
    TcRing<2> un, buf;
    uint32_t s_parity = 0, out_parity = 0;
    int rows_done = 0;
    // The warps of the mean's sum meet at a unit's start and end: a wait that ran out in one ends all, so that none waits in vain.
    auto meet = [&]() { ok = !tc::named_bar_or(1, PG_SOFT, !ok); };
    for (;; un.step()) {
      ok = tc_wait_warp(&sh.feed.full[un.at], un.parity, &sh.dead);
      if (MEANS) meet();
      if (!ok) break;
      const PgQueriesUnit u = sh.unit[un.at];
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
      if (u.len == 0) break;
      const int row = u.row0 + (tid & 127);
      const bool mine = row < u.len, sees = mine && (MEANS || (row > 0 && window > 1));
      const float2 stat = mine ? __ldcg(stats + (int64_t)u.h * a.T + u.t0 + row) : make_float2(0.f, 0.f);
      const float2 minus_lse = both(-stat.x), minus_d = both(-stat.y);
      float2 mean = both(0.f);
      for (int i = 0; i < u.n; ++i, buf.step()) {
        const int k0 = (u.lo + i) * PT_B, first = k0 + part * PG_COLS;
        const bool masked = k0 + PT_B - 1 > u.row0 || k0 <= u.row0 + PT_B - 1 - window;
        // of the thread's keys the row sees from .. to - 1; a row behind the sequence none, nor for dx one that sees a single key
        const int to = sees ? row + 1 - first : 0, from = row - first >= window ? row - first - window + 1 : 0;
        ok = tc_wait_warp(&sh.s_full, s_parity, &sh.dead);
        if (!ok) break;
        s_parity ^= 1;
        tc::fence_after_sync();
        float2 x[PG_COLS / 2];
        ld_columns(own_s, x);
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.s_read);
        if constexpr (CAP) pt_cap(x, factor, cap2);
#pragma unroll
        for (int j = 0; j < PG_COLS / 2; ++j) {
          float2 p = CAP ? add2(x[j], minus_lse) : fma2(x[j], both(factor), minus_lse);
          p = make_float2(ex2(p.x), ex2(p.y));
          x[j] = CAP && !MEANS ? mul2(p, cap_slope(x[j], over_cap2)) : p;
        }
        ok = tc_wait_warp(&sh.dp_full[buf.at], buf.parity, &sh.dead);
        if (!ok) break;
        tc::fence_after_sync();
        const uint32_t own_dp = t_dp + buf.at * 128 + part * PG_COLS + lanes;
        float2 dp[PG_COLS / 2];
        ld_columns(own_dp, dp);
        auto slopes = [&](auto some) {
          uint32_t w[PG_COLS / 2], rest[PG_COLS / 2];
#pragma unroll
          for (int j = 0; j < PG_COLS / 2; ++j) {
            float2 ds = mul2(x[j], MEANS ? dp[j] : add2(dp[j], minus_d));
            if (decltype(some)::value) ds = only(ds, 2 * j, from, to);
            if (MEANS) mean = add2(mean, ds);
            else tc::split_pair(ds.x, ds.y, w[j], rest[j]);
          }
          if (!MEANS) {
            tc::tmem_st16(own_dp + PG_COLS / 2, rest);
            st_columns(own_dp, w);
          }
        };
        if (masked) slopes(Yes());
        else slopes(No());
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.ds_full[buf.at]);
      }
      if constexpr (MEANS) {
        // the parts' sums of a row meet in tensor memory, in places that take turns
        float sums[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) sums[i] = mean.x + mean.y;
        const uint32_t at = t_dq + lanes + un.at * 32;
        tc::tmem_st8f(at + part * 8, sums);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        meet();
        if (!ok) break;
        tc::fence_after_sync();
        if (part == 0) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < PG_GROUPS; ++i) {
            tc::tmem_ld8(at + i * 8, sums);
            sum += sums[0];
          }
          if (mine) stats[(int64_t)u.h * a.T + u.t0 + row].y = sum;
        }
        continue;
      }
      if (!ok) break;
      ok = tc_wait_warp(&sh.out_full, out_parity, &sh.dead);
      if (!ok) break;
      out_parity ^= 1;
      tc::fence_after_sync();
      constexpr int N = D / PG_GROUPS < 32 ? 32 : D / PG_GROUPS;
      const int warp_row = (warp & 3) * 32;
      if (part * N < D)
        store_rows<N>(g.dq, g.bf16, (u.t0 + (int64_t)u.row0 + warp_row) * g.dq_stride + (int64_t)u.h * a.d, g.dq_stride,
                      u.len - u.row0 - warp_row, t_dq + lanes, part * N, a.scale, a.d);
      rows_done += min(PT_B, u.len - u.row0);
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    if (!MEANS && tid == 0) add_work(a.status, rows_done);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == PG_W) tc::tmem_dealloc(tmem, PT_TMEM);
  if (!MEANS) tc::pdl_wait();  // what comes after this kernel comes after the keys' too
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
cudaError_t grad_launch(const PromptAttnArgs& a, const PromptGradArgs& g, float2* stats, float* parts, int nparts, cudaStream_t s) {
  auto keys = prefill_attention_grad_keys_kernel<D, CAP>;
  auto queries = prefill_attention_grad_queries_kernel<D, CAP, false>;
  auto means = prefill_attention_grad_queries_kernel<D, CAP, true>;
  cudaError_t e = cudaFuncSetAttribute(keys, cudaFuncAttributeMaxDynamicSharedMemorySize, pg_keys_smem<D>());
  if (e == cudaSuccess) e = cudaFuncSetAttribute(means, cudaFuncAttributeMaxDynamicSharedMemorySize, pg_queries_smem<D>());
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
  const bool firsts = !(a.window > 0 && a.window <= (PG_FEW - 1) * PT_B + 1) && (int64_t)PG_FEW * a.N <= places;
  e = launch_pdl(means, dim3((unsigned)((firsts ? (int64_t)PG_FEW * a.N : places) * a.Hq)), dim3(PG_NT), pg_queries_smem<D>(), s, maps, a, g,
                 stats, places, firsts);
  if (e != cudaSuccess) return e;
  e = launch_pdl(keys, dim3((unsigned)(places * a.Hkv * nparts)), dim3(PG_NT), pg_keys_smem<D>(), s, maps, a, g, stats, parts, nparts, places);
  if (e != cudaSuccess) return e;
  e = launch_pdl(queries, dim3((unsigned)(places * a.Hq)), dim3(PG_NT), pg_queries_smem<D>(), s, maps, a, g, stats, places, false);
  if (e != cudaSuccess || nparts == 1) return e;
  return launch_pdl(pg_join_kernel, dim3((unsigned)places, 2 * a.Hkv), dim3(256), 0, s, a, g, parts, nparts);
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

cudaError_t pf_tc_grad(const PromptAttnArgs& a, const PromptGradArgs& g, float2* stats, float* parts, cudaStream_t s) {
  const bool cap = a.softcap > 0.f;
  const int n = pg_parts(a.T, a.Hq, a.Hkv);
  if (a.d == 128) return cap ? grad_launch<128, true>(a, g, stats, parts, n, s) : grad_launch<128, false>(a, g, stats, parts, n, s);
  return cap ? grad_launch<64, true>(a, g, stats, parts, n, s) : grad_launch<64, false>(a, g, stats, parts, n, s);
}

}  // namespace kda
