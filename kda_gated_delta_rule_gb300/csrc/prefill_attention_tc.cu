// Attention over packed prompts on the 5th-generation tensor cores: bf16 inputs, any head size.
//
// A unit is two blocks of 128 query rows that share their keys: the same tokens of two heads of a group where the group has an
// even number, else two neighbouring blocks of one head.  Per 128 keys and block, S = Q K^T (rows x keys) in tensor memory; a
// thread has one row of it, so its maximum and sum need no exchange; P = exp2(S - reference) goes back as bf16 over the
// scores it came from, as the row operand of O += P V.  While one block's softmax runs, the other's products do.
// One CTA per SM walks units: the grid has a CTA for each, and one that runs takes over the next that has not started, the longest
// rows first, so that a unit's start lies under the end of the one before.
//   warps 0 to 3, 4 to 7   softmax of block 0, 1
//   warp 8     issues the products (one thread)
//   warp 9     takes units, and brings their Q, and K and V tiles into rings, by TMA (128-byte swizzle; channels beyond d as zeros)
//   warps 10, 11   look at the V tiles with unseen keys: rows behind the sequence become zeros, values that are no numbers
//              too (0 * NaN would reach rows that do not see them); rows that do see one get it at the end
//
// The softmax's reference moves only when a score is 2^8 above it, so accumulators are hardly ever rescaled; the thread of the row does
// it, after the products that the scores' barrier already covers.  Probabilities are rounded to bf16 (2^-8) for the second
// product, half a step like the output's own rounding; their sum is taken before that, in fp32.
//
// Measured: 16384 tokens, 32 / 8 heads of 128: 1300 to 1410 us by the clocks, 1560 to 1690 TFLOP/s of cuBLAS' 1921; 16 prompts of 32771 tokens, 12 / 4
// heads: 309 to 317 us (1260 to 1290); window 1024 and cap 30, 16 / 2 heads of 64: 209 to 231 us; one of 137 tokens 11 to 12.  Bound by the chain of scores,
// softmax, products of each block (the products' pipe 57 to 62 % busy, no other fuller): two blocks per CTA because one alone leaves the pipe
// idle half the time, a whole row per thread because halves (sixteen warps) took 1432 us for 1425, tiles of 128 keys because 64 take as
// much of shared memory's bandwidth per product (1756).  Registers are shared out anew among the roles (setmaxnreg): without that 2
// to 5 % longer.  Heads of 64 halve the products and not the softmax: 897 to 912 TFLOP/s without window or cap.
#include "device.h"
#include "prefill_attention_tc.cuh"

namespace kda {

namespace {

constexpr int PT_O = 256;  // columns: scores of the two blocks, then their accumulators
constexpr float PT_SLACK = 8.f;

template <int D>
struct PtCfg {
  static constexpr int HALVES = D / 64;
  static constexpr int SLOT = HALVES * PT_HALF;
  static constexpr int KR = D == 128 ? 3 : 4, VR = D == 128 ? 2 : 4;
};

struct PtMaps {
  CUtensorMap q, k, v;
};

template <int N>
struct Count {
  static constexpr int value = N;
};

// The two blocks of a unit, and the key tiles that they walk.
struct PtUnit {
  int t0, len;  // len = 0: no more units
  int row0[2], head[2], rows[2];  // rows = 0: no such block
  int lo, hi[2], top;             // tiles lo .. hi[s]; top: the larger hi
  int kv_head;
};

struct PtShared {
  // every barrier is waited on only by roles that see each of its rounds
  PtFeed feed;
  uint64_t k_full[4], k_empty[4], v_full[4], v_ready[4], v_empty[4];
  uint64_t q_full, q_empty, s_full[2], p_full[2], o_full[2], drain;
  PtUnit unit[2];
  int odd_v[2];  // by unit: a value that is no number was left out
  uint32_t tmem;
  int dead;
};
template <int D>
constexpr int pt_smem() {
  using C = PtCfg<D>;
  return 1024 + (2 + C::KR + C::VR) * C::SLOT + (int)sizeof(PtShared);
}
static_assert(pt_smem<128>() <= 227 * 1024, "shared memory of one SM");

template <bool BY_HEADS>
__device__ __forceinline__ PtUnit pt_unit(const PromptAttnArgs& a, PfRanks<BY_HEADS ? 7 : 8>& ranks, int64_t places, int pairs, int id,
                                          int window) {
  const int pair = id % pairs;
  const PfBlock b = pf_ranked(a, ranks, id / pairs, places, false);
  PtUnit u;
  u.t0 = b.t0, u.len = b.len;
  u.top = -1;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    u.head[s] = BY_HEADS ? 2 * pair + s : pair;
    u.row0[s] = BY_HEADS ? b.row0 : b.row0 + s * PT_B;
    u.rows[s] = max(0, min(PT_B, b.len - u.row0[s]));
    u.hi[s] = u.rows[s] > 0 ? (u.row0[s] + u.rows[s] - 1) / PT_B : -1;
    u.top = max(u.top, u.hi[s]);
  }
  u.lo = max(0, u.row0[0] - window + 1) / PT_B;
  u.kv_head = u.head[0] / (a.Hq / a.Hkv);
  return u;
}
// Whether some row of the unit does not see some key of the tile.
__device__ __forceinline__ bool pt_masked(const PtUnit& u, int tile, int window) {
  const int k0 = tile * PT_B, last = u.rows[1] > 0 ? u.row0[1] + u.rows[1] - 1 : u.row0[0] + u.rows[0] - 1;
  return k0 + PT_B - 1 > u.row0[0] || k0 <= last - window;
}

// Zeros for the rows of a V tile from `keys` on, and for what is no number in the others; true where there was such.  Two warps.
template <int D>
__device__ __forceinline__ bool pt_clean(unsigned char* tile, int keys, int t) {
  constexpr int N = PT_B * 8 * (D / 64);  // pieces of 16 bytes: eight lie in a row's 128 bytes, in some order
  bool odd = false;
  uint4* pieces = reinterpret_cast<uint4*>(tile);
  const int whole = max(0, min(PT_B, keys)) * 8;  // pieces of a half that are rows of the sequence
#pragma unroll 1
  for (int i = whole + t; i < PT_B * 8; i += 64)
#pragma unroll
    for (int h = 0; h < D / 64; ++h) pieces[h * PT_B * 8 + i] = make_uint4(0, 0, 0, 0);
#pragma unroll 1
  for (int i0 = t; i0 < N; i0 += 64 * 8) {
    uint32_t any = 0;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
      const int i = i0 + 64 * n;
      const uint4 x = pieces[i];
      // an exponent of all ones carries into the next bit
      const uint32_t carry = ((x.x & 0x7f807f80u) + 0x00800080u) | ((x.y & 0x7f807f80u) + 0x00800080u) |
                             ((x.z & 0x7f807f80u) + 0x00800080u) | ((x.w & 0x7f807f80u) + 0x00800080u);
      any |= (i & (PT_B * 8 - 1)) < whole ? carry : 0u;
    }
    if (!(any & 0x80008000u)) continue;
#pragma unroll 1
    for (int n = 0; n < 8; ++n) {
      const int i = i0 + 64 * n;
      if ((i & (PT_B * 8 - 1)) >= whole) continue;
      uint32_t* w = reinterpret_cast<uint32_t*>(pieces + i);
      for (int c = 0; c < 4; ++c) {
        const uint32_t x = w[c], low = (x & 0x7f80u) == 0x7f80u, high = (x & 0x7f800000u) == 0x7f800000u;
        if (low || high) odd = true, w[c] = (low ? 0u : x & 0xffffu) | (high ? 0u : x & 0xffff0000u);
      }
    }
  }
  tc::fence_proxy_async();
  return odd;
}

// Which of 32 keys, from number `first` on, a row sees that sees from .. to - 1.
__device__ __forceinline__ uint32_t pt_seen(int first, int from, int to) {
  const int n = max(0, min(32, to - first)), skip = max(0, min(32, from - first));
  return (n < 32 ? (1u << n) - 1 : 0xffffffffu) & (skip < 32 ? 0xffffffffu << skip : 0u);
}
// `none` in the place of the scores of unseen keys.  A loop over 32 keys at a time: instructions that run once or twice in a unit are
// fetched for it, and most of the four have nothing to do.
__device__ __forceinline__ void pt_mask(uint32_t own_s, int from, int to, float none) {
#pragma unroll 1
  for (int c = 0; c < PT_B; c += 32) {
    const uint32_t seen = pt_seen(c, from, to);
    if (__all_sync(0xffffffffu, seen == 0xffffffffu)) continue;
    float x[32];
    tc::tmem_ld32(own_s + c, x);
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = seen >> i & 1 ? x[i] : none;
    tc::tmem_st32f(own_s + c, x);
  }
  tc::tmem_wait_st();
}

// Capped scores.  Which formula a score takes goes by its own product alone: the short polynomial up to `limit`, beyond it that of
// pt_cap.  A warp's votes only leave out what none of its scores takes, so that a row's bits do not depend on the other rows (and the
// next sequence's, which come along at a sequence's end) nor on keys that it does not see.  Where a warp has both kinds, both are worked out:
// window 1024, 16 / 2 heads of 64, 24001 tokens 209 us with cap 30, 408 with cap 6, 498 with cap 1 (318 and 402 when the warp chose one for all).
struct PtCap {
  CapNearer nearer;
  float factor, cap2;  // of a product, to the cap's argument; the cap in powers of two
  float limit;
  __device__ __forceinline__ PtCap(float factor, float cap2) : nearer(cap2, factor * (0.5f * PA_LN2)), factor(factor), cap2(cap2) {
    limit = factor > 0.f && nearer.usable() ? __fdividef(2.f * PA_LOG2E * PA_NEARER, factor) : -1.f;
  }
  // 16 scores in powers of two, less m
  __device__ __forceinline__ void less(const float2 (&x)[8], float m, float2 (&y)[8]) const {
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = fma2(x[i], nearer(x[i]), both(-m));
      far = fmaxf(far, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
    }
    if (__all_sync(0xffffffffu, far <= limit)) return;
    float2 z[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i];
    pt_cap(z, factor, cap2);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      z[i] = add2(z[i], both(-m));
      if (!(fabsf(x[i].x) <= limit)) y[i].x = z[i].x;
      if (!(fabsf(x[i].y) <= limit)) y[i].y = z[i].y;
    }
  }
  __device__ __forceinline__ float score(float s) const {
    if (fabsf(s) <= limit) return __fmul_rn(s, nearer(s));
    const float z = s * factor;
    return fabsf(z) <= PA_NEAR ? capped_near(z, cap2) : capped_far(z, cap2);
  }
};

// The largest capped score that a row sees of a tile, whose products stay in tensor memory.  `all_near`: halves of the keys that every row of
// the warp sees, within the short polynomial.
__device__ __forceinline__ float pt_capped_top(uint32_t own_s, bool masked, int from, int to, const PtCap& cap, int& all_near) {
  const bool falls = cap.factor < 0.f;  // the smallest product has the largest score
  float best = -INFINITY;
  if (masked) {
#pragma unroll 1
    for (int c = 0; c < PT_B; c += 32) {
      const uint32_t seen = pt_seen(c, from, to);
      if (__all_sync(0xffffffffu, seen == 0)) continue;
      float x[32];
      tc::tmem_ld32(own_s + c, x);
#pragma unroll
      for (int i = 0; i < 32; ++i) best = fmaxf(best, seen >> i & 1 ? (falls ? -x[i] : x[i]) : -INFINITY);
    }
    if (to <= 0 || from >= PT_B) return -INFINITY;
  } else {
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {
      float x[64], most[4], far[4];
      tc::tmem_ld64(own_s + 64 * half, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) far[i] = fabsf(x[i]), most[i] = x[i];
#pragma unroll
      for (int i = 4; i < 64; ++i) far[i & 3] = fmaxf(far[i & 3], fabsf(x[i])), most[i & 3] = fmaxf(most[i & 3], x[i]);
      if (falls) {
#pragma unroll
        for (int i = 0; i < 4; ++i) most[i] = -x[i];
#pragma unroll
        for (int i = 4; i < 64; ++i) most[i & 3] = fmaxf(most[i & 3], -x[i]);
      }
      best = fmaxf(best, fmaxf(fmaxf(most[0], most[1]), fmaxf(most[2], most[3])));
      if (__all_sync(0xffffffffu, fmaxf(fmaxf(far[0], far[1]), fmaxf(far[2], far[3])) <= cap.limit)) all_near |= 1 << half;
    }
  }
  return cap.score(falls ? -best : best);
}

// The sum of a channel's values that are no numbers, and so were left out of the tiles with unseen keys, over the keys that a row sees.
__device__ __noinline__ float pt_odd(const PromptAttnArgs& a, const PtUnit& u, int row, int hi, int window, int channel) {
  const bf16* v = static_cast<const bf16*>(a.v) + (int64_t)u.kv_head * a.d + channel;
  float sum = 0.f;
  for (int j = u.lo; j <= hi; ++j) {
    if (!pt_masked(u, j, window)) continue;
    for (int k = max(j * PT_B, row >= window ? row - window + 1 : 0); k <= min(j * PT_B + PT_B - 1, row); ++k) {
      const float x = to_f32(v[(int64_t)(u.t0 + k) * a.v_stride]);
      if (!(fabsf(x) <= 3.4e38f)) sum += x;
    }
  }
  return sum;
}

template <int D, bool CAP, bool BY_HEADS>
__global__ void __launch_bounds__(PT_NT, 1)
    prefill_attention_tc_kernel(const __grid_constant__ PtMaps maps, const PromptAttnArgs a, const int64_t places, const int pairs) {
  using C = PtCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* qbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* kslots = qbuf + 2 * C::SLOT;
  unsigned char* vslots = kslots + C::KR * C::SLOT;
  PtShared& sh = *reinterpret_cast<PtShared*>(vslots + C::VR * C::SLOT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int window = a.window > 0 ? a.window : 0x7fffffff;

  if (tid == 0) {
    sh.feed.init(8 + 1 + 2);
    for (int i = 0; i < C::KR; ++i) tc::bar_init(&sh.k_full[i], 1), tc::bar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < C::VR; ++i)
      tc::bar_init(&sh.v_full[i], 1), tc::bar_init(&sh.v_ready[i], 2), tc::bar_init(&sh.v_empty[i], 1);
    for (int i = 0; i < 2; ++i)
      tc::bar_init(&sh.s_full[i], 1), tc::bar_init(&sh.p_full[i], 4), tc::bar_init(&sh.o_full[i], 1);
    tc::bar_init(&sh.q_full, 1), tc::bar_init(&sh.q_empty, 1), tc::bar_init(&sh.drain, 1);
    tc::bar_fence_init();
    sh.dead = 0;
  }
  if (tid == 9 * 32) tc::prefetch_map(&maps.q), tc::prefetch_map(&maps.k), tc::prefetch_map(&maps.v);
  if (warp == 8) tc::tmem_alloc(&sh.tmem, PT_TMEM);
  pdl_begin();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  if (warp >= 8) {
    // 384 threads with 168 registers each were launched: 256 x 200 + 128 x 104 is as many
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 9) {
      // ---- units, and their loads
      PfRanks<BY_HEADS ? 7 : 8> ranks(a);
      bool ok = true, more = true;
      int sent_k = 0, sent_v = 0, units = 0, id = blockIdx.x;
      TcRing<2> un;
      TcRing<C::KR> kr;
      TcRing<C::VR> vr;
      while (more) {
        const PtUnit u = pt_unit<BY_HEADS>(a, ranks, places, pairs, id, window);
        if (u.len > 0) {
          ok = tc_wait(&sh.feed.empty[un.at], un.parity ^ 1, &sh.dead);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            sh.unit[un.at] = u, sh.odd_v[un.at] = 0;
            tc::bar_arrive(&sh.feed.full[un.at]);
            for (int j = u.lo; j <= u.top; ++j) {
              const int tok = u.t0 + j * PT_B;
              ok = tc_wait(&sh.k_empty[kr.at], kr.parity ^ 1, &sh.dead);
              if (!ok) break;
              tc::bar_arrive_expect_tx(&sh.k_full[kr.at], C::SLOT);
              pt_load<D>(kslots + kr.at * C::SLOT, &maps.k, u.kv_head, tok, &sh.k_full[kr.at]);
              ++sent_k;
              kr.step();
              if (j == u.lo) {
                ok = tc_wait(&sh.q_empty, (units & 1) ^ 1, &sh.dead);
                if (!ok) break;
                const int blocks = u.rows[1] > 0 ? 2 : 1;
                tc::bar_arrive_expect_tx(&sh.q_full, blocks * C::SLOT);
                for (int s = 0; s < blocks; ++s) pt_load<D>(qbuf + s * C::SLOT, &maps.q, u.head[s], u.t0 + u.row0[s], &sh.q_full);
                ++units;
              }
              if (j == u.top) sh.feed.ask();
              if (a.test_stall && j == u.lo + PT_STALL_AT) ok = tc_give_up(&sh.dead);
              ok = ok && tc_wait(&sh.v_empty[vr.at], vr.parity ^ 1, &sh.dead);
              if (!ok) break;
              tc::bar_arrive_expect_tx(&sh.v_full[vr.at], C::SLOT);
              pt_load<D>(vslots + vr.at * C::SLOT, &maps.v, u.kv_head, tok, &sh.v_full[vr.at]);
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
        if (id == 0) pf_check_offsets(a);  // once in a call: whichever CTA walks the unit
        ok = sh.feed.answered(&sh.dead, id);
        if (!ok) break;
        more = id >= 0;
      }
      if (ok) {
        ok = tc_wait(&sh.feed.empty[un.at], un.parity ^ 1, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0 && ok) {
          sh.unit[un.at].len = 0;
          tc::bar_arrive(&sh.feed.full[un.at]);
        }
      }
      if (!ok && lane == 0) {
        // let what is on its way arrive before the CTA ends: the last round of every slot
        flag_status(a.status, KDA_DEV_TIMEOUT);
        sh.feed.drain();
        if (units > 0) tc::bar_wait(&sh.q_full, (units - 1) & 1, 1u << 16);
        for (int i = max(0, sent_k - C::KR); i < sent_k; ++i) tc::bar_wait(&sh.k_full[i % C::KR], i / C::KR & 1, 1u << 16);
        for (int i = max(0, sent_v - C::VR); i < sent_v; ++i) tc::bar_wait(&sh.v_full[i % C::VR], i / C::VR & 1, 1u << 16);
      }
    } else if (warp == 8) {
      // ---- products: the warp waits and counts as one, one lane issues
      bool ok = true;
      TcRing<2> un;
      TcRing<C::KR> kr;
      TcRing<C::VR> vr;
      uint32_t p_parity[2] = {0, 0};
      const uint32_t tm = __reduce_max_sync(0xffffffffu, tmem);
      const uint64_t q0 = tc::sdesc(tc::smem_u32(qbuf)), k0 = tc::sdesc(tc::smem_u32(kslots));
      const uint64_t v0 = tc::sdesc_mn(tc::smem_u32(vslots), PT_HALF);
      constexpr uint32_t id_s = pt_idesc(PT_B), id_o = pt_idesc(D) | tc::IDESC_B_MN;
      auto scores = [&](int s) {
        const uint64_t qd = q0 + s * (C::SLOT / 16), kd = k0 + kr.at * (C::SLOT / 16);
        if (tc::elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // 16 channels per step
            const uint32_t at = (kk / 4 * PT_HALF + kk % 4 * 32) / 16;
            tc::mma_ss(tm + s * PT_B, qd + at, kd + at, id_s, kk > 0);
          }
          tc::commit(&sh.s_full[s]);
        }
      };
      for (uint32_t q_parity = 0;; q_parity ^= 1, un.step()) {
        ok = tc_wait_warp(&sh.feed.full[un.at], un.parity, &sh.dead);
        if (!ok) break;
        // numbers that are known to be the same for all lanes
        const int lo = __reduce_max_sync(0xffffffffu, sh.unit[un.at].lo), end = __reduce_max_sync(0xffffffffu, sh.unit[un.at].len);
        const int hi0 = __reduce_max_sync(0xffffffffu, sh.unit[un.at].hi[0]), hi1 = __reduce_max_sync(0xffffffffu, sh.unit[un.at].hi[1]);
        const int top = max(hi0, hi1);
        if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
        __syncwarp();
        if (end == 0) break;
        // the first tile's scores
        ok = tc_wait_warp(&sh.k_full[kr.at], kr.parity, &sh.dead) && tc_wait_warp(&sh.q_full, q_parity, &sh.dead);
        if (!ok) break;
        tc::fence_after_sync();
        scores(0);
        if (hi1 >= 0) scores(1);
        if (tc::elect_one()) {
          tc::commit(&sh.k_empty[kr.at]);
          if (lo == top) tc::commit(&sh.q_empty);
        }
        kr.step();
        for (int j = lo; j <= top; ++j) {
          ok = tc_wait_warp(&sh.v_ready[vr.at], vr.parity, &sh.dead);
          if (ok && j < top) ok = tc_wait_warp(&sh.k_full[kr.at], kr.parity, &sh.dead);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int hi = s ? hi1 : hi0;
            if (!ok || j > hi) continue;
            ok = tc_wait_warp(&sh.p_full[s], p_parity[s], &sh.dead);
            if (!ok) continue;
            p_parity[s] ^= 1;
            tc::fence_after_sync();
            const uint64_t vd = v0 + vr.at * (C::SLOT / 16);
            if (tc::elect_one()) {
#pragma unroll
              for (int kk = 0; kk < PT_B / 16; ++kk)  // 16 keys per step
                tc::mma_ts(tm + PT_O + s * 128, tm + s * PT_B + kk * 8, vd + kk * (2048 / 16), id_o, !(j == lo && kk == 0));
              if (j == hi) tc::commit(&sh.o_full[s]);
              if (s == 1 || j > hi1) tc::commit(&sh.v_empty[vr.at]);
            }
            // the next scores go where these probabilities lie: products run in the order of their issue
            if (j < hi) scores(s);
          }
          if (!ok) break;
          if (j < top) {
            if (tc::elect_one()) {
              tc::commit(&sh.k_empty[kr.at]);
              if (j + 1 == top) tc::commit(&sh.q_empty);
            }
            kr.step();
          }
          vr.step();
        }
        if (!ok) break;
      }
      // nothing of this warp's is on its way when the CTA ends
      if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
      __syncwarp();
      if (tc::elect_one()) tc::commit(&sh.drain);
      tc::bar_wait(&sh.drain, 0);
    } else {
      // ---- V tiles with keys that some row does not see
      TcRing<2> un;
      TcRing<C::VR> vr;
      bool ok = true;
      for (;; un.step()) {
        ok = tc_wait(&sh.feed.full[un.at], un.parity, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const PtUnit u = sh.unit[un.at];
        if (u.len == 0) break;
        for (int j = u.lo; j <= u.top; ++j, vr.step()) {
          ok = tc_wait(&sh.v_full[vr.at], vr.parity, &sh.dead);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (pt_masked(u, j, window)) {
            if (pt_clean<D>(vslots + vr.at * C::SLOT, u.len - j * PT_B, tid - 320)) *const_cast<volatile int*>(&sh.odd_v[un.at]) = 1;
            __threadfence_block();
          }
          __syncwarp();
          if (lane == 0) tc::bar_arrive(&sh.v_ready[vr.at]);
        }
        if (!ok) break;
        if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);
      }
      if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax: thread = row
    const int s = warp >> 2;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, own_s = tmem + s * PT_B + lanes, own_o = tmem + PT_O + s * 128 + lanes;
    const float cap2 = a.softcap * PA_LOG2E;
    // of a product, to powers of two (or the cap's argument); not 0, which would turn an unseen key's -infinity into a NaN
    float factor = pt_factor(a.scale, CAP ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E);
    const bool negative = !CAP && factor < 0.f;
    if (!CAP) factor = fmaxf(fabsf(factor), 1.2e-38f);
    const PtCap cap(factor, cap2);
    bool ok = true;
    uint32_t s_parity = 0, o_parity = 0;
    int rows_done = 0;
    for (TcRing<2> un;; un.step()) {
      ok = tc_wait(&sh.feed.full[un.at], un.parity, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const PtUnit u = sh.unit[un.at];
      if (u.len == 0) break;
      const int row0 = u.row0[s], row = row0 + (tid & 127), hi = u.hi[s];
      float m = PF_NONE, l = 0.f;
      for (int j = u.lo; j <= hi; ++j) {
        ok = tc_wait(&sh.s_full[s], s_parity, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        s_parity ^= 1;
        tc::fence_after_sync();
        // of the tile the row sees keys from .. to - 1
        const int k0 = j * PT_B;
        const bool masked = k0 + PT_B - 1 > row0 || k0 <= row0 + PT_B - 1 - window;
        const int to = row + 1 - k0, from = row - k0 < window ? 0 : row - k0 - window + 1;
        // the largest score in powers of two
        float top;
        float2 x[CAP ? 1 : PT_B / 2];
        int all_near = 0;  // halves of the keys for the short polynomial alone
        if constexpr (CAP) {
          top = pt_capped_top(own_s, masked, from, to, cap, all_near);
        } else {
          if (masked) pt_mask(own_s, from, to, negative ? INFINITY : -INFINITY);
          tc::tmem_ld128(own_s, reinterpret_cast<float*>(x));
          if (negative) {
#pragma unroll
            for (int i = 0; i < PT_B / 2; ++i) x[i] = make_float2(-x[i].x, -x[i].y);
          }
          float t[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) t[i] = fmaxf(x[i].x, x[i].y);
#pragma unroll
          for (int i = 4; i < PT_B / 2; ++i) t[i & 3] = fmaxf(fmaxf(t[i & 3], x[i].x), x[i].y);
          top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) * factor;
        }
        const bool move = top > m + PT_SLACK;
        if (__any_sync(0xffffffffu, move)) {
          const float mn = move ? top : m, by = ex2(m - mn);
          m = mn;
          l *= by;
          if (j > u.lo) {
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float o[16];
              uint32_t w[16];
              tc::tmem_ld16(own_o + c, o);
#pragma unroll
              for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * by);
              tc::tmem_st16(own_o + c, w);
            }
          }
        }
        float2 sum0 = make_float2(l, 0.f), sum1 = both(0.f);
        // N probabilities, to the columns of the scores that `at` counts in keys
        auto probabilities = [&](auto n, int at, const float2* x, auto argument) {
          constexpr int N = decltype(n)::value;
          uint32_t w[N / 2];
#pragma unroll
          for (int i = 0; i < N / 2; i += 2) {
            float2 e0 = argument(x[i]), e1 = argument(x[i + 1]);
            e0 = make_float2(ex2(e0.x), ex2(e0.y)), e1 = make_float2(ex2(e1.x), ex2(e1.y));
            sum0 = add2(sum0, e0), sum1 = add2(sum1, e1);
            w[i] = pack_bf16(e0.x, e0.y), w[i + 1] = pack_bf16(e1.x, e1.y);
          }
          if constexpr (N == 32) tc::tmem_st16(own_s + at / 2, w);
          else tc::tmem_st8f(own_s + at / 2, reinterpret_cast<const float*>(w));
        };
        if constexpr (CAP) {
          // by halves, over scores that have been read (a shorter body than the whole row's: instructions are fetched for each tile)
#pragma unroll 1
          for (int half = 0; half < 2; ++half) {
            if (all_near >> half & 1) {
              float2 y[32];
              tc::tmem_ld64(own_s + 64 * half, reinterpret_cast<float*>(y));
#pragma unroll
              for (int c = 0; c < 2; ++c)
                probabilities(Count<32>(), 64 * half + 32 * c, y + 16 * c, [&](float2 s) { return fma2(s, cap.nearer(s), both(-m)); });
              continue;
            }
#pragma unroll 1
            for (int c = 64 * half; c < 64 * half + 64; c += 16) {
              float2 x[8], y[8];
              tc::tmem_ld16(own_s + c, reinterpret_cast<float*>(x));
              cap.less(x, m, y);
              const uint32_t seen = masked ? pt_seen(c, from, to) : 0xffffffffu;
#pragma unroll
              for (int i = 0; i < 8; ++i)
                y[i] = make_float2(seen >> (2 * i) & 1 ? y[i].x : -INFINITY, seen >> (2 * i + 1) & 1 ? y[i].y : -INFINITY);
              probabilities(Count<16>(), c, y, [](float2 s) { return s; });
            }
          }
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) probabilities(Count<32>(), 32 * c, x + 16 * c, [&](float2 s) { return fma2(s, both(factor), both(-m)); });
        }
        sum0 = add2(sum0, sum1);
        l = sum0.x + sum0.y;
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.p_full[s]);
      }
      if (!ok) break;

      // ---- the rows' results
      if (u.rows[s] > 0) {
        ok = tc_wait(&sh.o_full[s], o_parity, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        o_parity ^= 1;
        tc::fence_after_sync();
        const bool mine = row - row0 < u.rows[s], odd = *const_cast<volatile int*>(&sh.odd_v[un.at]) != 0;
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.feed.empty[un.at]);  // before the stores, which an arrival behind them would wait for
        float by;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(by) : "f"(l));  // to 2^-23
        const int warp_row = (warp & 3) * 32;
        const int64_t at = (int64_t)(u.t0 + row0 + warp_row) * a.out_stride + (int64_t)u.head[s] * a.d;
#pragma unroll 1
        for (int c = 0; c < a.d; c += 32) {
          float o[32];
          tc::tmem_ld32(own_o + c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= by;
          if (odd && mine) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c + i < a.d) o[i] += pt_odd(a, u, row, hi, window, c + i);
          }
          __syncwarp();
          pt_store32(a.out, a.out_bf16, at + c, a.out_stride, u.rows[s] - warp_row, a.d - c, o);
        }
        if (mine && a.lse) a.lse[(int64_t)(u.t0 + row) * a.Hq + u.head[s]] = (m + log2f(l)) * PA_LN2;
        rows_done += u.rows[s];
      } else if (lane == 0) {
        tc::bar_arrive(&sh.feed.empty[un.at]);
      }
      __syncwarp();
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    if ((tid & 127) == 0) add_work(a.status, rows_done);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 8) tc::tmem_dealloc(tmem, PT_TMEM);
}

template <int D, bool CAP, bool BY_HEADS>
cudaError_t tc_launch(const PromptAttnArgs& a, cudaStream_t s) {
  auto kernel = prefill_attention_tc_kernel<D, CAP, BY_HEADS>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pt_smem<D>());
  if (e != cudaSuccess) return e;
  PtMaps maps;
  if (!encode_rows_map_sw128(&maps.q, a.q, a.T, a.Hq, a.d, a.q_stride, PT_B) ||
      !encode_rows_map_sw128(&maps.k, a.k, a.T, a.Hkv, a.d, a.k_stride, PT_B) ||
      !encode_rows_map_sw128(&maps.v, a.v, a.T, a.Hkv, a.d, a.v_stride, PT_B))
    return cudaErrorInvalidValue;
  const int pairs = BY_HEADS ? a.Hq / 2 : a.Hq;
  const int64_t places = pf_places(a.T, a.N, BY_HEADS ? PT_B : 2 * PT_B);
  if (places * pairs > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3((unsigned)(places * pairs)), dim3(PT_NT), pt_smem<D>(), s, maps, a, places, pairs);
}

template <int D>
cudaError_t tc_launch(const PromptAttnArgs& a, cudaStream_t s) {
  if (a.Hq / a.Hkv % 2 == 0) return a.softcap > 0.f ? tc_launch<D, true, true>(a, s) : tc_launch<D, false, true>(a, s);
  return a.softcap > 0.f ? tc_launch<D, true, false>(a, s) : tc_launch<D, false, false>(a, s);
}

}  // namespace

cudaError_t pf_tc(const PromptAttnArgs& a, cudaStream_t s) { return a.d == 128 ? tc_launch<128>(a, s) : tc_launch<64>(a, s); }

}  // namespace kda
