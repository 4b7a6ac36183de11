// Attention over packed prompts on the 5th-generation tensor cores: bf16 inputs, any head size.
//
// A CTA has two blocks of 128 query rows that share their keys: the same tokens of two heads of a group where the group has an
// even number, else two neighbouring blocks of one head.  Per 128 keys and block, S = Q K^T (rows x keys) in tensor memory; a
// thread has one row of it, so its maximum and sum need no exchange; P = exp2(S - reference) goes back as bf16 over the
// scores it came from, as the row operand of O += P V.  While one block's softmax runs, the other's products do.
//   warps 0 to 3, 4 to 7   softmax of block 0, 1
//   warp 8     issues the products (one thread)
//   warp 9     brings Q, and K and V tiles into rings, by TMA (128-byte swizzle; channels beyond d as zeros)
//   warps 10, 11   look at the V tiles with unseen keys: rows behind the sequence become zeros, values that are no numbers
//              too (0 * NaN would reach rows that do not see them); rows that do see one get it at the end
//
// The softmax's reference moves only when a score is 2^8 above it, so accumulators are hardly ever rescaled; the thread of the row does
// it, after the products that the scores' barrier already covers.  Probabilities are rounded to bf16 (2^-8) for the second
// product, half a step like the output's own rounding; their sum is taken before that, in fp32.
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

struct PtShared {
  // every barrier is waited on only by roles that see each of its rounds
  uint64_t k_full[4], k_empty[4], v_full[4], v_ready[4], v_empty[4];
  uint64_t q_full, s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int dead, odd_v;
};
template <int D>
constexpr int pt_smem() {
  using C = PtCfg<D>;
  return 1024 + (2 + C::KR + C::VR) * C::SLOT + (int)sizeof(PtShared);
}
static_assert(pt_smem<128>() <= 227 * 1024, "shared memory of one SM");

// The two blocks of a CTA, and the key tiles that they walk.
struct PtUnit {
  int t0, len;
  int row0[2], head[2], rows[2];  // rows = 0: no such block
  int lo, hi[2], top;             // tiles lo .. hi[s]; top: the larger hi
  int kv_head;
};

__device__ __forceinline__ PtUnit pt_unit(const PromptAttnArgs& a, int64_t places, int pairs, bool by_heads, int window) {
  const int64_t place = places - 1 - blockIdx.x / pairs;  // the longest rows first
  const int pair = blockIdx.x % pairs;
  const PfBlock b = pf_block(a, place, by_heads ? PT_B : 2 * PT_B);
  PtUnit u;
  u.t0 = b.t0, u.len = b.len;
  u.top = -1;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    u.head[s] = by_heads ? 2 * pair + s : pair;
    u.row0[s] = by_heads ? b.row0 : b.row0 + s * PT_B;
    u.rows[s] = max(0, min(PT_B, b.len - u.row0[s]));
    u.hi[s] = u.rows[s] > 0 ? (u.row0[s] + u.rows[s] - 1) / PT_B : -1;
    u.top = max(u.top, u.hi[s]);
  }
  u.lo = max(0, u.row0[0] - window + 1) / PT_B;
  u.kv_head = u.head[0] / (a.Hq / a.Hkv);
  return u;
}
// Whether some row of the CTA does not see some key of the tile.
__device__ __forceinline__ bool pt_masked(const PtUnit& u, int tile, int window) {
  const int k0 = tile * PT_B, last = u.rows[1] > 0 ? u.row0[1] + u.rows[1] - 1 : u.row0[0] + u.rows[0] - 1;
  return k0 + PT_B - 1 > u.row0[0] || k0 <= last - window;
}

__device__ __forceinline__ bool odd_bf16(uint32_t two) {  // a NaN or an infinity among the two
  return (two & 0x7f80u) == 0x7f80u || (two & 0x7f800000u) == 0x7f800000u;
}

template <int D, bool CAP>
__global__ void __launch_bounds__(PT_NT, 1)
    prefill_attention_tc_kernel(const __grid_constant__ PtMaps maps, const PromptAttnArgs a, const int64_t places, const int pairs,
                                const bool by_heads) {
  using C = PtCfg<D>;
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* qbuf = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* kslots = qbuf + 2 * C::SLOT;
  unsigned char* vslots = kslots + C::KR * C::SLOT;
  PtShared& sh = *reinterpret_cast<PtShared*>(vslots + C::VR * C::SLOT);
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int window = a.window > 0 ? a.window : 0x7fffffff;
  if (blockIdx.x == 0 && warp == 0) pf_check_offsets(a);
  const PtUnit u = pt_unit(a, places, pairs, by_heads, window);
  if (u.len == 0) return;

  if (tid == 0) {
    for (int i = 0; i < C::KR; ++i) tc::bar_init(&sh.k_full[i], 1), tc::bar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < C::VR; ++i)
      tc::bar_init(&sh.v_full[i], 1), tc::bar_init(&sh.v_ready[i], 2), tc::bar_init(&sh.v_empty[i], 1);
    for (int i = 0; i < 2; ++i)
      tc::bar_init(&sh.s_full[i], 1), tc::bar_init(&sh.p_full[i], 4), tc::bar_init(&sh.o_full[i], 1);
    tc::bar_init(&sh.q_full, 1), tc::bar_init(&sh.drain, 1);
    tc::bar_fence_init();
    sh.dead = sh.odd_v = 0;
  }
  if (warp == 8) tc::tmem_alloc(&sh.tmem, PT_TMEM);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sh.tmem;

  if (warp >= 8) {
    // 384 threads with 168 registers each were launched: 256 x 200 + 128 x 104 is as many
    asm volatile("setmaxnreg.dec.sync.aligned.u32 104;");
    if (warp == 9) {
      // ---- loads
      if (lane == 0) {
        bool ok = true;
        int sent_k = 0, sent_v = 0;
        const int blocks = u.rows[1] > 0 ? 2 : 1;
        tc::bar_arrive_expect_tx(&sh.q_full, blocks * C::SLOT);
        for (int s = 0; s < blocks; ++s)
          pt_load<D>(qbuf + s * C::SLOT, &maps.q, u.head[s], u.t0 + u.row0[s], &sh.q_full);
        TcRing<C::KR> kr;
        TcRing<C::VR> vr;
        for (int j = u.lo; j <= u.top; ++j) {
          const int tok = u.t0 + j * PT_B;
          ok = tc_wait(&sh.k_empty[kr.at], kr.parity ^ 1, &sh.dead);
          if (!ok) break;
          tc::bar_arrive_expect_tx(&sh.k_full[kr.at], C::SLOT);
          pt_load<D>(kslots + kr.at * C::SLOT, &maps.k, u.kv_head, tok, &sh.k_full[kr.at]);
          ++sent_k;
          kr.step();
          if (a.test_stall && j == u.lo + PT_STALL_AT) ok = tc_give_up(&sh.dead);
          ok = ok && tc_wait(&sh.v_empty[vr.at], vr.parity ^ 1, &sh.dead);
          if (!ok) break;
          tc::bar_arrive_expect_tx(&sh.v_full[vr.at], C::SLOT);
          pt_load<D>(vslots + vr.at * C::SLOT, &maps.v, u.kv_head, tok, &sh.v_full[vr.at]);
          ++sent_v;
          vr.step();
        }
        if (!ok) {
          // let what is on its way arrive before the CTA ends: the last round of every slot
          flag_status(a.status, KDA_DEV_TIMEOUT);
          tc::bar_wait(&sh.q_full, 0, 1u << 16);
          for (int i = max(0, sent_k - C::KR); i < sent_k; ++i) tc::bar_wait(&sh.k_full[i % C::KR], i / C::KR & 1, 1u << 16);
          for (int i = max(0, sent_v - C::VR); i < sent_v; ++i) tc::bar_wait(&sh.v_full[i % C::VR], i / C::VR & 1, 1u << 16);
        }
      }
    } else if (warp == 8) {
      // ---- products
      if (lane == 0) {
        bool ok = tc_wait(&sh.q_full, 0, &sh.dead);
        TcRing<C::KR> kr;
        TcRing<C::VR> vr;
        const uint64_t q0 = tc::sdesc(tc::smem_u32(qbuf)), k0 = tc::sdesc(tc::smem_u32(kslots));
        const uint64_t v0 = tc::sdesc_mn(tc::smem_u32(vslots), PT_HALF);
        constexpr uint32_t id_s = pt_idesc(PT_B), id_o = pt_idesc(D) | tc::IDESC_B_MN;
        auto scores = [&](int s) {
          const uint64_t qd = q0 + s * (C::SLOT / 16), kd = k0 + kr.at * (C::SLOT / 16);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {  // 16 channels per step
            const uint32_t at = (kk / 4 * PT_HALF + kk % 4 * 32) / 16;
            tc::mma_ss(tmem + s * PT_B, qd + at, kd + at, id_s, kk > 0);
          }
          tc::commit(&sh.s_full[s]);
        };
        // the first tile's scores
        ok = ok && tc_wait(&sh.k_full[0], 0, &sh.dead);
        if (ok) {
          tc::fence_after_sync();
          for (int s = 0; s < 2; ++s)
            if (u.lo <= u.hi[s]) scores(s);
          tc::commit(&sh.k_empty[0]);
          kr.step();
        }
        for (int j = u.lo; ok && j <= u.top; ++j) {
          const uint32_t parity = (j - u.lo) & 1;
          ok = tc_wait(&sh.v_ready[vr.at], vr.parity, &sh.dead);
          if (ok && j < u.top) ok = tc_wait(&sh.k_full[kr.at], kr.parity, &sh.dead);
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            if (!ok || j > u.hi[s]) continue;
            ok = tc_wait(&sh.p_full[s], parity, &sh.dead);
            if (!ok) continue;
            tc::fence_after_sync();
            const uint64_t vd = v0 + vr.at * (C::SLOT / 16);
#pragma unroll
            for (int kk = 0; kk < PT_B / 16; ++kk)  // 16 keys per step
              tc::mma_ts(tmem + PT_O + s * 128, tmem + s * PT_B + kk * 8, vd + kk * (2048 / 16), id_o, !(j == u.lo && kk == 0));
            if (j == u.hi[s]) tc::commit(&sh.o_full[s]);
            if (s == 1 || j > u.hi[1]) tc::commit(&sh.v_empty[vr.at]);
            // the next scores go where these probabilities lie: products run in the order of their issue
            if (j < u.hi[s]) scores(s);
          }
          if (!ok) break;
          if (j < u.top) {
            tc::commit(&sh.k_empty[kr.at]);
            kr.step();
          }
          vr.step();
        }
        // nothing of this thread's is on its way when the CTA ends
        if (!ok) flag_status(a.status, KDA_DEV_TIMEOUT);
        tc::commit(&sh.drain);
        tc::bar_wait(&sh.drain, 0);
      }
    } else {
      // ---- V tiles with keys that some row does not see
      TcRing<C::VR> vr;
      bool ok = true;
      for (int j = u.lo; j <= u.top; ++j, vr.step()) {
        ok = tc_wait(&sh.v_full[vr.at], vr.parity, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (pt_masked(u, j, window)) {
          unsigned char* tile = vslots + vr.at * C::SLOT;
          const int keys = u.len - j * PT_B;  // of the sequence
          bool odd = false;
          for (int i = tid - 320; i < PT_B * 8 * C::HALVES; i += 64) {
            const int row = (i >> 3) & (PT_B - 1);  // 16 bytes of it: eight lie in 128 bytes, in some order
            uint4* at = reinterpret_cast<uint4*>(tile) + i;
            if (row >= keys) {
              *at = make_uint4(0, 0, 0, 0);
              continue;
            }
            const uint4 x = *at;
            if (odd_bf16(x.x) || odd_bf16(x.y) || odd_bf16(x.z) || odd_bf16(x.w)) {
              odd = true;
              uint16_t* e = reinterpret_cast<uint16_t*>(at);
              for (int n = 0; n < 8; ++n)
                if ((e[n] & 0x7f80) == 0x7f80) e[n] = 0;
            }
          }
          if (odd) *const_cast<volatile int*>(&sh.odd_v) = 1;
          __threadfence_block();
          tc::fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.v_ready[vr.at]);
      }
      if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    // ---- softmax: thread = row
    const int s = warp >> 2, row = u.row0[s] + (tid & 127);
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16, own_s = tmem + s * PT_B + lanes, own_o = tmem + PT_O + s * 128 + lanes;
    const float cap2 = a.softcap * PA_LOG2E;
    // of a product, to powers of two (or the cap's argument); not 0, which would turn an unseen key's -infinity into a NaN
    float factor = a.scale * (CAP ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E);
    if (!CAP && fabsf(factor) < 1.2e-38f) factor = 1.2e-38f;
    bool ok = true;
    float m = PF_NONE, l = 0.f;
    for (int j = u.lo; j <= u.hi[s]; ++j) {
      ok = ok && tc_wait(&sh.s_full[s], (j - u.lo) & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      tc::fence_after_sync();
      float2 x[PT_B / 2];
#pragma unroll
      for (int c = 0; c < PT_B; c += 64) tc::tmem_ld64(own_s + c, reinterpret_cast<float*>(x) + c);
      const int k0 = j * PT_B;
      if constexpr (CAP) pt_cap(x, factor, cap2);
      // of the tile the row sees keys from .. to - 1
      if (k0 + PT_B - 1 > u.row0[s] || k0 <= u.row0[s] + PT_B - 1 - window) {
        const int to = row + 1 - k0, from = row - k0 < window ? 0 : row - k0 - window + 1;
        const float none = !CAP && factor < 0.f ? INFINITY : -INFINITY;
#pragma unroll
        for (int i = 0; i < PT_B / 2; ++i) {
          if (2 * i >= to || 2 * i < from) x[i].x = none;
          if (2 * i + 1 >= to || 2 * i + 1 < from) x[i].y = none;
        }
      }
      // the largest score in powers of two
      float top;
      if (CAP || factor >= 0.f) {
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int i = 0; i < PT_B / 2; ++i) t0 = fmaxf(t0, x[i].x), t1 = fmaxf(t1, x[i].y);
        top = fmaxf(t0, t1);
      } else {
        float t0 = INFINITY, t1 = INFINITY;
#pragma unroll
        for (int i = 0; i < PT_B / 2; ++i) t0 = fminf(t0, x[i].x), t1 = fminf(t1, x[i].y);
        top = fminf(t0, t1);
      }
      if constexpr (!CAP) top = top == -INFINITY || top == INFINITY ? (factor >= 0.f ? top : -top) : top * factor;
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
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t w[16];
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float2 e0 = x[16 * c + i], e1 = x[16 * c + i + 1];
          if constexpr (CAP) {
            e0 = add2(e0, both(-m)), e1 = add2(e1, both(-m));
          } else {
            e0 = fma2(e0, both(factor), both(-m)), e1 = fma2(e1, both(factor), both(-m));
          }
          e0 = make_float2(ex2(e0.x), ex2(e0.y)), e1 = make_float2(ex2(e1.x), ex2(e1.y));
          sum0 = add2(sum0, e0), sum1 = add2(sum1, e1);
          w[i] = pack_bf16(e0.x, e0.y), w[i + 1] = pack_bf16(e1.x, e1.y);
        }
        tc::tmem_st16(own_s + 16 * c, w);
      }
      sum0 = add2(sum0, sum1);
      l = sum0.x + sum0.y;
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.p_full[s]);
    }

    // ---- the rows' results
    if (u.rows[s] > 0) {
      ok = ok && tc_wait(&sh.o_full[s], 0, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      tc::fence_after_sync();
      if (ok) {
        const bool mine = row - u.row0[s] < u.rows[s], odd = *const_cast<volatile int*>(&sh.odd_v) != 0;
        const int64_t t = u.t0 + row;
        const float by = 1.f / l;
        const bf16* v = static_cast<const bf16*>(a.v) + u.kv_head * a.d;
        // values that are no numbers were left out of the tiles with unseen keys
        auto add_odd = [&](int c, float (&o)[16]) {
          for (int j = u.lo; j <= u.hi[s]; ++j) {
            if (!pt_masked(u, j, window)) continue;
            for (int k = max(j * PT_B, row >= window ? row - window + 1 : 0); k <= min(j * PT_B + PT_B - 1, row); ++k)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float x = c + i < a.d ? to_f32(v[(int64_t)(u.t0 + k) * a.v_stride + c + i]) : 0.f;
                if (!(fabsf(x) <= 3.4e38f)) o[i] += x;
              }
          }
        };
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          float o[16];
          tc::tmem_ld16(own_o + c, o);
          if (mine && c < a.d) {
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] *= by;
            if (odd) add_odd(c, o);
            pt_store16(a.out, a.out_bf16, t * a.out_stride + (int64_t)u.head[s] * a.d + c, o);
          }
          __syncwarp();  // the next load is the whole warp's
        }
        if (mine && a.lse) a.lse[t * a.Hq + u.head[s]] = (m + log2f(l)) * PA_LN2;
      }
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    if ((tid & 127) == 0 && ok) add_work(a.status, u.rows[s]);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 8) tc::tmem_dealloc(tmem, PT_TMEM);
}

template <int D, bool CAP>
cudaError_t tc_launch(const PromptAttnArgs& a, cudaStream_t s) {
  auto kernel = prefill_attention_tc_kernel<D, CAP>;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pt_smem<D>());
  if (e != cudaSuccess) return e;
  PtMaps maps;
  if (!encode_rows_map_sw128(&maps.q, a.q, a.T, a.Hq, a.d, a.q_stride, PT_B) ||
      !encode_rows_map_sw128(&maps.k, a.k, a.T, a.Hkv, a.d, a.k_stride, PT_B) ||
      !encode_rows_map_sw128(&maps.v, a.v, a.T, a.Hkv, a.d, a.v_stride, PT_B))
    return cudaErrorInvalidValue;
  const bool by_heads = a.Hq / a.Hkv % 2 == 0;
  const int pairs = by_heads ? a.Hq / 2 : a.Hq;
  const int64_t places = pf_places(a.T, a.N, by_heads ? PT_B : 2 * PT_B);
  if (places * pairs > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_pdl(kernel, dim3((unsigned)(places * pairs)), dim3(PT_NT), pt_smem<D>(), s, maps, a, places, pairs, by_heads);
}

}  // namespace

cudaError_t pf_tc(const PromptAttnArgs& a, cudaStream_t s) {
  const bool cap = a.softcap > 0.f;
  if (a.d == 128) return cap ? tc_launch<128, true>(a, s) : tc_launch<128, false>(a, s);
  return cap ? tc_launch<64, true>(a, s) : tc_launch<64, false>(a, s);
}

}  // namespace kda
