// Attention over a bf16 paged cache on the 5th-generation tensor cores: d = 128, bf16 queries and outputs.
//
// The mathematics, the line of tiles, the parts and their join are those of paged_attention.cuh; what differs is that
// cached rows never pass through registers.  One CTA per SM walks its share of the line in tiles of 128 tokens:
//   warp 0   copies the tile's K and V from their pages into rings of shared-memory slots (TMA, 128-byte swizzle, one box
//            of consecutive page rows per copy), running ahead of the others by the depth of the rings;
//   warps 1 and 3   issue S^T = K Q^T (128 tokens x the unit's query rows) and O^T += V^T P^T (128 channels x rows): K
//            is the row operand as it lies, V the same read along its channels;
//   warp 2   puts the next unit's queries into operand order;
//   warps 4 on   hold one token per thread: scores from tensor memory, their cap, mask and softmax, and the probabilities,
//            each as the sum of two bf16, to shared memory as the second product's column operand.
//
// Bound by HBM for few query rows: a tile's copies (64 KB) take 2800 cycles of the SM's share of it.  Every role is one
// warp or four, each passing through its code once per tile, so a role's time per tile is its instructions' latency (5
// to 10 cycles each): that is what was shortened (look-ups without divisions, roles on warps of their own).  With an 8-bit
// cache (1400 cycles a tile) the same roles were slower than the register form of paged_attention.cuh, multiplied as
// e4m3 with the 16-bit side in parts (125 us at 262144 tokens, where that form takes 109): that cache keeps it.
//
// One request with 32 heads over 8: of 262144 tokens 161 to 164 us (6.6 TB/s, 97 % of the copy rate), of 1000 tokens 10.7 us, a chain
// of launches, share-out, first copies and the join.
//
// Waits are bounded: one that gives up sets KDA_DEV_TIMEOUT and a flag on which every role leaves.
#include <stddef.h>

#include "device.h"
#include "paged_attention_tc.cuh"

namespace kda {

namespace {

constexpr int TC_SOFT0 = 128;          // first thread of the softmax warps

template <int RB>
struct TcCfg {
  static constexpr int PP = 2;                            // parts of a probability
  static constexpr int N1 = RB < 16 ? 16 : RB;            // columns of the products (multiples of 16)
  static constexpr int N2 = (PP * RB + 15) / 16 * 16;
  // softmax groups of four warps, each with RG of a tile's rows: several cover one another's latencies
  static constexpr int RG = RB < 8 ? RB : 8, RS = RB / RG;
  static constexpr int NT = TC_SOFT0 + RS * 128;
  static constexpr int S_COLS = (N1 + 31) / 32 * 32;      // tensor-memory columns of a score buffer
  static constexpr int SB = 2;                            // score and probability buffers
  static constexpr int O_COL = SB * S_COLS, TMEM_COLS = 128;
  static constexpr int SLOT = TC_TILE * TC_D * 2;        // bytes of a K or V tile
  static constexpr int Q_BYTES = N1 * TC_D * 2, P_BYTES = N2 * TC_TILE * 2;
  static constexpr int FIXED = 1024 + SB * P_BYTES + 2 * Q_BYTES + 2560 + 8 * NT;
  static constexpr int INFO = 8;  // tiles whose lists of boxes are kept: more than VS (see the copies)
  static constexpr int SLOTS_FIT = (227 * 1024 - FIXED) / SLOT;
  static constexpr int SLOTS = SLOTS_FIT > 10 ? 10 : SLOTS_FIT;
  static constexpr int KS = SLOTS / 2, VS = SLOTS - KS;  // slots of the two rings
};

template <int RB>
struct TcShared {
  using C = TcCfg<RB>;
  // Every barrier is waited on only by roles that see each of its rounds: a parity tells rounds apart no further.
  uint64_t k_full[C::KS], k_empty[C::KS], v_full[C::VS], v_empty[C::VS];
  uint64_t s_full[C::SB], s_free[C::SB], p_full[C::SB], p_free[C::SB], q_full[2], q_free[2], o_full, drain[2];
  int there[C::INFO];                                      // by tile: the boxes that were copied
  alignas(16) float factor[2][RB];  // per query row: score in powers of two per unit of the product
  int last[2][RB];                  // last seen position
  int head[2][RB];                  // place among the request's W x Hq output rows, -1 past the unit's rows
  float red[4][RB];
  int64_t sums[C::NT / 32];
  int64_t where[2];
  uint32_t tmem;
  int dead;
};

__device__ __forceinline__ void st_shared_u16(uint32_t at, uint32_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)v) : "memory");
}

// A thread's raw scores of a group's RG rows; `at`: their first column.
template <int RG>
__device__ __forceinline__ void load_scores(uint32_t at, float (&x)[RG]) {
  static_assert(RG <= 8, "one load");
  float s[8];
  tc::tmem_ld8(at, s);
#pragma unroll
  for (int i = 0; i < RG; ++i) x[i] = s[i];
}

template <int RB>
__global__ void __launch_bounds__(TcCfg<RB>::NT, 1)
    paged_attention_tc_kernel(const __grid_constant__ TcMaps maps, const PagedAttnArgs a, const PaPlan p, const int box) {
  using C = TcCfg<RB>;
  using Sh = TcShared<RB>;
  constexpr int N1 = C::N1, N2 = C::N2, SLOT = C::SLOT, KS = C::KS, VS = C::VS, PP = C::PP;
  constexpr int RS = C::RS, RG = C::RG, SB = C::SB, TC_NT = C::NT;
  static_assert(SB * C::S_COLS + N2 <= C::TMEM_COLS, "tensor memory asked for");
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* base = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* slots = base;
  unsigned char* vslots = slots + KS * SLOT;
  unsigned char* pbuf = vslots + VS * SLOT;
  unsigned char* qbuf = pbuf + SB * C::P_BYTES;
  Sh& sh = *reinterpret_cast<Sh*>(qbuf + 2 * C::Q_BYTES);
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hkv = a.c.Hkv, per_b = Hkv * p.blocks;

  if (tid == 0) {
    for (int i = 0; i < KS; ++i) tc::bar_init(&sh.k_full[i], 1), tc::bar_init(&sh.k_empty[i], 1);
    for (int i = 0; i < VS; ++i) tc::bar_init(&sh.v_full[i], 1), tc::bar_init(&sh.v_empty[i], 1);
    for (int i = 0; i < SB; ++i) {
      tc::bar_init(&sh.s_full[i], 2), tc::bar_init(&sh.s_free[i], 4 * RS);
      tc::bar_init(&sh.p_full[i], 4 * RS), tc::bar_init(&sh.p_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) tc::bar_init(&sh.q_full[i], 1), tc::bar_init(&sh.q_free[i], 1 + 4 * RS);
    tc::bar_init(&sh.o_full, 1);
    for (int i = 0; i < 2; ++i) tc::bar_init(&sh.drain[i], 1);
    tc::bar_fence_init();
    sh.dead = 0;
  }
  if (warp == 1) tc::tmem_alloc(&sh.tmem, C::TMEM_COLS);

  // ---- this CTA's share of the line (see paged_attention.cuh)
  const int run = (a.B + TC_NT - 1) / TC_NT;
  int64_t mine = 0;
  for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b)
    mine += pa_span<TC_TILE>(a, b, blockIdx.x == 0, box).tiles + TC_UNIT_COST;
  int64_t total;
  const int64_t upto = block_scan<TC_NT>(mine, sh.sums, total);
  total *= per_b;
  const int64_t workers = total < gridDim.x ? total : (int64_t)gridDim.x;
  const int64_t me = blockIdx.x;
  TcWalk walk;
  walk.at = me < workers ? me * total / workers : 0;
  walk.end = me < workers ? (me + 1) * total / workers : 0;
  const int64_t before = upto - mine;
  if (me < workers && walk.at >= before * per_b && walk.at < upto * per_b) {
    int64_t f = before;
    for (int b = tid * run;; ++b) {
      const int t = pa_span<TC_TILE>(a, b, false, box).tiles + TC_UNIT_COST;
      if (walk.at < (f + t) * per_b) {
        sh.where[0] = b;
        sh.where[1] = f * per_b;
        break;
      }
      f += t;
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  walk.b = me < workers ? (int)sh.where[0] : 0;
  walk.first_of_b = me < workers ? sh.where[1] : 0;
  const uint32_t tmem = sh.tmem, tmem_o = tmem + C::O_COL;
  const int window = a.window > 0 ? a.window : 0x7fffffff;

  if (warp == 0) {
    // ---- copies
    TcTiles it(walk);
    const int boxes = TC_TILE / box;
    bool ok = true;
    TcRing<KS> kr;
    TcRing<VS> vr;
    TcRing<C::INFO> info;
    // This lane's box of the next tile: its page's id is asked for a tile ahead, its place among the pages follows from the
    // last tile's.
    const int per_tile = TC_TILE / a.c.page_size, rest = TC_TILE - per_tile * a.c.page_size;
    int tile_no = 0;
    bool more = it.next(a, p, box), next_there = false;
    int next_page = 0, pg = 0, off = 0;
    const int32_t* table = nullptr;
    auto look_up = [&]() {
      const int tok = it.u.start + it.tile * TC_TILE + lane * box;
      if (it.first()) {
        pg = tok / a.c.page_size;
        off = tok - pg * a.c.page_size;
        table = a.block_table + (int64_t)it.u.b * a.max_pages;
      } else {
        pg += per_tile;
        off += rest;
        if (off >= a.c.page_size) off -= a.c.page_size, ++pg;
      }
      next_there = lane < boxes && tok < it.u.len;
      if (next_there) next_page = __ldg(table + pg);
    };
    if (more) look_up();
    while (more) {
      bool there = next_there;
      const int page = next_page, at = off, h = it.u.h;
      more = it.next(a, p, box);
      if (more) look_up();
      int row = 0;
      if (there) {
        there = (unsigned)page < (unsigned)a.c.num_pages;
        if (there) row = (page * Hkv + h) * a.c.page_size + at;
        else flag_status(a.status, KDA_DEV_PAGE_OOB);
      }
      const unsigned mask = __ballot_sync(0xffffffffu, there);
      const int count = __popc(mask);
      const uint32_t bytes = count * box * TC_D * 2;
      // A slot's n-th use waits for the release of the one before (the first finds the round before the first over).
      // The tile's list of boxes goes by its number: it has been read when its V is released, which the copies of VS tiles
      // later wait for.
      // The warp goes on or leaves as one: no lane copies what another does not wait for.
      ok = ok && tc_wait(&sh.k_empty[kr.at], kr.parity ^ 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0 && ok) {
        sh.there[info.at] = (int)mask;
        tc::bar_arrive_expect_tx(&sh.k_full[kr.at], bytes);
      }
      __syncwarp();
      // lane i has channels 0 .. 63 or 64 .. 127 of box i / 2
      const int two_row = __shfl_sync(0xffffffffu, row, lane >> 1), odd = lane & 1;
      const bool two = lane < 2 * boxes && (mask >> (lane >> 1) & 1);
      const uint32_t piece = odd * (TC_TILE * 128) + (lane >> 1) * box * 128;
      if (two && ok) tc::tma_load_2d(slots + kr.at * SLOT + piece, &maps.k, odd * 64, two_row, &sh.k_full[kr.at]);
      const bool k_sent = ok;
      if (p.stall && tile_no++ == TC_STALL_AT) ok = tc_give_up(&sh.dead);
      ok = ok && tc_wait(&sh.v_empty[vr.at], vr.parity ^ 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (lane == 0 && ok) tc::bar_arrive_expect_tx(&sh.v_full[vr.at], bytes);
      __syncwarp();
      if (two && ok) tc::tma_load_2d(vslots + vr.at * SLOT + piece, &maps.v, odd * 64, two_row, &sh.v_full[vr.at]);
      if (!ok) {
        // let what is on its way arrive before the CTA ends: this round's copies and those of the rounds just before
        if (lane == 0) {
          flag_status(a.status, KDA_DEV_TIMEOUT);
          for (int i = 0; i < KS; ++i) {
            const bool this_round = i < kr.at || (i == kr.at && k_sent);
            tc::bar_wait(&sh.k_full[i], this_round ? kr.parity : kr.parity ^ 1, 1u << 16);
          }
          for (int i = 0; i < VS; ++i)
            tc::bar_wait(&sh.v_full[i], i < vr.at || (i == vr.at && ok) ? vr.parity : vr.parity ^ 1, 1u << 16);
        }
        __syncwarp();
        break;
      }
      kr.step();
      vr.step();
      info.step();
    }
  } else if (warp == 1 || warp == 3) {
    // ---- products, one thread each; the tiles of the CTA's whole share take the buffers in turn.  (One thread for both
    // took 1700 cycles a tile, most of it its own instructions' latency.)
    bool ok = true;
    TcTiles it(walk);
    TcRing<SB> buf;
    if (warp == 1) {
      if (lane == 0) {
        constexpr uint32_t id = tc::idesc_bf16(128, N1);
        const uint64_t k0 = tc::sdesc(tc::smem_u32(slots)), q0 = tc::sdesc(tc::smem_u32(qbuf));
        TcRing<KS> ring;
        while (it.next(a, p, box)) {
          if (it.first()) ok = ok && tc_wait(&sh.q_full[it.unit_no & 1], (it.unit_no >> 1) & 1, &sh.dead);
          ok = ok && tc_wait(&sh.s_free[buf.at], buf.parity ^ 1, &sh.dead);
          ok = ok && tc_wait(&sh.k_full[ring.at], ring.parity, &sh.dead);
          if (!ok) break;
          tc::bar_arrive(&sh.s_full[buf.at]);  // hands on what came with K: the list of boxes
          tc::fence_after_sync();
          const uint64_t kd = k0 + ring.at * (SLOT / 16), qd = q0 + (it.unit_no & 1) * (C::Q_BYTES / 16);
          const uint32_t d = tmem + buf.at * C::S_COLS;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {  // 32 bytes of each row per step
            const uint64_t da = kd + (kk / 4 * (TC_TILE * 128) + kk % 4 * 32) / 16;
            const uint64_t db = qd + (kk / 4 * (N1 * 128) + kk % 4 * 32) / 16;
            tc::mma_ss(d, da, db, id, kk > 0);
          }
          tc::commit(&sh.s_full[buf.at]);
          tc::commit(&sh.k_empty[ring.at]);
          if (it.last()) tc::commit(&sh.q_free[it.unit_no & 1]);
          ring.step();
          buf.step();
        }
      }
    } else {
      constexpr uint32_t id = tc::idesc_bf16(128, N2) | tc::IDESC_A_MN;
      const uint64_t v0 = tc::sdesc_mn(tc::smem_u32(vslots), TC_TILE * 128), p0 = tc::sdesc(tc::smem_u32(pbuf));
      TcRing<VS> ring;
      TcRing<C::INFO> info;
      const int all_boxes = (int)((1u << (TC_TILE / box)) - 1);
      while (it.next(a, p, box)) {
        ok = ok && tc_wait(&sh.v_full[ring.at], ring.parity, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int64_t left = (int64_t)it.u.len - it.u.start - (int64_t)it.tile * TC_TILE;  // tokens from the tile's first on
        const int mask = sh.there[info.at];
        if (left < TC_TILE || mask != all_boxes) {
          // what lies in the slot for tokens that are not there must not be a NaN
          for (int t = lane; t < TC_TILE; t += 32)
            if (t >= left || !(mask >> (t / box) & 1)) {
              unsigned char* vrow = vslots + ring.at * SLOT + t * 128;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                reinterpret_cast<uint4*>(vrow)[i] = make_uint4(0, 0, 0, 0);
                reinterpret_cast<uint4*>(vrow + TC_TILE * 128)[i] = make_uint4(0, 0, 0, 0);
              }
            }
          tc::fence_proxy_async();
          __syncwarp();
        }
        if (lane == 0) {
          ok = tc_wait(&sh.p_full[buf.at], buf.parity, &sh.dead);
          if (ok) {
            tc::fence_after_sync();
            const uint64_t vd = v0 + ring.at * (SLOT / 16), pd = p0 + buf.at * (C::P_BYTES / 16);
            const uint32_t d = tmem_o;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // 16 tokens per step
              const uint64_t da = vd + kk * 2048 / 16;
              const uint64_t db = pd + (kk / 4 * (N2 * 128) + kk % 4 * 32) / 16;
              const uint32_t add = !(it.first() && kk == 0);
              tc::mma_ss(d, da, db, id, add);
            }
            tc::commit(&sh.p_free[buf.at]);
            tc::commit(&sh.v_empty[ring.at]);
            if (it.last()) tc::commit(&sh.o_full);
          }
        }
        ring.step();
        buf.step();
        info.step();
      }
    }
    if (lane == 0) {  // nothing of this thread's is on its way when the CTA ends
      if (!ok) flag_status(a.status, KDA_DEV_TIMEOUT);
      uint64_t* drain = &sh.drain[warp >> 1];
      tc::commit(drain);
      tc::bar_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---- queries of each unit, a row of 128 channels at a time, four channels a lane
    TcWalk w = walk;
    TcUnit u;
    bool ok = true;
    for (int un = 0; ok && next_unit(a, p, box, w, u); ++un) {
      const int buf = un & 1, row0 = u.rb * RB;
      if (un >= 2) ok = tc_wait(&sh.q_free[buf], ((un >> 1) - 1) & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const uint32_t qb = tc::smem_u32(qbuf + buf * C::Q_BYTES);
      constexpr int QCH = RB < 8 ? RB : 8;
#pragma unroll 1
      for (int r0 = 0; r0 < RB; r0 += QCH) {
        uint2 raw[QCH];
#pragma unroll
        for (int i = 0; i < QCH; ++i) {
          const int row = row0 + r0 + i, wt = row / p.G, g = row - wt * p.G;
          const int64_t head = ((int64_t)u.b * a.W + wt) * a.Hq + (int64_t)u.h * p.G + g;
          raw[i] = row < p.rows
                       ? __ldg(reinterpret_cast<const uint2*>(static_cast<const bf16*>(a.q) + head * TC_D + 4 * lane))
                       : make_uint2(0, 0);
        }
#pragma unroll
        for (int i = 0; i < QCH; ++i) {
          const int r = r0 + i, row = row0 + r;
          // channels 4 lane ..: block of 64 channels, 16-byte chunk of 8
          const uint32_t at = qb + (lane >> 4) * (N1 * 128) + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8;
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(raw[i].x), "r"(raw[i].y) : "memory");
          if (lane == 0) {
            const int wt = row / p.G, g = row - wt * p.G;
            sh.factor[buf][r] = a.scale * (a.softcap > 0.f ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E);
            sh.last[buf][r] = row < p.rows ? u.len - a.W + wt : -1;
            sh.head[buf][r] = row < p.rows ? wt * a.Hq + u.h * p.G + g : -1;
          }
        }
      }
      tc::fence_proxy_async();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.q_full[buf]);
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  } else if (warp >= 4) {
    // ---- softmax: thread = token of the tile, then channel of the output.  A role that gives up a wait goes on through
    // its tiles without results (no later wait holds it), so that the barriers between groups are always met.
    const int tk = (tid - TC_SOFT0) & 127, quarter = warp & 3, rs = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    const float cap2 = a.softcap * PA_LOG2E;
    const int bar_id = 1 + rs, rfirst = rs * RG;  // this group's rows of the unit
    float m[RG], l[RG];
    TcTiles it(walk);
    TcRing<SB> buf, before(SB - 1);  // this tile's buffers, and those of the tile before
    before.parity = 1;
    TcRing<C::INFO> info;
    int row0 = 0, nrows = 0, all_to = 0;
    int64_t all_from = 0;
    bool bad = false;
    const int box_bit = tk / box;
    PaMeta meta{-1, 0};
    int rows_done = 0;
    // where this thread's element of an operand row lies in a probability buffer: (place ^ (row % 8) * 16) + row * 128
    const uint32_t place = (uint32_t)(tk >> 6) * (N2 * 128) + ((uint32_t)((tk & 63) >> 3) << 4) + (tk & 7) * 2;
    for (; it.next(a, p, box); buf.step(), before.step(), info.step()) {
      const TcUnit& u = it.u;
      const int qb = it.unit_no & 1;
      if (it.first()) {
        row0 = u.rb * RB;
        nrows = min(RB, p.rows - row0);
        // tokens that every row of the unit sees
        all_to = u.len - a.W + row0 / p.G;
        all_from = (int64_t)u.len - a.W + (row0 + nrows - 1) / p.G - window + 1;
        bad |= !tc_wait(&sh.q_full[qb], (it.unit_no >> 1) & 1, &sh.dead);
#pragma unroll
        for (int r = 0; r < RG; ++r) m[r] = TC_NONE, l[r] = 0.f;
      }
      bad |= !tc_wait(&sh.s_full[buf.at], buf.parity, &sh.dead);
      tc::fence_after_sync();
      const int64_t tok0 = (int64_t)u.start + (int64_t)it.tile * TC_TILE;
      const int tok = (int)tok0 + tk;
      const bool there = tok < u.len && (sh.there[info.at] >> box_bit & 1);
      const bool masked = !there || tok0 + TC_TILE - 1 > all_to || tok0 < all_from;
      float x[RG];
      load_scores<RG>(tmem + buf.at * C::S_COLS + lanes + rfirst, x);
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.s_free[buf.at]);
#pragma unroll
      for (int r = 0; r < RG; r += 4) {
        const float4 f = *reinterpret_cast<const float4*>(&sh.factor[qb][rfirst + r]);
        x[r] *= f.x, x[r + 1] *= f.y, x[r + 2] *= f.z, x[r + 3] *= f.w;
      }
      if (a.softcap > 0.f) {
        bool near = true;
#pragma unroll
        for (int r = 0; r < RG; ++r) near = near && fabsf(x[r]) <= PA_NEAR;
        if (__all_sync(0xffffffffu, near)) {
#pragma unroll
          for (int r = 0; r < RG; ++r) x[r] = capped_near(x[r], cap2);
        } else {
#pragma unroll
          for (int r = 0; r < RG; ++r) x[r] = capped(x[r], cap2);
        }
      }
      if (masked) {
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const int last = sh.last[qb][rfirst + r];
          x[r] = there && tok <= last && tok > (int64_t)last - window ? x[r] : -INFINITY;
        }
      }
      float over = -INFINITY;
#pragma unroll
      for (int r = 0; r < RG; ++r) over = fmaxf(over, x[r] - m[r]);
      if (tc::named_bar_or(bar_id, 128, over > pa_slack(false))) {
        // ---- references move: the rows' maxima over the 128 tokens, then sums and accumulators follow
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          float t = x[r];
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
          if (lane == 0) sh.red[quarter][rfirst + r] = t;
        }
        // the group's last product into its accumulators is through
        if (!it.first()) bad |= !tc_wait(&sh.p_free[before.at], before.parity, &sh.dead);
        tc::fence_after_sync();
        tc::named_bar(bar_id, 128);
        float by[RG];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
          const float(&red)[4][RB] = sh.red;
          const int q = rfirst + r;
          const float mn = fmaxf(fmaxf(fmaxf(red[0][q], red[1][q]), fmaxf(red[2][q], red[3][q])), m[r]);
          by[r] = ex2(m[r] - mn);
          m[r] = mn;
          l[r] *= by[r];
        }
        if (!it.first()) {
          if constexpr (RG < 8) {  // column c is row c % RB's; the group has all rows
#pragma unroll
            for (int c = 0; c < PP * RB; c += 8) {
              float v[8];
              tc::tmem_ld8(tmem_o + lanes + c, v);
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] *= by[(c + i) % RB];
              tc::tmem_st8f(tmem_o + lanes + c, v);
            }
          } else {
#pragma unroll
            for (int part = 0; part < PP; ++part)
#pragma unroll
              for (int c = 0; c < RG; c += 8) {
                float v[8];
                const uint32_t at = tmem_o + lanes + part * RB + rfirst + c;
                tc::tmem_ld8(at, v);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= by[c + i];
                tc::tmem_st8f(at, v);
              }
          }
          tc::tmem_wait_st();
        }
        tc::named_bar(bar_id, 128);  // red may be written again
      }

      // ---- probabilities and their parts
      bad |= !tc_wait(&sh.p_free[buf.at], buf.parity ^ 1, &sh.dead);
      const uint32_t pb = tc::smem_u32(pbuf + buf.at * C::P_BYTES) + place;
#pragma unroll
      for (int r = 0; r < RG; r += 2) {
        float p0 = ex2(x[r] - m[r]), p1 = ex2(x[r + 1] - m[r + 1]);
        l[r] += p0;
        l[r + 1] += p1;
#pragma unroll
        for (int part = 0; part < PP; ++part) {
          const int c0 = part * RB + r;  // the operand's row is this plus rfirst (a multiple of 8, or 0)
          const uint32_t c = split_pair<false>(p0, p1);
          st_shared_u16((pb ^ ((c0 & 7) << 4)) + (rfirst + c0) * 128, c & 0xffffu);
          st_shared_u16((pb ^ (((c0 + 1) & 7) << 4)) + (rfirst + c0 + 1) * 128, c >> 16);
        }
      }
      tc::fence_proxy_async();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.p_full[buf.at]);
      if (!it.last()) continue;

      // ---- end of the unit's part
      __syncwarp();
      const bool whole = u.t0 == 0 && u.t1 == u.tiles;
      const int64_t part_at = (me * 2 + (u.t0 == 0 ? 1 : 0)) * RB;
      bool nan = false;
      // writes row r (of the unit) of the result: accumulator y of channel tk, reference mr, sum lr
      auto put = [&](int r, float y, float mr, float lr) {
        const bool none = mr == TC_NONE && lr == 0.f;
        if (mr == TC_NONE) mr = none ? -INFINITY : 0.f;  // nothing but NaN scores: let them through
        if (none) y = 0.f;
        const int hd = sh.head[qb][r];
        if (hd < 0 || bad) return;
        nan |= isnan(y);
        if (whole) {
          const int64_t head = (int64_t)u.b * a.W * a.Hq + hd;
          static_cast<bf16*>(a.out)[head * TC_D + tk] = __float2bfloat16_rn(none ? 0.f : y / lr);
          if (tk == 0 && a.lse) a.lse[head] = none ? -INFINITY : log_sum(mr, lr);
        } else {
          p.part_o[(part_at + r) * TC_D + tk] = y;
          if (tk == 0) *reinterpret_cast<float2*>(p.part_ml + (part_at + r) * 2) = make_float2(mr, lr);
        }
      };
#pragma unroll
      for (int r = 0; r < RG; ++r) {
        float t = l[r];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) sh.red[quarter][rfirst + r] = t;
      }
      bad |= !tc_wait(&sh.o_full, it.unit_no & 1, &sh.dead);
      bad = __any_sync(0xffffffffu, bad);  // the careful way out is a warp's
      tc::fence_after_sync();
      tc::named_bar(bar_id, 128);
      float o[PP * RG];
      if constexpr (RG < 8) {
        tc::tmem_ld8(tmem_o + lanes, o);
      } else {
#pragma unroll
        for (int part = 0; part < PP; ++part) tc::tmem_ld8(tmem_o + lanes + part * RB + rfirst, o + part * RG);
      }
      tc::fence_before_sync();
#pragma unroll
      for (int i = 0; i < RG; ++i) {
        const int r = rfirst + i;
        put(r, o[i] + o[RG + i], m[i], sh.red[0][r] + sh.red[1][r] + sh.red[2][r] + sh.red[3][r]);
      }
      if (tc::named_bar_or(bar_id, 128, nan)) {  // also: red may be written again
        for (int i = quarter; i < RG; i += 4) {
          const int r = rfirst + i;
          if (r >= nrows || bad) continue;
          float4 o;
          float mr, lr;
          careful_row<false>(a, p, u, row0 + r, o, mr, lr);
          const bool none = mr == TC_NONE && lr == 0.f;
          if (mr == TC_NONE) mr = none ? -INFINITY : 0.f;
          if (whole) {
            const int64_t head = (int64_t)u.b * a.W * a.Hq + sh.head[qb][r];
            const float by = none ? 0.f : 1.f / lr;
            uint2 y;
            y.x = tc::pack2(__float2bfloat16_rn(o.x * by), __float2bfloat16_rn(o.y * by));
            y.y = tc::pack2(__float2bfloat16_rn(o.z * by), __float2bfloat16_rn(o.w * by));
            *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + head * TC_D + 4 * lane) = y;
            if (lane == 0 && a.lse) a.lse[head] = none ? -INFINITY : log_sum(mr, lr);
          } else {
            *reinterpret_cast<float4*>(p.part_o + (part_at + r) * TC_D + 4 * lane) = o;
            if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + (part_at + r) * 2) = make_float2(mr, lr);
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.q_free[qb]);  // the unit's row table has been read
      if (whole) {
        rows_done += nrows;
      } else if (u.t0 == 0) {
        // the unit goes on in the following shares: this one ends t1 tiles into it
        const int cost = u.tiles + TC_UNIT_COST;
        const int64_t unit_end = walk.end - (u.t1 + TC_UNIT_COST) + cost;
        meta.unit = (u.b * Hkv + u.h) * p.blocks + u.rb;
        int64_t e = (unit_end - 1) * workers / total;
        while (e * total / workers > unit_end - 1) --e;
        while ((e + 1) * total / workers <= unit_end - 1) ++e;
        meta.end = (int)e;
      }
    }
    if (bad && tk == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    if (tid == TC_SOFT0) {
      p.meta[me] = bad ? PaMeta{-1, 0} : meta;
      add_work(a.status, rows_done);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 1) tc::tmem_dealloc(tmem, C::TMEM_COLS);
}

template <int RB>
cudaError_t tc_launch(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  using C = TcCfg<RB>;
  auto kernel = paged_attention_tc_kernel<RB>;
  static_assert(C::INFO > C::VS, "lists of boxes kept until they are read");
  constexpr int bytes = 1024 + C::SLOTS * C::SLOT + C::SB * C::P_BYTES + 2 * C::Q_BYTES +
                        (int)sizeof(TcShared<RB>);
  static_assert(bytes <= 227 * 1024 && C::KS >= 2, "shared memory of one SM");
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  const int box = page_box(a.c.page_size);
  const long long rows = (long long)a.c.num_pages * a.c.Hkv * a.c.page_size;
  TcMaps maps;
  if (!encode_cache_map(&maps.k, a.c.k_pages, rows, box) || !encode_cache_map(&maps.v, a.c.v_pages, rows, box))
    return cudaErrorInvalidValue;
  int64_t ctas = sms < PA_SMS ? sms : PA_SMS;
  const int64_t tiles = (int64_t)a.max_pages * a.c.page_size / TC_TILE + 2 + TC_UNIT_COST;
  const int64_t units = (int64_t)a.B * a.c.Hkv * p.blocks;
  if (tiles < ctas && units * tiles < ctas) ctas = units * tiles;
  PaPlan plan = p;
  plan.workers = (int)ctas;
  e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(C::NT), bytes, s, maps, a, plan, box);
  if (e != cudaSuccess) return e;
  return pa_join<TC_D, RB>(a, plan, units, s);
}

}  // namespace

bool pa_tc_supported(const PagedAttnArgs& a) {
  return a.c.d == TC_D && !a.c.e4m3 && a.q_bf16 && a.out_bf16 && a.c.num_pages > 0 &&
         (int64_t)a.c.num_pages * a.c.Hkv * a.c.page_size <= 0x7fffffff;
}

int pa_tc_row_block(int rows) { return rows <= 4 ? 4 : rows <= 8 ? 8 : 16; }

cudaError_t pa_tc(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  switch (pa_tc_row_block(p.rows)) {
    case 4: return tc_launch<4>(a, p, sms, s);
    case 8: return tc_launch<8>(a, p, sms, s);
    default: return tc_launch<16>(a, p, sms, s);
  }
}

}  // namespace kda
