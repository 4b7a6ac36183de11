// Attention of many query rows per cached row (drafts times grouped heads) on the 5th-generation tensor cores: d = 128,
// bf16 queries and outputs, both caches.
//
// The mathematics, the line of tiles, the parts and their join are those of paged_attention.cuh.  A unit has up to 128 query
// rows, and the query is the product's row operand: S = Q K^T (rows x 128 tokens), O += P V (rows x 128 channels).  So a
// thread has one query row of the scores, its maximum and sum need no exchange, and P goes back to tensor memory, over the
// scores it came from, as the second product's row operand.  One CTA per SM:
//   warps 0 to 3    bring K and V tiles into rings of operand slots: a bf16 cache's pages by TMA (128-byte swizzle, one box
//              of consecutive page rows per copy; warp 0 alone), an e4m3 cache's through registers, a tile ahead, where
//              codes become fp16 (exact);
//   warps 4 to 11   softmax: two groups of four, each with 64 of a tile's tokens and an accumulator of its own, so that they
//              meet only at a unit's end; two score buffers, so that the next tile's product runs under a tile's softmax;
//   warps 12 and 13   issue the two products;
//   warps 14 and 15   put the next unit's queries into operand order.
//
// Bound by the softmax warps, and with an e4m3 cache by the loaders next to them (forty instructions more in their loop over
// the tiles cost 10 %, so what can be seen elsewhere is not looked at there).  A tile's 128 x 128 scores are 128 exponentials a lane and scheduler, 1024 cycles of their unit,
// and with cap and scales about 20 more operations each; measured, a tile takes 3500 cycles (bf16) to 6000 (e4m3 with
// cap), the products 1024 to 1536 under them.  Code that runs once is dear (a cold instruction costs about 4 cycles, and a
// share has some ten tiles), so tiles go in two equal passes over one compact body, and rare cases in small loops.
// 64 requests of 500 to 6000 tokens (window 4096), 8 drafts, 12 heads over 1, cap: 37.5 us (bf16) and 45.5 us (e4m3); with the
// queries as the products' column operand 88 and 100 us.
//
// Waits are bounded: one that gives up sets KDA_DEV_TIMEOUT and a flag on which every role leaves.
#include "device.h"
#include "f32x2.cuh"
#include "paged_attention_tc.cuh"

namespace kda {

namespace {

constexpr int RW_RB = PA_ROWS_BLOCK;
constexpr int RW_SOFT0 = 128, RW_SOFT = 256, RW_NT = RW_SOFT0 + RW_SOFT + 128;
constexpr int RW_RING = 2;                        // slots of K and of V
constexpr int RW_INFO = 4;                        // tiles whose scales and tokens are kept: twice the ring
constexpr int RW_SLOT = TC_TILE * TC_D * 2;       // bytes of a K, V or Q tile: two blocks of 64 channels
constexpr int RW_BLOCK = TC_TILE * 128;           // bytes of a block
constexpr int RW_O = 256, RW_TMEM = 512;          // columns: two score buffers, two accumulators

struct RwShared {
  // Every barrier is waited on only by roles that see each of its rounds: a parity tells rounds apart no further.
  uint64_t k_full[RW_RING], k_empty[RW_RING], v_full[RW_RING], v_ready[RW_RING], v_empty[RW_RING];
  uint64_t s_full[2], p_full[2], p_free[2], q_full[2], q_free[2], o_full, drain[2];
  TcUnit unit[2];  // what the query warps walk to; t1 = 0 ends the share
  // by tile: which tokens there are, and their scales; lift is about log2 of the value's
  alignas(16) uint32_t there[RW_INFO][4];
  alignas(16) float k_scale[RW_INFO][TC_TILE], v_scale[RW_INFO][TC_TILE], lift[RW_INFO][TC_TILE];
  float lift_top[RW_INFO][4];  // largest lift of 32 tokens
  uint32_t v_tile[4];  // e4m3: number of the last tile whose V rows a warp has put in their slot, from 1
  float2 ml[2][RW_RB];
  // per query row of a unit: score in powers of two per unit of the product, last seen position, and place among the
  // request's W x Hq output rows (-1 past the unit's)
  float factor[2][RW_RB];
  int last[2][RW_RB], head[2][RW_RB];
  uint32_t nan[2][4];
  int64_t sums[RW_NT / 32];
  int64_t where[2];
  uint32_t tmem;
  int dead;
};
constexpr int RW_SMEM = 1024 + (2 * RW_RING + 2) * RW_SLOT + (int)sizeof(RwShared);
static_assert(RW_SMEM <= 227 * 1024, "shared memory of one SM");

__host__ __device__ constexpr uint32_t rw_idesc(bool f8) {  // 128 x 128, fp16 or bf16 operands
  return (1u << 4) | (f8 ? 0u : (1u << 7) | (1u << 10)) | (16u << 17) | (8u << 24);
}

// 16 codes as 16 fp16, to two chunks of a row's block.
__device__ __forceinline__ void put_codes(uint32_t slot, int row, int c, const uint4& w) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w}, at = slot + (c >> 2) * RW_BLOCK;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + tc::sw128_chunk(row, (c & 3) * 2 + i)),
                 "r"(half2_of_codes(x[2 * i] & 0xffffu)), "r"(half2_of_codes(x[2 * i] >> 16)),
                 "r"(half2_of_codes(x[2 * i + 1] & 0xffffu)), "r"(half2_of_codes(x[2 * i + 1] >> 16))
                 : "memory");
}
__device__ __forceinline__ uint4 load_codes(const void* pages, int64_t row, int c) {
  uint4 w = make_uint4(0, 0, 0, 0);
  if (row >= 0)
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(static_cast<const uint8_t*>(pages) + row * TC_D + c * 16));
  return w;
}

// capped_near of paged_attention.cuh for two scores, its coefficients multiplied out to powers of z.  Seven multiplications and
// additions instead of two operations of the exponential's unit.
struct CapPoly {
  float k[6];
  __device__ __forceinline__ explicit CapPoly(float cap2) {
    constexpr float h = 0.5f * PA_LN2, h2 = h * h;
    float w = cap2 * h;
#pragma unroll
    for (int i = 0; i < 6; ++i) k[i] = pa_tanh(i) * w, w *= h2;
  }
  __device__ __forceinline__ float2 operator()(float2 z) const {
    const float2 u = mul2(z, z);
    float2 t = both(k[5]);
#pragma unroll
    for (int i = 4; i >= 0; --i) t = fma2(t, u, both(k[i]));
    return mul2(z, t);
  }
};
__device__ __forceinline__ uint32_t pack_f16(float2 x) {
  const __half2 h = __floats2half2_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float4 ld_shared4(uint32_t at) {
  float4 x;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w) : "r"(at) : "memory");
  return x;
}

// Waits until the V rows of tile `tile_no` are in their slot (they stay there until this warp's probabilities are used); false
// when that takes too long, or another role has given up.
__device__ __forceinline__ bool rw_put(const volatile uint32_t* v_tile, uint32_t tile_no, int* dead) {
  for (int i = 0; i < 1 << 22; ++i) {
    if ((int)(*v_tile - tile_no) >= 0) {
      __threadfence_block();
      return true;
    }
    if (*reinterpret_cast<volatile int*>(dead)) return false;
  }
  *reinterpret_cast<volatile int*>(dead) = 1;
  return false;
}
// Whether a row of a V slot, one a lane, holds anything but zeros (fp16).  Most rows show it in their first chunk.
__device__ __forceinline__ uint32_t rw_nonzero(uint32_t slot, int row) {
  uint32_t any = 0;
#pragma unroll 1
  for (int c = 0; c < 16; ++c) {
    uint32_t x, y, z, w;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x), "=r"(y), "=r"(z), "=r"(w)
                 : "r"(slot + (c >> 3) * RW_BLOCK + tc::sw128_chunk(row, c & 7))
                 : "memory");
    any |= (x | y | z | w) & 0x7fff7fffu;
    if (__all_sync(0xffffffffu, any != 0)) break;
  }
  return any;
}

// A pair of probabilities times a power of two.
template <bool F8>
__device__ __forceinline__ uint32_t times16(uint32_t two, float by) {
  if constexpr (F8) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
    const __half2 h = __floats2half2_rn(f.x * by, f.y * by);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(two << 16) * by, __uint_as_float(two & 0xffff0000u) * by);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool F8>
__global__ void __launch_bounds__(RW_NT, 1)
    paged_attention_rows_kernel(const __grid_constant__ TcMaps maps, const PagedAttnArgs a, const PaPlan p, const int box) {
  extern __shared__ __align__(1024) unsigned char smem_raw[];
  unsigned char* kslots = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  unsigned char* vslots = kslots + RW_RING * RW_SLOT;
  unsigned char* qbuf = vslots + RW_RING * RW_SLOT;
  RwShared& sh = *reinterpret_cast<RwShared*>(qbuf + 2 * RW_SLOT);
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int Hkv = a.c.Hkv, per_b = Hkv * p.blocks;

  if (tid == 0) {
    for (int i = 0; i < RW_RING; ++i) {
      tc::bar_init(&sh.k_full[i], F8 ? 4 : 1), tc::bar_init(&sh.k_empty[i], 1);
      tc::bar_init(&sh.v_full[i], F8 ? 4 : 1), tc::bar_init(&sh.v_ready[i], 3), tc::bar_init(&sh.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::bar_init(&sh.s_full[i], 2), tc::bar_init(&sh.p_full[i], 8), tc::bar_init(&sh.p_free[i], 1);
      tc::bar_init(&sh.drain[i], 1);
      tc::bar_init(&sh.q_full[i], 2), tc::bar_init(&sh.q_free[i], 8);
    }
    tc::bar_init(&sh.o_full, 1);
    tc::bar_fence_init();
    sh.dead = 0;
    for (int i = 0; i < 4; ++i) sh.v_tile[i] = 0;
  }
  if (warp == 12) tc::tmem_alloc(&sh.tmem, RW_TMEM);

  // ---- this CTA's share of the line (see paged_attention.cuh)
  const int run = (a.B + RW_NT - 1) / RW_NT;
  int64_t mine = 0;
  for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b)
    mine += pa_span<TC_TILE>(a, b, blockIdx.x == 0, box).tiles + TC_UNIT_COST;
  int64_t total;
  const int64_t upto = block_scan<RW_NT>(mine, sh.sums, total);
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
  const uint32_t tmem = sh.tmem;
  const int window = a.window > 0 ? a.window : 0x7fffffff;

  if (warp < 4) {
    TcTiles it(walk);
    TcRing<RW_RING> ring;
    TcRing<RW_INFO> info;
    bool ok = true;
    if constexpr (F8) {
      // ---- e4m3: a lane places one token of its warp's 32; a tile's rows go 4 at a time, lanes 4 i to 4 i + 3 with half of one:
      // so the 8 lanes of a shared-memory store have half of two neighbouring rows, whose chunks meet all banks
      const int c = (lane & 3) + (lane >> 3 & 1) * 4, r4 = (lane >> 4) * 2 + (lane >> 2 & 1), tok_own = warp * 32 + lane;
      // the page's id is asked for two tiles ahead, the tile's rows one ahead
      int page = 0, off = 0, head = 0;
      bool more = true, next_there = false;
      auto look_up = [&]() {
        next_there = false;
        more = it.next(a, p, box);
        if (!more) return;
        head = it.u.h;
        const int64_t tok = (int64_t)it.u.start + (int64_t)it.tile * TC_TILE + tok_own;
        next_there = tok < it.u.len;
        if (next_there) {
          const int pg = (int)tok / a.c.page_size;
          off = (int)tok - pg * a.c.page_size;
          page = __ldg(a.block_table + (int64_t)it.u.b * a.max_pages + pg);
        }
      };
      auto place = [&]() -> int64_t {
        if (!next_there) return -1;
        if ((unsigned)page >= (unsigned)a.c.num_pages) {
          flag_status(a.status, KDA_DEV_PAGE_OOB);
          return -1;
        }
        return ((int64_t)page * Hkv + head) * a.c.page_size + off;
      };
      uint4 kw[8], vw[8];
      float ks = 0.f, vs = 0.f;
      int64_t row = -1;
      uint32_t tile_no = 0;  // of the CTA's share, from 1
      auto load_k = [&]() {
        ks = row >= 0 ? __ldg(a.c.k_scales + row) : 0.f;
        vs = row >= 0 ? __ldg(a.c.v_scales + row) : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) kw[i] = load_codes(a.c.k_pages, __shfl_sync(0xffffffffu, row, i * 4 + r4), c);
      };
      auto load_v = [&]() {
#pragma unroll
        for (int i = 0; i < 8; ++i) vw[i] = load_codes(a.c.v_pages, __shfl_sync(0xffffffffu, row, i * 4 + r4), c);
      };
      look_up();
      bool have = more;  // the tile whose rows are on their way
      if (have) {
        row = place();
        look_up();
        load_k();
        load_v();
      }
      while (have) {
        const uint32_t there = __ballot_sync(0xffffffffu, row >= 0);
        ok = ok && tc_wait(&sh.k_empty[ring.at], ring.parity ^ 1, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        // this tile's place among the kept was read by everyone before the product that freed the slot was issued
        const int lift = (int)(__float_as_uint(vs) >> 23) - 126, lift_top = __reduce_max_sync(0xffffffffu, lift);
        if (lane == 0) sh.there[info.at][warp] = there, sh.lift_top[info.at][warp] = (float)lift_top;
        sh.k_scale[info.at][tok_own] = ks;
        sh.v_scale[info.at][tok_own] = vs;
        sh.lift[info.at][tok_own] = (float)lift;
        const uint32_t k_at = tc::smem_u32(kslots + ring.at * RW_SLOT), v_at = tc::smem_u32(vslots + ring.at * RW_SLOT);
#pragma unroll
        for (int i = 0; i < 8; ++i) put_codes(k_at, warp * 32 + i * 4 + r4, c, kw[i]);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.k_full[ring.at]);
        // the next tile's keys are asked for before this one's values are put in place, but for the first tile, whose softmax
        // waits for them to move its reference
        const bool first = tile_no == 0;
        auto next_k = [&]() {
          have = more;
          if (have) {
            row = place();
            look_up();
            load_k();
          }
        };
        if (!first) next_k();
        ok = ok && tc_wait(&sh.v_empty[ring.at], ring.parity ^ 1, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 8; ++i) put_codes(v_at, warp * 32 + i * 4 + r4, c, vw[i]);
        tc::fence_proxy_async();
        __syncwarp();
        ++tile_no;
        if (lane == 0) {
          tc::bar_arrive(&sh.v_full[ring.at]);
          __threadfence_block();
          *const_cast<volatile uint32_t*>(&sh.v_tile[warp]) = tile_no;
        }
        if (first) next_k();
        if (have) load_v();
        ring.step();
        info.step();
      }
      if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    } else if (warp == 0) {
      // ---- bf16: lane i places box i of the next tile; its page's id is asked for a tile ahead
      const int boxes = TC_TILE / box;
      int page = 0, off = 0, tile_no = 0;
      bool next_there = false;
      auto look_up = [&]() {
        const int64_t tok = (int64_t)it.u.start + (int64_t)it.tile * TC_TILE + lane * box;
        next_there = lane < boxes && tok < it.u.len;
        if (next_there) {
          const int pg = (int)tok / a.c.page_size;
          off = (int)tok - pg * a.c.page_size;
          page = __ldg(a.block_table + (int64_t)it.u.b * a.max_pages + pg);
        }
      };
      bool more = it.next(a, p, box);
      if (more) look_up();
      while (more) {
        bool there = next_there;
        int row = 0;
        if (there) {
          there = (unsigned)page < (unsigned)a.c.num_pages;
          if (there) row = (page * Hkv + it.u.h) * a.c.page_size + off;
          else flag_status(a.status, KDA_DEV_PAGE_OOB);
        }
        const int left = (int)min((int64_t)TC_TILE, (int64_t)it.u.len - it.u.start - (int64_t)it.tile * TC_TILE);
        more = it.next(a, p, box);
        if (more) look_up();
        const unsigned mask = __ballot_sync(0xffffffffu, there);
        const uint32_t bytes = __popc(mask) * box * TC_D * 2;
        // the warp goes on or leaves as one: no lane copies what another does not wait for
        ok = ok && tc_wait(&sh.k_empty[ring.at], ring.parity ^ 1, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (lane < 4 && ok) {  // 32 tokens of the tile each; a box has at least 16
          uint32_t w = 0;
          for (int s = 0; s < 2; ++s)
            if (mask >> ((lane * 32 + s * 16) / box) & 1) w |= 0xffffu << (16 * s);
          const int n = left - lane * 32;  // of the request's tokens
          if (n < 32) w &= n <= 0 ? 0u : (1u << n) - 1;
          sh.there[info.at][lane] = w;
        }
        __syncwarp();
        if (lane == 0 && ok) tc::bar_arrive_expect_tx(&sh.k_full[ring.at], bytes);
        __syncwarp();
        // lane i has channels 0 .. 63 or 64 .. 127 of box i / 2
        const int two_row = __shfl_sync(0xffffffffu, row, lane >> 1), odd = lane & 1;
        const bool two = lane < 2 * boxes && (mask >> (lane >> 1) & 1);
        const uint32_t piece = odd * RW_BLOCK + (lane >> 1) * box * 128;
        if (two && ok) tc::tma_load_2d(kslots + ring.at * RW_SLOT + piece, &maps.k, odd * 64, two_row, &sh.k_full[ring.at]);
        const bool k_sent = ok;
        if (p.stall && tile_no++ == TC_STALL_AT) ok = tc_give_up(&sh.dead);
        ok = ok && tc_wait(&sh.v_empty[ring.at], ring.parity ^ 1, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 0 && ok) tc::bar_arrive_expect_tx(&sh.v_full[ring.at], bytes);
        __syncwarp();
        if (two && ok) tc::tma_load_2d(vslots + ring.at * RW_SLOT + piece, &maps.v, odd * 64, two_row, &sh.v_full[ring.at]);
        if (!ok) {
          // let what is on its way arrive before the CTA ends: this round's copies and those of the rounds just before
          if (lane == 0) {
            flag_status(a.status, KDA_DEV_TIMEOUT);
            for (int i = 0; i < RW_RING; ++i) {
              const bool this_round = i < ring.at || (i == ring.at && k_sent);
              tc::bar_wait(&sh.k_full[i], this_round ? ring.parity : ring.parity ^ 1, 1u << 16);
              tc::bar_wait(&sh.v_full[i], i < ring.at || (i == ring.at && ok) ? ring.parity : ring.parity ^ 1, 1u << 16);
            }
          }
          __syncwarp();
          break;
        }
        ring.step();
        info.step();
      }
    } else {
      // ---- bf16: what lies in a V slot for tokens that are not there must not be a NaN
      for (; it.next(a, p, box); ring.step(), info.step()) {
        ok = ok && tc_wait(&sh.v_full[ring.at], ring.parity, &sh.dead);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint4 there = *reinterpret_cast<const uint4*>(sh.there[info.at]);
        if ((there.x & there.y & there.z & there.w) != 0xffffffffu) {
          // two threads a row: the first 64 channels and the others
          for (int i = tid - 32; i < 2 * TC_TILE; i += 96) {
            const int t = i >> 1;
            if (sh.there[info.at][t >> 5] >> (t & 31) & 1) continue;
            uint4* vrow = reinterpret_cast<uint4*>(vslots + ring.at * RW_SLOT + (i & 1) * RW_BLOCK + t * 128);
#pragma unroll
            for (int j = 0; j < 8; ++j) vrow[j] = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async();
        }
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.v_ready[ring.at]);
      }
      if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    }
  } else if (warp == 12 || warp == 13) {
    // ---- products, one thread each
    if (lane == 0) {
      bool ok = true;
      TcRing<2> buf;
      TcRing<RW_RING> ring;
      constexpr uint32_t id = rw_idesc(F8);
      const uint64_t k0 = tc::sdesc(tc::smem_u32(kslots)), q0 = tc::sdesc(tc::smem_u32(qbuf));
      const uint64_t v0 = tc::sdesc_mn(tc::smem_u32(vslots), RW_BLOCK);
      for (int un = 0; ok; ++un) {
        ok = tc_wait(&sh.q_full[un & 1], un >> 1 & 1, &sh.dead);
        if (!ok) break;
        const int t0 = sh.unit[un & 1].t0, t1 = sh.unit[un & 1].t1;
        if (t1 == 0) break;
        for (int t = t0; t < t1; ++t) {
          if (warp == 12) {
            if (F8 && p.stall && t == t0 + TC_STALL_AT) ok = tc_give_up(&sh.dead);
            ok = ok && tc_wait(&sh.p_free[buf.at], buf.parity ^ 1, &sh.dead);
            ok = ok && tc_wait(&sh.k_full[ring.at], ring.parity, &sh.dead);
            if (!ok) break;
            tc::bar_arrive(&sh.s_full[buf.at]);  // hands on what came with K: the tokens and scales
            tc::fence_after_sync();
            const uint64_t kd = k0 + ring.at * (RW_SLOT / 16), qd = q0 + (un & 1) * (RW_SLOT / 16);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // 16 channels per step
              const uint32_t at = (kk / 4 * RW_BLOCK + kk % 4 * 32) / 16;
              tc::mma_ss(tmem + buf.at * 128, qd + at, kd + at, id, kk > 0);
            }
            tc::commit(&sh.s_full[buf.at]);
            tc::commit(&sh.k_empty[ring.at]);
          } else {
            ok = ok && tc_wait(F8 ? &sh.v_full[ring.at] : &sh.v_ready[ring.at], ring.parity, &sh.dead);
            ok = ok && tc_wait(&sh.p_full[buf.at], buf.parity, &sh.dead);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t vd = v0 + ring.at * (RW_SLOT / 16);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {  // 16 tokens per step; the first four are group 0's
              const uint32_t d = tmem + RW_O + kk / 4 * 128, at = tmem + buf.at * 128 + kk / 2 * 32 + kk % 2 * 8;
              const uint64_t db = vd + kk * (2048 / 16);
              tc::mma_ts(d, at, db, id | tc::IDESC_B_MN, !(t == t0 && kk % 4 == 0));
              if constexpr (!F8) tc::mma_ts(d, at + 16, db, id | tc::IDESC_B_MN, 1);
            }
            tc::commit(&sh.p_free[buf.at]);
            tc::commit(&sh.v_empty[ring.at]);
            if (t + 1 == t1) tc::commit(&sh.o_full);
          }
          ring.step();
          buf.step();
        }
      }
      // nothing of this thread's is on its way when the CTA ends
      if (!ok) flag_status(a.status, KDA_DEV_TIMEOUT);
      uint64_t* drain = &sh.drain[warp - 12];
      tc::commit(drain);
      tc::bar_wait(drain, 0);
    }
    __syncwarp();
  } else if (warp >= 14) {
    // ---- each unit for the others, and its queries: 16 lanes a row, all rows on their way at once
    TcWalk w = walk;
    TcUnit u;
    bool ok = true, more = true;
    const int c = lane & 15;
    const float per_unit = a.scale * (a.softcap > 0.f ? 2.f * PA_LOG2E / a.softcap : PA_LOG2E);
    for (int un = 0; more; ++un) {
      const int buf = un & 1;
      more = next_unit(a, p, box, w, u);
      if (un >= 2) ok = tc_wait(&sh.q_free[buf], ((un >> 1) - 1) & 1, &sh.dead);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (more) {
        const int row0 = u.rb * RW_RB, nrows = min(RW_RB, p.rows - row0), rows32 = (nrows + 31) & ~31;
        const uint4* q = static_cast<const uint4*>(a.q) + (int64_t)u.b * a.W * a.Hq * 16 + c;
        const uint32_t q_at = tc::smem_u32(qbuf + buf * RW_SLOT) + (c >> 3) * RW_BLOCK;
        const int r0 = (warp - 14) * 2 + (lane >> 4);
#pragma unroll 4
        for (int r = r0; r < rows32; r += 4) {
          const int wt = (row0 + r) / p.G, hd = r < nrows ? wt * a.Hq + u.h * p.G + (row0 + r - wt * p.G) : -1;
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(q_at + tc::sw128_chunk(r, c & 7)),
                       "l"(q + (int64_t)max(hd, 0) * 16), "r"(hd >= 0 ? 16 : 0)
                       : "memory");
          if (c == 0) {
            sh.head[buf][r] = hd;
            sh.last[buf][r] = hd >= 0 ? u.len - a.W + wt : -1;
            if constexpr (!F8) sh.factor[buf][r] = per_unit;
          }
        }
        if (warp == 14 && lane == 0) sh.unit[buf] = u;
        asm volatile("cp.async.wait_all;" ::: "memory");
        if constexpr (F8) {  // fp16: each row's maximum to [2^14, 2^15) by a power of two, exact down to 2^-31 of it
#pragma unroll 2
          for (int r = r0; r < rows32; r += 4) {
            const uint32_t at = q_at + tc::sw128_chunk(r, c & 7);  // what this thread copied
            uint32_t w4[4], top = 0;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w4[0]), "=r"(w4[1]), "=r"(w4[2]), "=r"(w4[3])
                         : "r"(at)
                         : "memory");
#pragma unroll
            for (int j = 0; j < 4; ++j) top = max(top, max((w4[j] & 0x7fffu) << 16, w4[j] & 0x7fff0000u));
#pragma unroll
            for (int j = 1; j < 16; j <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, j));
            int e = top > 0 && top <= 0x7f800000u ? 14 - ((int)(top >> 23) - 127) : 0;
            e = min(100, e);  // -114 at least
            const float up = __uint_as_float((uint32_t)(e + 127) << 23);
            if (c == 0) sh.factor[buf][r] = per_unit * __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j)
              w4[j] = pack_f16(make_float2(__uint_as_float(w4[j] << 16) * up, __uint_as_float(w4[j] & 0xffff0000u) * up));
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w4[0]), "r"(w4[1]), "r"(w4[2]), "r"(w4[3])
                         : "memory");
          }
        }
        tc::fence_proxy_async();
      } else if (warp == 14 && lane == 0) {
        sh.unit[buf].t1 = 0;
      }
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.q_full[buf]);
    }
    if (!ok && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
  } else {
    // ---- softmax: thread = query row; group g has tokens 64 g .. 64 g + 63 of each tile.  A role that gives up a wait goes
    // on through its unit without results (no later wait holds it), so that the barriers between groups are always met.
    const int tk = (tid - RW_SOFT0) & 127, quarter = warp & 3, g = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16, own_o = tmem + RW_O + g * 128 + lanes;
    const float cap2 = a.softcap * PA_LOG2E;
    const CapPoly cap_poly(cap2);
    bool bad = false;
    TcRing<2> buf, before(1);  // this tile's buffer, and that of the tile before
    before.parity = 1;
    TcRing<RW_INFO> info;
    uint32_t tile_no = 0;
    PaMeta meta{-1, 0};
    int rows_done = 0;
    for (int un = 0;; ++un) {
      const int qb = un & 1;
      bad |= !tc_wait(&sh.q_full[qb], un >> 1 & 1, &sh.dead);
      if (tc::named_bar_or(1, RW_SOFT, bad)) {
        bad = true;
        break;
      }
      const TcUnit u = sh.unit[qb];
      if (u.t1 == 0) break;
      const int row0 = u.rb * RW_RB, nrows = min(RW_RB, p.rows - row0);
      const bool active = quarter * 32 < nrows;
      // tokens that every row of the unit sees: [all_from, all_to]; a window longer than the request is no window
      const int width = min(window, max(u.len, 1));
      const int all_to = u.len - a.W + row0 / p.G, all_from = u.len - a.W + (row0 + nrows - 1) / p.G - width + 1;
      const int last = active ? sh.last[qb][tk] : -1, low = last - width + 1;
      const float factor = active ? sh.factor[qb][tk] : 0.f;
      float m = TC_NONE, l = 0.f;
      for (int tile = u.t0; tile < u.t1; ++tile, buf.step(), before.step(), info.step()) {
        const bool first_tile = tile == u.t0;
        ++tile_no;
        bad |= !tc_wait(&sh.s_full[buf.at], buf.parity, &sh.dead);
        bad = __any_sync(0xffffffffu, bad);
        const uint32_t own_s = tmem + buf.at * 128 + g * 64 + lanes;
        if (active) {
          tc::fence_after_sync();
          const int tok0 = u.start + tile * TC_TILE;
          const uint4 there = *reinterpret_cast<const uint4*>(sh.there[info.at]);
          const bool masked = tok0 > all_to - (TC_TILE - 1) || tok0 < all_from || (there.x & there.y & there.z & there.w) != 0xffffffffu;
          // 32 tokens at a time: few enough instructions to stay in the instruction cache, and no spilled scores
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            const int t0 = g * 64 + h * 32;  // first token within the tile
            float2 x[16];
            bool capped_yet = a.softcap <= 0.f;
            for (;;) {
              float raw[32];
              tc::tmem_ld32(own_s + 32 * h, raw);
#pragma unroll
              for (int i = 0; i < 16; ++i) x[i] = make_float2(raw[2 * i], raw[2 * i + 1]);
              if (a.softcap > 0.f && capped_yet) break;  // as they come
              if constexpr (F8) {
                const uint32_t ks = tc::smem_u32(sh.k_scale[info.at] + t0);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float4 s = ld_shared4(ks + 16 * i);
                  x[2 * i] = mul2(mul2(x[2 * i], make_float2(s.x, s.y)), both(factor));
                  x[2 * i + 1] = mul2(mul2(x[2 * i + 1], make_float2(s.z, s.w)), both(factor));
                }
              } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = mul2(x[i], both(factor));
              }
              if (capped_yet) break;
              float top = 0.f;
#pragma unroll
              for (int i = 0; i < 16; ++i) top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
              if (__all_sync(0xffffffffu, top <= PA_NEAR)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) x[i] = cap_poly(x[i]);
                break;
              }
              // scores near the cap: capped where they are, few at a time (little code for a rare case), and read again
#pragma unroll 1
              for (int c = 0; c < 32; c += 8) {
                float y[8];
                tc::tmem_ld8(own_s + 32 * h + c, y);
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = capped(y[i] * (F8 ? sh.k_scale[info.at][t0 + c + i] : 1.f) * factor, cap2);
                tc::tmem_st8f(own_s + 32 * h + c, y);
              }
              tc::tmem_wait_st();
              capped_yet = true;
            }
            if (masked) {
              // of the 32 the row sees those from `from` on, up to `to`
              const int first = tok0 + t0, to = max(0, min(32, last + 1 - first)), from = max(0, min(32, low - first));
              uint32_t seen = g == 0 ? (h == 0 ? there.x : there.y) : (h == 0 ? there.z : there.w);
              if (to < 32) seen &= (1u << to) - 1;
              seen &= from < 32 ? ~((1u << from) - 1) : 0u;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                x[i].x = seen >> (2 * i) & 1 ? x[i].x : -INFINITY;
                x[i].y = seen >> (2 * i + 1) & 1 ? x[i].y : -INFINITY;
              }
            }
            // ---- the reference moves only when a score is far above it (always on the first seen token), and by whole powers
            // of two, so that probabilities written already follow exactly
            float over = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; ++i) over = fmaxf(over, fmaxf(x[i].x, x[i].y));
            bool move = over + (F8 ? sh.lift_top[info.at][2 * g + h] : 0.f) > m + pa_slack(F8);
            if (F8 && __any_sync(0xffffffffu, move)) {  // so says a bound: now token by token
              // A value of zeros has a scale all the same: it adds nothing, and lifts the reference as the least scale does.  (All
              // warps of the group write the same; to one that does not move, either scale of such a token is right.)
              bad |= !rw_put(&sh.v_tile[2 * g + h], tile_no, &sh.dead);
              bad = __any_sync(0xffffffffu, bad);
              const uint32_t slot = tc::smem_u32(vslots + ((tile_no - 1) % RW_RING) * RW_SLOT);
              if (rw_nonzero(slot, t0 + lane) == 0)
                sh.v_scale[info.at][t0 + lane] = 0.f, sh.lift[info.at][t0 + lane] = PA_LEAST_LIFT + pa_head(F8, false);
              __syncwarp();
              const uint32_t lift = tc::smem_u32(sh.lift[info.at] + t0);
              over = -INFINITY;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float4 s = ld_shared4(lift + 16 * i);
                const float2 y = add2(x[2 * i], make_float2(s.x, s.y)), z = add2(x[2 * i + 1], make_float2(s.z, s.w));
                over = fmaxf(over, fmaxf(fmaxf(y.x, y.y), fmaxf(z.x, z.y)));
              }
              move = over > m + pa_slack(F8);
            }
            if (__any_sync(0xffffffffu, move)) {
              const float mn = fmaxf(m, ceilf(over) - pa_head(F8, false)), by = mn - m > 126.f ? 0.f : __uint_as_float((uint32_t)(127 - (int)(mn - m)) << 23);
              l = F8 && mn - m > 126.f ? times_pow2(l, m - mn) : l * by;
              m = mn;
              if (h == 1) {  // the first 32 tokens' probabilities
                tc::tmem_wait_st();  // what pass 0 stored, probabilities and accumulators, before it is read back
#pragma unroll 1
                for (int c = 0; c < (F8 ? 16 : 32); c += 8) {
                  float w[8];
                  tc::tmem_ld8(own_s + c, w);
#pragma unroll
                  for (int i = 0; i < 8; ++i) w[i] = __uint_as_float(times16<F8>(__float_as_uint(w[i]), by));
                  tc::tmem_st8f(own_s + c, w);
                }
              }
              if (!first_tile) {
                // the last product into this accumulator is through
                bad |= !tc_wait(&sh.p_free[before.at], before.parity, &sh.dead);
                bad = __any_sync(0xffffffffu, bad);
                tc::fence_after_sync();
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                  float o[16];
                  uint32_t w[16];
                  tc::tmem_ld16(own_o + c, o);
#pragma unroll
                  for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[i] * by);
                  tc::tmem_st16(own_o + c, w);
                }
              }
            }
            // ---- probabilities, to tensor memory over the scores: of 32 columns the first 16, for bf16 what they leave in the others
            uint32_t hi[16], lo[16];
            const uint32_t vs = tc::smem_u32(sh.v_scale[info.at] + t0);
            float2 sum = make_float2(l, 0.f), sum1 = both(0.f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float2 e0 = add2(x[2 * i], both(-m)), e1 = add2(x[2 * i + 1], both(-m));
              e0 = make_float2(ex2(e0.x), ex2(e0.y)), e1 = make_float2(ex2(e1.x), ex2(e1.y));
              sum = add2(sum, e0), sum1 = add2(sum1, e1);
              if constexpr (F8) {
                const float4 s = ld_shared4(vs + 16 * i);
                e0 = mul2(e0, make_float2(s.x, s.y)), e1 = mul2(e1, make_float2(s.z, s.w));
                hi[2 * i] = pack_f16(e0), hi[2 * i + 1] = pack_f16(e1);
              } else {
                hi[2 * i] = split_pair<false>(e0.x, e0.y), hi[2 * i + 1] = split_pair<false>(e1.x, e1.y);
                lo[2 * i] = pack_bf16(e0.x, e0.y), lo[2 * i + 1] = pack_bf16(e1.x, e1.y);
              }
            }
            sum = add2(sum, sum1);
            l = sum.x + sum.y;
            tc::tmem_st16(own_s + 32 * h, hi);
            if constexpr (!F8) tc::tmem_st16(own_s + 32 * h + 16, lo);
          }
          tc::tmem_wait_st();
        }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) tc::bar_arrive(&sh.p_full[buf.at]);
      }

      // ---- end of the unit's part: the groups' results joined, each writing 64 channels
      const bool whole = u.t0 == 0 && u.t1 == u.tiles;
      const int64_t part_at = (me * 2 + (u.t0 == 0 ? 1 : 0)) * RW_RB, heads = (int64_t)u.b * a.W * a.Hq;
      sh.ml[g][tk] = make_float2(m, l);
      bad |= !tc_wait(&sh.o_full, un & 1, &sh.dead);
      bad = __any_sync(0xffffffffu, bad);
      tc::fence_after_sync();
      tc::named_bar(1, RW_SOFT);
      bool nan = false;
      const int head = active ? sh.head[qb][tk] : -1;
      if (active && !bad) {
        const float2 other = sh.ml[1 - g][tk];
        float mr = fmaxf(m, other.x);
        const float own = ex2(m - mr), his = ex2(other.x - mr);
        float lr;
        if constexpr (F8) lr = __fadd_rn(times_pow2(l, m - mr), times_pow2(other.y, other.x - mr));
        else lr = g == 0 ? l * own + other.y * his : other.y * his + l * own;
        const float by0 = g == 0 ? own : his, by1 = g == 0 ? his : own;
        const bool none = mr == TC_NONE && lr == 0.f;
        if (mr == TC_NONE) mr = none ? -INFINITY : 0.f;  // nothing but NaN scores: let them through
        float over_l = 1.f;
        if (whole) asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(over_l) : "f"(lr));
        const float2 f0 = both(none ? 0.f : by0 * over_l), f1 = both(none ? 0.f : by1 * over_l);
        // over the queries, which the products have read: 32 channels of each group at a time, 128 bytes a row
        const uint32_t turn = tc::smem_u32(qbuf + qb * RW_SLOT) + g * RW_BLOCK;
        float2 check = both(0.f);
        const int r0 = quarter * 32 + (lane >> 3);
        int hd[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) hd[i] = sh.head[qb][r0 + 4 * i];
#pragma unroll 1
        for (int c = 0; c < 64; c += 32) {
          float o[32], o1[32];
          tc::tmem_ld32_two(tmem + RW_O + lanes + g * 64 + c, tmem + RW_O + 128 + lanes + g * 64 + c, o, o1);
#pragma unroll
          for (int i = 0; i < 32; i += 4) {
            float2 y0 = fma2(make_float2(o1[i], o1[i + 1]), f1, mul2(make_float2(o[i], o[i + 1]), f0));
            float2 y1 = fma2(make_float2(o1[i + 2], o1[i + 3]), f1, mul2(make_float2(o[i + 2], o[i + 3]), f0));
            check = fma2(y0, both(0.f), check), check = fma2(y1, both(0.f), check);  // NaN where one is NaN or infinite
            if (none) y0 = y1 = both(0.f);
            asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(turn + tc::sw128_chunk(tk, i / 4)), "f"(y0.x),
                         "f"(y0.y), "f"(y1.x), "f"(y1.y)
                         : "memory");
          }
          __syncwarp();
          const int ch = g * 64 + c + (lane & 7) * 4;
          float4 y[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = ld_shared4(turn + tc::sw128_chunk(r0 + 4 * i, lane & 7));
          if (whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              uint2 w;
              w.x = pack_bf16(y[i].x, y[i].y);
              w.y = pack_bf16(y[i].z, y[i].w);
              if (hd[i] >= 0) *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + (heads + hd[i]) * TC_D + ch) = w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (hd[i] >= 0) *reinterpret_cast<float4*>(p.part_o + (part_at + r0 + 4 * i) * TC_D + ch) = y[i];
          }
          __syncwarp();
        }
        nan = !none && isnan(check.x + check.y);
        if (head >= 0 && g == 0) {
          if (!whole) *reinterpret_cast<float2*>(p.part_ml + (part_at + tk) * 2) = make_float2(mr, lr);
          else if (a.lse) a.lse[heads + head] = none ? -INFINITY : log_sum(mr, lr);
        }
      }
      const uint32_t nans = __ballot_sync(0xffffffffu, nan && head >= 0);
      if (lane == 0) sh.nan[g][quarter] = nans;
      if (tc::named_bar_or(1, RW_SOFT, nans != 0)) {
        for (int r = warp - 4; r < nrows; r += 8) {
          if (bad || !((sh.nan[0][r >> 5] | sh.nan[1][r >> 5]) >> (r & 31) & 1)) continue;
          float4 o;
          float mr, lr;
          careful_row<F8>(a, p, u, row0 + r, o, mr, lr);
          const bool none = mr == TC_NONE && lr == 0.f;
          if (mr == TC_NONE) mr = none ? -INFINITY : 0.f;
          if (whole) {
            const int wt = (row0 + r) / p.G;
            const int64_t at = heads + (int64_t)wt * a.Hq + u.h * p.G + (row0 + r - wt * p.G);
            const float by = none ? 0.f : 1.f / lr;
            uint2 y;
            y.x = pack_bf16(o.x * by, o.y * by);
            y.y = pack_bf16(o.z * by, o.w * by);
            *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + at * TC_D + 4 * lane) = y;
            if (lane == 0 && a.lse) a.lse[at] = none ? -INFINITY : log_sum(mr, lr);
          } else {
            *reinterpret_cast<float4*>(p.part_o + (part_at + r) * TC_D + 4 * lane) = o;
            if (lane == 0) *reinterpret_cast<float2*>(p.part_ml + (part_at + r) * 2) = make_float2(mr, lr);
          }
        }
      }
      __syncwarp();
      if (lane == 0) tc::bar_arrive(&sh.q_free[qb]);  // the unit's rows have been read, and written from its queries' place
      if (whole) {
        rows_done += nrows;
      } else if (u.t0 == 0 && tid == RW_SOFT0) {
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
    if (bad && lane == 0) flag_status(a.status, KDA_DEV_TIMEOUT);
    if (tid == RW_SOFT0) {
      p.meta[me] = bad ? PaMeta{-1, 0} : meta;
      add_work(a.status, rows_done);
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 12) tc::tmem_dealloc(tmem, RW_TMEM);
}

template <bool F8>
cudaError_t rows_launch(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  auto kernel = paged_attention_rows_kernel<F8>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RW_SMEM);
  if (e != cudaSuccess) return e;
  const int box = page_box(a.c.page_size);
  TcMaps maps{};
  if (!F8) {
    const long long rows = (long long)a.c.num_pages * a.c.Hkv * a.c.page_size;
    if (!encode_cache_map(&maps.k, a.c.k_pages, rows, box) || !encode_cache_map(&maps.v, a.c.v_pages, rows, box))
      return cudaErrorInvalidValue;
  }
  int64_t ctas = sms < PA_SMS ? sms : PA_SMS;
  const int64_t tiles = (int64_t)a.max_pages * a.c.page_size / TC_TILE + 2 + TC_UNIT_COST;
  const int64_t units = (int64_t)a.B * a.c.Hkv * p.blocks;
  if (tiles < ctas && units * tiles < ctas) ctas = units * tiles;
  PaPlan plan = p;
  plan.workers = (int)ctas;
  e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(RW_NT), RW_SMEM, s, maps, a, plan, box);
  if (e != cudaSuccess) return e;
  return pa_join<TC_D, RW_RB>(a, plan, units, s);
}

}  // namespace

bool pa_rows_supported(const PagedAttnArgs& a) {
  return a.c.d == TC_D && a.q_bf16 && a.out_bf16 && a.c.num_pages > 0 &&
         (a.c.e4m3 || (int64_t)a.c.num_pages * a.c.Hkv * a.c.page_size <= 0x7fffffff);
}

cudaError_t pa_rows(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  return a.c.e4m3 ? rows_launch<true>(a, p, sms, s) : rows_launch<false>(a, p, sms, s);
}

}  // namespace kda
