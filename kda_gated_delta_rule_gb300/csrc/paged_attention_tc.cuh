// What the two tensor-memory forms of the attention share (d = 128): the walk over a CTA's share of the line of tiles, bounded
// waits, and the careful way out.
#pragma once

#include "paged_attention.cuh"
#include "tc_ptx.cuh"
#include "tmap.h"

namespace kda {

namespace {

constexpr int TC_TILE = 128, TC_D = 128;
constexpr int TC_UNIT_COST = 2;        // tiles a unit counts beyond its own (64 ragged requests with 96 rows: 43.8 us; 1: 44.7, 4: 46.8)
constexpr float TC_NONE = -3.402823466e38f;  // a softmax reference that has seen nothing (finite: no -inf - -inf)

// A place in a ring of N with the parity of its current round.
template <int N>
struct TcRing {
  int at = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ explicit TcRing(int first = 0) : at(first) {}
  __device__ __forceinline__ void step(int by = 1) {
    at += by;
    if (at >= N) at -= N, parity ^= 1;
  }
};

struct TcMaps {
  CUtensorMap k, v;
};

// ---- the share of this CTA, unit by unit and tile by tile; every role walks it on its own

struct TcUnit {
  int b, h, rb, row0, len, start, tiles, t0, t1;
};
struct TcWalk {
  int64_t at, end, first_of_b;
  int b;
};
__device__ __forceinline__ bool next_unit(const PagedAttnArgs& a, const PaPlan& p, int align, TcWalk& w, TcUnit& u) {
  const int per_b = a.c.Hkv * p.blocks;
  while (w.at < w.end) {
    const PaSpan span = pa_span<TC_TILE>(a, w.b, false, align);
    const int cost = span.tiles + TC_UNIT_COST;
    const int in_b = (int)((w.at - w.first_of_b) / cost);
    const int64_t first = w.first_of_b + (int64_t)in_b * cost, last = first + cost;
    u.b = w.b;
    u.h = in_b / p.blocks;
    u.rb = in_b - u.h * p.blocks;
    u.len = span.len, u.start = span.start, u.tiles = span.tiles;
    u.t0 = max(0, (int)(w.at - first) - TC_UNIT_COST);
    u.t1 = (int)((w.end < last ? w.end : last) - first) - TC_UNIT_COST;
    w.at = w.end < last ? w.end : last;
    if (in_b == per_b - 1 && w.at == last) {
      w.first_of_b = last;
      ++w.b;
    }
    if (u.t1 > u.t0) return true;
  }
  return false;
}
struct TcTiles {
  TcWalk w;
  TcUnit u;
  int tile, unit_no;
  __device__ __forceinline__ explicit TcTiles(const TcWalk& from) : w(from), tile(0), unit_no(-1) { u.t1 = 0; }
  __device__ __forceinline__ bool next(const PagedAttnArgs& a, const PaPlan& p, int align) {
    if (unit_no >= 0 && ++tile < u.t1) return true;
    if (!next_unit(a, p, align, w, u)) return false;
    tile = u.t0;
    ++unit_no;
    return true;
  }
  __device__ __forceinline__ bool first() const { return tile == u.t0; }
  __device__ __forceinline__ bool last() const { return tile + 1 == u.t1; }
};

// A bounded wait that also ends when another role has given up.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, int* dead) {
  if (tc::bar_test(bar, parity)) return true;
  for (int i = 0; i < 1 << 12; ++i) {
    if (*reinterpret_cast<volatile int*>(dead)) return false;
    if (tc::bar_wait(bar, parity, 1u << 10)) return true;
  }
  *reinterpret_cast<volatile int*>(dead) = 1;
  return false;
}

// For tests of the way out (kda_set_test_fault): the copying warp leaves as if its wait for a slot had run out, at this tile of its
// share, with the copies of those before it and of its keys on their way.  (Of an e4m3 cache, which has no such copies, the first
// product's warp, at this tile of a unit: any statement more in the loaders cost the calls 10 %.)
constexpr int TC_STALL_AT = 2;
__device__ __forceinline__ bool tc_give_up(int* dead) {
  *reinterpret_cast<volatile int*>(dead) = 1;
  return false;
}

// One row of a part by one warp, token by token in fp32: the way out when the accumulators hold a NaN, which may come from
// a query that meets a token it does not see (0 * NaN) or from an infinity meeting a split probability.  A lane has
// channels 4 lane .. 4 lane + 3.
template <bool F8>
__device__ __noinline__ void careful_row(const PagedAttnArgs& a, const PaPlan& p, const TcUnit& u, int qrow, float4& o,
                                         float& m, float& l) {
  const int lane = threadIdx.x & 31, w = qrow / p.G, g = qrow - w * p.G;
  const int64_t head = ((int64_t)u.b * a.W + w) * a.Hq + (int64_t)u.h * p.G + g;
  const bf16* q = static_cast<const bf16*>(a.q) + head * TC_D + 4 * lane;
  const float q0 = to_f32(q[0]), q1 = to_f32(q[1]), q2 = to_f32(q[2]), q3 = to_f32(q[3]);
  const int last = u.len - a.W + w, window = a.window > 0 ? a.window : 0x7fffffff;
  const int64_t lo = max((int64_t)u.start + (int64_t)u.t0 * TC_TILE, (int64_t)last - window + 1);
  const int64_t hi = min(min((int64_t)u.len, (int64_t)u.start + (int64_t)u.t1 * TC_TILE), (int64_t)last + 1);
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  m = TC_NONE;
  l = 0.f;
  for (int64_t tok = lo < 0 ? 0 : lo; tok < hi; ++tok) {
    const int pg = (int)(tok / a.c.page_size), page = __ldg(a.block_table + (int64_t)u.b * a.max_pages + pg);
    if ((unsigned)page >= (unsigned)a.c.num_pages) continue;
    const int64_t row = ((int64_t)page * a.c.Hkv + u.h) * a.c.page_size + (tok - (int64_t)pg * a.c.page_size);
    float k[4], v[4];
    if constexpr (F8) {
      const uint32_t kw = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.c.k_pages) + row * TC_D) + lane);
      const uint32_t vw = __ldg(reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(a.c.v_pages) + row * TC_D) + lane);
      const float ks = __ldg(a.c.k_scales + row), vs = __ldg(a.c.v_scales + row);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const uint32_t k2 = half2_of_codes(kw >> (8 * i)), v2 = half2_of_codes(vw >> (8 * i));
        const float2 kf = __half22float2(*reinterpret_cast<const __half2*>(&k2));
        const float2 vf = __half22float2(*reinterpret_cast<const __half2*>(&v2));
        k[i] = kf.x * ks, k[i + 1] = kf.y * ks, v[i] = vf.x * vs, v[i + 1] = vf.y * vs;
      }
    } else {
      const bf16* kp = static_cast<const bf16*>(a.c.k_pages) + row * TC_D + 4 * lane;
      const bf16* vp = static_cast<const bf16*>(a.c.v_pages) + row * TC_D + 4 * lane;
#pragma unroll
      for (int i = 0; i < 4; ++i) k[i] = to_f32(kp[i]), v[i] = to_f32(vp[i]);
    }
    float s = q0 * k[0] + q1 * k[1] + q2 * k[2] + q3 * k[3];
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= a.scale;
    s = a.softcap > 0.f ? a.softcap * tanhf(s / a.softcap) * PA_LOG2E : s * PA_LOG2E;
    const float mn = fmaxf(m, s), by = ex2(m - mn), e = ex2(s - mn);
    m = mn;
    l = l * by + e;
    o.x = o.x * by + e * v[0], o.y = o.y * by + e * v[1], o.z = o.z * by + e * v[2], o.w = o.w * by + e * v[3];
  }
}

inline int page_box(int page_size) {  // largest power of two that divides the page, at most a tile
  const int b = page_size & -page_size;
  return b < TC_TILE ? b : TC_TILE;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace

}  // namespace kda
