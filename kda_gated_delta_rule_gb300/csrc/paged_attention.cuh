// Attention of the newest tokens of each request over its paged key/value cache.
//
// Per query row (a query head of one window token), over the positions it sees, with x = scale q.k (capped:
// cap tanh(x / cap)):  out = sum exp(x - m) v / sum exp(x - m),  lse = m + log sum exp(x - m).
//
// Bound by HBM: a cached row of d channels feeds the few query rows of its head group (Hq / Hkv heads x W tokens),
// so each K or V element is read once and used for 2 multiplications per query row.
//
// Work.  A unit is one request, key/value head and block of RB = 8 NT query rows.  All units' caches, cut into tiles
// of TILE tokens, form one line of tiles; the CTAs take equal consecutive shares of it, so ragged lengths balance
// without the host knowing them, and a single long request spreads over the whole GPU.  A CTA that has a whole unit
// writes its output; the parts of a unit cut across CTAs go to the workspace (each CTA has at most one part that
// continues a unit and one that starts one) and a second, small kernel joins them in order.
//
// Inside a CTA four warps take the 16-token groups of a tile in turn, each with its own running maximum, sum and
// accumulators, joined at the end of the unit.  K and V go from global memory straight into the operand registers of
// mma.m16n8k16 (no shared memory, no transposes): the products are S^T = K Q^T and O^T = V^T P^T with the tokens
// resp. channels as the 16-row side and 8 query rows as columns.  The channel order inside a product's K steps is
// free as long as Q follows it, so a lane's operands for consecutive steps are one 16-byte piece of its token's row;
// V's pairs of tokens are put together from two such pieces by byte permutes.  The 5th-generation tensor instructions
// want 64 or 128 rows and both operands in shared or tensor memory; with 1 to 32 query rows they would sit idle
// behind the same loads.
//
// e4m3 caches: codes become fp16 (exact), q is scaled per row by a power of two into fp16's range (exact for bf16 q
// down to 2^-31 of the row's maximum), the key's scale multiplies the score and the value's scale the
// probability.  The running reference of the softmax is then the maximum of x + log2(value scale), so that the
// scaled probabilities fit fp16 for any scales.
//
// Rounding to fewer bits: probabilities enter the second product as 16-bit numbers.  fp16 (e4m3 cache) has 11 bits,
// well below the bf16 output's 8; bf16 (bf16 cache) has 8, so they go in as a sum of two bf16 (16 bits), else
// the output's error would grow by half.  With fp32 queries or outputs both products use more parts (FINE).
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "launch.h"

namespace kda {

constexpr int PA_NT = 128, PA_WARPS = 4;
constexpr int PA_MAX_CTAS = 608;  // four per SM
constexpr float PA_LOG2E = 1.4426950408889634f, PA_LN2 = 0.6931471805599453f;
// how far (in powers of two) scores may run above the softmax reference before it is moved
constexpr float PA_SLACK = 6.f;

// What the main kernel leaves for the join, per CTA.
struct PaMeta {
  int64_t tiles;  // tiles of all units
  int unit;       // the unit whose first part is this CTA's last, -1 if none
  int end_cta;    // the CTA with that unit's last part
};

__host__ __device__ constexpr int pa_nt(int rows) { return rows <= 8 ? 1 : rows <= 16 ? 2 : 4; }

struct PaPlan {  // derived on the host
  int G;         // query heads per key/value head
  int rows;      // query rows per key/value head: W * G
  int blocks;    // row blocks of RB per key/value head
  float* part_o;   // [CTA][2][RB][D]
  float* part_ml;  // [CTA][2][RB][2]
  PaMeta* meta;    // [CTA]
};

// ---------------------------------------------------------------- instructions

template <bool F8>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (F8)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t half2_of_codes(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)two));
  return r;
}
// Two fp32 as a 16-bit pair, and what the pair leaves of them.
template <bool F8>
__device__ __forceinline__ uint32_t split_pair(float& lo, float& hi) {
  uint32_t r;
  if constexpr (F8) {
    const __half2 h = __floats2half2_rn(lo, hi);
    const float2 f = __half22float2(h);
    r = *reinterpret_cast<const uint32_t*>(&h);
    lo -= f.x, hi -= f.y;
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    r = *reinterpret_cast<const uint32_t*>(&h);
    lo -= __uint_as_float(r << 16), hi -= __uint_as_float(r & 0xffff0000u);
  }
  return r;
}

// A lane's piece of a cached row: BYTES bytes as words (the last one half empty for 2 bytes).
template <int BYTES>
struct Piece {
  uint32_t w[BYTES < 4 ? 1 : BYTES / 4];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < (BYTES < 4 ? 1 : BYTES / 4); ++i) w[i] = 0;
  }
  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (BYTES == 16) {
      asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
          : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    } else if constexpr (BYTES == 8) {
      asm("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    } else if constexpr (BYTES == 4) {
      asm("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    } else {
      uint16_t h;
      asm("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(h) : "l"(p));
      w[0] = h;
    }
  }
};

// ---------------------------------------------------------------- the line of tiles

// Tokens a request's window sees: first seen position rounded down to 16, and the tiles from there to its length.
struct PaSpan {
  int len, start, tiles;
};
template <int TILE>
__device__ __forceinline__ PaSpan pa_span(const PagedAttnArgs& a, int b, bool flag) {
  PaSpan s;
  s.len = __ldg(a.seq_lens + b);
  if (s.len < 0 || s.len > (int64_t)a.max_pages * a.c.page_size) {
    if (flag) flag_status(a.status, KDA_DEV_SEQ_OOB);
    s.len = 0;
  }
  int64_t first = a.window > 0 ? (int64_t)s.len - a.W - a.window + 1 : 0;  // of the window's first query
  if (first < 0) first = 0;
  s.start = (int)first & ~15;
  const int64_t n = (int64_t)s.len - s.start;
  s.tiles = n > 0 ? (int)((n + TILE - 1) / TILE) : 1;  // a unit with nothing to see still writes its rows
  return s;
}

// ---------------------------------------------------------------- main kernel

template <int D, bool F8, int NT, bool FINE>
struct PaCfg {
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int RB = 8 * NT;
  static constexpr int GPI = F8 ? 2 : 1;                 // 16-token groups a warp works on at once
  static constexpr int TILE = 16 * GPI * PA_WARPS;       // tokens
  static constexpr int KC = D / 4 < 16 / ES ? D / 4 : 16 / ES;  // channels of a key piece
  static constexpr int KL = D / (4 * KC);                // key pieces per lane and token
  static constexpr int VC = D / 8 < 16 / ES ? D / 8 : 16 / ES;  // channels of a value piece
  static constexpr int VL = D / (8 * VC);
  static constexpr int KS = D / 16;                      // K steps of the first product, 16-channel tiles of the second
  static constexpr int QP = FINE ? (F8 ? 2 : 3) : 1;     // 16-bit parts of a query
  static constexpr int PP = FINE ? (F8 ? 2 : 3) : (F8 ? 1 : 2);  // and of a probability
};

template <int D, bool F8, int NT, bool FINE>
__global__ void __launch_bounds__(PA_NT) paged_attention_kernel(const PagedAttnArgs a, const PaPlan p) {
  using C = PaCfg<D, F8, NT, FINE>;
  constexpr int RB = C::RB, TILE = C::TILE, GPI = C::GPI, KS = C::KS;
  __shared__ uint2 qs[C::QP][NT][KS][32];    // Q in the operand order of the first product
  __shared__ float qscale[RB];               // per row: score in powers of two per unit of the first product
  __shared__ float red[RB][D + 4];           // a unit's accumulators, warps joined
  __shared__ float red_m[PA_WARPS][RB], red_l[PA_WARPS][RB];
  __shared__ int64_t scan[PA_NT];
  __shared__ int64_t where[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, j = lane & 3;
  const int Hkv = a.c.Hkv, per_b = Hkv * p.blocks;  // units per request

  // ---- this CTA's share of the line: each thread sums the tiles of a run of requests, then the sums are scanned
  const int run = (a.B + PA_NT - 1) / PA_NT;
  int64_t mine = 0;
  for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b) mine += pa_span<TILE>(a, b, blockIdx.x == 0).tiles;
  scan[tid] = mine;
  __syncthreads();
  for (int o = 1; o < PA_NT; o <<= 1) {
    const int64_t v = tid >= o ? scan[tid - o] : 0;
    __syncthreads();
    scan[tid] += v;
    __syncthreads();
  }
  const int64_t total = scan[PA_NT - 1] * per_b;
  const int64_t ctas = total < gridDim.x ? total : (int64_t)gridDim.x;
  if (blockIdx.x >= ctas) {
    if (tid == 0) p.meta[blockIdx.x] = PaMeta{total, -1, 0};
    return;
  }
  int64_t at = blockIdx.x * total / ctas;  // tile on the line
  const int64_t end = (blockIdx.x + 1) * total / ctas;
  // the request of `at`, and its first tile on the line
  const int64_t before = scan[tid] - mine;
  if (at >= before * per_b && at < scan[tid] * per_b) {
    int64_t f = before;
    for (int b = tid * run;; ++b) {
      const int t = pa_span<TILE>(a, b, false).tiles;
      if (at < (f + t) * per_b) {
        where[0] = b;
        where[1] = f * per_b;
        break;
      }
      f += t;
    }
  }
  __syncthreads();
  int b = (int)where[0];
  int64_t first_of_b = where[1];
  PaMeta meta{total, -1, 0};
  int rows_done = 0;

  while (at < end) {
    const PaSpan span = pa_span<TILE>(a, b, false);
    const int in_b = (int)((at - first_of_b) / span.tiles);  // unit within the request
    const int h = in_b / p.blocks, rb = in_b - h * p.blocks;
    const int64_t unit_first = first_of_b + (int64_t)in_b * span.tiles, unit_end = unit_first + span.tiles;
    const int t0 = (int)(at - unit_first), t1 = (int)((end < unit_end ? end : unit_end) - unit_first);
    const int row0 = rb * RB;

    // ---- queries of the unit, RB rows of D channels, into operand order
    __syncthreads();
    for (int r = warp; r < RB; r += PA_WARPS) {
      const int row = row0 + r, w = row / p.G, g = row - w * p.G;
      float x[D < 32 ? 1 : D / 32];
      float amax = 0.f;
      const int64_t base = (((int64_t)b * a.W + w) * a.Hq + (int64_t)h * p.G + g) * D;
#pragma unroll
      for (int i = 0; i < (D < 32 ? 1 : D / 32); ++i) {
        const int c = i * 32 + lane;
        x[i] = 0.f;
        if (row < p.rows && c < D)
          x[i] = a.q_bf16 ? to_f32(static_cast<const bf16*>(a.q)[base + c]) : static_cast<const float*>(a.q)[base + c];
        amax = fmaxf(amax, fabsf(x[i]));
      }
      float up = 1.f, down = 1.f;
      if constexpr (F8) {  // the row's maximum to [2^14, 2^15)
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        int e = amax > 0.f ? 14 - ((int)(__float_as_uint(amax) >> 23) - 127) : 0;
        e = max(-100, min(100, e));
        up = __uint_as_float((uint32_t)(e + 127) << 23);
        down = __uint_as_float((uint32_t)(127 - e) << 23);
      }
      if (lane == 0) qscale[r] = down * a.scale;
#pragma unroll
      for (int i = 0; i < (D < 32 ? 1 : D / 32); ++i) {
        const int c = i * 32 + lane;
        if (c >= D) break;
        float v = x[i] * up;
        // channel c belongs to key piece c / (4 KC), lane quarter jj, step s of the piece, place e of the step
        const int l = c / (4 * C::KC), jj = c / C::KC % 4, in = c % C::KC, s = l * (C::KC / 4) + in / 4, e = in % 4;
#pragma unroll
        for (int part = 0; part < C::QP; ++part) {
          uint16_t bits;
          if constexpr (F8) {
            const __half hv = __float2half_rn(v);
            v -= __half2float(hv);
            bits = __half_as_ushort(hv);
          } else {
            const bf16 bv = __float2bfloat16_rn(v);
            v -= __bfloat162float(bv);
            bits = __bfloat16_as_ushort(bv);
          }
          reinterpret_cast<uint16_t*>(&qs[part][r / 8][s][(r % 8) * 4 + jj])[e] = bits;
        }
      }
    }
    __syncthreads();

    // per lane: the two query rows of each 8-row column block, their last seen position and score factor
    int last[NT][2];
    float f[NT][2], m[NT][2], l[NT][2];
    float o[NT][KS][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = row0 + t * 8 + 2 * j + c;
        last[t][c] = row < p.rows ? span.len - a.W + row / p.G : -1;
        f[t][c] = qscale[t * 8 + 2 * j + c] * (a.softcap > 0.f ? 1.f : PA_LOG2E);
      }
    }
    const int window = a.window > 0 ? a.window : 0x7fffffff;
    // tokens every row of the unit sees: [all_from, all_to]
    const int w_lo = row0 / p.G, w_hi = min(p.rows - 1, row0 + RB - 1) / p.G;
    const int all_to = span.len - a.W + w_lo;
    const int64_t all_from = (int64_t)span.len - a.W + w_hi - window + 1;

    // ---- walk of the 16-token groups: this warp's group q of tile t is number (t * WARPS + warp) * GPI + q
    Piece<C::KC * C::ES> k[GPI][2][C::KL];
    Piece<C::VC * C::ES> v[GPI][4][C::VL];
    float ks[GPI][2], vs[GPI][2];
    int64_t row_of[GPI], next_row[GPI];  // cache row of the group's first token, -1: nothing to read
    const int32_t* table = a.block_table + (int64_t)b * a.max_pages;
    auto locate = [&](int tile, int64_t (&row)[GPI]) {
#pragma unroll
      for (int q = 0; q < GPI; ++q) {
        const int64_t tok = (int64_t)span.start + ((int64_t)(tile * PA_WARPS + warp) * GPI + q) * 16;
        row[q] = -1;
        if (tile < t1 && tok < span.len) {
          const int pg = (int)tok / a.c.page_size, off = (int)tok - pg * a.c.page_size;
          const int page = __ldg(table + pg);
          if ((unsigned)page < (unsigned)a.c.num_pages)
            row[q] = ((int64_t)page * Hkv + h) * a.c.page_size + off;
          else if (lane == 0)
            flag_status(a.status, KDA_DEV_PAGE_OOB);
        }
      }
    };
    // tokens of a group that exist: 16, fewer at the end of the request
    auto count = [&](int tile, int q) {
      const int64_t tok = (int64_t)span.start + ((int64_t)(tile * PA_WARPS + warp) * GPI + q) * 16;
      const int64_t c = span.len - tok;
      return c < 16 ? (int)c : 16;
    };
    auto load_k = [&](int tile, const int64_t (&row)[GPI]) {
#pragma unroll
      for (int q = 0; q < GPI; ++q) {
        const int cnt = row[q] < 0 ? 0 : count(tile, q);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tok = n + 8 * i;
          const uint8_t* at_k = static_cast<const uint8_t*>(a.c.k_pages) + (row[q] + tok) * (D * C::ES);
#pragma unroll
          for (int u = 0; u < C::KL; ++u) {
            if (tok < cnt) k[q][i][u].load(at_k + (u * 4 + j) * (C::KC * C::ES));
            else k[q][i][u].clear();
          }
          if constexpr (F8) {
            ks[q][i] = tok < cnt ? __ldg(a.c.k_scales + row[q] + tok) : 0.f;
            vs[q][i] = tok < cnt ? __ldg(a.c.v_scales + row[q] + tok) : 0.f;
          }
        }
      }
    };
    auto load_v = [&](int tile, const int64_t (&row)[GPI]) {
#pragma unroll
      for (int q = 0; q < GPI; ++q) {
        const int cnt = row[q] < 0 ? 0 : count(tile, q);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = 2 * j + (i & 1) + 8 * (i >> 1);
          const uint8_t* at_v = static_cast<const uint8_t*>(a.c.v_pages) + (row[q] + tok) * (D * C::ES);
#pragma unroll
          for (int u = 0; u < C::VL; ++u) {
            if (tok < cnt) v[q][i][u].load(at_v + (u * 8 + n) * (C::VC * C::ES));
            else v[q][i][u].clear();
          }
        }
      }
    };
    // O^T += V^T P^T for one group; pr[t]: this lane's probabilities (tokens n, n + 8; rows 2j, 2j + 1), times the
    // value scale where there is one
    auto add_pv = [&](int q, float (&pr)[NT][4]) {
      uint32_t pb[C::PP][NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int part = 0; part < C::PP; ++part) {
          pb[part][t][0] = transpose8x8(split_pair<F8>(pr[t][0], pr[t][1]));
          pb[part][t][1] = transpose8x8(split_pair<F8>(pr[t][2], pr[t][3]));
        }
#pragma unroll
      for (int u = 0; u < C::VL; ++u)
#pragma unroll
        for (int mt = 0; mt < C::VC / 2; ++mt) {  // channels 2 mt and 2 mt + 1 of the piece
          uint32_t va[4];
          if constexpr (F8) {
            const uint32_t sel = (mt & 1) ? 0x7362u : 0x5140u;
            const uint32_t x = __byte_perm(v[q][0][u].w[mt / 2], v[q][1][u].w[mt / 2], sel);
            const uint32_t y = __byte_perm(v[q][2][u].w[mt / 2], v[q][3][u].w[mt / 2], sel);
            va[0] = half2_of_codes(x & 0xffffu), va[1] = half2_of_codes(x >> 16);
            va[2] = half2_of_codes(y & 0xffffu), va[3] = half2_of_codes(y >> 16);
          } else {
            va[0] = __byte_perm(v[q][0][u].w[mt], v[q][1][u].w[mt], 0x5410);
            va[1] = __byte_perm(v[q][0][u].w[mt], v[q][1][u].w[mt], 0x7632);
            va[2] = __byte_perm(v[q][2][u].w[mt], v[q][3][u].w[mt], 0x5410);
            va[3] = __byte_perm(v[q][2][u].w[mt], v[q][3][u].w[mt], 0x7632);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int part = C::PP - 1; part >= 0; --part)
              mma16816<F8>(o[t][u * (C::VC / 2) + mt], va[0], va[1], va[2], va[3], pb[part][t][0], pb[part][t][1]);
        }
    };

    // A NaN among the accumulators may come from a row that meets a token it does not see (0 * NaN or 0 * infinity), or
    // from an infinite value meeting the parts of a split probability.  The part is then walked again with the second
    // product done token by token, each row taking only what it sees.
    bool careful = false;
    for (;;) {
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int c = 0; c < 2; ++c) m[t][c] = -INFINITY, l[t][c] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][s][i] = 0.f;
      }
      locate(t0, row_of);
      load_k(t0, row_of);
      load_v(t0, row_of);
      locate(t0 + 1, next_row);
      for (int tile = t0; tile < t1; ++tile) {
        // ---- S^T = K Q^T
        float s[GPI][NT][4];
#pragma unroll
        for (int q = 0; q < GPI; ++q)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[q][t][i] = 0.f;
#pragma unroll
        for (int u = 0; u < C::KL; ++u)
#pragma unroll
          for (int st = 0; st < C::KC / 4; ++st) {
            uint32_t ka[GPI][4];
#pragma unroll
            for (int q = 0; q < GPI; ++q) {
              if constexpr (F8) {
                ka[q][0] = half2_of_codes(k[q][0][u].w[st] & 0xffffu), ka[q][2] = half2_of_codes(k[q][0][u].w[st] >> 16);
                ka[q][1] = half2_of_codes(k[q][1][u].w[st] & 0xffffu), ka[q][3] = half2_of_codes(k[q][1][u].w[st] >> 16);
              } else {
                ka[q][0] = k[q][0][u].w[2 * st], ka[q][2] = k[q][0][u].w[2 * st + 1];
                ka[q][1] = k[q][1][u].w[2 * st], ka[q][3] = k[q][1][u].w[2 * st + 1];
              }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int part = C::QP - 1; part >= 0; --part) {
                const uint2 qb = qs[part][t][u * (C::KC / 4) + st][lane];
#pragma unroll
                for (int q = 0; q < GPI; ++q)
                  mma16816<F8>(s[q][t], ka[q][0], ka[q][1], ka[q][2], ka[q][3], qb.x, qb.y);
              }
          }
        float ksn[GPI][2], vsn[GPI][2];
        if constexpr (F8) {
#pragma unroll
          for (int q = 0; q < GPI; ++q)
#pragma unroll
            for (int i = 0; i < 2; ++i) ksn[q][i] = ks[q][i], vsn[q][i] = vs[q][i];
        }
        int64_t this_row[GPI];
#pragma unroll
        for (int q = 0; q < GPI; ++q) this_row[q] = row_of[q], row_of[q] = next_row[q];
        load_k(tile + 1, row_of);
        locate(tile + 2, next_row);

        // ---- scores in powers of two; unseen ones are -infinity
        float top[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) top[t][0] = top[t][1] = -INFINITY;
        bool partly[GPI];
#pragma unroll
        for (int q = 0; q < GPI; ++q) {
          const int64_t tok0 = (int64_t)span.start + ((int64_t)(tile * PA_WARPS + warp) * GPI + q) * 16;
          const bool none = this_row[q] < 0;
          partly[q] = none || tok0 + 15 > all_to || tok0 < all_from;
          float lift[2] = {0.f, 0.f};  // about log2 of the value scale
          if constexpr (F8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) lift[i] = (float)((int)(__float_as_uint(vsn[q][i]) >> 23) - 126);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x = s[q][t][i] * f[t][i & 1];
              if constexpr (F8) x *= ksn[q][i >> 1];
              if (a.softcap > 0.f) x = a.softcap * PA_LOG2E * tanhf(x / a.softcap);
              if (partly[q]) {
                const int64_t tok = tok0 + n + 8 * (i >> 1);
                const bool seen = !none && tok <= last[t][i & 1] && tok > (int64_t)last[t][i & 1] - window;
                x = seen ? x : -INFINITY;
              }
              s[q][t][i] = x;
              top[t][i & 1] = fmaxf(top[t][i & 1], F8 ? x + lift[i >> 1] : x);
            }
        }
        // ---- the reference moves only when a score is far above it (always on the first seen token)
        bool move = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) move |= top[t][c] > m[t][c] + PA_SLACK;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float x = top[t][c];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              const float mn = fmaxf(m[t][c], x);
              const float by = m[t][c] == mn ? 1.f : ex2(m[t][c] - mn);  // 0 from -infinity
              m[t][c] = mn;
              l[t][c] *= by;
#pragma unroll
              for (int st = 0; st < KS; ++st) o[t][st][c] *= by, o[t][st][c + 2] *= by;
            }
        }
        // ---- probabilities, their sum, and O^T += V^T P^T
#pragma unroll
        for (int q = 0; q < GPI; ++q) {
          float pr[NT][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float mr = m[t][i & 1] == -INFINITY ? 0.f : m[t][i & 1];
              const float e = ex2(s[q][t][i] - mr);
              l[t][i & 1] += e;
              pr[t][i] = F8 ? e * vsn[q][i >> 1] : e;
            }
          if (!careful) {
            add_pv(q, pr);
          } else {
            // token by token from memory, each row taking only what it sees; the probabilities rounded as above
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; i += 2) {
                float r0 = pr[t][i], r1 = pr[t][i + 1];
#pragma unroll
                for (int part = 0; part < C::PP; ++part) split_pair<F8>(r0, r1);
                pr[t][i] -= r0, pr[t][i + 1] -= r1;
              }
            const int64_t tok0 = (int64_t)span.start + ((int64_t)(tile * PA_WARPS + warp) * GPI + q) * 16;
            const int cnt = this_row[q] < 0 ? 0 : count(tile, q);
#pragma unroll 1
            for (int tk = 0; tk < cnt; ++tk) {
              float pt[NT][2];
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  pt[t][c] = __shfl_sync(0xffffffffu, tk < 8 ? pr[t][c] : pr[t][2 + c], (tk & 7) * 4 + j);
                  const int64_t tok = tok0 + tk;
                  if (!(tok <= last[t][c] && tok > (int64_t)last[t][c] - window)) pt[t][c] = -1.f;  // not seen
                }
#pragma unroll
              for (int u = 0; u < C::VL; ++u)
#pragma unroll
                for (int i = 0; i < C::VC; ++i) {
                  const int64_t e = (this_row[q] + tk) * D + (u * 8 + n) * C::VC + i;
                  float x;
                  if constexpr (F8) {
                    const uint32_t h2 = half2_of_codes(static_cast<const uint8_t*>(a.c.v_pages)[e]);
                    x = __half2float(__ushort_as_half((uint16_t)h2));
                  } else {
                    x = to_f32(static_cast<const bf16*>(a.c.v_pages)[e]);
                  }
#pragma unroll
                  for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                      if (!(pt[t][c] < 0.f)) o[t][u * (C::VC / 2) + i / 2][c + 2 * (i & 1)] += pt[t][c] * x;
                }
            }
          }
        }
        load_v(tile + 1, row_of);
      }
      bool nan = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) nan |= isnan(o[t][s][i]);
      if (careful || !__any_sync(0xffffffffu, nan)) break;
      careful = true;
    }

    // ---- join the four warps
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[t][c];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (m[t][c] == -INFINITY && !(x == 0.f)) m[t][c] = 0.f;  // nothing but NaN scores: let them through
        if (n == 0) red_l[warp][t * 8 + 2 * j + c] = x, red_m[warp][t * 8 + 2 * j + c] = m[t][c];
      }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < PA_WARPS; ++w) {
      if (warp == w) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int r = t * 8 + 2 * j + c;
            const float mt = fmaxf(fmaxf(red_m[0][r], red_m[1][r]), fmaxf(red_m[2][r], red_m[3][r]));
            const float by = m[t][c] == -INFINITY ? 0.f : ex2(m[t][c] - mt);
#pragma unroll
            for (int u = 0; u < C::VL; ++u)
#pragma unroll
              for (int mt2 = 0; mt2 < C::VC / 2; ++mt2)
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                  const int ch = (u * 8 + n) * C::VC + 2 * mt2 + hh;
                  const float x = m[t][c] == -INFINITY ? 0.f : o[t][u * (C::VC / 2) + mt2][c + 2 * hh] * by;
                  red[r][ch] = w == 0 ? x : red[r][ch] + x;
                }
          }
      }
      __syncthreads();
    }
    const bool whole = t0 == 0 && t1 == span.tiles;
    const int slot = t0 == 0 ? 1 : 0;  // 1: this part starts its unit
    for (int e = tid; e < RB * D; e += PA_NT) {
      const int r = e / D, c = e - r * D, row = row0 + r;
      float mt = -INFINITY, lt = 0.f;
#pragma unroll
      for (int w = 0; w < PA_WARPS; ++w) mt = fmaxf(mt, red_m[w][r]);
#pragma unroll
      for (int w = 0; w < PA_WARPS; ++w) lt += red_m[w][r] == -INFINITY ? 0.f : red_l[w][r] * ex2(red_m[w][r] - mt);
      if (whole) {
        if (row < p.rows) {
          const int w = row / p.G, g = row - w * p.G;
          const int64_t head = ((int64_t)b * a.W + w) * a.Hq + (int64_t)h * p.G + g;
          const float x = mt == -INFINITY ? 0.f : red[r][c] / lt;
          if (a.out_bf16) static_cast<bf16*>(a.out)[head * D + c] = __float2bfloat16_rn(x);
          else static_cast<float*>(a.out)[head * D + c] = x;
          if (c == 0 && a.lse) a.lse[head] = mt == -INFINITY ? -INFINITY : (mt + log2f(lt)) * PA_LN2;
        }
      } else {
        const int64_t base = ((int64_t)blockIdx.x * 2 + slot) * RB + r;
        p.part_o[base * D + c] = red[r][c];
        if (c == 0) p.part_ml[base * 2] = mt, p.part_ml[base * 2 + 1] = lt;
      }
    }
    if (whole) rows_done += min(RB, p.rows - row0);
    if (t0 == 0 && !whole) {
      // the unit goes on in the following CTAs; its last tile is in the CTA whose share holds it
      meta.unit = (b * Hkv + h) * p.blocks + rb;
      int64_t e = (unit_end - 1) * ctas / total;  // share boundaries are floors: at most one off
      while (e * total / ctas > unit_end - 1) --e;
      while ((e + 1) * total / ctas <= unit_end - 1) ++e;
      meta.end_cta = (int)e;
    }
    at = first_of_b + (int64_t)in_b * span.tiles + t1;
    if (in_b == per_b - 1 && t1 == span.tiles) {
      first_of_b = at;
      ++b;
    }
  }
  if (tid == 0) {
    p.meta[blockIdx.x] = meta;
    add_work(a.status, rows_done);
  }
}

// ---------------------------------------------------------------- join

// CTA (x, y) joins query rows y of the unit that main CTA x starts and others go on with: the parts' maxima and sums
// first, then their accumulators in CTA order.
template <int D, int RB>
__global__ void __launch_bounds__(128) paged_attention_join_kernel(const PagedAttnArgs a, const PaPlan p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const PaMeta meta = p.meta[blockIdx.x];
  if (meta.unit < 0) return;
  const int rb = meta.unit % p.blocks, bh = meta.unit / p.blocks, h = bh % a.c.Hkv, b = bh / a.c.Hkv;
  constexpr int ROWS = 128 / D;  // rows of a CTA
  const int r = blockIdx.y * ROWS + threadIdx.x / D, c = threadIdx.x % D, row = rb * RB + r;
  if (row >= p.rows) return;
  const int x0 = blockIdx.x, x1 = meta.end_cta;
  auto at = [&](int x) { return ((int64_t)x * 2 + (x == x0 ? 1 : 0)) * RB + r; };
  float m = -INFINITY;
  for (int x = x0; x <= x1; ++x) m = fmaxf(m, p.part_ml[at(x) * 2]);
  float l = 0.f, o = 0.f;
  if (m != -INFINITY) {
#pragma unroll 4
    for (int x = x0; x <= x1; ++x) {
      const float2 ml = *reinterpret_cast<const float2*>(p.part_ml + at(x) * 2);
      const float v = p.part_o[at(x) * D + c];
      const float by = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
      l += ml.y * by;
      o += v * by;
    }
    o /= l;
  }
  const int w = row / p.G, g = row - w * p.G;
  const int64_t head = ((int64_t)b * a.W + w) * a.Hq + (int64_t)h * p.G + g;
  if (a.out_bf16) static_cast<bf16*>(a.out)[head * D + c] = __float2bfloat16_rn(o);
  else static_cast<float*>(a.out)[head * D + c] = o;
  if (c == 0) {
    if (a.lse) a.lse[head] = m == -INFINITY ? -INFINITY : (m + log2f(l)) * PA_LN2;
    add_work(a.status, 1);
  }
}

// ---------------------------------------------------------------- launch

template <int D, bool F8, int NT, bool FINE>
cudaError_t pa_launch(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  using C = PaCfg<D, F8, NT, FINE>;
  static int resident = 0;  // CTAs of this kernel per SM
  if (!resident) {
    int n = 0;
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, paged_attention_kernel<D, F8, NT, FINE>,
                                                                        PA_NT, 0);
    if (e != cudaSuccess) return e;
    resident = n < 1 ? 1 : n > 4 ? 4 : n;
  }
  // no more CTAs than tiles the longest possible lengths could give
  const int64_t most = (int64_t)a.B * a.c.Hkv * p.blocks * (((int64_t)a.max_pages * a.c.page_size) / C::TILE + 1);
  int64_t ctas = (int64_t)resident * sms;
  if (ctas > PA_MAX_CTAS) ctas = PA_MAX_CTAS;
  if (ctas > most) ctas = most;
  paged_attention_kernel<D, F8, NT, FINE><<<(unsigned)ctas, PA_NT, 0, s>>>(a, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  constexpr int ROWS = 128 / D;
  return launch_pdl(paged_attention_join_kernel<D, C::RB>, dim3((unsigned)ctas, (C::RB + ROWS - 1) / ROWS), dim3(128), 0,
                    s, a, p);
}

template <int D, bool F8, bool FINE>
cudaError_t pa_rows(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  switch (pa_nt(p.rows)) {
    case 1: return pa_launch<D, F8, 1, FINE>(a, p, sms, s);
    case 2: return pa_launch<D, F8, 2, FINE>(a, p, sms, s);
    default: return pa_launch<D, F8, 4, FINE>(a, p, sms, s);
  }
}

template <bool F8, bool FINE>
cudaError_t pa_heads(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  switch (a.c.d) {
    case 16: return pa_rows<16, F8, FINE>(a, p, sms, s);
    case 32: return pa_rows<32, F8, FINE>(a, p, sms, s);
    case 64: return pa_rows<64, F8, FINE>(a, p, sms, s);
    default: return pa_rows<128, F8, FINE>(a, p, sms, s);
  }
}

// One translation unit each: paged_attention_{bf16,e4m3}{,_fine}.cu
cudaError_t pa_bf16(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s);
cudaError_t pa_bf16_fine(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s);
cudaError_t pa_e4m3(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s);
cudaError_t pa_e4m3_fine(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s);

}  // namespace kda
