// Attention of the newest tokens of each request over its paged key/value cache.
//
// Per query row (a query head of one window token), over the positions it sees, with x = scale q.k (capped:
// cap tanh(x / cap)):  out = sum exp(x - m) v / sum exp(x - m),  lse = m + log sum exp(x - m).
//
// Bound by HBM: a cached row of d channels feeds the few query rows of its head group (Hq / Hkv heads x W tokens), so each K
// or V element is used for 2 multiplications per query row.  It is read once per block of query rows: once where they are
// up to RB (8, 16 or 32; 16 at most with fp32 queries or outputs), three times for 96 bf16 rows, six times for 96 fp32 ones.
//
// Work.  A unit is one request, key/value head and block of RB = 8 NT query rows.  All units' caches, cut into tiles
// of TILE tokens, form one line; the warps take equal consecutive shares of it, so ragged lengths balance without
// the host knowing them, and a single long request spreads over the whole GPU.  A unit counts PA_UNIT_COST tiles more
// than it has, for its queries, first loads and output.  A warp that has a whole unit writes its output; the parts of a
// unit cut across warps go to the workspace (each warp has at most one part that continues a unit and one that
// starts one) and a second, small kernel joins them in order.  Warps never wait on one another after the share-out:
// the other warps of the SM cover one's latencies.  256 requests of 65 to 8191 tokens, 12 heads over 4: 96.5 us with e4m3 (4.8
// TB/s, 70 % of the copy rate: latency of dependent instructions at 12 warps per SM), 142 us with bf16 (92 %); with fp32
// queries and outputs 110 and 145 us; at d = 64 69 and 87 us (51 and 75 %: twice the rows for the same bytes).
//
// K and V go from global memory straight into the operand registers of mma.m16n8k16 (no transposes, no shared memory
// for them): the products are S^T = K Q^T and O^T = V^T P^T with the tokens resp. channels as the 16-row side and 8
// query rows as columns.  The channel order inside a product's K steps is free as long as Q follows it, so a lane's
// operands for consecutive steps are one 16-byte piece of its token's row; V's pairs of tokens are put together from two
// such pieces by byte permutes.  The 5th-generation tensor instructions take both operands from shared or tensor memory, where a
// bf16 cache comes by TMA as it lies: that is paged_attention_tc.cu, for few units, and paged_attention_rows.cu, for
// many query rows.  This form has all other calls: e4m3 codes need a pass through registers to become an operand, which
// this form makes of the operand's own load, and units that are many and short would pay those forms' starts and ends.
//
// e4m3 caches: codes become fp16 (exact), q is scaled per row by a power of two into fp16's range (exact for bf16 q
// down to 2^-31 of the row's maximum), the key's scale multiplies the score and the value's scale the
// probability.  The running reference of the softmax is then the maximum of x + log2(value scale), so that the
// scaled probabilities fit fp16 for any scales.  A value of zeros says nothing by its scale (1 in a row that kda_kv_write
// wrote): it counts with the least, and its probability, which multiplies zeros, is taken as 0 in the product.  Codes
// are looked at for that only when the reference moves, so it costs nothing else (256 ragged requests: 96 us with and without).
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
constexpr int PA_UNIT_COST = 2;
constexpr int PA_SHARE = 2;  // positions on the line that a warp takes at least
constexpr int PA_MAX_LEN = 0x7fffff00;  // token positions and the next tile's stay within 32 bits
constexpr float PA_LOG2E = 1.4426950408889634f, PA_LN2 = 0.6931471805599453f;
// How far (in powers of two) scores may run above the softmax reference before it is moved, and how far above it the largest
// lies when it has moved.  fp16 probabilities use that type's range: up to 2^15 (the value scale's rounding to `lift` included),
// so that they keep all their bits down to 2^-14 and are lost below 2^-25 only, 2^-34 of the largest.  fp32 calls move at
// less, for which the second part reaches to 2^-39: below fp32's own bits over a quarter of a million tokens.
constexpr float pa_head(bool f8, bool fine) { return f8 ? fine ? 14.f : 9.f : 0.f; }
constexpr float pa_slack(bool f8) { return f8 ? 15.f : 6.f; }
// The lift of the least value scale, 2^-63; where nothing else counts, the sum's terms are then up to 2^62 (and the rounding of such
// exponents, 2^-18, shows in the log-sum-exp as 1e-6).
constexpr float PA_LEAST_LIFT = -62.f;

// What the main kernel leaves for the join, per warp.
struct PaMeta {
  int unit;  // the unit whose first part is this warp's last, -1 if none
  int end;   // the warp with that unit's last part
};

// 8-row column blocks of a unit, and the CTAs per SM its kernel is built for
__host__ __device__ constexpr int pa_nt(int rows, bool fine) { return rows <= 8 ? 1 : rows <= 16 || fine ? 2 : 4; }
__host__ __device__ constexpr int pa_resident(int nt) { return nt == 1 ? 3 : 2; }
constexpr int PA_SMS = 152;

struct PaPlan {  // derived on the host
  int G;         // query heads per key/value head
  int rows;      // query rows per key/value head: W * G
  int blocks;    // row blocks of RB per key/value head
  float* part_o;   // [warp][2][RB][D]
  float* part_ml;  // [warp][2][RB][2]
  PaMeta* meta;    // [warp]
  int workers;     // warps launched (entries of meta)
  bool stall;      // a test of the bounded waits (tensor-memory forms)
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
// v 2^d, d <= 0, where 2^d alone may be below fp32's range (ex2 gives 0 there) though the product is not: references that
// include a value scale lie up to 126 powers of two apart at equal scores.  For d >= -64 the second factor is 1.
__device__ __forceinline__ float times_pow2(float v, float d) {
  const float near = fmaxf(d, -64.f);
  return v * ex2(near) * ex2(d - near);
}
// ln(l 2^m): l's power of two goes to m first, so that what is rounded has the result's size (l itself is up to 2^71 where
// references lie that far below the scores).
__device__ __forceinline__ float log_sum(float m, float l) {
  const uint32_t b = __float_as_uint(l);
  const int e = (int)(b >> 23) - 127;
  if (e < -126 || e > 127) return (m + log2f(l)) * PA_LN2;  // 0, infinity, NaN
  return (m + (float)e + log2f(__uint_as_float((b & 0x7fffffu) | 0x3f800000u))) * PA_LN2;
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
  __device__ __forceinline__ uint32_t any() const {
    uint32_t x = w[0];
#pragma unroll
    for (int i = 1; i < (BYTES < 4 ? 1 : BYTES / 4); ++i) x |= w[i];
    return x;
  }
  // Read once: not kept in L1 (one request of 262144 tokens, bf16: 172 to 174 us against 175 to 177).
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

// cap2 * tanh(y) given z = 2 log2(e) y, with cap2 = cap * log2(e).  Where all of a warp's |y| are up to 0.75 (|z| <= PA_NEAR) it is y
// times a polynomial in y^2 for tanh(y) / y (a weighted least-squares fit that levels the relative error, 1.3e-7 in fp32):
// no cancellation for small scores, and no use of the exponential's unit, which the exponentials fill already (256 ragged
// requests, e4m3 cache, cap 30: 103 us without it, 101 with).  Else 1 - 2 / (1 + 2^z), within 1.2e-7 absolutely, and below |y| = 0.15
// the odd series to y^7 (next term 6e-9 relatively there): 8e-7 relatively at worst.  fp32 calls take CUDA's tanhf.
constexpr float PA_NEAR = 1.5f * PA_LOG2E;
__host__ __device__ constexpr float pa_tanh(int i) {
  constexpr float c[6] = {1.f, -0.333329588f, 0.133254066f, -0.0533444285f, 0.0195829086f, -0.0047162571f};
  return c[i];
}
__device__ __forceinline__ float capped_near(float z, float cap2) {
  const float y = z * (0.5f * PA_LN2), u = y * y;
  float t = pa_tanh(5);
#pragma unroll
  for (int i = 4; i >= 0; --i) t = fmaf(t, u, pa_tanh(i));
  return cap2 * y * t;
}
__device__ __forceinline__ float capped(float z, float cap2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(z)));
  const float y = z * (0.5f * PA_LN2), u = y * y;
  const float small = cap2 * y * fmaf(u, fmaf(u, fmaf(u, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  return fabsf(z) < 0.3f * PA_LOG2E ? small : fmaf(-2.f * cap2, r, cap2);
}

// ---------------------------------------------------------------- the line of tiles

// Tokens a request's window sees: first seen position rounded down to `align` (a power of two that divides the page),
// and the tiles from there to its length.
struct PaSpan {
  int len, start, tiles;
};
template <int TILE>
__device__ __forceinline__ PaSpan pa_span(const PagedAttnArgs& a, int b, bool flag, int align = 16) {
  PaSpan s;
  s.len = __ldg(a.seq_lens + b);
  if (s.len < 0 || s.len > (int64_t)a.max_pages * a.c.page_size || s.len > PA_MAX_LEN) {
    if (flag) flag_status(a.status, KDA_DEV_SEQ_OOB);
    s.len = 0;
  }
  if (a.c.num_pages == 0 && s.len > 0) {
    if (flag) flag_status(a.status, KDA_DEV_PAGE_OOB);
    s.len = 0;
  }
  int64_t first = a.window > 0 ? (int64_t)s.len - a.W - a.window + 1 : 0;  // of the window's first query
  if (first < 0) first = 0;
  s.start = (int)first & -align;
  const int64_t n = (int64_t)s.len - s.start;
  s.tiles = n > 0 ? (int)((n + TILE - 1) / TILE) : 1;  // a unit with nothing to see still writes its rows
  return s;
}

// Sum of `mine` over the threads up to this one, and over all; `sums`: one place per warp.
template <int NT>
__device__ __forceinline__ int64_t block_scan(int64_t mine, int64_t* sums, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) sums[warp] = x;
  __syncthreads();
  total = 0;
  int64_t before = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    if (w == warp) before = total;
    total += sums[w];
  }
  return x + before;
}

// ---------------------------------------------------------------- main kernel

template <int D, bool F8, int NT, bool FINE>
struct PaCfg {
  static constexpr int ES = F8 ? 1 : 2;
  static constexpr int RS = D * ES;                      // bytes of a cached row
  static constexpr int RB = 8 * NT;
  static constexpr int GPI = F8 && NT < 4 ? 2 : 1;          // 16-token groups a warp works on at once
  static constexpr int TILE = 16 * GPI;                  // tokens
  static constexpr int KC = D / 4 < 16 / ES ? D / 4 : 16 / ES;  // channels of a key piece
  static constexpr int KL = D / (4 * KC);                // key pieces per lane and token
  static constexpr int VC = D / 8 < 16 / ES ? D / 8 : 16 / ES;  // channels of a value piece
  static constexpr int VL = D / (8 * VC);
  static constexpr int KS = D / 16;                      // K steps of the first product, 16-channel tiles of the second
  static constexpr int QP = FINE ? (F8 ? 2 : 3) : 1;     // 16-bit parts of a query
  static constexpr int PP = FINE ? (F8 ? 2 : 3) : (F8 ? 1 : 2);  // and of a probability
  static constexpr size_t SMEM = sizeof(uint2) * QP * NT * KS * 32 * PA_WARPS;
};

template <int D, bool F8, int NT, bool FINE>
__global__ void __launch_bounds__(PA_NT, pa_resident(NT)) paged_attention_kernel(const PagedAttnArgs a,
                                                                                 const PaPlan p) {
  using C = PaCfg<D, F8, NT, FINE>;
  constexpr int RB = C::RB, TILE = C::TILE, GPI = C::GPI, KS = C::KS;
  extern __shared__ uint2 q_operands[];  // [warp][part][NT][KS][lane]: Q as the first product takes it
  __shared__ int64_t sums[PA_WARPS];
  __shared__ int64_t where[PA_WARPS][2];
  pdl_begin();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = lane >> 2, j = lane & 3;
  const int Hkv = a.c.Hkv, per_b = Hkv * p.blocks;  // units per request
  uint2* qs = q_operands + warp * (C::QP * NT * KS * 32) + lane;

  // ---- the warps' shares of the line: each thread adds up the cost of a run of requests, then the sums are scanned
  const int run = (a.B + PA_NT - 1) / PA_NT;
  int64_t mine = 0;
  for (int b = tid * run; b < min(a.B, (tid + 1) * run); ++b)
    mine += pa_span<TILE>(a, b, blockIdx.x == 0).tiles + PA_UNIT_COST;
  int64_t total;
  const int64_t upto = block_scan<PA_NT>(mine, sums, total);
  total *= per_b;
  const int64_t all = (int64_t)gridDim.x * PA_WARPS, few = (total + PA_SHARE - 1) / PA_SHARE;
  const int64_t workers = few < all ? few : all;
  // the request in which each of this CTA's shares begins, and that request's first position
  const int64_t before = upto - mine;
  for (int w = 0; w < PA_WARPS; ++w) {
    const int64_t x = (int64_t)blockIdx.x * PA_WARPS + w, from = x * total / workers;
    if (x >= workers || from < before * per_b || from >= upto * per_b) continue;
    int64_t f = before;
    for (int b = tid * run;; ++b) {
      const int t = pa_span<TILE>(a, b, false).tiles + PA_UNIT_COST;
      if (from < (f + t) * per_b) {
        where[w][0] = b;
        where[w][1] = f * per_b;
        break;
      }
      f += t;
    }
  }
  __syncthreads();
  const int64_t me = (int64_t)blockIdx.x * PA_WARPS + warp;
  PaMeta meta{-1, 0};
  if (me >= workers) {
    if (lane == 0) p.meta[me] = meta;
    return;
  }
  int64_t at = me * total / workers;
  const int64_t end = (me + 1) * total / workers;
  int b = (int)where[warp][0];
  int64_t first_of_b = where[warp][1];
  int rows_done = 0;
  const int window = a.window > 0 ? a.window : 0x7fffffff;
  const float cap2 = a.softcap * PA_LOG2E;

  while (at < end) {
    const PaSpan span = pa_span<TILE>(a, b, false);
    const int cost = span.tiles + PA_UNIT_COST;
    const int in_b = (int)((at - first_of_b) / cost);  // unit within the request
    const int64_t unit_first = first_of_b + (int64_t)in_b * cost, unit_end = unit_first + cost;
    // the unit's overhead comes first on the line: a share that ends within it has no tile of the unit
    const int t0 = max(0, (int)(at - unit_first) - PA_UNIT_COST);
    const int t1 = (int)((end < unit_end ? end : unit_end) - unit_first) - PA_UNIT_COST;
    const int h = in_b / p.blocks, rb = in_b - h * p.blocks;
    const int this_b = b;
    at = end < unit_end ? end : unit_end;
    if (in_b == per_b - 1 && at == unit_end) {
      first_of_b = at;
      ++b;
    }
    if (t1 <= t0) continue;
    const int row0 = rb * RB;

    // ---- where the part's tokens are: a cursor over its 16-token groups, the next page's id asked for ahead
    const int32_t* table = a.block_table + (int64_t)this_b * a.max_pages;
    int tok_next = span.start + t0 * TILE;  // of the next group to place
    const int tok_end = (int)min((int64_t)span.len, (int64_t)span.start + (int64_t)t1 * TILE);
    int page_at = tok_next / a.c.page_size, off = tok_next - page_at * a.c.page_size;
    const int page_last = span.len > 0 ? (span.len - 1) / a.c.page_size : -1;
    int page = page_at <= page_last ? __ldg(table + page_at) : -1;
    int page_next = page_at < page_last ? __ldg(table + page_at + 1) : -1;
    // Places the next group: its first token's cache row, -1 where there is nothing to read.
    auto place = [&]() -> int64_t {
      int64_t row = -1;
      if (tok_next < tok_end) {
        if ((unsigned)page < (unsigned)a.c.num_pages) row = ((int64_t)page * Hkv + h) * a.c.page_size + off;
        else if (lane == 0) flag_status(a.status, KDA_DEV_PAGE_OOB);
      }
      tok_next = min(tok_next, 0x7fffffff - 64) + 16;
      off += 16;
      if (off == a.c.page_size) {
        off = 0;
        ++page_at;
        page = page_next;
        page_next = page_at < page_last ? __ldg(table + page_at + 1) : -1;
      }
      return row;
    };
    const int page_at0 = page_at, off0 = off, page0 = page, page_next0 = page_next;  // to walk again

    // ---- queries of the unit in the first product's operand order: row n of each column block, this lane's pieces
    float f[NT][2];   // per query row of this lane's results: score in powers of two (or the cap's argument) per unit of the product
    int last[NT][2];  // and its last seen position
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int row = row0 + t * 8 + n, w = row / p.G, g = row - w * p.G;
      const int64_t base = (((int64_t)this_b * a.W + w) * a.Hq + (int64_t)h * p.G + g) * D + j * C::KC;
      float x[C::KL][C::KC];
      float amax = 0.f;
#pragma unroll
      for (int u = 0; u < C::KL; ++u)
#pragma unroll
        for (int c = 0; c < C::KC; c += 4) {
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          if (row < p.rows) {
            const int64_t e = base + u * 4 * C::KC + c;
            if (a.q_bf16) {
              const uint2 r = __ldg(reinterpret_cast<const uint2*>(static_cast<const bf16*>(a.q) + e));
              v = make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                              __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
            } else {
              v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + e));
            }
          }
          x[u][c] = v.x, x[u][c + 1] = v.y, x[u][c + 2] = v.z, x[u][c + 3] = v.w;
          amax = fmaxf(amax, fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))));
        }
      float up = 1.f, down = 1.f;
      if constexpr (F8) {  // the row's maximum to [2^14, 2^15)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        int e = amax > 0.f ? 14 - ((int)(__float_as_uint(amax) >> 23) - 127) : 0;
        e = min(100, e);  // -114 at least
        up = __uint_as_float((uint32_t)(e + 127) << 23);
        down = __uint_as_float((uint32_t)(127 - e) << 23);
      }
#pragma unroll
      for (int u = 0; u < C::KL; ++u)
#pragma unroll
        for (int c = 0; c < C::KC; c += 4) {
          float v0 = x[u][c] * up, v1 = x[u][c + 1] * up, v2 = x[u][c + 2] * up, v3 = x[u][c + 3] * up;
#pragma unroll
          for (int part = 0; part < C::QP; ++part) {
            uint2 r;
            r.x = split_pair<F8>(v0, v1);
            r.y = split_pair<F8>(v2, v3);
            qs[((part * NT + t) * KS + u * (C::KC / 4) + c / 4) * 32] = r;
          }
        }
      const float own = down * a.scale * (a.softcap > 0.f ? (FINE ? 1.f : 2.f * PA_LOG2E) / a.softcap : PA_LOG2E);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        f[t][c] = __shfl_sync(0xffffffffu, own, (2 * j + c) * 4);
        const int r = row0 + t * 8 + 2 * j + c;
        last[t][c] = r < p.rows ? span.len - a.W + r / p.G : -1;
      }
    }
    // tokens every row of the unit sees: [all_from, all_to]
    const int all_to = span.len - a.W + row0 / p.G;
    const int64_t all_from = (int64_t)span.len - a.W + min(p.rows - 1, row0 + RB - 1) / p.G - window + 1;

    float m[NT][2], mu[NT][2], l[NT][2];  // softmax reference, the same with 0 for -infinity, sum
    float o[NT][KS][4];
    Piece<C::KC * C::ES> k[GPI][2][C::KL];
    Piece<C::VC * C::ES> v[GPI][4][C::VL];
    float ks[GPI][2], vs[GPI][2];

    // Loads of one group whose first token is tok0.  Past the request's end the last token is read again (unseen).
    auto load_k = [&](int q, int64_t row, int tok0) {
      if (row < 0) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int u = 0; u < C::KL; ++u) k[q][i][u].clear();
          ks[q][i] = vs[q][i] = 0.f;
        }
        return;
      }
      const int over = span.len - 1 - tok0;  // last token there is, within the group
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t r = row + min(n + 8 * i, over);
        const uint8_t* at_k = static_cast<const uint8_t*>(a.c.k_pages) + r * C::RS + j * (C::KC * C::ES);
#pragma unroll
        for (int u = 0; u < C::KL; ++u) k[q][i][u].load(at_k + u * (4 * C::KC * C::ES));
        if constexpr (F8) {
          ks[q][i] = __ldg(a.c.k_scales + r);
          vs[q][i] = __ldg(a.c.v_scales + r);
        }
      }
    };
    auto load_v = [&](int q, int64_t row, int tok0) {
      if (row < 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int u = 0; u < C::VL; ++u) v[q][i][u].clear();
        return;
      }
      const int over = span.len - 1 - tok0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t r = row + min(2 * j + (i & 1) + 8 * (i >> 1), over);
        const uint8_t* at_v = static_cast<const uint8_t*>(a.c.v_pages) + r * C::RS + n * (C::VC * C::ES);
#pragma unroll
        for (int u = 0; u < C::VL; ++u) v[q][i][u].load(at_v + u * (8 * C::VC * C::ES));
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
        for (int c = 0; c < 2; ++c) m[t][c] = -INFINITY, mu[t][c] = 0.f, l[t][c] = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[t][s][i] = 0.f;
      }
      int64_t row[GPI];
      int tok0 = span.start + t0 * TILE;  // of the tile's first group
      if (span.len > 0) {
#pragma unroll
        for (int q = 0; q < GPI; ++q) {
          row[q] = place();
          load_k(q, row[q], tok0 + 16 * q);
          load_v(q, row[q], tok0 + 16 * q);
        }
      }
      for (int tile = span.len > 0 ? t0 : t1; tile < t1; ++tile, tok0 += TILE) {
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
                ka[q][0] = half2_of_codes(k[q][0][u].w[st] & 0xffffu);
                ka[q][1] = half2_of_codes(k[q][1][u].w[st] & 0xffffu);
                ka[q][2] = half2_of_codes(k[q][0][u].w[st] >> 16);
                ka[q][3] = half2_of_codes(k[q][1][u].w[st] >> 16);
              } else {
                ka[q][0] = k[q][0][u].w[2 * st], ka[q][2] = k[q][0][u].w[2 * st + 1];
                ka[q][1] = k[q][1][u].w[2 * st], ka[q][3] = k[q][1][u].w[2 * st + 1];
              }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int part = C::QP - 1; part >= 0; --part) {
                const uint2 qb = qs[((part * NT + t) * KS + u * (C::KC / 4) + st) * 32];
#pragma unroll
                for (int q = 0; q < GPI; ++q)
                  mma16816<F8>(s[q][t], ka[q][0], ka[q][1], ka[q][2], ka[q][3], qb.x, qb.y);
              }
          }
        float ksn[GPI][2], vsn[GPI][2];
        int64_t this_row[GPI];
#pragma unroll
        for (int q = 0; q < GPI; ++q) {
          this_row[q] = row[q];
#pragma unroll
          for (int i = 0; i < 2; ++i) ksn[q][i] = F8 ? ks[q][i] : 1.f, vsn[q][i] = F8 ? vs[q][i] : 1.f;
          row[q] = place();
          load_k(q, row[q], tok0 + TILE + 16 * q);
        }

        // ---- scores in powers of two; unseen ones are -infinity
        float top[NT][2];
        float lift[GPI][2];  // about log2 of the value scale
#pragma unroll
        for (int t = 0; t < NT; ++t) top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
        for (int q = 0; q < GPI; ++q) {
          const int tq = tok0 + 16 * q;
          const bool none = this_row[q] < 0;
          const bool partly = none || tq > all_to - 15 || tq < all_from;
          if constexpr (F8) {
#pragma unroll
            for (int i = 0; i < 2; ++i) lift[q][i] = (float)((int)(__float_as_uint(vsn[q][i]) >> 23) - 126);
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x = s[q][t][i];
              if constexpr (F8) x *= ksn[q][i >> 1];  // first: a large query's factor and a small key's scale make up for one another
              s[q][t][i] = x * f[t][i & 1];
            }
          if (a.softcap > 0.f) {
            bool near = !FINE;  // all of them, as scores mostly are
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) near = near && fabsf(s[q][t][i]) <= PA_NEAR;
            if (__all_sync(0xffffffffu, near)) {
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[q][t][i] = capped_near(s[q][t][i], cap2);
            } else {
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) s[q][t][i] = FINE ? cap2 * tanhf(s[q][t][i]) : capped(s[q][t][i], cap2);
            }
          }
          if (partly) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int tok = tq + n + 8 * (i >> 1);
                const bool seen = !none && tok <= last[t][i & 1] && tok > (int64_t)last[t][i & 1] - window;
                s[q][t][i] = seen ? s[q][t][i] : -INFINITY;
              }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              top[t][i & 1] = fmaxf(top[t][i & 1], F8 ? s[q][t][i] + lift[q][i >> 1] : s[q][t][i]);
        }
        // ---- the reference moves only when a score is far above it (always on the first seen token)
        bool move = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int c = 0; c < 2; ++c) move |= top[t][c] > m[t][c] + pa_slack(F8);
        if (__any_sync(0xffffffffu, move)) {
          if constexpr (F8) {
            // a value of zeros has a scale all the same: it adds nothing, and lifts the reference as the least scale does
            bool zeros = false;
#pragma unroll
            for (int q = 0; q < GPI; ++q) {
              uint32_t other[4];  // bit n' 4 + j': lane's piece of token 2 j' + (i & 1) + 8 (i >> 1) has a nonzero code
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t any = 0;
#pragma unroll
                for (int u = 0; u < C::VL; ++u) any |= v[q][i][u].any();
                other[i] = __ballot_sync(0xffffffffu, any & 0x7f7f7f7fu);
              }
#pragma unroll
              for (int i = 0; i < 2; ++i) {  // this lane's tokens n and n + 8
                const uint32_t of = (n & 1 ? other[2 * i + 1] : other[2 * i]) >> (n >> 1) & 0x11111111u;
                if (of == 0) lift[q][i] = PA_LEAST_LIFT + pa_head(F8, FINE), vsn[q][i] = 0.f, zeros = true;
              }
            }
            if (__any_sync(0xffffffffu, zeros)) {
#pragma unroll
              for (int t = 0; t < NT; ++t) top[t][0] = top[t][1] = -INFINITY;
#pragma unroll
              for (int q = 0; q < GPI; ++q)
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                  for (int i = 0; i < 4; ++i) top[t][i & 1] = fmaxf(top[t][i & 1], s[q][t][i] + lift[q][i >> 1]);
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float x = top[t][c];
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
              const float mn = fmaxf(m[t][c], x - pa_head(F8, FINE));
              const float down = m[t][c] == mn ? 0.f : m[t][c] - mn, by = ex2(down);  // 0 from -infinity
              m[t][c] = mn;
              mu[t][c] = mn == -INFINITY ? 0.f : mn;
              l[t][c] = F8 ? times_pow2(l[t][c], down) : l[t][c] * by;
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
              const float e = ex2(s[q][t][i] - mu[t][i & 1]);
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
            const int tq = tok0 + 16 * q;
            const int cnt = this_row[q] < 0 ? 0 : min(16, span.len - tq);
#pragma unroll 1
            for (int tk = 0; tk < cnt; ++tk) {
              float pt[NT][2];
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                  pt[t][c] = __shfl_sync(0xffffffffu, tk < 8 ? pr[t][c] : pr[t][2 + c], (tk & 7) * 4 + j);
                  const int tok = tq + tk;
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
          load_v(q, row[q], tok0 + TILE + 16 * q);
        }
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
      tok_next = span.start + t0 * TILE;
      page_at = page_at0, off = off0, page = page0, page_next = page_next0;
    }

    // ---- the part's sums, and its rows: this lane has channels (8 u + n) VC .. of rows 2j and 2j + 1 of each block
    const bool whole = t0 == 0 && t1 == span.tiles;
    const int64_t part = (me * 2 + (t0 == 0 ? 1 : 0)) * RB;  // second place: the part that starts its unit
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = l[t][c];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        if (m[t][c] == -INFINITY && !(x == 0.f)) m[t][c] = 0.f;  // nothing but NaN scores: let them through
        const bool none = m[t][c] == -INFINITY;
        const int r = t * 8 + 2 * j + c, qrow = row0 + r;
        const float by = whole ? (none ? 0.f : 1.f / x) : 1.f;
        if (whole && qrow >= p.rows) continue;
        const int w = qrow / p.G, g = qrow - w * p.G;
        const int64_t head = ((int64_t)this_b * a.W + w) * a.Hq + (int64_t)h * p.G + g;
#pragma unroll
        for (int u = 0; u < C::VL; ++u) {
          float y[C::VC];
#pragma unroll
          for (int i = 0; i < C::VC; ++i) y[i] = o[t][u * (C::VC / 2) + i / 2][c + 2 * (i & 1)] * by;
          const int ch = (u * 8 + n) * C::VC;
          if (whole && a.out_bf16) {
            bf16* out = static_cast<bf16*>(a.out) + head * D + ch;
#pragma unroll
            for (int i = 0; i < C::VC; i += 2) {
              const __nv_bfloat162 z = __floats2bfloat162_rn(y[i], y[i + 1]);
              reinterpret_cast<__nv_bfloat162*>(out)[i / 2] = z;
            }
          } else {
            float* out = whole ? static_cast<float*>(a.out) + head * D + ch : p.part_o + (part + r) * D + ch;
#pragma unroll
            for (int i = 0; i < C::VC; i += 2) reinterpret_cast<float2*>(out)[i / 2] = make_float2(y[i], y[i + 1]);
          }
        }
        if (n == 0) {
          if (!whole) *reinterpret_cast<float2*>(p.part_ml + (part + r) * 2) = make_float2(m[t][c], x);
          else if (a.lse) a.lse[head] = none ? -INFINITY : log_sum(m[t][c], x);
        }
      }
    if (whole) {
      rows_done += min(RB, p.rows - row0);
    } else if (t0 == 0) {
      // the unit goes on in the following shares; its last tile is at unit_end - 1 on the line
      meta.unit = (this_b * Hkv + h) * p.blocks + rb;
      int64_t e = (unit_end - 1) * workers / total;  // share boundaries are floors: at most one off
      while (e * total / workers > unit_end - 1) --e;
      while ((e + 1) * total / workers <= unit_end - 1) ++e;
      meta.end = (int)e;
    }
  }
  if (lane == 0) {
    p.meta[me] = meta;
    add_work(a.status, rows_done);
  }
}

// ---------------------------------------------------------------- join

// The cut units' parts joined: a warp has a row (4 channels a lane) and every SL-th of its parts; a CTA has rows of the units
// whose first parts are the last of `chunk` workers: one, or half as many as a unit has parts where those are many.
// The time is a short chain of loads, so it goes as wide as there is work: 32 parts' references by one load, their rows
// eight at a time.  (With four workers and four rows per CTA, the parts over all its warps: 256 ragged requests 106 us
// instead of 96, one of 1000 tokens 11.1 instead of 10.6, one of 100000 47 instead of 37.)
template <int D, int RB, int SL>
__global__ void __launch_bounds__(SL == 1 ? 256 : 32 * SL) paged_attention_join_kernel(const PagedAttnArgs a, const PaPlan p,
                                                                          int chunk) {
  __shared__ float4 sum_o[SL > 1 ? 32 * SL : 1];
  __shared__ float2 sum_ml[SL];
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, slice = warp % SL, first = SL == 1 ? (int)blockIdx.x : (int)blockIdx.x * chunk;
  const int r = blockIdx.y * (blockDim.x / 32 / SL) + warp / SL;
  auto join = [&](int x0, PaMeta meta) {
    const int rb = meta.unit % p.blocks, bh = meta.unit / p.blocks, h = bh % a.c.Hkv, b = bh / a.c.Hkv;
    const int row = rb * RB + r, parts = meta.end - x0 + 1;
    const bool there = row < p.rows && r < RB, holds = lane * 4 < D;  // of a warp; of a lane
    auto at = [&](int i) { return ((int64_t)(x0 + i) * 2 + (i == 0 ? 1 : 0)) * RB + r; };
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    if (there) {
      // 32 of this warp's parts at a time, a lane with each one's reference and sum
      for (int i0 = slice; i0 < parts; i0 += 32 * SL) {
        const int own = i0 + lane * SL;
        const float2 ml = own < parts ? *reinterpret_cast<const float2*>(p.part_ml + at(own) * 2) : make_float2(-INFINITY, 0.f);
        float top = ml.x;
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, j));
        if (top > m) {
          const float by = ex2(m - top);  // 0 from -infinity
          o.x *= by, o.y *= by, o.z *= by, o.w *= by;
          l = times_pow2(l, m - top);
          m = top;
        }
        const float by = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
        if (ml.x != -INFINITY) l += times_pow2(ml.y, ml.x - m);
        const int n = min(32, (parts - i0 + SL - 1) / SL);
#pragma unroll 8
        for (int i = 0; i < n; ++i) {
          float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
          if (holds) x = *reinterpret_cast<const float4*>(p.part_o + at(i0 + i * SL) * D + lane * 4);
          const float w = __shfl_sync(0xffffffffu, by, i);
          if (w != 0.f) o.x += x.x * w, o.y += x.y * w, o.z += x.z * w, o.w += x.w * w;  // a part that saw nothing holds zeros
        }
      }
#pragma unroll
      for (int j = 16; j > 0; j >>= 1) l += __shfl_xor_sync(0xffffffffu, l, j);
    }
    if constexpr (SL > 1) {
      __syncthreads();  // the last unit's sums have been read
      sum_o[threadIdx.x] = o;
      if (lane == 0) sum_ml[slice] = make_float2(m, l);
      __syncthreads();
      if (slice == 0) {
        const float2 ml = lane < SL ? sum_ml[lane] : make_float2(-INFINITY, 0.f);
        m = ml.x;
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, j));
        const float by = ml.x == -INFINITY ? 0.f : ex2(ml.x - m);
        l = ml.x == -INFINITY ? 0.f : times_pow2(ml.y, ml.x - m);
        o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int i = 0; i < SL; ++i) {
          const float4 x = sum_o[32 * i + lane];
          const float w = __shfl_sync(0xffffffffu, by, i);
          if (w != 0.f) o.x += x.x * w, o.y += x.y * w, o.z += x.z * w, o.w += x.w * w;
        }
#pragma unroll
        for (int j = 16; j > 0; j >>= 1) l += __shfl_xor_sync(0xffffffffu, l, j);
      }
    }
    if (!there || slice != 0) return;
    const bool none = m == -INFINITY;
    const int wt = row / p.G, g = row - wt * p.G;
    const int64_t head = ((int64_t)b * a.W + wt) * a.Hq + (int64_t)h * p.G + g;
    const float by = none ? 0.f : 1.f / l;
    o = none ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(o.x * by, o.y * by, o.z * by, o.w * by);
    if (holds) {
      if (a.out_bf16) {
        const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x, o.y), hi = __floats2bfloat162_rn(o.z, o.w);
        *reinterpret_cast<uint2*>(static_cast<bf16*>(a.out) + head * D + lane * 4) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      } else {
        *reinterpret_cast<float4*>(static_cast<float*>(a.out) + head * D + lane * 4) = o;
      }
    }
    if (lane == 0) {
      if (a.lse) a.lse[head] = none ? -INFINITY : log_sum(m, l);
      add_work(a.status, 1);
    }
  };
  if constexpr (SL == 1) {
    const PaMeta meta = p.meta[first];
    if (meta.unit >= 0) join(first, meta);
  } else {
    PaMeta metas{-1, 0};  // lane i: worker first + i
    if (lane < chunk && first + lane < p.workers) metas = p.meta[first + lane];
    for (uint32_t left = __ballot_sync(0xffffffffu, metas.unit >= 0); left; left &= left - 1) {
      const int i = __ffs(left) - 1;
      join(first + i, PaMeta{__shfl_sync(0xffffffffu, metas.unit, i), __shfl_sync(0xffffffffu, metas.end, i)});
    }
  }
}

// ---------------------------------------------------------------- launch

template <int D, int RB>
cudaError_t pa_join(const PagedAttnArgs& a, const PaPlan& p, int64_t units, cudaStream_t s) {
  const int rows = p.rows < RB ? p.rows : RB, each = rows < 8 ? rows : 8;
  const int64_t parts = units > 0 ? p.workers / units : 1;  // of a unit, about
  if (parts >= 8) {
    const int chunk = parts > 64 ? 32 : (int)(parts / 2), ctas = (p.workers + chunk - 1) / chunk;
    return parts >= 64
               ? launch_pdl(paged_attention_join_kernel<D, RB, 32>, dim3(ctas, rows), dim3(1024), 0, s, a, p, chunk)
               : launch_pdl(paged_attention_join_kernel<D, RB, 8>, dim3(ctas, rows), dim3(256), 0, s, a, p, chunk);
  }
  return launch_pdl(paged_attention_join_kernel<D, RB, 1>, dim3(p.workers, (rows + each - 1) / each), dim3(32 * each), 0, s,
                    a, p, 1);
}

template <int D, bool F8, int NT, bool FINE>
cudaError_t pa_launch(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  using C = PaCfg<D, F8, NT, FINE>;
  auto kernel = paged_attention_kernel<D, F8, NT, FINE>;
  if (C::SMEM > 40 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    if (e != cudaSuccess) return e;
  }
  // no more warps than positions on the longest possible line
  const int64_t tiles = (int64_t)a.max_pages * a.c.page_size / C::TILE + 1 + PA_UNIT_COST;
  int64_t ctas = pa_resident(NT) * (sms < PA_SMS ? sms : PA_SMS);
  const int64_t units = (int64_t)a.B * a.c.Hkv * p.blocks;
  if (tiles < ctas * PA_WARPS && units * tiles < ctas * PA_WARPS) ctas = (units * tiles + PA_WARPS - 1) / PA_WARPS;
  PaPlan plan = p;
  plan.workers = (int)ctas * PA_WARPS;
  const cudaError_t e = launch_pdl(kernel, dim3((unsigned)ctas), dim3(PA_NT), C::SMEM, s, a, plan);
  if (e != cudaSuccess) return e;
  return pa_join<D, C::RB>(a, plan, units, s);
}

template <int D, bool F8, bool FINE>
cudaError_t pa_rows(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s) {
  const int nt = pa_nt(p.rows, FINE);
  if (nt == 1) return pa_launch<D, F8, 1, FINE>(a, p, sms, s);
  if constexpr (!FINE) {
    if (nt == 4) return pa_launch<D, F8, 4, FINE>(a, p, sms, s);
  }
  return pa_launch<D, F8, 2, FINE>(a, p, sms, s);
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
// the tensor-memory form (paged_attention_tc.cu), for d = 128 with bf16 queries and outputs
bool pa_tc_supported(const PagedAttnArgs& a);
int pa_tc_row_block(int rows);
cudaError_t pa_tc(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s);
constexpr int PA_ROWS_BLOCK = 128;  // query rows of a unit of the many-rows form
bool pa_rows_supported(const PagedAttnArgs& a);
cudaError_t pa_rows(const PagedAttnArgs& a, const PaPlan& p, int sms, cudaStream_t s);

}  // namespace kda
