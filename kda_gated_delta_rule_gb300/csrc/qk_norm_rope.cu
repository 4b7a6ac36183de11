// Per-head RMS norm of queries and keys with the position rotation, and its gradient.
//
// Forward, per row x (one token, one head) with weight w:  y = R(p) (x r w),  r = (mean x^2 + eps)^-1/2.
// Backward, with g = R(p)^T dy:  dx = r g w - x r^3 mean(g w x),  dw = sum over rows of g x r.
// R(p) only mixes the two channels of a pair, so its transpose is the rotation by the opposite angle.  All sums are in fp32: with
// fp32 rows dx is off by 6e-8 (rms) and dw, a sum over all rows, by 1.5e-7 (8000 tokens x 40 heads x 128: 2e-7); torch
// operations one after the other are off by 7e-8 and 1.2e-7 (3.8e-7).
//
// Both are bound by HBM (about 10 operations per element against 4 to 6 bytes), but only if the instructions are few.
// A row lies on D/8 lanes.  A lane has two runs of four channels, placed so that both channels of a pair are its own:
// lane i of the rotated part has channels 4i .. 4i + 3 and the same plus rot / 2 (half-split pairing), or
// 8i .. 8i + 7 (neighbouring pairs); either way its four pairs are 4i .. 4i + 3, one 16-byte read of each table, and
// its eight values are held as four float2, the pairs' lower channels in the first two and the upper ones in the others,
// so the arithmetic is on two values per instruction.  (With eight consecutive channels per lane the half-split
// rotation took a shuffle per channel and twice the table bytes: 41 us for 8192 x 40 x 128 bf16 rows; now 28.5, 89 % of the
// copy rate.)
// A group of lanes takes R rows of one token and one kind, queries or keys, issues all its loads before the first
// reduction, reads the angles and the weight once for them, and reduces the rows' sums together.
#include "f32x2.cuh"
#include "launch.h"
#include "rows8.cuh"

namespace kda {

constexpr int NORM_NT = 128, NORM_R = 4;
// CTAs per SM: as many as hold their rows without spills (8192 x 40 x 128 rows, bf16: 28.6 us with 7, 30.8 with 8, 30.0
// with 6; fp32: 55.8 with 6, 58.6 with 7, 64.9 with 8)
constexpr int norm_resident(bool bf16_in) { return bf16_in ? 7 : 6; }
constexpr int NORM_BWD_NT = 256, NORM_BWD_RESIDENT = 2;
// Rows that a group of the backward takes at once: fp32 rows fill the registers with two (16384 x 40 x 128 rows, bf16: 83 us
// with 4, 98 with 2; fp32: 150 us with 2, 163 with 4).
constexpr int norm_bwd_rows(bool bf16_in, bool bf16_grad) { return bf16_in && bf16_grad ? 4 : 2; }

// A lane's channels, and its four pairs.
struct NormLane {
  int a, b;  // first channel of each run
  int pair;  // first pair, or -1 where the channels are not rotated
};
template <int D, bool IL>
__device__ __forceinline__ NormLane norm_lane(int lr, int rot) {
  NormLane n;
  if (lr * 8 >= rot) {
    n.a = lr * 8, n.b = lr * 8 + 4, n.pair = -1;
  } else {
    n.pair = 4 * lr;
    n.a = IL ? 8 * lr : 4 * lr;
    n.b = IL ? 8 * lr + 4 : 4 * lr + rot / 2;
  }
  return n;
}
// Four channels of each run (e0 .. e3, f0 .. f3) as the four float2: half-split pairs are (e_i, f_i), neighbouring ones
// (e0, e1), (e2, e3), (f0, f1), (f2, f3).  spread() and gather() are each other's inverse.
template <bool IL>
__device__ __forceinline__ void spread(float2 (&x)[4], float4 e, float4 f) {
  if (IL) {
    x[0] = make_float2(e.x, e.z), x[1] = make_float2(f.x, f.z);
    x[2] = make_float2(e.y, e.w), x[3] = make_float2(f.y, f.w);
  } else {
    x[0] = make_float2(e.x, e.y), x[1] = make_float2(e.z, e.w);
    x[2] = make_float2(f.x, f.y), x[3] = make_float2(f.z, f.w);
  }
}
template <bool IL>
__device__ __forceinline__ void gather(const float2 (&x)[4], float4& e, float4& f) {
  if (IL) {
    e = make_float4(x[0].x, x[2].x, x[0].y, x[2].y);
    f = make_float4(x[1].x, x[3].x, x[1].y, x[3].y);
  } else {
    e = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    f = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
  }
}

template <bool BF>
struct RawRow;  // a lane's eight channels as loaded (plain loads: a call may work in place)
template <>
struct RawRow<true> {
  uint2 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t row, const NormLane& n) {
    const bf16* p = static_cast<const bf16*>(base) + row;
    a = *reinterpret_cast<const uint2*>(p + n.a);
    b = *reinterpret_cast<const uint2*>(p + n.b);
  }
  __device__ __forceinline__ float4 run(uint2 v) const {
    float4 f;
    unpack_bf16x2(v.x, f.x, f.y);
    unpack_bf16x2(v.y, f.z, f.w);
    return f;
  }
  template <bool IL>
  __device__ __forceinline__ void widen(float2 (&x)[4]) const { spread<IL>(x, run(a), run(b)); }
};
template <>
struct RawRow<false> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t row, const NormLane& n) {
    const float* p = static_cast<const float*>(base) + row;
    a = *reinterpret_cast<const float4*>(p + n.a);
    b = *reinterpret_cast<const float4*>(p + n.b);
  }
  template <bool IL>
  __device__ __forceinline__ void widen(float2 (&x)[4]) const { spread<IL>(x, a, b); }
};
template <bool BF, bool IL>
__device__ __forceinline__ void store_row(void* base, int64_t row, const NormLane& n, const float2 (&x)[4]) {
  float4 e, f;
  gather<IL>(x, e, f);
  if constexpr (BF) {
    bf16* p = static_cast<bf16*>(base) + row;
    *reinterpret_cast<uint2*>(p + n.a) = make_uint2(pack_bf16x2(e.x, e.y), pack_bf16x2(e.z, e.w));
    *reinterpret_cast<uint2*>(p + n.b) = make_uint2(pack_bf16x2(f.x, f.y), pack_bf16x2(f.z, f.w));
  } else {
    float* p = static_cast<float*>(base) + row;
    *reinterpret_cast<float4*>(p + n.a) = e;
    *reinterpret_cast<float4*>(p + n.b) = f;
  }
}

struct Angles {
  float2 c[2], s[2];
};
__device__ __forceinline__ Angles load_angles(const NormArgs& p, int pos, const NormLane& n) {
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (n.pair >= 0) {
    const int64_t at = (int64_t)pos * (p.rot / 2) + n.pair;
    c = __ldg(reinterpret_cast<const float4*>(p.cos + at));
    s = __ldg(reinterpret_cast<const float4*>(p.sin + at));
  }
  return Angles{{make_float2(c.x, c.y), make_float2(c.z, c.w)}, {make_float2(s.x, s.y), make_float2(s.z, s.w)}};
}
// Turns a lane's pairs by +angle (SIGN 1) or -angle (SIGN -1).
template <int SIGN>
__device__ __forceinline__ void rotate(float2 (&x)[4], const Angles& a) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 s = SIGN > 0 ? a.s[i] : make_float2(-a.s[i].x, -a.s[i].y), ns = make_float2(-s.x, -s.y);
    const float2 u = x[i], v = x[i + 2];
    x[i] = fma2(v, ns, mul2(u, a.c[i]));
    x[i + 2] = fma2(u, s, mul2(v, a.c[i]));
  }
}
template <bool IL>
__device__ __forceinline__ void load_weight(float2 (&w)[4], const float* p, const NormLane& n) {
  spread<IL>(w, __ldg(reinterpret_cast<const float4*>(p + n.a)), __ldg(reinterpret_cast<const float4*>(p + n.b)));
}
__device__ __forceinline__ float dot4(const float2 (&a)[4], const float2 (&b)[4]) {
  float2 v = mul2(a[0], b[0]);
#pragma unroll
  for (int i = 1; i < 4; ++i) v = fma2(a[i], b[i], v);
  return v.x + v.y;
}

// Sums of N values over the LPR lanes of a row, to all of them.  Four values over four lanes or more go together: two
// exchanges leave each lane of a quad with one value's partial sum, which is completed across the quads and dealt back (9
// shuffles instead of 16 at LPR = 16).
template <int LPR, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], int lane) {
  if constexpr (N % 4 == 0 && LPR >= 4) {
    const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
    for (int q = 0; q < N; q += 4) {
      float k0 = b0 ? v[q + 1] : v[q], k1 = b0 ? v[q + 3] : v[q + 2];
      k0 += __shfl_xor_sync(0xffffffffu, b0 ? v[q] : v[q + 1], 1);
      k1 += __shfl_xor_sync(0xffffffffu, b0 ? v[q + 2] : v[q + 3], 1);
      float k = b1 ? k1 : k0;
      k += __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2);
#pragma unroll
      for (int o = 4; o < LPR; o <<= 1) k += __shfl_xor_sync(0xffffffffu, k, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[q + i] = __shfl_sync(0xffffffffu, k, (lane & ~3) | i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = row_sum<LPR>(v[i]);
  }
}

// A group's place among the (token, chunk) pairs, chunk by chunk within a token, and how far it moves per turn.
struct NormCursor {
  unsigned t, c, step_t, step_c, chunks;
  __device__ __forceinline__ NormCursor(unsigned first, unsigned step, unsigned chunks_)
      : t(first / chunks_), c(first % chunks_), step_t(step / chunks_), step_c(step % chunks_), chunks(chunks_) {}
  __device__ __forceinline__ void advance() {
    t += step_t;
    c += step_c;
    if (c >= chunks) c -= chunks, ++t;
  }
};

// chunks_q, chunks: groups of R heads per token among the queries, and in all.  The CTAs walk the pairs; the next turn's
// position is read a turn ahead, so that rows and angles are asked for together.
template <int D, int R, bool INBF, bool OUTBF, bool IL>
__global__ void __launch_bounds__(NORM_NT, norm_resident(INBF)) qk_norm_rope_kernel(const NormArgs p, unsigned chunks_q,
                                                                              unsigned chunks, int turns) {
  constexpr int LPR = D / 8, NG = NORM_NT / LPR;
  pdl_begin();
  const int lane = threadIdx.x & 31, lr = threadIdx.x % LPR;
  const NormLane n = norm_lane<D, IL>(lr, p.rot);
  const unsigned T = (unsigned)p.T;
  NormCursor at(blockIdx.x * (unsigned)NG + threadIdx.x / LPR, gridDim.x * (unsigned)NG, chunks);
  int pos = p.rot && at.t < T ? __ldg(p.positions + at.t) : 0, written = 0;
  for (int turn_no = 0; turn_no < turns; ++turn_no) {
    const bool isq = at.c < chunks_q;
    const int h0 = (int)(isq ? at.c : at.c - chunks_q) * R, H = isq ? p.Hq : p.Hkv;
    const void* in = isq ? p.q : p.k;
    void* out = isq ? p.q_out : p.k_out;
    const int64_t in0 = at.t * (isq ? p.q_stride : p.k_stride) + h0 * D;
    const int64_t out0 = at.t * (isq ? p.q_out_stride : p.k_out_stride) + h0 * D;
    bool live = at.t < T;
    RawRow<INBF> raw[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (live && h0 + i < H) raw[i].load(in, in0 + i * D, n);
      else raw[i] = RawRow<INBF>{};
    }
    Angles ang{};
    if (p.rot) {
      if ((unsigned)pos >= (unsigned)p.num_positions) {
        if (live && lr == 0) flag_status(p.status, KDA_DEV_POS_OOB);
        live = false;
      } else {
        ang = load_angles(p, pos, n);
      }
    }
    at.advance();
    if (p.rot) pos = at.t < T ? __ldg(p.positions + at.t) : 0;
    float2 w[4];
    load_weight<IL>(w, isq ? p.wq : p.wk, n);
    float r[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float2 x[4];
      raw[i].template widen<IL>(x);
      r[i] = dot4(x, x);
    }
    row_sums<LPR, R>(r, lane);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float2 x[4];
      raw[i].template widen<IL>(x);
      const float2 scale = both(rsqrtf(r[i] * (1.f / D) + p.eps));
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = mul2(mul2(x[e], scale), w[e]);
      if (p.rot) rotate<1>(x, ang);
      if (live && h0 + i < H) {
        store_row<OUTBF, IL>(out, out0 + i * D, n, x);
        ++written;
      }
    }
  }
  if (p.status) {  // one atomic per warp
    const int sum = __reduce_add_sync(0xffffffffu, lr == 0 ? written : 0);
    if (lane == 0) add_work(p.status, sum);
  }
}

// Sum of N floats (a power of two) STRIDE apart, in pairs of pairs: a few roundings instead of one per term.
template <int N, int STRIDE>
__device__ __forceinline__ float pair_sum(const float* p) {
  if constexpr (N == 1) return *p;
  else return pair_sum<N / 2, STRIDE>(p) + pair_sum<N / 2, STRIDE>(p + N / 2 * STRIDE);
}

// Backward.  The first ctas_q CTAs walk the query rows, the others the key rows, in proportion to the heads, so a lane
// holds one weight and one set of weight gradients in registers over its whole walk.  The CTA adds its groups' sums
// up in shared memory in a fixed order, and one row of partial sums per CTA goes to the workspace.
template <int D, int R, bool INBF, bool GBF, bool OUTBF, bool IL>
__global__ void __launch_bounds__(NORM_BWD_NT, NORM_BWD_RESIDENT)
    qk_norm_rope_bwd_kernel(const NormArgs p, const void* __restrict__ dyq, const void* __restrict__ dyk,
                            float* __restrict__ partial, int ctas_q) {
  constexpr int LPR = D / 8, NG = NORM_BWD_NT / LPR;
  pdl_begin();
  const int lane = threadIdx.x & 31, lr = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const bool isq = blockIdx.x < ctas_q;
  const int H = isq ? p.Hq : p.Hkv;
  const unsigned chunks = (unsigned)(H + R - 1) / R;
  const unsigned cta = isq ? blockIdx.x : blockIdx.x - ctas_q, ctas = isq ? ctas_q : gridDim.x - ctas_q;
  const void *in = isq ? p.q : p.k, *dy = isq ? dyq : dyk;
  void* out = isq ? p.q_out : p.k_out;
  const int64_t in_stride = isq ? p.q_stride : p.k_stride, out_stride = isq ? p.q_out_stride : p.k_out_stride;
  const NormLane n = norm_lane<D, IL>(lr, p.rot);
  float2 w[4], acc[4] = {};
  load_weight<IL>(w, isq ? p.wq : p.wk, n);
  int written = 0;
  const unsigned T = (unsigned)p.T;
  NormCursor at(cta * NG + grp, ctas * NG, chunks);
  int pos_next = p.rot && at.t < T ? __ldg(p.positions + at.t) : 0;
  // every group of a CTA takes the same number of turns, so the shuffles below stay warp-wide
  const int64_t per_turn = (int64_t)ctas * NG;
  const int turns = (int)((p.T * chunks + per_turn - 1 - (int64_t)cta * NG) / per_turn);
  for (int turn_no = 0; turn_no < turns; ++turn_no) {
    bool live = at.t < T;
    const int h0 = (int)at.c * R;
    const int64_t in0 = at.t * in_stride + h0 * D, dy0 = ((int64_t)at.t * H + h0) * D, out0 = at.t * out_stride + h0 * D;
    RawRow<INBF> rx[R];
    RawRow<GBF> rg[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (live && h0 + i < H) {
        rx[i].load(in, in0 + i * D, n);
        rg[i].load(dy, dy0 + i * D, n);
      } else {
        rx[i] = RawRow<INBF>{};
        rg[i] = RawRow<GBF>{};
      }
    }
    Angles ang{};
    if (p.rot) {
      if ((unsigned)pos_next >= (unsigned)p.num_positions) {
        if (live && lr == 0) flag_status(p.status, KDA_DEV_POS_OOB);
        live = false;
      } else {
        ang = load_angles(p, pos_next, n);
      }
    }
    at.advance();
    if (p.rot) pos_next = at.t < T ? __ldg(p.positions + at.t) : 0;
    float2 g[R][4];
    float v[2 * R];  // per row: sum x^2, sum g w x
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float2 x[4], gx[4];
      rx[i].template widen<IL>(x);
      rg[i].template widen<IL>(g[i]);
      if (p.rot) rotate<-1>(g[i], ang);
      v[2 * i] = dot4(x, x);
#pragma unroll
      for (int e = 0; e < 4; ++e) gx[e] = mul2(g[i][e], x[e]);
      v[2 * i + 1] = dot4(gx, w);
    }
    row_sums<LPR, 2 * R>(v, lane);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (!live || h0 + i >= H) continue;
      float2 x[4];
      rx[i].template widen<IL>(x);
      const float r = rsqrtf(v[2 * i] * (1.f / D) + p.eps);
      const float2 r2 = both(r), k = both(-(r * r) * (r * v[2 * i + 1]) * (1.f / D));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 gr = mul2(g[i][e], r2);
        acc[e] = fma2(gr, x[e], acc[e]);
        x[e] = fma2(gr, w[e], mul2(x[e], k));
      }
      store_row<OUTBF, IL>(out, out0 + i * D, n, x);
      ++written;
    }
  }
  __shared__ float sum[NG][D + 4];
  {
    float4 e, f;
    gather<IL>(acc, e, f);
    *reinterpret_cast<float4*>(&sum[grp][n.a]) = e;
    *reinterpret_cast<float4*>(&sum[grp][n.b]) = f;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += NORM_BWD_NT) {
    partial[(int64_t)blockIdx.x * D + e] = pair_sum<NG, D + 4>(&sum[0][e]);
  }
  if (p.status) {
    const int total = __reduce_add_sync(0xffffffffu, lr == 0 ? written : 0);
    if (lane == 0) add_work(p.status, total);
  }
}

// Adds the CTAs' partial weight gradients, the queries' in blocks 0 .. D/16 - 1 and the keys' in the rest: 16 channels per
// CTA, the partial rows spread over its 32 half-warps and then added pair by pair, so the result does not depend on
// timing.
__global__ void __launch_bounds__(512) qk_norm_weight_grad_kernel(const float* __restrict__ partial, int ctas_q, int ctas,
                                                                  int D, float* __restrict__ dwq,
                                                                  float* __restrict__ dwk) {
  pdl_begin();
  __shared__ float part[32][17];
  const int c = threadIdx.x % 16, w = threadIdx.x / 16;
  const bool isq = blockIdx.x < D / 16;
  const int e = (isq ? blockIdx.x : blockIdx.x - D / 16) * 16 + c;
  const int lo = isq ? 0 : ctas_q, hi = isq ? ctas_q : ctas;
  float v = 0.f;
#pragma unroll 4
  for (int i = lo + w; i < hi; i += 32) v += partial[(int64_t)i * D + e];
  part[w][c] = v;
  __syncthreads();
  if (w == 0) (isq ? dwq : dwk)[e] = pair_sum<32, 17>(&part[0][c]);
}

namespace {

template <int D, int R, bool IL>
cudaError_t norm_fwd(const NormArgs& a, cudaStream_t s) {
  constexpr int NG = NORM_NT / (D / 8);
  const unsigned cq = (a.Hq + R - 1) / R, chunks = cq + (a.Hkv + R - 1) / R;
  int64_t blocks = (a.T * chunks + NG - 1) / NG;
  if (a.T > 0x7fffffff || blocks * NG > 0x7fffffff) return cudaErrorInvalidValue;
  const int64_t at_once = 152 * norm_resident(a.in_bf16), turns = (blocks + at_once - 1) / at_once;
  blocks = (blocks + turns - 1) / turns;  // as many as give every CTA that many turns
  auto kernel = a.in_bf16 ? (a.out_bf16 ? qk_norm_rope_kernel<D, R, true, true, IL> : qk_norm_rope_kernel<D, R, true, false, IL>)
                          : (a.out_bf16 ? qk_norm_rope_kernel<D, R, false, true, IL>
                                        : qk_norm_rope_kernel<D, R, false, false, IL>);
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(NORM_NT), 0, s, a, cq, chunks, (int)turns);
}

template <int D>
cudaError_t norm_fwd_d(const NormArgs& a, cudaStream_t s) {
  // Few rows: one per group, so that they spread over the SMs.  Otherwise NORM_R, for loads in flight and one
  // read of the angles.
  if (a.T * (a.Hq + a.Hkv) <= 4096) return a.interleaved ? norm_fwd<D, 1, true>(a, s) : norm_fwd<D, 1, false>(a, s);
  return a.interleaved ? norm_fwd<D, NORM_R, true>(a, s) : norm_fwd<D, NORM_R, false>(a, s);
}

template <int D, bool IL>
cudaError_t norm_bwd(const NormArgs& a, const void* dyq, const void* dyk, bool g_bf16, float* partial, int ctas_q,
                     int ctas, cudaStream_t s) {
  const int sel = (a.in_bf16 ? 4 : 0) | (g_bf16 ? 2 : 0) | (a.out_bf16 ? 1 : 0);
  switch (sel) {
#define KDA_CASE(n, i, g, o)                                                                                         \
  case n: return launch_pdl(qk_norm_rope_bwd_kernel<D, norm_bwd_rows(i, g), i, g, o, IL>, dim3(ctas),                \
                            dim3(NORM_BWD_NT), 0, s, a, dyq, dyk, partial, ctas_q);
    KDA_CASE(0, false, false, false)
    KDA_CASE(1, false, false, true)
    KDA_CASE(2, false, true, false)
    KDA_CASE(3, false, true, true)
    KDA_CASE(4, true, false, false)
    KDA_CASE(5, true, false, true)
    KDA_CASE(6, true, true, false)
    KDA_CASE(7, true, true, true)
#undef KDA_CASE
  }
  return cudaErrorInvalidValue;
}

template <int D>
cudaError_t norm_bwd_d(const NormArgs& a, const void* dyq, const void* dyk, bool g_bf16, float* dwq, float* dwk,
                       float* partial, cudaStream_t s) {
  constexpr int NG = NORM_BWD_NT / (D / 8), MOST = 152 * NORM_BWD_RESIDENT;
  const int R = norm_bwd_rows(a.in_bf16, g_bf16);
  static_assert(MOST <= NORM_BWD_CTAS, "one row of the workspace per CTA");
  const int64_t need_q = (a.T * ((a.Hq + R - 1) / R) + NG - 1) / NG, need_k = (a.T * ((a.Hkv + R - 1) / R) + NG - 1) / NG;
  int64_t ctas_q = need_q, ctas_k = need_k;
  if (need_q + need_k > MOST) {
    ctas_q = (MOST * need_q + (need_q + need_k) / 2) / (need_q + need_k);
    ctas_q = ctas_q < 1 ? 1 : ctas_q > MOST - 1 ? MOST - 1 : ctas_q;
    ctas_k = MOST - ctas_q;
  }
  const int ctas = (int)(ctas_q + ctas_k);
  if (ctas > 0) {  // without tokens the weights' gradients are zero
    const cudaError_t e = a.interleaved ? norm_bwd<D, true>(a, dyq, dyk, g_bf16, partial, (int)ctas_q, ctas, s)
                                        : norm_bwd<D, false>(a, dyq, dyk, g_bf16, partial, (int)ctas_q, ctas, s);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(qk_norm_weight_grad_kernel, dim3(2 * D / 16), dim3(512), 0, s, (const float*)partial, (int)ctas_q,
                    ctas, D, dwq, dwk);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const NormArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 16: return norm_fwd_d<16>(a, s);
    case 32: return norm_fwd_d<32>(a, s);
    case 64: return norm_fwd_d<64>(a, s);
    default: return norm_fwd_d<128>(a, s);
  }
}

cudaError_t launch_qk_norm_rope_backward(const NormArgs& a, const void* dyq, const void* dyk, bool g_bf16, float* dwq,
                                         float* dwk, float* partial, cudaStream_t s) {
  switch (a.d) {
    case 16: return norm_bwd_d<16>(a, dyq, dyk, g_bf16, dwq, dwk, partial, s);
    case 32: return norm_bwd_d<32>(a, dyq, dyk, g_bf16, dwq, dwk, partial, s);
    case 64: return norm_bwd_d<64>(a, dyq, dyk, g_bf16, dwq, dwk, partial, s);
    default: return norm_bwd_d<128>(a, dyq, dyk, g_bf16, dwq, dwk, partial, s);
  }
}

}  // namespace kda
