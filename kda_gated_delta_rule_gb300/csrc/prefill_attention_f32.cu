// Attention over packed prompts and its gradients on the CUDA cores: fp32 inputs, any head size.
//
//   x_ij = scale q_i . k_j, capped: y = cap tanh(x / cap);  p = softmax_j(y) over the keys that row i sees;  o_i = sum_j p_ij v_j
//   dv_j = sum_i p_ij do_i,  dy = p (do_i . v_j - D_i),  D_i = do_i . o_i,  dx = dy (1 - (y / cap)^2) scale
//   dq_i = sum_j dx_ij k_j,  dk_j = sum_i dx_ij q_i
//
// A CTA has 64 query rows of one head and walks the 64-key tiles that they see with the running maximum and sum, the next tile on its way
// (cp.async) under the present one's products; a thread has RI x 4 scores of a tile and the same RI rows of the output.  The gradients
// take two kernels, so that each output has one owner and no sum depends on an order of arrival: a CTA per 64 keys of a key/value
// head walks the query blocks of all its query heads (dk, dv), one per 64 query rows walks the keys (dq).  Both form the scores
// again from the log-sum-exp.  Where there are few units, their walks are what takes the time: then a cluster of CTAs deals a walk's
// tiles out, and adds its results up in order through distributed shared memory.
// Bound by shared memory, which feeds the fp32 pipe 16 bytes a lane in 4 cycles whether lanes share them or not (8 rows x 4 columns: 12 loads
// for 64 two-wide multiply-adds): 8 prompts of 2048 tokens, 12 / 4 heads of 64, forward 1249 us, 41 TFLOP/s of the pipe's 75; backward
// 4640.  3 prompts of 2047 tokens, 12 heads of 64: 140 us.
#include <cooperative_groups.h>

#include "f32x2.cuh"
#include "prefill_attention.cuh"

namespace kda {

namespace {

constexpr int PB = 64;  // rows and keys of a block (1 << 6)
// A thread has RI rows and 4 columns of a tile of scores.
constexpr int pf_threads(int ri) { return PB * PB / (4 * ri); }

namespace cg = cooperative_groups;

// What the CTAs of a cluster hand one another at the end: `N` floats for each of a thread's RI rows.  Row i of all threads is finished by CTA
// i * parts / RI, which adds the others' up in order.
template <int RI>
__device__ __forceinline__ int row_owner(int i, int parts) { return i * parts / RI; }
template <int RI, int N>
__device__ __forceinline__ void hand_over(float* slots, int i, const float (&x)[N]) {
#pragma unroll
  for (int c = 0; c < N; ++c) slots[(i * N + c) * pf_threads(RI) + threadIdx.x] = x[c];
}
template <int RI, int N>
__device__ __forceinline__ void take_over(cg::cluster_group& cluster, float* slots, int part, int i, float (&x)[N]) {
  const float* from = cluster.map_shared_rank(slots, part);
#pragma unroll
  for (int c = 0; c < N; ++c) x[c] = from[(i * N + c) * pf_threads(RI) + threadIdx.x];
}
// The sums of the cluster's CTAs, in order, at each row's owner.
template <int RI, int N>
__device__ __forceinline__ void add_parts(cg::cluster_group& cluster, float* slots, float (&acc)[RI][N]) {
  const int parts = cluster.num_blocks(), part = cluster.block_rank();
  if (parts == 1) return;
#pragma unroll
  for (int i = 0; i < RI; ++i) hand_over<RI>(slots, i, acc[i]);
  cluster.sync();
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    if (row_owner<RI>(i, parts) != part) continue;
    take_over<RI>(cluster, slots, 0, i, acc[i]);
    for (int n = 1; n < parts; ++n) {
      float x[N];
      take_over<RI>(cluster, slots, n, i, x);
#pragma unroll
      for (int c = 0; c < N; ++c) acc[i][c] += x[c];
    }
  }
}

template <int D>
struct PfShape {
  static constexpr int LD = D + 4;                 // floats between rows: the 16 rows a half-warp reads meet all banks
  static constexpr int CPT = D / 16;               // channels of a thread
  static constexpr int G = CPT < 4 ? CPT : 4;      // contiguous ones
  static constexpr int NG = CPT / G;               // groups of them, 16 G channels apart
  static constexpr int PLD = PB + 4;
};

// Rows 0 .. 63 of `base` (tokens `stride` apart) on their way; those from `valid` on are zeros.
template <int D, int RI>
__device__ __forceinline__ void load_block(float* dst, const float* base, int64_t stride, int valid) {
  constexpr int C4 = D / 4;
#pragma unroll 4
  for (int i = threadIdx.x; i < PB * C4; i += pf_threads(RI)) {
    const int r = i / C4, c = (i - r * C4) * 4;
    const bool there = r < valid;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + r * PfShape<D>::LD + c)),
                 "l"(base + (there ? r : 0) * stride + c), "r"(there ? 16 : 0)
                 : "memory");
  }
}
__device__ __forceinline__ void loads_sent() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last `N` groups of this thread's loads are there
template <int N>
__device__ __forceinline__ void loads_there() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// s[i][j] = row (ty + 16 i) of a times row (tx + 16 j) of b
template <int D, int RI>
__device__ __forceinline__ void dots(const float* a, const float* b, float (&s)[RI][4]) {
  constexpr int LD = PfShape<D>::LD;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float2 acc[RI][4];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = both(0.f);
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[RI], y[4];
#pragma unroll
    for (int i = 0; i < RI; ++i) x[i] = *reinterpret_cast<const float4*>(a + (ty + PB / RI * i) * LD + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * LD + c);
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fma2(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), acc[i][j]);
        acc[i][j] = fma2(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = acc[i][j].x + acc[i][j].y;
}

// A thread's channels of a row in shared memory.
template <int D>
__device__ __forceinline__ void ld_channels(const float* row, float (&v)[PfShape<D>::CPT]) {
  using S = PfShape<D>;
  const int tx = threadIdx.x & 15;
#pragma unroll
  for (int n = 0; n < S::NG; ++n) {
    const float* p = row + n * 16 * S::G + tx * S::G;
    if constexpr (S::G == 4) {
      const float4 x = *reinterpret_cast<const float4*>(p);
      v[4 * n] = x.x, v[4 * n + 1] = x.y, v[4 * n + 2] = x.z, v[4 * n + 3] = x.w;
    } else if constexpr (S::G == 2) {
      const float2 x = *reinterpret_cast<const float2*>(p);
      v[0] = x.x, v[1] = x.y;
    } else {
      v[0] = *p;
    }
  }
}

// acc += p v, two channels at once
template <int N>
__device__ __forceinline__ void axpy(float (&acc)[N], float p, const float (&v)[N]) {
  if constexpr (N >= 2) {
#pragma unroll
    for (int c = 0; c < N; c += 2) {
      const float2 r = fma2(both(p), make_float2(v[c], v[c + 1]), make_float2(acc[c], acc[c + 1]));
      acc[c] = r.x, acc[c + 1] = r.y;
    }
  } else {
    acc[0] = fmaf(p, v[0], acc[0]);
  }
}

// acc[i] += sum_j w(i, j) row_j over 4 rows of b at j0, w given per output row
template <int D, int RI>
__device__ __forceinline__ void add_rows(float (&acc)[RI][PfShape<D>::CPT], const float4 (&w)[RI], const float* b) {
  constexpr int CPT = PfShape<D>::CPT;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[CPT];
    ld_channels<D>(b + j * PfShape<D>::LD, v);
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const float p = j == 0 ? w[i].x : j == 1 ? w[i].y : j == 2 ? w[i].z : w[i].w;
      axpy(acc[i], p, v);
    }
  }
}

template <int D, typename Out>
__device__ __forceinline__ void store_channels(Out* row, const float (&v)[PfShape<D>::CPT]) {
  using S = PfShape<D>;
  const int tx = threadIdx.x & 15;
#pragma unroll
  for (int n = 0; n < S::NG; ++n) {
    Out* p = row + n * 16 * S::G + tx * S::G;
    if constexpr (S::G == 4 && sizeof(Out) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[4 * n], v[4 * n + 1], v[4 * n + 2], v[4 * n + 3]);
    } else {
#pragma unroll
      for (int c = 0; c < S::G; ++c) p[c] = from_f32<Out>(v[S::G * n + c]);
    }
  }
}
template <int D>
__device__ __forceinline__ void store_row(void* base, bool is_bf16, int64_t at, const float (&v)[PfShape<D>::CPT]) {
  if (is_bf16) store_channels<D>(static_cast<bf16*>(base) + at, v);
  else store_channels<D>(static_cast<float*>(base) + at, v);
}

// The score in powers of two, and the cap's slope there.
__device__ __forceinline__ float score2(float dot, float scale, float cap, float& slope) {
  const float x = dot * scale;
  if (cap > 0.f) {
    const float t = tanhf(x / cap);
    slope = 1.f - t * t;
    return cap * t * PA_LOG2E;
  }
  slope = 1.f;
  return x * PA_LOG2E;
}

// Whether a thread's share of a tile's values are numbers.
template <int D, int RI>
__device__ __forceinline__ bool numbers(const float* sv) {
  constexpr int C4 = D / 4;
  bool ok = true;
#pragma unroll 4
  for (int i = threadIdx.x; i < PB * C4; i += pf_threads(RI)) {
    const int r = i / C4, c = (i - r * C4) * 4;
    const float4 x = *reinterpret_cast<const float4*>(sv + r * PfShape<D>::LD + c);
    const float most = 3.402823466e38f;
    ok = ok && fabsf(x.x) <= most && fabsf(x.y) <= most && fabsf(x.z) <= most && fabsf(x.w) <= most;
  }
  return ok;
}

template <int D, int RI>
__global__ void __launch_bounds__(pf_threads(RI), D == 128 ? 1 : 2) pf_f32_kernel(const PromptAttnArgs a, const int64_t places) {
  using S = PfShape<D>;
  extern __shared__ __align__(16) float sm[];
  constexpr int BLOCK = PB * S::LD;
  float *sq = sm, *kv = sq + BLOCK, *sp = kv + 4 * BLOCK;  // kv: two tiles of K and V
  pdl_begin();
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank(), unit = blockIdx.x / parts;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, h = unit % a.Hq, kh = h / (a.Hq / a.Hkv);
  if (blockIdx.x == 0 && tid < 32) pf_check_offsets(a);
  PfRanks<6> ranks(a);
  const PfBlock b = pf_ranked(a, ranks, unit / a.Hq, places, false);
  if (b.len == 0) return;
  const int rows = min(PB, b.len - b.row0), window = a.window > 0 ? a.window : 0x7fffffff;
  load_block<D, RI>(sq, static_cast<const float*>(a.q) + (int64_t)(b.t0 + b.row0) * a.q_stride + h * D, a.q_stride, rows);
  float o[RI][S::CPT], m[RI], l[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    m[i] = PF_NONE, l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) o[i][c] = 0.f;
  }
  const int last = b.row0 + rows - 1, step = parts * PB;
  const int lowest = max(0, b.row0 - window + 1) / PB, first = (lowest + ((part - lowest) & (parts - 1))) * PB;
  auto load = [&](int k0) {
    float* to = kv + (k0 / step & 1) * 2 * BLOCK;
    const int64_t tok = b.t0 + k0;
    load_block<D, RI>(to, static_cast<const float*>(a.k) + tok * a.k_stride + kh * D, a.k_stride, b.len - k0);
    load_block<D, RI>(to + BLOCK, static_cast<const float*>(a.v) + tok * a.v_stride + kh * D, a.v_stride, b.len - k0);
  };
  if (first <= last) load(first);
  loads_sent();
  for (int k0 = first; k0 <= last; k0 += step) {
    const float *sk = kv + (k0 / step & 1) * 2 * BLOCK, *sv = sk + BLOCK;
    if (k0 + step <= last) load(k0 + step);  // over the tile before, which all have left
    loads_sent();
    loads_there<1>();
    __syncthreads();
    float s[RI][4];
    dots<D, RI>(sq, sk, s);
    const bool masked = k0 + PB - 1 > b.row0 || k0 <= last - window;
    // what unseen keys' values hold does not matter, NaN included (0 * NaN): a tile with such values takes the long way
    const bool careful = masked && !__syncthreads_and(numbers<D, RI>(sv));
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int row = b.row0 + ty + PB / RI * i;
      float top = m[i], slope;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 16 * j;
        s[i][j] = score2(s[i][j], a.scale, a.softcap, slope);
        if (masked && !(key <= row && key > row - window)) s[i][j] = -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int n = 1; n < 16; n <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, n));
      const float by = ex2(m[i] - top);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = ex2(s[i][j] - top);
        sum += p;
        sp[(ty + PB / RI * i) * S::PLD + tx + 16 * j] = p;
      }
      l[i] = l[i] * by + sum;
#pragma unroll
      for (int c = 0; c < S::CPT; ++c) o[i][c] *= by;
    }
    __syncwarp();  // a row's probabilities come from its own half-warp
    if (!careful) {
#pragma unroll 2
      for (int j = 0; j < PB; j += 4) {
        float4 w[RI];
#pragma unroll
        for (int i = 0; i < RI; ++i) w[i] = *reinterpret_cast<const float4*>(sp + (ty + PB / RI * i) * S::PLD + j);
        add_rows<D, RI>(o, w, sv + j * S::LD);
      }
    } else {
#pragma unroll 1
      for (int j = 0; j < PB; ++j) {
        float v[S::CPT];
        ld_channels<D>(sv + j * S::LD, v);
#pragma unroll
        for (int i = 0; i < RI; ++i) {
          const int row = b.row0 + ty + PB / RI * i;
          const bool seen = k0 + j <= row && k0 + j > row - window;
          const float p = sp[(ty + PB / RI * i) * S::PLD + j];
#pragma unroll
          for (int c = 0; c < S::CPT; ++c) o[i][c] = seen ? fmaf(p, v[c], o[i][c]) : o[i][c];
        }
      }
    }
    __syncthreads();
  }
  loads_there<0>();
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int n = 1; n < 16; n <<= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], n);
  if (parts > 1) {
    constexpr int N = S::CPT + 2;
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      float x[N] = {m[i], l[i]};
#pragma unroll
      for (int c = 0; c < S::CPT; ++c) x[2 + c] = o[i][c];
      hand_over<RI>(kv, i, x);
    }
    cluster.sync();
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      if (row_owner<RI>(i, parts) != part) continue;
      float x[N];
      for (int n = 0; n < parts; ++n) {
        take_over<RI>(cluster, kv, n, i, x);
        const float top = n == 0 ? x[0] : fmaxf(m[i], x[0]), by = n == 0 ? 0.f : ex2(m[i] - top), w = ex2(x[0] - top);
        if (n == 0) {
          l[i] = x[1];
#pragma unroll
          for (int c = 0; c < S::CPT; ++c) o[i][c] = x[2 + c];
        } else {
          l[i] = l[i] * by + x[1] * w;
#pragma unroll
          for (int c = 0; c < S::CPT; ++c) o[i][c] = o[i][c] * by + x[2 + c] * w;
        }
        m[i] = top;
      }
    }
  }
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = ty + PB / RI * i;
    if (r >= rows || row_owner<RI>(i, parts) != part) continue;
    const int64_t t = b.t0 + b.row0 + r;
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) o[i][c] /= l[i];
    store_row<D>(a.out, a.out_bf16, t * a.out_stride + h * D, o[i]);
    if (tx == 0 && a.lse) a.lse[t * a.Hq + h] = m[i] * PA_LN2 + logf(l[i]);
  }
  if (tid == 0 && part == 0) add_work(a.status, rows);
  if (parts > 1) cluster.sync();  // the others have read what is here
}

// Probabilities and dy of the tile (rows: queries, columns: keys) from the scores, with the masks; also in shared memory.
template <int D, int RI>
__device__ __forceinline__ void tile_grads(const PromptAttnArgs& a, const float2* stats, const float* sq, const float* sk,
                                           const float* sdo, const float* sv, int row0, int k0, int rows, int len, int window,
                                           float* sp, float* sds) {
  using S = PfShape<D>;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float2 st[RI];
#pragma unroll
  for (int i = 0; i < RI; ++i) st[i] = ty + PB / RI * i < rows ? __ldg(stats + ty + PB / RI * i) : make_float2(0.f, 0.f);
  float s[RI][4], dp[RI][4];
  dots<D, RI>(sq, sk, s);
  dots<D, RI>(sdo, sv, dp);
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = ty + PB / RI * i, row = row0 + r;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int key = k0 + tx + 16 * j;
      const bool seen = r < rows && key < len && key <= row && key > row - window;
      float slope;
      const float y = score2(s[i][j], a.scale, a.softcap, slope);
      const float p = seen ? ex2(y - st[i].x) : 0.f;
      if (sp) sp[r * S::PLD + tx + 16 * j] = p;
      sds[r * S::PLD + tx + 16 * j] = seen ? p * (dp[i][j] - st[i].y) * slope : 0.f;
    }
  }
  // a query that sees one key has p = 1 and dx = 0, whatever p and D are rounded to
  const int single = window == 1 ? PB : row0 == 0 ? 1 : 0;  // the block's first queries
  if (single > ty) {
#pragma unroll
    for (int i = 0; i < RI; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ty + PB / RI * i < single) sds[(ty + PB / RI * i) * S::PLD + tx + 16 * j] = 0.f;
  }
}

__host__ __device__ constexpr int kv_buffers(int d) { return d == 128 ? 1 : 2; }  // of Q and dO: what shared memory holds

template <int D, int RI>
__global__ void __launch_bounds__(pf_threads(RI), D == 128 ? 1 : 0)
    pf_f32_grad_kv_kernel(const PromptAttnArgs a, const PromptGradArgs g, const float2* __restrict__ stats, const int64_t places) {
  using S = PfShape<D>;
  extern __shared__ __align__(16) float sm[];
  constexpr int BLOCK = PB * S::LD, BUF = kv_buffers(D);
  float *sk = sm, *sv = sk + BLOCK, *qo = sv + BLOCK, *sp = qo + 2 * BUF * BLOCK, *sds = sp + PB * S::PLD;  // qo: Q and dO
  pdl_begin();
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank(), unit = blockIdx.x / parts;
  const int tid = threadIdx.x, ty = tid >> 4, kh = unit % a.Hkv, group = a.Hq / a.Hkv;
  if (blockIdx.x == 0 && tid < 32) pf_check_offsets(a);
  PfRanks<6> ranks(a);
  const PfBlock b = pf_ranked(a, ranks, unit / a.Hkv, places, true);
  if (b.len == 0) return;
  const int k0 = b.row0, keys = min(PB, b.len - k0), window = a.window > 0 ? a.window : 0x7fffffff;
  const int64_t tok = b.t0 + k0;
  load_block<D, RI>(sk, static_cast<const float*>(a.k) + tok * a.k_stride + kh * D, a.k_stride, keys);
  load_block<D, RI>(sv, static_cast<const float*>(a.v) + tok * a.v_stride + kh * D, a.v_stride, keys);
  float dk[RI][S::CPT], dv[RI][S::CPT];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) dk[i][c] = dv[i][c] = 0.f;
  const int64_t last = min((int64_t)b.len - 1, (int64_t)k0 + keys - 1 + window - 1);  // the last row that sees one of the keys
  // a round: a block of one head; this CTA's blocks are `part`, `part` + parts, ..
  const int blocks = max(0, ((int)(last / PB) - k0 / PB + parts - part) / parts), n = blocks * group;
  auto load = [&](int i) {
    const int h = kh * group + i / blocks, row0 = k0 + (part + i % blocks * parts) * PB;
    const int64_t t = b.t0 + row0;
    float* to = qo + (i % BUF) * 2 * BLOCK;
    load_block<D, RI>(to, static_cast<const float*>(a.q) + t * a.q_stride + h * D, a.q_stride, b.len - row0);
    load_block<D, RI>(to + BLOCK, static_cast<const float*>(g.d_out) + t * g.d_out_stride + h * D, g.d_out_stride, b.len - row0);
  };
  if (n > 0) load(0);
  loads_sent();
  for (int i = 0; i < n; ++i) {
    const int h = kh * group + i / blocks, row0 = k0 + (part + i % blocks * parts) * PB;
    const float *sq = qo + (i % BUF) * 2 * BLOCK, *sdo = sq + BLOCK;
    const int64_t t = b.t0 + row0;
    if (BUF == 2 && i + 1 < n) load(i + 1);  // over the round before, which all have left
    loads_sent();
    loads_there<BUF - 1>();
    __syncthreads();
    tile_grads<D, RI>(a, stats + h * a.T + t, sq, sk, sdo, sv, row0, k0, min(PB, b.len - row0), b.len, window, sp, sds);
    __syncthreads();
#pragma unroll 2
    for (int q = 0; q < PB; ++q) {
      float4 p[RI / 4], ds[RI / 4];
#pragma unroll
      for (int r = 0; r < RI / 4; ++r) {
        p[r] = *reinterpret_cast<const float4*>(sp + q * S::PLD + ty * RI + 4 * r);
        ds[r] = *reinterpret_cast<const float4*>(sds + q * S::PLD + ty * RI + 4 * r);
      }
      float x[S::CPT], y[S::CPT];
      ld_channels<D>(sdo + q * S::LD, x);
      ld_channels<D>(sq + q * S::LD, y);
#pragma unroll
      for (int r = 0; r < RI; ++r) {
        const float4 pr = p[r / 4], dr = ds[r / 4];
        axpy(dv[r], r % 4 == 0 ? pr.x : r % 4 == 1 ? pr.y : r % 4 == 2 ? pr.z : pr.w, x);
        axpy(dk[r], r % 4 == 0 ? dr.x : r % 4 == 1 ? dr.y : r % 4 == 2 ? dr.z : dr.w, y);
      }
    }
    __syncthreads();
    if (BUF == 1 && i + 1 < n) load(i + 1);
  }
  loads_there<0>();
  add_parts(cluster, qo, dk);
  add_parts(cluster, qo + PB * D, dv);
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = ty * RI + i;
    if (r >= keys || row_owner<RI>(i, parts) != part) continue;
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) dk[i][c] *= a.scale;
    store_row<D>(g.dk, g.bf16, (tok + r) * g.dk_stride + kh * D, dk[i]);
    store_row<D>(g.dv, g.bf16, (tok + r) * g.dv_stride + kh * D, dv[i]);
  }
  if (parts > 1) cluster.sync();
}

template <int D, int RI>
__global__ void __launch_bounds__(pf_threads(RI), D == 128 ? 1 : 2)
    pf_f32_grad_q_kernel(const PromptAttnArgs a, const PromptGradArgs g, const float2* __restrict__ stats, const int64_t places) {
  using S = PfShape<D>;
  extern __shared__ __align__(16) float sm[];
  constexpr int BLOCK = PB * S::LD;
  float *sq = sm, *sdo = sq + BLOCK, *kv = sdo + BLOCK, *sds = kv + 4 * BLOCK;
  pdl_begin();
  cg::cluster_group cluster = cg::this_cluster();
  const int parts = cluster.num_blocks(), part = cluster.block_rank(), unit = blockIdx.x / parts;
  const int tid = threadIdx.x, ty = tid >> 4, h = unit % a.Hq, kh = h / (a.Hq / a.Hkv);
  PfRanks<6> ranks(a);
  const PfBlock b = pf_ranked(a, ranks, unit / a.Hq, places, false);
  if (b.len == 0) return;
  const int rows = min(PB, b.len - b.row0), window = a.window > 0 ? a.window : 0x7fffffff;
  const int64_t t = b.t0 + b.row0;
  load_block<D, RI>(sq, static_cast<const float*>(a.q) + t * a.q_stride + h * D, a.q_stride, rows);
  load_block<D, RI>(sdo, static_cast<const float*>(g.d_out) + t * g.d_out_stride + h * D, g.d_out_stride, rows);
  float dq[RI][S::CPT];
#pragma unroll
  for (int i = 0; i < RI; ++i)
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) dq[i][c] = 0.f;
  const int last = b.row0 + rows - 1, step = parts * PB;
  const int lowest = max(0, b.row0 - window + 1) / PB, first = (lowest + ((part - lowest) & (parts - 1))) * PB;
  auto load = [&](int k0) {
    float* to = kv + (k0 / step & 1) * 2 * BLOCK;
    const int64_t tok = b.t0 + k0;
    load_block<D, RI>(to, static_cast<const float*>(a.k) + tok * a.k_stride + kh * D, a.k_stride, b.len - k0);
    load_block<D, RI>(to + BLOCK, static_cast<const float*>(a.v) + tok * a.v_stride + kh * D, a.v_stride, b.len - k0);
  };
  if (first <= last) load(first);
  loads_sent();
  for (int k0 = first; k0 <= last; k0 += step) {
    const float *sk = kv + (k0 / step & 1) * 2 * BLOCK, *sv = sk + BLOCK;
    if (k0 + step <= last) load(k0 + step);
    loads_sent();
    loads_there<1>();
    __syncthreads();
    tile_grads<D, RI>(a, stats + h * a.T + t, sq, sk, sdo, sv, b.row0, k0, rows, b.len, window, nullptr, sds);
    __syncwarp();
#pragma unroll 2
    for (int j = 0; j < PB; j += 4) {
      float4 w[RI];
#pragma unroll
      for (int i = 0; i < RI; ++i) w[i] = *reinterpret_cast<const float4*>(sds + (ty + PB / RI * i) * S::PLD + j);
      add_rows<D, RI>(dq, w, sk + j * S::LD);
    }
    __syncthreads();
  }
  loads_there<0>();
  add_parts(cluster, kv, dq);
#pragma unroll
  for (int i = 0; i < RI; ++i) {
    const int r = ty + PB / RI * i;
    if (r >= rows || row_owner<RI>(i, parts) != part) continue;
#pragma unroll
    for (int c = 0; c < S::CPT; ++c) dq[i][c] *= a.scale;
    store_row<D>(g.dq, g.bf16, (t + r) * g.dq_stride + h * D, dq[i]);
  }
  if (tid == 0 && part == 0) add_work(a.status, rows);
  if (parts > 1) cluster.sync();
}

// CTAs for a unit (a cluster), up to `most`: twice as many as long as there are tiles for them and all run within `rounds` times 152 CTAs
// of 128 channels, 304 of fewer.  (Shared memory holds one CTA of 128 channels an SM and two of fewer, but one in the gradients of 64: those
// run in up to two fillings, which took less than half as many CTAs in one: 509 tokens, 12 heads, forward and gradients 114 us for 159;
// 2000 tokens, 4 / 2 heads, 360 for 569.)  Both sides: 408 units of up to 23 tiles 194 -> 144 us with
// two CTAs, 420 of 11 tiles as before; 64 prompts of 512 tokens, 12 heads, 776 -> 963.  Gradients of 36 units of 8 query
// heads 1062 -> 347 us with four; 420 units 255 -> 305 with two, hence `rounds` of 1 there.
inline int parts_of(const PromptAttnArgs& a, int64_t units, int most, int rounds) {
  const int64_t slots = 152 * (a.d == 128 ? 1 : 2);
  int parts = 1;
  while (parts < most && parts * PB < a.max_seqlen && units * parts * 2 <= rounds * slots) parts *= 2;
  return parts;
}
template <typename Kernel, typename... Args>
cudaError_t launch_parts(Kernel* kernel, int threads, int64_t units, int parts, int smem, cudaStream_t s, const Args&... args) {
  if (units > 0x7fffffff) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * parts));
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)parts;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = parts > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Rows a thread has (RI).  Those of the queries' kernels: 8 up to 64 channels, in CTAs of 128 threads (512 prompts of 64 tokens, 12 heads of 64:
// forward 656 -> 360 us; 8 of 2048: 1303 -> 1249; the gradients 1392 -> 1246 and as they were), 4 for 128 (32 prompts of 512 tokens:
// forward 795 us, with 8 867).  The keys' kernel has 4: it holds two results, and with 8 took longer (509 tokens' gradients 76 -> 87).
template <int D>
constexpr int pf_rows() { return D == 128 ? 4 : 8; }
constexpr int PF_KEY_ROWS = 4;

template <int D>
cudaError_t forward_launch(const PromptAttnArgs& a, cudaStream_t s) {
  constexpr int RI = pf_rows<D>();
  using S = PfShape<D>;
  const int smem = (5 * PB * S::LD + PB * S::PLD) * 4;
  const int64_t places = pf_places(a.T, a.N, PB);
  return launch_parts(pf_f32_kernel<D, RI>, pf_threads(RI), places * a.Hq, parts_of(a, places * a.Hq, 2, 3), smem, s, a, places);
}

template <int D>
cudaError_t grad_launch(const PromptAttnArgs& a, const PromptGradArgs& g, const float2* stats, cudaStream_t s) {
  using S = PfShape<D>;
  constexpr int RQ = pf_rows<D>(), RK = PF_KEY_ROWS;
  const int smem_kv = ((2 + 2 * kv_buffers(D)) * PB * S::LD + 2 * PB * S::PLD) * 4, smem_q = (6 * PB * S::LD + PB * S::PLD) * 4;
  const int64_t places = pf_places(a.T, a.N, PB);
  const cudaError_t e = launch_parts(pf_f32_grad_kv_kernel<D, RK>, pf_threads(RK), places * a.Hkv, parts_of(a, places * a.Hkv, 4, 1), smem_kv, s, a, g, stats, places);
  if (e != cudaSuccess) return e;
  return launch_parts(pf_f32_grad_q_kernel<D, RQ>, pf_threads(RQ), places * a.Hq, parts_of(a, places * a.Hq, 4, 1), smem_q, s, a, g, stats, places);
}

}  // namespace

cudaError_t pf_f32(const PromptAttnArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 16: return forward_launch<16>(a, s);
    case 32: return forward_launch<32>(a, s);
    case 64: return forward_launch<64>(a, s);
    default: return forward_launch<128>(a, s);
  }
}

cudaError_t pf_f32_grad(const PromptAttnArgs& a, const PromptGradArgs& g, const float2* stats, cudaStream_t s) {
  switch (a.d) {
    case 16: return grad_launch<16>(a, g, stats, s);
    case 32: return grad_launch<32>(a, g, stats, s);
    case 64: return grad_launch<64>(a, g, stats, s);
    default: return grad_launch<128>(a, g, stats, s);
  }
}

}  // namespace kda
