// Acceptance of drafted tokens against the target's probabilities, and the token that follows the accepted ones.
//
// Draft i (token x, from a distribution q) is accepted when u_i q_i(x) < p_i(x), in exact arithmetic, up to the first that is not.
// Then one token is taken with the last random number r: the least v with w(0) + .. + w(v) > r sum(w), where w is max(p - q, 0)
// at a refused draft's place (p without x for a certain draft; p where nothing is left of it) and p behind the last accepted.
//
// The sums decide a whole number, so they must not depend on their order, and a place that fp32 rounds by 2^-24 would move past
// neighbouring tokens of a large vocabulary.  Probabilities are summed as 64-bit integers, in units of 2^-59: p is cut to whole units, and
// p - q, whose two fp32 terms are cut one by one, is less than two units off (2^-58 a token, 5.2e-13 for 150001; exact where p and
// q are whole units themselves).  Sums up to 31 stay within 64 bits, and any split gives the same result.
//
// One request per cluster of C CTAs of 8 warps, each warp a contiguous piece of the vocabulary.  It reads one row of p and of q
// once, for the sums; then the CTA in whose part the threshold falls reads one warp's piece again (from L2) to find the token.
// Measured: 64 windows of 7 drafts over 150001 tokens 26 to 28 us, where reading the rows takes 11 (odd rows: a token a load); 192 of 3 certain drafts over
// 65536 tokens, bf16, 20 to 24; one of 4 over 32768 tokens 5.7 to 6.3.  Bound by the instructions that make integers of probabilities,
// and in small calls by the chain draft, its probabilities, row, the cluster's sums, token.  Clusters because one CTA a
// request reads a row at its own latency, and partial sums in memory would need a second launch.
#include <cooperative_groups.h>

#include "device.h"
#include "common.cuh"
#include "launch.h"

namespace kda {

namespace {

namespace cg = cooperative_groups;

constexpr int VA_NT = 256, VA_WARPS = VA_NT / 32, VA_MOST = 8;  // threads, warps, CTAs of a cluster at most
constexpr int VA_UNROLL = 8;
constexpr int VA_CTAS = 608;  // CTAs at most, but for one a request: four an SM (192 requests of 65536 tokens: 20.2 us, with up to eight 22.0)
constexpr float VA_SUM = 31.f;

// p >= 0 in units of 2^-59: the mantissa with its leading one at the top of 64 bits, moved down by the exponent.  (CUDA's conversion to
// 64-bit integers runs at a fraction of these instructions' rate here: 64 requests of 150001 tokens took 57 us with it.)
__device__ __forceinline__ unsigned long long units(float p) {
  const uint32_t b = __float_as_uint(p), mantissa = b << 8 | 0x80000000u;
  const int down = 131 - (int)(b >> 23);  // below 0 for 32 and more, which the rough sum refuses
  uint32_t small, high, low;
  asm("shr.u32 %0, %1, %2;" : "=r"(small) : "r"(mantissa), "r"(max(down - 32, 0)));
  asm("shr.u32 %0, %1, %2;" : "=r"(high) : "r"(mantissa), "r"(down));
  asm("shf.r.clamp.b32 %0, %1, %2, %3;" : "=r"(low) : "r"(0), "r"(small), "r"(down));
  return (unsigned long long)high << 32 | low;
}

// A random number, brought into [0, 1).
__device__ __forceinline__ double within(float u) { return u > 0.f ? fmin((double)u, 1.0 - 0x1p-53) : 0.0; }

// What a token weighs.
template <typename In>
struct Weights {
  const In *p, *q;  // q null: no proposal to take off
  int without;      // with no q: a token that weighs nothing, or -1
  // NaN and negative values count as zero
  __device__ __forceinline__ unsigned long long operator()(float pv, float qv) const {
    // p - q is d + e exactly, d its rounding: where d > 0, p is the larger and (p - d) - q has no rounding.  Below 2^-4 e is at most
    // half of d's last place, 2^-29, so that it fits 32 bits in the sums' unit; few tokens of a row are above.
    const float a = fmaxf(pv, 0.f), b = fmaxf(qv, 0.f), d = fmaxf(__fsub_rn(a, b), 0.f);
    if (a >= 0x1p-4f) return a > b ? units(a) - units(b) : 0ull;
    const float e = d > 0.f ? __fsub_rn(__fsub_rn(a, d), b) : 0.f;
    return units(d) + (unsigned long long)(long long)__float2int_rz(__fmul_rn(e, 0x1p59f));
  }
  __device__ __forceinline__ unsigned long long alone(float pv, int v) const { return v != without ? units(fmaxf(pv, 0.f)) : 0ull; }
  __device__ __forceinline__ unsigned long long at(int v) const {
    return q ? (*this)(to_f32(p[v]), to_f32(q[v])) : alone(to_f32(p[v]), v);
  }
};

__device__ __forceinline__ void widen(const uint4& w, float (&f)[4], float) {
  f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y), f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void widen(const uint4& w, float (&f)[8], bf16) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[2 * i] = __uint_as_float(x[i] << 16), f[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
}

// U rounds of 16 bytes a lane, or of a token (which is what unaligned rows allow), from v on.
template <typename In, bool Q, int U, bool WIDE>
__device__ __forceinline__ void add_rounds(const Weights<In>& w, int v, int end, unsigned long long& sum, float& f) {
  constexpr int PER = WIDE ? 16 / sizeof(In) : 1, STEP = 32 * PER;
  v += (threadIdx.x & 31) * PER;
  float p[U][PER], q[U][PER];
  if constexpr (WIDE) {
    uint4 x[U], y[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      x[i] = __ldg(reinterpret_cast<const uint4*>(w.p + v + STEP * i));
      if (Q) y[i] = __ldg(reinterpret_cast<const uint4*>(w.q + v + STEP * i));
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      widen(x[i], p[i], In());
      if (Q) widen(y[i], q[i], In());
    }
  } else {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool there = v + STEP * i < end;
      p[i][0] = there ? to_f32(w.p[v + STEP * i]) : 0.f;
      q[i][0] = Q && there ? to_f32(w.q[v + STEP * i]) : 0.f;
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i)
#pragma unroll
    for (int e = 0; e < PER; ++e) {
      const int at = v + STEP * i + e;
      sum += Q ? w(p[i][e], q[i][e]) : w.alone(p[i][e], at);
      f += fmaxf(p[i][e], 0.f);
    }
}

// Sum of v0 .. v1; also in fp32, where it cannot wrap.
template <typename In, bool Q>
__device__ __forceinline__ unsigned long long warp_sum(const Weights<In>& w, int v0, int v1, float& rough) {
  unsigned long long sum = 0;
  float f = 0.f;
  int v = v0;
  const uintptr_t at = reinterpret_cast<uintptr_t>(w.p + v0) | (Q ? reinterpret_cast<uintptr_t>(w.q + v0) : 0);
  if ((at & 15) == 0) {
    constexpr int STEP = 32 * 16 / sizeof(In);
    for (; v + 4 * STEP <= v1; v += 4 * STEP) add_rounds<In, Q, 4, true>(w, v, v1, sum, f);
    for (; v + STEP <= v1; v += STEP) add_rounds<In, Q, 1, true>(w, v, v1, sum, f);
  }
  for (; v < v1; v += 32 * VA_UNROLL) add_rounds<In, Q, VA_UNROLL, false>(w, v, v1, sum, f);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1) {
    sum += __shfl_xor_sync(0xffffffffu, sum, i);
    f += __shfl_xor_sync(0xffffffffu, f, i);
  }
  rough = f;
  return sum;
}

template <typename In>
__global__ void __launch_bounds__(VA_NT) verify_accept_kernel(const VerifyAcceptArgs a) {
  __shared__ unsigned long long sums[VA_WARPS], scan[VA_WARPS];
  __shared__ float roughs[VA_WARPS];
  __shared__ unsigned long long totals[2][VA_MOST];  // of the cluster's CTAs, by pass
  __shared__ float rough_totals[2][VA_MOST];
  __shared__ int accepted, odd;
  cg::cluster_group cluster = cg::this_cluster();
  cluster.barrier_arrive();  // this CTA has started; waited for before the first store into another's shared memory
  pdl_begin();
  const int C = cluster.num_blocks(), rank = cluster.block_rank(), b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const In* target = static_cast<const In*>(a.target) + (int64_t)b * a.W * a.V;
  const In* proposal = static_cast<const In*>(a.proposal) + (a.proposal ? (int64_t)b * (a.W - 1) * a.V : 0);
  const float* u = a.uniform + (int64_t)b * a.W;
  const int32_t* drafts = a.drafts + (int64_t)b * (a.W - 1);

  int have = a.num_drafts ? __ldg(a.num_drafts + b) : a.W - 1;
  int flags = 0;
  if (have < 0 || have > a.W - 1) have = 0, flags |= KDA_DEV_ACCEPT_OOB;
  if (warp == 0) {
    // a lane tests a draft
    int n = 0;
    bool stray = false;
    for (int i0 = 0; i0 < have; i0 += 32) {
      const int i = i0 + lane;
      bool ok = false, out = false;
      if (i < have) {
        const int x = __ldg(drafts + i);
        out = (unsigned)x >= (unsigned)a.V;
        if (!out) {
          const int64_t at = (int64_t)i * a.V + x;
          // NaN and negative values count as zero, as in the weights
          const double p = fmaxf(to_f32(target[at]), 0.f), q = a.proposal ? fmaxf(to_f32(proposal[at]), 0.f) : 1.f;
          ok = within(__ldg(u + i)) * q < p;  // a product of two fp32 is exact in fp64; the largest number's is q or just below: p >= q decides
        }
      }
      const unsigned not_ok = ~__ballot_sync(0xffffffffu, ok);
      const int run = not_ok ? __ffs(not_ok) - 1 : 32;
      n += run;
      if (run < 32) {
        stray = __shfl_sync(0xffffffffu, out, run);
        break;
      }
    }
    if (lane == 0) accepted = n, odd = stray;
  }
  __syncthreads();
  const int n = accepted;
  const bool refused = n < have, stray = refused && odd != 0;
  if (stray) flags |= KDA_DEV_TOKEN_OOB;

  Weights<In> w{target + (int64_t)n * a.V, nullptr, -1};
  if (refused && !stray) {
    if (a.proposal) w.q = proposal + (int64_t)n * a.V;
    else w.without = __ldg(drafts + n);
  }
  const int piece = ((a.V + C * VA_WARPS - 1) / (C * VA_WARPS) + 255) & ~255;  // of a warp; 16 bytes a lane of either type
  const int64_t first = (int64_t)(rank * VA_WARPS + warp) * piece;
  const int v0 = (int)min((int64_t)a.V, first), v1 = (int)min((int64_t)a.V, first + piece);
  unsigned long long before = 0, total = 0, total_here = 0;
  int again = 0;
  float rough = 0.f;
  for (;;) {
    float f;
    const unsigned long long s = w.q ? warp_sum<In, true>(w, v0, v1, f) : warp_sum<In, false>(w, v0, v1, f);
    if (lane == 0) sums[warp] = s, roughs[warp] = f;
    __syncthreads();
    if (!again) cluster.barrier_wait();  // all have started
    if (tid < C) {  // this CTA's sums to each of the others
      unsigned long long t = 0;
      float r = 0.f;
      for (int i = 0; i < VA_WARPS; ++i) t += sums[i], r += roughs[i];
      *cluster.map_shared_rank(&totals[again][rank], tid) = t;
      *cluster.map_shared_rank(&rough_totals[again][rank], tid) = r;
    }
    cluster.sync();
    before = total = 0, rough = 0.f;
    for (int i = 0; i < C; ++i) {
      if (i < rank) before += totals[again][i];
      total += totals[again][i];
      rough += rough_totals[again][i];
    }
    total_here = totals[again][rank];
    if (total != 0 || (!w.q && w.without < 0)) break;
    w.q = nullptr, w.without = -1;  // nothing is left of the target there: it is taken as it stands
    again = 1;
    __syncthreads();
  }

  const bool usable = total != 0 && rough < VA_SUM;
  if (!usable) flags |= KDA_DEV_PROB_OOB;
  if (rank == 0 && tid == 0) {
    a.accepted[b] = n + 1;
    if (!usable) a.tokens[(int64_t)b * a.W + n] = -1;
    if (flags) flag_status(a.status, flags);
    add_work(a.status, n + 1);
  }
  if (rank == 0)
    for (int i = tid; i < a.W; i += VA_NT)
      if (i != n) a.tokens[(int64_t)b * a.W + i] = i < n ? __ldg(drafts + i) : -1;
  if (!usable) return;

  // the last random number in units of 2^-64, within [0, 1)
  const unsigned long long threshold = __umul64hi((unsigned long long)(within(__ldg(u + a.W - 1)) * 0x1p64), total);
  if (threshold < before || threshold - before >= total_here) return;
  // of this CTA's pieces the one that goes beyond it
  int at = 0;
  unsigned long long sum = before;
  while (at < VA_WARPS - 1 && sum + sums[at] <= threshold) sum += sums[at++];
  // and of its tokens: a thread has a run of them
  const int64_t p0 = (int64_t)(rank * VA_WARPS + at) * piece;
  const int each = piece / VA_NT;
  const int t0 = (int)min((int64_t)a.V, p0 + (int64_t)tid * each), t1 = (int)min((int64_t)a.V, p0 + (int64_t)(tid + 1) * each);
  unsigned long long run = 0;
  for (int v = t0; v < t1; ++v) run += w.at(v);
  unsigned long long upto = run;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const unsigned long long o = __shfl_up_sync(0xffffffffu, upto, i);
    if (lane >= i) upto += o;
  }
  if (lane == 31) scan[warp] = upto;
  __syncthreads();
  for (int i = 0; i < warp; ++i) sum += scan[i];
  sum += upto - run;
  if (threshold < sum || threshold - sum >= run) return;
  int v = t0;
  for (; v < t1 - 1; ++v) {
    sum += w.at(v);
    if (sum > threshold) break;
  }
  a.tokens[(int64_t)b * a.W + n] = v;
}

template <typename In>
cudaError_t accept_launch(const VerifyAcceptArgs& a, int cluster, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * cluster));
  cfg.blockDim = dim3(VA_NT);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_accept_kernel<In>, a);
}

}  // namespace

cudaError_t launch_verify_accept(const VerifyAcceptArgs& a, cudaStream_t s) {
  int cluster = VA_MOST;
  while (cluster > 1 && (int64_t)a.B * cluster > VA_CTAS) cluster >>= 1;
  return a.bf16 ? accept_launch<bf16>(a, cluster, s) : accept_launch<float>(a, cluster, s);
}

}  // namespace kda
