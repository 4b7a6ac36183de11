// What the forms of the prompt attention share: where a block of a packed batch's tokens lies, and which keys its rows see.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "softcap.cuh"

namespace kda {

namespace {

constexpr float PF_NONE = -3.402823466e38f;  // a softmax reference that has seen nothing (finite: no -inf - -inf)

// Blocks of `rows` tokens of all sequences, without sums over their lengths: the blocks of sequence i, at most
// ceil(length / rows) of them, lie among the places floor(start_i / rows) + i .. floor(start_i+1 / rows) + i, which
// are its own.  So a batch has floor(T / rows) + N places, some of them empty.
inline int64_t pf_places(int64_t T, int N, int rows) { return T / rows + N; }

struct PfBlock {
  int t0, len;  // the sequence's first token and length; len = 0: an empty place
  int row0;     // the block's first token within the sequence
};

// The block of 1 << SHIFT tokens at `place`; one whole warp asks.  A search with 32 probes at a time: N <= 32 is one load.
template <int SHIFT>
__device__ __forceinline__ PfBlock pf_block(const PromptAttnArgs& a, int64_t place) {
  const int lane = threadIdx.x & 31;
  const int T = (int)a.T;
  int lo = 0, hi = a.N, c0 = 0, c1 = -1;
  PfBlock b{0, 0, 0};
  while (hi > lo) {
    const int step = (hi - lo + 31) >> 5, i = lo + lane * step;
    if (i < hi) c0 = __ldcg(a.cu + i), c1 = __ldcg(a.cu + i + 1);
    const bool ok = i < hi && (int64_t)(max(0, min(T, c0)) >> SHIFT) + i <= place;
    const int n = __popc(__ballot_sync(0xffffffffu, ok));
    if (n == 0) return b;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
    if (step == 1) {
      c0 = __shfl_sync(0xffffffffu, c0, n - 1), c1 = __shfl_sync(0xffffffffu, c1, n - 1);
      break;
    }
  }
  if (c0 < 0 || c1 < c0 || c1 > T || c1 - c0 > a.max_seqlen) return b;
  const int64_t row0 = (place - ((int64_t)(c0 >> SHIFT) + lo)) << SHIFT;
  if (row0 < 0 || row0 >= c1 - c0) return b;  // (below zero only with offsets out of order, where the search may end anywhere)
  b.t0 = c0;
  b.len = c1 - c0;
  b.row0 = (int)row0;
  return b;
}

// The blocks of a batch in the order of how far they lie from their sequence's start: all sequences' last blocks of the longest
// length first.  Where the batch has up to 32 PF_RANKED sequences a warp keeps their lengths and finds block `rank` of that order by
// counting: level L has count(L) = sum_i max(0, blocks_i - L) blocks at L or above.  (Blocks of unlike work in the batch's own
// order end with whatever sequence came first: 16 prompts of 250 to 8000 tokens took 375 us.)
constexpr int PF_RANKED = 8;
template <int SHIFT>
struct PfRanks {
  int t0[PF_RANKED], len[PF_RANKED];
  __device__ __forceinline__ static bool serves(int N) { return N <= 32 * PF_RANKED; }
  __device__ __forceinline__ explicit PfRanks(const PromptAttnArgs& a) {
#pragma unroll
    for (int r = 0; r < PF_RANKED; ++r) {
      const int i = 32 * r + (int)(threadIdx.x & 31);
      t0[r] = len[r] = 0;
      if (32 * r < a.N && i < a.N) {
        const int c0 = __ldcg(a.cu + i), c1 = __ldcg(a.cu + i + 1);
        if (!(c0 < 0 || c1 < c0 || c1 > a.T || c1 - c0 > a.max_seqlen)) t0[r] = c0, len[r] = c1 - c0;
      }
    }
    int most = 1;
#pragma unroll
    for (int r = 0; r < PF_RANKED; ++r) most = max(most, blocks(r));
    level = top = __reduce_max_sync(0xffffffffu, most) - 1, above = 0;
  }
  __device__ __forceinline__ int blocks(int r) const { return (int)(((unsigned)len[r] + (1u << SHIFT) - 1) >> SHIFT); }
  __device__ __forceinline__ int64_t count(int level, int N) const {  // below 2^31 / 128 + N
    int n = 0;
#pragma unroll
    for (int r = 0; r < PF_RANKED; ++r)
      if (32 * r < N) n += max(0, blocks(r) - level);
    return __reduce_add_sync(0xffffffffu, n);
  }
  // Ranks mostly ascend, so the search starts at the level that the last one found (or at the top, where a rank lies above it): steps
  // that double, then halve.
  int level, above, top;  // above = count(level + 1)
  __device__ __forceinline__ PfBlock find(int64_t rank, int N) {
    PfBlock b{0, 0, 0};
    if (rank < above) level = top, above = 0;
    int hi = level + 1, lo = level, step = 1, n_hi = above, n;
    while ((n = (int)count(lo, N)) <= rank) {
      if (lo == 0) return b;
      hi = lo, n_hi = n;
      lo = max(0, lo - step);
      step *= 2;
    }
    while (hi - lo > 1) {  // count(lo) > rank >= count(hi)
      const int mid = (lo + hi) >> 1;
      n = (int)count(mid, N);
      if (n > rank) lo = mid;
      else hi = mid, n_hi = n;
    }
    level = lo, above = n_hi;
    int k = (int)(rank - n_hi);
    bool found = false;
#pragma unroll
    for (int r = 0; r < PF_RANKED; ++r) {
      if (32 * r >= N || found) continue;
      const unsigned mask = __ballot_sync(0xffffffffu, blocks(r) > lo);
      const int n = __popc(mask);
      if (k < n) {
        const unsigned lane = threadIdx.x & 31, below = mask & ((1u << lane) - 1);
        const unsigned it = __ballot_sync(0xffffffffu, (mask >> lane & 1) && __popc(below) == k);
        const int from = __ffs(it) - 1;
        b.t0 = __shfl_sync(0xffffffffu, t0[r], from);
        b.len = __shfl_sync(0xffffffffu, len[r], from);
        found = true;
      }
      k -= n;
    }
    return b;
  }
};
// Block number `rank`, the longest rows first (the farthest from their sequence's start), or, `reversed`, the farthest from its end.
template <int SHIFT>
__device__ __forceinline__ PfBlock pf_ranked(const PromptAttnArgs& a, PfRanks<SHIFT>& ranks, int64_t rank, int64_t places, bool reversed) {
  if (!PfRanks<SHIFT>::serves(a.N)) return pf_block<SHIFT>(a, reversed ? rank : places - 1 - rank);
  PfBlock b = ranks.find(rank, a.N);
  if (b.len > 0) b.row0 = (reversed ? (int)(((unsigned)b.len + (1u << SHIFT) - 1) >> SHIFT) - 1 - ranks.level : ranks.level) << SHIFT;
  if ((unsigned)b.row0 >= (unsigned)b.len) b.len = 0;  // (offsets out of order: their blocks' number may pass 32 bits)
  return b;
}

// (Offsets are read past L1: the gradient's second kernel starts without a wait for the one before.)
// Reports offsets that are out of order or out of range, and sequences beyond max_seqlen; one warp asks.
__device__ __forceinline__ void pf_check_offsets(const PromptAttnArgs& a) {
  bool bad = false;
  for (int i = threadIdx.x & 31; i < a.N; i += 32) {
    const int c0 = __ldcg(a.cu + i), c1 = __ldcg(a.cu + i + 1);
    bad |= c0 < 0 || c1 < c0 || c1 > a.T || c1 - c0 > a.max_seqlen;
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) flag_status(a.status, KDA_DEV_SEQ_OOB);
}

}  // namespace

// The register forms (any head size; prefill_attention_f32.cu) and the tensor-memory ones (prefill_attention_tc.cu,
// prefill_attention_grad_tc.cu).
cudaError_t pf_tc(const PromptAttnArgs& a, cudaStream_t s);
// How many fp32 parts of dk and dv a gradient on the tensor cores adds up (1: none are written), and the gradient.
int pg_parts(int64_t T, int Hq, int Hkv);
cudaError_t pf_tc_grad(const PromptAttnArgs& a, const PromptGradArgs& g, float2* stats, float* parts, cudaStream_t s);
cudaError_t pf_f32(const PromptAttnArgs& a, cudaStream_t s);
cudaError_t pf_f32_grad(const PromptAttnArgs& a, const PromptGradArgs& g, const float2* stats, cudaStream_t s);

}  // namespace kda
