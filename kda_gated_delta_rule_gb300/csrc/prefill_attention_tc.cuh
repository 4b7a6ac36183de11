// What the tensor-memory forms of the prompt attention share.
#pragma once

#include "prefill_attention.cuh"
#include "tc_roles.cuh"
#include "tmap.h"

namespace kda {

namespace {

constexpr int PT_B = 128;                 // rows of a block, keys of a tile
constexpr int PT_NT = 384;
constexpr int PT_HALF = PT_B * 128;       // bytes of 64 channels of a block or tile
constexpr int PT_TMEM = 512;              // columns: all
constexpr int PT_STALL_AT = 2;            // for tests of the way out (kda_set_test_fault): the tile at which a loader leaves

__host__ __device__ constexpr uint32_t pt_idesc(int n) {  // 128 x n, bf16 operands
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// 128 tokens of one head, from `tok` on, to a slot of D / 64 halves.
template <int D>
__device__ __forceinline__ void pt_load(unsigned char* slot, const CUtensorMap* map, int head, int tok, uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < D / 64; ++c) tc::tma_load_3d(slot + c * PT_HALF, map, c * 64, head, tok, bar);
}

// Units on their way to the roles of a CTA, two places, and the taking over of a CTA that has not started.
struct PtFeed {
  alignas(16) uint4 answer;
  uint64_t full[2], empty[2], taken;
  int asked, heard;
  __device__ __forceinline__ void init(int readers) {
    for (int i = 0; i < 2; ++i) tc::bar_init(&full[i], 1), tc::bar_init(&empty[i], readers);
    tc::bar_init(&taken, 1);
    asked = heard = 0;
  }
  // One thread asks, once before each answer; the whole warp hears it.
  __device__ __forceinline__ void ask() {
    tc::fence_proxy_async();  // the answer before has been read
    tc::take_cta(&answer, &taken);
    ++asked;
  }
  __device__ __forceinline__ bool answered(int* dead, int& id) {
    __syncwarp();
    const int n = heard;
    bool ok = tc_wait(&taken, n & 1, dead);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    id = tc::taken_cta(&answer);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) heard = n + 1;
    __syncwarp();
    return true;
  }
  // On the way out: an answer that has not been heard arrives.
  __device__ __forceinline__ void drain() {
    if (asked > heard) tc::bar_wait(&taken, heard & 1, 1u << 16);
  }
};

// 64 bytes of each of a warp's 32 rows, of which the lane has one row's in w: lanes exchange pieces in fours, so that a store's
// lanes have 64 bytes of eight rows instead of 16 of 32 (a store takes time by the 128-byte lines that it touches: with one row a
// lane the ends of a unit's 256 rows of 64 channels took 2000 cycles of it).  `to`: the first row's place; `rows`, `bytes`: how
// many of the 32 and of the 64 there are.  The whole warp calls.
__device__ __forceinline__ void pt_store64(char* to, int64_t row_bytes, int rows, int bytes, uint32_t (&w)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int b = 1; b < 4; b <<= 1) {
    const bool odd = (lane & b) != 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & b) continue;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t &low = w[4 * c + i], &high = w[4 * (c | b) + i];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? low : high, b);
        if (odd) low = got;
        else high = got;
      }
    }
  }
  // now w[4 i ..] is piece lane % 4 of row i of the lane's four
  const int row = lane & ~3, at = (lane & 3) * 16;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row + i < rows && at < bytes)
      *reinterpret_cast<uint4*>(to + (row + i) * row_bytes + at) = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// 32 results of each of a warp's 32 rows, the first at element `at` of `base`, rows `stride` elements apart; `rows` and `left`: how many
// rows and channels there are.
__device__ __forceinline__ void pt_store32(void* base, bool is_bf16, int64_t at, int64_t stride, int rows, int left, const float (&o)[32]) {
  uint32_t w[16];
  if (is_bf16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) w[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
    pt_store64(static_cast<char*>(base) + at * 2, stride * 2, rows, left * 2, w);
  } else {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(o[16 * half + i]);
      pt_store64(static_cast<char*>(base) + (at + 16 * half) * 4, stride * 4, rows, (left - 16 * half) * 4, w);
    }
  }
}

// What takes a product to the softmax's or the cap's argument; finite, so that a product of zero stays one.
__device__ __forceinline__ float pt_factor(float scale, float per) {
  constexpr float most = 3.402823466e38f;
  return fminf(fmaxf(scale * per, -most), most);
}

// Scores in powers of two, capped; `factor` takes a product to the cap's argument.  Each takes its formula by its own argument; the vote only
// leaves the exponential out where no score of the warp needs it, so that none depends on what the other lanes hold.
template <int N>
__device__ __forceinline__ void pt_cap(float2 (&x)[N], float factor, float cap2) {
  const CapPoly near(cap2);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    x[i] = mul2(x[i], both(factor));
    top = fmaxf(top, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
  }
  if (__all_sync(0xffffffffu, top <= PA_NEAR)) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = near(x[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 y = near(x[i]);
      x[i] = make_float2(fabsf(x[i].x) <= PA_NEAR ? y.x : capped_far(x[i].x, cap2), fabsf(x[i].y) <= PA_NEAR ? y.y : capped_far(x[i].y, cap2));
    }
  }
}

}  // namespace

}  // namespace kda
