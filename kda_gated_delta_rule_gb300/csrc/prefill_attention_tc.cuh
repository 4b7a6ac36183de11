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

// 16 results of a row, from channel c on.
__device__ __forceinline__ void pt_store16(void* base, bool is_bf16, int64_t at, const float (&o)[16]) {
  if (is_bf16) {
    uint4* y = reinterpret_cast<uint4*>(static_cast<bf16*>(base) + at);
    y[0] = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
    y[1] = make_uint4(pack_bf16(o[8], o[9]), pack_bf16(o[10], o[11]), pack_bf16(o[12], o[13]), pack_bf16(o[14], o[15]));
  } else {
    float4* y = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
  }
}

// The same with 32, of which there are `left` (a multiple of 16).
__device__ __forceinline__ void pt_store32(void* base, bool is_bf16, int64_t at, const float (&o)[32], int left) {
  pt_store16(base, is_bf16, at, reinterpret_cast<const float(&)[16]>(o[0]));
  if (left > 16) pt_store16(base, is_bf16, at + 16, reinterpret_cast<const float(&)[16]>(o[16]));
}

// Scores in powers of two, capped; `factor` takes a product to the cap's argument.
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
    for (int i = 0; i < N; ++i) x[i] = make_float2(capped(x[i].x, cap2), capped(x[i].y, cap2));
  }
}

}  // namespace

}  // namespace kda
