// What kernels of several roles share: rings of operand slots and bounded waits on their barriers.
#pragma once

#include "tc_ptx.cuh"

namespace kda {

namespace {

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

// The same by a whole warp, which goes on or leaves as one.
__device__ __forceinline__ bool tc_wait_warp(uint64_t* bar, uint32_t parity, int* dead) {
  return __all_sync(0xffffffffu, tc_wait(bar, parity, dead));
}

__device__ __forceinline__ bool tc_give_up(int* dead) {
  *reinterpret_cast<volatile int*>(dead) = 1;
  return false;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

}  // namespace

}  // namespace kda
