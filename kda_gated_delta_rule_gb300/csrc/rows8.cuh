// Row access shared by the attention layers' row kernels: a row of D channels is spread over D/8 lanes, eight
// consecutive channels each, so a lane's bf16 share is one 16-byte access and its fp32 share two.
#pragma once

#include "common.cuh"

namespace kda {

// A lane's eight channels as loaded (plain loads: a call may work in place).
template <bool BF>
struct Raw8;
template <>
struct Raw8<true> {
  uint4 v;
};
template <>
struct Raw8<false> {
  float4 a, b;
};

__device__ __forceinline__ void load8(Raw8<true>& r, const void* base, int64_t elem) {
  r.v = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(base) + elem);
}
__device__ __forceinline__ void load8(Raw8<false>& r, const void* base, int64_t elem) {
  const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + elem);
  r.a = p[0];
  r.b = p[1];
}

__device__ __forceinline__ void unpack_bf16x2(uint32_t v, float& lo, float& hi) {
  lo = __uint_as_float(v << 16);
  hi = __uint_as_float(v & 0xffff0000u);
}
__device__ __forceinline__ void widen8(const Raw8<true>& r, float (&x)[8]) {
  unpack_bf16x2(r.v.x, x[0], x[1]);
  unpack_bf16x2(r.v.y, x[2], x[3]);
  unpack_bf16x2(r.v.z, x[4], x[5]);
  unpack_bf16x2(r.v.w, x[6], x[7]);
}
__device__ __forceinline__ void widen8(const Raw8<false>& r, float (&x)[8]) {
  x[0] = r.a.x; x[1] = r.a.y; x[2] = r.a.z; x[3] = r.a.w;
  x[4] = r.b.x; x[5] = r.b.y; x[6] = r.b.z; x[7] = r.b.w;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <bool BF>
__device__ __forceinline__ void store8(void* base, int64_t elem, const float (&x)[8]) {
  if constexpr (BF) {
    *reinterpret_cast<uint4*>(static_cast<bf16*>(base) + elem) =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
  } else {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + elem);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  }
}

// Sum / maximum over the LPR lanes of a row (LPR a power of two, rows aligned to LPR lanes).
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LPR>
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

}  // namespace kda
