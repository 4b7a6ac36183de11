// The softmax's exponential and the scores' tanh cap, in powers of two.
#pragma once

#include "f32x2.cuh"

namespace kda {

namespace {

constexpr float PA_LOG2E = 1.4426950408889634f, PA_LN2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// cap2 * tanh(y) given z = 2 log2(e) y, with cap2 = cap * log2(e).  Where all of a warp's |y| are up to 0.75 (|z| <= PA_NEAR; the prompt's
// forms choose score by score) it is y
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
// The form with the exponential alone: for |z| beyond PA_NEAR, 2e-7 relatively there.
__device__ __forceinline__ float capped_far(float z, float cap2) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(z)));
  return fmaf(-2.f * cap2, r, cap2);
}
__device__ __forceinline__ float capped(float z, float cap2) {
  const float y = z * (0.5f * PA_LN2), u = y * y;
  const float small = cap2 * y * fmaf(u, fmaf(u, fmaf(u, -17.f / 315.f, 2.f / 15.f), -1.f / 3.f), 1.f);
  return fabsf(z) < 0.3f * PA_LOG2E ? small : capped_far(z, cap2);
}

// capped_near for two scores, its coefficients multiplied out to powers of z.  Seven multiplications and
// additions instead of two operations of the exponential's unit.
struct CapPoly {
  float k[6];
  __device__ __forceinline__ explicit CapPoly(float cap2) {
    constexpr float h = 0.5f * PA_LN2, h2 = h * h;
    float w = cap2 * h;
#pragma unroll
    for (int i = 0; i < 6; ++i) k[i] = pa_tanh(i) * w, w *= h2;
  }
  __device__ __forceinline__ float2 operator()(float2 z) const {
    const float2 u = mul2(z, z);
    float2 t = both(k[5]);
#pragma unroll
    for (int i = 4; i >= 0; --i) t = fma2(t, u, both(k[i]));
    return mul2(z, t);
  }
};

// The same for |y| up to 0.35 with four coefficients (1.7e-7 in fp32, fitted likewise), as a polynomial p in the square of the product s that
// y is `per` times: the capped score is s p(s^2).  Two multiplications and additions less, and s p - m is one more that the
// exponential's argument needs anyway.
constexpr float PA_NEARER = 0.35f;
struct CapNearer {
  float k[4];
  __device__ __forceinline__ CapNearer(float cap2, float per) {
    constexpr float c[4] = {1.f, -0.33332664f, 0.13299826f, -0.04914852f};
    float w = cap2 * per;
#pragma unroll
    for (int i = 0; i < 4; ++i) k[i] = c[i] * w, w *= per * per;
  }
  // The coefficients go with per, per^3, .. per^7: caps far below or above the scale leave fp32's range, and so may s^2 under the latter.
  __device__ __forceinline__ bool usable() const {
    bool ok = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) ok = ok && fabsf(k[i]) >= 1.175494351e-38f && fabsf(k[i]) <= 3.402823466e38f;
    return ok;
  }
  __device__ __forceinline__ float2 operator()(float2 s) const {
    const float2 u = mul2(s, s);
    return fma2(fma2(fma2(both(k[3]), u, both(k[2])), u, both(k[1])), u, both(k[0]));
  }
  __device__ __forceinline__ float operator()(float s) const {
    const float u = s * s;
    return fmaf(fmaf(fmaf(k[3], u, k[2]), u, k[1]), u, k[0]);
  }
};

}  // namespace

}  // namespace kda
