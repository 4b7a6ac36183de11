// Per-head RMS norm of queries and keys with the position rotation, and its gradient.
//
// Forward, per row x (one token, one head) with weight w:  y = R(p) (x r w),  r = (mean x^2 + eps)^-1/2.
// Backward, with g = R(p)^T dy and u = x r:  dx = r (g w - u mean(g w u)),  dw = sum over rows of g u.
// R(p) only mixes the two channels of a pair, so its transpose is the rotation by the opposite angle.
//
// Both are bound by HBM (about 10 operations per element against 4 to 6 bytes).  A row lies on D/8 lanes; a
// group of lanes takes R rows of one token, issues all its loads before the first reduction and reads the
// token's angles once for them.  In the rotation the partner channel of the half-split pairing is eight-channel
// aligned (rot is a multiple of 16), so it sits in the same register of another lane: one shuffle per channel;
// neighbouring pairs never leave the lane.
#include "launch.h"
#include "rows8.cuh"

namespace kda {

constexpr int NORM_NT = 128;

// The token's angles as this lane needs them: cos and sin per channel (half-split) or per pair (interleaved,
// entries 0..3).  Lanes past the rotated channels keep cos = 1, sin = 0.
struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ void load_angles(Angles& a, const NormArgs& p, int pos, int lane_in_row) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a.c[i] = 1.f, a.s[i] = 0.f;
  const int c0 = lane_in_row * 8, half = p.rot / 2;
  if (c0 >= p.rot) return;
  if (p.interleaved) {
    const int64_t at = (int64_t)pos * half + c0 / 2;
    const float4 c = __ldg(reinterpret_cast<const float4*>(p.cos + at));
    const float4 s = __ldg(reinterpret_cast<const float4*>(p.sin + at));
    a.c[0] = c.x, a.c[1] = c.y, a.c[2] = c.z, a.c[3] = c.w;
    a.s[0] = s.x, a.s[1] = s.y, a.s[2] = s.z, a.s[3] = s.w;
  } else {
    const int64_t at = (int64_t)pos * half + (c0 < half ? c0 : c0 - half);
    const float sign = c0 < half ? -1.f : 1.f;  // the lower channel of a pair gets -sin, the upper +sin
    const float4* cp = reinterpret_cast<const float4*>(p.cos + at);
    const float4* sp = reinterpret_cast<const float4*>(p.sin + at);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 c = __ldg(cp + i), s = __ldg(sp + i);
      a.c[4 * i] = c.x, a.c[4 * i + 1] = c.y, a.c[4 * i + 2] = c.z, a.c[4 * i + 3] = c.w;
      a.s[4 * i] = sign * s.x, a.s[4 * i + 1] = sign * s.y, a.s[4 * i + 2] = sign * s.z, a.s[4 * i + 3] = sign * s.w;
    }
  }
}

// Turns this lane's eight channels by +angle (sgn = 1) or -angle (sgn = -1).  All lanes of the warp call it.
__device__ __forceinline__ void rotate8(float (&x)[8], const Angles& a, const NormArgs& p, int partner_lane,
                                        float sgn) {
  if (p.rot == 0) return;
  if (p.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float u = x[2 * i], v = x[2 * i + 1], s = sgn * a.s[i];
      x[2 * i] = u * a.c[i] - v * s;
      x[2 * i + 1] = u * s + v * a.c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_sync(0xffffffffu, x[i], partner_lane);
      x[i] = x[i] * a.c[i] + other * (sgn * a.s[i]);
    }
  }
}

// Warp lane that holds the partner channels of this lane's (half-split pairing).
__device__ __forceinline__ int partner_of(const NormArgs& p, int lane, int lane_in_row) {
  const int hl = p.rot / 16;
  if (lane_in_row >= 2 * hl) return lane;
  return lane_in_row < hl ? lane + hl : lane - hl;
}

template <int D, int R, bool INBF, bool OUTBF>
__global__ void __launch_bounds__(NORM_NT) qk_norm_rope_kernel(const NormArgs p, int chunks) {
  constexpr int LPR = D / 8, NG = NORM_NT / LPR;
  const int lane = threadIdx.x & 31, lr = threadIdx.x % LPR;
  const unsigned gid = blockIdx.x * (unsigned)NG + threadIdx.x / LPR;
  const int64_t t = gid / (unsigned)chunks;
  const int h0 = (int)(gid % (unsigned)chunks) * R;
  const int H = p.Hq + p.Hkv;
  bool live = t < p.T;
  Raw8<INBF> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int h = h0 + i;
    if (live && h < H) {
      if (h < p.Hq) load8(raw[i], p.q, t * p.q_stride + h * D + lr * 8);
      else load8(raw[i], p.k, t * p.k_stride + (h - p.Hq) * D + lr * 8);
    } else {
      raw[i] = Raw8<INBF>{};
    }
  }
  Angles ang;
  if (p.rot) {
    const int pos = live ? __ldg(p.positions + t) : 0;
    if ((unsigned)pos >= (unsigned)p.num_positions) {
      if (live && lr == 0) flag_status(p.status, KDA_DEV_POS_OOB);
      live = false;
    } else {
      load_angles(ang, p, pos, lr);
    }
  }
  const int partner = partner_of(p, lane, lr);
  int written = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int h = h0 + i;
    float x[8];
    widen8(raw[i], x);
    float ss = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) ss += x[c] * x[c];
    ss = row_sum<LPR>(ss);
    const float r = rsqrtf(ss * (1.f / D) + p.eps);
    const float* w = h < p.Hq ? p.wq : p.wk;
    const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + lr * 8));
    const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + lr * 8) + 1);
    x[0] *= r * w0.x, x[1] *= r * w0.y, x[2] *= r * w0.z, x[3] *= r * w0.w;
    x[4] *= r * w1.x, x[5] *= r * w1.y, x[6] *= r * w1.z, x[7] *= r * w1.w;
    rotate8(x, ang, p, partner, 1.f);
    if (live && h < H) {
      if (h < p.Hq) store8<OUTBF>(p.q_out, t * p.q_out_stride + h * D + lr * 8, x);
      else store8<OUTBF>(p.k_out, t * p.k_out_stride + (h - p.Hq) * D + lr * 8, x);
      ++written;
    }
  }
  if (p.status) {  // one atomic per warp
    const int n = __reduce_add_sync(0xffffffffu, lr == 0 ? written : 0);
    if (lane == 0) add_work(p.status, n);
  }
}

// Backward.  A fixed number of CTAs (NORM_BWD_CTAS at most) walk the tokens' row chunks; each lane keeps the
// weight gradients of its eight channels in registers over the whole walk, the CTA adds its groups up in shared
// memory in a fixed order, and one row of partial sums per CTA goes to the workspace.
template <int D, int R, bool INBF, bool GBF, bool OUTBF>
__global__ void __launch_bounds__(NORM_NT) qk_norm_rope_bwd_kernel(const NormArgs p, const void* __restrict__ dyq,
                                                                   const void* __restrict__ dyk,
                                                                   float* __restrict__ partial, int chunks) {
  constexpr int LPR = D / 8, NG = NORM_NT / LPR;
  const int lane = threadIdx.x & 31, lr = threadIdx.x % LPR, grp = threadIdx.x / LPR;
  const int H = p.Hq + p.Hkv;
  const int partner = partner_of(p, lane, lr);
  float accq[8] = {}, acck[8] = {};
  int written = 0;
  const int64_t total = p.T * chunks;
  // every group of a warp takes the same number of turns, so the shuffles below stay warp-wide
  for (int64_t base = (int64_t)blockIdx.x * NG; base < total; base += (int64_t)gridDim.x * NG) {
    const int64_t gid = base + grp;
    bool live = gid < total;
    const int64_t t = live ? gid / chunks : 0;
    const int h0 = live ? (int)(gid - t * chunks) * R : 0;
    Raw8<INBF> rx[R];
    Raw8<GBF> rg[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int h = h0 + i;
      if (live && h < p.Hq) {
        load8(rx[i], p.q, t * p.q_stride + h * D + lr * 8);
        load8(rg[i], dyq, (t * p.Hq + h) * D + lr * 8);
      } else if (live && h < H) {
        load8(rx[i], p.k, t * p.k_stride + (h - p.Hq) * D + lr * 8);
        load8(rg[i], dyk, (t * p.Hkv + h - p.Hq) * D + lr * 8);
      } else {
        rx[i] = Raw8<INBF>{};
        rg[i] = Raw8<GBF>{};
      }
    }
    Angles ang;
    if (p.rot) {
      const int pos = live ? __ldg(p.positions + t) : 0;
      if ((unsigned)pos >= (unsigned)p.num_positions) {
        if (live && lr == 0) flag_status(p.status, KDA_DEV_POS_OOB);
        live = false;
      } else {
        load_angles(ang, p, pos, lr);
      }
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int h = h0 + i;
      const bool on = live && h < H, isq = h < p.Hq;
      float x[8], g[8];
      widen8(rx[i], x);
      widen8(rg[i], g);
      rotate8(g, ang, p, partner, -1.f);
      const float* w = isq ? p.wq : p.wk;
      const float4 w0 = __ldg(reinterpret_cast<const float4*>(w + lr * 8));
      const float4 w1 = __ldg(reinterpret_cast<const float4*>(w + lr * 8) + 1);
      const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      float ss = 0.f, dot = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) ss += x[c] * x[c], dot += g[c] * wv[c] * x[c];
      ss = row_sum<LPR>(ss);
      dot = row_sum<LPR>(dot);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const float m = dot * r * (1.f / D);  // mean(g w u)
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const float u = x[c] * r, gu = g[c] * u;
        if (on && isq) accq[c] += gu;
        if (on && !isq) acck[c] += gu;
        x[c] = r * (g[c] * wv[c] - u * m);
      }
      if (on) {
        if (isq) store8<OUTBF>(p.q_out, t * p.q_out_stride + h * D + lr * 8, x);
        else store8<OUTBF>(p.k_out, t * p.k_out_stride + (h - p.Hq) * D + lr * 8, x);
        ++written;
      }
    }
  }
  __shared__ float sum[NG][2][D + 4];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    sum[grp][0][lr * 8 + c] = accq[c];
    sum[grp][1][lr * 8 + c] = acck[c];
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 2 * D; e += NORM_NT) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < NG; ++i) v += sum[i][e / D][e % D];
    partial[(int64_t)blockIdx.x * 2 * D + e] = v;
  }
  if (p.status) {
    const int n = __reduce_add_sync(0xffffffffu, lr == 0 ? written : 0);
    if (lane == 0) add_work(p.status, n);
  }
}

// Adds the CTAs' partial weight gradients: 32 channels per CTA, the partial rows spread over its warps and then
// added in warp order, so the result does not depend on timing.
__global__ void __launch_bounds__(512) qk_norm_weight_grad_kernel(const float* __restrict__ partial, int rows, int D,
                                                                  float* __restrict__ dwq, float* __restrict__ dwk) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float part[16][33];
  const int e = blockIdx.x * 32 + threadIdx.x % 32, w = threadIdx.x / 32;
  float v = 0.f;
  for (int i = w; i < rows; i += 16) v += partial[(int64_t)i * 2 * D + e];
  part[w][threadIdx.x % 32] = v;
  __syncthreads();
  if (w == 0) {
    v = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v += part[i][threadIdx.x];
    if (e < D) dwq[e] = v;
    else dwk[e - D] = v;
  }
}

namespace {

template <int D, int R>
cudaError_t norm_fwd(const NormArgs& a, int64_t blocks, int chunks, cudaStream_t s) {
  const unsigned g = (unsigned)blocks;
  if (a.in_bf16 && a.out_bf16) qk_norm_rope_kernel<D, R, true, true><<<g, NORM_NT, 0, s>>>(a, chunks);
  else if (a.in_bf16) qk_norm_rope_kernel<D, R, true, false><<<g, NORM_NT, 0, s>>>(a, chunks);
  else if (a.out_bf16) qk_norm_rope_kernel<D, R, false, true><<<g, NORM_NT, 0, s>>>(a, chunks);
  else qk_norm_rope_kernel<D, R, false, false><<<g, NORM_NT, 0, s>>>(a, chunks);
  return cudaGetLastError();
}

template <int D>
cudaError_t norm_fwd_d(const NormArgs& a, cudaStream_t s) {
  constexpr int NG = NORM_NT / (D / 8);
  const int H = a.Hq + a.Hkv;
  // Few rows: one per group, so that they spread over the SMs.  Otherwise four, for loads in flight and one
  // read of the angles.
  const int R = a.T * H <= 4096 ? 1 : 4;
  const int chunks = (H + R - 1) / R;
  const int64_t blocks = (a.T * chunks + NG - 1) / NG;
  if (a.T > 0x7fffffff || blocks * NG > 0x7fffffff) return cudaErrorInvalidValue;
  return R == 1 ? norm_fwd<D, 1>(a, blocks, chunks, s) : norm_fwd<D, 4>(a, blocks, chunks, s);
}

template <int D, int R>
cudaError_t norm_bwd(const NormArgs& a, const void* dyq, const void* dyk, bool g_bf16, float* partial, int ctas,
                     int chunks, cudaStream_t s) {
  const int sel = (a.in_bf16 ? 4 : 0) | (g_bf16 ? 2 : 0) | (a.out_bf16 ? 1 : 0);
  switch (sel) {
#define KDA_CASE(n, i, g, o)                                                                             \
  case n: qk_norm_rope_bwd_kernel<D, R, i, g, o><<<ctas, NORM_NT, 0, s>>>(a, dyq, dyk, partial, chunks); \
    break;
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
  return cudaGetLastError();
}

template <int D>
cudaError_t norm_bwd_d(const NormArgs& a, const void* dyq, const void* dyk, bool g_bf16, float* dwq, float* dwk,
                       float* partial, cudaStream_t s) {
  constexpr int NG = NORM_NT / (D / 8), R = 2;
  const int chunks = (a.Hq + a.Hkv + R - 1) / R;
  const int64_t need = (a.T * chunks + NG - 1) / NG;
  const int ctas = (int)(need < NORM_BWD_CTAS ? need : NORM_BWD_CTAS);
  if (ctas > 0) {  // without tokens the weights' gradients are zero
    const cudaError_t e = norm_bwd<D, R>(a, dyq, dyk, g_bf16, partial, ctas, chunks, s);
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(qk_norm_weight_grad_kernel, dim3(2 * D / 32), dim3(512), 0, s, (const float*)partial, ctas, D, dwq,
                    dwk);
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
