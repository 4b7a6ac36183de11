// The paged key/value cache's row kernels: writing tokens into it (quantised where the cache is 8-bit) and reading
// rows back.
//
// Quantisation of a row x:  e = the least integer in [-63, 63] with max|x| <= 448 * 2^e,  c = e4m3(x * 2^-e).
// With max|x| = m * 2^E, 1 <= m < 2, and 448 = 1.75 * 2^8 this is e = E - 8, plus one where m > 1.75: integer
// arithmetic on the maximum's bits.  A power-of-two scale makes the scaling exact, costs no division, and loses
// nothing against the exact ratio max|x| / 448: e4m3 is a floating-point grid, so its relative step is the same
// wherever in [224, 448] the largest channel lands.
//
// Bound by HBM: each row is read once and written once.  A row lies on D/8 lanes (rows8.cuh); a group of lanes takes
// R of the token's 2 Hkv rows (keys, then values) and issues all its loads before the first reduction.
#include "launch.h"
#include <cuda_fp16.h>

#include "rows8.cuh"

namespace kda {

constexpr int KV_NT = 128;

// Two e4m3 codes (the low byte is `lo`'s), round to nearest even, saturating.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// The values of two e4m3 codes (exact in fp16).
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  const __half2 v = *reinterpret_cast<const __half2*>(&h);
  return __half22float2(v);
}

// Scale exponent of a row with maximum magnitude amax (0 for a zero row).
__device__ __forceinline__ int scale_exponent(float amax) {
  if (amax == 0.f) return 0;
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, -63), 63);
}
__device__ __forceinline__ float exp2_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Row index (in [num_pages][Hkv][page_size] order) of head 0 of a slot; heads are page_size rows apart.
__device__ __forceinline__ int64_t slot_row(int64_t slot, const KvCacheArgs& c) {
  int64_t page, off;
  if (slot <= 0xffffffffll) {  // 32-bit division where it suffices
    const uint32_t s = (uint32_t)slot, q = s / (uint32_t)c.page_size;
    page = q;
    off = s - q * (uint32_t)c.page_size;
  } else {
    page = slot / c.page_size;
    off = slot - page * c.page_size;
  }
  return page * c.Hkv * c.page_size + off;
}

template <int D, int R, bool INBF, bool F8>
__global__ void __launch_bounds__(KV_NT) kv_write_kernel(const KvWriteArgs p, int chunks) {
  constexpr int LPR = D / 8, NG = KV_NT / LPR;
  pdl_begin();
  const int lane = threadIdx.x & 31, lr = threadIdx.x % LPR;
  const unsigned gid = blockIdx.x * (unsigned)NG + threadIdx.x / LPR;
  const int64_t t = gid / (unsigned)chunks;
  const int r0 = (int)(gid % (unsigned)chunks) * R;
  const int rows = 2 * p.c.Hkv;
  Raw8<INBF> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    if (t < p.T && r < rows) {
      if (r < p.c.Hkv) load8(raw[i], p.k, t * p.k_stride + r * D + lr * 8);
      else load8(raw[i], p.v, t * p.v_stride + (r - p.c.Hkv) * D + lr * 8);
    } else {
      raw[i] = Raw8<INBF>{};
    }
  }
  const int64_t slot = t < p.T ? __ldg(p.slots + t) : -1;
  const bool beyond = slot >= (int64_t)p.c.num_pages * p.c.page_size;
  if (beyond && lr == 0) flag_status(p.status, KDA_DEV_PAGE_OOB);
  const bool live = slot >= 0 && !beyond;
  const int64_t row0 = live ? slot_row(slot, p.c) : 0;
  int written = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    const bool isk = r < p.c.Hkv, on = live && r < rows;
    const int64_t row = row0 + (int64_t)(isk ? r : r - p.c.Hkv) * p.c.page_size;
    void* pages = isk ? p.c.k_pages : p.c.v_pages;
    float x[8];
    if constexpr (F8) {
      widen8(raw[i], x);
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) amax = fmaxf(amax, fabsf(x[c]));  // fmaxf drops NaN
      const int e = scale_exponent(row_max<LPR>(amax));
      const float inv = exp2_int(-e);
      uint2 codes;
      codes.x = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
      codes.y = e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16;
      if (on) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + row * D + lr * 8) = codes;
        if (lr == 0) (isk ? p.c.k_scales : p.c.v_scales)[row] = exp2_int(e);
      }
    } else {
      if (on) {
        if constexpr (INBF) {
          *reinterpret_cast<uint4*>(static_cast<bf16*>(pages) + row * D + lr * 8) = raw[i].v;
        } else {
          widen8(raw[i], x);
          store8<true>(pages, row * D + lr * 8, x);
        }
      }
    }
    written += on && isk;
  }
  if (p.status) {
    const int n = __reduce_add_sync(0xffffffffu, lr == 0 ? written : 0);
    if (lane == 0) add_work(p.status, n);
  }
}

template <int D, int R, bool F8, bool OUTBF>
__global__ void __launch_bounds__(KV_NT) kv_read_kernel(const KvReadArgs p, int chunks) {
  constexpr int LPR = D / 8, NG = KV_NT / LPR;
  pdl_begin();
  const int lr = threadIdx.x % LPR;
  const unsigned gid = blockIdx.x * (unsigned)NG + threadIdx.x / LPR;
  const int64_t t = gid / (unsigned)chunks;
  const int r0 = (int)(gid % (unsigned)chunks) * R;
  const int rows = 2 * p.c.Hkv;
  if (t >= p.T) return;
  const int64_t slot = __ldg(p.slots + t);
  const bool beyond = slot >= (int64_t)p.c.num_pages * p.c.page_size;
  if (beyond && lr == 0) flag_status(p.status, KDA_DEV_PAGE_OOB);
  const bool live = slot >= 0 && !beyond;
  const int64_t row0 = live ? slot_row(slot, p.c) : 0;
  uint2 codes[R];
  uint4 bits[R];
  float scale[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    const bool isk = r < p.c.Hkv;
    const int64_t row = row0 + (int64_t)(isk ? r : r - p.c.Hkv) * p.c.page_size;
    const void* pages = isk ? p.c.k_pages : p.c.v_pages;
    codes[i] = make_uint2(0, 0);
    bits[i] = make_uint4(0, 0, 0, 0);
    scale[i] = 0.f;
    if (live && r < rows) {
      if constexpr (F8) {
        codes[i] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + row * D + lr * 8);
        scale[i] = (isk ? p.c.k_scales : p.c.v_scales)[row];
      } else {
        bits[i] = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(pages) + row * D + lr * 8);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int r = r0 + i;
    if (r >= rows) break;
    const bool isk = r < p.c.Hkv;
    void* out = isk ? p.k_out : p.v_out;
    const int64_t at = (t * p.c.Hkv + (isk ? r : r - p.c.Hkv)) * D + lr * 8;
    float x[8];
    if constexpr (F8) {
      const float2 a = from_e4m3x2(codes[i].x & 0xffffu), b = from_e4m3x2(codes[i].x >> 16);
      const float2 c = from_e4m3x2(codes[i].y & 0xffffu), d = from_e4m3x2(codes[i].y >> 16);
      x[0] = a.x * scale[i], x[1] = a.y * scale[i], x[2] = b.x * scale[i], x[3] = b.y * scale[i];
      x[4] = c.x * scale[i], x[5] = c.y * scale[i], x[6] = d.x * scale[i], x[7] = d.y * scale[i];
      store8<OUTBF>(out, at, x);
    } else if constexpr (OUTBF) {
      *reinterpret_cast<uint4*>(static_cast<bf16*>(out) + at) = bits[i];
    } else {
      widen8(Raw8<true>{bits[i]}, x);
      store8<false>(out, at, x);
    }
  }
}

namespace {

// Rows per group: one for a few tokens (they spread over the SMs), else four.
inline int kv_rows(int64_t T, int Hkv) { return T * Hkv <= 2048 ? 1 : 4; }

template <int D, int R>
cudaError_t write_r(const KvWriteArgs& a, bool f8, cudaStream_t s) {
  constexpr int NG = KV_NT / (D / 8);
  const int chunks = (2 * a.c.Hkv + R - 1) / R;
  const int64_t blocks = (a.T * chunks + NG - 1) / NG;
  if (blocks * NG > 0x7fffffff) return cudaErrorInvalidValue;
  auto kernel = f8 ? (a.in_bf16 ? kv_write_kernel<D, R, true, true> : kv_write_kernel<D, R, false, true>)
                   : (a.in_bf16 ? kv_write_kernel<D, R, true, false> : kv_write_kernel<D, R, false, false>);
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(KV_NT), 0, s, a, chunks);
}

template <int D, int R>
cudaError_t read_r(const KvReadArgs& a, bool f8, cudaStream_t s) {
  constexpr int NG = KV_NT / (D / 8);
  const int chunks = (2 * a.c.Hkv + R - 1) / R;
  const int64_t blocks = (a.T * chunks + NG - 1) / NG;
  if (blocks * NG > 0x7fffffff) return cudaErrorInvalidValue;
  auto kernel = f8 ? (a.out_bf16 ? kv_read_kernel<D, R, true, true> : kv_read_kernel<D, R, true, false>)
                   : (a.out_bf16 ? kv_read_kernel<D, R, false, true> : kv_read_kernel<D, R, false, false>);
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(KV_NT), 0, s, a, chunks);
}

template <int D>
cudaError_t write_d(const KvWriteArgs& a, bool f8, cudaStream_t s) {
  return kv_rows(a.T, a.c.Hkv) == 1 ? write_r<D, 1>(a, f8, s) : write_r<D, 4>(a, f8, s);
}
template <int D>
cudaError_t read_d(const KvReadArgs& a, bool f8, cudaStream_t s) {
  return kv_rows(a.T, a.c.Hkv) == 1 ? read_r<D, 1>(a, f8, s) : read_r<D, 4>(a, f8, s);
}

}  // namespace

cudaError_t launch_kv_write(const KvWriteArgs& a, cudaStream_t s) {
  switch (a.c.d) {
    case 16: return write_d<16>(a, a.c.e4m3, s);
    case 32: return write_d<32>(a, a.c.e4m3, s);
    case 64: return write_d<64>(a, a.c.e4m3, s);
    default: return write_d<128>(a, a.c.e4m3, s);
  }
}

cudaError_t launch_kv_read(const KvReadArgs& a, cudaStream_t s) {
  switch (a.c.d) {
    case 16: return read_d<16>(a, a.c.e4m3, s);
    case 32: return read_d<32>(a, a.c.e4m3, s);
    case 64: return read_d<64>(a, a.c.e4m3, s);
    default: return read_d<128>(a, a.c.e4m3, s);
  }
}

}  // namespace kda
