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
// R of the token's key rows, or value rows, and issues all its loads before the first reduction.  The groups of a
// CTA take the same rows of consecutive tokens, which lie next to one another in a page: whole sectors of scales and
// runs of 1 KB of codes at D = 128.  65536 tokens x 8 heads x 128, bf16 rows and an e4m3 cache: written in 60.4 us, read in
// 61.7 (6.7 and 6.6 TB/s, 100 and 97 % of the copy rate).
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

// Largest magnitude of a row, over its lanes; NaN left out.  bf16 rows compare as bf16 pairs.
template <int LPR>
__device__ __forceinline__ float row_amax(const Raw8<true>& r) {
  auto mag = [](uint32_t v) {
    v &= 0x7fff7fffu;
    return *reinterpret_cast<__nv_bfloat162*>(&v);
  };
  __nv_bfloat162 m = __hmax2(__hmax2(mag(r.v.x), mag(r.v.y)), __hmax2(mag(r.v.z), mag(r.v.w)));
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) m = __hmax2(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float lo = __low2float(m), hi = __high2float(m);
  return fmaxf(fmaxf(lo, hi), 0.f);  // a row of NaN only: 0
}
template <int LPR>
__device__ __forceinline__ float row_amax(const Raw8<false>& r) {
  float m = fmaxf(fmaxf(fabsf(r.a.x), fabsf(r.a.y)), fmaxf(fabsf(r.a.z), fabsf(r.a.w)));
  m = fmaxf(m, fmaxf(fmaxf(fabsf(r.b.x), fabsf(r.b.y)), fmaxf(fabsf(r.b.z), fabsf(r.b.w))));
  return fmaxf(row_max<LPR>(m), 0.f);
}

// chunks: groups of R heads among the keys, as many again among the values.
template <int D, int R, bool INBF, bool F8>
__global__ void __launch_bounds__(KV_NT) kv_write_kernel(const KvWriteArgs p, unsigned chunks) {
  constexpr int LPR = D / 8, NG = KV_NT / LPR;
  pdl_begin();
  const int lane = threadIdx.x & 31, lr = threadIdx.x % LPR;
  const int64_t t = (int64_t)(blockIdx.x / (2 * chunks)) * NG + threadIdx.x / LPR;
  const unsigned c = blockIdx.x % (2 * chunks);
  const bool isk = c < chunks;
  const int h0 = (int)(isk ? c : c - chunks) * R, H = p.c.Hkv;
  const void* in = isk ? p.k : p.v;
  const int64_t in0 = t * (isk ? p.k_stride : p.v_stride) + h0 * D + lr * 8;
  Raw8<INBF> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (t < p.T && h0 + i < H) load8(raw[i], in, in0 + i * D);
    else raw[i] = Raw8<INBF>{};
  }
  const int64_t slot = t < p.T ? __ldg(p.slots + t) : -1;
  const bool beyond = slot >= (int64_t)p.c.num_pages * p.c.page_size;
  if (beyond && lr == 0) flag_status(p.status, KDA_DEV_PAGE_OOB);
  const bool live = slot >= 0 && !beyond;
  const int64_t row0 = (live ? slot_row(slot, p.c) : 0) + (int64_t)h0 * p.c.page_size;
  void* pages = isk ? p.c.k_pages : p.c.v_pages;
  float* scales = isk ? p.c.k_scales : p.c.v_scales;
  int written = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const bool on = live && h0 + i < H;
    const int64_t row = row0 + (int64_t)i * p.c.page_size;
    if constexpr (F8) {
      const int e = scale_exponent(row_amax<LPR>(raw[i]));
      const float inv = exp2_int(-e);
      float x[8];
      widen8(raw[i], x);
      uint2 codes;
      codes.x = e4m3x2(x[0] * inv, x[1] * inv) | e4m3x2(x[2] * inv, x[3] * inv) << 16;
      codes.y = e4m3x2(x[4] * inv, x[5] * inv) | e4m3x2(x[6] * inv, x[7] * inv) << 16;
      if (on) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pages) + row * D + lr * 8) = codes;
        if (lr == 0) scales[row] = exp2_int(e);
      }
    } else if (on) {
      if constexpr (INBF) {
        *reinterpret_cast<uint4*>(static_cast<bf16*>(pages) + row * D + lr * 8) = raw[i].v;
      } else {
        float x[8];
        widen8(raw[i], x);
        store8<true>(pages, row * D + lr * 8, x);
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
__global__ void __launch_bounds__(KV_NT) kv_read_kernel(const KvReadArgs p, unsigned chunks) {
  constexpr int LPR = D / 8, NG = KV_NT / LPR;
  pdl_begin();
  const int lr = threadIdx.x % LPR;
  const int64_t t = (int64_t)(blockIdx.x / (2 * chunks)) * NG + threadIdx.x / LPR;
  const unsigned c = blockIdx.x % (2 * chunks);
  const bool isk = c < chunks;
  const int h0 = (int)(isk ? c : c - chunks) * R, H = p.c.Hkv;
  if (t >= p.T) return;
  const int64_t slot = __ldg(p.slots + t);
  const bool beyond = slot >= (int64_t)p.c.num_pages * p.c.page_size;
  if (beyond && lr == 0) flag_status(p.status, KDA_DEV_PAGE_OOB);
  const bool live = slot >= 0 && !beyond;
  const int64_t row0 = (live ? slot_row(slot, p.c) : 0) + (int64_t)h0 * p.c.page_size;
  const void* pages = isk ? p.c.k_pages : p.c.v_pages;
  const float* scales = isk ? p.c.k_scales : p.c.v_scales;
  uint2 codes[R];
  Raw8<true> bits[R];
  float scale[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = row0 + (int64_t)i * p.c.page_size;
    codes[i] = make_uint2(0, 0);
    bits[i] = Raw8<true>{};
    scale[i] = 0.f;
    if (live && h0 + i < H) {
      if constexpr (F8) {
        codes[i] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(pages) + row * D + lr * 8);
        scale[i] = scales[row];
      } else {
        load8(bits[i], pages, row * D + lr * 8);
      }
    }
  }
  void* out = isk ? p.k_out : p.v_out;
  const int64_t out0 = (t * H + h0) * D + lr * 8;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (h0 + i >= H) break;
    float x[8];
    if constexpr (F8) {
      const float2 a = from_e4m3x2(codes[i].x & 0xffffu), b = from_e4m3x2(codes[i].x >> 16);
      const float2 cc = from_e4m3x2(codes[i].y & 0xffffu), d = from_e4m3x2(codes[i].y >> 16);
      x[0] = a.x * scale[i], x[1] = a.y * scale[i], x[2] = b.x * scale[i], x[3] = b.y * scale[i];
      x[4] = cc.x * scale[i], x[5] = cc.y * scale[i], x[6] = d.x * scale[i], x[7] = d.y * scale[i];
      store8<OUTBF>(out, out0 + i * D, x);
    } else if constexpr (OUTBF) {
      *reinterpret_cast<uint4*>(static_cast<bf16*>(out) + out0 + i * D) = bits[i].v;
    } else {
      widen8(bits[i], x);
      store8<false>(out, out0 + i * D, x);
    }
  }
}

namespace {

// Rows per group: one for a few tokens (they spread over the SMs), else four.
inline int kv_rows(int64_t T, int Hkv) { return T * Hkv <= 2048 ? 1 : 4; }

template <int D, int R>
cudaError_t write_r(const KvWriteArgs& a, bool f8, cudaStream_t s) {
  constexpr int NG = KV_NT / (D / 8);
  const unsigned chunks = (a.c.Hkv + R - 1) / R;
  const int64_t blocks = (a.T + NG - 1) / NG * 2 * chunks;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  auto kernel = f8 ? (a.in_bf16 ? kv_write_kernel<D, R, true, true> : kv_write_kernel<D, R, false, true>)
                   : (a.in_bf16 ? kv_write_kernel<D, R, true, false> : kv_write_kernel<D, R, false, false>);
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3(KV_NT), 0, s, a, chunks);
}

template <int D, int R>
cudaError_t read_r(const KvReadArgs& a, bool f8, cudaStream_t s) {
  constexpr int NG = KV_NT / (D / 8);
  const unsigned chunks = (a.c.Hkv + R - 1) / R;
  const int64_t blocks = (a.T + NG - 1) / NG * 2 * chunks;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
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
