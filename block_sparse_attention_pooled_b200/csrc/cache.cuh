// The paged cache of K and V: writing new tokens (bf16, or e4m3 with a power
// of two for each token and head) and reading positions back.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ptx.cuh"

namespace sparge {

struct CacheView {
  uint8_t *k, *v;
  uint8_t *k_exp, *v_exp;
  const int32_t *table, *first, *cu;
  int pages, Hkv, page_shift, B, max_pages, tokens;  // a page holds 1 << page_shift tokens
};

// The sequence that packed token t belongs to (cu ascending, t < cu[B]).
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int t) {
  int lo = 0, hi = B;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Row index (page, head 0, place) * Hkv of position p of sequence b in units
// of (token, head) rows: head h's row is that + h << page_shift; -1 where the
// place does not exist.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, int b, int p) {
  const int col = p >> c.page_shift;
  if (p < 0 || col >= c.max_pages) return -1;
  const int id = __ldg(c.table + (int64_t)b * c.max_pages + col);
  if (id < 0 || id >= c.pages) return -1;
  return (((int64_t)id * c.Hkv) << c.page_shift) + (p & ((1 << c.page_shift) - 1));
}

// 2^(byte - 127), NaN for byte 255 (bytes 10 .. 246 are written).
__device__ __forceinline__ float exp_scale(uint8_t byte) {
  return byte == 255 ? __int_as_float(0x7FC00000) : __uint_as_float((uint32_t)byte << 23);
}

// The power of a row whose largest magnitude is a (finite): the least with
// a <= 448 * 2^power, in [-117, 119]. 448 = 1.75 * 2^8: the power is a's
// exponent - 8, one more where a's mantissa passes 1.75.
__device__ __forceinline__ int e4m3_power(float a) {
  const uint32_t u = __float_as_uint(a);
  const int k = (int)(u >> 23) - 127;
  return min(max(k - ((u & 0x7FFFFFu) > 0x600000u ? 7 : 8), -117), 119);
}

// One thread per 8 channels; the row's threads find its largest magnitude by
// shuffles.
template <int D, bool E4M3>
__global__ void __launch_bounds__(256)
    cache_write_kernel(const CacheView c, const __nv_bfloat16* __restrict__ K, int64_t ks,
                       const __nv_bfloat16* __restrict__ V, int64_t vs) {
  constexpr int TPR = D / 8;
  const int n = min(__ldg(c.cu + c.B), c.tokens);
  const int64_t rows = (int64_t)c.tokens * c.Hkv * 2;
  const int64_t r = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const int c8 = (threadIdx.x % TPR) * 8;
  const int which = (int)(r / c.Hkv & 1), h = (int)(r % c.Hkv);
  const int64_t t = r / c.Hkv / 2;
  const bool live = r < rows && t < n;
  int64_t row = -1;
  uint4 x = make_uint4(0, 0, 0, 0);
  if (live) {
    const int b = find_seq(c.cu, c.B, (int)t);
    row = cache_row(c, b, __ldg(c.first + b) + (int)t - __ldg(c.cu + b));
    const __nv_bfloat16* src = which ? V + t * vs : K + t * ks;
    x = *reinterpret_cast<const uint4*>(src + h * D + c8);
  }
  if (row >= 0) row += (int64_t)h << c.page_shift;
  if (!E4M3) {
    if (row >= 0) *reinterpret_cast<uint4*>((which ? c.v : c.k) + (row * D + c8) * 2) = x;
    return;
  }
  // Magnitudes of bf16 compare as their bits; 0x7F80 and up are not finite.
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
#pragma unroll
  for (int o = TPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (row < 0) return;
  const bool finite = top < 0x7F80u;
  const int e = e4m3_power(__uint_as_float(top << 16));
  const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
  uint32_t code[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t r4 = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t u = w[2 * j + i];
      const float2 f = make_float2(__uint_as_float(u << 16) * inv, __uint_as_float(u & 0xFFFF0000u) * inv);
      r4 |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * i);
    }
    code[j] = finite ? r4 : 0u;
  }
  *reinterpret_cast<uint2*>((which ? c.v : c.k) + row * D + c8) = make_uint2(code[0], code[1]);
  if (c8 == 0) (which ? c.v_exp : c.k_exp)[row] = finite ? (uint8_t)(127 + e) : (uint8_t)255;
}

// 4 codes -> 4 values times s, as two bf16 pairs (exact).
__device__ __forceinline__ uint2 decode4(uint32_t code, float s) {
  uint32_t o[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(code >> (16 * i)), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    o[i] = pack_bf16x2(f.x * s, f.y * s);
  }
  return make_uint2(o[0], o[1]);
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(256)
    cache_read_kernel(const CacheView c, __nv_bfloat16* __restrict__ K, __nv_bfloat16* __restrict__ V) {
  constexpr int TPR = D / 8;
  const int n = min(__ldg(c.cu + c.B), c.tokens);
  const int64_t r = (int64_t)blockIdx.x * (256 / TPR) + threadIdx.x / TPR;
  const int c8 = (threadIdx.x % TPR) * 8;
  const int which = (int)(r / c.Hkv & 1), h = (int)(r % c.Hkv);
  const int64_t t = r / c.Hkv / 2;
  if (t >= n) return;
  const int b = find_seq(c.cu, c.B, (int)t);
  int64_t row = cache_row(c, b, __ldg(c.first + b) + (int)t - __ldg(c.cu + b));
  uint4 x = make_uint4(0, 0, 0, 0);
  if (row >= 0) {
    row += (int64_t)h << c.page_shift;
    const uint8_t* src = which ? c.v : c.k;
    if (E4M3) {
      const float s = exp_scale(__ldg((which ? c.v_exp : c.k_exp) + row));
      const uint2 u = *reinterpret_cast<const uint2*>(src + row * D + c8);
      const uint2 a = decode4(u.x, s), d = decode4(u.y, s);
      x = make_uint4(a.x, a.y, d.x, d.y);
    } else {
      x = *reinterpret_cast<const uint4*>(src + (row * D + c8) * 2);
    }
  }
  *reinterpret_cast<uint4*>((which ? V : K) + (t * c.Hkv + h) * D + c8) = x;
}

}  // namespace sparge
