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

// 2^(byte - 127), NaN for byte 255 (bytes 10 .. 246 are written; 0 is subnormal).
__device__ __forceinline__ float exp_scale(uint8_t byte) {
  return byte == 255 ? __int_as_float(0x7FC00000) : __uint_as_float(max((uint32_t)byte << 23, 0x400000u));
}

// The power of a row whose largest magnitude is a (finite): the least with
// a <= 448 * 2^power, in [-117, 119]. 448 = 1.75 * 2^8: the power is a's
// exponent - 8, one more where a's mantissa passes 1.75.
__device__ __forceinline__ int e4m3_power(float a) {
  const uint32_t u = __float_as_uint(a);
  const int k = (int)(u >> 23) - 127;
  return min(max(k - ((u & 0x7FFFFFu) > 0x600000u ? 7 : 8), -117), 119);
}

// Both kernels are bound by their bytes. One warp per token and 16 (d = 128) or
// 32 rows of its K and V heads, so that the walk from the packed token to its
// place (sequence, position, page: three loads that wait for one another) is
// made once for them; a lane takes 16 channels, four rows of each in flight.
// 25 k tokens of 12 heads read back: from e4m3 67 us with a thread per 8
// channels, 44 so (230 MB, two thirds of it written: 5.2 TB/s); from bf16 51 us
// (6.0 TB/s).
constexpr int kCacheWarps = 8;  // per block

struct TokenPlace {
  bool live;
  int64_t row;  // of head 0 (cache_row), -1: does not exist
};

__device__ __forceinline__ TokenPlace token_place(const CacheView& c, int t) {
  TokenPlace p{t < min(__ldg(c.cu + c.B), c.tokens), -1};
  if (p.live) {
    const int b = find_seq(c.cu, c.B, t);
    p.row = cache_row(c, b, __ldg(c.first + b) + t - __ldg(c.cu + b));
  }
  return p;
}

template <int D, bool E4M3>
__global__ void __launch_bounds__(kCacheWarps * 32)
    cache_write_kernel(const CacheView c, const __nv_bfloat16* __restrict__ K, int64_t ks,
                       const __nv_bfloat16* __restrict__ V, int64_t vs) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, U = 4;
  const int lane = threadIdx.x % 32, ch = lane % LPR * 16;
  const int t = blockIdx.x * kCacheWarps + threadIdx.x / 32;
  const TokenPlace at = token_place(c, t);
  if (!at.live || at.row < 0) return;
  {
    const int r0 = blockIdx.y * (U * RPS);
    uint4 x[U][2];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPS + lane / LPR, h = r >> 1;  // row r: head r / 2, K then V
      if (h >= c.Hkv) continue;
      const uint4* src =
          reinterpret_cast<const uint4*>(((r & 1) ? V + (int64_t)t * vs : K + (int64_t)t * ks) + h * D + ch);
      x[u][0] = __ldg(src);
      x[u][1] = __ldg(src + 1);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPS + lane / LPR, h = r >> 1;
      const bool here = h < c.Hkv;
      const int64_t row = at.row + ((int64_t)h << c.page_shift);
      if (!E4M3) {
        if (here) {
          uint4* dst = reinterpret_cast<uint4*>(((r & 1) ? c.v : c.k) + (row * D + ch) * 2);
          dst[0] = x[u][0];
          dst[1] = x[u][1];
        }
        continue;
      }
      // Magnitudes of bf16 compare as their bits; 0x7F80 and up are not finite.
      const uint32_t w[8] = {x[u][0].x, x[u][0].y, x[u][0].z, x[u][0].w, x[u][1].x, x[u][1].y, x[u][1].z, x[u][1].w};
      uint32_t top = 0;
      if (here) {
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
      }
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (!here) continue;
      const bool finite = top < 0x7F80u;
      const int e = e4m3_power(__uint_as_float(top << 16));
      const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
      uint32_t code[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t r4 = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t v = w[2 * j + i];
          const float2 f = make_float2(__uint_as_float(v << 16) * inv, __uint_as_float(v & 0xFFFF0000u) * inv);
          r4 |= (uint32_t)__nv_cvt_float2_to_fp8x2(f, __NV_SATFINITE, __NV_E4M3) << (16 * i);
        }
        code[j] = finite ? r4 : 0u;
      }
      *reinterpret_cast<uint4*>(((r & 1) ? c.v : c.k) + row * D + ch) = make_uint4(code[0], code[1], code[2], code[3]);
      if (ch == 0) ((r & 1) ? c.v_exp : c.k_exp)[row] = finite ? (uint8_t)(127 + e) : (uint8_t)255;
    }
  }
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
__global__ void __launch_bounds__(kCacheWarps * 32)
    cache_read_kernel(const CacheView c, __nv_bfloat16* __restrict__ K, __nv_bfloat16* __restrict__ V) {
  constexpr int LPR = D / 16, RPS = 32 / LPR, U = 4;
  const int lane = threadIdx.x % 32, ch = lane % LPR * 16;
  const int t = blockIdx.x * kCacheWarps + threadIdx.x / 32;
  const TokenPlace at = token_place(c, t);
  if (!at.live) return;
  {
    const int r0 = blockIdx.y * (U * RPS);
    uint4 x[U][2];
    uint8_t e[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPS + lane / LPR, h = r >> 1;  // row r: head r / 2, K then V
      x[u][0] = x[u][1] = make_uint4(0, 0, 0, 0);
      e[u] = 0;
      if (h >= c.Hkv || at.row < 0) continue;
      const int64_t row = at.row + ((int64_t)h << c.page_shift);
      const uint8_t* src = ((r & 1) ? c.v : c.k) + (row * D + ch) * (E4M3 ? 1 : 2);
      x[u][0] = *reinterpret_cast<const uint4*>(src);
      if (E4M3) e[u] = ((r & 1) ? c.v_exp : c.k_exp)[row];
      else x[u][1] = *reinterpret_cast<const uint4*>(src + 16);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * RPS + lane / LPR, h = r >> 1;
      if (h >= c.Hkv) continue;
      if (E4M3) {
        const float f = exp_scale(e[u]);
        const uint2 a = decode4(x[u][0].x, f), b = decode4(x[u][0].y, f), d = decode4(x[u][0].z, f),
                    g = decode4(x[u][0].w, f);
        x[u][0] = make_uint4(a.x, a.y, b.x, b.y);
        x[u][1] = make_uint4(d.x, d.y, g.x, g.y);
      }
      uint4* dst = reinterpret_cast<uint4*>(((r & 1) ? V : K) + ((int64_t)t * c.Hkv + h) * D + ch);
      dst[0] = x[u][0];
      dst[1] = x[u][1];
    }
  }
}

}  // namespace sparge
