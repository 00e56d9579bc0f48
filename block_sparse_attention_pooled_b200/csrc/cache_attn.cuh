// Attention of new tokens over the paged cache.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "cache.cuh"
#include "window.cuh"

namespace sparge {

struct CacheAttnParams {
  CacheView c;
  Window w;
  const __nv_bfloat16* Q;
  int64_t q_stride;
  __nv_bfloat16* O;
  float* lse;
  int H;
  float scale;
};

// One warp per (token, head): lane l holds channels l, l + 32, ...
template <int D, bool E4M3>
__global__ void __launch_bounds__(128) cache_attn_simple(const CacheAttnParams p) {
  constexpr int C = D / 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, h = (int)(row % p.H);
  const int64_t t = row / p.H;
  if (t >= min(__ldg(p.c.cu + p.c.B), p.c.tokens)) return;
  const int b = find_seq(p.c.cu, p.c.B, (int)t);
  const int c0 = __ldg(p.c.cu + b), first = __ldg(p.c.first + b);
  const int L = first + __ldg(p.c.cu + b + 1) - c0, i = first + (int)t - c0;
  const int hk = h / (p.H / p.c.Hkv);
  float q[C], o[C] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) q[c] = __bfloat162float(p.Q[t * p.q_stride + h * D + c * 32 + lane]);
  const int lo = p.w.lo(i), hi = p.w.hi(i, L), ns = min(min(p.w.sinks, lo), hi);
  for (int k = 0; k < ns + max(hi - lo, 0); ++k) {
    int64_t at = cache_row(p.c, b, k < ns ? k : lo + k - ns);
    if (at < 0) continue;
    at += (int64_t)hk << p.c.page_shift;
    auto val = [&](const uint8_t* x, const uint8_t* e, int c) -> float {
      const int64_t a = at * D + c * 32 + lane;
      if (!E4M3) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(x)[a]);
      const __half_raw hr = __nv_cvt_fp8_to_halfraw(x[a], __NV_E4M3);
      return __half2float(*reinterpret_cast<const __half*>(&hr)) * exp_scale(e[at]);
    };
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) s += q[c] * val(p.c.k, p.c.k_exp, c);
    s = warp_sum(s) * p.scale;
    const float mn = fmaxf(m, s), f = __expf(m - mn), e = __expf(s - mn);
    m = mn;
    l = l * f + e;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = o[c] * f + e * val(p.c.v, p.c.v_exp, c);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) p.O[row * D + c * 32 + lane] = __float2bfloat16_rn(l > 0.0f ? o[c] / l : 0.0f);
  if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace sparge
