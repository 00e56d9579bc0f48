// Windowed attention: which keys a row sees, and the kernels over whole
// sequences [B, H, N, d].
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace sparge {

// The row at position i sees [lo(i), hi(i, L)) and [0, min(sinks, hi)).
struct Window {
  int left, right, sinks, unit;
  __device__ __forceinline__ int lo(int i) const {
    const int f = i / unit - left;
    return left < 0 || f <= 0 ? 0 : f * unit;
  }
  __device__ __forceinline__ int hi(int i, int L) const {
    if (right < 0) return L;
    const long long e = ((long long)(i / unit) + right + 1) * unit;
    return e < L ? (int)e : L;
  }
};

struct WindowParams {
  const __nv_bfloat16 *Q, *K, *V;
  const int32_t* lens;
  __nv_bfloat16* O;
  float* lse;
  Window w;
  int H, Hkv, N;
  float scale;
  // backward
  const __nv_bfloat16 *O_in, *dO;
  const float* lse_in;
  float* dsum;
  __nv_bfloat16 *dQ, *dK, *dV;
};

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int N) {
  return lens ? min(max(__ldg(lens + b), 0), N) : N;
}

// Forward, one warp per row: lane l holds channels l, l + 32, ...
template <int D>
__global__ void __launch_bounds__(128) window_fwd_simple(const WindowParams p, int64_t rows) {
  constexpr int C = D / 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= rows) return;
  const int lane = threadIdx.x % 32;
  const int i = (int)(row % p.N), h = (int)(row / p.N % p.H), b = (int)(row / p.N / p.H);
  const int L = seq_len(p.lens, b, p.N);
  const int64_t kv0 = ((int64_t)b * p.Hkv + h / (p.H / p.Hkv)) * p.N * D;
  float q[C], o[C] = {}, m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) q[c] = __bfloat162float(p.Q[row * D + c * 32 + lane]);
  const int lo = p.w.lo(i), hi = i < L ? p.w.hi(i, L) : 0, ns = min(min(p.w.sinks, lo), hi);
  for (int t = 0; t < ns + max(hi - lo, 0); ++t) {
    const int64_t at = kv0 + (int64_t)(t < ns ? t : lo + t - ns) * D + lane;
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) s += q[c] * __bfloat162float(p.K[at + c * 32]);
    s = warp_sum(s) * p.scale;
    const float mn = fmaxf(m, s), f = __expf(m - mn), e = __expf(s - mn);
    m = mn;
    l = l * f + e;
#pragma unroll
    for (int c = 0; c < C; ++c) o[c] = o[c] * f + e * __bfloat162float(p.V[at + c * 32]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) p.O[row * D + c * 32 + lane] = __float2bfloat16_rn(l > 0.0f ? o[c] / l : 0.0f);
  if (p.lse && lane == 0) p.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

// dQ and D_i, one warp per row.
template <int D>
__global__ void __launch_bounds__(128) window_dq_simple(const WindowParams p, int64_t rows) {
  constexpr int C = D / 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= rows) return;
  const int lane = threadIdx.x % 32;
  const int i = (int)(row % p.N), h = (int)(row / p.N % p.H), b = (int)(row / p.N / p.H);
  const int L = seq_len(p.lens, b, p.N);
  const int64_t kv0 = ((int64_t)b * p.Hkv + h / (p.H / p.Hkv)) * p.N * D;
  float q[C], g[C], a[C] = {}, di = 0.0f;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    q[c] = __bfloat162float(p.Q[row * D + c * 32 + lane]);
    g[c] = __bfloat162float(p.dO[row * D + c * 32 + lane]);
    di += g[c] * __bfloat162float(p.O_in[row * D + c * 32 + lane]);
  }
  di = warp_sum(di);
  const float lse = p.lse_in[row];
  if (lane == 0) p.dsum[row] = di;
  const int lo = p.w.lo(i), hi = i < L ? p.w.hi(i, L) : 0, ns = min(min(p.w.sinks, lo), hi);
  for (int t = 0; t < ns + max(hi - lo, 0); ++t) {
    const int64_t at = kv0 + (int64_t)(t < ns ? t : lo + t - ns) * D + lane;
    float s = 0.0f, dp = 0.0f;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      s += q[c] * __bfloat162float(p.K[at + c * 32]);
      dp += g[c] * __bfloat162float(p.V[at + c * 32]);
    }
    s = warp_sum(s) * p.scale;
    dp = warp_sum(dp);
    const float ds = __expf(s - lse) * (dp - di);
#pragma unroll
    for (int c = 0; c < C; ++c) a[c] += ds * __bfloat162float(p.K[at + c * 32]);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) p.dQ[row * D + c * 32 + lane] = __float2bfloat16_rn(a[c] * p.scale);
}

// dK and dV, one warp per key, over the rows that may see it.
template <int D>
__global__ void __launch_bounds__(128) window_dkdv_simple(const WindowParams p, int64_t keys) {
  constexpr int C = D / 32;
  const int64_t key = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  if (key >= keys) return;
  const int lane = threadIdx.x % 32;
  const int j = (int)(key % p.N), hk = (int)(key / p.N % p.Hkv), b = (int)(key / p.N / p.Hkv);
  const int L = seq_len(p.lens, b, p.N), G = p.H / p.Hkv;
  float k[C], v[C], dk[C] = {}, dv[C] = {};
#pragma unroll
  for (int c = 0; c < C; ++c) {
    k[c] = __bfloat162float(p.K[key * D + c * 32 + lane]);
    v[c] = __bfloat162float(p.V[key * D + c * 32 + lane]);
  }
  for (int g = 0; g < G && j < L; ++g) {
    const int64_t r0 = ((int64_t)b * p.H + hk * G + g) * p.N;
    for (int i = 0; i < L; ++i) {
      if (j >= p.w.hi(i, L) || (j < p.w.lo(i) && j >= p.w.sinks)) continue;
      const int64_t at = (r0 + i) * D + lane;
      float s = 0.0f, dp = 0.0f, q[C], go[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        q[c] = __bfloat162float(p.Q[at + c * 32]);
        go[c] = __bfloat162float(p.dO[at + c * 32]);
        s += q[c] * k[c];
        dp += go[c] * v[c];
      }
      s = warp_sum(s) * p.scale;
      dp = warp_sum(dp);
      const float pr = __expf(s - p.lse_in[r0 + i]), ds = pr * (dp - p.dsum[r0 + i]);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        dv[c] += pr * go[c];
        dk[c] += ds * q[c];
      }
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    p.dK[key * D + c * 32 + lane] = __float2bfloat16_rn(dk[c] * p.scale);
    p.dV[key * D + c * 32 + lane] = __float2bfloat16_rn(dv[c]);
  }
}

}  // namespace sparge
