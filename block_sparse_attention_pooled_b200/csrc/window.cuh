// Windowed attention: which keys a row sees.
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

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

__device__ __forceinline__ int seq_len(const int32_t* lens, int b, int N) {
  return lens ? min(max(__ldg(lens + b), 0), N) : N;
}

}  // namespace sparge
