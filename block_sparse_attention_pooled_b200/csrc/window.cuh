// Windowed attention: which keys a row sees.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "ptx.cuh"

namespace sparge {

// The row at position i sees [lo(i), hi(i, L)) and [0, min(sinks, hi)).
struct Window {
  int left, right, sinks, unit;
  __device__ __forceinline__ int unit_of(int i) const { return unit == 1 ? i : i / unit; }
  __device__ __forceinline__ int lo(int i) const {
    if (left < 0) return 0;
    const int f = unit_of(i) - left;
    return f <= 0 ? 0 : f * unit;
  }
  __device__ __forceinline__ int hi(int i, int L) const {
    if (right < 0) return L;
    const long long e = ((long long)unit_of(i) + right + 1) * unit;
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
