// Windowed attention backward on the 5th-generation tensor cores.
//
//   P_ij = exp(s_ij - lse_i), dP_ij = dO_i . v_j, dS_ij = P_ij (dP_ij - D_i)
//   dQ_i = sum_j dS_ij k_j / sqrt(d);  dK_j = sum_i dS_ij q_i / sqrt(d);  dV_j = sum_i P_ij dO_i
//
// Two kernels recompute the scores, one per direction of the sums, so that
// each sum stays in TMEM and no atomics are needed: 7 products of 128 x 128 x d
// per tile pair instead of 5.
//   window_dq_kernel    one CTA per 128 query rows, over their key tiles; forms D_i
//                       and leaves it for the other;
//   window_dkdv_kernel  one CTA per 128 keys (and part of the query tiles),
//                       over the query tiles of all heads that share them.
// Both: 128 x 128 score tiles (a 64-wide tile would be bound by the reads of
// its operands from shared memory), warp 0 producer, warp 1 MMA issuer, warps 4..11 the
// elementwise part: row = TMEM lane, warps 4..7 the tile's first 64 columns,
// warps 8..11 the last.
#pragma once
#include <cuda.h>
#include <cstdint>
#include <cuda_bf16.h>

#include "attn_bwd.cuh"
#include "wattn.cuh"

namespace sparge {

enum : unsigned int {
  kErrWbIn = 0xA00, kErrWbFull, kErrWbEmpty, kErrWbS, kErrWbDp, kErrWbDpFree, kErrWbP, kErrWbDs, kErrWbVecFull,
  kErrWbVecEmpty, kErrWbFinal, kErrWbDrain
};

struct WBwdParams {
  Window w;
  const int32_t* lens;
  const __nv_bfloat16 *O, *dO;
  const float* lse;
  float* dsum;  // [B,H,N] D_i
  __nv_bfloat16 *dQ, *dK, *dV;
  float* part;  // dK/dV of keys whose rows are split: [piece][2][128][D] fp32
  int B, H, Hkv, N;
  int rtiles;                   // 128-row tiles (dQ), 128-key tiles (dK/dV)
  int sink_tiles, sink_pieces;  // dK/dV: the first tiles' rows are in so many pieces
  int pieces;                   // and the other tiles' in so many
  float scale_log2, scale;
};

// In place of D_i: the row sees a single key. (A NaN of no computation.)
constexpr uint32_t kOneKey = 0x7FC05EE1u;

// Rows [lo, hi) that see key j.
__device__ __forceinline__ int key_row_lo(const Window& w, int j) {
  const int f = j / w.unit - w.right;
  return w.right < 0 || f <= 0 ? 0 : f * w.unit;
}
__device__ __forceinline__ int key_row_hi(const Window& w, int j, int L) {
  if (w.left < 0 || j < w.sinks) return L;
  const long long e = ((long long)(j / w.unit) + w.left + 1) * w.unit;
  return e < L ? (int)e : L;
}

// Loads a 128-row tile; where it reaches past the end of its sequence
// (len < N), zeros there, whatever memory holds.
template <int D>
__device__ __forceinline__ bool load_rows(uint32_t dst, uint32_t bar, const CUtensorMap* tm, int row0, int len, int N,
                                          int head, int lane, FixUp& fix, volatile int* abort_flag) {
  if (len < N && row0 + kWTile > len) {
    if (!load_and_zero<D>(dst, tm, row0, head, lane, fix, abort_flag, [&](int r) { return row0 + r >= len; })) return false;
    if (lane == 0) mbar_arrive(bar);
  } else if (lane == 0) {
    mbar_arrive_expect_tx(bar, kWTile * D * 2);
    for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * (kWTile * 128), tm, bar, c * 64, row0, head);
  }
  return true;
}

// D = A B^T over d, both operands [128][D] tiles, K-major.
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint64_t a, uint64_t b) {
  constexpr uint32_t id = idesc_bf16_f32(kWTile, kWTile, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint32_t o = ((kk >> 2) * (kWTile * 128) + (kk & 3) * 32) >> 4;
    mma_ss(d_tmem, a + o, b + o, id, kk > 0 ? 1u : 0u);
  }
}

// The same with A as bf16 pairs in TMEM (D / 2 columns).
template <int D>
__device__ __forceinline__ void mma_rows_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b) {
  constexpr uint32_t id = idesc_bf16_f32(kWTile, kWTile, false, false);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk)
    mma_ts(d_tmem, a_tmem + kk * 8, b + (((kk >> 2) * (kWTile * 128) + (kk & 3) * 32) >> 4), id, kk > 0 ? 1u : 0u);
}

// Row r of a [128][D] tile in shared memory (128-byte swizzle) into TMEM.
template <int D>
__device__ __forceinline__ void row_to_tmem(uint32_t tile, int r, uint32_t taddr) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int ch = 4 * c + k;
      asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(w[4 * k]), "=r"(w[4 * k + 1]), "=r"(w[4 * k + 2]), "=r"(w[4 * k + 3])
                   : "r"(tile + (ch / 8) * (kWTile * 128) + r * 128 + (((ch % 8) ^ (r & 7)) * 16))
                   : "memory");
    }
    tmem_st16(taddr + 16 * c, w);
  }
}

// D (+)= A B over the tile's 128 columns: A bf16 pairs in TMEM, columns 0..63
// of the tile at a_tmem, 64..127 at a_tmem + 64; B a [128][D] tile, MN-major.
template <int D>
__device__ __forceinline__ void mma_cols(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, bool accumulate) {
  constexpr uint32_t id = idesc_bf16_f32(kWTile, D, false, true);
#pragma unroll
  for (int kk = 0; kk < kWTile / 16; ++kk)
    mma_ts(d_tmem, a_tmem + (kk >> 2) * 64 + (kk & 3) * 8, b + kk * 128, id, accumulate || kk > 0 ? 1u : 0u);
}

__device__ __forceinline__ void tmem_ld64(uint32_t taddr, float (&s)[64]) { load_scores(taddr, s); }

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&pk)[32]) {
  tmem_st16(taddr, *reinterpret_cast<const uint32_t(*)[16]>(&pk[0]));
  tmem_st16(taddr + 16, *reinterpret_cast<const uint32_t(*)[16]>(&pk[16]));
  tmem_st_wait();
}

template <int D>
__device__ __forceinline__ void store_zero(__nv_bfloat16* out) {
#pragma unroll
  for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// dQ. TMEM columns: S [0,128), dP [128,256), dQ [256,256+D), Q [384,384+D/2),
// dO [448,448+D/2) (bf16 pairs); dS(t) (bf16 pairs) over dP(t). Q and dO are the
// A operands of every tile's products: from TMEM they are not read from shared
// memory again and again, whose bandwidth bounds this kernel (about 95 of 128
// bytes a clock go through): 96 KB instead of 160 a tile, and their 64 KB become
// ring slots. Issue order: S(t+1) once S(t) is in registers; dQ += dS(t) K(t);
// dP(t+1). While the warps finish dS(t), S(t+1) runs; while they form P(t+1),
// dQ(t) and dP(t+1) do.
// ---------------------------------------------------------------------------
template <int D>
struct WDqSmem {
  static constexpr int NS = D == 128 ? 7 : 10;
  static constexpr int kTileBytes = kWTile * D * 2;
  static constexpr int kOffDot = NS * kTileBytes;  // [2][128] fp32; Q and dO land in the last two slots first
  static constexpr int kOffBar = kOffDot + 1024;
  static constexpr int kBarIn = 0, kBarFull = 1, kBarEmpty = 1 + NS, kBarS = 1 + 2 * NS, kBarDp = 2 + 2 * NS,
                       kBarSFree = 3 + 2 * NS, kBarDs = 4 + 2 * NS, kBarTaken = 5 + 2 * NS, kBarFinal = 6 + 2 * NS,
                       kBarDrain = 7 + 2 * NS, kBarFix = 8 + 2 * NS;
  static constexpr int kNumBars = 9 + 2 * NS;
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffTmem + 16 + 1024;
  static_assert(kBytes <= 227 * 1024);
};

template <int D>
__global__ void __launch_bounds__(kWThreads, 1)
    window_dq_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                     const WBwdParams p) {
  using L = WDqSmem<D>;
  constexpr int NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t sKv = sbase, sQ = sKv + (NS - 2) * L::kTileBytes, sDO = sQ + L::kTileBytes;
  auto bar = [&](int i) { return sbase + L::kOffBar + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sgen + L::kOffTmem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kOffTmem + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  const int BH = p.B * p.H;
  const int bh = blockIdx.x % BH, q0 = (p.rtiles - 1 - (int)(blockIdx.x / BH)) * kWTile;
  const int b = bh / p.H, kvh = b * p.Hkv + (bh % p.H) / (p.H / p.Hkv);
  const int len = seq_len(p.lens, b, p.N);
  KeyTiles kt{0, 0, 0, 0};
  if (q0 < len) kt = key_tiles(p.w.lo(q0), p.w.hi(min(q0 + kWTile, len) - 1, len), p.w.sinks, 0);
  const int T = kt.total;
  // D_i comes from the forward's O, whose rounding to bf16 moves it by up to
  // 2^-8 |dO_i| |O_i|: harmless where O_i is a mean of many values, but of the
  // size of dS where a row sees few keys. So with few key tiles they are gone
  // through twice, first for D_i = sum_j P_ij dP_ij in fp32. Relative error of dQ
  // over 8 x 4000 rows (the roundings of dS and dQ alone: 2.35e-3): 2 keys 4.1e-3
  // -> 2.4e-3, 512 keys 2.53e-3 -> 2.44e-3; from nine tiles on it is below 2.5e-3
  // without. A step of 2 x 8 heads x 2047 tokens that see 511 keys: 62 -> 67 us.
  const bool twice = T <= 8;
  const int U = twice ? 2 * T : T;
  auto key_of = [&](int u) { return kt.key0(u < T ? u : u - T); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar(i), i == L::kBarSFree || i == L::kBarDs || i == L::kBarTaken ? 256 : 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + L::kOffTmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_let_next();
  auto few_registers = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 80;"); };

  if (warp == 0) {
    few_registers();
    if (T > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(L::kBarIn), 2 * L::kTileBytes);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(sQ + c * (kWTile * 128), &tmQ, bar(L::kBarIn), c * 64, q0, bh);
          tma_load_3d(sDO + c * (kWTile * 128), &tmDO, bar(L::kBarIn), c * 64, q0, bh);
        }
      }
      FixUp fix{bar(L::kBarFix), 0};
      int n = 0;
      for (; n < 2 * U; ++n) {  // K(0), V(0), K(1), ...
        const int slot = n % NS;
        const bool ok = n == NS - 2 ? role_wait(bar(L::kBarTaken), 0, kErrWbIn, abort_flag)
                                    : n < NS || role_wait(bar(L::kBarEmpty + slot), (n / NS - 1) & 1, kErrWbEmpty, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (!load_rows<D>(sKv + slot * L::kTileBytes, bar(L::kBarFull + slot), (n & 1) ? &tmV : &tmK, key_of(n >> 1),
                          len, p.N, kvh, lane, fix, abort_flag))
          break;
      }
      if (lane == 0) {
        mbar_wait(bar(L::kBarIn), 0, kErrWbIn);
        for (int i = n > NS ? n - NS : 0; i < n; ++i) mbar_wait(bar(L::kBarFull + i % NS), (i / NS) & 1, kErrWbFull);
      }
    }
  } else if (warp == 1) {
    few_registers();
    const bool leader = elect_one();
    const uint64_t dKv = sdesc_sw128(sKv, 16, 1024), dKvM = sdesc_sw128(sKv, kWTile * 128, 1024);
    auto wait = [&](int i, uint32_t parity, unsigned int site) {
      return __all_sync(0xffffffffu, role_wait(bar(i), parity, site, abort_flag));
    };
    auto slot = [&](int n) { return (uint64_t)(((n % NS) * L::kTileBytes) >> 4); };
    auto full = [&](int n) { return wait(L::kBarFull + n % NS, (n / NS) & 1, kErrWbFull); };
    bool ok = T > 0 && wait(L::kBarTaken, 0, kErrWbIn);
    for (int t = -1; ok && t < U; ++t) {
      const bool more = t + 1 < U;
      const int k = 2 * (t + 1), v = k + 1;
      if (more) {
        ok = full(k) && (t < 0 || wait(L::kBarSFree, t & 1, kErrWbS));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          mma_rows_ts<D>(tmem, tmem + 384, dKv + slot(k));
          mma_commit(bar(L::kBarS));
        }
        __syncwarp();
      }
      if (t >= 0) {
        ok = wait(L::kBarDs, t & 1, kErrWbDs);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          if (t >= U - T) mma_cols<D>(tmem + 256, tmem + 128, dKvM + slot(2 * t), t > U - T);
          mma_commit(bar(L::kBarEmpty + (2 * t) % NS));
          if (!more) mma_commit(bar(L::kBarFinal));
        }
        __syncwarp();
      }
      if (more) {
        ok = full(v);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          mma_rows_ts<D>(tmem + 128, tmem + 448, dKv + slot(v));
          mma_commit(bar(L::kBarDp));
          mma_commit(bar(L::kBarEmpty + v % NS));
        }
        __syncwarp();
      }
    }
    if (leader) mma_commit(bar(L::kBarDrain));
    __syncwarp();
    mbar_wait(bar(L::kBarDrain), 0, kErrWbDrain);
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int wg = (warp - 4) / 4;
    const int r = (warp & 3) * 32 + lane, i = q0 + r;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const bool live = i < len;
    const int at = max(min(i, len - 1), 0);
    const int lo = p.w.lo(at), hi = p.w.hi(at, len);
    const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
    const int64_t row = (int64_t)bh * p.N + i;
    // A row that sees a single key has P = 1 whatever its score, and a gradient of
    // the score that is exactly 0 (dP - D would be rounding noise): its P is left
    // out here (-inf), and a mark in place of D tells the other kernel.
    const bool one = max(hi - lo, 0) + min(min(p.w.sinks, hi), lo) == 1;
    const float nl2 = !live ? 0.0f : one ? -INFINITY : -__ldg(p.lse + row) * 1.4426950408889634f;
    // dO_i . O_i in fp32, 16 rows per warp, a row's 16-byte pieces on neighbouring lanes.
    float* dots = reinterpret_cast<float*>(sgen + L::kOffDot);
    if (!twice) {
      constexpr int LPR = D / 8, RPS = 32 / LPR, U = 16 / RPS;
      const int r0 = (warp - 4) * 16 + lane / LPR;
      const int64_t base = ((int64_t)bh * p.N + q0 + r0) * D + lane % LPR * 8;
      uint4 a[U], g[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = q0 + r0 + u * RPS < len;
        a[u] = in ? __ldg(reinterpret_cast<const uint4*>(p.O + base + u * RPS * D)) : make_uint4(0, 0, 0, 0);
        g[u] = in ? __ldg(reinterpret_cast<const uint4*>(p.dO + base + u * RPS * D)) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t av[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, gv[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          dot = fmaf(__uint_as_float(av[k] << 16), __uint_as_float(gv[k] << 16), dot);
          dot = fmaf(__uint_as_float(av[k] & 0xFFFF0000u), __uint_as_float(gv[k] & 0xFFFF0000u), dot);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
        if (lane % LPR == 0) dots[r0 + u * RPS] = dot;
      }
    }
    auto all_rows = [] { asm volatile("bar.sync 2, 256;" ::: "memory"); };
    // The sum of both groups' shares of a row. The second barrier keeps the next
    // call's shares out until all rows have read these: with one key tile no
    // other wait lies between two calls.
    auto both = [&](float v) {
      dots[128 * wg + r] = v;
      all_rows();
      const float sum = dots[r] + dots[128 + r];
      all_rows();
      return sum;
    };
    all_rows();
    float D_i = twice ? 0.0f : dots[r], more_D = 0.0f;
    all_rows();
    const uint64_t sc2 = f2(p.scale_log2, p.scale_log2), nl = f2(nl2, nl2);
    uint64_t nd2 = f2(-D_i, -D_i);
    // Q and dO into TMEM, one by each group of warps.
    bool ok = true;
    if (T > 0) {
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarIn), 0, kErrWbIn, abort_flag));
      if (ok) {
        row_to_tmem<D>(wg == 0 ? sQ : sDO, r, tmem + (wg == 0 ? 384 : 448) + lane_off);
        tmem_st_wait();
        tc_fence_before();
        fence_async_smem();
        mbar_arrive(bar(L::kBarTaken));
      }
    }
    const uint32_t ts = tmem + 64 * wg + lane_off, tp = tmem + 128 + 64 * wg + lane_off;
    for (int u = 0; u < U; ++u) {
      const int t = u < T ? u : u - T, key0 = kt.key0(t);
      if (u == T) {  // the second time: D_i is known
        D_i = both(more_D);
        nd2 = f2(-D_i, -D_i);
        more_D = 0.0f;
      }
      if (!ok) continue;
      const bool sink = t < kt.ns;
      const bool whole = sink ? key0 + kWTile <= min(kt.cut, all_hi) : key0 >= all_lo && key0 + kWTile <= all_hi;
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarS), u & 1, kErrWbS, abort_flag));
      if (!ok) continue;
      tc_fence_after();
      float s[64], dp[64];
      tmem_ld64(ts, s);
      tc_fence_before();
      mbar_arrive(bar(L::kBarSFree));
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 x = f2_split(fma2(f2(s[2 * j], s[2 * j + 1]), sc2, nl));
        s[2 * j] = ex2_approx(x.x);
        s[2 * j + 1] = ex2_approx(x.y);
      }
      if (!whole) {
        const int c0 = key0 + 64 * wg;
        const int e = (sink ? min(hi, kt.cut) : hi) - c0, a = sink ? 0 : lo - c0, k = p.w.sinks - c0;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t seen = bits_below(e - 32 * c) & (~bits_below(a - 32 * c) | bits_below(k - 32 * c));
#pragma unroll
          for (int j = 0; j < 32; ++j) s[32 * c + j] = (seen >> j) & 1u ? s[32 * c + j] : 0.0f;
        }
      }
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarDp), u & 1, kErrWbDp, abort_flag));
      if (!ok) continue;
      tc_fence_after();
      tmem_ld64(tp, dp);
      uint64_t sum = 0ull;  // of P dP (dP - 0) the first time, of dS the second: what D_i lacks
      uint32_t pk[32];
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        const float2 g = f2_split(add2(f2(dp[2 * j], dp[2 * j + 1]), nd2));
        const float d0 = s[2 * j] * g.x, d1 = s[2 * j + 1] * g.y;
        sum = add2(sum, f2(d0, d1));
        pk[j] = pack_bf16x2(d0, d1);
      }
      const float2 su = f2_split(sum);
      more_D += su.x + su.y;
      if (u >= U - T) tmem_st32(tp, pk);
      tc_fence_before();
      mbar_arrive(bar(L::kBarDs));
    }
    // For the other kernel: D_i with what the sum of dS over the keys (0 but for
    // D_i's error) says it lacks.
    D_i += both(more_D);
    if (wg == 0 && live) p.dsum[row] = one ? __uint_as_float(kOneKey) : D_i;
    if (ok && T > 0) {
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarFinal), 0, kErrWbFinal, abort_flag));
      tc_fence_after();
    }
    // Each group of warps stores half of the channels.
    __nv_bfloat16* out = p.dQ + row * D + wg * (D / 2);
    if (ok && T > 0) store_row<D / 2>(out, tmem + 256 + wg * (D / 2) + lane_off, p.scale, !live, i < p.N);
    else if (i < p.N) store_zero<D / 2>(out);
  } else {
    few_registers();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// dK, dV. Scores transposed (rows = keys): S^T = K Q^T, dP^T = V dO^T, so that
// P^T and dS^T are already the A operands of dV += P^T dO and dK += dS^T Q.
// TMEM columns: S^T [0,128), dP^T [128,256), dV [256,256+D), dK [384,384+D);
// P^T and dS^T (bf16 pairs) over S^T and dP^T. Issue order:
// dV(t); S(t+1); dK(t); dP(t+1): while the warps form P(t+1), the tensor core
// has dK(t) and dP(t+1) to do, and while they form dS(t+1), dV(t+1) and S(t+2).
// Warp 2 brings each query tile's lse and D.
// ---------------------------------------------------------------------------
// Where a piece's sums go, in units of [2][128][D]: the sinks' tiles first.
__device__ __forceinline__ int64_t part_slot(const WBwdParams& p, int kvh, int tile, int piece) {
  const int st = p.sink_tiles;
  if (tile < st) return ((int64_t)kvh * st + tile) * p.sink_pieces + piece;
  const int64_t sinks = p.sink_pieces > 1 ? (int64_t)p.B * p.Hkv * st * p.sink_pieces : 0;
  return sinks + ((int64_t)kvh * (p.rtiles - st) + tile - st) * p.pieces + piece;
}

template <int D>
struct WDkvSmem {
  static constexpr int NS = D == 128 ? 5 : 8;
  static constexpr int kTileBytes = kWTile * D * 2;
  static constexpr int kOffK = 0, kOffV = kTileBytes, kOffRing = 2 * kTileBytes;
  static constexpr int kOffVec = kOffRing + NS * kTileBytes;  // [2][128] fp32, then 128 bits
  static constexpr int kOffBar = kOffVec + 1024 + 16;
  static constexpr int kBarKV = 0, kBarFull = 1, kBarEmpty = 1 + NS, kBarS = 1 + 2 * NS, kBarDp = 2 + 2 * NS,
                       kBarP = 3 + 2 * NS, kBarDs = 4 + 2 * NS, kBarVecFull = 5 + 2 * NS, kBarVecEmpty = 7 + 2 * NS,
                       kBarFinal = 9 + 2 * NS, kBarDrain = 10 + 2 * NS, kBarFix = 11 + 2 * NS;
  static constexpr int kNumBars = 12 + 2 * NS;
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffTmem + 16 + 1024;
  static_assert(kBytes <= 227 * 1024);
};

template <int D>
__global__ void __launch_bounds__(kWThreads, 1)
    window_dkdv_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CUtensorMap tmDO,
                       const WBwdParams p) {
  using L = WDkvSmem<D>;
  constexpr int NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t sK = sbase + L::kOffK, sV = sbase + L::kOffV, sRing = sbase + L::kOffRing;
  float* vec = reinterpret_cast<float*>(sgen + L::kOffVec);
  auto bar = [&](int i) { return sbase + L::kOffBar + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sgen + L::kOffTmem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kOffTmem + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  // The sinks' tiles (all their pieces) come first, then the others.
  const int BHkv = p.B * p.Hkv, G = p.H / p.Hkv;
  const int kvh = blockIdx.x % BHkv, u = blockIdx.x / BHkv, nsink = p.sink_tiles * p.sink_pieces;
  const bool in_sink = u < nsink;
  const int pieces = in_sink ? p.sink_pieces : p.pieces;
  const int tile = in_sink ? u / pieces : p.sink_tiles + (u - nsink) / pieces;
  const int piece = in_sink ? u % pieces : (u - nsink) % pieces;
  const int b = kvh / p.Hkv, h0 = b * p.H + (kvh % p.Hkv) * G;
  const int len = seq_len(p.lens, b, p.N), k0 = tile * kWTile;
  // Query tiles [row0, row0 + 128 nq) of each of the G heads; this CTA's are t0 .. t0 + T - 1.
  int row0 = 0, nq = 0;
  if (k0 < len) {
    const int last = min(k0 + kWTile, len) - 1;
    row0 = key_row_lo(p.w, k0);
    const int end = max(key_row_hi(p.w, last, len), k0 < p.w.sinks ? len : 0);
    nq = max(end - row0 + kWTile - 1, 0) / kWTile;
  }
  const int64_t all = (int64_t)G * nq;
  const int t0 = (int)(all * piece / pieces), T = (int)(all * (piece + 1) / pieces) - t0;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      const bool rows = i == L::kBarP || i == L::kBarDs || i == L::kBarVecEmpty || i == L::kBarVecEmpty + 1;
      mbar_init(bar(i), rows ? 256 : 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sbase + L::kOffTmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  grid_wait();  // for D_i
  grid_let_next();
  auto few_registers = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 80;"); };

  if (warp == 0) {
    few_registers();
    if (T > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(L::kBarKV), 2 * L::kTileBytes);
        for (int c = 0; c < D / 64; ++c) {
          tma_load_3d(sK + c * (kWTile * 128), &tmK, bar(L::kBarKV), c * 64, k0, kvh);
          tma_load_3d(sV + c * (kWTile * 128), &tmV, bar(L::kBarKV), c * 64, k0, kvh);
        }
      }
      FixUp fix{bar(L::kBarFix), 0};
      int n = 0, g = t0 / nq, qt = t0 % nq;
      for (; n < 2 * T; ++n) {  // Q(0), dO(0), Q(1), ...
        const int slot = n % NS;
        const bool ok = n < NS || role_wait(bar(L::kBarEmpty + slot), (n / NS - 1) & 1, kErrWbEmpty, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) break;
        if (!load_rows<D>(sRing + slot * L::kTileBytes, bar(L::kBarFull + slot), (n & 1) ? &tmDO : &tmQ,
                          row0 + qt * kWTile, len, p.N, h0 + g, lane, fix, abort_flag))
          break;
        if ((n & 1) && ++qt == nq) qt = 0, ++g;
      }
      if (lane == 0) {
        mbar_wait(bar(L::kBarKV), 0, kErrWbIn);
        for (int i = n > NS ? n - NS : 0; i < n; ++i) mbar_wait(bar(L::kBarFull + i % NS), (i / NS) & 1, kErrWbFull);
      }
    }
  } else if (warp == 1) {
    few_registers();
    const bool leader = elect_one();
    const uint64_t dK = sdesc_sw128(sK, 16, 1024), dV = sdesc_sw128(sV, 16, 1024);
    const uint64_t dR = sdesc_sw128(sRing, 16, 1024), dRm = sdesc_sw128(sRing, kWTile * 128, 1024);
    auto wait = [&](int i, uint32_t parity, unsigned int site) {
      return __all_sync(0xffffffffu, role_wait(bar(i), parity, site, abort_flag));
    };
    auto slot = [&](int n) { return (uint64_t)(((n % NS) * L::kTileBytes) >> 4); };
    auto full = [&](int n) { return wait(L::kBarFull + n % NS, (n / NS) & 1, kErrWbFull); };
    bool ok = T > 0 && wait(L::kBarKV, 0, kErrWbIn);
    for (int t = -1; ok && t < T; ++t) {
      if (t >= 0) {
        ok = wait(L::kBarP, t & 1, kErrWbP);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          mma_cols<D>(tmem + 256, tmem, dRm + slot(2 * t + 1), t > 0);
          mma_commit(bar(L::kBarEmpty + (2 * t + 1) % NS));
        }
        __syncwarp();
      }
      if (t + 1 < T) {
        ok = full(2 * (t + 1));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          mma_rows<D>(tmem, dK, dR + slot(2 * (t + 1)));
          mma_commit(bar(L::kBarS));
        }
        __syncwarp();
      }
      if (t >= 0) {
        ok = wait(L::kBarDs, t & 1, kErrWbDs);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          mma_cols<D>(tmem + 384, tmem + 128, dRm + slot(2 * t), t > 0);
          mma_commit(bar(L::kBarEmpty + (2 * t) % NS));
          if (t == T - 1) mma_commit(bar(L::kBarFinal));
        }
        __syncwarp();
      }
      if (t + 1 < T) {
        ok = full(2 * (t + 1) + 1);
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          mma_rows<D>(tmem + 128, dV, dR + slot(2 * (t + 1) + 1));
          mma_commit(bar(L::kBarDp));
        }
        __syncwarp();
      }
    }
    if (leader) mma_commit(bar(L::kBarDrain));
    __syncwarp();
    mbar_wait(bar(L::kBarDrain), 0, kErrWbDrain);
  } else if (warp == 2) {
    // Row scalars of each query tile: -lse log2 e, read for P, and -D, read for
    // dS; the next tile's wait in registers. A row past the end gets -inf: its
    // P is 0.
    few_registers();
    int g = T > 0 ? t0 / nq : 0, qt = T > 0 ? t0 % nq : 0;
    float nl[4], nd[4];
    uint32_t one[4];  // rows that see a single key
    auto fetch = [&] {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = row0 + qt * kWTile + 32 * k + lane;
        const int64_t row = (int64_t)(h0 + g) * p.N + i;
        nl[k] = i < len ? -__ldg(p.lse + row) * 1.4426950408889634f : -INFINITY;
        const float D_i = i < len ? __ldcg(p.dsum + row) : 0.0f;
        const bool mark = __float_as_uint(D_i) == kOneKey;
        one[k] = __ballot_sync(0xffffffffu, mark);
        nd[k] = mark ? 0.0f : -D_i;
      }
      if (++qt == nq) qt = 0, ++g;
    };
    if (T > 0) fetch();
    bool ok = true;
    for (int t = 0; ok && t < T; ++t) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ok = ok && (t == 0 || role_wait(bar(L::kBarVecEmpty + h), (t - 1) & 1, kErrWbVecEmpty, abort_flag));
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            vec[128 * h + 32 * k + lane] = h == 0 ? nl[k] : nd[k];
            if (h == 1 && lane == k) reinterpret_cast<uint32_t*>(vec)[256 + k] = one[k];
          }
        }
        __syncwarp();
        if (ok && lane == 0) mbar_arrive(bar(L::kBarVecFull + h));
      }
      if (t + 1 < T) fetch();
    }
  } else if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int wg = (warp - 4) / 4;
    const int r = (warp & 3) * 32 + lane, j = k0 + r;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const bool live = j < len;
    const int at = max(min(j, len - 1), 0);
    const int lo = live ? key_row_lo(p.w, at) : 0, hi = live ? key_row_hi(p.w, at, len) : 0;
    const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
    const uint64_t sc2 = f2(p.scale_log2, p.scale_log2);
    int qt = T > 0 ? t0 % nq : 0;
    bool ok = true;
    for (int t = 0; t < T; ++t) {
      const int c0 = row0 + qt * kWTile + 64 * wg;  // this thread's first query row
      if (++qt == nq) qt = 0;
      const bool whole = c0 >= all_lo && c0 + 64 <= all_hi;
      const float* v = vec + 64 * wg;
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarVecFull), t & 1, kErrWbVecFull, abort_flag)) &&
           __all_sync(0xffffffffu, role_wait(bar(L::kBarS), t & 1, kErrWbS, abort_flag));
      if (!ok) break;
      tc_fence_after();
      float s[64];
      uint32_t pk[32];
      tmem_ld64(tmem + 64 * wg + lane_off, s);
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float4 n4 = *reinterpret_cast<const float4*>(v + 4 * c);
        const float2 x = f2_split(fma2(f2(s[4 * c], s[4 * c + 1]), sc2, f2(n4.x, n4.y)));
        const float2 y = f2_split(fma2(f2(s[4 * c + 2], s[4 * c + 3]), sc2, f2(n4.z, n4.w)));
        s[4 * c] = ex2_approx(x.x);
        s[4 * c + 1] = ex2_approx(x.y);
        s[4 * c + 2] = ex2_approx(y.x);
        s[4 * c + 3] = ex2_approx(y.y);
      }
      mbar_arrive(bar(L::kBarVecEmpty));
      if (!whole) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t seen = bits_below(hi - c0 - 32 * c) & ~bits_below(lo - c0 - 32 * c);
#pragma unroll
          for (int i = 0; i < 32; ++i) s[32 * c + i] = (seen >> i) & 1u ? s[32 * c + i] : 0.0f;
        }
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) pk[i] = pack_bf16x2(s[2 * i], s[2 * i + 1]);
      tmem_st32(tmem + 64 * wg + lane_off, pk);
      tc_fence_before();
      mbar_arrive(bar(L::kBarP));
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarVecFull + 1), t & 1, kErrWbVecFull, abort_flag)) &&
           __all_sync(0xffffffffu, role_wait(bar(L::kBarDp), t & 1, kErrWbDp, abort_flag));
      if (!ok) break;
      tc_fence_after();
      float dp[64];
      tmem_ld64(tmem + 128 + 64 * wg + lane_off, dp);
      const uint2 one = *reinterpret_cast<const uint2*>(vec + 256 + 2 * wg);
      if (one.x | one.y) {
#pragma unroll
        for (int i = 0; i < 64; ++i) s[i] = ((i < 32 ? one.x : one.y) >> (i % 32)) & 1u ? 0.0f : s[i];
      }
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float4 n4 = *reinterpret_cast<const float4*>(v + 128 + 4 * c);
        const float2 x = f2_split(add2(f2(dp[4 * c], dp[4 * c + 1]), f2(n4.x, n4.y)));
        const float2 y = f2_split(add2(f2(dp[4 * c + 2], dp[4 * c + 3]), f2(n4.z, n4.w)));
        pk[2 * c] = pack_bf16x2(s[4 * c] * x.x, s[4 * c + 1] * x.y);
        pk[2 * c + 1] = pack_bf16x2(s[4 * c + 2] * y.x, s[4 * c + 3] * y.y);
      }
      mbar_arrive(bar(L::kBarVecEmpty + 1));
      tmem_st32(tmem + 128 + 64 * wg + lane_off, pk);
      tc_fence_before();
      mbar_arrive(bar(L::kBarDs));
    }
    if (ok && T > 0) {
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarFinal), 0, kErrWbFinal, abort_flag));
      tc_fence_after();
    }
    // The first four warps store dV, the others dK.
    const uint32_t acc = tmem + (wg == 0 ? 256 : 384) + lane_off;
    const float f = wg == 0 ? 1.0f : p.scale;
    if (pieces > 1) {
      const int64_t slot = part_slot(p, kvh, tile, piece);
      float* out = p.part + ((slot * 2 + wg) * kWTile + r) * D;
      if (ok && T > 0) {
        store_row_f32<D>(out, acc, f, !live, true);
      } else {
#pragma unroll
        for (int c = 0; c < D; c += 4) *reinterpret_cast<float4*>(out + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    } else {
      __nv_bfloat16* out = (wg == 0 ? p.dV : p.dK) + ((int64_t)kvh * p.N + j) * D;
      if (ok && T > 0) store_row<D>(out, acc, f, !live, j < p.N);
      else if (j < p.N) store_zero<D>(out);
    }
  } else {
    few_registers();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// dK, dV of the keys whose rows were split: the pieces added in order. One
// thread per four channels of a (K/V head, tile, which, key).
template <int D>
__global__ void __launch_bounds__(256) window_reduce_kernel(const WBwdParams p, int64_t quads) {
  grid_wait();
  constexpr int QD = D / 4;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= quads) return;
  const int c = (int)(i % QD) * 4, r = (int)(i / QD % kWTile), which = (int)(i / QD / kWTile % 2);
  const int ct = (int)(i / QD / kWTile / 2), kvh = ct / p.rtiles, tile = ct % p.rtiles;
  const bool in_sink = tile < p.sink_tiles;
  const int pieces = in_sink ? p.sink_pieces : p.pieces, key = tile * kWTile + r;
  if (pieces <= 1 || key >= p.N) return;
  const int64_t slot = part_slot(p, kvh, tile, 0);
  const float* src = p.part + ((slot * 2 + which) * kWTile + r) * D + c;
  float4 a = *reinterpret_cast<const float4*>(src);
  for (int k = 1; k < pieces; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(src + (int64_t)k * 2 * kWTile * D);
    a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
  }
  __nv_bfloat16* out = (which == 0 ? p.dV : p.dK) + ((int64_t)kvh * p.N + key) * D + c;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
}

}  // namespace sparge
