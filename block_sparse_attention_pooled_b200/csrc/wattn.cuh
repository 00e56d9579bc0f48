// Windowed attention forward on the 5th-generation tensor cores, over whole
// sequences (cache_chunk.cuh has the same over the paged cache).
//
//   O_i = sum_j softmax_j(q_i . k_j / sqrt(d)) v_j over the keys visible to i,
// in one pass over the keys with a running maximum and sum per row.
//
// A CTA per work item of 256 rows (two 128-row tiles A and B) of one head; the
// one on each SM goes on with the items of CTAs that have not started. It walks
// the 128-key tiles that any of the rows may see: the sinks below the window,
// then the window. Roles:
//   warp 0       producer: Q, then K and V tiles into a ring, by TMA; a tile
//                that reaches past the sequence's end gets zeros in the rows
//                that do not exist, so that what memory holds there never meets
//                a probability of 0;
//   warp 1       MMA issuer and TMEM owner;
//   warps 4..7   softmax of tile A: one row (TMEM lane) per thread;
//   warps 8..11  softmax of tile B.
// The two tiles alternate: while the tensor core works on one tile's products,
// the other tile's softmax runs. Issue order per key tile:
//   O_A += P_A(t) V(t); S_A(t+1) = Q_A K(t+1)^T; O_B += P_B(t) V(t); S_B(t+1).
// The products complete in order, so "S(t+1) is there" also says that O(t) is,
// and a row may be rescaled without a wait of its own. A key tile that none of
// a row tile's rows see (the window's ends) is left out for that row tile.
// TMEM columns: S_A [0,128), S_B [128,256), O_A [256,256+D), O_B [384,384+D);
// P(t) (bf16, two per column) lies over the first 64 columns of its S(t).
#pragma once
#include <cuda.h>
#include <cstdint>
#include <cuda_bf16.h>

#include "attn.cuh"
#include "cache_sched.cuh"
#include "ptx.cuh"
#include "window.cuh"

namespace sparge {

enum : unsigned int {
  kErrWinQ = 0x900, kErrWinQEmpty, kErrWinKvFull, kErrWinKvEmpty, kErrWinS, kErrWinP, kErrWinO, kErrWinOFree,
  kErrWinDrain, kErrWinFix, kErrWinNext
};

constexpr int kWTile = 128;       // rows per tile and keys per tile
constexpr int kWThreads = 384;

struct WAttnParams {
  Window w;
  const int32_t* lens;  // whole sequences: [B] or null
  __nv_bfloat16* O;
  float* lse;
  int B, H, Hkv, N, rtiles;
  float scale_log2;
};

template <int D>
struct WSmem {
  static constexpr int NS = D == 128 ? 5 : 8;
  static constexpr int kTileBytes = kWTile * D * 2;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKv = 2 * kTileBytes;
  static constexpr int kOffBar = kOffKv + NS * kTileBytes;
  static constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarKvFull = 2, kBarKvEmpty = 2 + NS, kBarS = 2 + 2 * NS,
                       kBarP = 4 + 2 * NS, kBarP2 = 6 + 2 * NS, kBarO = 8 + 2 * NS, kBarOFree = 10 + 2 * NS,
                       kBarDrain = 12 + 2 * NS, kBarFix = 13 + 2 * NS, kBarNext = 14 + 2 * NS, kBarNextRead = 16 + 2 * NS;
  static constexpr int kNumBars = 18 + 2 * NS;
  static constexpr int kOffNext = kOffBar + kNumBars * 8;  // two answers of 16 bytes
  static constexpr int kOffTmem = kOffNext + 32;
  static constexpr int kBytes = kOffTmem + 16 + 1024;
};

// Zeros in the rows of a [128][D] tile (64-column boxes, 128-byte swizzle) for
// which bad(r), by a warp's lanes, after its loads have landed and before the
// tensor core may read it: memory may hold NaN in places that no row sees, and
// 0 * NaN is not 0. (Loading such a tile by the lanes instead took 12 us, 24
// through a page table, which was most of a short call.)
template <int D, typename Bad>
__device__ __forceinline__ void zero_rows(uint32_t dst, int lane, Bad bad) {
  constexpr int CH = D / 8;  // 16-byte pieces per row; a row's all go, so the swizzle does not matter
  const int c = lane % CH;
  const uint32_t box = dst + (c / 8) * (kWTile * 128) + (c % 8) * 16;
  for (int r = lane / CH; r < kWTile; r += 32 / CH)
    if (bad(r)) asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(box + r * 128), "r"(0) : "memory");
  fence_async_smem();
  __syncwarp();
}

// A producer warp's way to such tiles: their loads land on a barrier of its own.
struct FixUp {
  uint32_t bar;
  uint32_t phase;
};

template <int D, typename Bad>
__device__ __forceinline__ bool load_and_zero(uint32_t dst, const CUtensorMap* tm, int row0, int head, int lane, FixUp& fix,
                                              volatile int* abort_flag, Bad bad) {
  if (lane == 0) {
    mbar_arrive_expect_tx(fix.bar, kWTile * D * 2);
    for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * (kWTile * 128), tm, fix.bar, c * 64, row0, head);
  }
  const bool ok = role_wait(fix.bar, fix.phase & 1, kErrWinFix, abort_flag);
  ++fix.phase;
  if (!__all_sync(0xffffffffu, ok)) return false;
  zero_rows<D>(dst, lane, bad);
  return true;
}

using KeyTiles = KeyTilesT<kWTile>;

__device__ __forceinline__ KeyTiles key_tiles(int lo, int hi, int sinks, int align_mask) {
  return key_tiles_of<kWTile>(lo, hi, sinks, align_mask);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&r)[32]) {
  uint32_t v[2][16];
  tmem_ld16(taddr, v[0]);
  tmem_ld16(taddr + 16, v[1]);
#pragma unroll
  for (int j = 0; j < 32; ++j) r[j] = __uint_as_float(v[j / 16][j % 16]);
}

// 32 bytes to global memory: in one piece where `wide` (the address is a
// multiple of 32; a warp's rows then fill whole sectors), else in two.
__device__ __forceinline__ void store32(void* dst, const uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                 "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}
__device__ __forceinline__ bool is_wide(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

// A row of D accumulator columns times f, as bf16.
template <int D>
__device__ __forceinline__ void store_row(__nv_bfloat16* out, uint32_t taddr, float f, bool zero, bool store) {
  const bool wide = is_wide(out);
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_ld32(taddr + c, o);
    tmem_ld_wait();
    if (store) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = zero ? 0u : pack_bf16x2(o[16 * h + 2 * j] * f, o[16 * h + 2 * j + 1] * f);
        store32(out + c + 16 * h, w, wide);
      }
    }
  }
}

// The same in fp32 (out: a multiple of 32 bytes).
template <int D>
__device__ __forceinline__ void store_row_f32(float* out, uint32_t taddr, float f, bool zero, bool store) {
#pragma unroll 1
  for (int c = 0; c < D; c += 32) {
    float o[32];
    tmem_ld32(taddr + c, o);
    tmem_ld_wait();
    if (store) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = zero ? 0u : __float_as_uint(o[8 * h + j] * f);
        store32(out + c + 8 * h, w, true);
      }
    }
  }
}

// Bits 0 .. n - 1 (n at most 0: none, 32 or more: all).
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n >= 32 ? 0xFFFFFFFFu : n <= 0 ? 0u : (1u << n) - 1u;
}

// 2^(s scale - ref) -> P (bf16 pairs) over the scores' columns; the row's sum.
// half() runs when the first 64 keys' P is in TMEM. All exponentials go to the
// MUFU: a polynomial on the FMA pipe for a quarter of them measured 3% slower
// (480p frames: 1094 against 1062 us), half of them 10%.
template <typename Half>
__device__ __forceinline__ float exp_store(const float (&s)[kWTile], uint32_t ts, float scale_log2, float ref, Half half) {
  const uint64_t scale2 = f2(scale_log2, scale_log2), negm2 = f2(-ref, -ref);
  uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t pk[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float2 x = f2_split(fma2(f2(s[32 * c + 2 * j], s[32 * c + 2 * j + 1]), scale2, negm2));
      const uint64_t ex = f2(ex2_approx(x.x), ex2_approx(x.y));
      acc[j & 3] = add2(acc[j & 3], ex);
      const float2 ev = f2_split(ex);
      pk[j] = pack_bf16x2(ev.x, ev.y);
    }
    tmem_st16(ts + 16 * c, pk);
    if (c == 1) {
      tmem_st_wait();
      half();
    }
  }
  const float2 t = f2_split(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])));
  tmem_st_wait();
  return t.x + t.y;
}

// One softmax step of a row: 128 scores at taddr -> P (bf16 pairs) over them.
// [a, e): the row's window relative to the tile, k: its sinks relative to it;
// `whole`: every key of the tile is visible to every row of the warp; gone: a
// bit for each 16 keys that do not exist.
template <int D, typename Half>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, bool first, bool whole, int a, int e, int k,
                                             float scale_log2, float& m_run, float& l_run, uint32_t gone,
                                             Half half) {
  float s[kWTile];
  {
    uint32_t v[8][16];
#pragma unroll
    for (int c = 0; c < 8; ++c) tmem_ld16(ts + 16 * c, v[c]);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
      for (int j = 0; j < 16; ++j) s[16 * c + j] = __uint_as_float(v[c][j]);
  }
  if (!whole) {
    // One bit per key, 32 at a time: tests of single bits compile to selects,
    // not to branches.
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t seen = bits_below(e - 32 * c) & (~bits_below(a - 32 * c) | bits_below(k - 32 * c));
      seen &= ~(((gone >> (2 * c)) & 1u ? 0xFFFFu : 0u) | ((gone >> (2 * c + 1)) & 1u ? 0xFFFF0000u : 0u));
#pragma unroll
      for (int j = 0; j < 32; ++j) s[32 * c + j] = (seen >> j) & 1u ? s[32 * c + j] : -INFINITY;
    }
  }
  float m8[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    m8[j] = fmaxf(s[j], s[8 + j]);
#pragma unroll
    for (int i = 2; i < 16; i += 2) m8[j] = fmax3(m8[j], s[8 * i + j], s[8 * i + 8 + j]);
  }
  const float top = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
  const float m_new = fmaxf(m_run, top * scale_log2);
  if (first) {
    m_run = m_new;
  } else if (__any_sync(0xffffffffu, m_new > m_run + kRescaleThreshold)) {
    // O and l hold sums of 2^(s - m_run): move them to the new reference. The
    // TMEM access is the warp's, so all its rows move (by 1 where the maximum
    // held; a row that has seen nothing has 0 to move).
    const float f = m_new == -INFINITY ? 1.0f : ex2_approx(m_run - m_new);
    rescale_row<D>(to, f);
    l_run *= f;
    m_run = m_new;
  }
  const float ref = m_run == -INFINITY ? 0.0f : m_run;
  l_run += exp_store(s, ts, scale_log2, ref, half);
}

template <int D>
__global__ void __launch_bounds__(kWThreads, 1)
    window_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                      const __grid_constant__ CUtensorMap tmV, const WAttnParams p) {
  using L = WSmem<D>;
  constexpr int NS = L::NS;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t sQ = sbase + L::kOffQ, sKv = sbase + L::kOffKv;
  auto bar = [&](int i) { return sbase + L::kOffBar + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sgen + L::kOffTmem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kOffTmem + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      const bool rows = (i >= L::kBarP && i < L::kBarP + 4) || (i >= L::kBarOFree && i < L::kBarOFree + 2);
      mbar_init(bar(i), rows ? 128 : i >= L::kBarNextRead && i < L::kBarNextRead + 2 ? 10 : 1);
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
  // The block's registers (384 x 168) are shared out anew: the first four
  // warps keep 80 each, so that the softmax's eight can hold a row's 128 scores.
  auto few_registers = [] { asm volatile("setmaxnreg.dec.sync.aligned.u32 80;"); };

  // The block starts with the item of its index and then takes over items of
  // blocks that have not started: each SM gets its next item when it is free
  // (dealing them out in turn left 7% of the SMs' time unused on the 480p clip,
  // a quarter on a ragged batch of three). Answers go through two slots that
  // the ten warps with a role read.
  struct Items {
    uint32_t k;  // answers read
  };
  auto next_item = [&](Items& items) {
    const int slot = items.k & 1;
    const bool ok = role_wait(bar(L::kBarNext + slot), (items.k >> 1) & 1, kErrWinNext, abort_flag);
    if (!__all_sync(0xffffffffu, ok)) return -1;
    const int id = canceled_block(sbase + L::kOffNext + 16 * slot);
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(L::kBarNextRead + slot));
    ++items.k;
    return id;
  };

  // Work item `it`: rows [q0, q0 + 256) of head bh. The last rows come first:
  // they see the most where the past is not limited.
  const int BH = p.B * p.H;
  auto item = [&](int it, int& bh, int& q0, int& len, KeyTiles& kt) {
    bh = it % BH;
    q0 = (p.rtiles - 1 - it / BH) * 2 * kWTile;
    len = seq_len(p.lens, bh / p.H, p.N);
    if (q0 >= len) {
      kt.total = 0;
      return;
    }
    const int last = min(q0 + 2 * kWTile, len) - 1;
    kt = key_tiles(p.w.lo(q0), p.w.hi(last, len), p.w.sinks, 0);
  };
  // Which of an item's key tiles the rows of its 128-row tile x see at all.
  struct Reach {
    int lo, hi, sinks;
    __device__ __forceinline__ bool sees(int key0) const {
      return key0 < hi && (key0 + kWTile > lo || key0 < sinks);
    }
  };
  auto reach = [&](int x, int q0, int len) {
    const int first = q0 + x * kWTile;
    if (first >= len) return Reach{0, 0, 0};
    return Reach{p.w.lo(first), p.w.hi(min(first + kWTile, len) - 1, len), p.w.sinks};
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    few_registers();
    uint32_t n = 0, nq = 0;  // ring slots filled, items with work
    FixUp fix{bar(L::kBarFix), 0};
    Items items{0};
    bool ok = true;
    // Asked for when the item's loads are all on their way (earlier, and a long
    // item would hold another back); the ring covers the answer's time.
    auto ask = [&] {
      const int slot = items.k & 1;
      const bool free = items.k < 2 || role_wait(bar(L::kBarNextRead + slot), ((items.k >> 1) - 1) & 1, kErrWinNext, abort_flag);
      if (!__all_sync(0xffffffffu, free)) return -1;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(L::kBarNext + slot), 16);
        try_cancel(sbase + L::kOffNext + 16 * slot, bar(L::kBarNext + slot));
      }
      __syncwarp();
      return next_item(items);
    };
    for (int it = blockIdx.x; ok && it >= 0; it = ok ? ask() : -1) {
      int bh, q0, len;
      KeyTiles kt;
      item(it, bh, q0, len, kt);
      if (kt.total == 0) continue;
      const int b = bh / p.H, kvh = b * p.Hkv + (bh % p.H) / (p.H / p.Hkv);
      ok = nq == 0 || role_wait(bar(L::kBarQEmpty), (nq - 1) & 1, kErrWinQEmpty, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(bar(L::kBarQFull), 2 * L::kTileBytes);
        for (int h = 0; h < 2; ++h)
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(sQ + h * L::kTileBytes + c * (kWTile * 128), &tmQ, bar(L::kBarQFull), c * 64, q0 + h * kWTile,
                        bh);
      }
      ++nq;
      for (int t = 0; ok && t < 2 * kt.total; ++t, ++n) {  // K(0), V(0), K(1), V(1), ...
        const int slot = n % NS, key0 = kt.key0(t >> 1);
        ok = n < NS || role_wait(bar(L::kBarKvEmpty + slot), (n / NS - 1) & 1, kErrWinKvEmpty, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dst = sKv + slot * L::kTileBytes;
        if (len < p.N && key0 + kWTile > len) {
          ok = load_and_zero<D>(dst, (t & 1) ? &tmV : &tmK, key0, kvh, lane, fix, abort_flag,
                                [&](int r) { return key0 + r >= len; });
          if (!ok) break;
          if (lane == 0) mbar_arrive(bar(L::kBarKvFull + slot));
        } else if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::kBarKvFull + slot), L::kTileBytes);
          for (int c = 0; c < D / 64; ++c)
            tma_load_3d(dst + c * (kWTile * 128), (t & 1) ? &tmV : &tmK, bar(L::kBarKvFull + slot), c * 64, key0, kvh);
        }
      }
    }
    // Never leave with copies in flight.
    if (lane == 0) {
      if (nq) mbar_wait(bar(L::kBarQFull), (nq - 1) & 1, kErrWinQ);
      for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i)
        mbar_wait(bar(L::kBarKvFull + i % NS), (i / NS) & 1, kErrWinKvFull);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    few_registers();
    const bool leader = elect_one();
    constexpr uint32_t idS = idesc_bf16_f32(kWTile, kWTile, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(kWTile, D, false, true);
    const uint64_t dQ = sdesc_sw128(sQ, 16, 1024);
    const uint64_t dKm = sdesc_sw128(sKv, 16, 1024);              // K-major (S = Q K^T)
    const uint64_t dVm = sdesc_sw128(sKv, kWTile * 128, 1024);    // MN-major (O += P V)
    auto wait = [&](int b, uint32_t parity, unsigned int site) {
      return __all_sync(0xffffffffu, role_wait(bar(b), parity, site, abort_flag));
    };
    uint32_t n = 0, nq = 0;                         // ring slots used, items
    uint32_t steps0 = 0, steps1 = 0, done0 = 0, done1 = 0;  // key tiles and items of each row tile
    bool ok = true;
    auto issue_s = [&](int x, int slot) {  // S_x = Q_x K^T
      if (leader) {
        const uint64_t q = dQ + (uint64_t)((x * L::kTileBytes) >> 4), k = dKm + (uint64_t)((slot * L::kTileBytes) >> 4);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t o = ((kk >> 2) * (kWTile * 128) + (kk & 3) * 32) >> 4;
          mma_ss(tmem + x * 128, q + o, k + o, idS, kk > 0 ? 1u : 0u);
        }
        mma_commit(bar(L::kBarS + x));
      }
      __syncwarp();
    };
    Items items{0};
    for (int it = blockIdx.x; ok && it >= 0; it = ok ? next_item(items) : -1) {
      int bh, q0, len;
      KeyTiles kt;
      item(it, bh, q0, len, kt);
      if (kt.total == 0) continue;
      const Reach ra = reach(0, q0, len), rb = reach(1, q0, len);
      bool begun0 = false, begun1 = false;
      ok = wait(L::kBarQFull, nq & 1, kErrWinQ) && wait(L::kBarKvFull + n % NS, (n / NS) & 1, kErrWinKvFull);
      if (!ok) break;
      tc_fence_after();
      if (ra.sees(kt.key0(0))) issue_s(0, n % NS);
      if (rb.sees(kt.key0(0))) issue_s(1, n % NS);
      if (leader) {
        mma_commit(bar(L::kBarKvEmpty + n % NS));
        if (kt.total == 1) mma_commit(bar(L::kBarQEmpty));
      }
      __syncwarp();
      ++n;
      for (int t = 0; ok && t < kt.total; ++t) {
        const int vs = n % NS, ks = (n + 1) % NS, key0 = kt.key0(t), key1 = kt.key0(t + 1);
        const bool more = t + 1 < kt.total;
        ok = wait(L::kBarKvFull + vs, (n / NS) & 1, kErrWinKvFull);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const Reach& r = x == 0 ? ra : rb;
          uint32_t &steps = x == 0 ? steps0 : steps1, &done = x == 0 ? done0 : done1;
          bool& begun = x == 0 ? begun0 : begun1;
          if (ok && r.sees(key0)) {
            if (!begun && done > 0) ok = wait(L::kBarOFree + x, (done - 1) & 1, kErrWinOFree);
            ok = ok && wait(L::kBarP + x, steps & 1, kErrWinP);
            if (!ok) break;
            tc_fence_after();
            const uint64_t v = dVm + (uint64_t)((vs * L::kTileBytes) >> 4);
            if (leader) {
#pragma unroll
              for (int kk = 0; kk < kWTile / 32; ++kk)  // 16 keys = 2048 bytes of V = 8 columns of P
                mma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, v + kk * 128, idO, (begun || kk > 0) ? 1u : 0u);
            }
            __syncwarp();
            ok = wait(L::kBarP2 + x, steps & 1, kErrWinP);
            if (!ok) break;
            tc_fence_after();
            const bool last = t == kt.ns + (r.hi - 1 - kt.lo) / kWTile;  // holds the last key it sees
            if (leader) {
#pragma unroll
              for (int kk = kWTile / 32; kk < kWTile / 16; ++kk)
                mma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, v + kk * 128, idO, 1u);
              if (last) mma_commit(bar(L::kBarO + x));
            }
            __syncwarp();
            begun = true;
            ++steps;
            if (last) ++done;
          }
          if (ok && more && r.sees(key1)) {
            ok = wait(L::kBarKvFull + ks, ((n + 1) / NS) & 1, kErrWinKvFull);
            if (!ok) break;
            tc_fence_after();
            issue_s(x, ks);
          }
        }
        if (ok && leader) {
          mma_commit(bar(L::kBarKvEmpty + vs));
          if (more) mma_commit(bar(L::kBarKvEmpty + ks));
          if (t + 2 == kt.total) mma_commit(bar(L::kBarQEmpty));
        }
        __syncwarp();
        n += more ? 2 : 1;
      }
      ++nq;
    }
    // Every MMA issued has completed before TMEM is freed.
    if (leader) mma_commit(bar(L::kBarDrain));
    __syncwarp();
    mbar_wait(bar(L::kBarDrain), 0, kErrWinDrain);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = (warp - 4) / 4;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + x * 128 + lane_off, to = tmem + 256 + x * 128 + lane_off;
    uint32_t nq = 0, np = 0;
    bool ok = true;
    Items items{0};
    for (int it = blockIdx.x; ok && it >= 0; it = ok ? next_item(items) : -1) {
      int bh, q0, len;
      KeyTiles kt;
      item(it, bh, q0, len, kt);
      const int i = q0 + x * kWTile + r;
      // Rows past the end compute what the last row sees (so that no tile
      // needs a mask for their sake) and store zeros.
      const int at = max(min(i, len - 1), 0);
      const int lo = p.w.lo(at), hi = p.w.hi(at, len);
      // Keys that all rows of the warp see without looking at the sinks.
      const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
      const Reach rx = reach(x, q0, len);
      float m_run = -INFINITY, l_run = 0.0f;
      bool begun = false;
      for (int t = 0; t < kt.total; ++t) {
        const int key0 = kt.key0(t);
        if (!rx.sees(key0)) continue;
        ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarS + x), np++ & 1, kErrWinS, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const bool sink = t < kt.ns;
        const bool whole = sink ? key0 + kWTile <= min(kt.cut, all_hi) : key0 >= all_lo && key0 + kWTile <= all_hi;
        const int e = (sink ? min(hi, kt.cut) : hi) - key0;
        softmax_tile<D>(ts, to, !begun, whole, sink ? 0 : lo - key0, e, p.w.sinks - key0, p.scale_log2, m_run, l_run,
                        0, [&] {
                          tc_fence_before();
                          mbar_arrive(bar(L::kBarP + x));
                        });
        tc_fence_before();
        mbar_arrive(bar(L::kBarP2 + x));
        begun = true;
      }
      if (!ok) break;
      if (i >= len) l_run = 0.0f;
      const bool none = l_run == 0.0f;
      const float inv = none ? 0.0f : 1.0f / l_run;
      if (begun) {
        ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarO + x), nq & 1, kErrWinO, abort_flag));
        if (!ok) break;
        tc_fence_after();
        ++nq;
      }
      __nv_bfloat16* out = p.O + ((int64_t)bh * p.N + i) * D;
      if (begun) {
        store_row<D>(out, to, inv, none, i < p.N);
      } else if (i < p.N) {
#pragma unroll
        for (int c = 0; c < D; c += 8) *reinterpret_cast<uint4*>(out + c) = make_uint4(0, 0, 0, 0);
      }
      if (begun) {
        tc_fence_before();
        mbar_arrive(bar(L::kBarOFree + x));
      }
      if (p.lse != nullptr && i < p.N)
        p.lse[(int64_t)bh * p.N + i] = l_run == 0.0f ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
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

}  // namespace sparge
