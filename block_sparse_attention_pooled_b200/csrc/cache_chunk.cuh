// Attention of a chunk of new tokens over the paged cache on the 5th-generation
// tensor cores: window_fwd_kernel's structure (two 128-row tiles that alternate
// between the tensor core and their softmax) over the equal runs of key tiles
// of cache_sched.cuh.
//
// A row is a (token, head of the K/V head's group) pair, token by token, so a
// tile holds 128 / G tokens and K and V are read once for the whole group. The
// rows of Q come by a 4-D TMA box {64 channels, G heads, 128 / G tokens}.
// K and V come by TMA, one box per page, from a warp each (a box costs its
// issuing lane some hundred cycles). bf16: straight into the ring. e4m3:
// the codes into a slot of their own, from where four more warps write them
// into the ring as bf16, each times its row's power: exact. A row of V that is
// NaN goes there as zeros, or rows of the tile that do not see it would get
// 0 * NaN, and sets a flag; the softmax warps that find it set at the end of an
// item look for such rows among the keys of each of their rows. (Looking at the
// powers of every tile took 171 -> 179 us for five chunks of 700 tokens.)
#pragma once
#include <cuda.h>
#include <cstdint>
#include <cuda_bf16.h>

#include "cache_attn.cuh"
#include "cache_sched.cuh"
#include "wattn.cuh"

namespace sparge {

enum : unsigned int {
  kErrCcQ = 0xC00, kErrCcQEmpty, kErrCcKvFull, kErrCcKvEmpty, kErrCcS, kErrCcP, kErrCcO, kErrCcOFree, kErrCcDrain
};

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  const __nv_bfloat162 v = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Waits for a phase for a millisecond at most, and says nothing.
__device__ __forceinline__ void wait_quietly(uint32_t bar, uint32_t parity) {
  const unsigned long long t0 = globaltimer_ns();
  while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 < 1000000ull) {
  }
}

// Whether a row that sees [lo, hi) and the sinks of an item's key tiles t0 .. t1 - 1
// sees a row of V that is NaN. Called by a whole warp, each lane with its row.
__device__ __noinline__ bool sees_nan_value(const CacheAttnParams& p, KeyTiles kt, int b, int hk, int len, int t0, int t1,
                                            int lo, int hi) {
  const int lane = threadIdx.x % 32;
  bool sees = false;
  for (int t = t0; t < t1; ++t) {
    const bool sink = t < kt.ns;
    const int key0 = kt.key0(t), most = sink ? min(hi, kt.cut) : hi, mine = key0 + 4 * lane;
    const int64_t row = mine < len ? cache_row(p.c, b, mine) : -1;  // of four keys: they lie in one page
    uint32_t bytes = 0;
    if (row >= 0) bytes = *reinterpret_cast<const uint32_t*>(p.c.v_exp + row + ((int64_t)hk << p.c.page_shift));
    for (unsigned left = __ballot_sync(0xffffffffu, __vcmpeq4(bytes, 0xFFFFFFFFu) != 0); left; left &= left - 1) {
      const int src = __ffs(left) - 1;
      const uint32_t four = __shfl_sync(0xffffffffu, bytes, src);
      for (int j = 0; j < 4; ++j) {
        const int key = key0 + 4 * src + j;
        sees |= (four >> (8 * j) & 0xFFu) == 0xFFu && key < most && (sink || key >= lo || key < p.w.sinks);
      }
    }
  }
  return sees;
}

template <bool E4M3>
__host__ __device__ constexpr int chunk_threads() { return E4M3 ? 512 : 384; }

// Shared memory: two Q tiles, the ring, and for e4m3 a slot of K's codes and one of V's.
template <int D, bool E4M3>
struct ChunkSmem {
  static constexpr int NS = E4M3 ? 4 : D == 128 ? 5 : 8;
  static constexpr int kTileBytes = kWTile * D * 2;
  static constexpr int kOffQ = 0, kOffKv = 2 * kTileBytes;
  static constexpr int kOffCode = kOffKv + NS * kTileBytes;
  static constexpr int kOffExp = kOffCode + (E4M3 ? kTileBytes : 0);  // [2][128]
  static constexpr int kOffMask = kOffExp + (E4M3 ? 256 : 0);         // [2]
  static constexpr int kOffBar = kOffMask + 16;
  static constexpr int kBarQFull = 0, kBarQEmpty = 1, kBarKvFull = 2, kBarKvEmpty = 2 + NS, kBarS = 2 + 2 * NS,
                       kBarP = 4 + 2 * NS, kBarP2 = 6 + 2 * NS, kBarO = 8 + 2 * NS, kBarOFree = 10 + 2 * NS,
                       kBarDrain = 12 + 2 * NS, kBarCodeFull = 13 + 2 * NS, kBarFix = 15 + 2 * NS,
                       kBarCodeEmpty = 17 + 2 * NS;
  static constexpr int kNumBars = 19 + 2 * NS;
  static constexpr int kOffTmem = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffTmem + 16 + 1024;
  static_assert(kBytes <= 227 * 1024);
};

template <int D, bool E4M3>
__global__ void __launch_bounds__(chunk_threads<E4M3>(), 1)
    cache_chunk_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const __grid_constant__ CacheAttnParams p) {
  using L = ChunkSmem<D, E4M3>;
  constexpr int NS = L::NS, KT = kWTile;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  const uint32_t sQ = sbase + L::kOffQ, sKv = sbase + L::kOffKv;
  auto bar = [&](int i) { return sbase + L::kOffBar + 8u * (uint32_t)i; };
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(sgen + L::kOffTmem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kOffTmem + 4);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  volatile uint32_t* code_mask = reinterpret_cast<volatile uint32_t*>(sgen + L::kOffMask);  // boxes that exist
  volatile uint32_t* nan_flag = code_mask + 2;  // e4m3: some row of V so far is NaN

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      const bool rows = (i >= L::kBarP && i < L::kBarP + 4) || (i >= L::kBarOFree && i < L::kBarOFree + 2);
      const bool conv = E4M3 && ((i >= L::kBarKvFull && i < L::kBarKvFull + NS) || i >= L::kBarCodeEmpty);
      mbar_init(bar(i), rows || conv ? 128 : 1);
    }
    *abort_flag = 0;
    *nan_flag = 0;
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
  const int tq = p.tpt / 2;  // tokens per 128-row tile

  // This CTA's run of units.
  CacheRun<KT> run;
  run.find(p, blockIdx.x, lane);
  const int64_t W = run.W;
  const int ctas = run.ctas;
  const bool work = run.left > 0;
  CacheItem<KT> it = run.it;
  int at = run.at;
  const int64_t start = run.start, end = start + run.left;
  int64_t left = run.left;
  auto few_registers = [] {
    if (E4M3) asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
  };
  // Ends a piece of an item; false when the run is done.
  auto advance = [&](int stop) {
    left -= stop - at;
    at = 0;
    return left > 0 && it.next(p);
  };

  if (warp == 0 || warp == 2) {
    // ------------------------------------------------------------ producers: Q and K, V
    few_registers();
    const bool is_v = warp == 2;
    const CUtensorMap* tm = is_v ? &tmV : &tmK;
    const uint8_t* exps = is_v ? p.c.v_exp : p.c.k_exp;
    const int box_shift = p.box_shift, boxes = KT >> box_shift;
    uint32_t n = is_v, nq = 0;  // ring order K(0), V(0), K(1), ...
    FixUp fix{bar(L::kBarFix + is_v), 0};
    bool ok = true;
    if (work) do {
      const int stop = (int)min((int64_t)it.T, at + left), len = it.len();
      if (!is_v) {
        ok = nq == 0 || role_wait(bar(L::kBarQEmpty), (nq - 1) & 1, kErrCcQEmpty, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(L::kBarQFull), 2 * (D / 64) * tq * p.G * 128);
          for (int h = 0; h < 2; ++h)
            for (int c = 0; c < D / 64; ++c)
              tma_load_4d(sQ + h * L::kTileBytes + c * (kWTile * 128), &tmQ, bar(L::kBarQFull), c * 64, 0,
                          it.cu + it.tile * p.tpt + h * tq, it.hk);
        }
        ++nq;
      }
      PageAhead<KT> pages;
      pages.start(p, it, at, stop, lane);
      for (int t = at; t < stop; ++t, n += 2) {
        const int key0 = it.kt.key0(t), pos = key0 + (lane << box_shift);
        int64_t row = pages.get(p, it, t, lane);
        if (lane >= boxes) row = -1;
        const unsigned there = __ballot_sync(0xffffffffu, row >= 0);
        const int place = pos & ((1 << p.c.page_shift) - 1);
        const int64_t head = row + ((int64_t)it.hk << p.c.page_shift);
        const int z = (int)((head - place) >> p.c.page_shift);
        if (E4M3) {
          const uint32_t full = bar(L::kBarCodeFull + is_v);
          ok = n < 2 || role_wait(bar(L::kBarCodeEmpty + is_v), (n / 2 - 1) & 1, kErrCcKvEmpty, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) {
            code_mask[is_v] = there;
            mbar_arrive_expect_tx(full, ((uint32_t)__popc(there) << box_shift) * (D + 1));
          }
          __syncwarp();
          if (row >= 0) {
            tma_load_3d(sbase + L::kOffCode + is_v * (kWTile * D) + (lane << box_shift) * D, tm, full, 0, place, z);
            bulk_load(sbase + L::kOffExp + is_v * 128 + (lane << box_shift), exps + head, 1u << box_shift, full);
          }
        } else {
          const int slot = n % NS;
          const uint32_t full = bar(L::kBarKvFull + slot), dst = sKv + slot * L::kTileBytes;
          ok = n < NS || role_wait(bar(L::kBarKvEmpty + slot), (n / NS - 1) & 1, kErrCcKvEmpty, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          // A tile with places that do not exist lands on the warp's own barrier
          // first and gets zeros there.
          const bool broken = key0 + KT > len || __popc(there) < boxes;
          const uint32_t land = broken ? fix.bar : full;
          if (lane == 0) mbar_arrive_expect_tx(land, ((uint32_t)__popc(there) << box_shift) * (D * 2));
          __syncwarp();
          if (row >= 0)
            for (int c = 0; c < D / 64; ++c)
              tma_load_3d(dst + c * (KT * 128) + (lane << box_shift) * 128, tm, land, c * 64, place, z);
          if (broken) {
            ok = role_wait(fix.bar, fix.phase++ & 1, kErrCcKvFull, abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            zero_rows<D>(dst, lane, [&](int r) { return key0 + r >= len || !(there >> (r >> box_shift) & 1u); });
            if (lane == 0) mbar_arrive(full);
          }
        }
        __syncwarp();
      }
      if (!ok || !advance(stop)) break;
    } while (true);
    // Never leave with copies in flight.
    if (lane == 0) {
      if (nq) mbar_wait(bar(L::kBarQFull), (nq - 1) & 1, kErrCcQ);
      if (E4M3) {
        if (n >= 2) mbar_wait(bar(L::kBarCodeFull + is_v), (n / 2 - 1) & 1, kErrCcKvFull);
      } else {
        // Its loads that no later one has followed into their slot: where one
        // has (the other warp's, the ring being odd), the slot was empty again.
        // When a role gave up that is not known: each wait gets a millisecond.
        const int last = (int)n - (is_v ? 2 : 1);  // the ring's last index
        for (int i = max((int)n - 2 * (NS + 1), (int)is_v); i < (int)n; i += 2) {
          if (ok && i + NS > last) mbar_wait(bar(L::kBarKvFull + i % NS), (i / NS) & 1, kErrCcKvFull);
          else if (!ok) wait_quietly(bar(L::kBarKvFull + i % NS), (i / NS) & 1);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    few_registers();
    const bool leader = elect_one();
    constexpr uint32_t idS = idesc_bf16_f32(kWTile, kWTile, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(kWTile, D, false, true);
    const uint64_t dQ = sdesc_sw128(sQ, 16, 1024);
    const uint64_t dKm = sdesc_sw128(sKv, 16, 1024);
    const uint64_t dVm = sdesc_sw128(sKv, kWTile * 128, 1024);
    auto wait = [&](int b, uint32_t parity, unsigned int site) {
      return __all_sync(0xffffffffu, role_wait(bar(b), parity, site, abort_flag));
    };
    uint32_t n = 0, nq = 0;
    uint32_t steps[2] = {0, 0}, items[2] = {0, 0};  // of each tile
    bool ok = true;
    auto issue_s = [&](int x, int slot) {
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
    if (work) do {
      const int stop = (int)min((int64_t)it.T, at + left), total = stop - at;
      const int nx = it.n - it.tile * p.tpt > tq ? 2 : 1;  // tile B may have no rows
      ok = wait(L::kBarQFull, nq & 1, kErrCcQ) && wait(L::kBarKvFull + n % NS, (n / NS) & 1, kErrCcKvFull);
      if (!ok) break;
      tc_fence_after();
      issue_s(0, n % NS);
      if (nx == 2) issue_s(1, n % NS);
      if (leader) {
        mma_commit(bar(L::kBarKvEmpty + n % NS));
        if (total == 1) mma_commit(bar(L::kBarQEmpty));
      }
      __syncwarp();
      ++n;
      for (int t = 0; ok && t < total; ++t) {
        const int vs = n % NS, ks = (n + 1) % NS;
        const bool more = t + 1 < total;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (x >= nx) break;
          if (x == 0) ok = wait(L::kBarKvFull + vs, (n / NS) & 1, kErrCcKvFull);
          if (ok && t == 0 && items[x] > 0) ok = wait(L::kBarOFree + x, (items[x] - 1) & 1, kErrCcOFree);
          ok = ok && wait(L::kBarP + x, steps[x] & 1, kErrCcP);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t v = dVm + (uint64_t)((vs * L::kTileBytes) >> 4);
#pragma unroll
            for (int kk = 0; kk < kWTile / 32; ++kk)
              mma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, v + kk * 128, idO, (t > 0 || kk > 0) ? 1u : 0u);
          }
          __syncwarp();
          ok = wait(L::kBarP2 + x, steps[x] & 1, kErrCcP);
          ++steps[x];
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t v = dVm + (uint64_t)((vs * L::kTileBytes) >> 4);
#pragma unroll
            for (int kk = kWTile / 32; kk < kWTile / 16; ++kk)
              mma_ts(tmem + 256 + x * 128, tmem + x * 128 + kk * 8, v + kk * 128, idO, 1u);
            if (x == nx - 1) mma_commit(bar(L::kBarKvEmpty + vs));
            if (!more) mma_commit(bar(L::kBarO + x));
          }
          __syncwarp();
          if (more) {
            if (x == 0) ok = wait(L::kBarKvFull + ks, ((n + 1) / NS) & 1, kErrCcKvFull);
            if (!ok) break;
            tc_fence_after();
            issue_s(x, ks);
            if (x == nx - 1 && leader) {
              mma_commit(bar(L::kBarKvEmpty + ks));
              if (t + 2 == total) mma_commit(bar(L::kBarQEmpty));
            }
            __syncwarp();
          }
        }
        n += more ? 2 : 1;
      }
      ++nq;
      ++items[0];
      if (nx == 2) ++items[1];
      if (!ok || !advance(stop)) break;
    } while (true);
    if (leader) mma_commit(bar(L::kBarDrain));
    __syncwarp();
    mbar_wait(bar(L::kBarDrain), 0, kErrCcDrain);
  } else if (warp >= 4 && warp < 12) {
    // ------------------------------------------------------------ softmax and epilogue
    if (E4M3) asm volatile("setmaxnreg.inc.sync.aligned.u32 192;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 200;");
    const int x = (warp - 4) / 4;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + x * 128 + lane_off, to = tmem + 256 + x * 128 + lane_off;
    uint32_t nq = 0, np = 0;
    bool ok = true;
    if (work) do {
      const int at0 = at, stop = (int)min((int64_t)it.T, at + left), len = it.len();
      const int64_t unit0 = end - left - at;
      if (x == 1 && it.n - it.tile * p.tpt <= tq) {  // no rows here
        if (!advance(stop)) break;
        continue;
      }
      const int tok = it.tile * p.tpt + x * tq + r / p.G;
      const bool live = r < tq * p.G && tok < it.n;
      const int i = it.first + min(tok, it.n - 1);
      const int lo = p.w.lo(i), hi = p.w.hi(i, len);
      const int all_lo = __reduce_max_sync(0xffffffffu, lo), all_hi = __reduce_min_sync(0xffffffffu, hi);
      float m_run = -INFINITY, l_run = 0.0f;
      // Lane l < 8: whether the tile's l-th 16 keys lie in a page that does not
      // exist; looked up a tile ahead.
      auto absent = [&](int t) {
        const int g16 = it.kt.key0(t) + lane * 16;
        return lane < 8 && t < stop && g16 < len && cache_row(p.c, it.b, g16) < 0;
      };
      bool next_absent = absent(at);
      for (int t = at; t < stop; ++t, ++np) {
        const int key0 = it.kt.key0(t);
        const unsigned m = __ballot_sync(0xffffffffu, next_absent);
        next_absent = absent(t + 1);
        ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarS + x), np & 1, kErrCcS, abort_flag));
        if (!ok) break;
        tc_fence_after();
        const bool sink = t < it.kt.ns;
        const bool whole = m == 0 &&
                           (sink ? key0 + KT <= min(it.kt.cut, all_hi) : key0 >= all_lo && key0 + KT <= all_hi);
        const int e = (sink ? min(hi, it.kt.cut) : hi) - key0;
        softmax_tile<D>(ts, to, t == at, whole, sink ? 0 : lo - key0, e, p.w.sinks - key0, p.scale_log2, m_run, l_run,
                        m, [&] {
                          tc_fence_before();
                          mbar_arrive(bar(L::kBarP + x));
                        });
        tc_fence_before();
        mbar_arrive(bar(L::kBarP2 + x));
      }
      if (!ok) break;
      ok = __all_sync(0xffffffffu, role_wait(bar(L::kBarO + x), nq & 1, kErrCcO, abort_flag));
      if (!ok) break;
      tc_fence_after();
      ++nq;
      const int64_t row = (int64_t)(it.cu + tok) * p.H + it.hk * p.G + r % p.G;
      const bool none = l_run == 0.0f;
      // What O is multiplied by: NaN if the row sees a row of V that is NaN. All
      // of the item's V tiles are in O, so the flag is there.
      float one = 1.0f;
      if (E4M3 && __any_sync(0xffffffffu, *nan_flag != 0) && sees_nan_value(p, it.kt, it.b, it.hk, len, at0, stop, lo, hi))
        one = __int_as_float(0x7FC00000);
      if (at0 == 0 && live && r % p.G == 0)
        p.owners[(int64_t)(it.cu + tok) * p.c.Hkv + it.hk] =
            make_int4(blockIdx.x, start < unit0, stop == it.T ? (int)blockIdx.x : run_owner(W, ctas, unit0 + it.T - 1),
                      x * tq * p.G + r);
      if (at0 == 0 && stop == it.T) {
        store_row<D>(p.O + row * D, to, none ? 0.0f : one / l_run, none, live);
        if (live && p.lse) p.lse[row] = none ? -INFINITY : (m_run + log2f(l_run)) * 0.69314718055994531f;
      } else {
        const int64_t slot = (int64_t)(2 * blockIdx.x + (start < unit0 ? 1 : 0)) * (2 * kWTile) + (x * tq * p.G + r);
        store_row_f32<D>(p.part_o + slot * D, to, one, false, live);
        if (live) p.part_ml[slot] = make_float2(m_run, l_run);
      }
      tc_fence_before();
      mbar_arrive(bar(L::kBarOFree + x));
      if (!advance(stop)) break;
    } while (true);
  } else if (E4M3 && warp >= 12) {
    // ------------------------------------------------------------ codes to bf16
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    constexpr int CH = D / 16;             // 16-code pieces per row
    constexpr int N = kWTile * CH / 128;   // pieces per thread and tile
    constexpr int U = 4;                   // at a time
    constexpr int RS = 128 / CH;           // rows between a thread's pieces
    // Eight neighbouring threads take four pieces of an even row and, of the odd row after it, the four of D = 64 or
    // the other four of D = 128: their 16-byte reads and writes then lie in different banks (a row of eight pieces
    // would write each bank twice).
    const int tid = threadIdx.x - 384, odd = tid / 4 % 2;
    const int c = tid % 4 + (CH == 8 ? 4 * (tid / 8 % 2 ^ odd) : 0), r0 = tid / (2 * CH) * 2 + odd;
    uint32_t n = 0;
    bool ok = true;
    if (work) do {
      const int stop = (int)min((int64_t)it.T, at + left), len = it.len();
      const int box_shift = p.box_shift;
      for (int t = 2 * at; ok && t < 2 * stop; ++t, ++n) {
        const int slot = n % NS, is_v = t & 1, key0 = it.kt.key0(t >> 1);
        ok = role_wait(bar(L::kBarCodeFull + is_v), (n / 2) & 1, kErrCcKvFull, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t there = code_mask[is_v], src = sbase + L::kOffCode + is_v * (kWTile * D);
        ok = n < NS || role_wait(bar(L::kBarKvEmpty + slot), (n / NS - 1) & 1, kErrCcKvEmpty, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t dst = sKv + slot * L::kTileBytes;
        const uint32_t line0 = dst + (2 * c / 8) * (kWTile * 128);
        const uint32_t nan_row = is_v ? 0u : 0x7FC0u;  // what such a row's codes are multiplied by
#pragma unroll 1
        for (int k0 = 0; k0 < N; k0 += U) {
          uint4 code[U];
          uint32_t e[U];
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int r = r0 + (k0 + k) * RS;
            code[k] = lds128(src + r * D + ((D == 128 ? c ^ (r & 7) : c ^ ((r >> 1) & 3)) * 16));
            e[k] = lds_u8(sbase + L::kOffExp + is_v * 128 + r);
          }
#pragma unroll
          for (int k = 0; k < U; ++k) {
            const int r = r0 + (k0 + k) * RS;
            const bool here = key0 + r < len && (there >> (r >> box_shift) & 1u);
            // 2^(e + 120) as bf16, twice; 2^120 and 2^e in two steps where that is out of range. 0: does not exist
            // (the codes there may be anything, but as bf16 they are finite). A row that is NaN counts as far.
            const bool far = here && e[k] > 134;
            const uint32_t p1 = !here ? 0u : (e[k] == 255 ? nan_row : (far ? 247u : e[k] + 120u) << 7) * 0x10001u;
            const uint32_t w[4] = {code[k].x, code[k].y, code[k].z, code[k].w};
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
              v[j] = bf16x2_mul(codes_to_bf16(__byte_perm(w[j / 2], 0, j & 1 ? 0x4342 : 0x4140)), p1);
            if (far) {
              if (e[k] == 255 && is_v) *nan_flag = 1;
              const uint32_t p2 = (e[k] == 255 ? 0x3F80u : e[k] << 7) * 0x10001u;
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = bf16x2_mul(v[j], p2);
            }
            const uint32_t line = line0 + r * 128;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + ((((2 * c) % 8 + h) ^ (r & 7)) * 16)),
                           "r"(v[4 * h]), "r"(v[4 * h + 1]), "r"(v[4 * h + 2]), "r"(v[4 * h + 3])
                           : "memory");
          }
        }
        mbar_arrive(bar(L::kBarCodeEmpty + is_v));
        fence_async_smem();
        mbar_arrive(bar(L::kBarKvFull + slot));
      }
      if (!ok || !advance(stop)) break;
    } while (true);
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
