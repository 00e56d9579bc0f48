// Attention of few new tokens over the paged cache (one token of each of G
// heads when decoding): bound by reading the cache once.
//
// Persistent CTAs with equal runs of key tiles (cache_sched.cuh; 64 keys of bf16,
// 128 of e4m3). Two producer
// warps fill a ring of K and V tiles by TMA through the page table (one box per
// page and 64 columns; 128 bytes of swizzle); the other warps take whole tiles
// in turn, each with a running maximum and sum and an accumulator of its own,
// so that nothing but the ring orders them, and are joined in shared memory at
// the end of an item. Scores are kept transposed (keys x rows): with at most 8
// rows the 16-wide side of mma.m16n8k16 is the keys' and the channels', and a
// tile costs half the instructions. P^T turns from accumulator to operand by
// movmatrix, in registers.
//   S^T = K Q^T (16 keys x 8 rows x 16 channels a step), O^T += V^T P^T.
// e4m3: a lane takes 16 codes of a row at a time, which fixes the order of the
// channels within a step (Q is read in the same order). Every code is exact in
// fp16, so these products are fp16's, with what does not fit its range kept
// outside: a row of Q enters times the power of two that puts its largest
// element at 2^14 (exact but below 2^-39 of that), a key's power joins its
// score, and a value's power joins the exponent of its probability: with
// x_j the score in log2 units and e_j the power of v_j, the product takes
// P_j = 2^(x_j + e_j - M + 15), M the running maximum of x_j + e_j: at the top
// of fp16's range, so that what lies down to 2^-29 of the largest keeps 11 bits
// and half a step below that is 2^-40 of it. (Half a step of the largest key's
// own codes is 2^-10 of its power.) The row sum is
// kept apart, sum 2^(x_j - X) with X the running maximum of x_j: powers lie up
// to 240 apart (a row of zeros has the least), so neither sum can be had from
// the other's terms. The product is moved to the reference X when a warp is done.
#pragma once
#include <cuda.h>
#include <cstdint>
#include <cuda_bf16.h>

#include "cache_sched.cuh"
#include "ptx.cuh"

namespace sparge {

enum : unsigned int { kErrCaFull = 0xB00, kErrCaEmpty, kErrCaDrain };

// Keys per tile: 32 KB of K and V either way (16 KB tiles cost as much to hand
// over, 121 us against 105 for 24 sequences of 16 k tokens).
template <bool E4M3>
__host__ __device__ constexpr int dec_keys() { return E4M3 ? 128 : 64; }

template <int D, bool E4M3, int R8>
struct DecSmem {
  // Consumer warps; SPLIT of them share a tile, each with its part of the keys.
  // bf16: the tensor instructions and ldmatrix of three warps keep up with
  // memory. e4m3: half the bytes and ten instructions per four codes need more.
  static constexpr int SPLIT = E4M3 ? 2 : 1;
  static constexpr int NW = E4M3 ? (R8 == 1 ? 10 : 8) : D == 128 ? 3 : 4;
  static constexpr int kRows = 8 * R8;
  static constexpr int kRowBytes = D * (E4M3 ? 1 : 2);
  static constexpr int KT = dec_keys<E4M3>();
  static constexpr int kTile = KT * kRowBytes;           // K or V
  static constexpr int kStage = 2 * kTile;
  static constexpr int kOStride = D + 4;                 // floats; + 4: the lanes' rows fall into different banks
  static constexpr int kMerge = NW * kRows * (kOStride * 4 + 8);
  static constexpr int kBudget = 225 * 1024 - kMerge - 2048;
  // A multiple of the warps' turns, so that a slot is always the same warp's: a warp
  // that met a slot first in a later round could take the round before, still
  // on its way, for its own (the barrier tells odd rounds from even ones only).
  static constexpr int kFit = kBudget / (kStage + 2 * KT + 32);
  static constexpr int NS = (kFit > 16 ? 16 : kFit) / (NW / SPLIT) * (NW / SPLIT);
  static_assert(NS >= 4);
  static constexpr int kOffExp = NS * kStage;            // per stage: K's and V's powers
  static constexpr int kOffMask = kOffExp + NS * 2 * KT; // per stage: which 16-key groups exist
  static constexpr int kOffBar = kOffMask + NS * 4 + (NS & 1) * 4;
  static constexpr int kOffMl = kOffBar + 2 * NS * 8;
  static constexpr int kOffO = (kOffMl + NW * kRows * 8 + 15) / 16 * 16;
  static constexpr int kOffAbort = kOffO + NW * kRows * kOStride * 4;
  static constexpr int kBytes = kOffAbort + 16 + 1024;
  static constexpr int kThreads = (NW + 2) * 32;
  static_assert(kBytes <= 227 * 1024);
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// c += a b, 16 x 8 x 16.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma16816_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two e4m3 codes in the low half -> fp16 pair.
__device__ __forceinline__ uint32_t codes_to_f16(uint32_t u) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)u, __NV_E4M3);
  return (uint32_t)h.x | ((uint32_t)h.y << 16);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Two e4m3 codes in the lower bytes of u's halves, times 2^-120, as a bf16 pair
// (sign, exponent and mantissa in place; exact, also below 2^-6): magnitude up
// by 4 bits, sign by 8, 2^7 16 + 2^7 240 = 2^15. Mostly multiplies: the integer
// pipe has half their rate.
__device__ __forceinline__ uint32_t codes_to_bf16(uint32_t u) { return u * 16u + (u & 0x00800080u) * 240u; }

template <int D, bool E4M3, int R8>
__global__ void __launch_bounds__(DecSmem<D, E4M3, R8>::kThreads)
    cache_decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                        const CacheAttnParams p) {
  using L = DecSmem<D, E4M3, R8>;
  constexpr int NS = L::NS, NW = L::NW, KT = L::KT, SPLIT = L::SPLIT;
  constexpr int MT = KT / 16 / SPLIT;  // a warp's 16-key steps of a tile
  constexpr float kPTop = 15.0f;       // e4m3: the largest P is 2^15 (fp16 ends at 2^16)
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* sgen = smem_raw + (sbase - raw);
  auto full = [&](int i) { return sbase + L::kOffBar + 8u * (uint32_t)i; };
  auto empty = [&](int i) { return sbase + L::kOffBar + 8u * (uint32_t)(NS + i); };
  uint32_t* masks = reinterpret_cast<uint32_t*>(sgen + L::kOffMask);
  float2* wml = reinterpret_cast<float2*>(sgen + L::kOffMl);
  float* wo = reinterpret_cast<float*>(sgen + L::kOffO);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(sgen + L::kOffAbort);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full(i), 2);
      mbar_init(empty(i), SPLIT);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  grid_let_next();
  CacheRun<KT> run;
  run.find(p, blockIdx.x, lane);
  if (run.left == 0) return;
  const int64_t W = run.W;
  const int ctas = run.ctas;
  CacheItem<KT> it = run.it;
  int at = run.at;
  const int64_t start = run.start, end = start + run.left;
  int64_t left = run.left;

  if (warp >= NW) {
    // ------------------------------------------------------------ producers: one warp for K, one for V
    const bool is_v = warp > NW;
    const CUtensorMap* tm = is_v ? &tmV : &tmK;
    const uint8_t* exps = is_v ? p.c.v_exp : p.c.k_exp;
    const int box_shift = p.box_shift, boxes = KT >> box_shift;
    uint32_t n = 0;
    bool ok = true;
    while (ok && left > 0) {
      const int stop = (int)min((int64_t)it.T, at + left);
      left -= stop - at;
      PageAhead<KT> pages;
      pages.start(p, it, at, stop, lane);
      for (int t = at; t < stop; ++t, ++n) {
        const int slot = n % NS;
        const int pos = it.kt.key0(t) + (lane << box_shift);
        int64_t row = pages.get(p, it, t, lane);  // a page's row, head 0
        if (lane >= boxes) row = -1;
        ok = n < NS || role_wait(empty(slot), (n / NS - 1) & 1, kErrCaEmpty, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const unsigned there = __ballot_sync(0xffffffffu, row >= 0);
        if (lane == 0) {
          if (!is_v) {
            uint32_t m = 0;  // one bit per 16 keys
            for (int x = 0; x < boxes; ++x)
              if (there >> x & 1u) m |= ((1u << (1 << (box_shift - 4))) - 1u) << (x << (box_shift - 4));
            masks[slot] = m;
          }
          const uint32_t bytes = (uint32_t)__popc(there) << box_shift;
          mbar_arrive_expect_tx(full(slot), bytes * (L::kRowBytes + (E4M3 ? 1 : 0)));
        }
        __syncwarp();
        if (row >= 0) {
          const uint32_t dst =
              sbase + slot * L::kStage + (is_v ? L::kTile : 0) + (lane << box_shift) * (E4M3 ? D : 128);
          const int place = pos & ((1 << p.c.page_shift) - 1);
          const int64_t head = row + ((int64_t)it.hk << p.c.page_shift);
          const int z = (int)((head - place) >> p.c.page_shift);
          if (E4M3) {
            tma_load_3d(dst, tm, full(slot), 0, place, z);
            bulk_load(sbase + L::kOffExp + slot * 2 * KT + (is_v ? KT : 0) + (lane << box_shift), exps + head,
                      1u << box_shift, full(slot));
          } else {
#pragma unroll
            for (int c = 0; c < D / 64; ++c) tma_load_3d(dst + c * (KT * 128), tm, full(slot), c * 64, place, z);
          }
        }
        __syncwarp();
      }
      if (left > 0 && !it.next(p)) break;
      at = 0;
    }
    // Never leave with copies in flight.
    if (lane == 0)
      for (uint32_t i = n > NS ? n - NS : 0; i < n; ++i) mbar_wait(full(i % NS), (i / NS) & 1, kErrCaDrain);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int g = lane >> 2, c = lane & 3;
  const int turn = warp / SPLIT, k16 = warp % SPLIT * MT;  // its first 16-key step
  uint32_t n = 0;
  bool ok = true;
  while (ok && left > 0) {
    const int at0 = at, stop = (int)min((int64_t)it.T, at + left);
    const int t0 = it.tile * p.tpt, tokens = min(p.tpt, it.n - t0), len = it.len();
    const int64_t unit0 = end - left - at;  // the item's first unit
    left -= stop - at;
    // Q as operand B: rows 8 x + g, channels as the keys' operand has them.
    uint32_t q[R8][D / 16][2];
    float unq[R8][2], unq2[R8][2];  // e4m3: two factors that undo the scaling of the lane's accumulator rows
#pragma unroll
    for (int x = 0; x < R8; ++x) {
      const int r = 8 * x + g;
      const bool live = r < tokens * p.G;
      const __nv_bfloat16* src =
          p.Q + (int64_t)(it.cu + t0 + (live ? r / p.G : 0)) * p.q_stride + (it.hk * p.G + (live ? r % p.G : 0)) * D;
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {
        if (E4M3) {
          const uint2 v = *reinterpret_cast<const uint2*>(src + 64 * (k / 4) + 16 * c + 4 * (k % 4));
          q[x][k][0] = v.x;
          q[x][k][1] = v.y;
        } else {
          q[x][k][0] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * c);
          q[x][k][1] = *reinterpret_cast<const uint32_t*>(src + 16 * k + 2 * c + 8);
        }
      }
      if (E4M3) {
        uint32_t top = 0;  // the row's largest magnitude, as bf16 bits
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h) top = max(top, max(q[x][k][h] & 0x7FFFu, (q[x][k][h] >> 16) & 0x7FFFu));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const int shift = min(14 - ((int)(top >> 7) - 127), 127);
        const float f = __uint_as_float((uint32_t)(127 + shift) << 23);
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            q[x][k][h] = pack_f16x2(__uint_as_float(q[x][k][h] << 16) * f, __uint_as_float(q[x][k][h] & 0xFFFF0000u) * f);
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          // One before and one after the key's power: all of 2^-shift at once
          // could leave the range where the score does not.
          const int sh = __shfl_sync(0xffffffffu, shift, 4 * (2 * c + y)), half = sh / 2;
          unq[x][y] = p.scale_log2 * __uint_as_float((uint32_t)(127 - half) << 23);
          unq2[x][y] = __uint_as_float((uint32_t)(127 - (sh - half)) << 23);
        }
      }
    }
    // The lane's rows in the accumulators: 8 x + 2 c + y.
    int lo[R8][2], hi[R8][2];
    float m_run[R8][2], l_run[R8][2], o[D / 16][R8][4];
    float x_run[R8][2];  // e4m3: the reference of l_run, over the lane's own keys
#pragma unroll
    for (int x = 0; x < R8; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = it.first + t0 + min((8 * x + 2 * c + y) / p.G, tokens - 1);
        lo[x][y] = p.w.lo(i);
        hi[x][y] = p.w.hi(i, len);
        m_run[x][y] = x_run[x][y] = -INFINITY;
        l_run[x][y] = 0.0f;
      }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
      for (int x = 0; x < R8; ++x)
#pragma unroll
        for (int y = 0; y < 4; ++y) o[k][x][y] = 0.0f;
    const int all_lo = p.w.lo(it.first + t0 + tokens - 1), all_hi = p.w.hi(it.first + t0, len);

    for (int t = at; t < stop; ++t, ++n) {
      if (n % (NW / SPLIT) != turn) continue;
      const int slot = n % NS, key0 = it.kt.key0(t);
      const bool sink = t < it.kt.ns;
      ok = __all_sync(0xffffffffu, role_wait(full(slot), (n / NS) & 1, kErrCaFull, abort_flag));
      if (!ok) break;
      const uint32_t mask = *reinterpret_cast<volatile uint32_t*>(masks + slot);
      const uint32_t sk = sbase + slot * L::kStage, sv = sk + L::kTile, ex = sbase + L::kOffExp + slot * 2 * KT;
      const bool exists = mask == (1u << (KT / 16)) - 1u && key0 + KT <= len;
      const bool whole = exists && (sink ? key0 + KT <= min(it.kt.cut, all_hi) : key0 >= all_lo && key0 + KT <= all_hi);
      if (!exists) {
        // Zeros in V's rows that do not exist: memory may hold NaN there, and 0 * NaN is not 0.
        // (Each warp its own keys; a row's pieces all go, so their order does not matter.)
        constexpr int PPR = L::kRowBytes / 16;
        for (int e = lane; e < 16 * MT * PPR; e += 32) {
          const int r = 16 * k16 + e / PPR, ch = e % PPR;
          if (key0 + r >= len || !(mask >> (r >> 4) & 1u))
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                             E4M3 ? sv + r * D + ch * 16 : sv + (ch / 8) * (KT * 128) + r * 128 + (ch % 8) * 16),
                         "r"(0)
                         : "memory");
        }
        fence_async_smem();
        __syncwarp();
      }
      // S^T
      float s[MT][R8][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int x = 0; x < R8; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y) s[mt][x][y] = 0.0f;
        if (E4M3) {
#pragma unroll
          for (int j = 0; j < D / 64; ++j) {
            uint32_t w[2][4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int r = 16 * (k16 + mt) + g + 8 * y, ch = 4 * j + c;
              const uint4 v = lds128(sk + r * D + (D == 128 ? (ch ^ (r & 7)) : (ch ^ ((r >> 1) & 3))) * 16);
              w[y][0] = v.x, w[y][1] = v.y, w[y][2] = v.z, w[y][3] = v.w;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t a[4] = {codes_to_f16(w[0][k]), codes_to_f16(w[1][k]), codes_to_f16(w[0][k] >> 16),
                                     codes_to_f16(w[1][k] >> 16)};
#pragma unroll
              for (int x = 0; x < R8; ++x) mma16816_f16(s[mt][x], a, q[x][4 * j + k][0], q[x][4 * j + k][1]);
            }
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int r = 16 * (k16 + mt) + (lane & 15), ch = 2 * k + (lane >> 4);
            uint32_t a[4];
            ldsm4(sk + (ch / 8) * (KT * 128) + r * 128 + (((ch % 8) ^ (r & 7)) * 16), a);
#pragma unroll
            for (int x = 0; x < R8; ++x) mma16816(s[mt][x], a, q[x][k][0], q[x][k][1]);
          }
        }
      }
      // To log2 units; keys that a row does not see to -inf.
      float ev[MT][2];  // e4m3: the powers of the lane's keys' values
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int z = 0; z < 2; ++z) {
          float pk = 1.0f;
          if (E4M3) {
            const int r = 16 * (k16 + mt) + g + 8 * z;
            pk = exp_scale((uint8_t)lds_u8(ex + r));
            const uint32_t b = lds_u8(ex + KT + r);
            ev[mt][z] = b == 255 ? __int_as_float(0x7FC00000) : (float)((int)b - 127);
          }
#pragma unroll
          for (int x = 0; x < R8; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float& v = s[mt][x][2 * z + y];
              v = E4M3 ? v * unq[x][y] * pk * unq2[x][y] : v * p.scale_log2;
            }
        }
      if (!whole) {
        const int most = sink ? it.kt.cut : len;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int j = key0 + 16 * (k16 + mt) + g + 8 * z;
            const bool here = (mask >> (k16 + mt) & 1u) && j < most;
#pragma unroll
            for (int x = 0; x < R8; ++x)
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                const bool seen = here & (j < hi[x][y]) & ((j >= lo[x][y]) | (j < p.w.sinks));
                s[mt][x][2 * z + y] = seen ? s[mt][x][2 * z + y] : -INFINITY;
              }
          }
      }
      // Running maximum and sum; P^T as operand B, two 16-bit keys a register.
      uint32_t b[MT][R8][2];
#pragma unroll
      for (int x = 0; x < R8; ++x) {
        float top[2];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          float m;
          if (E4M3) {
            float mx = fmaxf(s[0][x][y], s[0][x][2 + y]);
            m = fmaxf(s[0][x][y] + ev[0][0], s[0][x][2 + y] + ev[0][1]);
#pragma unroll
            for (int mt = 1; mt < MT; ++mt) {
              mx = fmax3(mx, s[mt][x][y], s[mt][x][2 + y]);
              m = fmax3(m, s[mt][x][y] + ev[mt][0], s[mt][x][2 + y] + ev[mt][1]);
            }
            mx = fmaxf(mx, x_run[x][y]);
            if (mx > x_run[x][y]) l_run[x][y] *= ex2_approx(x_run[x][y] - mx);
            x_run[x][y] = mx;
            const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              l_run[x][y] += ex2_approx(s[mt][x][y] - ref) + ex2_approx(s[mt][x][2 + y] - ref);
          } else {
            m = fmaxf(s[0][x][y], s[0][x][2 + y]);
#pragma unroll
            for (int mt = 1; mt < MT; ++mt) m = fmax3(m, s[mt][x][y], s[mt][x][2 + y]);
          }
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
          top[y] = fmaxf(m, m_run[x][y]);
        }
        if (__any_sync(0xffffffffu, top[0] > m_run[x][0] || top[1] > m_run[x][1])) {
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            // x_j + e_j is rounded: the reference lies a step above it, so that P
            // stays in fp16's range where a step is more than its last binade.
            if (E4M3 && top[y] > m_run[x][y]) top[y] = fmaf(fabsf(top[y]), 0x1p-23f, top[y]);
            const float f = top[y] == -INFINITY ? 1.0f : ex2_approx(m_run[x][y] - top[y]);
            if (!E4M3) l_run[x][y] *= f;
            m_run[x][y] = top[y];
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              o[k][x][y] *= f;
              o[k][x][2 + y] *= f;
            }
          }
        }
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const float ref = m_run[x][y] == -INFINITY ? 0.0f : m_run[x][y];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              float& v = s[mt][x][2 * z + y];
              if (E4M3) {
                const float e = ex2_approx(v - ref + (ev[mt][z] + kPTop));
                v = whole || v != -INFINITY ? e : 0.0f;  // a masked key's power may be anything
              } else {
                v = ex2_approx(v - ref);
                l_run[x][y] += v;
              }
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          b[mt][x][0] = movmatrix_t(E4M3 ? pack_f16x2(s[mt][x][0], s[mt][x][1]) : pack_bf16x2(s[mt][x][0], s[mt][x][1]));
          b[mt][x][1] = movmatrix_t(E4M3 ? pack_f16x2(s[mt][x][2], s[mt][x][3]) : pack_bf16x2(s[mt][x][2], s[mt][x][3]));
        }
      }
      // O^T
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (E4M3) {
          constexpr int NB = D / 8;  // codes per lane and key row
          uint32_t w[4][NB / 4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            const int r = 16 * (k16 + mt) + 2 * c + (y & 1) + 8 * (y >> 1);
            if (D == 128) {
              const uint4 v = lds128(sv + r * D + ((g ^ (r & 7)) * 16));
              w[y][0] = v.x, w[y][1] = v.y, w[y][NB / 4 - 2] = v.z, w[y][NB / 4 - 1] = v.w;
            } else {
              const uint2 v = lds64(sv + r * D + (((g >> 1) ^ ((r >> 1) & 3)) * 16) + (g & 1) * 8);
              w[y][0] = v.x, w[y][1] = v.y;
            }
          }
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {  // rows g and g + 8 of step k: channels NB g + 2 k and + 1
            const int i = k / 2, h = (k & 1) * 2;
            uint32_t a[4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              // bytes h and h + 1 of both keys' words, key by key
              const uint32_t u = __byte_perm(w[2 * y][i], w[2 * y + 1][i], h == 0 ? 0x5140 : 0x7362);
              a[2 * y] = codes_to_f16(u);
              a[2 * y + 1] = codes_to_f16(u >> 16);
            }
#pragma unroll
            for (int x = 0; x < R8; ++x) mma16816_f16(o[k][x], a, b[mt][x][0], b[mt][x][1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const int r = 16 * (k16 + mt) + (lane & 7) + 8 * (lane >> 4), ch = 2 * k + ((lane >> 3) & 1);
            uint32_t a[4];
            ldsm4_t(sv + (ch / 8) * (KT * 128) + r * 128 + (((ch % 8) ^ (r & 7)) * 16), a);
#pragma unroll
            for (int x = 0; x < R8; ++x) mma16816(o[k][x], a, b[mt][x][0], b[mt][x][1]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(slot));
    }
    // Join the warps.
#pragma unroll
    for (int x = 0; x < R8; ++x)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float ref = m_run[x][y], f = 1.0f;
        if (E4M3) {
          ref = x_run[x][y];
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) ref = fmaxf(ref, __shfl_xor_sync(0xffffffffu, ref, d));
          if (x_run[x][y] != -INFINITY) l_run[x][y] *= ex2_approx(x_run[x][y] - ref);
          // From M to X in two halves: the whole may lie below 2^-126.
          if (m_run[x][y] != -INFINITY && ref != -INFINITY) f = ex2_approx(0.5f * (m_run[x][y] - ref - kPTop));
        }
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l_run[x][y] += __shfl_xor_sync(0xffffffffu, l_run[x][y], d);
        const int r = 8 * x + 2 * c + y;
        if (g == 0) wml[warp * L::kRows + r] = make_float2(ref, l_run[x][y]);
        float* dst = wo + (warp * L::kRows + r) * L::kOStride;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const int ch = E4M3 ? (D / 8) * g + 2 * k : 16 * k + g, ch2 = E4M3 ? ch + 1 : ch + 8;
          dst[ch] = E4M3 ? o[k][x][y] * f * f : o[k][x][y];
          dst[ch2] = E4M3 ? o[k][x][2 + y] * f * f : o[k][x][2 + y];
        }
      }
    asm volatile("bar.sync 1, %0;" ::"n"(NW * 32) : "memory");
    const bool all = at0 == 0 && stop == it.T;
    if (at0 == 0 && threadIdx.x < tokens)
      p.owners[(int64_t)(it.cu + t0 + threadIdx.x) * p.c.Hkv + it.hk] =
          make_int4(blockIdx.x, start < unit0, all ? (int)blockIdx.x : run_owner(W, ctas, unit0 + it.T - 1),
                    threadIdx.x * p.G);
    const int64_t slot0 = (int64_t)(2 * blockIdx.x + (start < unit0 ? 1 : 0)) * L::kRows;
    constexpr int TPR = D / 4;  // threads per row, four channels each
    for (int r = threadIdx.x / TPR; r < tokens * p.G; r += NW * 32 / TPR) {  // NW * 32 is a multiple of TPR
      const int ch = (threadIdx.x % TPR) * 4;
      float m = -INFINITY, l = 0.0f;
      float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < NW; ++w) m = fmaxf(m, wml[w * L::kRows + r].x);
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float2 ml = wml[w * L::kRows + r];
        const float f = ml.x == -INFINITY ? 0.0f : ex2_approx(ml.x - m);
        const float4 v = *reinterpret_cast<const float4*>(wo + (w * L::kRows + r) * L::kOStride + ch);
        l += ml.y * f;
        acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
      }
      if (all) {
        const int64_t row = (int64_t)(it.cu + t0 + r / p.G) * p.H + it.hk * p.G + r % p.G;
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
        *reinterpret_cast<uint2*>(p.O + row * D + ch) =
            make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
        if (p.lse && ch == 0) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
      } else {
        *reinterpret_cast<float4*>(p.part_o + (slot0 + r) * D + ch) = acc;
        if (ch == 0) p.part_ml[slot0 + r] = make_float2(m, l);
      }
    }
    // All leave together if one gave up.
    int gone;
    asm volatile(
        "{\n\t.reg .pred q, r;\n\tsetp.ne.b32 q, %1, 0;\n\tbarrier.cta.red.or.pred r, 1, %2, q;\n\t"
        "selp.b32 %0, 1, 0, r;\n\t}"
        : "=r"(gone)
        : "r"((int)(!ok || *abort_flag)), "n"(NW * 32)
        : "memory");
    if (gone || (left > 0 && !it.next(p))) break;
    at = 0;
  }
}

}  // namespace sparge
