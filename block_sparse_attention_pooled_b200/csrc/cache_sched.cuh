// How the work of attention over the paged cache is cut up. All lengths are in
// device memory, so the kernels find their shares themselves, in a few
// microseconds: that is most of a short call, so the walk keeps to 32 bits and
// one round of loads where it can.
//
// An item is a row tile (up to `tpt` consecutive new tokens of a sequence,
// times the G heads that share a K/V head) of one K/V head; its units are the
// key tiles of KT keys that any of its rows may see. The units of all items in
// order (sequence, row tile, K/V head) are dealt to the CTAs in equal
// contiguous runs: every CTA gets the same number of key tiles (to one),
// however ragged the batch is. A run that ends inside an item leaves a partial
// result; the CTA that has an item's first unit notes who holds the others
// (`owners`), and cache_combine_kernel joins them.
#pragma once
#include <cstdint>

#include "cache.cuh"
#include "window.cuh"

namespace sparge {

// The key tiles of a run of rows: `ns` tiles from key 0 that hold the sinks
// below `lo`, then tiles from `lo` on. A sink tile's keys at or past `cut` are
// not its own: they belong to the window's tiles or to nobody.
template <int KT>
struct KeyTilesT {
  int ns, total, lo, cut;
  __device__ __forceinline__ int key0(int t) const { return t < ns ? t * KT : lo + (t - ns) * KT; }
};

// lo: the first row's first key, rounded down by align_mask; hi: the last row's end.
template <int KT>
__device__ __forceinline__ KeyTilesT<KT> key_tiles_of(int lo, int hi, int sinks, int align_mask) {
  KeyTilesT<KT> k;
  k.lo = lo & ~align_mask;
  k.cut = min(min(sinks, hi), k.lo);
  k.ns = (k.cut + KT - 1) / KT;
  if (k.ns * KT >= k.lo) k.lo = k.cut = k.ns = 0;  // the sinks' tiles reach the window: one run of tiles
  k.total = k.ns + (max(hi - k.lo, 0) + KT - 1) / KT;
  return k;
}

struct CacheAttnParams {
  CacheView c;
  Window w;
  const __nv_bfloat16* Q;
  int64_t q_stride;
  __nv_bfloat16* O;
  float* lse;
  float* part_o;    // [2 * CTAs][rows][D]: a CTA's first and last partial
  float2* part_ml;  // [2 * CTAs][rows]: reference (log2) and sum
  int4* owners;     // [tokens][Hkv]: first CTA of the token's item, whether in its last partial, last CTA, row of head 0
  int H, G;
  int tpt;          // tokens per row tile
  int box_shift;    // log2 of the keys in one TMA box of pages
  int ctas;         // CTAs that the units are dealt to
  float scale_log2;
};

// One item and where its units lie. Held alike by all lanes of a warp.
template <int KT>
struct CacheItem {
  int b, tile, hk;      // sequence, row tile, K/V head
  int n, first, cu;     // the sequence's new tokens, its position, its first packed token
  KeyTilesT<KT> kt;
  int T;                // key tiles, at least 1

  __device__ __forceinline__ void seq(const CacheAttnParams& p, int seq) {
    b = seq;
    const int end = min(__ldg(p.c.cu + b + 1), p.c.tokens);
    cu = max(__ldg(p.c.cu + b), 0);
    n = max(end - cu, 0);
    first = max(__ldg(p.c.first + b), 0);
  }
  __device__ __forceinline__ int len() const { return first + n; }
  __device__ __forceinline__ void keys(const CacheAttnParams& p) {
    const int t0 = tile * p.tpt, t1 = min(n, t0 + p.tpt) - 1;
    kt = key_tiles_of<KT>(p.w.lo(first + t0), p.w.hi(first + t1, len()), p.w.sinks, (1 << p.c.page_shift) - 1);
    T = max(kt.total, 1);
  }
  // Unit `in` of the row tile's: its K/V head, and its place there.
  __device__ __forceinline__ void place(int64_t in, int& at) {
    if (in < INT32_MAX) {
      hk = (int)in / T;
      at = (int)in - hk * T;
    } else {
      hk = (int)(in / T);
      at = (int)(in % T);
    }
  }
  // To the next item; false past the last.
  __device__ __forceinline__ bool next(const CacheAttnParams& p) {
    if (++hk < p.c.Hkv) return true;
    hk = 0;
    if ((tile + 1) * p.tpt < n) {
      ++tile;
      keys(p);
      return true;
    }
    tile = 0;
    do {
      if (b + 1 >= p.c.B) return false;
      seq(p, b + 1);
    } while (n == 0);
    keys(p);
    return true;
  }
};

// Walks all (sequence, row tile) pairs, 32 at a time, and calls
// f(b, tile, units of one K/V head) on the lanes that hold one; f returns true
// to stop the walk. Called by a whole warp.
template <int KT, typename F>
__device__ __forceinline__ void walk_tiles(const CacheAttnParams& p, int lane, F f) {
  for (int b0 = 0; b0 < p.c.B; b0 += 32) {
    CacheItem<KT> it;
    int tiles = 0;
    it.n = it.first = it.cu = 0;
    if (b0 + lane < p.c.B) {
      it.seq(p, b0 + lane);
      tiles = (it.n + p.tpt - 1) / p.tpt;
    }
    int sum = tiles;  // inclusive prefix over the lanes
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const int all = __shfl_sync(0xffffffffu, sum, 31);
    for (int q0 = 0; q0 < all; q0 += 32) {
      const int q = q0 + lane;
      int src = 0;  // the lane whose sequence holds pair q: the first with sum > q
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const int v = __shfl_sync(0xffffffffu, sum, min(src + o - 1, 31));
        if (v <= q) src += o;
      }
      src = min(src, 31);
      CacheItem<KT> x;
      x.b = b0 + src;
      x.n = __shfl_sync(0xffffffffu, it.n, src);
      x.first = __shfl_sync(0xffffffffu, it.first, src);
      x.cu = __shfl_sync(0xffffffffu, it.cu, src);
      x.tile = q - (__shfl_sync(0xffffffffu, sum, src) - __shfl_sync(0xffffffffu, tiles, src));
      x.hk = 0;
      x.T = 0;
      if (q < all) x.keys(p);
      if (f(x)) return;
    }
  }
}

// The item that holds unit u (below their number) and u's place in it. Called by a whole warp.
template <int KT>
__device__ __forceinline__ CacheItem<KT> find_unit(const CacheAttnParams& p, int64_t u, int lane, int& at) {
  int64_t base = 0;
  CacheItem<KT> found;
  walk_tiles<KT>(p, lane, [&](const CacheItem<KT>& x) {
    int64_t sum = (int64_t)x.T * p.c.Hkv;
    const int64_t own = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    const unsigned past = __ballot_sync(0xffffffffu, base + sum > u);
    if (past == 0) {
      base += __shfl_sync(0xffffffffu, sum, 31);
      return false;
    }
    const int src = __ffs(past) - 1;
    found.b = __shfl_sync(0xffffffffu, x.b, src);
    found.tile = __shfl_sync(0xffffffffu, x.tile, src);
    found.n = __shfl_sync(0xffffffffu, x.n, src);
    found.first = __shfl_sync(0xffffffffu, x.first, src);
    found.cu = __shfl_sync(0xffffffffu, x.cu, src);
    base += __shfl_sync(0xffffffffu, sum - own, src);
    return true;
  });
  found.keys(p);
  found.place(u - base, at);
  return found;
}

// The page rows (cache_row) of an item's key tiles, a batch of tiles at a time:
// lane l holds box l % boxes of tile `base` + l / boxes, and the next batch is
// on its way, so no tile waits for the page table (its latency, once a tile,
// is as long as a tile's own bytes take).
template <int KT>
struct PageAhead {
  int boxes_shift, box_shift, base, stop;
  int64_t cur, nxt;
  __device__ __forceinline__ int64_t fetch(const CacheAttnParams& p, const CacheItem<KT>& it, int from, int lane) const {
    const int t = from + (lane >> boxes_shift);
    const int pos = it.kt.key0(t) + ((lane & ((1 << boxes_shift) - 1)) << box_shift);
    return t < stop && pos < it.len() ? cache_row(p.c, it.b, pos) : -1;
  }
  __device__ __forceinline__ int tiles() const { return 32 >> boxes_shift; }
  // Tiles at .. end - 1 of the item.
  __device__ __forceinline__ void start(const CacheAttnParams& p, const CacheItem<KT>& it, int at, int end, int lane) {
    box_shift = p.box_shift;
    boxes_shift = 31 - __clz(KT) - box_shift;
    base = at;
    stop = end;
    cur = fetch(p, it, base, lane);
    nxt = fetch(p, it, base + tiles(), lane);
  }
  // The row of box `lane` of tile t (lanes past the boxes: of some other box);
  // t does not decrease.
  __device__ __forceinline__ int64_t get(const CacheAttnParams& p, const CacheItem<KT>& it, int t, int lane) {
    if (t >= base + tiles()) {
      base += tiles();
      cur = nxt;
      nxt = fetch(p, it, base + tiles(), lane);
    }
    return __shfl_sync(0xffffffffu, cur, (((t - base) << boxes_shift) + lane) & 31);
  }
};

// CTAs that get a run: two units at least, so that a short cache does not end
// up in more partials than tiles.
__device__ __forceinline__ int ctas_used(int64_t W, int ctas) { return (int)max((int64_t)1, min((int64_t)ctas, W / 2)); }

// CTA c's units: [c W / ctas, (c + 1) W / ctas); and the CTA that has unit u.
__device__ __forceinline__ int64_t run_start(int64_t W, int ctas, int c) {
  return W < (1 << 20) ? (int64_t)((uint32_t)W * (uint32_t)c / (uint32_t)ctas) : W * c / ctas;
}
__device__ __forceinline__ int run_owner(int64_t W, int ctas, int64_t u) {
  return W < (1 << 20) ? (int)(((uint32_t)(u + 1) * (uint32_t)ctas - 1) / (uint32_t)W) : (int)(((u + 1) * ctas - 1) / W);
}

// CTA `cta`'s run: its first unit's item, that unit's place in it, and the
// units (0: none). ctas: the CTAs that get a run. Called by a whole warp. Up to
// 32 row tiles are gone through once (counting them and searching them in two
// walks took 2 us more, of 12 for one token of one stream); more take both.
template <int KT>
struct CacheRun {
  CacheItem<KT> it;
  int at, ctas;
  int64_t W, start, left;

  __device__ __forceinline__ void find(const CacheAttnParams& p, int cta, int lane) {
    CacheItem<KT> x;
    int rounds = 0;
    int64_t total = 0;
    x.T = 0;
    walk_tiles<KT>(p, lane, [&](const CacheItem<KT>& y) {
      total += y.T;
      if (y.T) x = y;
      ++rounds;
      return false;
    });
    at = 0;
    if (rounds != 1) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
      share(p, total, cta);
      if (left > 0) it = find_unit<KT>(p, start, lane, at);
      return;
    }
    int sum = x.T;  // at most 32 x 2^31 / KT: 32 bits do
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += v;
    }
    share(p, __shfl_sync(0xffffffffu, sum, 31), cta);
    if (left == 0) return;
    const int src = __ffs(__ballot_sync(0xffffffffu, (int64_t)sum * p.c.Hkv > start)) - 1;
    it.b = __shfl_sync(0xffffffffu, x.b, src);
    it.tile = __shfl_sync(0xffffffffu, x.tile, src);
    it.n = __shfl_sync(0xffffffffu, x.n, src);
    it.first = __shfl_sync(0xffffffffu, x.first, src);
    it.cu = __shfl_sync(0xffffffffu, x.cu, src);
    it.kt.ns = __shfl_sync(0xffffffffu, x.kt.ns, src);
    it.kt.total = __shfl_sync(0xffffffffu, x.kt.total, src);
    it.kt.lo = __shfl_sync(0xffffffffu, x.kt.lo, src);
    it.kt.cut = __shfl_sync(0xffffffffu, x.kt.cut, src);
    it.T = __shfl_sync(0xffffffffu, x.T, src);
    it.place(start - (int64_t)(__shfl_sync(0xffffffffu, sum, src) - it.T) * p.c.Hkv, at);
  }

 private:
  __device__ __forceinline__ void share(const CacheAttnParams& p, int64_t tiles, int cta) {
    W = tiles * p.c.Hkv;
    ctas = ctas_used(W, p.ctas);
    start = run_start(W, ctas, cta);
    left = cta < ctas ? run_start(W, ctas, cta + 1) - start : 0;
  }
};

// L lanes per (packed token, head): joins the partials of the item that the
// token's rows lie in, if there is more than one. rows: of a partial. A row is
// a chain of four loads (length, owner, sums, partials), so with many rows a
// warp takes four of them at once (a call over five chunks 130 -> 123 us); with
// few, whole warps share out the many partials that a row then has.
template <int D, int L>
__global__ void __launch_bounds__(128) cache_combine_kernel(const CacheAttnParams p, int rows) {
  grid_wait();
  constexpr int C = D / L, V = C < 4 ? C : 4, N = C / V;  // channels per lane, N runs of V neighbours
  const int lane = threadIdx.x % 32, sub = lane % L;
  const unsigned group = L == 32 ? 0xffffffffu : ((1u << (L % 32)) - 1u) << (lane - sub);
  const int64_t id = (int64_t)blockIdx.x * (128 / L) + threadIdx.x / L;
  const int t = (int)(id / p.H), h = (int)(id % p.H);
  if (t >= min(__ldg(p.c.cu + p.c.B), p.c.tokens)) return;
  const int4 own = p.owners[(int64_t)t * p.c.Hkv + h / p.G];
  const int c0 = own.x, c1 = own.z, r = own.w + h % p.G;
  if (c0 == c1) return;  // one CTA did it all
  if (c0 < 0 || c0 > c1 || c1 >= p.ctas || r < 0 || r >= rows) return;  // never noted: the kernel before gave up a wait
  auto slot = [&](int c) { return (int64_t)(2 * c + (c == c0 ? own.y : 0)) * rows + r; };
  float m = -INFINITY;
  for (int c = c0 + sub; c <= c1; c += L) m = fmaxf(m, p.part_ml[slot(c)].x);
#pragma unroll
  for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(group, m, o));
  float l = 0.0f, o[N][V] = {};
  for (int b = c0; b <= c1; b += L) {
    const int n = min(L, c1 + 1 - b);
    const float2 ml = sub < n ? p.part_ml[slot(b + sub)] : make_float2(0.0f, 0.0f);
    const float f = ml.y == 0.0f ? 0.0f : exp2f(ml.x - m);  // 0: saw nothing
    l += ml.y * f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float fi = __shfl_sync(group, f, i, L);
      const float* src = p.part_o + slot(b + i) * D + sub * V;
      float v[N][V];
#pragma unroll
      for (int j = 0; j < N; ++j) {
        if (V == 4) *reinterpret_cast<float4*>(v[j]) = *reinterpret_cast<const float4*>(src + j * L * V);
        else *reinterpret_cast<float2*>(v[j]) = *reinterpret_cast<const float2*>(src + j * L * V);
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) o[j][k] += v[j][k] * fi;
    }
  }
#pragma unroll
  for (int x = L / 2; x > 0; x >>= 1) l += __shfl_xor_sync(group, l, x);
  const int64_t row = (int64_t)t * p.H + h;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    uint32_t w[V / 2];
#pragma unroll
    for (int k = 0; k < V / 2; ++k) w[k] = pack_bf16x2(o[j][2 * k] * inv, o[j][2 * k + 1] * inv);
    __nv_bfloat16* out = p.O + row * D + (j * L + sub) * V;
    if (V == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[V / 2 - 1]);
    else *reinterpret_cast<uint32_t*>(out) = w[0];
  }
  if (p.lse && sub == 0) p.lse[row] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace sparge
