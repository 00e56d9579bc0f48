// Host side of the windowed-attention and paged-cache entry points (included
// by sparge.cu, which holds the shared checks and descriptor helpers).
#pragma once

namespace {

struct WDims {
  int64_t BH, BHkv, rows, keys;
};

bool window_ok(const sparge_window* w) {
  return w != nullptr && w->left >= -1 && w->right >= -1 && w->sinks >= 0 && w->unit >= 1;
}

Window device_window(const sparge_window* w) { return Window{w->left, w->right, w->sinks, w->unit}; }

sparge_status check_window(const sparge_window_shape* s, const sparge_window* w, WDims* out) {
  if (s == nullptr || !window_ok(w)) return SPARGE_ERR_INVALID_ARG;
  if (s->B <= 0 || s->H <= 0 || s->Hkv <= 0 || s->N <= 0 || s->d <= 0 || s->H % s->Hkv) return SPARGE_ERR_INVALID_ARG;
  if (s->d != 64 && s->d != 128) return SPARGE_ERR_UNSUPPORTED;
  out->BH = (int64_t)s->B * s->H;
  out->BHkv = (int64_t)s->B * s->Hkv;
  if (out->BHkv > 65535 || out->BH > INT32_MAX / 8) return SPARGE_ERR_UNSUPPORTED;
  out->rows = out->BH * s->N;
  out->keys = out->BHkv * s->N;
  if (ceil_div(out->rows, 4) > INT32_MAX || s->N > (1 << 30)) return SPARGE_ERR_UNSUPPORTED;
  return SPARGE_OK;
}

bool all_aligned16(std::initializer_list<const void*> ps) {
  for (const void* p : ps)
    if (p == nullptr || !aligned16(p)) return false;
  return true;
}

// Launches a kernel that waits itself (grid_wait) for the one before it in the
// stream, which this call launched: its blocks start, and get ready, while that
// one's last blocks still run.
template <typename... Params, typename... Args>
cudaError_t launch_next(void (*kernel)(Params...), unsigned grid, unsigned threads, size_t smem, cudaStream_t st,
                        const Args&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3(grid);
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &early;
  c.numAttrs = 1;
  cudaLaunchKernelEx(&c, kernel, Params(args)...);
  return cudaGetLastError();
}

// How the rows of dK and dV's key tiles are split, from what the host knows.
// A key that every later row sees (a sink, or any key where the past is not
// limited) has up to N rows per head, another as many as the window is wide;
// one CTA works through its rows in order, so long runs are cut into pieces of
// at most about a third of an SM's share of the whole work, or about its share
// where that is small (a piece's fp32 sums are written and read once more).
// Whole backward, us, with pieces of a sixth / a third / the whole share: 480p
// clip of frames 3180 / 3100 / 3099 (half the time is this kernel's), 12 heads x
// 8000 tokens that see 1024: 376 / 291 / 269, 8 x 4096 causal: 196 / 165 / 117.
// The third is not the best where runs are long. With little work, pieces of at
// least 2 / 8 tiles: 4 heads x 1000 tokens of d 64 29 / 35, 2 x 8 x 2047 76 / 78.
// (148: the SMs of the one GPU this is built for, so that the workspace does not
// depend on the current device.)
struct KvSplit {
  int tiles, sink_tiles, sink_pieces, pieces;
  size_t slots;  // of [2][128][d] fp32
};

KvSplit kv_split(const sparge_window_shape* s, const sparge_window* w, const WDims& d) {
  KvSplit k;
  k.tiles = (int)ceil_div(s->N, kWTile);
  const int64_t G = s->H / s->Hkv;
  const int64_t reach = std::min<int64_t>(
      s->N, w->left < 0 || w->right < 0 ? s->N : ((int64_t)w->left + w->right + 1) * w->unit + kWTile);
  k.sink_tiles = w->left < 0 ? 0 : (int)ceil_div(std::min(w->sinks, s->N), kWTile);
  const int64_t run = G * ceil_div(reach, kWTile), sink_run = G * k.tiles;
  const int64_t all = d.BHkv * (run * (k.tiles - k.sink_tiles) + sink_run * k.sink_tiles);
  // Little work is dealt in one piece per SM (a second round of CTAs would take
  // as long as the first).
  const int64_t sms = 148, share = ceil_div(all, sms);
  int64_t most = share > 24 ? share / 3 : std::max<int64_t>(8, share);
  for (;; ++most) {
    k.pieces = (int)std::min<int64_t>(ceil_div(run, most), 64);
    k.sink_pieces = (int)std::min<int64_t>(ceil_div(sink_run, most), 64);
    if (share > 24 || most >= sink_run ||
        d.BHkv * ((int64_t)k.sink_tiles * k.sink_pieces + (int64_t)(k.tiles - k.sink_tiles) * k.pieces) <= sms)
      break;
  }
  k.slots = k.sink_pieces > 1 ? (size_t)d.BHkv * k.sink_tiles * k.sink_pieces : 0;
  if (k.pieces > 1) k.slots += (size_t)d.BHkv * (k.tiles - k.sink_tiles) * k.pieces;
  return k;
}

size_t window_ws(int op, const sparge_window_shape* s, const sparge_window* w, const WDims& d) {
  if (op != SPARGE_OP_WINDOW_BWD) return 0;
  return align256((size_t)d.rows * 4) + kv_split(s, w, d).slots * 2 * kWTile * s->d * 4;
}

sparge_status check_ws(const void* ws, size_t have, size_t need) {
  if (need == 0) return SPARGE_OK;
  if (ws == nullptr || have < need || (reinterpret_cast<uintptr_t>(ws) & 255u)) return SPARGE_ERR_WORKSPACE;
  return SPARGE_OK;
}

// SMs of the current device.
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 148;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

template <int D>
sparge_status launch_window_fwd(const void* Q, const void* K, const void* V, const sparge_window_shape* s,
                                const sparge_window* w, const int32_t* lens, void* O, float* lse, const WDims& dm,
                                void* stream) {
  CUtensorMap mq, mk, mv;
  if (!make_map_bhnd(&mq, Q, dm.BH, s->N, D, kWTile) || !make_map_bhnd(&mk, K, dm.BHkv, s->N, D, kWTile) ||
      !make_map_bhnd(&mv, V, dm.BHkv, s->N, D, kWTile))
    return SPARGE_ERR_CUDA;
  WAttnParams p{};
  p.w = device_window(w);
  p.lens = lens;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.B = s->B;
  p.H = s->H;
  p.Hkv = s->Hkv;
  p.N = s->N;
  p.rtiles = (int)ceil_div(s->N, 2 * kWTile);
  if (dm.BH * p.rtiles > INT32_MAX / 2) return SPARGE_ERR_UNSUPPORTED;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)D));
  cudaError_t e = ensure_smem(window_fwd_kernel<D>, WSmem<D>::kBytes, D == 64 ? 20 : 21);
  if (e != cudaSuccess) return cuda_status(e);
  window_fwd_kernel<D><<<(unsigned)(dm.BH * p.rtiles), kWThreads, WSmem<D>::kBytes,
                         static_cast<cudaStream_t>(stream)>>>(mq, mk, mv, p);
  return cuda_status(cudaGetLastError());
}

template <int D>
sparge_status launch_window_bwd(const void* Q, const void* K, const void* V, const sparge_window_shape* s,
                                const sparge_window* w, const int32_t* lens, const void* O, const float* lse,
                                const void* dO, void* dQ, void* dK, void* dV, const WDims& dm, void* workspace,
                                void* stream) {
  CUtensorMap mq, mk, mv, mdo;
  if (!make_map_bhnd(&mq, Q, dm.BH, s->N, D, kWTile) || !make_map_bhnd(&mk, K, dm.BHkv, s->N, D, kWTile) ||
      !make_map_bhnd(&mv, V, dm.BHkv, s->N, D, kWTile) || !make_map_bhnd(&mdo, dO, dm.BH, s->N, D, kWTile))
    return SPARGE_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const KvSplit k = kv_split(s, w, dm);
  WBwdParams p{};
  p.w = device_window(w);
  p.lens = lens;
  p.O = static_cast<const __nv_bfloat16*>(O);
  p.dO = static_cast<const __nv_bfloat16*>(dO);
  p.lse = lse;
  p.dsum = static_cast<float*>(workspace);
  p.dQ = static_cast<__nv_bfloat16*>(dQ);
  p.dK = static_cast<__nv_bfloat16*>(dK);
  p.dV = static_cast<__nv_bfloat16*>(dV);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256((size_t)dm.rows * 4));
  p.B = s->B;
  p.H = s->H;
  p.Hkv = s->Hkv;
  p.N = s->N;
  p.rtiles = k.tiles;
  p.sink_tiles = k.sink_tiles;
  p.sink_pieces = k.sink_pieces;
  p.pieces = k.pieces;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)D));
  p.scale = (float)(1.0 / std::sqrt((double)D));
  const int64_t gq = dm.BH * k.tiles;
  const int64_t gk = dm.BHkv * ((int64_t)k.sink_tiles * k.sink_pieces + (int64_t)(k.tiles - k.sink_tiles) * k.pieces);
  if (gq > INT32_MAX || gk > INT32_MAX) return SPARGE_ERR_UNSUPPORTED;
  cudaError_t e = ensure_smem(window_dq_kernel<D>, WDqSmem<D>::kBytes, D == 64 ? 22 : 23);
  if (e != cudaSuccess) return cuda_status(e);
  window_dq_kernel<D><<<(unsigned)gq, kWThreads, WDqSmem<D>::kBytes, st>>>(mq, mk, mv, mdo, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  e = ensure_smem(window_dkdv_kernel<D>, WDkvSmem<D>::kBytes, D == 64 ? 24 : 25);
  if (e != cudaSuccess) return cuda_status(e);
  e = launch_next(window_dkdv_kernel<D>, (unsigned)gk, kWThreads, WDkvSmem<D>::kBytes, st, mq, mk, mv, mdo, p);
  if (e == cudaSuccess && k.slots > 0) {
    const int64_t quads = dm.BHkv * k.tiles * 2 * kWTile * (D / 4);
    if (ceil_div(quads, 256) > INT32_MAX) return SPARGE_ERR_UNSUPPORTED;
    e = launch_next(window_reduce_kernel<D>, (unsigned)ceil_div(quads, 256), 256, 0, st, p, quads);
  }
  return cuda_status(e);
}

// ---------------------------------------------------------------- paged cache
sparge_status check_cache(const sparge_cache* c, const sparge_cache_batch* b, CacheView* v) {
  if (c == nullptr || b == nullptr) return SPARGE_ERR_INVALID_ARG;
  if (c->pages <= 0 || c->Hkv <= 0 || c->page <= 0 || c->d <= 0 || b->B <= 0 || b->max_pages <= 0 || b->tokens < 0)
    return SPARGE_ERR_INVALID_ARG;
  if (c->type != SPARGE_CACHE_BF16 && c->type != SPARGE_CACHE_E4M3) return SPARGE_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return SPARGE_ERR_UNSUPPORTED;
  if (c->page != 16 && c->page != 32 && c->page != 64 && c->page != 128) return SPARGE_ERR_UNSUPPORTED;
  if (!all_aligned16({c->k, c->v})) return SPARGE_ERR_INVALID_ARG;
  if (c->type == SPARGE_CACHE_E4M3 && !all_aligned16({c->k_exp, c->v_exp})) return SPARGE_ERR_INVALID_ARG;
  if (!b->page_table || !b->first || !b->cu) return SPARGE_ERR_INVALID_ARG;
  if ((int64_t)c->pages * c->Hkv > INT32_MAX || c->Hkv > 65535) return SPARGE_ERR_UNSUPPORTED;
  if ((int64_t)b->tokens * c->Hkv * 2 > INT32_MAX) return SPARGE_ERR_UNSUPPORTED;
  v->k = static_cast<uint8_t*>(c->k);
  v->v = static_cast<uint8_t*>(c->v);
  v->k_exp = c->k_exp;
  v->v_exp = c->v_exp;
  v->table = b->page_table;
  v->first = b->first;
  v->cu = b->cu;
  v->pages = c->pages;
  v->Hkv = c->Hkv;
  v->page_shift = c->page == 16 ? 4 : c->page == 32 ? 5 : c->page == 64 ? 6 : 7;
  v->B = b->B;
  v->max_pages = b->max_pages;
  v->tokens = b->tokens;
  return SPARGE_OK;
}

// Which kernel, and its workspace: per CTA a first and a last partial of `rows` rows.
struct AttnPlan {
  int rows;  // 8, 16: cache_decode_kernel; 256: cache_chunk_kernel
  int tpt, ctas;
  size_t owners, bytes;  // offset of the owners, and all
};

// Up to 16 rows a sequence the time is the cache's bytes and mma.sync keeps up
// with them; more rows go to tcgen05, whose tiles have 128. 24 sequences of
// 16 k keys and 4 K/V heads, 16 rows, us by mma.sync / by tcgen05: d 128 bf16
// 130 / 169, e4m3 160 / 197; d 64 92 / 136 and 90 / 150; two such sequences
// 29 / 37 and 37 / 38. 20 rows take 157 (bf16) and 198 (e4m3) by tcgen05.
AttnPlan attn_plan(const sparge_cache* c, const sparge_cache_batch* b, int32_t H, int32_t max_new) {
  AttnPlan a;
  const int64_t G = H / c->Hkv, rows = G * std::min(max_new, b->tokens);
  a.rows = rows <= 8 ? 8 : rows <= 16 ? 16 : 2 * kWTile;
  a.tpt = a.rows <= 16 ? (int)(a.rows / G) : (int)(kWTile / G) * 2;
  a.ctas = sm_count();
  // Row tiles of one sequence read the same keys. Where all sequences have as
  // many, a whole number of CTAs per row tile keeps them at the same keys at the
  // same time, so that L2 serves all but the first (1560 rows over 32760 cached
  // tokens of 12 heads, 7 row tiles: 147 CTAs read 0.2 GB from memory, 148 1.3 GB).
  // It pays where few CTAs stand aside for it. Aligned from 15/16 of the CTAs on /
  // never / from 7/8 on, us over bf16: that frame 292 / 332 / 292, 4000 rows x 8
  // heads over 24 k 328 / 389 / 349, 2 x 700 tokens over 20 k 243 / 240 / 257,
  // 5 x 640 over 9 k 150 / 146 / 138.
  if (a.rows > 16 && (int64_t)b->B * max_new == b->tokens) {
    const int64_t tiles = (int64_t)b->B * ceil_div(max_new, a.tpt);
    const int64_t even = tiles > 0 ? a.ctas / tiles * tiles : 0;
    if (even * 16 >= (int64_t)a.ctas * 15) a.ctas = (int)even;
  }
  a.owners = align256((size_t)2 * a.ctas * a.rows * 8) + align256((size_t)2 * a.ctas * a.rows * c->d * 4);
  a.bytes = a.owners + align256((size_t)b->tokens * c->Hkv * 16);
  return a;
}

// Pages [pages * Hkv][page][d] with boxes of a page's rows: bf16 in 64-column
// boxes (64 rows at most) with the 128-byte swizzle, codes in whole rows with
// the swizzle of their width.
int box_rows(const sparge_cache* c) { return std::min(c->page, c->type == SPARGE_CACHE_E4M3 ? 128 : 64); }

bool make_map_pages(CUtensorMap* m, const void* base, const sparge_cache* c) {
  const bool q = c->type == SPARGE_CACHE_E4M3;
  const cuuint64_t width = q ? 1 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)c->d, (cuuint64_t)c->page, (cuuint64_t)c->pages * c->Hkv};
  cuuint64_t strides[2] = {c->d * width, (cuuint64_t)c->page * c->d * width};
  cuuint32_t box[3] = {q ? (cuuint32_t)c->d : 64, (cuuint32_t)box_rows(c), 1};
  return encode_map(m, q ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box,
                    q && c->d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Q as [Hkv][tokens][G][d] with (64 channels x G heads x tq tokens) boxes.
bool make_map_q(CUtensorMap* m, const CacheAttnParams& p, int d, int tq) {
  cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)p.G, (cuuint64_t)p.c.tokens, (cuuint64_t)p.c.Hkv};
  cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)p.q_stride * 2, (cuuint64_t)p.G * d * 2};
  cuuint32_t box[4] = {64, (cuuint32_t)p.G, (cuuint32_t)tq, 1};
  return encode_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p.Q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int D, bool E4M3, int R8>
cudaError_t launch_decode(const CUtensorMap& mk, const CUtensorMap& mv, const CacheAttnParams& p, cudaStream_t st) {
  using L = DecSmem<D, E4M3, R8>;
  cudaError_t e = ensure_smem(cache_decode_kernel<D, E4M3, R8>, L::kBytes, (D == 64 ? 0 : 4) + (E4M3 ? 2 : 0) + R8 - 1 + 32);
  if (e != cudaSuccess) return e;
  cache_decode_kernel<D, E4M3, R8><<<p.ctas, L::kThreads, L::kBytes, st>>>(mk, mv, p);
  return cudaGetLastError();
}

// Whole warps where the rows fit on the SMs at once that way (64 warps each), else eight lanes a row.
template <int D>
cudaError_t launch_combine(const CacheAttnParams& p, int rows, cudaStream_t st) {
  const int64_t n = (int64_t)p.c.tokens * p.H;
  if (n <= 64 * (int64_t)sm_count())
    return launch_next(cache_combine_kernel<D, 32>, (unsigned)ceil_div(n, 4), 128, 0, st, p, rows);
  return launch_next(cache_combine_kernel<D, 8>, (unsigned)ceil_div(n, 16), 128, 0, st, p, rows);
}

template <int D, bool E4M3>
sparge_status launch_cache_attn(const sparge_cache* c, const CacheAttnParams& p, const AttnPlan& plan, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!make_map_pages(&mk, c->k, c) || !make_map_pages(&mv, c->v, c)) return SPARGE_ERR_CUDA;
  cudaError_t e;
  if (plan.rows <= 16) {
    e = plan.rows == 8 ? launch_decode<D, E4M3, 1>(mk, mv, p, st) : launch_decode<D, E4M3, 2>(mk, mv, p, st);
    if (e != cudaSuccess) return cuda_status(e);
    return cuda_status(launch_combine<D>(p, plan.rows, st));
  }
  CUtensorMap mq;
  if (!make_map_q(&mq, p, D, plan.tpt / 2)) return SPARGE_ERR_CUDA;
  e = ensure_smem(cache_chunk_kernel<D, E4M3>, ChunkSmem<D, E4M3>::kBytes, 40 + (D == 64 ? 0 : 2) + (E4M3 ? 1 : 0));
  if (e != cudaSuccess) return cuda_status(e);
  cache_chunk_kernel<D, E4M3><<<p.ctas, chunk_threads<E4M3>(), ChunkSmem<D, E4M3>::kBytes, st>>>(mq, mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return cuda_status(e);
  return cuda_status(launch_combine<D>(p, plan.rows, st));
}

}  // namespace

extern "C" {

size_t sparge_window_workspace_bytes(int op, const sparge_window_shape* shape, const sparge_window* window) {
  WDims dm;
  if (check_window(shape, window, &dm) != SPARGE_OK) return 0;
  return window_ws(op, shape, window, dm);
}

sparge_status sparge_window_fwd(const void* Q, const void* K, const void* V, const sparge_window_shape* shape,
                                const sparge_window* window, const int32_t* lens, void* O, float* lse,
                                void* workspace, size_t workspace_bytes, void* stream) {
  WDims dm;
  sparge_status st = check_window(shape, window, &dm);
  if (st != SPARGE_OK) return st;
  if (!all_aligned16({Q, K, V, O})) return SPARGE_ERR_INVALID_ARG;
  st = check_ws(workspace, workspace_bytes, window_ws(SPARGE_OP_WINDOW_FWD, shape, window, dm));
  if (st != SPARGE_OK) return st;
  if (shape->d == 64) return launch_window_fwd<64>(Q, K, V, shape, window, lens, O, lse, dm, stream);
  return launch_window_fwd<128>(Q, K, V, shape, window, lens, O, lse, dm, stream);
}

sparge_status sparge_window_bwd(const void* Q, const void* K, const void* V, const sparge_window_shape* shape,
                                const sparge_window* window, const int32_t* lens, const void* O, const float* lse,
                                const void* dO, void* dQ, void* dK, void* dV, void* workspace,
                                size_t workspace_bytes, void* stream) {
  WDims dm;
  sparge_status st = check_window(shape, window, &dm);
  if (st != SPARGE_OK) return st;
  if (!all_aligned16({Q, K, V, O, dO, dQ, dK, dV}) || !lse) return SPARGE_ERR_INVALID_ARG;
  st = check_ws(workspace, workspace_bytes, window_ws(SPARGE_OP_WINDOW_BWD, shape, window, dm));
  if (st != SPARGE_OK) return st;
  if (shape->d == 64)
    return launch_window_bwd<64>(Q, K, V, shape, window, lens, O, lse, dO, dQ, dK, dV, dm, workspace, stream);
  return launch_window_bwd<128>(Q, K, V, shape, window, lens, O, lse, dO, dQ, dK, dV, dm, workspace, stream);
}

sparge_status sparge_cache_write(const sparge_cache* cache, const sparge_cache_batch* batch, const void* K,
                                 int64_t k_stride, const void* V, int64_t v_stride, void* stream) {
  CacheView v;
  sparge_status st = check_cache(cache, batch, &v);
  if (st != SPARGE_OK) return st;
  if (batch->tokens == 0) return SPARGE_OK;
  const int64_t least = (int64_t)cache->Hkv * cache->d;
  if (!all_aligned16({K, V}) || k_stride < least || v_stride < least || k_stride % 8 || v_stride % 8)
    return SPARGE_ERR_INVALID_ARG;
  const __nv_bfloat16 *k = static_cast<const __nv_bfloat16*>(K), *vv = static_cast<const __nv_bfloat16*>(V);
  const dim3 grid((unsigned)ceil_div(batch->tokens, kCacheWarps), (unsigned)ceil_div(2 * cache->Hkv, 4 * (cache->d == 64 ? 8 : 4)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool q = cache->type == SPARGE_CACHE_E4M3;
  if (cache->d == 64) {
    if (q) cache_write_kernel<64, true><<<grid, kCacheWarps * 32, 0, s>>>(v, k, k_stride, vv, v_stride);
    else cache_write_kernel<64, false><<<grid, kCacheWarps * 32, 0, s>>>(v, k, k_stride, vv, v_stride);
  } else {
    if (q) cache_write_kernel<128, true><<<grid, kCacheWarps * 32, 0, s>>>(v, k, k_stride, vv, v_stride);
    else cache_write_kernel<128, false><<<grid, kCacheWarps * 32, 0, s>>>(v, k, k_stride, vv, v_stride);
  }
  return cuda_status(cudaGetLastError());
}

sparge_status sparge_cache_read(const sparge_cache* cache, const sparge_cache_batch* batch, void* K, void* V,
                                void* stream) {
  CacheView v;
  sparge_status st = check_cache(cache, batch, &v);
  if (st != SPARGE_OK) return st;
  if (batch->tokens == 0) return SPARGE_OK;
  if (!all_aligned16({K, V})) return SPARGE_ERR_INVALID_ARG;
  __nv_bfloat16 *k = static_cast<__nv_bfloat16*>(K), *vv = static_cast<__nv_bfloat16*>(V);
  const dim3 grid((unsigned)ceil_div(batch->tokens, kCacheWarps), (unsigned)ceil_div(2 * cache->Hkv, 4 * (cache->d == 64 ? 8 : 4)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool q = cache->type == SPARGE_CACHE_E4M3;
  if (cache->d == 64) {
    if (q) cache_read_kernel<64, true><<<grid, kCacheWarps * 32, 0, s>>>(v, k, vv);
    else cache_read_kernel<64, false><<<grid, kCacheWarps * 32, 0, s>>>(v, k, vv);
  } else {
    if (q) cache_read_kernel<128, true><<<grid, kCacheWarps * 32, 0, s>>>(v, k, vv);
    else cache_read_kernel<128, false><<<grid, kCacheWarps * 32, 0, s>>>(v, k, vv);
  }
  return cuda_status(cudaGetLastError());
}

size_t sparge_cache_attn_workspace_bytes(const sparge_cache* cache, const sparge_cache_batch* batch, int32_t H,
                                         int32_t max_new, int32_t max_len, const sparge_window* window) {
  CacheView v;
  if (check_cache(cache, batch, &v) != SPARGE_OK) return 0;
  if (!window_ok(window) || H <= 0 || H % cache->Hkv || max_new < 1 || max_len < 1 || batch->tokens == 0) return 0;
  if ((int64_t)batch->tokens * H > INT32_MAX || H / cache->Hkv > kWTile) return 0;
  return attn_plan(cache, batch, H, max_new).bytes;
}

sparge_status sparge_cache_attn(const sparge_cache* cache, const sparge_cache_batch* batch, const void* Q,
                                int64_t q_stride, int32_t H, int32_t max_new, int32_t max_len,
                                const sparge_window* window, void* O, float* lse, void* workspace,
                                size_t workspace_bytes, void* stream) {
  CacheAttnParams p{};
  sparge_status st = check_cache(cache, batch, &p.c);
  if (st != SPARGE_OK) return st;
  if (!window_ok(window) || H <= 0 || H % cache->Hkv || max_new < 1 || max_len < 1) return SPARGE_ERR_INVALID_ARG;
  if ((int64_t)batch->tokens * H > INT32_MAX || H / cache->Hkv > kWTile) return SPARGE_ERR_UNSUPPORTED;
  if (batch->tokens == 0) return SPARGE_OK;
  if (!all_aligned16({Q, O}) || q_stride < (int64_t)H * cache->d || q_stride % 8) return SPARGE_ERR_INVALID_ARG;
  const AttnPlan plan = attn_plan(cache, batch, H, max_new);
  st = check_ws(workspace, workspace_bytes, plan.bytes);
  if (st != SPARGE_OK) return st;
  p.w = device_window(window);
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.q_stride = q_stride;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.lse = lse;
  p.part_ml = static_cast<float2*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + align256((size_t)2 * plan.ctas * plan.rows * 8));
  p.owners = reinterpret_cast<int4*>(static_cast<uint8_t*>(workspace) + plan.owners);
  p.H = H;
  p.G = H / cache->Hkv;
  p.tpt = plan.tpt;
  p.box_shift = 0;
  while ((1 << p.box_shift) < box_rows(cache)) ++p.box_shift;
  p.ctas = plan.ctas;
  p.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)cache->d));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool q = cache->type == SPARGE_CACHE_E4M3;
  if (cache->d == 64) return q ? launch_cache_attn<64, true>(cache, p, plan, s) : launch_cache_attn<64, false>(cache, p, plan, s);
  return q ? launch_cache_attn<128, true>(cache, p, plan, s) : launch_cache_attn<128, false>(cache, p, plan, s);
}

}  // extern "C"
