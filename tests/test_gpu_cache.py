"""The paged cache (write, read back, attention of new tokens) against the 64-bit definition."""
import math

import pytest
import torch

from window_ref import close, e4m3_rows, rows_fwd, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sparge():
    from block_sparse_attention_pooled_b200 import build

    build.build()
    from block_sparse_attention_pooled_b200 import sparge as m

    return m


def ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Paged:
    """A cache of NaN places, its page table, and what every position of each sequence should hold (float64)."""

    def __init__(self, kind, Hkv, d, page, lengths, seed=0, spare=2):
        self.g = torch.Generator(device="cuda")
        self.g.manual_seed(seed)
        self.kind, self.Hkv, self.d, self.page, self.B = kind, Hkv, d, page, len(lengths)
        need = [-(-n // page) for n in lengths]
        self.pages = sum(need) + spare
        ids = torch.randperm(self.pages, generator=self.g, device="cuda").to(torch.int32)
        self.table = torch.full((self.B, max(1, max(need))), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        shape = (self.pages, Hkv, page, d)
        if kind == "bf16":
            self.k, self.v = (torch.full(shape, math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2))
            self.exp = {}
        else:
            self.k, self.v = (torch.full(shape, 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
                              for _ in range(2))
            self.exp = {n: torch.full(shape[:3], 255, dtype=torch.uint8, device="cuda") for n in ("k_exp", "v_exp")}

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def fill(self, sparge, lengths):
        """Writes all positions; returns the values per sequence, [Hkv, n, d] in 64 bits, for K and V."""
        T = sum(lengths)
        k, v = self.normal(T, self.Hkv, self.d), self.normal(T, self.Hkv, self.d)
        cu = ints(*[sum(lengths[:b]) for b in range(self.B + 1)])
        sparge.sparge_cache_write(k, v, self.k, self.v, self.table, ints(*[0] * self.B), cu, **self.exp)
        if self.kind == "e4m3":
            k, v = e4m3_rows(k)[0], e4m3_rows(v)[0]
        cut = lambda x: [x[int(cu[b]):int(cu[b + 1])].double().transpose(0, 1) for b in range(self.B)]  # noqa: E731
        return cut(k), cut(v)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_write_then_read(sparge, kind, page, d):
    """Ragged batches (an empty one among them) at odd positions: every written place reads back as its one rounding,
    every other place keeps its bits, absent pages are neither written nor read."""
    past, new = [0, 5, page - 1, 3 * page + 7, 40], [page + 3, 0, 2, 1, 2 * page]
    c = Paged(kind, 3, d, page, [a + b for a, b in zip(past, new)])
    c.table[4, -(-(40 + 2 * page) // page) - 1] = c.pages  # the last page of the last sequence does not exist
    before = [t.view(torch.uint8).clone() for t in (c.k, c.v)]
    T = sum(new)
    wide = c.normal(T + 2, 3 * 3 * d)  # k and v as slices of a fused projection, two rows behind the last sequence
    wide[:, 3 * d:] *= torch.exp(torch.randn(T + 2, 1, generator=c.g, device="cuda") * 3).to(torch.bfloat16)
    k, v = wide[:, 3 * d:6 * d].unflatten(1, (3, d)), wide[:, 6 * d:].unflatten(1, (3, d))
    cu, first = ints(*[sum(new[:b]) for b in range(6)]), ints(*past)
    sparge.sparge_cache_write(k, v, c.k, c.v, c.table, first, cu, **c.exp)
    K = torch.full((T + 2, 3, d), 7.0, dtype=torch.bfloat16, device="cuda")
    V = K.clone()
    sparge.sparge_cache_read(c.k, c.v, c.table, first, cu, T + 2, K=K, V=V, **c.exp)
    torch.cuda.synchronize()
    want_k, want_v = (k.double(), v.double()) if kind == "bf16" else (e4m3_rows(k)[0], e4m3_rows(v)[0])
    touched = torch.zeros(c.pages, page, dtype=torch.bool, device="cuda")
    for b in range(5):
        for t in range(new[b]):
            p, row = past[b] + t, int(cu[b]) + t
            page_id = int(c.table[b, p // page])
            if page_id == c.pages:
                assert not K[row].any() and not V[row].any()
                continue
            touched[page_id, p % page] = True
            assert torch.equal(K[row].double(), want_k[row]) and torch.equal(V[row].double(), want_v[row])
    assert (K[T:] == 7).all() and (V[T:] == 7).all()
    for t, old in zip((c.k, c.v), before):
        now = t.view(torch.uint8)
        same = (now == old).flatten(3).all(-1)  # [pages, Hkv, page]
        assert same.transpose(1, 2)[~touched].all()


def test_exponents_at_the_edges(sparge):
    """Largest magnitudes around the type's 448, the ends of bf16's range, zeros, and rows that are not finite."""
    d = 64
    tops = [448.0, 449.0, 450.0, 447.0, 1.75, 1.7578125, 3.5, 7.0, 1.0, 3.0e38, 3.3e38, 2.0 ** -100, 2.0 ** -126, 1e-39, 0.0,
            math.inf, -math.inf, math.nan]
    c = Paged("e4m3", 1, d, 32, [len(tops)])
    k = c.normal(len(tops), d).float()
    k = (k / k.abs().amax(-1, keepdim=True) * 0.9).to(torch.bfloat16).float()
    t = torch.tensor(tops, device="cuda")[:, None]
    k = torch.where(torch.isfinite(t), k * torch.where(torch.isfinite(t), t, 0.0), k)
    k[:, 3] = t[:, 0]
    k = k[:, None].to(torch.bfloat16)
    cu, first = ints(0, len(tops)), ints(0)
    sparge.sparge_cache_write(k, k, c.k, c.v, c.table, first, cu, **c.exp)
    K, V = sparge.sparge_cache_read(c.k, c.v, c.table, first, cu, len(tops), **c.exp)
    want, byte = e4m3_rows(k)
    page = int(c.table[0, 0])
    assert torch.equal(c.exp["k_exp"][page, 0, :len(tops)], byte[:, 0])
    for got in (K, V):
        close(got, want, torch.zeros_like(want), "values")
    assert torch.isnan(K[-3:]).all()


def attn_check(sparge, kind, H, Hkv, d, page, past, new, win, seed=0, max_new=None, max_len=None, extra=0, drop=()):
    """Attention of ragged chunks; `drop`: (sequence, page column) pairs whose pages are gone."""
    left, right, sinks, unit = win
    total = [a + b for a, b in zip(past, new)]
    c = Paged(kind, Hkv, d, page, total, seed)
    ks, vs = c.fill(sparge, total)
    gone = {b: [col for bb, col in drop if bb == b] for b in range(c.B)}
    for b, col in drop:
        c.table[b, col] = -1
    T = sum(new)
    Q = c.normal(T + extra, H, d)
    O = torch.full((T + extra, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + extra, H), 7.0, device="cuda")
    cu = ints(*[sum(new[:b]) for b in range(c.B + 1)])
    got = sparge.sparge_cache_attn(Q, c.k, c.v, c.table, ints(*past), cu, max_new or max(1, max(new)),
                                   max_len or max(1, max(total)), left, right, sinks=sinks, unit=unit, O=O, lse=lse,
                                   **c.exp)
    assert got is O
    torch.cuda.synchronize()
    assert sparge.device_status() == 0
    assert (O[T:] == 7).all() and (lse[T:] == 7).all()
    for b in range(c.B):
        if not new[b]:
            continue
        at = torch.arange(total[b], device="cuda")
        seen = visible(at[past[b]:], at, total[b], left, right, sinks, unit)
        for col in gone[b]:
            seen[:, col * page:(col + 1) * page] = False
        r = slice(int(cu[b]), int(cu[b + 1]))
        for h in range(H):
            o, ls, to, _, tl = rows_fwd(Q[r, h], ks[b][h // (H // Hkv)], vs[b][h // (H // Hkv)], seen)
            close(O[r, h], o, to, f"O[{b}], head {h}")
            close(lse[r, h], ls, tl, f"lse[{b}], head {h}")


CAUSAL = (-1, 0, 0, 1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (4, 1), (8, 2), (6, 2), (16, 1), (40, 2), (12, 12)])
def test_single_tokens(sparge, kind, H, Hkv, d):
    attn_check(sparge, kind, H, Hkv, d, 16, [0, 1, 15, 63, 64, 130, 700], [1] * 7, CAUSAL)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("win", [CAUSAL, (100, 0, 0, 1), (100, 0, 5, 1), (63, 0, 200, 1), (0, 0, 0, 1), (0, 0, 1, 1),
                                 (1, 0, 50, 50)])
def test_single_tokens_with_windows(sparge, kind, page, win):
    attn_check(sparge, kind, 4, 2, 128, page, [0, 300, 999, 1500], [1, 1, 1, 1], win)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("new", [2, 3, 5, 16, 17, 33])
def test_few_tokens(sparge, kind, d, new):
    attn_check(sparge, kind, 6, 2, d, 32, [0, 200, 517], [new, 1, new], CAUSAL)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64, 128])
@pytest.mark.parametrize("win", [CAUSAL, (-1, -1, 0, 1), (150, 0, 70, 1), (1, 0, 100, 100), (0, 0, 0, 60), (30, 20, 3, 1)])
def test_ragged_chunks(sparge, kind, d, page, win):
    attn_check(sparge, kind, 4, 2, d, page, [0, 77, 1000, 5, 300], [300, 0, 129, 1, 256], win, extra=3)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (5, 1), (14, 2), (24, 1)])
def test_chunks_with_shared_heads(sparge, kind, H, Hkv):
    attn_check(sparge, kind, H, Hkv, 128, 64, [0, 321, 64], [130, 70, 64], (-1, 0, 0, 1))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 40, 150])
def test_dropped_pages_and_rows_that_see_nothing(sparge, kind, new):
    """Pages gone at the start, in the middle and under the rows themselves; sequence 1 has none left."""
    attn_check(sparge, kind, 4, 2, 128, 16, [400, 20, 100], [new, new, new], (200, 0, 40, 1),
               drop=[(0, 0), (0, 1), (0, 20), (0, 21)] + [(1, c) for c in range(-(-(20 + new) // 16))] + [(2, 6)])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 20, 200])
def test_bounds_only_split_the_work(sparge, kind, new):
    """max_new and max_len too small or far too large change nothing but the split."""
    for max_new, max_len in ((1, 1), (new, 4096), (10 ** 6, 10 ** 8)):
        attn_check(sparge, kind, 4, 1, 128, 32, [900, 17], [new, new], CAUSAL, max_new=max_new, max_len=max_len)


def test_long_cache_one_stream(sparge):
    attn_check(sparge, "bf16", 8, 2, 128, 64, [40000], [1], CAUSAL)
    attn_check(sparge, "e4m3", 8, 2, 128, 64, [40000], [9], CAUSAL)


def test_nothing_to_do(sparge):
    c = Paged("bf16", 1, 64, 16, [5])
    Q = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    assert sparge.sparge_cache_attn(Q, c.k, c.v, c.table, ints(5), ints(0, 0), 1, 5).shape == (0, 2, 64)
    kv = torch.empty(0, 1, 64, dtype=torch.bfloat16, device="cuda")
    sparge.sparge_cache_write(kv, kv, c.k, c.v, c.table, ints(5), ints(0, 0))
    assert sparge.sparge_cache_read(c.k, c.v, c.table, ints(0), ints(0, 0), 0)[0].shape == (0, 1, 64)
    attn_check(sparge, "bf16", 2, 1, 64, 16, [5], [0], CAUSAL, extra=4)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_new", [1, 16, 200])
@pytest.mark.parametrize("B", [1, 40])
def test_all_sequences_without_new_tokens(sparge, kind, max_new, B):
    """Whatever max_new promised: no row is written."""
    attn_check(sparge, kind, 4, 2, 128, 16, [100] * B, [0] * B, CAUSAL, max_new=max_new, extra=6)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 70])
def test_where_the_new_tokens_stand_in_a_batch(sparge, kind, new):
    """The sequences with new tokens among the first 32, behind them, in both parts; more than 32 row tiles of one."""
    for has in ((0, 31), (32,), (35, 37), (31, 32), (5, 39)):
        attn_check(sparge, kind, 4, 2, 64, 16, [30 * (b % 7) for b in range(40)], [new if b in has else 0 for b in range(40)],
                   CAUSAL, extra=2)
    attn_check(sparge, kind, 4, 1, 64, 64, [10, 300], [1, 2200 if new > 1 else 1], (50, 0, 0, 1), max_new=new)


def test_offsets_past_32_bits(sparge):
    """A pool of over 2^32 bytes and 2^31 values for each of K and V, its last pages in use."""
    Hkv, page, d = 8, 128, 128
    pages = (1 << 31) // (Hkv * page * d) + 40
    k = torch.empty(pages, Hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    table = (pages - 1 - torch.arange(20, device="cuda")).to(torch.int32)[None]
    n = 20 * page - 3
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    kn, vn, Q = (torch.randn(n, h, d, generator=g, device="cuda").to(torch.bfloat16) for h in (Hkv, Hkv, 8))
    cu = ints(0, n)
    sparge.sparge_cache_write(kn, vn, k, v, table, ints(0), cu)
    K, V = sparge.sparge_cache_read(k, v, table, ints(0), cu, n)
    assert torch.equal(K, kn) and torch.equal(V, vn)
    for new in (1, 300):
        O = sparge.sparge_cache_attn(Q[-new:], k, v, table, ints(n - new), ints(0, new), new, n)
        at = torch.arange(n, device="cuda")
        seen = visible(at[-new:], at, n, *CAUSAL)
        for h in (0, 7):
            o, _, to, _, _ = rows_fwd(Q[-new:, h], kn[:, h], vn[:, h], seen)
            close(O[:, h], o, to, f"head {h}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("new", [1, 100])
def test_strides_streams_and_graphs(sparge, kind, new):
    """Q as a slice of a fused projection; two streams at once; two graphs captured with one workspace pool and
    replayed after the lengths in device memory have moved."""
    past = [500, 130]
    c = Paged(kind, 2, 128, 32, [p + 2 * new for p in past])
    c.fill(sparge, [p + 2 * new for p in past])
    fused = c.normal(2 * new, 3 * 8 * 128)
    Q = fused[:, 8 * 128:2 * 8 * 128].unflatten(1, (8, 128))
    cu = ints(0, new, 2 * new)

    def call(first, stream=None):
        return sparge.sparge_cache_attn(Q, c.k, c.v, c.table, first, cu, new, 700, -1, 0, stream=stream, **c.exp)

    first, later = ints(*past), ints(*[p + new for p in past])
    dense = sparge.sparge_cache_attn(Q.contiguous(), c.k, c.v, c.table, first, cu, new, 700, -1, 0, **c.exp)
    assert torch.equal(call(first), dense)
    want = call(later)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [call(f, s) for f, s in zip((first, later), streams)]
    torch.cuda.synchronize()
    assert torch.equal(got[0], dense) and torch.equal(got[1], want)
    at = first.clone()
    graphs, outs = [], []
    for _ in range(2):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(at))
    for g, o in zip(graphs, outs):
        at.copy_(later)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        at.copy_(first)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, dense)
    assert sparge.device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_a_clip_generated_frame_by_frame(sparge, d):
    """The operators together: writing a clip's frames into a rolling bf16 cache, whose old pages are dropped, and
    attending frame by frame gives the windowed forward over the whole clip."""
    unit, frames, H, Hkv, page, left, sinks = 90, 7, 4, 2, 16, 2, 90
    N = unit * frames
    c = Paged("bf16", Hkv, d, page, [N, N])
    Q, K, V = (c.normal(2, h, N, d) for h in (H, Hkv, Hkv))
    lse = torch.empty(2, H, N, device="cuda")
    whole = sparge.sparge_window_fwd(Q, K, V, left, 0, sinks=sinks, unit=unit, lse=lse)
    at = torch.arange(N, device="cuda")
    seen = visible(at, at, N, left, 0, sinks, unit)
    keep = -(-sinks // page)
    for f in range(frames):
        now = slice(f * unit, (f + 1) * unit)
        pack = lambda x: x[:, :, now].transpose(1, 2).reshape(2 * unit, x.shape[1], d)  # noqa: E731
        first, cu = ints(f * unit, f * unit), ints(0, unit, 2 * unit)
        sparge.sparge_cache_write(pack(K), pack(V), c.k, c.v, c.table, first, cu)
        dead = max(0, f - left) * unit // page  # pages before the window, but for the sinks'
        c.table[:, keep:max(keep, dead)] = -1
        O = sparge.sparge_cache_attn(pack(Q), c.k, c.v, c.table, first, cu, unit, (f + 1) * unit, left, 0, sinks=sinks,
                                     unit=unit).view(2, unit, H, d).transpose(1, 2)
        for b in range(2):
            for h in range(H):
                o, _, to, _, _ = rows_fwd(Q[b, h, now], K[b, h // 2], V[b, h // 2], seen[now])
                close(O[b, h], o, to, f"frame {f}")
                close(whole[b, h, now], o, to, f"frame {f} of the whole clip")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("H", [8, 16, 32])
def test_a_large_batch_again_and_again(sparge, kind, H):
    """More sequences than lanes, runs that cross many items, calls back to back: every call gives the same bits."""
    Hkv, d, past = 4, 128, [3000 + 131 * b for b in range(40)]
    c = Paged(kind, Hkv, d, 64, [p + 1 for p in past])
    ks, vs = c.fill(sparge, [p + 1 for p in past])
    Q = c.normal(40, H, d)
    cu, first = torch.arange(41, dtype=torch.int32, device="cuda"), ints(*past)
    runs = [sparge.sparge_cache_attn(Q, c.k, c.v, c.table, first, cu, 1, max(past) + 1, **c.exp) for _ in range(20)]
    torch.cuda.synchronize()
    assert sparge.device_status() == 0
    for o in runs[1:]:
        assert torch.equal(o, runs[0])
    for b in (0, 17, 31, 32, 39):
        at = torch.arange(past[b] + 1, device="cuda")
        seen = visible(at[-1:], at, past[b] + 1, *CAUSAL)
        for h in range(0, H, 3):
            o, _, to, _, _ = rows_fwd(Q[b:b + 1, h], ks[b][h // (H // Hkv)], vs[b][h // (H // Hkv)], seen)
            close(runs[0][b:b + 1, h], o, to, f"sequence {b}, head {h}")


@pytest.mark.parametrize("new", [1, 50])
def test_a_row_of_the_cache_that_is_nan(sparge, new):
    """A token written with an infinity reads as NaN and makes the rows that see it NaN; rows that do not see it, and a
    row whose window has passed it, stay as they are."""
    c = Paged("e4m3", 1, 128, 32, [200 + new])
    k, v = c.normal(200 + new, 1, 128), c.normal(200 + new, 1, 128)
    k[150, 0, 3] = math.inf
    cu, first = ints(0, 200 + new), ints(0)
    sparge.sparge_cache_write(k, v, c.k, c.v, c.table, first, cu, **c.exp)
    K, V = sparge.sparge_cache_read(c.k, c.v, c.table, first, cu, 200 + new, **c.exp)
    assert torch.isnan(K[150]).all() and torch.isfinite(V).all() and torch.isfinite(K[151:]).all()
    Q = c.normal(new, 4, 128)
    for left, seen in ((-1, True), (20, False)):
        lse = torch.empty(new, 4, device="cuda")
        O = sparge.sparge_cache_attn(Q, c.k, c.v, c.table, ints(200), ints(0, new), new, 200 + new, left, 0, lse=lse, **c.exp)
        assert torch.isnan(O).all() == seen and torch.isnan(lse).all() == seen and torch.isfinite(O).all() == (not seen)


@pytest.mark.parametrize("new", [1, 60])
def test_output_at_any_16_bytes(sparge, new):
    c = Paged("bf16", 2, 64, 16, [300])
    c.fill(sparge, [300])
    Q = c.normal(new, 4, 64)
    args = (Q, c.k, c.v, c.table, ints(300 - new), ints(0, new), new, 300)
    want = sparge.sparge_cache_attn(*args)
    odd = torch.empty(Q.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(Q.shape)
    assert odd.data_ptr() % 32 == 16 and torch.equal(sparge.sparge_cache_attn(*args, O=odd), want)


@pytest.mark.parametrize("new", [1, 40])
def test_powers_at_both_ends(sparge, new):
    """Keys so small and values so large (and the other way round) that their powers lie near the ends of the range."""
    for ks, vs, qs in ((2.0 ** -60, 2.0 ** 60, 2.0 ** 60), (2.0 ** 40, 2.0 ** -40, 2.0 ** -40), (2.0 ** 10, 2.0 ** 100, 2.0 ** -10)):
        c = Paged("e4m3", 2, 64, 32, [300])
        k, v = c.normal(300, 2, 64) * ks, c.normal(300, 2, 64) * vs
        first, cu = ints(0), ints(0, 300)
        sparge.sparge_cache_write(k, v, c.k, c.v, c.table, first, cu, **c.exp)
        k64, v64 = (e4m3_rows(x)[0].transpose(0, 1) for x in (k, v))
        Q = c.normal(new, 4, 64) * qs
        O = sparge.sparge_cache_attn(Q, c.k, c.v, c.table, ints(300 - new), ints(0, new), new, 300, **c.exp)
        at = torch.arange(300, device="cuda")
        seen = visible(at[-new:], at, 300, *CAUSAL)
        for h in range(4):
            o, _, to, _, _ = rows_fwd(Q[:, h], k64[h // 2], v64[h // 2], seen)
            close(O[:, h], o, to, f"head {h}, keys {ks}")


def test_the_most_shared_heads(sparge):
    attn_check(sparge, "bf16", 128, 1, 64, 16, [70, 5], [1, 3], CAUSAL)
    attn_check(sparge, "e4m3", 100, 1, 128, 32, [150], [2], (40, 0, 3, 1))


def test_a_shared_prefix(sparge):
    """Two sequences whose tables begin with the same pages, and one sequence listed twice."""
    c = Paged("bf16", 2, 64, 16, [100, 100])
    ks, vs = c.fill(sparge, [100, 100])
    c.table[1, :4] = c.table[0, :4]
    k1, v1 = (torch.cat([x[0][:, :64], x[1][:, 64:]], 1) for x in (ks, vs))
    table = torch.stack([c.table[0], c.table[1], c.table[0]])
    for new in (1, 40):
        q = c.normal(new, 4, 64)
        Q = torch.cat([q, c.normal(new, 4, 64), q])
        O = sparge.sparge_cache_attn(Q, c.k, c.v, table, ints(*[100 - new] * 3), ints(0, new, 2 * new, 3 * new), new, 100)
        assert torch.equal(O[:new], O[2 * new:])
        at = torch.arange(100, device="cuda")
        seen = visible(at[-new:], at, 100, *CAUSAL)
        for b, (kk, vv) in enumerate(((ks[0], vs[0]), (k1, v1))):
            for h in range(4):
                o, _, to, _, _ = rows_fwd(Q[b * new:(b + 1) * new, h], kk[h // 2], vv[h // 2], seen)
                close(O[b * new:(b + 1) * new, h], o, to, f"sequence {b}, head {h}")
