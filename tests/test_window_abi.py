"""Refusals of the windowed-attention and paged-cache entry points (no GPU needed: nothing reaches a CUDA call)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_pooled_b200 import build

    build.build()
    from block_sparse_attention_pooled_b200 import sparge

    return sparge


P = ctypes.c_void_p(16 * 1024)  # never dereferenced: the checks come first
ODD = ctypes.c_void_p(16 * 1024 + 8)


def ref(x):
    return ctypes.byref(x)


def fwd(lib, shape=(1, 4, 2, 100, 128), win=(10, 0, 4, 1), args=None):
    a = dict(Q=P, K=P, V=P, lens=None, O=P, lse=None, ws=P, n=1 << 40)
    a.update(args or {})
    s = None if shape is None else ref(lib.WindowShape(*shape))
    w = None if win is None else ref(lib.Window(*win))
    return lib.raw().sparge_window_fwd(a["Q"], a["K"], a["V"], s, w, a["lens"], a["O"], a["lse"], a["ws"], a["n"], None)


def test_window_arguments(lib):
    bad = lib.ERR_INVALID_ARG
    assert fwd(lib, shape=None) == bad and fwd(lib, win=None) == bad
    for shape in ((0, 4, 2, 100, 128), (1, 4, 0, 100, 128), (1, 5, 2, 100, 128), (1, 4, 2, 0, 128), (1, 4, 2, -1, 128),
                  (1, 4, 2, 100, 0)):
        assert fwd(lib, shape=shape) == bad, shape
    for win in ((-2, 0, 0, 1), (0, -2, 0, 1), (0, 0, -1, 1), (0, 0, 0, 0)):
        assert fwd(lib, win=win) == bad, win
    for shape in ((1, 4, 2, 100, 96), (1, 4, 2, 100, 256), (1, 65536, 65536, 100, 64)):
        assert fwd(lib, shape=shape) == lib.ERR_UNSUPPORTED, shape
    for name in ("Q", "K", "V", "O"):
        assert fwd(lib, args={name: None}) == bad and fwd(lib, args={name: ODD}) == bad


def test_window_backward_arguments(lib):
    s, w = lib.WindowShape(1, 4, 2, 100, 128), lib.Window(10, 0, 4, 1)
    need = lib.raw().sparge_window_workspace_bytes(lib.OP_WINDOW_BWD, ref(s), ref(w))
    assert need >= 4 * 100 * 4
    assert lib.raw().sparge_window_workspace_bytes(lib.OP_WINDOW_BWD, ref(lib.WindowShape(1, 4, 3, 100, 128)), ref(w)) == 0

    def bwd(**k):
        a = [P, P, P, ref(s), ref(w), None] + [k.get(n, P) for n in ("O", "lse", "dO", "dQ", "dK", "dV", "ws")]
        return lib.raw().sparge_window_bwd(*a, k.get("n", need), None)

    for name in ("O", "lse", "dO", "dQ", "dK", "dV"):
        assert bwd(**{name: None}) == lib.ERR_INVALID_ARG, name
    for name in ("O", "dO", "dQ", "dK", "dV"):
        assert bwd(**{name: ODD}) == lib.ERR_INVALID_ARG, name
    assert bwd(ws=None) == lib.ERR_WORKSPACE and bwd(n=need - 1) == lib.ERR_WORKSPACE
    assert bwd(ws=ctypes.c_void_p(16 * 1024 + 64)) == lib.ERR_WORKSPACE


def cache(lib, **k):
    a = dict(k=16384, v=16384, k_exp=16384, v_exp=16384, pages=10, Hkv=2, page=64, d=128, type=lib.CACHE_E4M3)
    a.update(k)
    return lib.Cache(**a)


def batch(lib, **k):
    a = dict(page_table=16384, first=16384, cu=16384, B=3, max_pages=5, tokens=7)
    a.update(k)
    return lib.CacheBatch(**a)


def test_cache_arguments(lib):
    raw = lib.raw()

    def calls(c, b):
        w = lib.Window(-1, 0, 0, 1)
        cr, br = (None if x is None else ref(x) for x in (c, b))
        return {raw.sparge_cache_write(cr, br, P, 256, P, 256, None), raw.sparge_cache_read(cr, br, P, P, None),
                raw.sparge_cache_attn(cr, br, P, 1024, 8, 1, 100, ref(w), P, None, P, 1 << 40, None)}

    bad, not_done = {lib.ERR_INVALID_ARG}, {lib.ERR_UNSUPPORTED}
    assert calls(None, batch(lib)) == bad and calls(cache(lib), None) == bad
    for k in (dict(pages=0), dict(Hkv=0), dict(page=0), dict(d=0), dict(type=2), dict(type=-1), dict(k=None), dict(v=None),
              dict(k=16384 + 4), dict(k_exp=None), dict(v_exp=None)):
        assert calls(cache(lib, **k), batch(lib)) == bad, k
    for k in (dict(page=8), dict(page=48), dict(page=256), dict(d=96), dict(d=256), dict(pages=1 << 30, Hkv=4)):
        assert calls(cache(lib, **k), batch(lib)) == not_done, k
    for k in (dict(B=0), dict(max_pages=0), dict(tokens=-1), dict(page_table=None), dict(first=None), dict(cu=None)):
        assert calls(cache(lib), batch(lib, **k)) == bad, k
    assert calls(cache(lib), batch(lib, tokens=0)) == {lib.OK}
    c, b, w = cache(lib), batch(lib), lib.Window(-1, 0, 0, 1)
    for ks, vs in ((255, 256), (256, 248), (260, 256)):
        assert raw.sparge_cache_write(ref(c), ref(b), P, ks, P, vs, None) == lib.ERR_INVALID_ARG
    assert raw.sparge_cache_write(ref(c), ref(b), ODD, 256, P, 256, None) == lib.ERR_INVALID_ARG
    assert raw.sparge_cache_read(ref(c), ref(b), None, P, None) == lib.ERR_INVALID_ARG

    def attn(stride=1024, H=8, max_new=1, max_len=100, w=w, Q=P, O=P):
        return raw.sparge_cache_attn(ref(c), ref(b), Q, stride, H, max_new, max_len, ref(w), O, None, P, 1 << 40, None)

    for k in (dict(H=0), dict(H=7), dict(max_new=0), dict(max_len=0), dict(stride=1023), dict(stride=1028), dict(Q=None),
              dict(Q=ODD), dict(O=ODD), dict(w=lib.Window(0, 0, 0, 0)), dict(w=lib.Window(-3, 0, 0, 1))):
        assert attn(**k) == lib.ERR_INVALID_ARG, k


def test_shared_heads_have_a_limit(lib):
    """More than 128 query heads per K/V head: refused, and no workspace asked for (not a division by zero)."""
    raw, w = lib.raw(), lib.Window(-1, 0, 0, 1)
    c, b = cache(lib, Hkv=1), batch(lib, B=1, tokens=9)
    for H in (129, 256, 100000):
        assert raw.sparge_cache_attn(ref(c), ref(b), P, H * 128, H, 9, 100, ref(w), P, None, P, 1 << 40,
                                     None) == lib.ERR_UNSUPPORTED
        assert raw.sparge_cache_attn_workspace_bytes(ref(c), ref(b), H, 9, 100, ref(w)) == 0
    assert raw.sparge_cache_attn_workspace_bytes(ref(c), ref(b), 128, 9, 100, ref(w)) > 0
    for k in (dict(H=7, Hkv=2), dict(max_new=0), dict(max_len=0)):
        a = dict(H=8, Hkv=2, max_new=1, max_len=10) | k
        assert raw.sparge_cache_attn_workspace_bytes(ref(cache(lib, Hkv=a["Hkv"])), ref(b), a["H"], a["max_new"], a["max_len"],
                                                     ref(w)) == 0


def test_binding_refuses_cpu_tensors_and_wrong_shapes(lib):
    q = torch.zeros(1, 2, 64, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.sparge_window_fwd(q, q, q, 1, 0)
    with pytest.raises(ValueError):
        lib.sparge_window_bwd(q, q, q, q, q, q, 1, 0)
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lib.sparge_cache_write(t, t, q, q, i[None], i[:1], i)
    with pytest.raises(ValueError):
        lib.sparge_cache_read(q, q, i[None], i[:1], i, 3)
    with pytest.raises(ValueError):
        lib.sparge_cache_attn(t, q, q, i[None], i[:1], i, 1, 1)


@pytest.mark.parametrize("i,j,win,want", [
    (5, 5, (0, 0, 0, 1), True), (5, 4, (0, 0, 0, 1), False), (5, 6, (0, 0, 0, 1), False), (5, 6, (0, 1, 0, 1), True),
    (5, 0, (0, 0, 1, 1), True), (5, 1, (0, 0, 1, 1), False), (2, 5, (0, 0, 9, 1), False), (2, 5, (0, 0, 9, 3), False),
    (2, 2, (0, 0, 0, 3), True), (0, 2, (0, 0, 0, 3), True), (3, 2, (0, 0, 0, 3), False), (3, 2, (1, 0, 0, 3), True),
    (7, 0, (-1, 0, 0, 1), True), (0, 7, (-1, -1, 0, 1), True), (0, 8, (-1, -1, 0, 1), False), (8, 0, (-1, -1, 0, 1), False)])
def test_the_reference_rule(i, j, win, want):
    from window_ref import visible

    assert bool(visible(torch.tensor([i]), torch.tensor([j]), 8, *win)[0, 0]) is want
