"""What the compiled binding of the windowed and cached entry points refuses by itself, before the C ABI sees it."""
import threading

import pytest
import torch


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_pooled_b200 import build

    build.build()
    from block_sparse_attention_pooled_b200 import sparge

    return sparge


def test_tensors_of_the_host_are_refused(lib):
    q = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    n = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: lib.sparge_window_fwd(q, q, q, -1, 0),
                 lambda: lib.sparge_window_bwd(q, q, q, q, q, q, -1, 0),
                 lambda: lib.sparge_cache_write(q[0], q[0], q, q, n, n, n),
                 lambda: lib.sparge_cache_read(q, q, n, n, n, 3),
                 lambda: lib.sparge_cache_attn(q[0], q, q, n, n, n, 1, 8)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        lib.sparge_window_fwd(q, q, None, -1, 0)


def window_inputs(B=2, H=4, Hkv=2, N=40, d=64):
    g = torch.Generator(device="cuda").manual_seed(3)
    return [torch.randn(B, h, N, d, device="cuda", dtype=torch.bfloat16, generator=g) for h in (H, Hkv, Hkv)]


@pytest.mark.gpu
def test_window_tensors(lib):
    Q, K, V = window_inputs()
    O, lse = torch.empty_like(Q), torch.empty(Q.shape[:3], device="cuda")
    lib.sparge_window_fwd(Q, K, V, 5, 0, O=O, lse=lse)
    good = dict(Q=Q, K=K, V=V, O=O, lse=lse, lens=None)

    def refused(**k):
        a = {**good, **k}
        with pytest.raises(ValueError):
            lib.sparge_window_fwd(a["Q"], a["K"], a["V"], 5, 0, lens=a["lens"], O=a["O"], lse=a["lse"])
        with pytest.raises(ValueError):
            lib.sparge_window_bwd(a["Q"], a["K"], a["V"], a["O"], a["lse"], torch.ones_like(O), 5, 0, lens=a["lens"])

    for name in ("Q", "K", "V", "O", "lse"):
        t = good[name]
        refused(**{name: t.half()})
        refused(**{name: t.cpu()})
        refused(**{name: t[:1]})
        refused(**{name: t.transpose(1, 2)})
        refused(**{name: t.repeat_interleave(2, -1)[..., ::2]})
    n = torch.full((2,), 7, dtype=torch.int32, device="cuda")
    for lens in (n.long(), n.cpu(), n[:1], n.repeat_interleave(2)[::2], n[None]):
        refused(lens=lens)
    for name, like in (("dQ", Q), ("dK", K), ("dV", V)):
        for t in (like.half(), like[:1], like.cpu()):
            with pytest.raises(ValueError):
                lib.sparge_window_bwd(Q, K, V, O, lse, O, 5, 0, **{name: t})
    with pytest.raises(ValueError):
        lib.sparge_window_bwd(Q, K, V, O, lse, O, 5, 0, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(lib.SpargeError) as e:
        lib.sparge_window_bwd(Q, K, V, O, lse, O, 5, 0, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == lib.ERR_WORKSPACE
    with pytest.raises(lib.SpargeError) as e:
        lib.sparge_window_fwd(Q, K, V, -2, 0)
    assert e.value.code == lib.ERR_INVALID_ARG and "sparge_window_fwd" in str(e.value)
    for bad in (1 << 31, 0.5, None):
        with pytest.raises(TypeError):
            lib.sparge_window_fwd(Q, K, V, bad, 0)


@pytest.mark.gpu
def test_cache_tensors(lib):
    dev = "cuda"
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device=dev)
    codes = pages.to(torch.float8_e4m3fn)
    exps = torch.full((4, 2, 16), 127, dtype=torch.uint8, device=dev)
    table = torch.arange(4, dtype=torch.int32, device=dev).view(2, 2)
    first = torch.zeros(2, dtype=torch.int32, device=dev)
    cu = torch.tensor([0, 3, 5], dtype=torch.int32, device=dev)
    new = torch.randn(5, 2, 64, device=dev).bfloat16()
    Q = torch.randn(5, 4, 64, device=dev).bfloat16()
    good = dict(k=new, v=new, kp=pages, vp=pages.clone(), table=table, first=first, cu=cu, ke=None, ve=None, Q=Q, tokens=5)
    fp8 = dict(kp=codes, vp=codes.clone(), ke=exps, ve=exps)

    def calls(a):
        return (lambda: lib.sparge_cache_write(a["k"], a["v"], a["kp"], a["vp"], a["table"], a["first"], a["cu"],
                                               a["ke"], a["ve"]),
                lambda: lib.sparge_cache_read(a["kp"], a["vp"], a["table"], a["first"], a["cu"], a["tokens"], a["ke"],
                                              a["ve"]),
                lambda: lib.sparge_cache_attn(a["Q"], a["kp"], a["vp"], a["table"], a["first"], a["cu"], 3, 32,
                                              k_exp=a["ke"], v_exp=a["ve"]))

    for base in (good, {**good, **fp8}):
        for call in calls(base):
            call()

    def refused(which=(0, 1, 2), **k):
        for i, call in enumerate(calls({**good, **k})):
            if i in which:
                with pytest.raises((ValueError, lib.SpargeError)):  # one query head for two K/V heads: the C ABI's refusal
                    call()

    for name in ("kp", "vp"):
        for t in (pages.half(), pages.cpu(), pages[:2], pages.transpose(1, 2), codes, pages[0]):
            refused(**{name: t})
    refused(kp=pages.half(), vp=pages.half())
    refused(ke=exps)
    refused(**{**fp8, "ke": None})
    refused(**{**fp8, "ve": exps[:2]})
    refused(**{**fp8, "ve": exps.char()})
    refused(**{**fp8, "ve": exps.cpu()})
    for name in ("table", "first", "cu"):
        t = good[name]
        for bad in (t.long(), t.cpu(), t[:1], t[None], t.repeat_interleave(2, -1)[..., ::2]):
            refused(**{name: bad})
    for name, which in (("k", (0,)), ("v", (0,)), ("Q", (2,))):
        t = good[name]
        for bad in (t.half(), t.cpu(), t[0], t[:, :1], t[..., :32], t.repeat_interleave(2, -1)[..., ::2],
                    t.transpose(0, 1).contiguous().transpose(0, 1)):
            refused(which, **{name: bad})
    refused((0,), k=new[:4])
    refused((1,), tokens=-1)
    refused((1,), tokens=1 << 31)
    huge = torch.empty(1, 2, 64, dtype=torch.bfloat16, device=dev).expand(1 << 31, 2, 64)  # one token's memory
    refused((0,), k=huge, v=huge)
    refused((2,), Q=torch.empty(1, 4, 64, dtype=torch.bfloat16, device=dev).expand(1 << 31, 4, 64))
    for out in (dict(O=Q[:4].contiguous()), dict(O=Q.half()), dict(lse=torch.empty(4, 5, device=dev)),
                dict(lse=torch.empty(5, 4)), dict(workspace=torch.empty(1 << 20, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            lib.sparge_cache_attn(Q, pages, pages, table, first, cu, 3, 32, **out)
    for out in (dict(K=new[:4].contiguous()), dict(V=new.half())):
        with pytest.raises(ValueError):
            lib.sparge_cache_read(pages, pages, table, first, cu, 5, **out)
    with pytest.raises(lib.SpargeError) as e:
        lib.sparge_cache_attn(Q, pages, pages, table, first, cu, 0, 32)
    assert e.value.code == lib.ERR_INVALID_ARG


@pytest.mark.gpu
def test_threads_call_at_once(lib):
    """Four threads, each with its own stream: the same results as one after the other."""
    ins = [window_inputs(N=100 + 37 * i) for i in range(4)]
    want = [lib.sparge_window_fwd(*t, 20, 0) for t in ins]
    torch.cuda.synchronize()
    got = [[] for _ in ins]

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(50):
            got[i].append(lib.sparge_window_fwd(*ins[i], 20, 0, stream=s))
        s.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(4):
        assert len(got[i]) == 50 and all(torch.equal(o, want[i]) for o in got[i])


@pytest.mark.gpu
def test_outputs_for_another_stream(lib):
    """Memory that the current stream has freed, with work on it still queued there, does not become another stream's
    output; and an output is not handed out again while the current stream still reads it."""
    ins = window_inputs(B=1, H=8, Hkv=2, N=1000)
    want = lib.sparge_window_fwd(*ins, 20, 0)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(40_000_000)  # some 20 ms
    torch.empty_like(want).fill_(7)
    got = lib.sparge_window_fwd(*ins, 20, 0, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda._sleep(40_000_000)
    copy = got.clone()
    del got
    with torch.cuda.stream(s):
        torch.empty_like(want).fill_(9)
    torch.cuda.synchronize()
    assert torch.equal(copy, want)


@pytest.mark.gpu
def test_forward_workspace_is_checked(lib):
    """The windowed forward looks at a workspace as the other calls do."""
    Q, K, V = window_inputs()
    want = lib.sparge_window_fwd(Q, K, V, 5, 0)
    assert torch.equal(lib.sparge_window_fwd(Q, K, V, 5, 0, workspace=torch.empty(256, dtype=torch.uint8, device="cuda")), want)
    for bad in (torch.empty(256, dtype=torch.uint8), torch.empty(256, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError):
            lib.sparge_window_fwd(Q, K, V, 5, 0, workspace=bad)
    with pytest.raises(TypeError):
        lib.sparge_window_fwd(Q, K, V, 5, 0, workspace=256)


def test_binding_is_rebuilt_for_another_torch(lib, monkeypatch, tmp_path):
    """Up to date: left alone. Built for another torch, or not known for which: built anew, and noted."""
    from block_sparse_attention_pooled_b200 import build

    built, note = [], tmp_path / "sub" / "bind_for.txt"
    monkeypatch.setattr(build, "_build_bind", lambda: built.append(1))
    build.build()
    assert built == []
    monkeypatch.setattr(build, "BIND_FOR", str(note))
    build.build()
    assert built == [1]
    build.build()
    assert built == [1]
    note.write_text("torch 2.10.0, Python 3.12.3")
    build.build()
    assert built == [1, 1]
    build.build()
    assert built == [1, 1]


def test_without_the_compiled_binding(lib):
    """The entry points that it does not serve work without it; the others say what is missing when they are called."""
    import subprocess
    import sys

    code = """
import sys
sys.modules["block_sparse_attention_pooled_b200._bind"] = None  # its import raises ImportError
from block_sparse_attention_pooled_b200 import sparge
assert sparge.workspace_bytes(sparge.OP_ATTN_BWD, sparge.Shape(1, 2, 1000, 128, 128, 64)) > 0
for name, args in (("sparge_window_fwd", (1, 1, 1, 0, 0)), ("sparge_window_bwd", (1,) * 6 + (0, 0)),
                   ("sparge_cache_write", (1,) * 7), ("sparge_cache_read", (1,) * 6), ("sparge_cache_attn", (1,) * 8)):
    try:
        getattr(sparge, name)(*args)
    except ImportError as e:
        assert "_bind" in str(e) and "build" in str(e), e
    else:
        raise AssertionError(name)
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=build_root())


def build_root():
    from block_sparse_attention_pooled_b200 import build

    return build.ROOT
