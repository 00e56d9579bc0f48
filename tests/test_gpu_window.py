"""Windowed attention (forward and backward) against the 64-bit definition, at the sizes and masks where a tiled
kernel can go wrong."""
import pytest
import torch

from window_ref import close, rows_bwd, rows_fwd, visible

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sparge():
    from block_sparse_attention_pooled_b200 import build

    build.build()
    from block_sparse_attention_pooled_b200 import sparge as m

    return m


def inputs(B, H, Hkv, N, d, seed=0, lens=None, pad=float("nan")):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = [torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
         for s in ((B, H, N, d), (B, Hkv, N, d), (B, Hkv, N, d), (B, H, N, d))]
    if lens is not None:
        for b, n in enumerate(lens):
            for t in x:
                t[b, :, n:] = pad
    return x


def check(sparge, Q, K, V, dO, win, lens=None, grads=True):
    B, H, N, d = Q.shape
    Hkv = K.shape[1]
    left, right, sinks, unit = win
    lt = None if lens is None else torch.tensor(lens, dtype=torch.int32, device="cuda")
    lse = torch.empty(B, H, N, device="cuda")
    O = sparge.sparge_window_fwd(Q, K, V, left, right, sinks=sinks, unit=unit, lens=lt, lse=lse)
    G = sparge.sparge_window_bwd(Q, K, V, O, lse, dO, left, right, sinks=sinks, unit=unit, lens=lt) if grads else None
    torch.cuda.synchronize()
    assert sparge.device_status() == 0
    at = torch.arange(N, device="cuda")
    for b in range(B):
        L = N if lens is None else lens[b]
        seen = visible(at, at, L, left, right, sinks, unit)
        for hk in range(Hkv):
            dk = dv = tk = tv = 0.0
            for h in range(hk * (H // Hkv), (hk + 1) * (H // Hkv)):
                o, ls, to, P, tl = rows_fwd(Q[b, h], K[b, hk], V[b, hk], seen)
                close(O[b, h], o, to, f"O[{b},{h}]")
                close(lse[b, h], ls, tl, f"lse[{b},{h}]")
                if grads:
                    (dq, a, c), (tq, ta, tc) = rows_bwd(Q[b, h], K[b, hk], V[b, hk], dO[b, h], P, o, to, seen)
                    close(G[0][b, h], dq, tq + dq.abs() * 2.0 ** -8, f"dQ[{b},{h}]")
                    dk, dv, tk, tv = dk + a, dv + c, tk + ta, tv + tc
            if grads:
                close(G[1][b, hk], dk, tk + dk.abs() * 2.0 ** -8, f"dK[{b},{hk}]")
                close(G[2][b, hk], dv, tv + dv.abs() * 2.0 ** -8, f"dV[{b},{hk}]")
    return O, lse, G


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 513])
def test_lengths(sparge, N, d):
    check(sparge, *inputs(1, 2, 2, N, d, seed=N), (-1, 0, 0, 1))
    check(sparge, *inputs(1, 2, 1, N, d, seed=N + 1), (33, 5, 3, 1))


WINDOWS = [(-1, -1, 0, 1), (-1, 0, 0, 1), (0, 0, 0, 1), (0, 0, 1, 1), (63, 0, 4, 1), (64, 0, 128, 1), (127, 127, 0, 1),
           (200, 0, 130, 1), (0, -1, 7, 1), (1, 0, 100, 100), (2, 1, 65, 64), (0, 0, 0, 97), (0, 0, 97, 97),
           (5, 0, 10 ** 9, 1), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (3, 0, 129, 50), (1, 2, 1, 300)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("win", WINDOWS)
def test_windows(sparge, win, d):
    check(sparge, *inputs(1, 2, 2, 700, d, seed=5), win)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv", [(3, 1), (6, 2), (8, 1), (4, 4)])
def test_shared_heads(sparge, H, Hkv, d):
    check(sparge, *inputs(2, H, Hkv, 333, d, seed=H), (100, 0, 20, 1))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("win", [(-1, 0, 0, 1), (100, 0, 70, 1), (-1, -1, 0, 1), (1, 0, 64, 64), (90, 90, 0, 1)])
def test_padded_batch_with_nan_in_the_padding(sparge, win, d):
    lens = [400, 0, 1, 129, 256]
    x = inputs(5, 2, 1, 400, d, seed=9, lens=lens)
    O, lse, G = check(sparge, *x, win, lens=lens)
    for b, n in enumerate(lens):
        assert not O[b, :, n:].any() and (lse[b, :, n:] == -float("inf")).all()
        for t in G:
            assert not t[b, :, n:].any()


def test_lengths_past_the_tensor_are_cut(sparge):
    x = inputs(2, 1, 1, 100, 128)
    far = torch.tensor([10 ** 6, -5], dtype=torch.int32, device="cuda")
    O = sparge.sparge_window_fwd(*x[:3], -1, 0, lens=far)
    assert torch.equal(O[0], sparge.sparge_window_fwd(*x[:3], -1, 0)[0]) and not O[1].any()


@pytest.mark.parametrize("scale", [12.0, 0.0])
def test_peaked_and_flat_rows(sparge, scale):
    """Scores of hundreds (one key takes all, the running maximum jumps late) and all equal."""
    Q, K, V, dO = inputs(1, 1, 1, 600, 128, seed=3)
    check(sparge, Q * scale, K, V, dO, (-1, 0, 0, 1))


def test_long_sequence_against_sampled_rows(sparge):
    """Far rows of a long clip with frame units: sinks and window tiles far apart."""
    N, unit, sinks = 32760, 1560, 1560
    Q, K, V, _ = inputs(1, 2, 1, N, 128, seed=4)
    lse = torch.empty(1, 2, N, device="cuda")
    O = sparge.sparge_window_fwd(Q, K, V, 2, 0, sinks=sinks, unit=unit, lse=lse)
    rows = torch.arange(0, N, 97, device="cuda")
    seen = visible(rows, torch.arange(N, device="cuda"), N, 2, 0, sinks, unit)
    for h in range(2):
        o, ls, to, _, tl = rows_fwd(Q[0, h][rows], K[0, 0], V[0, 0], seen)
        close(O[0, h][rows], o, to, "O")
        close(lse[0, h][rows], ls, tl, "lse")


def test_gradients_against_differences(sparge):
    """d/dx of sum(O dO) from the 64-bit forward's central differences along random directions: the definition's
    gradient and the kernel's agree with it (the kernel's within its own tolerance along the direction)."""
    Q, K, V, dO = inputs(1, 2, 1, 150, 64, seed=11)
    win = (40, 3, 5, 1)
    _, _, G = check(sparge, Q, K, V, dO, win)
    at = torch.arange(150, device="cuda")
    seen = visible(at, at, 150, *win)

    def loss(q, k, v):
        return sum((rows_fwd(q[0, h], k[0, 0], v[0, 0], seen)[0] * dO[0, h].double()).sum() for h in range(2))

    x = [Q.double(), K.double(), V.double()]
    for n in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(n)
        u = torch.randn(x[n].shape, generator=g, device="cuda", dtype=torch.float64)
        h = 1e-5
        up, down = [list(x), list(x)]
        up[n], down[n] = x[n] + h * u, x[n] - h * u
        want = (loss(*up) - loss(*down)) / (2 * h)
        got = (G[n].double() * u).sum()
        # the sum of 9600 or more products, each off by a few 2^-8 of values of this norm, of either sign
        assert abs(got - want) <= 8 * 2.0 ** -8 * G[n].double().norm(), (n, got, want)


def test_identical_calls_give_identical_bits(sparge):
    Q, K, V, dO = inputs(2, 4, 2, 1111, 128, seed=6)
    runs = []
    for _ in range(3):
        lse = torch.empty(2, 4, 1111, device="cuda")
        O = sparge.sparge_window_fwd(Q, K, V, 300, 0, sinks=200, lse=lse)
        runs.append((O, lse) + sparge.sparge_window_bwd(Q, K, V, O, lse, dO, 300, 0, sinks=200))
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_other_stream_and_graph(sparge):
    """On a stream of its own, two at once, and captured and replayed on new inputs."""
    Q, K, V, dO = inputs(1, 4, 2, 777, 128, seed=7)
    args = (200, 0, 64)
    lse = torch.empty(1, 4, 777, device="cuda")
    O = sparge.sparge_window_fwd(Q, K, V, *args, lse=lse)
    want = (O,) + sparge.sparge_window_bwd(Q, K, V, O, lse, dO, *args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got, own = [], [torch.empty_like(lse) for _ in streams]  # the caller's buffers live until the streams are done
    for s, l2 in zip(streams, own):
        o = sparge.sparge_window_fwd(Q, K, V, *args, lse=l2, stream=s)
        got.append((o,) + sparge.sparge_window_bwd(Q, K, V, o, l2, dO, *args, stream=s))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    q = torch.zeros_like(Q)
    l3 = torch.empty_like(lse)
    with torch.cuda.graph(graph):
        o = sparge.sparge_window_fwd(q, K, V, *args, lse=l3)
        g = (o,) + sparge.sparge_window_bwd(q, K, V, o, l3, dO, *args)
    for _ in range(2):
        q.copy_(Q)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    assert sparge.device_status() == 0


def test_given_outputs_are_used(sparge):
    Q, K, V, dO = inputs(1, 2, 2, 200, 64, seed=8)
    O, lse = torch.empty_like(Q), torch.empty(1, 2, 200, device="cuda")
    assert sparge.sparge_window_fwd(Q, K, V, 10, 0, O=O, lse=lse) is O
    out = [torch.empty_like(t) for t in (Q, K, V)]
    got = sparge.sparge_window_bwd(Q, K, V, O, lse, dO, 10, 0, dQ=out[0], dK=out[1], dV=out[2])
    assert all(a is b for a, b in zip(got, out))


def test_outputs_at_any_16_bytes(sparge):
    """Outputs whose address is a multiple of 16 but not of 32 bytes."""
    Q, K, V, dO = inputs(1, 2, 1, 150, 128, seed=10)
    lse = torch.empty(1, 2, 150, device="cuda")
    O = sparge.sparge_window_fwd(Q, K, V, 30, 0, lse=lse)
    G = sparge.sparge_window_bwd(Q, K, V, O, lse, dO, 30, 0)
    odd = [torch.empty(t.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(t.shape) for t in (Q, Q, K, V)]
    sparge.sparge_window_fwd(Q, K, V, 30, 0, O=odd[0])
    sparge.sparge_window_bwd(Q, K, V, O, lse, dO, 30, 0, dQ=odd[1], dK=odd[2], dV=odd[3])
    for a, b in zip(odd, (O,) + G):
        assert a.data_ptr() % 32 == 16 and torch.equal(a, b)


def test_a_row_of_nan_stays_a_row(sparge):
    """A NaN in one query row gives that row NaN, in O and the log-sum-exp, and no other."""
    Q, K, V, _ = inputs(1, 1, 1, 300, 64, seed=12)
    lse, clean = torch.empty(1, 1, 300, device="cuda"), torch.empty(1, 1, 300, device="cuda")
    want = sparge.sparge_window_fwd(Q, K, V, -1, 0, lse=clean)
    Q[0, 0, 77, 5] = float("nan")
    O = sparge.sparge_window_fwd(Q, K, V, -1, 0, lse=lse)
    assert torch.isnan(O[0, 0, 77]).all() and torch.isnan(lse[0, 0, 77])
    keep = torch.arange(300, device="cuda") != 77
    assert torch.equal(O[0, 0, keep], want[0, 0, keep]) and torch.equal(lse[0, 0, keep], clean[0, 0, keep])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,win", [(1, (-1, 0, 0, 1)), (1, (0, 0, 1, 5)), (300, (0, 0, 0, 1)), (5, (0, 0, 0, 1))])
def test_rows_that_see_one_key_have_no_score_gradient(sparge, N, win, d):
    """Their probability is 1 whatever the score: O is the key's v, dQ and dK are exactly 0, dV sums dO."""
    Q, K, V, dO = inputs(2, 4, 2, N, d, seed=13)
    lse = torch.empty(2, 4, N, device="cuda")
    O = sparge.sparge_window_fwd(Q, K, V, *win[:2], sinks=win[2], unit=win[3], lse=lse)
    dQ, dK, dV = sparge.sparge_window_bwd(Q, K, V, O, lse, dO, *win[:2], sinks=win[2], unit=win[3])
    assert torch.equal(O, V.repeat_interleave(2, 1))
    assert not dQ.any() and not dK.any()
    want = dO.double().view(2, 2, 2, N, d).sum(2)
    assert ((dV.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -20 * dO.double().abs().amax()).all()


@pytest.mark.parametrize("win", [(1, 0, 0, 1), (3, 0, 4, 1), (0, 0, 0, 2), (30, 30, 0, 1)])
def test_gradients_of_rows_that_see_few_keys(sparge, win):
    """dS sums to 0 over a row's keys, and with few of them D's error does not average out: the relative error (2-norm)
    of dQ and dK stays at what rounding dS and the result leaves, 2^-9 each in the mean of a uniform last bit times
    sqrt(2): at most 2^-8 in all."""
    Q, K, V, dO = inputs(1, 4, 2, 1500, 128, seed=14)
    lse = torch.empty(1, 4, 1500, device="cuda")
    O = sparge.sparge_window_fwd(Q, K, V, *win[:2], sinks=win[2], unit=win[3], lse=lse)
    G = sparge.sparge_window_bwd(Q, K, V, O, lse, dO, *win[:2], sinks=win[2], unit=win[3])
    at = torch.arange(1500, device="cuda")
    seen = visible(at, at, 1500, *win)
    dK = torch.zeros(2, 1500, 128, dtype=torch.float64, device="cuda")
    for h in range(4):
        o, _, to, P, _ = rows_fwd(Q[0, h], K[0, h // 2], V[0, h // 2], seen)
        (dq, dk, _), _ = rows_bwd(Q[0, h], K[0, h // 2], V[0, h // 2], dO[0, h], P, o, to, seen)
        assert (G[0][0, h].double() - dq).norm() <= 2.0 ** -8 * dq.norm()
        dK[h // 2] += dk
    assert (G[1][0].double() - dK).norm() <= 2.0 ** -8 * dK.norm()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,unit,right", [(128, 1, 0), (77, 1, 0), (128 * 12, 128, 0), (100, 1, -1)])
def test_backward_of_single_key_tiles_repeats_itself(sparge, N, unit, right, d):
    """Row tiles with one key tile sum each row over both halves of its columns twice, with nothing but the row sums'
    own barriers in between: every one of many calls gives the same bits, which are the definition's gradients."""
    Q, K, V, dO = inputs(2, 40, 20, N, d, seed=15)
    win = (0 if unit > 1 else -1, right, 0, unit)
    O, lse, want = check(sparge, *(t[:1, :2 if t.shape[1] == 40 else 1].contiguous() for t in (Q, K, V, dO)), win)
    lse = torch.empty(2, 40, N, device="cuda")
    O = sparge.sparge_window_fwd(Q, K, V, *win[:2], unit=unit, lse=lse)
    runs = [sparge.sparge_window_bwd(Q, K, V, O, lse, dO, *win[:2], unit=unit) for _ in range(100)]
    torch.cuda.synchronize()
    assert sparge.device_status() == 0
    assert torch.equal(runs[0][0][:1, :2], want[0])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)
