"""Attention over an e4m3 cache whose rows have powers far apart, against the 64-bit definition: through the kernel for
up to 16 rows a sequence (4 heads, 1 and 4 new tokens) and the one for more (20 new tokens)."""
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


def normal(seed, *shape):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda")


def cache_of(sparge, k, v, page=64):
    """k, v [n, d] as the cache of one sequence with one K/V head."""
    n, d = k.shape
    pages = -(-n // page)
    kp, vp = (torch.full((pages, 1, page, d), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    exp = {x: torch.full((pages, 1, page), 255, dtype=torch.uint8, device="cuda") for x in ("k_exp", "v_exp")}
    table = torch.arange(pages, dtype=torch.int32, device="cuda").flip(0)[None].contiguous()
    bf = [x.to(torch.bfloat16)[:, None].contiguous() for x in (k, v)]
    sparge.sparge_cache_write(*bf, kp, vp, table, ints(0), ints(0, n), **exp)
    return (kp, vp, table), exp, [e4m3_rows(x)[0][:, 0] for x in bf]


def attend(sparge, Q, cache, exp, n, win=(-1, 0, 0, 1)):
    new, lse = Q.shape[0], torch.empty(Q.shape[:2], device="cuda")
    O = sparge.sparge_cache_attn(Q, *cache, ints(n - new), ints(0, new), new, n, *win[:2], sinks=win[2], unit=win[3],
                                 lse=lse, **exp)
    torch.cuda.synchronize()
    assert sparge.device_status() == 0
    return O, lse


def compare(O, lse, Q, k64, v64, win=(-1, 0, 0, 1), floor=None):
    """floor: [rows, d] for each head, what a probability's rounding may add (none where probabilities are bf16)."""
    n, new = k64.shape[0], Q.shape[0]
    at = torch.arange(n, device="cuda")
    seen = visible(at[-new:], at, n, *win)
    for h in range(Q.shape[1]):
        o, ls, to, P, tl = rows_fwd(Q[:, h], k64, v64, seen)
        close(lse[:, h], ls, tl, f"lse, head {h}")
        close(O[:, h], o, to if floor is None else to + floor(P), f"O, head {h}")


def check(sparge, k, v, Q, win=(-1, 0, 0, 1), page=64):
    cache, exp, (k64, v64) = cache_of(sparge, k, v, page)
    O, lse = attend(sparge, Q, cache, exp, k.shape[0], win)
    compare(O, lse, Q, k64, v64, win)
    return O, lse


def one_against_many(many, below, d, new, seed):
    """The first key scores 0 and the others `below` (log2) less, for 4 heads; the last `new` tokens are among them."""
    k = torch.zeros(many + 1, d, device="cuda")
    k[1:, 0] = -8.0
    Q = torch.zeros(new, 4, d, device="cuda")
    Q[..., 0] = below / 8.0 * math.sqrt(d) / math.log2(math.e)
    return k, Q.to(torch.bfloat16), normal(seed, many + 1, d)


NEW = pytest.mark.parametrize("new", [1, 4, 20])


@NEW
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top,many,below", [(100.0, 4096, 12), (3.0, 4096, 17), (2.0 ** 20, 40, 0), (2.0 ** 90, 40, 0)])
def test_keys_whose_value_is_zero_count(sparge, top, many, below, d, new):
    """One key with a value of `top` among many whose value is 0: they only dilute it."""
    k, Q, v = one_against_many(many, below, d, new, 1)
    v = v.clamp(-1, 1) * top
    v[1:] = 0
    check(sparge, k, v, Q)


@NEW
@pytest.mark.parametrize("zeros", [2048, 30000])
def test_long_runs_of_zero_rows(sparge, zeros, new):
    """Keys and values of 0 (a stretch that was never written but is seen), then ordinary rows; then nothing else."""
    n = zeros + 5000
    k, v = normal(2, n, 128), normal(3, n, 128)
    k[:zeros] = 0
    v[:zeros] = 0
    Q = normal(4, new, 4, 128).to(torch.bfloat16)
    check(sparge, k, v, Q)
    O, _ = check(sparge, k[:zeros].contiguous(), v[:zeros].contiguous(), Q)
    assert not O.any()


@NEW
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("win", [(-1, 0, 0, 1), (700, 0, 30, 1)])
def test_rows_of_different_powers(sparge, win, d, new):
    """Magnitudes of K and V that differ from row to row by up to 2^12, some rows 0, scores of some dozens."""
    n = 1500
    k, v = normal(5, n, d), normal(6, n, d)
    k *= torch.exp2(normal(7, n, 1).clamp(-3, 3))
    v *= torch.exp2(2 * normal(8, n, 1).clamp(-3, 3))
    v[::7] = 0
    k[::5] = 0
    check(sparge, k, v, normal(9, new, 4, d).to(torch.bfloat16) * 2, win, page=16)


def fp16_floor(code, power):
    """What probabilities in fp16 may add. A P_j 2^e_j enters as a multiple of its row's largest, W, which stands at
    2^15: half a step of fp16 below 2^-14 is 2^-25, that is 2^-40 W, for each key's code."""
    def floor(P):
        W = (P * power[None]).amax(1)
        return 2.0 ** -40 * W[:, None] * ((P > 0).double() @ code.abs())
    return floor


def check_with_floor(sparge, k, v, Q):
    cache, exp, (k64, v64) = cache_of(sparge, k, v)
    byte = e4m3_rows(v.to(torch.bfloat16))[1]
    power = torch.exp2(byte.double() - 127)
    O, lse = attend(sparge, Q, cache, exp, k.shape[0])
    compare(O, lse, Q, k64, v64, floor=fp16_floor(v64 / power[:, None], power))


@pytest.mark.parametrize("new", [1, 4])
@pytest.mark.parametrize("below", [17.3, 21.7, 26])
@pytest.mark.parametrize("many", [63, 6000])  # all with the best key in one warp's hands; most of them elsewhere
@pytest.mark.parametrize("d", [64, 128])
def test_channels_that_the_best_key_leaves_empty(sparge, d, many, below, new):
    """The best key holds 0 in half of its channels: there O comes from the many keys `below` binades down, each
    kept to fp16's 11 bits, as they are with more rows (bf16's 8 bits). The tolerance has no part for lost keys."""
    k, Q, v = one_against_many(many, below, d, 20, 10)
    v = v.abs().clamp(0.25, 3)
    v[0, ::2] = 0
    v[0, 1::2] = 3.0
    few, _ = check(sparge, k, v, Q[-new:].contiguous())
    many, _ = check(sparge, k, v, Q)
    assert ((few.double() - many[-new:].double()).abs() <= 2.5 * 2.0 ** -8 * few.double().abs()).all()


@pytest.mark.parametrize("new", [1, 4, 20])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_powers_dozens_apart(sparge, d, new):
    """V's rows between 2^-40 and 2^40 (some rows 0), scores of some dozens, K's rows 2^6 apart."""
    n = 1500
    k, v = normal(11, n, d), normal(12, n, d)
    k *= torch.exp2(normal(13, n, 1).clamp(-3, 3))
    v *= torch.exp2(20 * normal(14, n, 1).clamp(-2, 2))
    v[::9] = 0
    check_with_floor(sparge, k, v, normal(15, new, 4, d).to(torch.bfloat16))


@NEW
@pytest.mark.parametrize("power", [10, 20, 27])
def test_equal_scores_however_large(sparge, power, new):
    """Scores of 8 * 2^power for three keys (exact in 32 bits) and of the opposite sign for the others: O is the mean of
    the three's values."""
    n, d = 300, 64
    k, v = torch.zeros(n, d, device="cuda"), normal(18, n, d)
    k[:, 0] = -8.0
    k[[3, 70, 200], 0] = 8.0
    Q = torch.zeros(new, 4, d, device="cuda")
    Q[..., 0] = 2.0 ** power
    check(sparge, k, v, Q.to(torch.bfloat16))


@NEW
@pytest.mark.parametrize("power", [-124, -110, -90, 90, 110, 116])
def test_queries_of_any_magnitude(sparge, power, new):
    """Q around 2^power and K around 2^-power: scores as of ordinary ones, down to rows of Q that are almost subnormal."""
    n, d = 300, 128
    k, v = normal(19, n, d).clamp(-3, 3), normal(20, n, d)
    Q = normal(21, new, 4, d)
    Q = torch.where(Q.abs() < 0.25, 0.25, Q) * 2.0 ** power
    check(sparge, k * 2.0 ** -power, v, Q.to(torch.bfloat16))


@NEW
def test_large_scores_of_large_queries(sparge, new):
    """Scores of some 2^12 from a Q of 2^126 and keys near the least power: no product on the way overflows."""
    n, d = 300, 64
    k, v = torch.zeros(n, d, device="cuda"), normal(22, n, d)
    k[:, 0] = -(2.0 ** -111)
    k[[3, 70, 200], 0] = 2.0 ** -111
    Q = torch.zeros(new, 4, d, device="cuda")
    Q[..., 0] = 2.0 ** 126
    check(sparge, k, v, Q.to(torch.bfloat16))


@pytest.mark.parametrize("new", [1, 4, 20])
@pytest.mark.parametrize("byte", [0, 1, 9, 247, 254])
def test_bytes_that_the_writer_does_not_store(sparge, byte, new):
    """Every byte but 255 is the power byte - 127, in reading and in attention, as far as bf16 holds the values: in K
    (with a Q of the opposite magnitude) and in V, where the sums before the division by the row's have to fit 32 bits
    (150 keys of 2^120 do, of 2^127 do not)."""
    n, d, page = 150, 64, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(16)
    pages = -(-n // page)
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None].contiguous()
    # codes between 1/2 and 15/8: their values are exact in bf16 at every power, subnormal ones included
    codes = [(torch.randint(0x30, 0x40, (pages, 1, page, d), generator=g, device="cuda", dtype=torch.uint8)
              | torch.randint(0, 2, (pages, 1, page, d), generator=g, device="cuda", dtype=torch.uint8) << 7)
             .view(torch.float8_e4m3fn) for _ in range(2)]
    for which in (0, 1):
        exp = [torch.full((pages, 1, page), b, dtype=torch.uint8, device="cuda") for b in ((byte, 127) if which == 0 else (127, byte))]
        kv = [(c.float().double() * torch.exp2(e.double() - 127)[..., None]).transpose(1, 2).flatten(0, 1)[:n, 0]
              for c, e in zip(codes, exp)]
        both = {"k_exp": exp[0], "v_exp": exp[1]}
        got = sparge.sparge_cache_read(*codes, table, ints(0), ints(0, n), n, **both)
        for x, want in zip(got, kv):
            assert torch.equal(x[:, 0].double(), want)
        if byte == 254 and which == 1:
            continue
        Q = (normal(17, new, 4, d) * 2.0 ** (max(-120, min(120, 127 - byte)) if which == 0 else 0)).to(torch.bfloat16)
        O, lse = attend(sparge, Q, (*codes, table), both, n)
        compare(O, lse, Q, *kv)


@pytest.mark.parametrize("new", [1, 4, 20, 90])
@pytest.mark.parametrize("where", ["v", "k"])
@pytest.mark.parametrize("d", [64, 128])
def test_rows_of_nan_reach_only_those_who_see_them(sparge, d, where, new):
    """Rows with an infinity among the new tokens and just outside a window: O is NaN for the rows that see one, in V or
    K, and as if it were not there for the others of its tile; V does not reach the log-sum-exp."""
    n = 700
    k, v, Q = normal(23, n, d), normal(24, n, d), normal(25, new, 4, d).to(torch.bfloat16)
    first = n - new
    bad = [first - 41, 5] + ([first + new // 2] if new > 1 else [])
    x = v if where == "v" else k
    x[bad, 7] = math.inf
    clean = k.clone(), v.clone()
    clean[0 if where == "k" else 1][bad] = 0
    cache, exp, _ = cache_of(sparge, k, v, 16)
    at = torch.arange(n, device="cuda")
    for win in ((40, 0, 0, 1), (40, 0, 10, 1), (-1, 0, 0, 1)):
        O, lse = attend(sparge, Q, cache, exp, n, win)
        seen = visible(at[-new:], at, n, *win)
        hit = seen[:, bad].any(1)
        k64, v64 = (e4m3_rows(t.to(torch.bfloat16))[0] for t in clean)
        for h in range(4):
            assert torch.isnan(O[hit, h]).all()
            o, ls, to, _, tl = rows_fwd(Q[:, h], k64, v64, seen)
            close(O[~hit, h], o[~hit], to[~hit], f"O, window {win}")
            keep = ~hit if where == "k" else torch.ones_like(hit)
            close(lse[keep, h], ls[keep], tl[keep], f"lse, window {win}")
            assert torch.isnan(lse[~keep, h]).all()


def test_nan_rows_in_a_long_split_cache(sparge):
    """The same where many CTAs share an item: the partial that holds the row makes O NaN, the log-sum-exp stays."""
    n, d = 40000, 128
    k, v = normal(26, n, d), normal(27, n, d)
    v[31000, 0] = -math.inf
    clean = v.clone()
    clean[31000] = 0
    cache, exp, (k64, _) = cache_of(sparge, k, v)
    v64 = e4m3_rows(clean.to(torch.bfloat16))[0]
    for new in (1, 20, 200):
        Q = normal(28, new, 4, d).to(torch.bfloat16)
        O, lse = attend(sparge, Q, cache, exp, n)
        assert torch.isnan(O).all()
        at = torch.arange(n, device="cuda")
        seen = visible(at[-new:], at, n, -1, 0, 0, 1)
        for h in range(4):
            _, ls, _, _, tl = rows_fwd(Q[:, h], k64, v64, seen)
            close(lse[:, h], ls, tl, "lse")


@pytest.mark.parametrize("new", [1, 4, 20])
@pytest.mark.parametrize("power", [3, 12, 20, 22, 23, 24])
def test_equal_large_scores_of_rows_of_different_powers(sparge, power, new):
    """Scores of 2^power for some keys (exact in 32 bits), of the opposite sign for the others, and V's powers from row to
    row: sums of score and power are rounded, the mean over the best keys stays."""
    n, d = 600, 64
    for seed in range(4):
        k, v = torch.zeros(n, d, device="cuda"), normal(30 + seed, n, d)
        v *= torch.exp2(torch.randint(-9, 10, (n, 1), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        k[:, 0] = -8.0
        k[::37, 0] = 8.0
        Q = torch.zeros(new, 4, d, device="cuda")
        Q[..., 0] = 2.0 ** power * torch.tensor([1.0, 1.25, 1.5, 1.75], device="cuda")
        check(sparge, k, v, Q.to(torch.bfloat16))
