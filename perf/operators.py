"""Cases of the windowed and cached attention operators: what each computes in plain torch operations, the
framework's calls, and the definition in 64 bits.

The operators share one rule of visibility. Positions are counted in units of `unit` tokens (a video frame, or
1 for single tokens); row i sees key j < length when j's unit lies within `left` units before and `right` units
after i's own (-1: no limit), and the first `sinks` tokens as far as `right` lets it:

    lo_i = max(0, (i div unit - left) unit),  hi_i = min(length, (i div unit + right + 1) unit)
    visible(i) = [lo_i, hi_i)  and  [0, min(sinks, hi_i))

  fwd    forward over [B, H, N, d] with grouped K/V heads: O and the log-sum-exp of each row
  train  forward and backward of the same: O, dQ, dK, dV
  cache  new tokens' K and V written into a paged cache (bf16, or e4m3 with a power of two for each token and
         head), and a range of positions read back as bf16
  attn   a chunk of new tokens of each sequence (one token when decoding) attends to the paged cache

Lengths of ragged batches come from the case's own `ragged` number, so that the work of a case is known from
the case alone.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------------------------------------- the cases
def listed():
    return [
        # the smallest training shape: a few hundred tokens of two narrow heads, where the launch counts
        dict(name="fwd small d64", op="fwd", B=1, H=2, Hkv=2, N=300, d=64, left=63, right=0, sinks=4, unit=1, ragged=0),
        # a 480p clip (21 frames of 30 x 52 tokens), each frame sees itself, two frames back and the first frame
        dict(name="fwd 480p frames", op="fwd", B=1, H=12, Hkv=12, N=32760, d=128, left=2, right=0, sinks=1560, unit=1560,
             ragged=0),
        # a padded batch of clips of different lengths with grouped heads and a window in tokens
        dict(name="fwd grouped ragged", op="fwd", B=3, H=8, Hkv=2, N=5003, d=128, left=1023, right=0, sinks=64, unit=1,
             ragged=1),
        # a training step of attention on the 480p clip
        dict(name="train 480p frames", op="train", B=1, H=12, Hkv=12, N=32760, d=128, left=2, right=0, sinks=1560,
             unit=1560, ragged=0),
        # a training step with narrow grouped heads, an odd length and a window to both sides
        dict(name="train grouped d64", op="train", B=2, H=8, Hkv=2, N=2047, d=64, left=255, right=255, sinks=17, unit=1,
             ragged=2),
        # one decoding step's tokens into a bf16 cache, and a short tail read back: launch latency
        dict(name="cache step bf16", op="cache", B=16, Hkv=8, d=128, page=64, kind="bf16", new=1, past=300, back=16,
             ragged=3),
        # two 480p frames of each of four streams quantised into the cache, and the window read back
        dict(name="cache frames e4m3", op="cache", B=4, Hkv=12, d=128, page=64, kind="e4m3", new=2 * 1560, past=9361,
             back=4 * 1560, ragged=4),
        # one token of one stream over a short cache: the latency of a decoding step
        dict(name="attn one stream", op="attn", B=1, H=8, Hkv=2, d=128, page=16, kind="bf16", new=1, past=1023, left=-1,
             right=0, sinks=0, unit=1, ragged=0),
        # a large decoding batch over long ragged caches
        dict(name="attn decode bf16", op="attn", B=32, H=32, Hkv=8, d=128, page=64, kind="bf16", new=1, past=16383,
             left=-1, right=0, sinks=0, unit=1, ragged=5),
        # decoding over a quantised cache with a rolling window and sinks
        dict(name="attn decode e4m3", op="attn", B=24, H=16, Hkv=4, d=128, page=32, kind="e4m3", new=1, past=30000,
             left=16383, right=0, sinks=64, unit=1, ragged=6),
        # the next frame of a 480p clip over all the frames before it
        dict(name="attn frame bf16", op="attn", B=1, H=12, Hkv=12, d=128, page=128, kind="bf16", new=1560, past=20 * 1560,
             left=-1, right=0, sinks=0, unit=1560, ragged=0),
        # ragged chunks of prompts over a quantised cache with grouped heads, a window and sinks
        dict(name="attn chunks e4m3", op="attn", B=5, H=16, Hkv=4, d=128, page=64, kind="e4m3", new=701, past=9000,
             left=4095, right=0, sinks=64, unit=1, ragged=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("fwd", "train", "cache", "attn"))
    group = rng.choice((1, 1, 2, 3, 4, 8))
    d = rng.choice((64, 128, 128))
    ragged = rng.choice((0, rng.randint(1, 10**6)))
    if op in ("fwd", "train"):
        N = _log(rng, 1, 12000)
        unit = rng.choice((1, 1, _log(rng, 2, max(2, N // 3))))
        units = max(1, -(-N // unit))
        Hkv = rng.randint(1, max(1, min(8, 40000 // (N * group))))
        reach = max(1, min(units, 4096 // unit))
        return dict(op=op, B=rng.randint(1, 3), H=Hkv * group, Hkv=Hkv, N=N, d=d,
                    left=rng.choice((_log(rng, 1, reach), -1)) if N <= 4096 else _log(rng, 1, reach),
                    right=rng.choice((0, 0, _log(rng, 1, reach))) if N > 4096 else rng.choice((0, _log(rng, 1, reach), -1)),
                    sinks=rng.choice((0, _log(rng, 1, min(N, 2048)))), unit=unit, ragged=ragged)
    page = rng.choice((16, 32, 64, 128))
    kind = rng.choice(("bf16", "e4m3"))
    past = _log(rng, 1, 30000) - 1
    Hkv = rng.choice((1, 2, 3, 4, 8, 12)) if group <= 4 else rng.choice((1, 2, 4))
    if op == "cache":
        B = _log(rng, 1, max(1, min(32, 100000 // (past + 1))))
        new = _log(rng, 1, 4000)
        return dict(op=op, B=B, Hkv=Hkv, d=d, page=page, kind=kind, new=new, past=past, back=_log(rng, 1, past + new),
                    ragged=ragged)
    new = rng.choice((1, 1, rng.randint(2, 16), _log(rng, 17, 1600)))
    rows = new * Hkv * group
    B = _log(rng, 1, max(1, min(32, 500000 // (past + new), 1_000_000_000 // (rows * (past + new)))))
    unit = rng.choice((1, 1, _log(rng, 2, 2000)))
    return dict(op=op, B=B, H=Hkv * group, Hkv=Hkv, d=d, page=page, kind=kind, new=new, past=past,
                left=rng.choice((-1, _log(rng, 1, max(1, 8192 // unit)))), right=rng.choice((0, 0, -1)),
                sinks=rng.choice((0, _log(rng, 1, 256))), unit=unit, ragged=ragged)


def _lengths(case):
    """Per sequence: the clips' lengths (fwd, train), or new and past tokens (cache, attn)."""
    rng = random.Random(case["ragged"])
    if case["op"] in ("fwd", "train"):
        if not case["ragged"]:
            return [case["N"]] * case["B"]
        return [case["N"]] + [rng.randint(0, case["N"]) for _ in range(case["B"] - 1)]
    if not case["ragged"]:
        return [case["new"]] * case["B"], [case["past"]] * case["B"]
    if case["new"] == 1:
        new = [1] * case["B"]
    else:
        new = [case["new"]] + [rng.randint(0, case["new"]) for _ in range(case["B"] - 1)]
    return new, [case["past"]] + [rng.randint(case["past"] // 2, case["past"]) for _ in range(case["B"] - 1)]


def _range(i, length, case):
    """[lo, hi) of the rows at positions i, before the sinks."""
    u, left, right = case["unit"], case["left"], case["right"]
    f = torch.div(i, u, rounding_mode="floor")
    lo = torch.clamp((f - left) * u, min=0) if left >= 0 else torch.zeros_like(i)
    hi = torch.clamp((f + right + 1) * u, max=length) if right >= 0 else torch.full_like(i, length)
    return lo, hi


def _pairs(case, first, last, length):
    """(visible pairs, keys that some row sees) of the rows at positions first .. last - 1."""
    if last <= first:
        return 0, 0
    lo, hi = _range(torch.arange(first, last), length, case)
    more = torch.minimum(torch.minimum(hi, lo), torch.tensor(case["sinks"]))
    start, end = int(lo[0]), int(hi[-1])
    return int((hi - lo + more).sum()), end - start + min(start, case["sinks"])


def work(case):
    d, op = case["d"], case["op"]
    width = 2 if case.get("kind", "bf16") == "bf16" else 1
    row = d * width + (1 if width == 1 else 0)  # a token and head in the cache
    if op in ("fwd", "train"):
        B, H, Hkv, N = case["B"], case["H"], case["Hkv"], case["N"]
        pairs = sum(_pairs(case, 0, n, n)[0] for n in _lengths(case))
        q, kv = B * H * N * d * 2, B * Hkv * N * d * 2
        if op == "fwd":
            return {"bytes": 2 * q + 2 * kv + B * H * N * 4, "flops": 4.0 * pairs * H * d}
        return {"bytes": 4 * q + 4 * kv, "flops": 14.0 * pairs * H * d}
    new, past = _lengths(case)
    if op == "cache":
        n, back = sum(new), sum(min(case["back"], a + b) for a, b in zip(new, past))
        return {"bytes": 2.0 * case["Hkv"] * (n * (2 * d + row) + back * (2 * d + row)), "flops": 0.0}
    both = [_pairs(case, p, p + n, p + n) for n, p in zip(new, past)]
    return {"bytes": 4.0 * sum(new) * case["H"] * d + 2.0 * case["Hkv"] * row * sum(k for _, k in both),
            "flops": 4.0 * case["H"] * d * sum(p for p, _ in both)}


# ------------------------------------------------------------------------------------------------- the inputs
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _drift(g, positions, *shape):
    """What neighbouring tokens share: a slow wave of its own phase for each head and channel."""
    phase = torch.rand(shape, generator=g, device="cuda") * 6.2831853
    return 0.5 * torch.sin(positions * 0.002 + phase)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    d, op = case["d"], case["op"]
    s = dict(case)
    if op in ("fwd", "train"):
        B, H, Hkv, N = case["B"], case["H"], case["Hkv"], case["N"]
        at = torch.arange(N, device="cuda", dtype=torch.float32)[:, None]
        for name, heads in (("Q", H), ("K", Hkv)):
            s[name] = (_normal(g, B, heads, N, d) + _drift(g, at, B, heads, 1, d)).to(torch.bfloat16)
        s["V"] = _normal(g, B, Hkv, N, d).to(torch.bfloat16)
        if op == "train":
            s["dO"] = _normal(g, B, H, N, d).to(torch.bfloat16)
        s["lens"] = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda") if case["ragged"] else None
        return s
    new, past = _lengths(case)
    B, Hkv, page = case["B"], case["Hkv"], case["page"]
    total = [a + b for a, b in zip(new, past)]
    need = [-(-n // page) for n in total]
    most, pool = max(1, max(need)), sum(need) + 3
    pages = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
    first = torch.tensor([sum(need[:b]) for b in range(B)], device="cuda")[:, None]
    column = torch.arange(most, device="cuda")[None, :]
    used = column < torch.tensor(need, device="cuda")[:, None]
    s["table"] = torch.where(used, pages[torch.where(used, first + column, 0)], -1).to(torch.int32).contiguous()
    s["past_t"] = torch.tensor(past, dtype=torch.int32, device="cuda")
    s["cu_new"] = torch.tensor([sum(new[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["max_new"], s["max_len"] = max(new), max(1, max(total))
    shape = (pool, Hkv, page, d)
    for name in ("k", "v"):
        if case["kind"] == "bf16":
            s[name + "_pages"] = _normal(g, *shape).to(torch.bfloat16)
            s[name + "_exp"] = None
        else:  # a row's largest code lies in the top binades of the type, its power of two near 2^-7
            s[name + "_pages"] = (_normal(g, *shape) * 110).clamp(-448, 448).to(torch.float8_e4m3fn)
            s[name + "_exp"] = torch.randint(119, 122, shape[:3], generator=g, device="cuda", dtype=torch.uint8)
    T = sum(new)
    if op == "attn":
        s["Q"] = _normal(g, T, case["H"], d).to(torch.bfloat16)
        return s
    spread = torch.exp(_normal(g, T, Hkv, 1))  # the tokens' norms differ
    s["k_new"] = (_normal(g, T, Hkv, d) * spread).to(torch.bfloat16)
    s["v_new"] = _normal(g, T, Hkv, d).to(torch.bfloat16)
    back = [min(case["back"], n) for n in total]
    s["start"] = torch.tensor([n - b for n, b in zip(total, back)], dtype=torch.int32, device="cuda")
    s["cu_back"] = torch.tensor([sum(back[:b]) for b in range(B + 1)], dtype=torch.int32, device="cuda")
    s["n_back"] = sum(back)
    return s


# ------------------------------------------------------------------------------------------------- one pass
def run(s):
    op = s["op"]
    if own:
        from block_sparse_attention_pooled_b200 import sparge

        if op in ("fwd", "train"):
            lse = torch.empty(s["Q"].shape[:3], dtype=torch.float32, device=s["Q"].device)
            O = sparge.sparge_window_fwd(s["Q"], s["K"], s["V"], s["left"], s["right"], sinks=s["sinks"], unit=s["unit"],
                                         lens=s["lens"], lse=lse)
            if op == "fwd":
                return O, lse
            return (O,) + sparge.sparge_window_bwd(s["Q"], s["K"], s["V"], O, lse, s["dO"], s["left"], s["right"],
                                                   sinks=s["sinks"], unit=s["unit"], lens=s["lens"])
        if op == "cache":
            sparge.sparge_cache_write(s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["past_t"],
                                      s["cu_new"], k_exp=s["k_exp"], v_exp=s["v_exp"])
            return sparge.sparge_cache_read(s["k_pages"], s["v_pages"], s["table"], s["start"], s["cu_back"], s["n_back"],
                                            k_exp=s["k_exp"], v_exp=s["v_exp"])
        return sparge.sparge_cache_attn(s["Q"], s["k_pages"], s["v_pages"], s["table"], s["past_t"], s["cu_new"],
                                        s["max_new"], s["max_len"], s["left"], s["right"], sinks=s["sinks"],
                                        unit=s["unit"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    if op in ("fwd", "train"):
        return _plain_window(s)
    return _plain_cache(s) if op == "cache" else _plain_attn(s)


def _plain_window(s):
    """Rows in blocks; each block gathers the keys that any of its rows may see, the sinks first."""
    Q, K, V = s["Q"].float(), s["K"].float(), s["V"].float()
    B, H, N, d = Q.shape
    Hkv, G, u = K.shape[1], H // K.shape[1], s["unit"]
    reach = N if min(s["left"], s["right"]) < 0 else min(N, (s["left"] + s["right"] + 1) * u)
    c = max(1, min(N, max(128, reach // 4)))
    blocks, sinks = -(-N // c), min(s["sinks"], N)
    row = torch.arange(blocks * c, device=Q.device)
    lo, hi = _range(row, N, s)
    lo, hi = lo.view(blocks, c), hi.view(blocks, c)
    first, last = lo[:, 0], hi.amax(1)
    width = min(N, c + u + reach)  # at least as wide as any block's last - first, known without a look at the GPU
    col = torch.cat([torch.arange(sinks, device=Q.device).expand(blocks, sinks),
                     first[:, None] + torch.arange(width, device=Q.device)], 1)
    in_window = torch.arange(sinks + width, device=Q.device) >= sinks
    j = col[:, None, :]
    seen = torch.where(in_window, (j >= lo[..., None]) & (j < last[:, None, None]), j < lo[..., None]) & (j < hi[..., None])
    lens = s["lens"].long() if s["lens"] is not None else torch.full((B,), N, device=Q.device)
    seen = seen & (j < lens[:, None, None, None]) & (row.view(blocks, c, 1) < lens[:, None, None, None])
    seen = seen[:, None, :, None]  # [B, 1, blocks, 1, c, keys]
    col = col.clamp(max=N - 1)

    def rows(x):  # [B, H, N, d] -> [B, Hkv, blocks, G c, d]
        x = torch.cat([x, x.new_zeros(B, H, blocks * c - N, d)], 2)
        return x.view(B, Hkv, G, blocks, c, d).transpose(2, 3).reshape(B, Hkv, blocks, G * c, d)

    def back(x, w):
        return x.view(B, Hkv, blocks, G, c, w).transpose(2, 3).reshape(B, H, blocks * c, w)[:, :, :N]

    q, k, v = rows(Q), K[:, :, col], V[:, :, col]
    p = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, blocks, G, c, sinks + width)
    p.masked_fill_(~seen, -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    p.div_(torch.where(total == 0, 1.0, total))
    p = p.view(B, Hkv, blocks, G * c, sinks + width)
    o = p @ v
    if s["op"] == "fwd":
        return back(o, d).to(torch.bfloat16), back((top + total.log()).view(B, Hkv, blocks, G * c, 1), 1)[..., 0]
    g = rows(s["dO"].float())
    ds = g @ v.transpose(-1, -2)
    ds.sub_((g * o).sum(-1, keepdim=True)).mul_(p).mul_(1.0 / math.sqrt(d))
    flat = col.reshape(-1)
    dk, dv = torch.zeros_like(K), torch.zeros_like(V)
    dv.index_add_(2, flat, (p.transpose(-1, -2) @ torch.where(p.sum(-1, keepdim=True) > 0, g, 0.0)).flatten(2, 3))
    dk.index_add_(2, flat, (ds.transpose(-1, -2) @ q).flatten(2, 3))
    return tuple(x.to(torch.bfloat16) for x in (back(o, d), back(ds @ k, d), dk, dv))


def _tokens(cu, n):
    """Sequence and place within it of each of n packed tokens."""
    t = torch.arange(n, device=cu.device, dtype=torch.int32)
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return b, t - cu[b]


def _power(e):
    """2^e in 32 bits, from its bits: pow() on the GPU is an ulp off for some whole numbers."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _values(pages, exp, page, at):
    """The values that the cache holds at (page, place), in 32 bits: [..., Hkv, d]."""
    x = pages.view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn) if exp is not None else pages[page, :, at]
    return x.float() if exp is None else x.float() * _power(exp[page, :, at].int() - 127)[..., None]


def _plain_cache(s):
    b, t = _tokens(s["cu_new"], s["k_new"].shape[0])
    pos = (s["past_t"][b] + t).long()
    page, at = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    for new, pages, exp in ((s["k_new"], s["k_pages"], s["k_exp"]), (s["v_new"], s["v_pages"], s["v_exp"])):
        if exp is None:
            pages[page, :, at] = new
            continue
        x = new.float()
        m, e = torch.frexp(x.abs().amax(-1))  # a = m 2^e with m in [1/2, 1)
        e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-117, 119)
        e = torch.where(m == 0, -117, e)
        codes = (x * _power(-e)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        pages.view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
        exp[page, :, at] = (e + 127).to(torch.uint8)
    b, t = _tokens(s["cu_back"], s["n_back"])
    pos = (s["start"][b] + t).long()
    page, at = s["table"][b, pos // s["page"]].long(), pos % s["page"]
    return tuple(_values(p, e, page, at).to(torch.bfloat16) for p, e in
                 ((s["k_pages"], s["k_exp"]), (s["v_pages"], s["v_exp"])))


def _plain_attn(s):
    Q, cu, past = s["Q"].float(), s["cu_new"], s["past_t"].long()
    T, H, d = Q.shape
    B, Hkv, n, L = past.shape[0], s["Hkv"], s["max_new"], s["max_len"]
    G = H // Hkv
    new = (cu[1:] - cu[:-1]).long()
    length = past + new
    j = torch.arange(L, device=Q.device)
    page = s["table"][:, j // s["page"]].long().clamp(min=0)
    k = _values(s["k_pages"], s["k_exp"], page, j % s["page"])
    v = _values(s["v_pages"], s["v_exp"], page, j % s["page"])
    gone = (j >= length[:, None])[..., None, None]
    k, v = (x.masked_fill_(gone, 0.0).transpose(1, 2) for x in (k, v))  # [B, Hkv, L, d]
    t = torch.arange(n, device=Q.device)
    lo, hi = _range(past[:, None] + t, L, s)
    lo, hi = lo[..., None], torch.minimum(hi, length[:, None])[..., None]
    seen = (j < hi) & ((j >= lo) | (j < s["sinks"])) & (t < new[:, None])[..., None]  # [B, n, L]
    at = (cu[:-1].long()[:, None] + t).clamp(max=T - 1)
    q = Q[at].view(B, n, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    p = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, G, n, L)
    p.masked_fill_(~seen[:, None, None], -math.inf)
    top = p.amax(-1, keepdim=True)
    p.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * n, L) @ v).view(B, Hkv, G, n, d) / torch.where(total == 0, 1.0, total)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H, d)
    b, place = _tokens(cu, T)
    return o[b, place].to(torch.bfloat16)


# ------------------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """From the definition, a few rows at a time over the keys between the first and the last they see."""
    s = prepare(case, seed)
    w = work(case)
    if w["flops"] > 4e13:
        return None
    if case["op"] in ("fwd", "train"):
        return _exact_window(s)
    if case["op"] == "cache":
        return _exact_cache(s)
    table = s["table"].cpu()
    new, past = _lengths(case)
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, p) in enumerate(zip(new, past)):
        if not n:
            continue
        pages = table[b, : -(-(n + p) // case["page"])].long().cuda()
        K, V = (_dense(s[x + "_pages"], s[x + "_exp"], pages)[:, : n + p] for x in ("k", "v"))
        out[at : at + n] = _softmax_rows(s["Q"][at : at + n].transpose(0, 1), K, V, p, s)[0].transpose(0, 1)
        at += n
    return out


def _power64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _dense(pages, exp, which):
    """[Hkv, tokens, d] in 64 bits of the pages listed."""
    x = pages[which] if exp is None else pages.view(torch.uint8)[which].view(torch.float8_e4m3fn)
    x = x.float().double()
    if exp is not None:
        x = x * _power64(exp[which].long() - 127)[..., None]
    return x.transpose(0, 1).flatten(1, 2)


def _seen(i, j, length, s):
    """Whether the row at position i sees key j, from the rule's words."""
    fi, fj = i[:, None] // s["unit"], j[None, :] // s["unit"]
    near = torch.ones_like(fi - fj, dtype=torch.bool)
    ahead = near.clone()
    if s["left"] >= 0:
        near = fj >= fi - s["left"]
    if s["right"] >= 0:
        ahead = fj <= fi + s["right"]
    return ahead & (near | (j[None, :] < s["sinks"])) & (j[None, :] < length)


def _softmax_rows(Q, K, V, past, s, step=1024):
    """O [H, n, d] and the log-sum-exp [H, n] of rows at positions past.. over K, V [Hkv, length, d]."""
    H, n, d = Q.shape
    G, length = H // K.shape[0], K.shape[1]
    O = torch.zeros(H, n, d, dtype=torch.float64, device="cuda")
    lse = torch.full((H, n), -math.inf, dtype=torch.float64, device="cuda")
    for r in range(0, n, step):
        i = torch.arange(r, min(n, r + step), device="cuda") + past
        seen = _seen(i, torch.arange(length, device="cuda"), length, s)
        cols = seen.any(0).nonzero()[:, 0]
        if not cols.numel():
            continue
        seen = seen[:, cols]
        for h in range(H):
            S = Q[h, r : r + step].double() @ K[h // G][cols].double().T / math.sqrt(d)
            S = torch.where(seen, S, -math.inf)
            lse[h, r : r + step] = torch.logsumexp(S, 1)
            O[h, r : r + step] = torch.nan_to_num(torch.softmax(S, 1)) @ V[h // G][cols].double()
    return O, lse


def _exact_window(s):
    Q, K, V = s["Q"], s["K"], s["V"]
    B, H, N, d = Q.shape
    G = H // K.shape[1]
    O = torch.zeros(Q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(Q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    dQ, dK, dV = (torch.zeros(x.shape, dtype=torch.float64, device="cuda") for x in (Q, K, V))
    for b, n in enumerate(_lengths(s)):
        if not n:
            continue
        O[b, :, :n], lse[b, :, :n] = _softmax_rows(Q[b, :, :n], K[b, :, :n], V[b, :, :n], 0, s)
        if s["op"] == "fwd":
            continue
        for r in range(0, n, 1024):
            end = min(n, r + 1024)
            seen = _seen(torch.arange(r, end, device="cuda"), torch.arange(n, device="cuda"), n, s)
            cols = seen.any(0).nonzero()[:, 0]
            seen = seen[:, cols]
            for h in range(H):
                q, g = Q[b, h, r:end].double(), s["dO"][b, h, r:end].double()
                k, v = K[b, h // G][cols].double(), V[b, h // G][cols].double()
                P = torch.softmax(torch.where(seen, q @ k.T / math.sqrt(d), -math.inf), 1)
                dP = g @ v.T
                dS = P * (dP - (P * dP).sum(1, keepdim=True)) / math.sqrt(d)
                dQ[b, h, r:end] = dS @ k
                dK[b, h // G].index_add_(0, cols, dS.T @ q)
                dV[b, h // G].index_add_(0, cols, P.T @ g)
    return (O, lse) if s["op"] == "fwd" else (O, dQ, dK, dV)


def _exact_cache(s):
    """Each position read back holds the new token's rounded value, or what the cache held there before."""
    new, past = _lengths(s)
    table, start, cu = s["table"].cpu(), s["start"].tolist(), s["cu_new"].tolist()
    both = []
    for x in ("k", "v"):
        fresh = s[x + "_new"].double()
        if s[x + "_exp"] is not None:
            m, e = torch.frexp(fresh.abs().amax(-1, keepdim=True) / 448.0)
            e = torch.where(m > 0.5, e, e - 1).clamp(-117, 119)  # the least e with 448 2^e at or over the largest value
            y = fresh / _power64(e)
            step = _power64(torch.frexp(y.abs().clamp(min=2.0**-6))[1] - 4)  # of the binade that y lies in
            fresh = torch.round(y / step) * step * _power64(e)
        rows = []
        for b, (n, p) in enumerate(zip(new, past)):
            pages = table[b, : -(-(n + p) // s["page"])].long().cuda()
            old = _dense(s[x + "_pages"], s[x + "_exp"], pages).transpose(0, 1)[: n + p].clone()
            old[p:] = fresh[cu[b] : cu[b + 1]]
            rows.append(old[start[b] :])
        both.append(torch.cat(rows))
    return tuple(both)
