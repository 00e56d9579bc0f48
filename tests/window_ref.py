"""64-bit reference of windowed attention and of the e4m3 rows of a paged cache, and the tolerances that follow
from the roundings the kernels are documented to make.

A rounding to bf16 is off by at most eps = 2^-8 of the value. The kernels round P (and dS in the backward) to bf16
for their products and the results once; scores, exponentials and sums are in 32 bits, whose part is taken as
eps / 4 of the same sums of magnitudes. Hence, with A = sum_j P_ij |v_j|:

    |O - O64|   <= eps |O64| + (1 + 1/4) eps A                                     =: tO
    |dV - dV64| <= eps |dV64| + (1 + 1/4) eps sum_i P_ij |dO_i|
    D_i = dO_i . O_i takes the forward's O: off by at most |dO_i| . tO_i           =: tD_i
    |dQ - dQ64| <= eps |dQ64| + sum_j ((1 + 1/4) eps |dS_ij| + P_ij tD_i) |k_j| / sqrt(d)
    |dK - dK64| <= the same with sums over i and |q_i|

The log-sum-exp moves by no more than the scores do, whose sums of d products in 32 bits are off by at most
d 2^-24 of the sum of magnitudes each step (2^-23 for a sum that truncates); 1e-5 is added for exp and log.
"""
import math

import torch

EPS = 2.0 ** -8
SMALL = 1e-30  # both sides zero


def visible(i, j, L, left, right, sinks, unit):
    """[len(i), len(j)] from the rule's words."""
    fi, fj = i[:, None] // unit, j[None, :] // unit
    ahead = torch.ones((len(i), len(j)), dtype=torch.bool, device=i.device)
    near = ahead.clone()
    if right >= 0:
        ahead = fj <= fi + right
    if left >= 0:
        near = fj >= fi - left
    return ahead & (near | (j[None, :] < sinks)) & (j[None, :] < L) & (i[:, None] < L)


def rows_fwd(Q, K, V, seen):
    """One head's rows: O, lse, tO, P and the lse's tolerance. seen: [rows, keys]."""
    Q, K, V = Q.double(), K.double(), V.double()
    K, V = (torch.where(seen.any(0)[:, None], x, 0.0) for x in (K, V))
    Q = torch.where(seen.any(1)[:, None], Q, 0.0)
    scale = 1.0 / math.sqrt(Q.shape[1])
    S = torch.where(seen, Q @ K.T * scale, -math.inf)
    lse = torch.logsumexp(S, 1)
    P = torch.where(seen, torch.exp(S - lse[:, None]), 0.0)
    O = P @ V
    t = EPS * O.abs() + 1.25 * EPS * (P @ V.abs())
    tl = 1e-5 + Q.shape[1] * 2.0 ** -23 * scale * (Q.abs() @ K.abs().T).amax(1)
    return O, lse, t, P, tl


def rows_bwd(Q, K, V, dO, P, O, tO, seen):
    """One head's (dQ, dK, dV) and their tolerances before the rounding of the result, summed by the caller."""
    q, k, v, g = (x.double() for x in (Q, K, V, dO))
    k, v = (torch.where(seen.any(0)[:, None], x, 0.0) for x in (k, v))
    q, g = (torch.where(seen.any(1)[:, None], x, 0.0) for x in (q, g))
    scale = 1.0 / math.sqrt(q.shape[1])
    dS = P * (g @ v.T - (g * O).sum(1, keepdim=True))
    E = 1.25 * EPS * dS.abs() + P * (g.abs() * tO).sum(1, keepdim=True)
    return (dS @ k * scale, dS.T @ q * scale, P.T @ g), \
        (E @ k.abs() * scale, E.T @ q.abs() * scale, 1.25 * EPS * (P.T @ g.abs()))


def close(got, want, tol, what):
    got = got.double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), f"{what}: infinities or NaN differ"
    fine = torch.isfinite(want)
    bad = (got - want).abs()[fine] - tol[fine] - SMALL
    assert not fine.any() or bad.max() <= 0, f"{what}: off by {bad.max():.3g} more than allowed, at {int((bad > 0).sum())} places"
    g, w = got[~fine], want[~fine]
    assert torch.equal(g.isnan(), w.isnan()) and torch.equal(g[~g.isnan()], w[~w.isnan()]), f"{what}: other infinities"


def e4m3_rows(x):
    """(code values, exponent bytes) of bf16 rows, by frexp and by rounding in 64 bits; NaN rows get byte 255."""
    x = x.double()
    finite = torch.isfinite(x).all(-1)
    x = torch.where(finite[..., None], x, 0.0)
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(m == 0, -117, e).clamp(-117, 119)
    p = ((e.long() + 1023) << 52).view(torch.float64)[..., None]
    y = x / p
    step = ((torch.frexp(y.abs().clamp(min=2.0 ** -6))[1].long() - 4 + 1023) << 52).view(torch.float64)
    y = (torch.round(y / step) * step).clamp(-448, 448)
    value = torch.where(finite[..., None], y * p, math.nan)
    return value, torch.where(finite, e + 127, 255).to(torch.uint8)
