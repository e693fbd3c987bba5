"""Attention in 64 bits with what its roundings can be expected to move it by,
and a check against that: much closer than a worst case at long contexts, where
rounding errors average out and a lost key does not.

Rounding errors are taken as independent and uniform within half a step:
  output          h(o), half a step of the type at |o|: variance h^2 / 3
  probabilities   rounded once (two query tiles): u^2 / 3 sum p^2 v^2 at most,
                  u half a step at 1; in two terms (single tokens): u^2 of that
  scores          off by e at most (d products summed in fp32): e^2 sum p^2 v^2
and errors common to a row (fp32 sums, ex2, cut-off MMA sums: c of itself).
Over the d dimensions of a row of 128 keys or more the mean square is within
2.5 times its expectation: six deviations, of 0.89 / sqrt d for uniform terms,
of sqrt(2 / d + 0.8 / keys that matter) for sums over keys.  Over all rows of a
call (8,192 outputs or more: deviations of 2% at most) it is within 1.21."""
from __future__ import annotations

import torch


def half_step(x, dtype):
    """Half a step of the type at |x| (of its smallest normal below that)."""
    fi = torch.finfo(dtype)
    return torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=fi.tiny)))) * fi.eps / 2


def expected(q, k, v, first, scale, dtype, rounded_p):
    """q [n, Hq, d] over k, v [m, Hkv, d] in fp64: row i sees keys j <= first + i
    (first None: all).  Returns out and, per element, the expected square of its
    error and the row's common error."""
    n, hq, d = q.shape
    m, hkv, _ = k.shape
    u = torch.finfo(dtype).eps / 2
    out, var = torch.zeros_like(q), torch.zeros_like(q)
    for h in range(hq):
        hk = h // (hq // hkv)
        z = q[:, h] @ k[:, hk].T * scale
        if first is not None:
            seen = torch.arange(m, device=q.device)[None, :] <= first + torch.arange(n, device=q.device)[:, None]
            z = torch.where(seen, z, float("-inf"))
        p = torch.softmax(z, -1)
        out[:, h] = p @ v[:, hk]
        e = d * 2.0 ** -24 * q[:, h].norm(dim=-1).max() * k[:, hk].norm(dim=-1).max() * scale
        rounding = (u if rounded_p else u * u) ** 2 / 3
        var[:, h] = (rounding + e * e) * ((p * p) @ (v[:, hk] * v[:, hk]))
    var += half_step(out, dtype) ** 2 / 3
    mma = (8 if rounded_p else 16) * min(m / 128, 256)
    common = (2.0 ** -22 + (128 + m / 128) * 2.0 ** -24 + mma * 2.0 ** -23) * out.abs()
    return out, var, common


def excess(got, out, var, common, keys):
    """(rows, all): the largest root mean square error of a row of 128 keys or
    more, and that of all of them, each over its limit (at most 1 is right).
    keys [n]: the keys that each row sees."""
    rows = keys >= 128
    err = ((got - out).abs() - common).clamp(min=0)[rows] ** 2
    row = (err.mean(-1) / (2.56 * var[rows].mean(-1))).max().sqrt()
    return float(row), float((err.mean() / (1.21 * var[rows].mean())).sqrt())
