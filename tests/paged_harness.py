"""Set-up and bounds shared by the GPU tests of the paged cache and of cross
attention."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged_oracle as PO

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def f64(t):
    return t.double().cpu().numpy()


def randn(seed, shape, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def score_error(d, q_norm, k_norm, scale):
    """Bound on a score's error: its d products summed in fp32 (a half step of
    each of d partial sums, none above |q| |k|)."""
    return d * 2.0 ** -24 * q_norm * k_norm * scale


def check(got, lse, want, want_lse, mass, dtype, q_norm, k_norm, scale, d, n_key, what=""):
    """Output and lse against the oracle.

    u = half a step of the type.  The output is rounded once (u |o|), the
    probabilities at most once (each by u of itself, so u sum p|v|), and a score that
    is off by e moves its probability by e of itself and the sum by as much
    (2 e sum p|v|); e adds the error of ex2 (2^-22) and of the fp32 row sum
    ((128 + n / 128) 2^-24).  Values under the type's smallest normal have an
    absolute step instead.  lse has no rounded probability in it: e, and
    fp32 steps of its own size.
    """
    live = ~np.isnan(want)
    u = torch.finfo(dtype).eps / 2
    e = score_error(d, q_norm, k_norm, scale) + 2.0 ** -22 + (128 + n_key / 128) * 2.0 ** -24
    tol = u * (np.abs(want) * (1 + u) + mass) + 2 * e * mass + 2.0 ** -24
    err = np.abs(got - want)
    assert np.isfinite(got[live]).all(), what
    worst = float((err / tol)[live].max()) if live.any() else 0.0
    assert worst <= 1.0, "%s: %.3g times the bound, error %.3g" % (what, worst, np.nanmax(err))
    if lse is not None:
        ok = np.isfinite(want_lse)
        assert np.array_equal(lse[np.isneginf(want_lse)], want_lse[np.isneginf(want_lse)]), what
        err = np.abs(lse[ok] - want_lse[ok])
        ltol = e + 2.0 ** -22 * (1 + np.abs(want_lse[ok]))
        assert (err <= ltol).all(), "%s: lse off by %.3g" % (what, err.max())
    return worst


class Pages:
    """A pool with the requests' keys and values on shuffled pages; what lies
    past a request's length and on unused pages is NaN."""

    def __init__(self, seed, kv_len, page, hkv, d, dtype, extra_cols=2, fill=float("nan")):
        rng = np.random.default_rng(seed)
        used = [-(-int(n) // page) for n in kv_len]
        self.n_page = sum(used) + 3
        self.page, self.hkv, self.d = page, hkv, d
        cols = max(used + [1]) + extra_cols
        ids = rng.permutation(self.n_page)[:sum(used)]
        self.table = np.full((len(kv_len), cols), -7, dtype=np.int32)
        self.k = torch.full((self.n_page, hkv, page, d), fill, dtype=dtype)
        self.v = self.k.clone()
        g = torch.Generator().manual_seed(seed)
        at = 0
        for b, n in enumerate(kv_len):
            for j in range(used[b]):
                p, rows = int(ids[at]), min(page, int(n) - j * page)
                at += 1
                self.table[b, j] = p
                for pool in (self.k, self.v):
                    pool[p, :, :rows] = torch.randn((hkv, rows, d), generator=g).to(dtype)
        self.k, self.v = self.k.cuda(), self.v.cuda()

    def cache(self, skv, **kw):
        return skv.PagedCache.wrap(k=self.k, v=self.v, block_table=torch.from_numpy(self.table).cuda(), **kw)


def run_paged(skv, seed, q_len, kv_len, page, hq, hkv, d, dtype, scale=None, q_mul=1.0, what="", ws=None):
    """paged_attn against the oracle on shuffled pages; returns (out, lse)."""
    scale = d ** -0.5 if scale is None else scale
    pg = Pages(seed, kv_len, page, hkv, d, dtype)
    cache = pg.cache(skv)
    qs = starts(q_len)
    q = (randn(seed + 1, (int(qs[-1]), hq, d), dtype).float() * q_mul).to(dtype)
    out, lse = skv.paged_attn(cache, q, ints(qs), ints(kv_len), scale, lse=True, ws=ws)
    want, wlse, mass = PO.paged(f64(q), f64(pg.k), f64(pg.v), pg.table, qs, kv_len, scale)
    assert cache.device_status() == 0, what
    k = pg.k.float()
    k_norm = float(torch.where(torch.isnan(k), 0.0, k).norm(dim=-1).max())
    q_norm = float(q.float().norm(dim=-1).max()) if q.numel() else 0.0
    check(f64(out), f64(lse), want, wlse, mass, dtype, q_norm, k_norm, scale, d, max(kv_len), what)
    return out, lse
