"""Sampled rows of large paged batches, and bounds that count each rounding."""
from __future__ import annotations

import numpy as np
import torch

from oracle import relation_oracle as RO

import _paged as P


def gathered(cache, table_row, T, g):
    """Rows 0 .. T-1 of cached head g of a request, fp64; a page outside the cache is zeros."""
    n_pages, _, page, d = cache.shape
    pages = table_row[:-(-T // page)].to(cache.device).long()
    live = (pages >= 0) & (pages < n_pages)
    x = cache[pages.clamp(0, n_pages - 1), g]
    x = torch.where(live[:, None, None], x, torch.zeros_like(x))
    return P.f64(x).reshape(-1, d)[:T]


def rows_of(m, b, picks, heads, lam):
    """fp64 rows of the new tokens picks of request b at the query heads given: Y and sum_j F_ij (|V_j| + |Y_i|),
    [len(picks), len(heads), d]."""
    H, d = m["P1"].shape[1:]
    G = H // m["cP2"].shape[1]
    cu, T = m["cu"].cpu().numpy(), int(m["total"][b])
    q = int(cu[b + 1] - cu[b])
    Y, W = np.zeros((len(picks), len(heads), d)), np.zeros((len(picks), len(heads), d))
    for x, h in enumerate(heads):
        k, v = (gathered(m[c], m["table"][b], T, h // G) for c in ("cP2", "cV"))
        for y, i in enumerate(picks):
            p = T - q + i
            u = RO.evidence(P.f64(m["P1"][int(cu[b]) + i, h])[None], k[:p + 1])[0]
            logit = RO.silu(u) - lam * np.log(p + 1.0)
            logit[p] = RO.sigmoid(u[p:] / float(m["tau"][h]))[0]
            w = np.exp(logit - logit.max())
            w /= w.sum()
            Y[y, x] = w @ v[:p + 1]
            W[y, x] = w @ (np.abs(v[:p + 1]) + np.abs(Y[y, x]))
    return Y, W


def check_rows(m, Y, b, picks, heads, lam, lim):
    """Y (all packed rows) at those rows against rows_of; lim(ref, spread) bounds the difference."""
    ref, spread = rows_of(m, b, picks, heads, lam)
    at = [int(m["cu"][b]) + i for i in picks]
    err = np.abs(P.f64(Y[at][:, list(heads)]) - ref)
    top = lim(ref, spread)
    worst = np.unravel_index(np.argmax(err - top), err.shape)
    assert np.all(err <= top), (b, picks[worst[0]], heads[worst[1]], err[worst], top[worst], ref[worst])


def weights_bound(ref, spread, n, du, e_max):
    """|Y - Y*| of bf16 rows whose weights stay whole for the transport (two bf16 terms of each).

    Output: half a step, 2^-8 |Y*|. Weights: the first term leaves at most 2^-8 of a weight, exactly, and the second
    rounds that by 2^-8 of it: 2^-16. Numerator and row sum: n fp32 additions each, at most n 2^-24 relative. The
    exponent: an evidence off by du moves SiLU by at most 1.1 du, and E = SiLU(u) log2 e is formed with at most eight
    roundings of 2^-24, |E| <= e_max; the exponential itself and its sum with the others' 2^-22."""
    return (2.0**-16 + 2 * n * 2.0**-24 + 1.1 * du + 8 * e_max * 2.0**-24 + 2.0**-22) * spread + 2.0**-8 * np.abs(ref)


def evidence_error(P1, P2):
    """The most that fp32 sums of d bf16 products (exact in fp32) can be off, scaled by 1 / sqrt(d): d 2^-24 of the sum of
    their magnitudes, itself at most the product of the norms."""
    d = P1.shape[-1]
    top = float(np.sqrt((P.f64(P1)**2).sum(-1).max()) * np.sqrt(np.nanmax((P.f64(P2)**2).sum(-1))))
    return d * 2.0**-24 * top / np.sqrt(d), top / np.sqrt(d) * 1.4427
