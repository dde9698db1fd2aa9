"""Inputs of the tests of 8-bit pages and trees of drafted tokens."""
from __future__ import annotations

import numpy as np
import torch

from oracle import paged_ex_oracle as XO

import _paged as P


def random_parents(nn, rng, reach=5, roots=0.1):
    """A tree over each request's new tokens: some roots, the others under one of the `reach` before them."""
    out = []
    for n in nn:
        out += [-1 if k == 0 or rng.random() < roots else int(rng.integers(max(0, k - reach), k)) for k in range(n)]
    return np.array(out, dtype=np.int32)


def bits_of(parent, cu, total, words, N, junk=None):
    """Ancestor bits [N, words] int32. junk: a generator that sets the bits at and past each token's own place."""
    tree, _ = XO.tree_plan(parent, total, cu, words, np.zeros((N, words)), np.zeros(N))
    tree = tree & 0xffffffff
    if junk is not None:
        for b in range(len(total)):
            for k in range(int(cu[b + 1]) - int(cu[b])):
                for a in range(k, 32 * words):
                    if junk.random() < 0.5:
                        tree[int(cu[b]) + k, a // 32] |= 1 << (a % 32)
    return np.where(tree >= 1 << 31, tree - (1 << 32), tree).astype(np.int32)


def as_8bit(m, rng=None, spread=0):
    """m of _paged.make (bf16) with its caches quantised: float8 caches, scales, and the values they stand for as
    fp64 arrays (k64, v64). spread: V rows times powers of two of up to that many steps, P2 rows of up to two."""
    out = dict(m)
    n_pages, Hkv, page, d = m["cP2"].shape
    scale = np.zeros((n_pages, Hkv, 2, page), dtype=np.uint8)
    for part, name in ((0, "cP2"), (1, "cV")):
        x = P.f64(m[name])
        if spread:
            x = x * 2.0**rng.integers(-min(spread, 2) if part == 0 else -spread, (2 if part == 0 else spread) + 1, x.shape[:3])[..., None]
        q, k = XO.quantise(x)
        hole = np.isnan(x).all(-1)                       # rows that no request holds: NaN, and bytes that are no scale
        scale[:, :, part] = np.where(hole, 255, k + 127)
        out[name] = torch.from_numpy(q).to(torch.float32).to(torch.float8_e4m3fn)
        out["k64" if part == 0 else "v64"] = np.where(hole[..., None], 0.0, q * 2.0**k[..., None])
    out["scale"] = torch.from_numpy(scale).view(torch.float8_e8m0fnu)
    return out


def to_device(m, dev="cuda"):
    out = P.to_device(m, dev)
    for k in ("scale", "tree"):
        if m.get(k) is not None:
            out[k] = m[k].to(dev)
    return out
