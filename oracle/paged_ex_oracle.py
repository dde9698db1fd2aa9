"""Plain evaluation of the paged Relation Cache's 8-bit rows, trees of drafted tokens
and cut to the kept ones (fp64 and Python integers, from the definitions). Test
infrastructure; shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

from . import paged_oracle as PO
from . import relation_oracle as RO

LOW, HIGH = -100, 119


def scale_exponents(x):
    """The least k in [LOW, HIGH] with max |x| <= 448 * 2^k over the finite elements of each row (last axis)."""
    top = np.where(np.isfinite(x), np.abs(x), 0.0).max(-1)
    k = np.full(top.shape, LOW)
    for e in range(LOW, HIGH):
        k = np.where(top > 448.0 * 2.0**e, e + 1, k)
    return k


def e4m3_round(y):
    """The nearest e4m3 value of each element of y, |y| <= 448 (ties to the even significand); NaN stays."""
    a = np.abs(np.where(np.isnan(y), 0.0, y))
    step = 2.0**(np.floor(np.log2(np.maximum(a, 2.0**-6))) - 3)
    q = np.sign(y) * np.round(a / step) * step
    return np.where(np.isnan(y), np.nan, q)


def quantise(x):
    """(values, exponents) of rows x: value * 2^exponent stands for x."""
    k = scale_exponents(x)
    y = np.where(np.isfinite(x), np.clip(x / 2.0**k[..., None], -448.0, 448.0), np.nan)
    return e4m3_round(y), k


def ancestors(parent, k):
    """Places of the ancestors of a request's k'th token."""
    out, p = [], parent[k]
    at = k
    while 0 <= p < at:
        out.append(int(p))
        at, p = p, parent[p]
    return out


def valid(cu, total, b, N, rows):
    q = int(cu[b + 1]) - int(cu[b])
    return 0 <= cu[b] and q >= 0 and cu[b + 1] <= N and q <= total[b] <= rows


def tree_plan(parent, total, cu, words, tree0, pos0):
    """(tree, pos); rows and entries that are left alone come from tree0 and pos0."""
    N = len(parent)
    tree, pos = np.array(tree0, dtype=np.int64), np.array(pos0, dtype=np.int64)
    # Behind the last request; where that one ends past N, behind the last that does not.
    last = int(cu[-1])
    pos[max([0] + [int(c) for c in cu if c <= N]) if last > N else max(last, 0):] = -1
    for b in range(len(total)):
        f, q = int(cu[b]), int(cu[b + 1]) - int(cu[b])
        if not (0 <= f and q > 0 and f + q <= N):
            continue
        for k in range(q):
            if total[b] < q:
                pos[f + k] = -1
            elif q > 32 * words:
                pos[f + k] = total[b] - q + k
            else:
                up = ancestors(parent[f:f + q], k)
                pos[f + k] = total[b] - q + len(up)
                tree[f + k] = 0
                for a in up:
                    tree[f + k, a // 32] |= 1 << (a % 32)
    return np.where(tree >= 1 << 31, tree - (1 << 32), tree), pos


def seen(tree_row, k, words, q):
    """Places of the new tokens that token k of q sees."""
    if tree_row is None or q > 32 * words:
        return list(range(k))
    return [a for a in range(k) if (int(tree_row[a // 32]) >> (a % 32)) & 1]


def paged_fwd(P1, cP2, cV, table, total, cu, tau, lam, Y0, max_new, tree=None):
    """(Y, sum_j F_ij (|V_j| + |Y_i|)) fp64, with trees [N, words]; caches as the values that they stand for."""
    N, H, _ = P1.shape
    n_pages, Hkv, page, _ = cP2.shape
    words = 0 if tree is None else tree.shape[1]
    Y, W = np.array(Y0, dtype=np.float64), np.zeros(P1.shape)
    for b in range(len(total)):
        q, T = int(cu[b + 1]) - int(cu[b]), int(total[b])
        if not (0 < q <= max_new and valid(cu, total, b, N, table.shape[1] * page)):
            continue
        k, v = PO.gather(cP2, table[b], T, n_pages), PO.gather(cV, table[b], T, n_pages)
        for i in range(q):
            p, t = T - q + i, int(cu[b]) + i
            rows = list(range(T - q)) + [T - q + a for a in seen(None if tree is None else tree[t], i, words, q)] + [p]
            for h in range(H):
                g = h // (H // Hkv)
                u = RO.evidence(P1[t, h][None], k[g][rows])[0]
                logit = RO.silu(u) - lam * np.log(float(len(rows)))
                logit[-1] = RO.sigmoid(u[-1:] / float(tau[h]))[0]
                w = np.exp(logit - logit.max())
                w /= w.sum()
                Y[t, h] = w @ v[g][rows]
                W[t, h] = w @ (np.abs(v[g][rows]) + np.abs(Y[t, h]))
    return Y, W


def paged_keep(caches, table, total, cu, keep, n_keep, lens, free, n_free, page):
    """Moves rows of caches (arrays [n_pages, H_kv, page, ...], copied) and returns dict(caches, lens, free, n_free)."""
    caches = [c.copy() for c in caches]
    n_pages, rows = caches[0].shape[0], table.shape[1] * page
    lens, free = [int(x) for x in lens], [int(x) for x in free]
    have = min(max(int(n_free), 0), len(free))
    for b in range(len(total)):
        if not valid(cu, total, b, len(keep), rows):
            continue
        f, T = int(cu[b]), int(total[b])
        q = int(cu[b + 1]) - f
        n = int(n_keep[b])
        places = [int(x) for x in keep[f:f + n]] if 0 <= n <= q else []
        if any(not (y > x) for x, y in zip([-1] + places, places)) or any(x >= q for x in places):
            places = []
        n = len(places)
        at = [T - q + x for x in places]
        old = [[c[table[b, p // page], :, p % page].copy() if 0 <= table[b, p // page] < n_pages else
                np.zeros_like(c[0, :, 0]) for p in at] for c in caches]
        for k in range(n):
            p = T - q + k
            if at[k] != p and 0 <= table[b, p // page] < n_pages:
                for c, x in zip(caches, old):
                    c[table[b, p // page], :, p % page] = x[k]
        lens[b] = T - q + n
        for j in range(PO.ceil_div(lens[b], page), PO.ceil_div(T, page)):
            if have < len(free):
                free[have] = int(table[b, j])
                have += 1
    return dict(caches=caches, lens=lens, free=free, n_free=have)
