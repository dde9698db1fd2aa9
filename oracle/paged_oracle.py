"""Plain evaluation of the paged Relation Cache: the page map in Python
integers, and the forward of packed tokens as rows of the Relation forward on
each request's gathered rows (fp64, from the definition). Test infrastructure;
shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

from . import relation_oracle as RO

INT_MAX = 2**31 - 1


def ceil_div(a, b):
    return -(-a // b)


def page_map(lens, n_new, table, free, n_free, N, page, n_pages):
    """One request at a time; returns dict(cu, total, slot, pos, n_free, table, free)."""
    lens, n_new = [int(x) for x in lens], [int(x) for x in n_new]
    table, free = np.array(table, dtype=np.int64), [int(x) for x in free]
    S, width = table.shape
    F = len(free)
    have = min(max(int(n_free), 0), F)
    total = [-1] * S
    # Finished requests return their pages; what does not fit the list is dropped.
    for b in range(S):
        if n_new[b] == -1 and 0 <= lens[b] <= width * page:
            total[b] = 0
            for k in range(ceil_div(lens[b], page)):
                if have < F:
                    free[have] = int(table[b, k])
                    have += 1
    cu, wanted, spent = [0], 0, 0
    slot, pos = [-1] * N, [-1] * N
    top = have
    for b in range(S):
        q = max(n_new[b], 0)
        first = cu[-1]
        cu.append(first + q)
        if n_new[b] < 0 or lens[b] < 0 or lens[b] + q > width * page or cu[-1] > N:
            continue
        held = ceil_div(lens[b], page)
        need = ceil_div(lens[b] + q, page) - held
        wanted += need
        if need and wanted > top:
            continue
        for k in range(need):
            have -= 1
            table[b, held + k] = free[have]
        spent += need
        total[b] = lens[b] + q
        for k in range(q):
            p = lens[b] + k
            pg = int(table[b, p // page])
            pos[first + k] = p
            slot[first + k] = pg * page + p % page if 0 <= pg < n_pages else -1
    cu = [min(c, INT_MAX) for c in cu]
    return dict(cu=cu, total=total, slot=slot, pos=pos, n_free=[top - spent], table=table, free=free)


def gather(cache, table_row, T, n_pages):
    """Rows 0 .. T-1 of a request, [H_kv, T, d]; a page outside the cache is zeros."""
    _, Hkv, page, d = cache.shape
    out = np.zeros((Hkv, T, d))
    for p in range(0, T, page):
        pg, n = int(table_row[p // page]), min(page, T - p)
        if 0 <= pg < n_pages:
            out[:, p:p + n] = cache[pg, :, :n]
    return out


def paged_fwd(P1, cP2, cV, table, total, cu, tau, lam, Y0, max_new, with_spread=False):
    """Y [N, H, d] fp64: Y0 where no request writes. with_spread: also
    sum_j F_ij (|V_j| + |Y_i|) per output, the scale of a relative error of the weights."""
    N, H, d = P1.shape
    n_pages, Hkv, page, _ = cP2.shape
    Y, W = np.array(Y0, dtype=np.float64), np.zeros((N, H, d))
    for b in range(len(total)):
        q, T = int(cu[b + 1]) - int(cu[b]), int(total[b])
        if not (0 < q <= max_new and 0 <= cu[b] and cu[b + 1] <= N and q <= T <= table.shape[1] * page):
            continue
        k, v = gather(cP2, table[b], T, n_pages), gather(cV, table[b], T, n_pages)
        for h in range(H):
            g = h // (H // Hkv)
            for i in range(q):
                p, t = T - q + i, int(cu[b]) + i
                u = RO.evidence(P1[t, h][None], k[g, :p + 1])[0]
                logit = RO.silu(u) - lam * np.log(p + 1.0)
                logit[p] = RO.sigmoid(u[p:] / float(tau[h]))[0]
                w = np.exp(logit - logit.max())
                w /= w.sum()
                Y[t, h] = w @ v[g, :p + 1]
                W[t, h] = w @ (np.abs(v[g, :p + 1]) + np.abs(Y[t, h]))
    return (Y, W) if with_spread else Y
