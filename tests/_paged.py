"""Inputs of the paged Relation Cache tests, and the bounds of its outputs."""
from __future__ import annotations

import numpy as np
import torch

from causal_self_exchange_amd import workloads as W

BAD = -7                        # a page number outside every cache


def make(dt, H, Hkv, d, page, reqs, seed, scale=1.0, stride_pad=0, pad_rows=0, spare=2, tau=None):
    """A batch of requests (cached, new): pages in shuffled order, NaN in every
    cache row that no request holds, table entries past a request's pages BAD.
    CPU tensors; P1 with stride_pad extra elements between tokens."""
    rng = np.random.default_rng(seed)
    tdt = W.torch_dtype(dt)
    total = [c + n for c, n in reqs]
    held = [-(-t // page) for t in total]
    n_pages = sum(held) + spare
    width = max(max(held), 1) + 1
    order = rng.permutation(n_pages)
    table = np.full((len(reqs), width), BAD, dtype=np.int32)
    cP2 = torch.full((n_pages, Hkv, page, d), float("nan"), dtype=tdt)
    cV = torch.full((n_pages, Hkv, page, d), float("nan"), dtype=tdt)
    at = 0
    for b, t in enumerate(total):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
        for k in range(held[b]):
            n = min(page, t - k * page)
            cP2[table[b, k], :, :n] = torch.from_numpy(scale * rng.standard_normal((Hkv, n, d))).to(tdt)
            cV[table[b, k], :, :n] = torch.from_numpy(rng.standard_normal((Hkv, n, d))).to(tdt)
    cu = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
    N = max(1, int(cu[-1]) + pad_rows)
    wide = torch.from_numpy(scale * rng.standard_normal((N, H * d + stride_pad))).to(tdt)
    P1 = wide[:, :H * d].unflatten(1, (H, d))
    tau = rng.uniform(0.5, 2.0, H).astype(np.float32) if tau is None else np.full(H, tau, np.float32)
    return dict(P1=P1, cP2=cP2, cV=cV, table=torch.from_numpy(table),
                total=torch.tensor(total, dtype=torch.int32), cu=torch.from_numpy(cu), tau=tau,
                max_new=max([1] + [n for _, n in reqs]), N=N)


def to_device(m, dev="cuda"):
    """The same on the device; P1 keeps its token stride."""
    out = dict(m)
    for k in ("cP2", "cV", "table", "total", "cu"):
        out[k] = m[k].to(dev)
    P1 = m["P1"]
    wide = torch.empty((P1.shape[0], P1.stride(0)), dtype=P1.dtype, device=dev).fill_(float("nan"))
    view = wide[:, :P1.shape[1] * P1.shape[2]].unflatten(1, tuple(P1.shape[1:]))
    view.copy_(P1)
    out["P1"] = view
    return out


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def bound(ref, spread, dt, du=0.0):
    """Elementwise bound of |Y - Y*|.

    bf16: the weights of the transport and the row of Y are rounded once each, by
    at most 2^-8 relative, and the normaliser is formed from the weights before or
    after rounding: at most 2^-8 sum_j F_j (|V_j| + |Y|) and 2^-8 |Y|. The rest is
    fp32: an error du of the evidence moves a weight by at most 1.1 du relative
    (|SiLU'| < 1.1). With du below 1e-4 it stays within 5% of the rounding terms.
    fp32: the weights carry du (given) and about 2^-19 from the exponentials, the
    sums 2^-19 sum_j F_j |V_j| for the lengths here (6 sqrt(n) 2^-24, n <= 2^15 / 4)."""
    if dt == "bf16":
        return (1.05 * 2.0**-8 + 1.1 * du) * (spread + np.abs(ref)) + 1e-7
    return (2.0**-18 + 1.1 * du) * (spread + np.abs(ref)) + 1e-9
