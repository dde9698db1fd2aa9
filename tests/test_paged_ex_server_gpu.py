"""A server that drafts trees and keeps a path of each, against one that never drafts."""
import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from causal_self_exchange_amd import workloads as W
from oracle import paged_ex_oracle as XO

import _paged as P
import _paged_ex as X
import test_paged_ex_gpu as TX

pytestmark = pytest.mark.gpu
DEV = "cuda"
i32 = TX.i32


class Server:
    def __init__(self, pages, H, Hkv, d, page, n_pages, S, width, rng):
        self.tdt = torch.bfloat16 if pages == "e4m3" else W.torch_dtype(pages)
        self.H, self.Hkv, self.d, self.page, self.n_pages = H, Hkv, d, page, n_pages
        cdt = torch.float8_e4m3fn if pages == "e4m3" else self.tdt
        self.caches = [torch.zeros((n_pages, Hkv, page, d), device=DEV).to(cdt) for _ in range(2)]
        self.scale = TX.scales(n_pages, Hkv, page) if pages == "e4m3" else None
        self.table = torch.full((S, width), P.BAD, dtype=torch.int32, device=DEV)
        self.free, self.n_free, self.lens = i32(rng.permutation(n_pages)), i32([n_pages]), i32([0] * S)

    def step(self, x, nn, tau, theta, rope, parent=None):
        """Y of the packed tokens x of nn new tokens a request; parent: they are trees."""
        N, H, Hkv, S = x.shape[0], self.H, self.Hkv, len(nn)
        out = tuple(torch.empty(k, dtype=torch.int32, device=DEV) for k in (S + 1, S, N, N)) + (self.n_free,)
        self.cu, self.total, slot, pos, _ = R.page_map(self.lens, i32(nn), self.table, self.free, self.n_free, N, self.page, self.n_pages, out=out)
        assert min(self.total.tolist()) >= 0
        tree = None
        if parent is not None:
            tree, pos = R.tree_plan(i32(parent), self.total, self.cu, 2)
        self.q = R.paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], slot, *self.caches, P1=x[:, :H], pos=pos, rope=rope, theta=theta,
                                scale=self.scale)
        self.pos = pos
        return R.paged_fwd(self.q, *self.caches, self.table, self.total, self.cu, tau, 0.5, max_new=max(1, *nn), scale=self.scale, tree=tree)

    def rows(self, b, n):
        tb = self.table[b].cpu().numpy()
        return [np.stack([c[tb[p // self.page], :, p % self.page] for p in range(n)]) for c in TX.rows_of(self.caches, self.scale)]

    def values(self):
        return [P.f64(c) * (2.0**TX.exps(self.scale)[:, :, j, :, None] if self.scale is not None else 1.0) for j, c in enumerate(self.caches)]


@pytest.mark.parametrize("pages,rope", [("e4m3", "half"), ("bf16", "interleaved"), ("f32", "half"), ("e4m3", "interleaved")])
def test_drafts_leave_no_trace(pages, rope):
    """The kept tokens' rows in the cache are, bit for bit, those of a server that appends the same tokens at
    relation_page_map's positions; their Y are both within the bound of that server's plain forward."""
    H, Hkv, d, page, S = 8, 2, 64, 16, 4
    rng = np.random.default_rng(17)
    a, b_ = (Server(pages, H, Hkv, d, page, 60, S, 20, rng) for _ in range(2))
    tau, theta = rng.uniform(0.5, 2.0, H).astype(np.float32), rng.uniform(-2, 2, 1).astype(np.float32)
    for step, nn in enumerate([[40, 7, 1, 65], [9, 20, 33, 1], [1, 12, 4, 30], [30, 6, 25, 6], [64, 18, 8, 3], [5, 5, 5, 5]]):
        N = sum(nn)
        x = torch.from_numpy(rng.standard_normal((N, H + 2 * Hkv, d))).to(a.tdt).to(DEV)
        parent = np.concatenate([np.arange(n) - 1 for n in nn]) if step == 0 else X.random_parents(nn, rng)
        Ya = a.step(x, nn, tau, theta, rope, parent)
        at = a.cu.tolist()
        paths = []
        for r, n in enumerate(nn):
            leaf = n - 1 if step == 0 else int(rng.integers(0, n))
            paths.append(sorted(XO.ancestors(parent[at[r]:at[r + 1]], leaf)) + [leaf])
        keep = np.zeros(N, dtype=np.int64)
        for r, p in enumerate(paths):
            keep[at[r]:at[r] + len(p)] = p
        picked = [at[r] + i for r, p in enumerate(paths) for i in p]
        Yb = b_.step(x[picked].contiguous(), [len(p) for p in paths], tau, theta, rope)
        torch.cuda.synchronize()
        assert a.pos[picked].tolist() == b_.pos.tolist()
        assert torch.equal(a.q[picked], b_.q)
        R.paged_keep(*a.caches, a.table, a.total, a.cu, i32(keep), i32([len(p) for p in paths]), a.lens, a.free, a.n_free,
                     n_free_out=a.n_free, scale=a.scale)
        b_.lens = b_.total.clone()
        torch.cuda.synchronize()
        assert a.lens.tolist() == b_.lens.tolist() and int(a.n_free) == int(b_.n_free)
        for r in range(S):
            for g, w in zip(a.rows(r, int(a.lens[r])), b_.rows(r, int(a.lens[r]))):
                np.testing.assert_array_equal(g, w)
        k, v = b_.values()
        ref, spread = XO.paged_fwd(P.f64(b_.q), k, v, b_.table.cpu().numpy(), b_.total.cpu().numpy(), b_.cu.cpu().numpy(), tau, 0.5,
                                   np.zeros(tuple(b_.q.shape)), max(len(p) for p in paths))
        lim = TX.limit(dict(P1=b_.q, cP2=b_.caches[0], table=b_.table, total=b_.total, max_new=max(len(p) for p in paths), N=len(picked),
                            tree=None), ref, spread, k)
        for y in (Ya[picked], Yb):
            assert np.all(np.abs(P.f64(y) - ref) <= lim)
