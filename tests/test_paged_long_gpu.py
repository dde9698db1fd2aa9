"""The paged forward over segments of more than 4,096 keys, whose block-table entries a wave takes in several windows.
Every 1,024 rows of a request have an evidence level and a V of their own, so that rows of another part of the table
give another output; sampled rows against fp64."""
import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from causal_self_exchange_amd import workloads as W

import _paged as P
import _paged_rows as PR

pytestmark = pytest.mark.gpu
DEV = "cuda"


def levels(dt, H, Hkv, d, page, reqs, seed):
    """A batch over one set of pages: the table of request b is a permutation's turn by 37 b pages. P2 holds an evidence level
    (0 or 3) of its 1,024 rows in column 0, noise elsewhere; P1's column 0 is sqrt(d). V holds a level too."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    tdt = W.torch_dtype(dt)
    total = [c + n for c, n in reqs]
    n_pages = -(-max(total) // page)
    perm = torch.randperm(n_pages, generator=g, device=DEV)
    table = torch.stack([perm.roll(37 * b) for b in range(len(reqs))]).to(torch.int32)
    cP2 = torch.randn((n_pages, Hkv, page, d), generator=g, device=DEV) * 0.3
    cV = torch.randn((n_pages, Hkv, page, d), generator=g, device=DEV) * 0.3
    part = torch.empty(n_pages, dtype=torch.long, device=DEV)
    part[perm] = torch.arange(n_pages, device=DEV) * page // 1024
    k = int(part.max()) + 1
    cP2[..., 0] = 3.0 * torch.randint(0, 2, (k, Hkv), generator=g, device=DEV)[part][:, :, None]
    cV += 2.0 * torch.randn((k, Hkv, d), generator=g, device=DEV)[part][:, :, None]
    N = sum(n for _, n in reqs)
    P1 = torch.randn((N, H, d), generator=g, device=DEV)
    P1[..., 0] = float(np.sqrt(d))
    cu = np.concatenate([[0], np.cumsum([n for _, n in reqs])]).astype(np.int32)
    tau = np.random.default_rng(seed).uniform(0.5, 2.0, H).astype(np.float32)
    return dict(P1=P1.to(tdt), cP2=cP2.to(tdt), cV=cV.to(tdt), table=table, total=torch.tensor(total, dtype=torch.int32, device=DEV),
                cu=torch.from_numpy(cu).to(DEV), tau=tau, max_new=max(n for _, n in reqs), N=N)


def bound(dt, n):
    """Numerator and row sum have n fp32 additions at most each, 2^-24 of it relative. bf16: besides, P.bound, du below 1e-4
    (d 2^-24 of magnitudes below 100 over sqrt(d)); fp32: weights 1.1 du + 2^-18, du as above."""
    sums = 2 * n * 2.0**-24
    if dt == "bf16":
        return lambda r, s: sums * s + P.bound(r, s, "bf16", 1e-4)
    return lambda r, s: (sums + 1.1e-4 + 2.0**-18) * s


def check(m, dt, lam, picks):
    Y = R.paged_fwd(m["P1"], m["cP2"], m["cV"], m["table"], m["total"], m["cu"], m["tau"], lam, max_new=m["max_new"])
    torch.cuda.synchronize()
    H = m["P1"].shape[1]
    for b, rows in picks:
        PR.check_rows(m, Y, b, rows, sorted({0, H // 2, H - 1}), lam, bound(dt, int(m["total"][b])))


@pytest.mark.parametrize("dt,d,H,Hkv,page,S,T,n", [
    # Scan units (314 of 128 keys and two a row block) over the work-groups of the launch: about 78 each, a step of every
    # wave per unit in bf16 and two in fp32, of 32 and 64 in a window.
    ("bf16", 128, 8, 8, 16, 16, 40000, 1),       # 128 row blocks, 512 work-groups
    ("bf16", 64, 16, 16, 64, 16, 40000, 1),      # 256 row blocks, 1,024 work-groups
    ("bf16", 64, 32, 4, 16, 32, 40003, 3),       # 24 rows a block of 32: 128 row blocks, 512 work-groups
    ("bf16", 80, 8, 8, 128, 16, 40000, 1),
    ("bf16", 32, 16, 16, 256, 16, 40000, 1),
    ("f32", 64, 16, 16, 16, 16, 40000, 1),
    ("f32", 128, 32, 4, 64, 32, 40003, 3),
    ("f32", 48, 8, 8, 16, 32, 40000, 1),
])
def test_scan_segments_past_one_window(dt, d, H, Hkv, page, S, T, n):
    m = levels(dt, H, Hkv, d, page, [(T - n - 101 * b, n) for b in range(S)], seed=d + H)
    check(m, dt, 0.5, [(0, [0, n - 1]), (3, [n - 1]), (S - 1, [0])])


@pytest.mark.parametrize("d,H,Hkv,page", [(64, 8, 2, 16), (128, 8, 8, 64), (80, 6, 2, 128)])
def test_tile_segments_past_one_window(d, H, Hkv, page):
    """A chunk of 2,048 tokens over 40,001 rows: about 8 tiles a head of 650 key tiles, over 256 work-groups more than 110 each."""
    m = levels("bf16", H, Hkv, d, page, [(40001, 2048), (39000, 1)], seed=d)
    check(m, "bf16", 0.5, [(0, [0, 30, 31, 32, 1000, 2047]), (1, [0])])
