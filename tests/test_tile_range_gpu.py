"""Query tiles whose weights at the fixed offset times V pass the fp32 range, with values of both signs: such sums are NaN
and not infinite, and the outputs are finite."""
import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from oracle import relation_oracle as RO

import _paged as P
import _paged_ex as X
import _paged_rows as PR
import test_paged_ex_gpu as TX
import test_paged_gpu as T

pytestmark = pytest.mark.gpu
DEV = "cuda"


def evident(m, top):
    """m with evidence of some 57 (sqrt(d) times 2.66^2, and less for d = 128; weights of about 2^80) and V of magnitude 2^top."""
    d = m["P1"].shape[-1]
    a = {64: 2.65625, 80: 2.5, 48: 2.859375, 128: 2.234375}[d]
    m["P1"] = torch.full_like(m["P1"], a)
    m["cP2"] = torch.where(m["cP2"].isnan(), m["cP2"], a + 0.25 * m["cP2"].float()).to(m["cP2"].dtype)
    m["cV"] *= 2.0**top
    return m


@pytest.mark.parametrize("d,T_,top,lse", [(64, 700, 60, False), (128, 600, 60, False), (64, 700, 100, True), (128, 520, 60, True),
                                          (80, 600, 100, False), (48, 600, 60, True)])
def test_forward(d, T_, top, lse):
    """P1 is one number, which the inference forward scales and rounds again: by half a step (2^-8) of all evidence alike, so
    two keys' weights part by 2^-8 of the difference of their evidence. fp32 sums as in _paged_rows."""
    m = evident(P.make("bf16", 2, 2, d, 16, [(0, T_)], seed=d + T_), top)
    pages = m["table"][0, :-(-T_ // 16)].long()
    P1 = m["P1"].transpose(0, 1)[None].contiguous()
    P2, V = (m[c][pages].transpose(0, 1).reshape(2, -1, d)[:, :T_][None].contiguous() for c in ("cP2", "cV"))
    Y = (R.fwd_lse(P1.to(DEV), P2.to(DEV), V.to(DEV), m["tau"], 0.5)[0] if lse else R.fwd(P1.to(DEV), P2.to(DEV), V.to(DEV), m["tau"], 0.5))
    torch.cuda.synchronize()
    at_most, e_max = PR.evidence_error(P1, P2)
    picks = [0, 1, 31, 32, 255, 256, 300, 511, 512, T_ - 1]
    for h in range(2):
        u = RO.evidence(P.f64(P1[0, h]), P.f64(P2[0, h]))
        apart = 0.0 if lse else float(u.max() - u.min()) * 2.0**-8
        ref, spread = PR.rows_of(m, 0, picks, [h], 0.5)
        err = np.abs(P.f64(Y[0, h])[picks] - ref[:, 0])
        assert np.all(err <= P.bound(ref[:, 0], spread[:, 0], "bf16", at_most + apart + 8 * e_max * 2.0**-24))


@pytest.mark.parametrize("d,top", [(64, 60), (128, 100)])
def test_paged_chunks(d, top):
    """Chunks on the forward's tiles, whole and in parts."""
    m = evident(P.make("bf16", 4, 2, d, 16, [(400, 300), (700, 70), T.filler(4)], seed=d), top)
    Y = T.run_fwd(m, 0.5, None)
    at_most, e_max = PR.evidence_error(m["P1"], m["cP2"])
    for b, n in ((0, 300), (1, 70), (2, T.filler(4)[1])):
        PR.check_rows(m, Y, b, sorted({0, 1, n // 2, n - 1, min(n - 1, 256)}), [0, 3], 0.5,
                      lambda r, s: P.bound(r, s, "bf16", at_most + 8 * e_max * 2.0**-24))


@pytest.mark.parametrize("pages,d,H,Hkv,reqs", [
    ("e4m3", 128, 4, 2, [(400, 90), (700, 64), (300, 33)]), ("e4m3", 64, 8, 2, [(400, 20), (900, 31), (333, 17)]),
    ("e4m3", 64, 4, 1, [(12000, 90)]), ("e4m3", 80, 4, 1, [(12000, 30)]), ("e4m3", 48, 8, 1, [(9000, 12)]),
    ("bf16", 128, 4, 1, [(500, 60), (9000, 64)]), ("bf16", 64, 4, 1, [(500, 30), (9000, 32)]), ("bf16", 64, 4, 2, [(400, 64), (330, 64)]),
])
@pytest.mark.parametrize("top", [60, 100])
def test_query_tiles(pages, d, H, Hkv, reqs, top):
    """8-bit pages and trees, tiles of 128 and of 256 rows, whole and in parts."""
    m = evident(P.make("bf16", H, Hkv, d, 16, reqs, seed=d + H), top)
    if pages == "e4m3":
        m = X.as_8bit(m)
    tree = TX.with_trees(dict(m), reqs, 3, d)
    for x in ([m] if pages == "e4m3" else []) + [tree]:
        assert TX.tile_rows(TX.widened(x)) == 0
        TX.check_ex(x, 0.5)


@pytest.mark.parametrize("top", [99.5, 102.0])
@pytest.mark.parametrize("d,H,n", [(64, 8, 16), (64, 8, 32)])
def test_parts_of_large_values(d, H, n, top):
    """A row block in as many parts as there are ranges, of four waves (512) and of eight (256): 140,000 rows of one evidence
    of 9 (weights of 2^13) and V about 2^top, so parts just below the range over their number, and more than the range together.
    du as in test_joined_tiles_of_large_values."""
    m = P.make("bf16", H, 1, d, 64, [(140000, n)], seed=1)
    m["P1"] = torch.full_like(m["P1"], 1.0625)
    m["cP2"] = torch.where(m["cP2"].isnan(), m["cP2"], 1.0625)
    m["cV"] = (2.0**(top - 2) * (1.0 + 0.25 * m["cV"].float())).to(torch.bfloat16)
    m = X.as_8bit(m)
    assert TX.tile_rows(m) == 0
    Y = TX.run_ex(m, 0.5)
    assert bool(torch.isfinite(Y).all())
    w = dict(m, cP2=torch.from_numpy(m["k64"]), cV=torch.from_numpy(m["v64"]))
    PR.check_rows(w, Y, 0, [0, n - 1], [0, H - 1], 0.5, lambda r, s: P.bound(r, s, "bf16", 4e-5))
