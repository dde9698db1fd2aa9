"""Query tiles whose weights at the fixed offset times V pass the fp32 range, with values of both signs: such sums are NaN
and not infinite, and the outputs are finite."""
import pytest
import torch

import _paged as P
import _paged_ex as X
import test_paged_ex_gpu as TX

pytestmark = pytest.mark.gpu


def evident(m, top):
    """m with evidence of some 57 (sqrt(d) times 2.66^2, and less for d = 128; weights of about 2^80) and V of magnitude 2^top."""
    d = m["P1"].shape[-1]
    a = {64: 2.65625, 80: 2.5, 48: 2.859375, 128: 2.234375}[d]
    m["P1"] = torch.full_like(m["P1"], a)
    m["cP2"] = torch.where(m["cP2"].isnan(), m["cP2"], a + 0.25 * m["cP2"].float()).to(m["cP2"].dtype)
    m["cV"] *= 2.0**top
    return m


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
