"""Single tokens in batches that go to query tiles whole: their weights are kept as in the scan, whatever the others are."""
import numpy as np
import pytest
import torch

from oracle import paged_ex_oracle as XO

import _paged as P
import _paged_ex as X
import _paged_rows as PR
import test_paged_ex_gpu as TX
import test_paged_weights_gpu as TW

pytestmark = pytest.mark.gpu

REQS = [(40, 1), (300, 19), (701, 1), (20, 24), (63, 1), (1, 30), (2, 1), (0, 1), (64, 1), (1500, 20), (65, 1), (5000, 1), (300, 21), (0, 33)]


@pytest.mark.parametrize("pages", ["e4m3", "bf16"])
@pytest.mark.parametrize("d,H,Hkv,page", [(128, 8, 2, 16), (64, 8, 2, 16), (64, 4, 1, 64), (80, 16, 2, 16), (48, 12, 2, 32), (32, 24, 1, 16)])
def test_single_tokens_keep_their_weights(pages, d, H, Hkv, page):
    """Cached rows of four kinds, so that roundings of a weight add up (test_paged_weights_gpu)."""
    m = TW.classes(H, Hkv, d, page, REQS, seed=d + H)
    k, v = (np.nan_to_num(P.f64(m[c])) for c in ("cP2", "cV"))
    if pages == "e4m3":
        m = X.as_8bit(m)
        k, v = m["k64"], m["v64"]
    for x in ([m] if pages == "e4m3" else []) + [TX.with_trees(dict(m), REQS, 2, d)]:
        x = TX.widened(x)
        assert TX.tile_rows(x) == 0
        tree = x["tree"].numpy() if x.get("tree") is not None else None
        ref, spread = XO.paged_fwd(P.f64(x["P1"]), k, v, x["table"].numpy(), x["total"].numpy(), x["cu"].numpy(), x["tau"], 0.5,
                                   np.zeros(tuple(x["P1"].shape)), x["max_new"], tree=tree)
        Y = P.f64(TX.run_ex(x, 0.5))
        at_most, e_max = PR.evidence_error(x["P1"], torch.from_numpy(k))
        kept = PR.weights_bound(ref, spread, int(x["total"].max()), at_most, e_max)
        one = np.zeros((x["N"], 1, 1), bool)
        for a, b in zip(x["cu"].tolist(), x["cu"].tolist()[1:]):
            one[a] |= b - a == 1
        lim = np.where(one, kept, P.bound(ref, spread, "bf16", at_most + 8 * e_max * 2.0**-24))
        err = np.abs(Y - ref)
        worst = np.unravel_index(np.argmax((err - lim) * one), err.shape)
        assert np.all(err <= lim), (worst, err[worst], lim[worst], ref[worst])
