"""The weights of the paged forward: rows of the scan keep them whole for the transport."""
import numpy as np
import pytest
import torch

import _paged as P
import _paged_rows as PR
import test_paged_gpu as T
from oracle import paged_oracle as PO

pytestmark = pytest.mark.gpu


def classes(H, Hkv, d, page, reqs, seed):
    """A batch whose cached rows are of four kinds, each a P2 and a V of its own: the roundings of a kind's weights add up
    and do not average out, while Y itself is small where the kinds' V cancel."""
    m = P.make("bf16", H, Hkv, d, page, reqs, seed, stride_pad=8)
    rng = np.random.default_rng(seed)
    kinds = [torch.from_numpy(rng.standard_normal((Hkv, 4, d))).to(torch.bfloat16) for _ in range(2)]
    for b, (c, n) in enumerate(reqs):
        for p0 in range(0, c + n, page):
            k = min(page, c + n - p0)
            kind = torch.from_numpy(rng.integers(0, 4, k))
            for cache, x in zip(("cP2", "cV"), kinds):
                m[cache][m["table"][b, p0 // page], :, :k] = x[:, kind]
    return m


@pytest.mark.parametrize("H,Hkv,reqs", [
    (8, 8, [(0, 1), (1, 1), (2, 1), (5, 1), (40, 1), (300, 1), (701, 1)]), (8, 1, [(3, 1), (129, 2), (600, 1)]),
    (4, 2, [(2, 3), (70, 9), (200, 40)]), (6, 2, [(900, 5), (1, 2)]),
])
@pytest.mark.parametrize("d,page", [(32, 16), (48, 32), (64, 16), (80, 64), (128, 16)])
def test_scan_rows_keep_their_weights(d, page, H, Hkv, reqs):
    m = classes(H, Hkv, d, page, reqs, seed=d + H)
    Y = T.run_fwd(m, 0.5, None)
    zero = np.zeros(tuple(m["P1"].shape))
    ref, spread = PO.paged_fwd(P.f64(m["P1"]), np.nan_to_num(P.f64(m["cP2"])), np.nan_to_num(P.f64(m["cV"])),
                               m["table"].numpy(), m["total"].numpy(), m["cu"].numpy(), m["tau"], 0.5, zero, m["max_new"],
                               with_spread=True)
    du, e_max = PR.evidence_error(m["P1"], m["cP2"])
    lim = PR.weights_bound(ref, spread, int(m["total"].max()), du, e_max)
    err = np.abs(P.f64(Y) - ref)
    worst = np.unravel_index(np.argmax(err - lim), err.shape)
    assert np.all(err <= lim), (worst, err[worst], lim[worst], ref[worst])
