"""8-bit V rows of the largest scales: the products that are summed are finite, and so is every step towards them."""
import numpy as np
import pytest
import torch

import _paged as P
import _paged_ex as X
import test_paged_ex_gpu as TX

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d,H,Hkv", [(64, 4, 2), (128, 8, 1), (80, 2, 2), (48, 24, 1), (32, 16, 2)])
@pytest.mark.parametrize("scale,u,reqs", [(254, 1.5, [(7, 1), (3, 2), (0, 4)]), (250, 4.5, [(20, 1), (12, 9), (40, 1)]),
                                          (246, 4.5, [(200, 1), (12, 9), (90, 40)]), (254, 1.5, [(3, 3)])])
def test_largest_scales(d, H, Hkv, scale, u, reqs):
    """Evidence u of all rows (weights of 2^1.8 and 2^6.4) and V of 2^-9 to 3 * 2^-9 times the scale: n weights times V stay
    below 2^127, a weight times the scale does not."""
    m = P.make("bf16", H, Hkv, d, 16, reqs, seed=d)
    a = (u / d**0.5)**0.5
    m["P1"] = torch.full_like(m["P1"], a)
    m["cP2"] = torch.where(m["cP2"].isnan(), m["cP2"], a)
    m = X.as_8bit(m)
    rng = np.random.default_rng(d)
    q = rng.integers(1, 4, tuple(m["cV"].shape)) * rng.choice([-1.0, 1.0], tuple(m["cV"].shape)) * 2.0**-9
    bits = m["scale"].view(torch.uint8).numpy().copy()
    held = bits[:, :, 1] != 255
    bits[:, :, 1][held] = scale
    m["scale"] = torch.from_numpy(bits).view(torch.float8_e8m0fnu)
    m["cV"] = torch.from_numpy(q).float().to(torch.float8_e4m3fn)
    m["v64"] = np.where(held[..., None], q * 2.0**(scale - 127), 0.0)
    TX.check_ex(m, 0.5)
    TX.check_ex(TX.with_trees(m, reqs, 2, d), 0.5)
