"""The paged forward where unshifted weights times V pass the fp32 range while the outputs do not."""
import pytest
import torch

import _paged as P
import _paged_rows as PR
import test_paged_gpu as T

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,d,H,Hkv,reqs", [
    ("bf16", 64, 4, 2, [(40, 1), (300, 3), (700, 1), (10, 33)]), ("bf16", 128, 2, 2, [(500, 1), (90, 1)]),
    ("bf16", 80, 4, 1, [(60, 70)]), ("f32", 64, 4, 2, [(40, 1), (300, 3), (10, 33)]), ("f32", 128, 2, 1, [(400, 1), (0, 40)]),
])
def test_scan_of_large_values(dt, d, H, Hkv, reqs):
    """V of magnitude 2^100 beside evidence of some tens. The stabiliser follows a score within 2^8, so n keys' weights times
    V stay below n 2^8 2^103. du as for evidence of some hundreds in test_paged_fwd_large_evidence, over d = 128: the sum
    of magnitudes below 128 * 9 * 2 / pi * 3, 128 of them: 128 2^-24 2200 / sqrt(128) = 1.5e-3; |E| 2^-22 below 1e-4."""
    m = P.make(dt, H, Hkv, d, 16, reqs, seed=d + H, scale=3.0)
    m["cV"] *= 2.0**100
    T.check_fwd(m, 0.5, dt, du=2e-3)


def test_joined_tiles_of_large_values():
    """Query tiles cut into many parts, each of which sums to less than the fp32 range while all of them together do not:
    16,000 rows of one evidence of 9 (weights of 2^13) and V about 2^102. du: 64 equal products, sums of up to 72, each
    addition 2^-24 of it: 64 * 72 * 2^-24 / 8 = 3.5e-5; |E| 2^-22 = 4e-6."""
    H, d, (ctx, n) = 2, 64, T.filler(2)
    m = P.make("bf16", H, 1, d, 64, [(ctx, n)], seed=1)
    m["P1"] = torch.full_like(m["P1"], 1.0625)
    m["cP2"] = torch.where(m["cP2"].isnan(), m["cP2"], 1.0625)
    m["cV"] = (2.0**102 * (1.0 + 0.25 * m["cV"].float())).to(torch.bfloat16)
    Y = T.run_fwd(m, 0.5, None)
    assert bool(torch.isfinite(Y).all())
    PR.check_rows(m, Y, 0, [0, 1, 255, 256, 700, n - 1], [0, 1], 0.5, lambda r, s: P.bound(r, s, "bf16", 4e-5))
