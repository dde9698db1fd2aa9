"""Positions of tokens of requests that run past the packed batch, which relation_page_map refuses."""
import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from oracle import paged_ex_oracle as XO
from oracle import paged_oracle as PO

BATCHES = [([3, 4, 5], 9), ([3, 4, 5], 7), ([9], 4), ([2, 0, 50, 1, 0, 3], 20), ([1] * 300 + [40] + [1] * 700, 320), ([600, 700], 1000),
           ([2**30, 2**30, 2**30, 1], 6), ([5, 6], 11)]


def maps(nn, N):
    S = len(nn)
    return PO.page_map([7] * S, nn, np.zeros((S, 300)), list(range(5000)), 5000, N, 16, 5000)


@pytest.mark.parametrize("nn,N", BATCHES)
def test_plain_plan_has_the_page_maps_positions(nn, N):
    m = maps(nn, N)
    _, pos = XO.tree_plan(np.arange(N) - 1, m["total"], m["cu"], 1, np.zeros((N, 1)), np.full(N, 77))
    refused = np.array(m["pos"]) < 0
    assert (pos[refused] == -1).all() and (pos[~refused] >= 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("nn,N", BATCHES)
def test_tokens_of_requests_past_the_batch(nn, N):
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    m, S = maps(nn, N), len(nn)
    cu, total, _, pos0, _ = R.page_map(i32([7] * S), i32(nn), i32(np.zeros((S, 300))), i32(np.arange(5000)), i32([5000]), N, 16, 5000)
    rng = np.random.default_rng(N)
    parent = rng.integers(-1, 12, N)
    for words in (1, 32):
        out = tuple(torch.full(s, 77, dtype=torch.int32, device="cuda") for s in ((N, words), (N,)))
        R.tree_plan(i32(parent), total, cu, words, out=out)
        torch.cuda.synchronize()
        want = XO.tree_plan(parent, m["total"], m["cu"], words, np.full((N, words), 77), np.full(N, 77))
        for g, w in zip(out, want):
            np.testing.assert_array_equal(g.cpu().numpy(), w)
        assert (out[1][pos0 < 0] == -1).all()
