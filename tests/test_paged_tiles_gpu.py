"""Chunks on query tiles of the paged forward, next to the same calls in the scan."""
import pytest
import torch

from causal_self_exchange_amd import relation as R

import _paged as P
import _paged_rows as PR
import test_paged_gpu as T
import test_paged_weights_gpu as TW

pytestmark = pytest.mark.gpu
DEV = "cuda"


def call(m, fwd="auto", fill=3.0, max_new=None, caches=None, table=None):
    d = P.to_device(m)
    Y = torch.full(tuple(m["P1"].shape), fill, dtype=m["P1"].dtype, device=DEV)
    cP2, cV = (d["cP2"], d["cV"]) if caches is None else caches
    with R.kernels(fwd=fwd):
        R.paged_fwd(d["P1"], cP2, cV, d["table"] if table is None else table, d["total"], d["cu"], m["tau"], 0.5,
                    max_new=m["max_new"] if max_new is None else max_new, out=Y)
    torch.cuda.synchronize()
    return Y


def same(a, b):
    return torch.equal(a, b)


def check_tiles(m, b, dt="bf16", du=1e-6, max_new=None, heads=(0, -1), caches=None, table=None):
    """The batch with work enough for query tiles in request b: the call takes them (its bits are not the scan's), and of
    request b the rows around the tiles' and blocks' ends are compared."""
    Y = call(m, max_new=max_new, caches=caches, table=table)
    S = call(m, "scan", max_new=max_new, caches=caches, table=table)
    differ = not same(Y, S)
    assert differ
    H = m["P1"].shape[1]
    n = int(m["cu"][b + 1] - m["cu"][b])
    picks = sorted({0, 1, n // 3, n // 2, n - 33, n - 1, min(n - 1, 255), min(n - 1, 256)} & set(range(n)))
    for y in (Y, S):
        PR.check_rows(m, y, b, picks, [h % H for h in heads], 0.5, lambda r, s: P.bound(r, s, dt, du))
    return Y, S


def test_selection_of_kernels():
    """REL_KERNEL_SCAN keeps chunks off the query tiles; a batch that has no work for tiles is the same either way."""
    m = P.make("bf16", 8, 2, 64, 16, T.CHUNKS + [T.filler(8)], seed=2)
    Y, S = check_tiles(m, len(T.CHUNKS))
    assert torch.equal(call(m, "scan"), S) and torch.equal(call(m), Y)
    m = P.make("bf16", 8, 2, 64, 16, T.CHUNKS, seed=2)
    assert torch.equal(call(m), call(m, "scan"))
    m = P.make("f32", 8, 2, 64, 16, T.CHUNKS, seed=2)
    assert torch.equal(call(m), call(m, "scan"))


def test_rows_of_the_scan_keep_their_weights_in_prompts():
    """A prompt with enough work for tiles, in the scan by selection. A wave adds a quarter of the keys, then the waves and up
    to 257 parts meet."""
    m = TW.classes(8, 2, 64, 16, [T.filler(8)], seed=3)
    du, e_max = PR.evidence_error(m["P1"], m["cP2"])
    n = int(m["total"][0]) // 4 + 300
    PR.check_rows(m, call(m, "scan"), 0, [0, 5, 100, m["max_new"] - 1], [0, 3, 7], 0.5,
                  lambda r, s: PR.weights_bound(r, s, n, du, e_max))
