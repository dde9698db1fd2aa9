"""Chunks on query tiles of the paged forward, next to the same calls in the scan: the selection of kernels, and what the
scan's small batches do not reach of the tiles."""
import numpy as np
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


@pytest.mark.parametrize("d,page,H,Hkv", [(128, 16, 4, 2), (64, 64, 2, 2), (80, 32, 3, 1), (48, 16, 2, 1), (32, 128, 2, 2)])
def test_chunks(d, page, H, Hkv):
    reqs = T.CHUNKS + [T.filler(H)]
    m = P.make("bf16", H, Hkv, d, page, reqs, seed=d + H, stride_pad=32, pad_rows=5)
    T.check_fwd(m, 0.5, "bf16", skip=len(T.CHUNKS))
    check_tiles(m, len(T.CHUNKS))


@pytest.mark.parametrize("reqs", [T.CHUNKS, T.RAGGED + [(500, 300)]])
def test_large_evidence(reqs):
    """Evidence far beyond the exponent range of an unshifted exponential: the tiles' second pass, and joins of states with
    a stabiliser of their own. du as in test_paged_fwd_large_evidence (scale 5, d = 64)."""
    m = P.make("bf16", 4, 2, 64, 16, reqs + [T.filler(4)], seed=5, scale=5.0)
    T.check_fwd(m, 0.5, "bf16", du=2e-3, skip=len(reqs))
    check_tiles(m, len(reqs), du=2e-3)


def test_pages_outside_the_cache_read_as_zeros():
    m = P.make("bf16", 4, 2, 64, 16, T.CHUNKS + [T.filler(4)], seed=8)
    bad = [P.BAD, m["cP2"].shape[0], 2**31 - 1]
    for b in range(len(T.CHUNKS)):
        m["table"][b, 0] = bad[b % 3]
    for k, p in enumerate((0, 7, 8, 63, 64, 130, 400, 401, 402, 403, 999)):
        m["table"][len(T.CHUNKS), p] = bad[k % 3]
    T.check_fwd(m, 0.5, "bf16", skip=len(T.CHUNKS))
    check_tiles(m, len(T.CHUNKS))


def test_shared_pages():
    m = P.make("bf16", 8, 2, 128, 16, [(64, 170), T.filler(8), (64, 150)], seed=4)
    for b in (0, 2):
        m["table"][b, :4] = m["table"][1, :4]
    T.check_fwd(m, 0.5, "bf16", skip=1)
    check_tiles(m, 1)


def test_other_rows_stay():
    """Refused, empty, oversized and inconsistent requests next to tiles."""
    m = P.make("bf16", 4, 2, 64, 16, [(10, 150), (0, 0), (40, 300), (7, 1), (30, 900), (5, 200), (2, 130), T.filler(4)], seed=3,
               pad_rows=40)
    m["total"][2] = -1
    m["total"][3] = 0
    m["total"][5] = m["table"].shape[1] * 16 + 1
    T.check_fwd(m, 0.5, "bf16", max_new=700, skip=7)      # request 4 has more than 700 new tokens
    check_tiles(m, 7, max_new=700)
    m["cu"][0] = -2
    T.check_fwd(m, 0.5, "bf16", max_new=1000, skip=7)


def test_caches_past_32_bit_offsets():
    """Tiles over pages on both sides of 2^31 and 2^32 elements, against the same pages in a small cache."""
    H, Hkv, d, page = 4, 2, 128, 256
    per = Hkv * page * d
    n_pages = (1 << 32) // per + 40
    m = P.make("bf16", H, Hkv, d, page, [(100, 160), T.filler(4)], seed=7)
    held = int(m["cP2"].shape[0])
    marks = [(1 << 31) // per, (1 << 32) // per]
    where = np.array([0, n_pages - 1] + [k + j for k in marks for j in range(-15, 15)] + list(range(50, 50 + held)))[:held]
    assert len(set(where)) == held
    big = [torch.empty((n_pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    at = torch.from_numpy(where).to(DEV)
    for b, c in zip(big, (m["cP2"], m["cV"])):
        b[at] = c.to(DEV)
    small = m["table"].numpy()
    table = torch.from_numpy(np.where(small >= 0, where[np.clip(small, 0, None)], P.BAD).astype(np.int32)).to(DEV)
    Y, S = check_tiles(m, 1)
    assert torch.equal(call(m, caches=big, table=table), Y)
    assert torch.equal(call(m, "scan", caches=big, table=table), S)


def test_serving_loop_on_tiles():
    """A prompt and its continuation on tiles (10,000 and 11,700 units of work), single tokens and a
    chunk in the scan: the rows of one forward. The bar of test_serving_loop."""
    s = T.Server("bf16", 8, 2, 64, 16, 300, 3, 250, seed=5)
    s.step([2100, 0, 70], 2200)
    s.step([1500, 300, 1], 1801)
    s.step([1, 2, 1], 5)
    s.step([300, 1, 0], 301)
    s.check(3e-2)
