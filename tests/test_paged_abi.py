"""Refusals of the paged Relation Cache that need no GPU: the C ABI rejects
every invalid call before any HIP call, the binding checks its tensors, and the
plain page map keeps its invariants."""
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from oracle import paged_oracle as PO

(OK, E_NULL, E_SHAPE, E_DTYPE, E_HEADDIM, E_TAU, E_LAMBDA, E_ALIGN, E_ALIAS, E_WS, E_LAUNCH, E_PRESTEP, E_KERNEL, E_PAGE,
 E_GROUP, E_STRIDE) = range(16)
BIG = 1 << 40


def at(k):
    """Fake, never-dereferenced device addresses, 1 TiB apart."""
    return BIG * (k + 1)


def fptr(vals):
    import ctypes
    if vals is None:
        return None, None
    arr = np.asarray(vals, dtype=np.float32)
    return arr, arr.ctypes.data_as(ctypes.POINTER(ctypes.c_float))


MAP = dict(len=at(0), n_new=at(1), table=at(2), free=at(3), n_free=at(4), n_free_out=at(5), cu=at(6), total=at(7), slot=at(8),
           pos=at(9), S=4, N=32, F=10, max_pages=8, page=16, n_pages=50)


def page_map(**kw):
    m = {**MAP, **kw}
    return R.lib().relation_page_map(*(m[k] for k in MAP), None)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, E_NULL) for k in list(MAP)[:10]],
    (dict(S=0), E_SHAPE), (dict(S=65536), E_SHAPE), (dict(N=0), E_SHAPE), (dict(F=0), E_SHAPE), (dict(N=-1), E_SHAPE),
    (dict(page=8), E_PAGE), (dict(page=48), E_PAGE), (dict(page=512), E_PAGE), (dict(page=0), E_PAGE), (dict(n_pages=0), E_PAGE),
    (dict(n_pages=1 << 27), E_PAGE), (dict(max_pages=0), E_PAGE), (dict(max_pages=1 << 27), E_PAGE),
    (dict(len=at(0) + 2), E_ALIGN), (dict(pos=at(9) + 1), E_ALIGN),
    (dict(cu=at(0) + 12), E_ALIAS), (dict(total=at(0)), E_ALIAS), (dict(slot=at(9) - 4), E_ALIAS), (dict(free=at(2) + 124), E_ALIAS),
    (dict(n_free_out=at(1)), E_ALIAS), (dict(n_free=at(3) + 4), E_ALIAS), (dict(n_free=at(6), n_free_out=at(6)), E_ALIAS),
])
def test_page_map_rejects(kw, code):
    assert page_map(**kw) == code


APP = dict(P1=at(0), P2=at(1), I=at(2), ld1=512, ld2=128, ldi=128, slot=at(3), pos=at(4), rope=1, base=1e4, theta=(0.1,), pairing=0,
           P1o=at(5), cP2=at(6), cV=at(7), N=9, H=8, Hkv=2, d=64, n_pages=20, page=16, dt=R.REL_BF16)


def append(**kw):
    m = {**APP, **kw}
    keep, th = fptr(m["theta"])
    return R.lib().relation_paged_append(*(th if k == "theta" else m[k] for k in APP), None)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, E_NULL) for k in ("P1", "P2", "I", "slot", "pos", "P1o", "cP2", "cV")],
    (dict(N=0), E_SHAPE), (dict(H=0), E_SHAPE), (dict(H=257, ld1=257 * 64), E_SHAPE), (dict(Hkv=0), E_SHAPE), (dict(Hkv=257), E_SHAPE),
    (dict(Hkv=1, theta=(0.1,)), E_SHAPE), (dict(dt=5), E_DTYPE), (dict(d=96), E_HEADDIM), (dict(d=0), E_HEADDIM),
    (dict(page=17), E_PAGE), (dict(n_pages=-1), E_PAGE), (dict(n_pages=1 << 30), E_PAGE),
    (dict(ld1=511), E_STRIDE), (dict(ld1=516), E_STRIDE), (dict(ld2=64), E_STRIDE), (dict(ldi=132), E_STRIDE),
    (dict(ldi=-128), E_STRIDE), (dict(ld2=1 << 31), E_STRIDE), (dict(ld2=130, dt=R.REL_F32), E_STRIDE),
    (dict(rope=3), E_PRESTEP), (dict(pairing=2), E_PRESTEP), (dict(base=1.0), E_PRESTEP), (dict(base=float("nan")), E_PRESTEP),
    (dict(theta=(float("inf"),)), E_PRESTEP),
    (dict(P2=at(1) + 8), E_ALIGN), (dict(cV=at(7) + 2), E_ALIGN), (dict(slot=at(3) + 2), E_ALIGN), (dict(pos=at(4) + 3), E_ALIGN),
    (dict(P1o=at(0) + 16), E_ALIAS), (dict(P1o=at(0), ld1=520), E_ALIAS), (dict(cP2=at(1)), E_ALIAS), (dict(cV=at(6) + 1024), E_ALIAS),
    (dict(cP2=at(3)), E_ALIAS), (dict(cV=at(4)), E_ALIAS), (dict(P1o=at(2) + 16), E_ALIAS), (dict(cV=at(2) - 16), E_ALIAS),
])
def test_paged_append_rejects(kw, code):
    assert append(**kw) == code


FWD = dict(P1=at(0), ld1=512, cP2=at(1), cV=at(2), table=at(3), total=at(4), cu=at(5), tau=(1.0,) * 8, lam=0.5, Y=at(6), N=9, S=3, H=8,
           Hkv=2, d=64, n_pages=20, page=16, max_pages=8, max_new=9, dt=R.REL_BF16, ws=at(7), nb=1 << 30)


def fwd(**kw):
    m = {**FWD, **kw}
    keep, tp = fptr(m["tau"])
    return R.lib().relation_paged_fwd(*(tp if k == "tau" else m[k] for k in FWD), None)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, E_NULL) for k in ("P1", "cP2", "cV", "table", "total", "cu", "tau", "Y")],
    (dict(N=0), E_SHAPE), (dict(S=0), E_SHAPE), (dict(S=70000), E_SHAPE), (dict(H=0), E_SHAPE), (dict(H=258, tau=(1.0,) * 258), E_SHAPE),
    (dict(Hkv=0), E_SHAPE), (dict(max_new=0), E_SHAPE), (dict(Hkv=3), E_GROUP), (dict(Hkv=16), E_GROUP), (dict(dt=-1), E_DTYPE),
    (dict(d=16), E_HEADDIM), (dict(page=20), E_PAGE), (dict(n_pages=0), E_PAGE), (dict(max_pages=0), E_PAGE),
    (dict(max_pages=1 << 28), E_PAGE), (dict(n_pages=1 << 26, page=256), E_PAGE),
    (dict(max_pages=(1 << 27) - 4095), E_PAGE), (dict(n_pages=(1 << 23) - 255, page=256), E_PAGE),
    (dict(tau=(1.0,) * 7 + (0.0,)), E_TAU), (dict(tau=(float("nan"),) * 8), E_TAU), (dict(lam=float("inf")), E_LAMBDA),
    (dict(ld1=504), E_STRIDE), (dict(ld1=514), E_STRIDE), (dict(ws=None), E_WS), (dict(nb=0), E_WS),
    (dict(P1=at(0) + 4), E_ALIGN), (dict(Y=at(6) + 8), E_ALIGN), (dict(ws=at(7) + 4), E_ALIGN), (dict(table=at(3) + 2), E_ALIGN),
    (dict(cu=at(5) + 1), E_ALIGN), (dict(total=at(4) + 2), E_ALIGN),
    (dict(Y=at(0)), E_ALIAS), (dict(Y=at(1) + 64), E_ALIAS), (dict(Y=at(2)), E_ALIAS), (dict(Y=at(3)), E_ALIAS), (dict(ws=at(6)), E_ALIAS),
    (dict(ws=at(0)), E_ALIAS), (dict(ws=at(4)), E_ALIAS), (dict(ws=at(2)), E_ALIAS), (dict(Y=at(5) - 16), E_ALIAS),
])
def test_paged_fwd_rejects(kw, code):
    assert fwd(**kw) == code


def test_workspace_query():
    q = R.paged_workspace_bytes
    assert q(9, 3, 8, 2, 64) > 0
    assert fwd(nb=q(9, 3, 8, 2, 64) - 1) == E_WS
    for bad in ((0, 3, 8, 2, 64), (9, 0, 8, 2, 64), (9, 70000, 8, 2, 64), (9, 3, 0, 2, 64), (9, 3, 8, 3, 64), (9, 3, 8, 0, 64),
                (9, 3, 300, 2, 64), (9, 3, 8, 2, 72)):
        assert q(*bad) == 0, bad


def test_status_strings():
    names = [R.lib().relation_status_str(c) for c in (E_PAGE, E_GROUP, E_STRIDE)]
    assert len(set(names)) == 3 and b"unknown status" not in names


# ---- the binding -----------------------------------------------------------------

bf, i4 = torch.bfloat16, torch.int32


def z(*shape, dtype=bf):
    return torch.zeros(shape, dtype=dtype)


def b_map(**kw):
    a = dict(lens=z(3, dtype=i4), n_new=z(3, dtype=i4), block_table=z(3, 5, dtype=i4), free_pages=z(9, dtype=i4),
             n_free=z(1, dtype=i4), N=7, page_size=16, n_pages=20)
    a.update(kw)
    return lambda: R.page_map(**a)


def b_append(**kw):
    a = dict(P2=z(7, 2, 64), I=z(7, 2, 64), slot=z(7, dtype=i4), cache_P2=z(20, 2, 16, 64), cache_V=z(20, 2, 16, 64),
             P1=z(7, 8, 64), pos=z(7, dtype=i4), rope="half")
    a.update(kw)
    return lambda: R.paged_append(**a)


def b_fwd(**kw):
    a = dict(P1=z(7, 8, 64), cache_P2=z(20, 2, 16, 64), cache_V=z(20, 2, 16, 64), block_table=z(3, 5, dtype=i4),
             total=z(3, dtype=i4), cu=z(4, dtype=i4), tau=1.0)
    a.update(kw)
    return lambda: R.paged_fwd(**a)


@pytest.mark.parametrize("call,exc,words", [
    (b_map(block_table=z(15, dtype=i4)), ValueError, "block_table must be"), (b_map(free_pages=z(3, 3, dtype=i4)), ValueError, "free_pages"),
    (b_map(lens=z(4, dtype=i4)), ValueError, "lens has shape"), (b_map(n_new=z(3, dtype=torch.int64)), TypeError, "n_new has dtype"),
    (b_map(n_free=z(2, dtype=i4)), ValueError, "n_free has shape"), (b_map(out=(z(4, dtype=i4),)), ValueError, "out must be"),
    (b_map(out=tuple(z(n, dtype=i4) for n in (4, 3, 7, 8, 1))), ValueError, "pos has shape"), (b_map(), ValueError, "device tensor"),
    (b_append(cache_P2=z(20, 16, 64)), ValueError, "cache_P2 must be"), (b_append(cache_V=z(20, 2, 16, 32)), ValueError, "cache_V has shape"),
    (b_append(P2=z(7, 128)), ValueError, "P2 must be"), (b_append(I=z(7, 2, 64, dtype=torch.float32)), TypeError, "I has dtype"),
    (b_append(slot=z(6, dtype=i4)), ValueError, "slot has shape"), (b_append(P1=z(6, 8, 64)), ValueError, "P1 has shape"),
    (b_append(P1=None, out=z(7, 8, 64)), ValueError, "without P1"), (b_append(P2=z(7, 64, 2).transpose(1, 2)), ValueError, "contiguous"),
    (b_append(P1=z(7, 8, 128)[:, :, :64]), ValueError, "contiguous"), (b_append(out=z(7, 8, 32)), ValueError, "out has shape"),
    (b_append(), ValueError, "device tensor"),
    (b_fwd(P1=z(7, 512)), ValueError, "P1 must be"), (b_fwd(block_table=z(3, dtype=i4)), ValueError, "block_table must be"),
    (b_fwd(total=z(2, dtype=i4)), ValueError, "total has shape"), (b_fwd(cu=z(3, dtype=i4)), ValueError, "cu has shape"),
    (b_fwd(P1=z(7, 8, 32)), ValueError, "P1 has shape"), (b_fwd(cache_V=z(20, 2, 16, 64, dtype=torch.float32)), TypeError, "cache_V has dtype"),
    (b_fwd(out=z(7, 8, 63)), ValueError, "out has shape"), (b_fwd(workspace=z(4, dtype=torch.uint8)), ValueError, "workspace holds"),
    (b_fwd(cu=z(4, dtype=torch.int64)), TypeError, "cu has dtype"), (b_fwd(), ValueError, "device tensor"),
    (b_map(N=2**32 + 7), ValueError, "32 bits"), (b_map(page_size=2**32 + 16), ValueError, "32 bits"),
    (b_map(n_pages=2**31), ValueError, "32 bits"), (b_fwd(max_new=2**32 + 1), ValueError, "32 bits"),
])
def test_binding_checks(call, exc, words):
    with pytest.raises(exc, match=words):
        call()


# ---- the plain page map -------------------------------------------------------------

@pytest.mark.parametrize("seed", range(6))
def test_plain_page_map_keeps_every_page_once(seed):
    """Steps of random growth and release: pages in tables and free pages are always the same set, slots are distinct."""
    rng = np.random.default_rng(seed)
    S, width, page, n_pages = 9, 12, 16, 60
    table, lens = np.full((S, width), -1), np.zeros(S, int)
    free, n_free = rng.permutation(n_pages), n_pages
    for _ in range(30):
        nn = np.where(rng.random(S) < 0.1, -1, rng.integers(0, 40, S))
        m = PO.page_map(lens, nn, table, free, n_free, 300, page, n_pages)
        table, free, n_free = m["table"], m["free"], m["n_free"][0]
        lens = np.where(np.array(m["total"]) >= 0, m["total"], lens)
        used = [int(table[b, k]) for b in range(S) for k in range(-(-lens[b] // page))]
        assert sorted(used + list(free[:n_free])) == list(range(n_pages))
        slots = [s for s in m["slot"] if s >= 0]
        assert len(set(slots)) == len(slots)
        for b in range(S):
            if nn[b] > 0 and m["total"][b] >= 0:
                assert m["pos"][m["cu"][b]:m["cu"][b + 1]] == list(range(lens[b] - nn[b], lens[b]))


BOOT = """
import sys
import causal_self_exchange_amd.relation as R
R.LIB_PATH = sys.argv[1]
import pytest
sys.exit(pytest.main(['-q', '-x', '-k', 'rejects or workspace_query or status', '-p', 'no:cacheprovider', sys.argv[2]]))
"""


@pytest.mark.timeout(600)
def test_refusals_under_host_sanitizers(tmp_path):
    if shutil.which(os.environ.get("CXX_HOST", "g++")) is None:
        pytest.skip("no host C++ compiler")
    from causal_self_exchange_amd.sanitize import build_host
    lib = build_host.build(str(tmp_path))
    env = dict(os.environ, ASAN_OPTIONS="verify_asan_link_order=0:detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", BOOT, lib, os.path.abspath(__file__)], cwd=root, env=env, capture_output=True,
                       text=True, timeout=550)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])
    assert " passed" in r.stdout
