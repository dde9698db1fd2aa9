"""8-bit pages, trees and the cut to kept tokens without a GPU: refusals of the C ABI and
of the binding, and pins of the plain evaluations."""
import ctypes
import os
import shutil
import subprocess
import sys

import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from oracle import paged_ex_oracle as XO
from oracle import paged_oracle as PO

import _paged as P
import _paged_ex as X
from test_paged_abi import (APP, E_ALIAS, E_ALIGN, E_DTYPE, E_GROUP, E_HEADDIM, E_LAMBDA, E_NULL, E_PAGE, E_PRESTEP, E_SHAPE,
                            E_STRIDE, E_TAU, E_WS, FWD, at, fptr)

APP8 = {k: v for k, v in APP.items() if k != "dt"}
APP8 = {**dict(list(APP8.items())[:list(APP8).index("cV") + 1]), "scale": at(8),
        **dict(list(APP8.items())[list(APP8).index("cV") + 1:])}


def append(**kw):
    m = {**APP8, **kw}
    th = None if m["theta"] is None else (ctypes.c_double * len(m["theta"]))(*m["theta"])
    return R.lib().relation_paged_append_q8(*(th if k == "theta" else m[k] for k in APP8), None)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, E_NULL) for k in ("P1", "P2", "I", "slot", "pos", "P1o", "cP2", "cV", "scale")],
    (dict(N=0), E_SHAPE), (dict(Hkv=257), E_SHAPE), (dict(Hkv=1, theta=(0.1,)), E_SHAPE), (dict(d=96), E_HEADDIM),
    (dict(page=17), E_PAGE), (dict(n_pages=1 << 30), E_PAGE), (dict(ld1=511), E_STRIDE), (dict(ld2=132), E_STRIDE),
    (dict(rope=3), E_PRESTEP), (dict(theta=(float("nan"),)), E_PRESTEP), (dict(cP2=at(6) + 8), E_ALIGN), (dict(scale=at(8) + 4), E_ALIGN),
    (dict(scale=at(6) + 20 * 2 * 16 * 64 - 16), E_ALIAS), (dict(scale=at(1)), E_ALIAS), (dict(scale=at(5) - 16), E_ALIAS),
    (dict(cV=at(6) + 1024), E_ALIAS), (dict(P1o=at(0) + 16), E_ALIAS),
])
def test_paged_append_q8_rejects(kw, code):
    assert append(**kw) == code


EX = {}
for _k, _v in FWD.items():
    EX[_k] = _v
    if _k == "cV":
        EX["scale"] = None
    if _k == "cu":
        EX.update(tree=at(8), words=1)
    if _k == "dt":
        pass


def fwd(**kw):
    m = {**EX, **kw}
    keep, tp = fptr(m["tau"])
    return R.lib().relation_paged_fwd_ex(*(tp if k == "tau" else m[k] for k in EX), None)


Q8 = dict(dt=R.REL_E4M3, scale=at(9))


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, E_NULL) for k in ("P1", "cP2", "cV", "table", "total", "cu", "tau", "Y")],
    (dict(dt=R.REL_E4M3), E_NULL), (dict(scale=at(9)), E_DTYPE), (dict(scale=at(9), dt=R.REL_F32, ld1=512), E_DTYPE), (dict(dt=3), E_DTYPE),
    (dict(words=0), E_SHAPE), (dict(words=33), E_SHAPE), (dict(words=-1), E_SHAPE), (dict(tree=None), E_SHAPE), (dict(max_new=0), E_SHAPE),
    (dict(H=7), E_GROUP), (dict(d=40), E_HEADDIM), (dict(page=8), E_PAGE), (dict(max_pages=1 << 28), E_PAGE), (dict(tau=(0.0,) * 8), E_TAU),
    (dict(lam=float("inf")), E_LAMBDA), (dict(ld1=508), E_STRIDE), (dict(nb=100), E_WS), (dict(ws=None), E_WS),
    (dict(tree=at(8) + 2), E_ALIGN), (dict(**{**Q8, "scale": at(9) + 8}), E_ALIGN), (dict(Y=at(8)), E_ALIAS), (dict(Y=at(8) + 16), E_ALIAS),
    (dict(**{**Q8, "scale": at(6)}), E_ALIAS), (dict(**Q8, ws=at(9) + 16), E_ALIAS), (dict(ws=at(8)), E_ALIAS), (dict(**Q8, Y=at(1)), E_ALIAS),
])
def test_paged_fwd_ex_rejects(kw, code):
    assert fwd(**kw) == code


@pytest.mark.parametrize("call", ["paged_fwd", "paged_append", "fwd", "linear"])
def test_8bit_is_a_page_type_only(call):
    t = np.ones(8, np.float32)
    tp = fptr(t)[1]
    lib, d = R.lib(), R.REL_E4M3
    if call == "paged_fwd":
        m = {**FWD, "dt": d}
        st = lib.relation_paged_fwd(*(tp if k == "tau" else m[k] for k in FWD), None)
    elif call == "paged_append":
        m = {**APP, "dt": d, "theta": None}
        st = lib.relation_paged_append(*(m[k] for k in APP), None)
    elif call == "fwd":
        st = lib.relation_fwd(at(0), at(1), at(2), tp, at(3), 1, 8, 64, 64, d, None)
    else:
        st = lib.relation_linear_fwd(at(0), at(1), at(2), at(3), tp, at(4), None, 1, 8, 64, 64, d, at(5), 1 << 30, None)
    assert st == E_DTYPE


PLAN = dict(parent=at(0), total=at(1), cu=at(2), tree=at(3), pos=at(4), N=40, S=5, words=2)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, E_NULL) for k in list(PLAN)[:5]], (dict(N=0), E_SHAPE), (dict(S=0), E_SHAPE), (dict(S=65536), E_SHAPE),
    (dict(words=0), E_SHAPE), (dict(words=33), E_SHAPE), (dict(parent=at(0) + 1), E_ALIGN), (dict(tree=at(3) + 2), E_ALIGN),
    (dict(pos=at(3) + 316), E_ALIAS), (dict(pos=at(0)), E_ALIAS), (dict(tree=at(2) + 20), E_ALIAS), (dict(tree=at(1) - 316), E_ALIAS),
])
def test_tree_plan_rejects(kw, code):
    assert R.lib().relation_tree_plan(*{**PLAN, **kw}.values(), None) == code


KEEP = dict(cP2=at(0), cV=at(1), scale=None, table=at(2), total=at(3), cu=at(4), keep=at(5), n_keep=at(6), len=at(7), free=at(8),
            n_free=at(9), n_free_out=at(10), N=40, S=5, F=9, Hkv=2, d=64, n_pages=20, page=16, max_pages=8, dt=R.REL_BF16)


@pytest.mark.parametrize("kw,code", [
    *[({k: None}, E_NULL) for k in KEEP if k != "scale" and KEEP[k] is not None and KEEP[k] >= at(0)],
    (dict(dt=R.REL_E4M3), E_NULL), (dict(scale=at(11)), E_DTYPE), (dict(dt=4), E_DTYPE), (dict(N=0), E_SHAPE), (dict(S=0), E_SHAPE),
    (dict(F=0), E_SHAPE), (dict(Hkv=0), E_SHAPE), (dict(Hkv=257), E_SHAPE), (dict(d=33), E_HEADDIM), (dict(page=15), E_PAGE),
    (dict(n_pages=0), E_PAGE), (dict(max_pages=1 << 27), E_PAGE), (dict(cP2=at(0) + 4), E_ALIGN), (dict(len=at(7) + 3), E_ALIGN),
    (dict(dt=R.REL_E4M3, scale=at(11) + 8), E_ALIGN), (dict(cV=at(0) + 16), E_ALIAS), (dict(len=at(3)), E_ALIAS), (dict(free=at(2) + 156), E_ALIAS),
    (dict(n_free_out=at(8)), E_ALIAS), (dict(keep=at(7) + 16), E_ALIAS), (dict(dt=R.REL_E4M3, scale=at(1) + 16), E_ALIAS),
    (dict(n_free=at(7)), E_ALIAS),
])
def test_paged_keep_rejects(kw, code):
    assert R.lib().relation_paged_keep(*{**KEEP, **kw}.values(), None) == code


# ---- binding -------------------------------------------------------------------------

def case(dt="bf16"):
    m = P.make(dt, 4, 2, 32, 16, [(5, 3), (20, 2)], 1)
    m["tree"] = torch.zeros((5, 1), dtype=torch.int32)
    return m


def call_fwd(m, **kw):
    return R.paged_fwd(m["P1"], m["cP2"], m["cV"], m["table"], m["total"], m["cu"], 1.0, **kw)


def test_binding_checks():
    m = case()
    m8 = X.as_8bit(m)
    i = lambda n: torch.zeros(n, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="device tensor"):
        call_fwd(m8, scale=m8["scale"], tree=m["tree"])
    with pytest.raises(TypeError, match="scale must be"):
        call_fwd(m8)
    with pytest.raises(TypeError, match="scale belongs"):
        call_fwd(m, scale=m8["scale"])
    with pytest.raises(TypeError, match="dtype"):
        call_fwd(m8, scale=m8["scale"].view(torch.uint8))
    with pytest.raises(ValueError, match="shape"):
        call_fwd(m8, scale=m8["scale"][:, :, :1])
    with pytest.raises(TypeError, match="P1 has dtype"):
        call_fwd({**m8, "P1": m["P1"].float()}, scale=m8["scale"])
    with pytest.raises(ValueError, match="tree"):
        call_fwd(m, tree=m["tree"][:, 0])
    with pytest.raises(ValueError, match="words"):
        call_fwd(m, tree=torch.zeros((5, 33), dtype=torch.int32))
    with pytest.raises(ValueError, match="shape"):
        call_fwd(m, tree=torch.zeros((4, 1), dtype=torch.int32))
    with pytest.raises(TypeError, match="dtype"):
        call_fwd(m, tree=m["tree"].long())
    tok = torch.zeros((5, 2, 32), dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="scale must be"):
        R.paged_append(tok, tok, i(5), m8["cP2"], m8["cV"])
    with pytest.raises(TypeError, match="P2 has dtype"):
        R.paged_append(tok.float(), tok, i(5), m8["cP2"], m8["cV"], scale=m8["scale"])
    with pytest.raises(ValueError, match="device tensor"):
        R.paged_append(tok, tok, i(5), m8["cP2"], m8["cV"], scale=m8["scale"])
    with pytest.raises(ValueError, match="words"):
        R.tree_plan(i(5), i(2), i(3), 0)
    with pytest.raises(ValueError, match="1-d"):
        R.tree_plan(m["tree"], i(2), i(3), 1)
    with pytest.raises(ValueError, match="shape"):
        R.tree_plan(i(5), i(2), i(4), 1)
    with pytest.raises(ValueError, match="out must"):
        R.tree_plan(i(5), i(2), i(3), 1, out=(m["tree"],))
    with pytest.raises(ValueError, match="device tensor"):
        R.tree_plan(i(5), i(2), i(3), 1)
    keep = (m["table"], m["total"], m["cu"], i(5), i(2), i(2), i(4), i(1))
    with pytest.raises(ValueError, match="device tensor"):
        R.paged_keep(m["cP2"], m["cV"], *keep)
    with pytest.raises(TypeError, match="scale must be"):
        R.paged_keep(m8["cP2"], m8["cV"], *keep)
    with pytest.raises(TypeError, match="scale belongs"):
        R.paged_keep(m["cP2"], m["cV"], *keep, scale=m8["scale"])
    with pytest.raises(ValueError, match="shape"):
        R.paged_keep(m["cP2"], m["cV"], *keep[:5], i(3), *keep[6:])
    with pytest.raises(TypeError, match="unsupported dtype"):
        R.paged_keep(m["cP2"].half(), m["cV"].half(), *keep)


def test_host_code_under_sanitizers(tmp_path):
    """The refusals above against the host code built with AddressSanitizer and UndefinedBehaviorSanitizer."""
    if os.environ.get("REL_SANITIZED_RUN") or shutil.which(os.environ.get("CXX_HOST", "g++")) is None:
        pytest.skip("no host C++ compiler, or the run inside")
    from causal_self_exchange_amd.sanitize import build_host
    from test_abi_sanitized import BOOT, ROOT
    lib = build_host.build(str(tmp_path))
    env = dict(os.environ, REL_SANITIZED_RUN="1", ASAN_OPTIONS="verify_asan_link_order=0:detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-c", BOOT, lib, os.path.join(ROOT, "tests", "test_paged_ex_abi.py")], cwd=ROOT, env=env,
                       capture_output=True, text=True, timeout=550)
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-3000:])


# ---- pins of the plain evaluations ---------------------------------------------------

def test_quantise_pins():
    # All 8-bit values stand for themselves; the rounding is the nearest of them, ties to the even code.
    codes = torch.arange(256, dtype=torch.uint8)
    vals = codes.view(torch.float8_e4m3fn).double().numpy()
    fine = ~np.isnan(vals)
    np.testing.assert_array_equal(XO.e4m3_round(vals[fine]), vals[fine])
    x = np.random.default_rng(0).uniform(-448, 448, 4000)
    x = np.concatenate([x, x * 2.0**-9, (vals[:126] + vals[1:127]) / 2, [448.0, -448.0, 0.0, 2.0**-10, 3 * 2.0**-10]])
    grid = np.sort(vals[fine])
    got = XO.e4m3_round(x)
    np.testing.assert_array_equal(np.abs(got - x), np.abs(grid[None] - x[:, None]).min(1))
    np.testing.assert_array_equal(got, torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())
    # Scales: the least power of two that leaves no value above 448.
    rows = np.array([[0.0, 0.0], [448.0, 1.0], [448.001, 0.0], [-896.0, 3.0], [1e-40, 0.0], [3e38, 1.0], [np.inf, 2.0], [np.nan, -7.0], [0.875, 0.0]])
    np.testing.assert_array_equal(XO.scale_exponents(rows), [-100, 0, 1, 1, -100, 119, -7, -6, -9])
    q, _ = XO.quantise(rows)
    assert np.isnan(q[6, 0]) and np.isnan(q[7, 0]) and q[6, 1] == 256.0 and q[5, 0] == 448.0 and q[1, 0] == 448.0 and q[8, 0] == 448.0


def test_tree_plan_pins():
    # 0 <- 1 <- 2, 0 <- 3, root 4 <- 5; a parent that is not before its token makes a root.
    tree, pos = XO.tree_plan([-1, 0, 1, 0, 7, 4, 0, 9], [16, 12], [0, 6, 8], 1, np.full((8, 1), 9), np.full(8, 9))
    assert tree[:, 0].tolist() == [0, 1, 3, 1, 0, 16, 0, 0] and pos.tolist() == [10, 11, 12, 11, 10, 11, 10, 10]
    tree, pos = XO.tree_plan([-1] + list(range(39)) + [-1, -1], [50], [0, 40], 1, np.full((42, 1), 9), np.full(42, 9))
    assert (tree == 9).all() and pos.tolist() == list(range(10, 50)) + [-1, -1]
    tree, pos = XO.tree_plan([-1] + list(range(39)), [50], [0, 40], 2, np.zeros((40, 2)), np.zeros(40))
    assert tree[39].tolist() == [-1, 127] and tree[32].tolist() == [-1, 0] and pos.tolist() == list(range(10, 50))


def test_tree_rows_equal_their_path_alone():
    """A token of a tree equals the last token of its path in a request that holds the cached rows and that path; a
    tree that is a chain, and no tree, equal the forward of the chunk."""
    m = P.make("f32", 4, 2, 32, 16, [(21, 9), (0, 6)], 3)
    rng = np.random.default_rng(3)
    parent = X.random_parents([9, 6], rng)
    a = {k: P.f64(m[k]) for k in ("P1", "cP2", "cV")}
    tb, total, cu = m["table"].numpy(), m["total"].numpy(), m["cu"].numpy()
    tree = X.bits_of(parent, cu, total, 1, m["N"], junk=rng)
    Y, _ = XO.paged_fwd(a["P1"], a["cP2"], a["cV"], tb, total, cu, m["tau"], 0.5, np.zeros(a["P1"].shape), 9, tree=tree)
    for b, (c, n) in enumerate([(21, 9), (0, 6)]):
        k, v = (PO.gather(a[x], tb[b], c + n, len(a[x])) for x in ("cP2", "cV"))
        for i in range(n):
            rows = list(range(c)) + [c + x for x in sorted(XO.ancestors(parent[cu[b]:cu[b + 1]], i))] + [c + i]
            one = lambda x: x[:, rows][None].transpose(0, 1, 2, 3)  # noqa: E731
            page = len(rows)
            y = PO.paged_fwd(a["P1"][cu[b] + i][None], one(k), one(v), np.zeros((1, 1), int), [page], [0, 1], m["tau"], 0.5,
                             np.zeros((1, 4, 32)), 1)
            np.testing.assert_allclose(Y[cu[b] + i], y[0], rtol=1e-12, atol=1e-14)
    chain = X.bits_of(np.array([k - 1 for n in (9, 6) for k in range(n)]), cu, total, 1, m["N"])
    want = PO.paged_fwd(a["P1"], a["cP2"], a["cV"], tb, total, cu, m["tau"], 0.5, np.zeros(a["P1"].shape), 9)
    for t in (chain, None):
        Y, _ = XO.paged_fwd(a["P1"], a["cP2"], a["cV"], tb, total, cu, m["tau"], 0.5, np.zeros(a["P1"].shape), 9, tree=t)
        np.testing.assert_allclose(Y, want, rtol=1e-12, atol=1e-14)


def test_keep_pins():
    c = np.arange(4 * 1 * 4 * 1.0).reshape(4, 1, 4, 1)                       # pages of four rows
    table = np.array([[2, 0, 3], [1, 9, 9]])
    r = XO.paged_keep([c], table, [11, 2], [0, 6, 8], [1, 3, 4, 0, 0, 0, 0, 1], [3, 3], [5, 0], [-1] * 3, 1, 4)
    # Request 0: rows 5 .. 10 are new; 6, 8, 9 move to 5, 6, 7, and the third page goes back. Request 1: 3 of 2, keeps none.
    assert r["caches"][0][0, 0, :, 0].tolist() == [0, 2, 12, 13] and r["caches"][0][3, 0, :2, 0].tolist() == [12, 13]
    assert r["lens"] == [8, 0] and r["free"] == [-1, 3, 1] and r["n_free"] == 3
    r = XO.paged_keep([c], table, [11, 2], [0, 6, 8], [3, 1, 4, 0, 0, 0, 1, 0], [2, 1], [5, 0], [-1] * 2, 0, 4)
    assert r["lens"] == [5, 1] and r["free"] == [3, -1] and r["n_free"] == 1 and r["caches"][0][1, 0, 0, 0] == 5
