"""8-bit pages of the paged Relation Cache, trees of drafted tokens and the cut to the kept ones on the GPU, against plain
evaluations (oracle/paged_ex_oracle.py), alone and together."""
import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from causal_self_exchange_amd import workloads as W
from oracle import paged_ex_oracle as XO
from oracle import prestep_oracle as PR

import _paged as P
import _paged_ex as X
import _paged_rows as PW

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def scales(n_pages, Hkv, page, fill=200):
    return torch.full((n_pages, Hkv, 2, page), fill, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)


def exps(scale):
    return scale.view(torch.uint8).cpu().numpy().astype(np.int64) - 127


# ---- append -------------------------------------------------------------------------

def check_rows(got, k, x, slack):
    """Stored values got (e4m3, fp64) and exponents k of rows whose fp64 values are x, known to within slack: k is that of
    a maximum within slack, and each value is off by at most half a step of e4m3 (2^-4 of it, 2^-10 below 2^-6) and slack."""
    lo, hi = (XO.scale_exponents(np.maximum(np.abs(x) + s, 0.0)) for s in (-slack, slack))
    assert np.all((k >= lo) & (k <= hi))
    step = 2.0**k[..., None]
    half = np.maximum(2.0**-4 * np.abs(x), 2.0**-10 * step)
    assert np.all(np.abs(got * step - x) <= half + 2 * slack), float(np.max(np.abs(got * step - x) - half))


@pytest.mark.parametrize("N,H,Hkv,d,page,rope,mix,pairing,fused", [
    (1, 8, 8, 64, 16, "interleaved", True, "A", True), (37, 12, 4, 128, 64, "half", True, "B", True),
    (33, 6, 2, 80, 32, "interleaved", True, "B", False), (5, 3, 3, 48, 16, "half", False, "A", True),
    (130, 5, 1, 32, 256, "none", False, "A", False), (64, 16, 16, 80, 128, "half", True, "A", False),
    (21, 4, 4, 48, 16, "interleaved", True, "A", True), (9, 2, 2, 32, 16, "half", True, "B", True),
    (700, 32, 8, 128, 16, "interleaved", True, "B", True), (50, 0, 256, 64, 16, "half", True, "A", True),
])
def test_paged_append_q8(N, H, Hkv, d, page, rope, mix, pairing, fused):
    rng = np.random.default_rng(N + d)
    n_pages = -(-N // page) + 3
    rows = rng.standard_normal((N, H + 2 * Hkv, d)) * 2.0**rng.integers(-20, 20, (N, H + 2 * Hkv, 1))
    x = torch.from_numpy(rows).to(torch.bfloat16).to(DEV)
    P1, P2, I = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if not fused:
        P1, P2, I = P1.contiguous(), P2.contiguous(), I.contiguous()
    slot = rng.permutation(n_pages * page)[:N].astype(np.int32)
    if N > 4:
        slot[rng.integers(0, N, 3)] = [-1, -9, n_pages * page]
    pos = rng.integers(0, 70000, N).astype(np.int32)
    theta = rng.uniform(-3, 3, Hkv // 2).astype(np.float32) if mix else None
    cP2, cV = (torch.full((n_pages, Hkv, page, d), 5.0, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
    sc = scales(n_pages, Hkv, page)
    out = torch.full((N, H, d), 7.0, dtype=torch.bfloat16, device=DEV) if H else None
    got = R.paged_append(P2, I, i32(slot), cP2, cV, P1=P1 if H else None, pos=i32(pos), rope=rope, theta=theta, pairing=pairing,
                         out=out, scale=sc)
    torch.cuda.synchronize()
    assert got is out
    live = (slot >= 0) & (slot < n_pages * page)
    k = PR.rope(P.f64(P2).transpose(1, 0, 2), pos, 1e4, rope).transpose(1, 0, 2)
    v = P.f64(I) if theta is None else PR.givens_mix(P.f64(I)[:, :, None], theta, pairing)[:, :, 0]
    pages, offs = slot[live] // page, slot[live] % page
    e = exps(sc)
    # fp32 roundings of a rotation, its sine and cosine, or of a mixing: a few 2^-24 of the magnitudes that meet. 2^-21 of
    # the largest element of the row, or of the two rows of a pair of heads, is more than all of them.
    def slack(t):
        return 2.0**-21 * np.abs(t).max(-1, keepdims=True)
    top = slack(P.f64(I))
    mate = np.arange(Hkv) ^ 1 if pairing == "A" else (np.arange(Hkv) + np.where(np.arange(Hkv) % 2, 1, -1)) % Hkv
    mixed = np.maximum(top, top[:, mate]) if mix else 0.0 * top
    check_rows(P.f64(cP2)[pages, :, offs], e[pages, :, 0, offs], k[live], slack(P.f64(P2))[live])
    check_rows(P.f64(cV)[pages, :, offs], e[pages, :, 1, offs], v[live], mixed[live])
    if H:
        a = PR.rope(P.f64(P1).transpose(1, 0, 2), pos, 1e4, rope).transpose(1, 0, 2)
        assert np.all(np.abs(P.f64(out) - a)[live] <= (2.0**-8 * np.abs(a) + slack(P.f64(P1)))[live])
        assert np.all(P.f64(out)[~live] == 7.0)
    rest = np.ones((n_pages, page), dtype=bool)
    rest[pages, offs] = False
    for c in (cP2, cV):
        assert np.all(P.f64(c).transpose(0, 2, 1, 3)[rest] == 5.0)
    assert np.all(e.transpose(0, 3, 1, 2)[rest] == 200 - 127)


def test_paged_append_q8_equals_the_quantised_append():
    """Without rotation or mixing the rows are the inputs: bit for bit the plain quantisation, at zeros, the borders of a
    scale, the smallest and largest numbers, infinities and NaN."""
    d, Hkv = 64, 2
    rng = np.random.default_rng(0)
    rows = [np.zeros(d), np.full(d, 448.0), np.full(d, 450.0), np.full(d, -896.0), np.full(d, 1e-39), np.full(d, 3.3e38),
            np.full(d, -1e-30), np.full(d, 2.0**-110), np.full(d, 2.0**-91), np.full(d, 448 * 2.0**119)]
    rows += [rng.standard_normal(d) * 2.0**k for k in range(-126, 126, 6)]
    rows += [np.where(rng.random(d) < 0.2, bad, rng.standard_normal(d) * 30) for bad in (np.inf, -np.inf, np.nan)] + [np.full(d, np.nan)]
    x = torch.from_numpy(np.stack(rows)).to(torch.bfloat16)
    x = torch.stack([x, x.flip(0)], 1)
    N = x.shape[0]
    c = [torch.zeros((8, Hkv, 16, d), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    sc = scales(8, Hkv, 16)
    slot = np.arange(N)
    R.paged_append(x.to(DEV), x.flip(2).contiguous().to(DEV), i32(slot), *c, scale=sc)
    torch.cuda.synchronize()
    for part, w in ((0, P.f64(x)), (1, P.f64(x.flip(2)))):
        q, k = XO.quantise(w)
        np.testing.assert_array_equal(exps(sc)[slot // 16, :, part, slot % 16], k)
        np.testing.assert_array_equal(P.f64(c[part])[slot // 16, :, slot % 16], q)


def test_paged_append_q8_mixes_by_fp64_angles():
    """Every stored value is one of the nearest to a number within 2^-23 of the exact one (fp32 sums of exact products,
    rounded twice), and the nearest to the exact one where fp32 leaves two."""
    N, Hkv, d, page = 2048, 8, 128, 16
    rng = np.random.default_rng(5)
    theta = rng.uniform(-3, 3, Hkv // 2)
    x = torch.from_numpy(rng.standard_normal((N, Hkv, d))).to(torch.bfloat16)
    c = [torch.zeros((N // page, Hkv, page, d), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    sc = scales(N // page, Hkv, page)
    R.paged_append(x.to(DEV), x.to(DEV), i32(np.arange(N)), *c, theta=list(theta), scale=sc)
    torch.cuda.synchronize()
    k = exps(sc)[:, :, 1].transpose(0, 2, 1).reshape(N, Hkv, 1)
    q = P.f64(c[1]).transpose(0, 2, 1, 3).reshape(N, Hkv, d)
    a, b = P.f64(x)[:, 0::2], P.f64(x)[:, 1::2]
    cs, sn = np.cos(theta)[:, None], np.sin(theta)[:, None]
    y = np.stack([cs * a - sn * b, sn * a + cs * b], 2).reshape(N, Hkv, d) / 2.0**k
    top = np.abs(y).max(-1)
    assert np.all(top <= 448 * (1 + 2.0**-22)) and np.all(top >= 224 * (1 - 2.0**-22))
    half = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0**-40))), -6) - 4)
    # Where e4m3 has four bits, the nearest: the factors are within 2^-39, their products and sum in fp64.
    mag = np.repeat(np.abs(a) + np.abs(b), 2, axis=1) / 2.0**k
    off = np.where(np.abs(y) >= 2.0**-6, mag * 2.0**-38, np.abs(y) * 2.0**-23)
    assert np.all(np.abs(q - y) <= half + off)


@pytest.mark.parametrize("rope", ["interleaved", "half"])
def test_paged_append_q8_rotates_to_the_nearest(rope):
    """As above, of P2. The angles are below 2^15, so those in fp64 (and the frequencies' last bit) are within 2^-37."""
    N, Hkv, d, page = 2048, 8, 128, 16
    rng = np.random.default_rng(6)
    x = torch.from_numpy(rng.standard_normal((N, Hkv, d))).to(torch.bfloat16)
    pos = rng.integers(0, 20000, N)
    c = [torch.zeros((N // page, Hkv, page, d), device=DEV).to(torch.float8_e4m3fn) for _ in range(2)]
    sc = scales(N // page, Hkv, page)
    R.paged_append(x.to(DEV), x.to(DEV), i32(np.arange(N)), *c, pos=i32(pos), rope=rope, scale=sc)
    torch.cuda.synchronize()
    k = exps(sc)[:, :, 0].transpose(0, 2, 1).reshape(N, Hkv, 1)
    q = P.f64(c[0]).transpose(0, 2, 1, 3).reshape(N, Hkv, d)
    ang = pos[:, None, None] * 10000.0 ** (-2.0 * np.arange(d // 2) / d)
    half = rope == "half"
    a, b = (P.f64(x)[..., :d // 2], P.f64(x)[..., d // 2:]) if half else (P.f64(x)[..., 0::2], P.f64(x)[..., 1::2])
    both = [np.cos(ang) * a - np.sin(ang) * b, np.sin(ang) * a + np.cos(ang) * b]
    mag = np.abs(a) + np.abs(b)
    y, mag = (np.concatenate(both, -1), np.concatenate([mag, mag], -1)) if half else (
        np.stack(both, -1).reshape(N, Hkv, d), np.repeat(mag, 2, -1))
    y, mag = y / 2.0**k, mag / 2.0**k
    step = 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(np.abs(y), 2.0**-40))), -6) - 4)
    # Below four bits, fp32: two roundings of the sum, and those of the split factors (2^-39 each).
    off = np.where(np.abs(y) >= 2.0**-6, 0.0, np.abs(y) * 2.0**-22) + mag * 2.0**-36
    assert np.all(np.abs(q - y) <= step + off)


# ---- plan ----------------------------------------------------------------------------

@pytest.mark.parametrize("S,n_hi,words,pad,seed", [(1, 1, 1, 0, 1), (3, 12, 1, 0, 2), (40, 32, 1, 7, 3), (17, 64, 2, 300, 4),
                                                    (9, 70, 3, 1, 5), (300, 6, 1, 0, 6), (4, 1024, 32, 3, 7), (6, 100, 2, 5, 8)])
def test_tree_plan(S, n_hi, words, pad, seed):
    rng = np.random.default_rng(seed)
    nn = rng.integers(0, n_hi + 1, S)
    nn[0] = n_hi
    cu = np.concatenate([[0], np.cumsum(nn)]).astype(np.int32)
    N = int(cu[-1]) + pad
    total = nn + rng.integers(0, 5000, S)
    if S > 4:
        total[1], total[3] = -1, nn[3] - 1
    parent = np.concatenate([X.random_parents(nn, rng), rng.integers(-9, 9, pad)])
    wild = rng.random(N) < 0.05
    parent[wild] = rng.integers(-2**31, 2**31 - 1, int(wild.sum()))
    if seed == 7:
        parent[:n_hi] = np.arange(-1, n_hi - 1)              # one path of 1,024
    tree, pos = torch.full((N, words), 77, dtype=torch.int32, device=DEV), torch.full((N,), 77, dtype=torch.int32, device=DEV)
    want = XO.tree_plan(parent, total, cu, words, tree.cpu().numpy(), pos.cpu().numpy())
    got = R.tree_plan(i32(parent), i32(total), i32(cu), words, out=(tree, pos))
    torch.cuda.synchronize()
    assert got[0] is tree
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)
    # Offsets that are not valid are skipped.
    bad = cu.copy()
    bad[0] = -3
    if S > 2:
        bad[2] = N + 5
    want = XO.tree_plan(parent, total, bad, words, np.full((N, words), 5), np.full(N, 5))
    tree.fill_(5)
    pos.fill_(5)
    R.tree_plan(i32(parent), i32(total), i32(bad), words, out=(tree, pos))
    torch.cuda.synchronize()
    for g, w in zip((tree, pos), want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


# ---- forward ---------------------------------------------------------------------------

def run_ex(m, lam, ws=None, fill=3.0, max_new=None):
    d = X.to_device(m)
    Y = torch.full(tuple(m["P1"].shape), fill, dtype=m["P1"].dtype, device=DEV)
    R.paged_fwd(d["P1"], d["cP2"], d["cV"], d["table"], d["total"], d["cu"], m["tau"], lam,
                max_new=m["max_new"] if max_new is None else max_new, out=Y, workspace=ws, scale=d.get("scale"), tree=d.get("tree"))
    torch.cuda.synchronize()
    return Y


def many_rows(m, max_new=None):
    """Whether requests may have more than 64 rows to a cached head, in a batch of 8-bit pages or of 16-bit trees whose
    workspace has the part for query tiles."""
    H, Hkv = m["P1"].shape[1], m["cP2"].shape[1]
    most = min(m["max_new"] if max_new is None else max_new, m["N"])
    return most * (H // Hkv) > 64 and most * min(H // Hkv, 8) >= 65 and (m.get("tree") is not None or "k64" in m)


def tile_rows(m, max_new=None):
    """The most rows to a cached head of requests that stay with the scan: by the batch's rows times the most keys that its
    table admits (and 500), and by how like its requests are."""
    H, Hkv = m["P1"].shape[1], m["cP2"].shape[1]
    most = min(m["max_new"] if max_new is None else max_new, m["N"])
    if not many_rows(m, max_new) or H // Hkv > 128 or m["N"] * H * (m["table"].shape[1] * m["cP2"].shape[2] + 500) < 12000000:
        return 2**31
    if 4 * m["N"] >= m["total"].shape[0] * most:
        return 0
    return 64 if most * (H // Hkv) >= 512 else 2**31


def widened(m):
    """The same batch with a table wide enough for query tiles."""
    cols = -(-12000000 // (m["N"] * m["P1"].shape[1] * m["cP2"].shape[2])) + 1
    return dict(m, table=torch.cat([m["table"], torch.full((m["table"].shape[0], cols), P.BAD, dtype=torch.int32)], 1))


def limit(m, ref, spread, k, du=None, max_new=None):
    """Bound of a batch's rows; on query tiles the weights are rounded to bf16 once (relation.h), elsewhere kept."""
    if m["P1"].dtype == torch.float32:
        return P.bound(ref, spread, "f32", 1e-6 if du is None else du)
    at_most, e_max = PW.evidence_error(m["P1"], torch.from_numpy(k))
    kept = PW.weights_bound(ref, spread, int(m["total"].max()), at_most, e_max)
    least = tile_rows(m, max_new)
    if least == 2**31:
        return kept
    G, tiled = m["P1"].shape[1] // m["cP2"].shape[1], np.zeros((m["N"], 1, 1), bool)
    for a, b in zip(m["cu"].tolist(), m["cu"].tolist()[1:]):
        if 0 <= a < b <= m["N"] and (b - a) * G > least:
            tiled[a:b] = True
    return np.where(tiled, P.bound(ref, spread, "bf16", at_most + 8 * e_max * 2.0**-24), kept)


def check_ex(m, lam, fill=3.0, max_new=None, du=None):
    """A batch against the plain evaluation; where it has the rows for query tiles, in a wide table too."""
    y0 = np.full(tuple(m["P1"].shape), fill)
    k, v = (m["k64"], m["v64"]) if "k64" in m else (np.nan_to_num(P.f64(m[c])) for c in ("cP2", "cV"))
    tree = m["tree"].numpy() if m.get("tree") is not None else None
    ref, spread = XO.paged_fwd(P.f64(m["P1"]), k, v, m["table"].numpy(), m["total"].numpy(), m["cu"].numpy(), m["tau"], lam, y0,
                               m["max_new"] if max_new is None else max_new, tree=tree)
    for b in [m] + ([widened(m)] if many_rows(m, max_new) and m["P1"].dtype == torch.bfloat16 else []):
        Y = run_ex(b, lam, fill=fill, max_new=max_new)
        lim = np.where(spread > 0, limit(b, ref, spread, k, du, max_new), 0.0)     # rows nobody writes stay exactly
        err = np.abs(P.f64(Y) - ref)
        worst = np.unravel_index(np.argmax(err - lim), err.shape)
        assert np.all(err <= lim), (tile_rows(b, max_new), worst, err[worst], lim[worst], ref[worst])
    return Y


def make8(H, Hkv, d, page, reqs, seed, spread=3, **kw):
    return X.as_8bit(P.make("bf16", H, Hkv, d, page, reqs, seed, **kw), np.random.default_rng(seed + 1), spread)


def with_trees(m, reqs, words, seed, **kw):
    rng = np.random.default_rng(seed)
    parent = X.random_parents([n for _, n in reqs], rng, **kw)
    m["tree"] = torch.from_numpy(X.bits_of(parent, m["cu"].numpy(), m["total"].numpy(), words, m["N"], junk=rng))
    m["parent"] = parent
    return m


DECODE = [(0, 1), (1, 1), (15, 1), (16, 1), (17, 1), (31, 1), (63, 1), (64, 1), (65, 1), (255, 1), (700, 1)]
RAGGED = [(0, 1), (0, 2), (3, 5), (60, 9), (0, 33), (129, 7), (31, 32), (500, 1), (1, 70)]
CHUNKS = [(0, 130), (77, 300), (1000, 57), (64, 64)]
TREES = [(0, 1), (0, 2), (3, 5), (60, 9), (0, 33), (129, 7), (31, 32), (500, 1), (1, 64), (16, 16), (700, 50), (13, 3)]


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (6, 2), (7, 1), (24, 1)])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 64), (80, 32), (48, 16), (32, 256)])
def test_fwd_8bit_decode(d, page, H, Hkv):
    check_ex(make8(H, Hkv, d, page, DECODE, seed=d + H, stride_pad=16), 0.5)


@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (5, 1)])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 32), (80, 16), (48, 64), (32, 128)])
def test_fwd_8bit_ragged(d, page, H, Hkv):
    check_ex(make8(H, Hkv, d, page, RAGGED, seed=d + H, pad_rows=3), 0.25)


@pytest.mark.parametrize("d,page,H,Hkv", [(128, 16, 4, 2), (64, 64, 2, 2), (80, 32, 3, 1), (48, 16, 2, 1), (32, 128, 2, 2)])
def test_fwd_8bit_chunks(d, page, H, Hkv):
    check_ex(make8(H, Hkv, d, page, CHUNKS, seed=d + H, stride_pad=32, pad_rows=5), 1.0)


@pytest.mark.parametrize("d,H,Hkv", [(128, 4, 2), (64, 2, 1), (80, 1, 1)])
def test_fwd_8bit_long_history(d, H, Hkv):
    check_ex(make8(H, Hkv, d, 16, [(20001, 1), (9000, 3), (5, 1), (8190, 18)], seed=d), 0.5)


@pytest.mark.parametrize("S,H,Hkv,d,ctx_hi,new_hi,words", [(128, 4, 2, 64, 200, 1, 0), (129, 4, 2, 64, 200, 3, 1), (300, 2, 1, 128, 90, 4, 1),
                                                           (700, 1, 1, 32, 40, 2, 0)])
def test_fwd_8bit_many_requests(S, H, Hkv, d, ctx_hi, new_hi, words):
    rng = np.random.default_rng(S)
    reqs = [(int(rng.integers(0, ctx_hi)), int(rng.integers(0 if new_hi > 1 else 1, new_hi + 1))) for _ in range(S)]
    m = make8(H, Hkv, d, 16, reqs, seed=S, pad_rows=2)
    if words:
        m = with_trees(m, reqs, words, S)
    m["total"][S // 3] = -1
    check_ex(m, 0.5)


@pytest.mark.parametrize("pages", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (5, 1), (24, 1)])
@pytest.mark.parametrize("d,page", [(128, 16), (64, 32), (80, 64), (48, 16), (32, 128)])
def test_fwd_trees(d, page, H, Hkv, pages):
    reqs = TREES if H < 8 else TREES[:8]
    m = make8(H, Hkv, d, page, reqs, d + H, pad_rows=3) if pages == "e4m3" else P.make(pages, H, Hkv, d, page, reqs, d + H, stride_pad=8)
    check_ex(with_trees(m, reqs, 2, d), 0.5)


@pytest.mark.parametrize("pages,d,H,Hkv", [("e4m3", 128, 8, 2), ("bf16", 64, 4, 1), ("f32", 48, 2, 2)])
def test_fwd_trees_long_and_mixed(pages, d, H, Hkv):
    """Trees over divided histories, wide ones, and chunks of more tokens than a tree's bits, whose rows hold anything."""
    reqs = [(20000, 7), (0, 200), (3000, 31), (40, 129), (9, 128), (5000, 1)]
    m = make8(H, Hkv, d, 16, reqs, d, spread=0) if pages == "e4m3" else P.make(pages, H, Hkv, d, 16, reqs, d)
    m = with_trees(m, reqs, 4, d, reach=40, roots=0.02)
    junk = torch.randint(-2**31, 2**31 - 1, m["tree"].shape, dtype=torch.int64).to(torch.int32)
    for b, (_, n) in enumerate(reqs):
        if n > 128:
            m["tree"][m["cu"][b]:m["cu"][b + 1]] = junk[m["cu"][b]:m["cu"][b + 1]]
    check_ex(m, 0.5)


@pytest.mark.parametrize("pages,d,H,Hkv,reqs", [
    ("e4m3", 128, 2, 1, [(6000, 128), (31, 129), (0, 1)]), ("e4m3", 64, 8, 2, [(63, 255), (64, 256), (65, 257), (1, 511)]),
    ("e4m3", 80, 5, 1, [(4097, 300), (20, 51), (20, 52)]), ("e4m3", 48, 8, 8, [(0, 256), (3, 1), (0, 64), (100, 900)]),
    ("e4m3", 32, 3, 3, [(10, 1500)]), ("e4m3", 128, 24, 2, [(129, 30), (2, 5), (500, 140), (0, 21), (90, 22)]),
    ("e4m3", 64, 128, 1, [(70, 3), (5, 1), (300, 2)]), ("e4m3", 128, 256, 2, [(70, 3), (5, 1), (300, 2)]),
    ("bf16", 128, 7, 1, [(700, 60), (31, 37), (0, 9)]), ("bf16", 64, 4, 2, [(9000, 64), (64, 65), (63, 33)]),
    ("bf16", 80, 16, 2, [(129, 100), (4000, 17), (0, 1)]),
])
def test_fwd_query_tiles(pages, d, H, Hkv, reqs):
    """At and around the tiles' 128 and 256 rows, groups that do not divide them, histories in few and many pieces."""
    m = make8(H, Hkv, d, 16, reqs, d + H, stride_pad=8, pad_rows=2) if pages == "e4m3" else P.make(pages, H, Hkv, d, 32, reqs, d + H)
    words = min(32, -(-max(n for _, n in reqs) // 32))
    if pages == "e4m3":
        check_ex(m, 0.5)
    check_ex(with_trees(m, reqs, words, d), 0.5)


@pytest.mark.parametrize("S,H,Hkv,d,new_hi", [(128, 16, 2, 64, 12), (129, 16, 2, 64, 12), (140, 8, 2, 128, 40), (300, 4, 1, 32, 60)])
def test_fwd_query_tiles_many_requests(S, H, Hkv, d, new_hi):
    rng = np.random.default_rng(S)
    reqs = [(int(rng.integers(0, 200)), int(rng.integers(0, new_hi + 1))) for _ in range(S)]
    reqs[S // 2] = (reqs[S // 2][0], new_hi)
    m = with_trees(make8(H, Hkv, d, 16, reqs, seed=S, pad_rows=2), reqs, 2, S)
    m["total"][S // 3] = -1
    check_ex(m, 0.5)


@pytest.mark.parametrize("pages,S,H,Hkv,d", [("e4m3", 40, 8, 2, 128), ("bf16", 40, 8, 8, 64), ("e4m3", 150, 4, 4, 48), ("bf16", 150, 16, 2, 80)])
def test_fwd_single_tokens_beside_chunks(pages, S, H, Hkv, d):
    """Requests for the scan and for query tiles in one call, both with histories that are divided."""
    rng = np.random.default_rng(S + d)
    reqs = [(int(rng.integers(0, 2500)), int(rng.integers(0, 3))) for _ in range(S)]
    reqs[3], reqs[S // 2], reqs[S - 1] = (3000, 512 // (H // Hkv) + 3), (9000, 1), (70, 64 // (H // Hkv) + 1)
    reqs[5] = (100, 64 // (H // Hkv))
    m = widened(make8(H, Hkv, d, 32, reqs, S) if pages == "e4m3" else P.make(pages, H, Hkv, d, 32, reqs, S))
    if pages == "e4m3":
        assert tile_rows(m) == 64
        check_ex(m, 0.5)
    m = with_trees(m, reqs, 3, S)
    assert tile_rows(m) == 64
    check_ex(m, 0.5)


@pytest.mark.parametrize("pages", ["e4m3", "bf16", "f32"])
def test_fwd_tree_of_a_path_is_the_chunk(pages):
    """Trees that are one path, under any number of words, are the chunks' rows, bit for bit in the scan."""
    reqs = [(0, 33), (50, 9), (1000, 3), (7, 64), (4, 1)]
    m = make8(8, 2, 64, 16, reqs, 3) if pages == "e4m3" else P.make(pages, 8, 2, 64, 16, reqs, 3)
    with R.kernels(fwd="scan"):
        want = run_ex(m, 0.5)
        for words in (2, 3, 32):
            m["tree"] = torch.from_numpy(X.bits_of(np.concatenate([np.arange(n) - 1 for _, n in reqs]), m["cu"].numpy(),
                                                   m["total"].numpy(), words, m["N"], junk=np.random.default_rng(words)))
            assert torch.equal(run_ex(m, 0.5), want)


@pytest.mark.parametrize("pages", ["e4m3", "bf16"])
def test_fwd_all_roots_see_the_cache_alone(pages):
    reqs = [(0, 5), (40, 40), (16, 2)]
    m = make8(4, 2, 128, 16, reqs, 5) if pages == "e4m3" else P.make(pages, 4, 2, 128, 16, reqs, 5)
    m["tree"] = torch.zeros((m["N"], 2), dtype=torch.int32)
    Y = check_ex(m, 0.5)
    # With nothing cached a root is its own V alone.
    own = P.f64(m["cV"])[m["table"][0, 0], :, :5].transpose(1, 0, 2) if pages == "bf16" else m["v64"][m["table"][0, 0], :, :5].transpose(1, 0, 2)
    np.testing.assert_array_equal(P.f64(Y[:5]), own.repeat(2, axis=1))


@pytest.mark.parametrize("new", [20, 200])
def test_fwd_8bit_leaves_other_rows(new):
    reqs = [(10, 3), (0, 0), (40, 4), (7, 1), (30, new), (5, 2), (2, 2), (9, 90)]
    m = make8(4, 2, 64, 16, reqs, seed=3, pad_rows=4)
    m = with_trees(m, reqs, 1, 3)
    m["total"][2], m["total"][3], m["total"][5] = -1, 0, 2**31 - 1
    check_ex(m, 0.5, max_new=8)
    check_ex(m, 0.5, max_new=100)
    for tree in (m["tree"], None):
        m["tree"] = tree
        for k, v in ((-1, m["N"] + 1), (0, -2)):
            cu = m["cu"].clone()
            m["cu"][k] = v
            check_ex(m, 0.5, max_new=300)
            m["cu"] = cu


@pytest.mark.parametrize("reqs,words", [(DECODE, 0), (RAGGED, 0), (TREES, 2)])
def test_fwd_8bit_pages_outside_the_cache_read_as_zeros(reqs, words):
    m = make8(4, 2, 64, 16, reqs, seed=8)
    if words:
        m = with_trees(m, reqs, words, 8)
    for b in range(len(reqs)):
        m["table"][b, 0] = [P.BAD, m["cP2"].shape[0], 2**31 - 1][b % 3]
    check_ex(m, 0.5)


@pytest.mark.parametrize("pages,reqs", [("e4m3", RAGGED), ("bf16", TREES[:8]), ("f32", TREES[:8])])
def test_fwd_ex_large_evidence(pages, reqs):
    """Evidence to some hundreds: the stabiliser moves. fp32: du as for the forward without trees."""
    m = make8(4, 2, 64, 16, reqs, 5, spread=0, scale=5.0) if pages == "e4m3" else P.make(pages, 4, 2, 64, 16, reqs, 5, scale=5.0)
    check_ex(with_trees(m, reqs, 3, 5), 0.5, du=2e-3)
    m["tree"] = None
    if pages == "e4m3":
        check_ex(m, 0.5)


@pytest.mark.parametrize("pages,d", [("e4m3", 128), ("bf16", 64), ("e4m3", 48)])
def test_fwd_query_tiles_large_evidence_over_long_history(pages, d):
    """Row blocks that the tiles scan a second time, over more tiles than a wave holds table entries of, beside others."""
    reqs = [(9000, 40), (6000, 64), (70, 30)]
    m = make8(4, 1, d, 16, reqs, d, spread=0, scale=5.0) if pages == "e4m3" else P.make(pages, 4, 1, d, 16, reqs, d, scale=5.0)
    m["P1"][m["cu"][1]:m["cu"][2]] *= 0.125
    check_ex(with_trees(m, reqs, 2, d), 0.5)
    m["tree"] = None
    if pages == "e4m3":
        check_ex(m, 0.5)


def test_fwd_8bit_far_scales():
    """V rows of scales up to 2^90 and down to 2^-90 in one request: the bound is relative to what a row sums."""
    m = P.make("bf16", 2, 1, 64, 16, [(300, 1), (90, 40)], seed=2)
    check_ex(X.as_8bit(m, np.random.default_rng(3), 90), 0.5)


def test_fwd_8bit_past_32_bit_offsets():
    """Pages on both sides of 2^31 and 2^32 bytes: written by the append, read by single tokens, chunks and trees, moved."""
    H, Hkv, d, page = 4, 2, 128, 256
    per = Hkv * page * d
    n_pages = (1 << 32) // per + 40
    reqs = [(600, 1), (100, 160), (300, 5)]
    m = with_trees(make8(H, Hkv, d, page, reqs, 7), reqs, 1, 7)
    held = int(m["cP2"].shape[0])
    marks = [(1 << 31) // per, (1 << 32) // per]
    where = np.array([0, n_pages - 1] + [k + j for k in marks for j in (-2, -1, 0, 1)] + list(range(50, 50 + held)))[:held]
    at = torch.from_numpy(where).to(DEV)
    big = [torch.empty((n_pages, Hkv, page, d), dtype=torch.float8_e4m3fn, device=DEV) for _ in range(2)]
    sc = torch.zeros((n_pages, Hkv, 2, page), dtype=torch.uint8, device=DEV)
    dev = X.to_device(m)
    for b, c in zip(big, ("cP2", "cV")):
        b.view(torch.uint8)[at] = dev[c].view(torch.uint8)
    sc[at] = dev["scale"].view(torch.uint8)
    sc = sc.view(torch.float8_e8m0fnu)
    small = m["table"].numpy()
    table = i32(np.where(small >= 0, where[np.clip(small, 0, None)], P.BAD))
    wide = torch.full((len(reqs), 100), P.BAD, dtype=torch.int32, device=DEV)
    for tree, cols in ((None, 0), (dev["tree"], 0), (None, 100), (dev["tree"], 100)):
        kw = dict(max_new=160, tree=tree)
        assert (tile_rows(dict(m, table=torch.cat([m["table"], wide.cpu()[:, :cols]], 1))) == 0) == (cols > 0)
        want = R.paged_fwd(dev["P1"], dev["cP2"], dev["cV"], torch.cat([dev["table"], wide[:, :cols]], 1), dev["total"], dev["cu"], m["tau"],
                           0.5, scale=dev["scale"], **kw)
        got = R.paged_fwd(dev["P1"], *big, torch.cat([table, wide[:, :cols]], 1), dev["total"], dev["cu"], m["tau"], 0.5, scale=sc, **kw)
        assert torch.equal(got, want)
    n = len(where)
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((n, 2 * Hkv, d))).to(torch.bfloat16).to(DEV)
    R.paged_append(x[:, :Hkv], x[:, Hkv:], i32(where * page + page - 1), *big, scale=sc)
    torch.cuda.synchronize()
    q, k = XO.quantise(P.f64(x))
    for part, c in enumerate(big):
        np.testing.assert_array_equal(P.f64(c.view(torch.uint8)[at][:, :, -1].view(torch.float8_e4m3fn)), q[:, part * Hkv:(part + 1) * Hkv])
        np.testing.assert_array_equal(sc.view(torch.uint8)[at][:, :, part, -1].cpu().numpy() - 127.0, k[:, part * Hkv:(part + 1) * Hkv])
    # A request whose new tokens lie in pages past both marks.
    tb = i32([[where[4], where[8], where[7], where[1]]])
    before = [c.view(torch.uint8)[at].cpu().numpy() for c in (*big, sc.view(torch.uint8).transpose(2, 3))]
    lens, free, n_free, odd = i32([0]), i32([-1] * 4), i32([0]), np.concatenate([np.arange(300) * 2 + 1, np.zeros(300)])
    R.paged_keep(*big, tb, i32([1000]), i32([0, 600]), i32(odd), i32([300]), lens, free, n_free, n_free_out=n_free, scale=sc)
    R.paged_keep(*big, tb, i32([1000]), i32([0, 600]), i32(np.arange(600) + 300), i32([300]), lens, free, n_free, n_free_out=n_free, scale=sc)
    torch.cuda.synchronize()
    spots = {int(w): j for j, w in enumerate(where)}
    t2 = np.array([[spots[int(p)] for p in tb[0].cpu()]])
    r = XO.paged_keep(before, t2, [1000], [0, 600], odd, [300], [0], [-1] * 4, 0, page)
    assert r["n_free"] == 1                                       # the second call returns the same page again
    r = XO.paged_keep(r["caches"], t2, [1000], [0, 600], np.arange(600) + 300, [300], r["lens"], r["free"], 1, page)
    for c, w in zip((*big, sc.view(torch.uint8).transpose(2, 3)), r["caches"]):
        np.testing.assert_array_equal(c.view(torch.uint8)[at].cpu().numpy(), w)
    assert int(n_free) == 2 and lens.tolist() == [700]


# ---- cut ---------------------------------------------------------------------------------

def cache_of(pages, n_pages, Hkv, page, d, rng):
    """Pages of random bytes, so that any row moved wrongly is seen."""
    if pages == "e4m3":
        raw = [torch.from_numpy(rng.integers(0, 256, (n_pages, Hkv, page, d)).astype(np.uint8)) for _ in range(2)]
        sc = torch.from_numpy(rng.integers(0, 256, (n_pages, Hkv, 2, page)).astype(np.uint8))
        return [c.to(DEV).view(torch.float8_e4m3fn) for c in raw], sc.to(DEV).view(torch.float8_e8m0fnu)
    dt = W.torch_dtype(pages)
    return [torch.from_numpy(rng.standard_normal((n_pages, Hkv, page, d))).to(dt).to(DEV) for _ in range(2)], None


def rows_of(caches, scale):
    """Host copies [n_pages, H_kv, page, ...] of the bytes."""
    out = [c.view(torch.uint8).cpu().numpy() if scale is not None else c.float().cpu().numpy() for c in caches]
    return out + ([scale.view(torch.uint8).cpu().numpy().transpose(0, 1, 3, 2).copy()] if scale is not None else [])


def check_keep(pages, Hkv, d, page, table, total, cu, keep, n_keep, F, n_free, seed, n_pages=None, in_place=False):
    rng = np.random.default_rng(seed)
    n_pages = int(np.max(table)) + 2 if n_pages is None else n_pages
    caches, sc = cache_of(pages, n_pages, Hkv, page, d, rng)
    free = np.full(F, -5)
    lens = np.full(len(total), 12345)
    want = XO.paged_keep(rows_of(caches, sc), np.asarray(table), total, cu, keep, n_keep, lens, free, n_free, page)
    ln, fr, nf = i32(lens), i32(free), i32([n_free])
    got = R.paged_keep(*caches, i32(table), i32(total), i32(cu), i32(keep), i32(n_keep), ln, fr, nf,
                       n_free_out=nf if in_place else None, scale=sc)
    torch.cuda.synchronize()
    for g, w in zip(rows_of(caches, sc), want["caches"]):
        np.testing.assert_array_equal(g, w)
    assert ln.tolist() == want["lens"] and fr.tolist() == want["free"] and int(got) == want["n_free"]
    assert in_place or int(nf) == n_free


@pytest.mark.parametrize("pages", ["e4m3", "bf16", "f32"])
@pytest.mark.parametrize("S,Hkv,d,page,ctx_hi,new_hi,most,seed", [
    (1, 1, 32, 16, 0, 1, 1, 1), (5, 3, 48, 16, 40, 9, 4, 2), (48, 4, 64, 32, 100, 24, 6, 3), (256, 2, 128, 16, 60, 40, 40, 4),
    (257, 1, 80, 64, 300, 64, 8, 5), (600, 2, 32, 16, 30, 12, 12, 6), (3, 8, 128, 16, 200, 700, 600, 7), (2, 1, 64, 256, 1000, 300, 300, 8),
])
def test_paged_keep(pages, S, Hkv, d, page, ctx_hi, new_hi, most, seed):
    rng = np.random.default_rng(seed)
    ctx, nn = rng.integers(0, ctx_hi + 1, S), rng.integers(0 if S > 2 else new_hi, new_hi + 1, S)
    total = ctx + nn
    held = -(-total // page)
    width = int(held.max()) + 1
    table = np.full((S, width), P.BAD)
    order = rng.permutation(int(held.sum()) + 3)
    cu = np.concatenate([[0], np.cumsum(nn)])
    keep = np.full(int(cu[-1]) + 5, 99)
    n_keep = np.array([rng.integers(0, min(most, n) + 1) for n in nn])
    if S <= 2:
        n_keep[:] = np.minimum(most, nn)
        n_keep[0] = max(1, nn[0] * 2 // 3)
    at = 0
    for b in range(S):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
        keep[cu[b]:cu[b] + n_keep[b]] = np.sort(rng.permutation(nn[b])[:n_keep[b]])
    if S > 4:                                        # requests that are refused, and choices that are not valid
        total[1] = -1
        n_keep[2] = nn[2] + 1
        n_keep[3] = -1
        b = int(np.argmax(n_keep))
        if n_keep[b] > 2:
            keep[cu[b] + 1] = keep[cu[b]]
    check_keep(pages, Hkv, d, page, table, total, cu, keep, n_keep, max(4, int(held.sum()) // 2), 3, seed, n_pages=len(order), in_place=seed % 2 == 0)


def test_paged_keep_edges():
    # Offsets that overlap or leave the batch, pages outside the cache, a count outside the list, a full list.
    table = np.array([[0, 1, 2], [3, 99, 4], [5, -7, 6], [7, 8, 9]])
    keep = [1, 2, 5, 0, 0, 0, 1, 17, 20, 0, 0, 0, 3, 4, 19, 0, 0, 0, 0, 0, 18]
    for cu in ([0, 6, 12, 18, 21], [0, 21, 0, 21, 21], [-1, 6, 30, 18, 21], [6, 0, 12, 21, 18]):
        for n_keep in ([3, 3, 3, 1], [6, 2, 1, 3], [0, 0, 0, 0], [2**31 - 1, -2**31, 7, 21]):
            for total in ([40, 33, 30, 48], [6, 6, 49, 20], [0, -1, 2**31 - 1, 21]):
                for n_free in (-4, 2, 900):
                    check_keep("e4m3", 2, 32, 16, table, total, cu, keep, n_keep, 5, n_free, 1, n_pages=10)


# ---- together ------------------------------------------------------------------------------

@pytest.mark.parametrize("pages", ["e4m3", "bf16", "f32"])
def test_speculative_serving_loop(pages):
    """Prompts, then trees of drafted tokens of which a path is kept: every step's rows against the plain forward of what
    the pages hold, the kept rows against those that were written, and the pages' accounts."""
    H, Hkv, d, page, n_pages, S, width = 8, 2, 64, 16, 60, 4, 20
    rng = np.random.default_rng(11)
    tdt = torch.bfloat16 if pages == "e4m3" else W.torch_dtype(pages)
    caches = [torch.zeros((n_pages, Hkv, page, d), device=DEV).to(torch.float8_e4m3fn if pages == "e4m3" else tdt) for _ in range(2)]
    sc = scales(n_pages, Hkv, page) if pages == "e4m3" else None
    table = torch.full((S, width), P.BAD, dtype=torch.int32, device=DEV)
    free, n_free, lens = i32(rng.permutation(n_pages)), i32([n_pages]), i32([0] * S)
    tau, theta = rng.uniform(0.5, 2.0, H).astype(np.float32), rng.uniform(-2, 2, 1).astype(np.float32)
    kept = [[] for _ in range(S)]

    def held_rows(b, T):
        """Bytes of rows 0 .. T-1 of request b: P2, V and scales, [T, ...]."""
        tb = table[b].cpu().numpy()
        return [np.stack([c[tb[p // page], :, p % page] for p in range(T)]) if T else None for c in rows_of(caches, sc)]

    for step, nn in enumerate([[40, 7, 0, 65], [9, 20, 33, 1], [1, 12, 4, 30], [30, -1, 25, 6], [64, 18, 8, 3], [5, 5, 5, 5]]):
        N = sum(max(n, 0) for n in nn) + 3
        x = torch.from_numpy(rng.standard_normal((N, H + 2 * Hkv, d))).to(tdt).to(DEV)
        cu, total, slot, _, _ = R.page_map(lens, i32(nn), table, free, n_free, N, page, n_pages, out=tuple(
            torch.empty(k, dtype=torch.int32, device=DEV) for k in (S + 1, S, N, N)) + (n_free,))
        assert min(total.tolist()) >= 0
        count = [max(n, 0) for n in nn]
        parent = np.concatenate([X.random_parents(count, rng), [-1] * 3])
        if step == 0:
            parent = np.concatenate([np.arange(n) - 1 for n in count] + [[-1] * 3])      # prompts
        tree, pos = R.tree_plan(i32(parent), total, cu, 2)
        q = R.paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], slot, *caches, P1=x[:, :H], pos=pos, rope="half", theta=theta, scale=sc)
        Y = R.paged_fwd(q, *caches, table, total, cu, tau, 0.5, max_new=max(count), scale=sc, tree=tree)
        torch.cuda.synchronize()
        at, tot = cu.cpu().numpy(), total.cpu().numpy()
        k64, v64 = (P.f64(c) * (2.0**exps(sc)[:, :, j, :, None] if sc is not None else 1.0) for j, c in enumerate(caches))
        ref, spread = XO.paged_fwd(P.f64(q), k64, v64, table.cpu().numpy(), tot, at, tau, 0.5, np.zeros((N, H, d)), max(count),
                                   tree=tree.cpu().numpy())
        lim = limit(dict(P1=q, cP2=caches[0], table=table, total=total, max_new=max(count), N=N, tree=tree), ref, spread, k64)
        assert np.all(np.abs(P.f64(Y) - ref) <= lim)
        # Keep a path of each tree (prompts: all of it).
        keep, n_keep, rows = np.zeros(N, dtype=np.int64), [], [held_rows(b, int(tot[b])) for b in range(S)]
        for b, n in enumerate(count):
            path = list(range(n))
            if n and step:
                leaf = int(rng.integers(0, n))
                path = sorted(XO.ancestors(parent[at[b]:at[b + 1]], leaf)) + [leaf]
            if nn[b] < 0:
                kept[b] = []
            ctx = int(tot[b]) - n
            assert ctx == len(kept[b])
            for k, i in enumerate(path):
                assert int(pos[at[b] + i]) == ctx + k if n <= 64 else True
                kept[b].append([c[ctx + i] for c in rows[b]])
            keep[at[b]:at[b] + len(path)] = path
            n_keep.append(len(path))
        R.paged_keep(*caches, table, total, cu, i32(keep), i32(n_keep), lens, free, n_free, n_free_out=n_free, scale=sc)
        torch.cuda.synchronize()
        assert lens.tolist() == [len(r) for r in kept]
        for b in range(S):
            if kept[b]:
                for c, g in enumerate(held_rows(b, len(kept[b]))):
                    np.testing.assert_array_equal(g, np.stack([r[c] for r in kept[b]]))
        used = [int(table[b, k]) for b in range(S) for k in range(-(-int(lens[b]) // page))]
        assert sorted(used + free[:int(n_free)].tolist()) == list(range(n_pages))


@pytest.mark.parametrize("width", [60, 1100])
@pytest.mark.parametrize("pages", ["e4m3", "bf16"])
def test_calls_replay_in_a_graph(pages, width):
    """A whole step captured once and replayed with new lengths, trees and inputs, against the eager calls: in the scan, and
    in a table wide enough for query tiles."""
    S, N, H, Hkv, d, page, n_pages, held = 6, 300, 8, 2, 64, 16, 460, 60
    assert (N * H * (width * page + 500) >= 12000000) == (width > held)
    rng = np.random.default_rng(2)
    lens0, nn, parent, keep, n_keep = (torch.zeros(k, dtype=torch.int32, device=DEV) for k in (S, S, N, N, S))
    base = rng.permutation(n_pages)
    base = base[base >= S * held]                     # the table rows hold the others
    x = torch.zeros((N, H + 2 * Hkv, d), dtype=torch.bfloat16, device=DEV)
    cdt = torch.float8_e4m3fn if pages == "e4m3" else torch.bfloat16
    state = {}
    for name in ("graph", "eager"):
        state[name] = dict(table=torch.zeros((S, width), dtype=torch.int32, device=DEV), free=i32(np.tile(base, 4)), n_free=i32([len(base)]), lens=i32([0] * S),
                           c=[torch.zeros((n_pages, Hkv, page, d), device=DEV).to(cdt) for _ in range(2)],
                           sc=scales(n_pages, Hkv, page, 120) if pages == "e4m3" else None,
                           out=tuple(torch.zeros(k, dtype=torch.int32, device=DEV) for k in (S + 1, S, N, N, 1)),
                           plan=(torch.zeros((N, 2), dtype=torch.int32, device=DEV), torch.zeros(N, dtype=torch.int32, device=DEV)),
                           q=torch.zeros((N, H, d), dtype=torch.bfloat16, device=DEV), Y=torch.zeros((N, H, d), dtype=torch.bfloat16, device=DEV),
                           last=i32([0]), ws=torch.empty(R.paged_workspace_bytes(N, S, H, Hkv, d), dtype=torch.uint8, device=DEV))

    def work(s):
        cu, total, slot, _, left = R.page_map(lens0, nn, s["table"], s["free"], s["n_free"], N, page, n_pages, out=s["out"])
        tree, pos = R.tree_plan(parent, total, cu, 2, out=s["plan"])
        R.paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], slot, *s["c"], P1=x[:, :H], pos=pos, rope="interleaved", out=s["q"], scale=s["sc"])
        R.paged_fwd(s["q"], *s["c"], s["table"], total, cu, 1.0, 0.5, max_new=N, out=s["Y"], workspace=s["ws"], scale=s["sc"], tree=tree)
        R.paged_keep(*s["c"], s["table"], total, cu, keep, n_keep, s["lens"], s["free"], left, n_free_out=s["last"], scale=s["sc"])
        return [s["Y"], s["q"], s["table"], s["lens"], s["free"], s["last"], pos, tree, *(c.view(torch.uint8) for c in s["c"])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        work(state["graph"])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work(state["graph"])
    torch.cuda.synchronize()
    for ln, n in (([0] * 6, [64, 1, 0, 30, 2, 64]), ([300, 0, 16, 700, 2, 129], [33] * 6), ([301, 5, 0, 1, 3, 600], [40, 1, 130, 1, 1, 1]),
                  ([10, 9, 8, 7, 6, 5], [0] * 6)):
        lens0.copy_(i32(ln))
        nn.copy_(i32(n))
        parent.copy_(i32(np.concatenate([X.random_parents(n, rng), np.zeros(N - sum(n))])))
        at, kp, nk = 0, np.zeros(N), []
        for k in n:
            nk.append(int(rng.integers(0, min(k, 8) + 1)))
            kp[at:at + nk[-1]] = np.sort(rng.permutation(k)[:nk[-1]])
            at += k
        keep.copy_(i32(kp))
        n_keep.copy_(i32(nk))
        x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape))).to(torch.bfloat16))
        own = torch.full((S, width), P.BAD, dtype=torch.int32, device=DEV)
        own[:, :held] = i32(np.arange(S * held).reshape(S, held))
        # Eager from the graph's state, then the replay from the same.
        for name in ("eager", "graph"):
            s = state[name]
            for a, b in zip(s["c"], state["graph"]["c"]):
                a.view(torch.uint8).copy_(b.view(torch.uint8).clone())
            if s["sc"] is not None:
                s["sc"].view(torch.uint8).copy_(state["graph"]["sc"].view(torch.uint8).clone())
            s["free"].copy_(i32(np.tile(base, 4)))
            s["Y"].fill_(0.0)
            s["q"].fill_(0.0)
            s["plan"][0].fill_(0)
            s["lens"].fill_(0)
            s["table"].copy_(own)
            torch.cuda.synchronize()
            if name == "eager":
                want = [t.clone() for t in work(s)]
                torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), k


def test_calls_on_streams_at_once():
    """Forwards on three streams at once, a workspace each, and other calls of the kind beside them."""
    ms = [make8(8, 2, 128, 16, [(6000, 1), (300, 9), (0, 200)], 1), with_trees(make8(4, 4, 64, 16, TREES, 2), TREES, 2, 2),
          widened(with_trees(P.make("bf16", 8, 2, 128, 16, TREES, 3), TREES, 2, 3)), widened(make8(8, 2, 128, 16, CHUNKS, 4))]
    want = [run_ex(m, 0.5) for m in ms]
    ds = [X.to_device(m) for m in ms]
    streams, outs = [torch.cuda.Stream() for _ in ms], [torch.full_like(y, 3.0) for y in want]
    wss = [torch.empty(R.paged_workspace_bytes(m["N"], len(m["total"]), *(m["P1"].shape[1], m["cP2"].shape[1], m["P1"].shape[2])),
                       dtype=torch.uint8, device=DEV) for m in ms]
    plans = [R.tree_plan(i32(m["parent"]), d["total"], d["cu"], 2)[1].clone() for m, d in list(zip(ms, ds))[1:3]]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s, y, ws in zip(ds, streams, outs, wss):
            R.paged_fwd(d["P1"], d["cP2"], d["cV"], d["table"], d["total"], d["cu"], d["tau"], 0.5, max_new=d["max_new"], out=y,
                        stream=s, workspace=ws, scale=d.get("scale"), tree=d.get("tree"))
        again = [R.tree_plan(i32(m["parent"]), d["total"], d["cu"], 2, stream=s)[1] for m, d, s in list(zip(ms, ds, streams))[1:3]]
    torch.cuda.synchronize()
    for y, w in zip(outs, want):
        assert torch.equal(y, w)
    for a, b in zip(again, plans):
        assert torch.equal(a, b)


def test_same_call_same_bits_through_one_workspace():
    ms = [make8(8, 2, 128, 16, [(9000, 1), (300, 1), (5000, 4)], 1), with_trees(make8(8, 8, 64, 16, TREES, 2), TREES, 2, 2),
          with_trees(P.make("f32", 4, 1, 48, 32, TREES, 3), TREES, 2, 3), widened(make8(8, 2, 128, 16, CHUNKS, 4)),
          widened(with_trees(P.make("bf16", 8, 2, 64, 16, TREES, 5), TREES, 2, 5))]
    need = max(R.paged_workspace_bytes(m["N"], len(m["total"]), m["P1"].shape[1], m["cP2"].shape[1], m["P1"].shape[2]) for m in ms)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    first = [run_ex(m, 0.5, ws=ws) for m in ms]
    for m, y in zip(ms[::-1], first[::-1]):
        assert torch.equal(run_ex(m, 0.5, ws=ws), y)
