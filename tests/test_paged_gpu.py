"""The paged Relation Cache on the GPU: page map, packed append and chunk
forward against plain evaluations (oracle/paged_oracle.py), alone and together."""
import numpy as np
import pytest
import torch

from causal_self_exchange_amd import relation as R
from causal_self_exchange_amd import workloads as W
from oracle import paged_oracle as PO
from oracle import prestep_oracle as PR
from oracle import relation_oracle as RO

import _paged as P

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ---- page map -----------------------------------------------------------------

def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def check_map(lens, n_new, table, free, n_free, N, page, n_pages, in_place=False):
    want = PO.page_map(lens, n_new, table, free, n_free, N, page, n_pages)
    tb, fr, nf = i32(table), i32(free), i32([n_free])
    out = None
    if in_place:
        out = tuple(torch.full((n,), 77, dtype=torch.int32, device=DEV) for n in (len(lens) + 1, len(lens), N, N)) + (nf,)
    cu, total, slot, pos, n_out = R.page_map(i32(lens), i32(n_new), tb, fr, nf, N, page, n_pages, out=out)
    torch.cuda.synchronize()
    got = dict(cu=cu, total=total, slot=slot, pos=pos, n_free=n_out, table=tb, free=fr)
    for k, t in got.items():
        np.testing.assert_array_equal(t.cpu().numpy(), np.asarray(want[k]), err_msg=k)
    return want


@pytest.mark.parametrize("S,len_hi,new_hi,page,release,frac,pad,seed", [
    (1, 0, 1, 16, 0.0, 1.0, 0, 1), (1, 40, 0, 16, 0.0, 1.0, 3, 2), (7, 100, 1, 16, 0.0, 1.0, 0, 3),
    (64, 300, 1, 64, 0.2, 1.0, 0, 4), (65, 50, 70, 16, 0.3, 0.5, 9, 5), (300, 200, 30, 32, 0.1, 0.8, 100, 6),
    (1023, 33, 3, 16, 0.1, 0.9, 0, 7), (1024, 33, 3, 256, 0.1, 2.0, 1, 8), (1025, 33, 3, 128, 0.5, 0.2, 0, 9),
    (2500, 90, 5, 16, 0.3, 0.6, 17, 10), (3, 5, 5000, 16, 0.0, 1.0, 0, 11), (40, 20000, 3000, 16, 0.4, 0.7, 5, 12),
])
def test_page_map(S, len_hi, new_hi, page, release, frac, pad, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, len_hi + 1, S)
    n_new = np.where(rng.random(S) < release, -1, rng.integers(0, new_hi + 1, S))
    held = -(-lens // page)
    need = -(-(lens + np.maximum(n_new, 0)) // page) - held
    width = int((held + need).max()) + 1
    n_free = max(1, int(need.sum() * frac))
    n_pages = int(held.sum()) + n_free
    order = rng.permutation(n_pages)
    table = np.full((S, width), P.BAD)
    at = 0
    for b in range(S):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    free = np.full(n_pages, -1)
    free[:n_free] = order[at:]
    N = max(1, int(np.maximum(n_new, 0).sum()) + pad)
    check_map(lens, n_new, table, free, n_free, N, page, n_pages, in_place=seed % 2 == 0)


def test_page_map_refuses_request_by_request():
    big = 2**31 - 1
    # Lengths, counts and page numbers that do not fit, next to good ones; the list runs out in between.
    lens = [0, -1, 16, 64, big, 5, 17, 15, 0, -5, 30, 0]
    n_new = [1, 3, -2, 1, big, 27, 40, 1, 16, -1, -1, 100]
    table = np.full((12, 4), P.BAD)
    table[2, :1], table[5, 0], table[6, :2], table[7, 0], table[10, :2] = 3, 900, [4, 5], 6, [7, 8]
    free = [10, 11, 999, 12, 13, 0, 0, 0, 0, 0]
    want = check_map(lens, n_new, table, free, 5, 200, 16, 20)
    assert want["total"][0] == 1 and want["total"][3] == -1 and want["total"][10] == 0
    check_map(lens, n_new, table, free, 5, 40, 16, 20)            # fewer packed rows than tokens
    check_map(lens, n_new, table, free, -3, 200, 16, 20)          # counts outside the list
    check_map(lens, n_new, table, free, 500, 200, 16, 20)
    check_map([64] * 5, [-1] * 5, np.arange(20).reshape(5, 4), [-1] * 7, 3, 4, 16, 20)   # more returned than fit


# ---- append --------------------------------------------------------------------

APPEND = [
    # dt, N, H, Hkv, d, page, rope, mix, pairing, fused
    ("bf16", 1, 8, 8, 64, 16, "interleaved", True, "A", True), ("bf16", 37, 12, 4, 128, 64, "half", True, "B", True),
    ("f32", 33, 6, 2, 80, 32, "interleaved", True, "B", False), ("f32", 5, 3, 3, 48, 16, "half", False, "A", True),
    ("bf16", 130, 5, 1, 32, 256, "none", False, "A", False), ("bf16", 64, 16, 16, 80, 128, "half", True, "A", False),
    ("f32", 19, 4, 4, 128, 16, "none", True, "A", True), ("bf16", 700, 32, 8, 128, 16, "interleaved", True, "B", True),
]


def token_slots(N, n_pages, page, rng, gaps=True):
    slot = rng.permutation(n_pages * page)[:N].astype(np.int32)
    if gaps and N > 4:
        slot[rng.integers(0, N, 3)] = [-1, -9, n_pages * page]     # no slot, and past the last page
    return slot


@pytest.mark.parametrize("dt,N,H,Hkv,d,page,rope,mix,pairing,fused", APPEND)
def test_paged_append(dt, N, H, Hkv, d, page, rope, mix, pairing, fused):
    rng = np.random.default_rng(N + d)
    tdt = W.torch_dtype(dt)
    n_pages = -(-N // page) + 3
    x = torch.from_numpy(rng.standard_normal((N, H + 2 * Hkv, d))).to(tdt).to(DEV)
    P1, P2, I = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
    if not fused:
        P1, P2, I = P1.contiguous(), P2.contiguous(), I.contiguous()
    slot = token_slots(N, n_pages, page, rng)
    pos = rng.integers(0, 70000, N).astype(np.int32)
    theta = rng.uniform(-3, 3, Hkv // 2).astype(np.float32) if mix else None
    cP2, cV = (torch.full((n_pages, Hkv, page, d), 5.0, dtype=tdt, device=DEV) for _ in range(2))
    out = torch.full((N, H, d), 7.0, dtype=tdt, device=DEV)
    got = R.paged_append(P2, I, i32(slot), cP2, cV, P1=P1, pos=i32(pos), rope=rope, theta=theta, pairing=pairing, out=out)
    torch.cuda.synchronize()
    assert got is out
    live = (slot >= 0) & (slot < n_pages * page)
    # Against the fp64 pre-steps: |x - x*| <= half a step of the output + a few fp32 roundings of the two products.
    a = PR.rope(P.f64(P1).transpose(1, 0, 2), pos, 1e4, rope).transpose(1, 0, 2)
    k = PR.rope(P.f64(P2).transpose(1, 0, 2), pos, 1e4, rope).transpose(1, 0, 2)
    v = P.f64(I) if theta is None else PR.givens_mix(P.f64(I)[:, :, None], theta, pairing)[:, :, 0]
    half = 2.0**-8 if dt == "bf16" else 2.0**-24
    big = float(np.abs(P.f64(x)).max()) * 2
    pages, offs = slot[live] // page, slot[live] % page
    for name, g, w in (("P1", P.f64(out)[live], a[live]), ("P2", P.f64(cP2)[pages, :, offs], k[live]),
                       ("V", P.f64(cV)[pages, :, offs], v[live])):
        assert np.all(np.abs(g - w) <= half * np.abs(w) + 2.0**-20 * big), name
    # Everything else is as it was.
    assert np.all(P.f64(out)[~live] == 7.0)
    rest = np.ones((n_pages, page), dtype=bool)
    rest[pages, offs] = False
    for c in (cP2, cV):
        assert np.all(P.f64(c).transpose(0, 2, 1, 3)[rest] == 5.0)


def test_paged_append_of_more_tokens_than_one_launch_takes():
    N = (1 << 23) + 5
    n_pages = -(-N // 256)
    x = torch.randn((N, 2, 32), device=DEV).to(torch.bfloat16)
    slot = torch.arange(N - 1, -1, -1, dtype=torch.int32, device=DEV)
    c = [torch.zeros((n_pages, 1, 256, 32), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    R.paged_append(x[:, :1], x[:, 1:], slot, *c)
    torch.cuda.synchronize()
    for k in range(2):
        assert torch.equal(c[k].view(-1, 32)[:N].flip(0), x[:, k])


@pytest.mark.parametrize("dt,N,H,d,rope,pairing", [("bf16", 50, 4, 128, "half", "A"), ("f32", 21, 6, 48, "interleaved", "B"),
                                                   ("bf16", 9, 2, 80, "interleaved", "A"), ("f32", 64, 8, 64, "half", "B")])
def test_paged_append_equals_prestep(dt, N, H, d, rope, pairing):
    """The same rotations and mixings as relation_prestep on one-token sequences, bit for bit."""
    rng = np.random.default_rng(d)
    tdt = W.torch_dtype(dt)
    P1, P2, I = (torch.from_numpy(rng.standard_normal((N, H, d))).to(tdt).to(DEV) for _ in range(3))
    pos, theta = i32(rng.integers(0, 9000, N)), rng.uniform(-3, 3, H // 2).astype(np.float32)
    slot = rng.permutation(80)[:N].astype(np.int32)
    cP2, cV = torch.zeros((5, H, 16, d), dtype=tdt, device=DEV), torch.zeros((5, H, 16, d), dtype=tdt, device=DEV)
    w1, w2, wi = R.prestep(P1[:, :, None], P2[:, :, None], I[:, :, None], pos, rope, 1e4, theta, pairing)
    got = R.paged_append(P2, I, i32(slot), cP2, cV, P1=P1, pos=pos, rope=rope, theta=theta, pairing=pairing, out=P1)
    torch.cuda.synchronize()
    assert got is P1 and torch.equal(P1, w1[:, :, 0])
    pages, offs = torch.from_numpy(slot // 16).long().to(DEV), torch.from_numpy(slot % 16).long().to(DEV)
    assert torch.equal(cP2[pages, :, offs], w2[:, :, 0]) and torch.equal(cV[pages, :, offs], wi[:, :, 0])
    # Without P1 only the cache is written.
    c2, cv = torch.zeros_like(cP2), torch.zeros_like(cV)
    assert R.paged_append(P2, I, i32(slot), c2, cv, pos=pos, rope=rope, theta=theta, pairing=pairing) is None
    torch.cuda.synchronize()
    assert torch.equal(c2, cP2) and torch.equal(cv, cV)


# ---- chunk forward ---------------------------------------------------------------

def run_fwd(m, lam, dt, ws=None, fill=3.0, max_new=None):
    d = P.to_device(m)
    Y = torch.full(tuple(m["P1"].shape), fill, dtype=m["P1"].dtype, device=DEV)
    R.paged_fwd(d["P1"], d["cP2"], d["cV"], d["table"], d["total"], d["cu"], m["tau"], lam,
                max_new=m["max_new"] if max_new is None else max_new, out=Y, workspace=ws)
    torch.cuda.synchronize()
    return Y


def check_fwd(m, lam, dt, du=1e-6, fill=3.0, max_new=None, skip=None):
    """Y against the plain evaluation, but for the rows of request skip."""
    Y = run_fwd(m, lam, dt, fill=fill, max_new=max_new)
    y0 = np.full(tuple(m["P1"].shape), fill)
    total, cu = m["total"].numpy().copy(), m["cu"].numpy()
    if skip is not None:
        total[skip] = -1
    ref, spread = PO.paged_fwd(P.f64(m["P1"]), np.nan_to_num(P.f64(m["cP2"])), np.nan_to_num(P.f64(m["cV"])),
                               m["table"].numpy(), total, cu, m["tau"], lam, y0,
                               m["max_new"] if max_new is None else max_new, with_spread=True)
    err = np.abs(P.f64(Y) - ref)
    if skip is not None:
        rows = slice(cu[skip], cu[skip + 1])
        assert np.all(np.isfinite(err[rows])) and np.any(err[rows] > 0)
        err[rows] = 0.0
    lim = np.where(spread > 0, P.bound(ref, spread, dt, du), 0.0)      # rows nobody writes stay exactly
    worst = np.unravel_index(np.argmax(err - lim), err.shape)
    assert np.all(err <= lim), (worst, err[worst], lim[worst], float(np.max(err / (lim + 1e-30))))
    return Y


def filler(H):
    """A request with enough work to put the batch's chunks on query tiles (8,000 units of 32 rows by 128 keys, two more a
    row block): 75 row blocks and more over 16,000 rows. Its own rows are not looked at (check_fwd's skip)."""
    return (16000, 75 * 32 // H + 1)


DECODE = [(0, 1), (1, 1), (15, 1), (16, 1), (17, 1), (31, 1), (63, 1), (64, 1), (65, 1), (255, 1), (700, 1)]
RAGGED = [(0, 1), (0, 2), (3, 5), (60, 9), (0, 33), (129, 7), (31, 32), (500, 1), (1, 70)]
CHUNKS = [(0, 130), (77, 300), (1000, 257), (64, 64), (0, 513)]


@pytest.mark.parametrize("H,Hkv", [(4, 4), (8, 2), (6, 2), (7, 1), (24, 1)])
@pytest.mark.parametrize("dt,d,page", [("bf16", 128, 16), ("bf16", 64, 64), ("bf16", 80, 32), ("bf16", 48, 16),
                                       ("bf16", 32, 256), ("f32", 128, 16), ("f32", 64, 32), ("f32", 80, 16),
                                       ("f32", 48, 128), ("f32", 32, 16)])
def test_paged_fwd_decode(dt, d, page, H, Hkv):
    check_fwd(P.make(dt, H, Hkv, d, page, DECODE, seed=d + H, stride_pad=16), 0.5, dt)


@pytest.mark.parametrize("H,Hkv", [(2, 2), (8, 2), (5, 1)])
@pytest.mark.parametrize("dt,d,page", [("bf16", 128, 16), ("bf16", 64, 32), ("bf16", 80, 16), ("bf16", 48, 64),
                                       ("bf16", 32, 128), ("f32", 128, 32), ("f32", 64, 16), ("f32", 80, 256),
                                       ("f32", 48, 16), ("f32", 32, 64)])
def test_paged_fwd_ragged(dt, d, page, H, Hkv):
    check_fwd(P.make(dt, H, Hkv, d, page, RAGGED, seed=d + H, pad_rows=3), 0.25, dt)


@pytest.mark.parametrize("dt,d,page,H,Hkv", [("bf16", 128, 16, 4, 2), ("bf16", 64, 64, 2, 2), ("bf16", 80, 32, 3, 1),
                                             ("bf16", 48, 16, 2, 1), ("bf16", 32, 128, 2, 2), ("f32", 128, 64, 2, 1),
                                             ("f32", 80, 16, 2, 2), ("f32", 48, 32, 3, 1)])
def test_paged_fwd_chunks(dt, d, page, H, Hkv):
    check_fwd(P.make(dt, H, Hkv, d, page, CHUNKS, seed=d + H, stride_pad=32, pad_rows=5), 1.0, dt)


@pytest.mark.parametrize("dt,d", [("bf16", 128), ("bf16", 64), ("f32", 64)])
def test_paged_fwd_long_history(dt, d):
    """Few rows over histories long enough to be split, and a chunk over one."""
    check_fwd(P.make(dt, 4, 2, d, 16, [(20001, 1), (9000, 3), (5, 1), (8190, 18)], seed=d), 0.5, dt)


@pytest.mark.parametrize("d,page,H,Hkv,reqs", [
    (128, 16, 2, 1, [(6000, 128), (31, 129), (0, 1)]), (64, 256, 8, 2, [(63, 255), (64, 256), (65, 257), (1, 511)]),
    (80, 64, 1, 1, [(4097, 300)]), (48, 16, 8, 8, [(0, 256), (3, 1), (0, 64), (100, 900)]),
    (32, 128, 3, 3, [(10, 1500)]), (128, 32, 16, 4, [(129, 190), (2, 5), (500, 140), (0, 127)]),
])
def test_paged_fwd_long_chunks(d, page, H, Hkv, reqs):
    """Chunks of 128 tokens and more, at and around the tile sizes, mixed with short ones; few and many pieces per tile.
    Alone (in the scan), and next to as much work as puts them on tiles."""
    check_fwd(P.make("bf16", H, Hkv, d, page, reqs, seed=d + H, stride_pad=8, pad_rows=2), 0.5, "bf16")
    check_fwd(P.make("bf16", H, Hkv, d, page, reqs + [filler(H)], seed=d + H, stride_pad=8, pad_rows=2), 0.5, "bf16",
              skip=len(reqs))


@pytest.mark.parametrize("d,page,H,Hkv,reqs", [
    # Chunks whose rows share query tiles with those of the other heads: one block of 32 positions to eight, from
    # positions at and off their multiples, groups that do not divide the eight waves, histories long enough to be cut.
    (64, 16, 8, 1, [(0, 16), (16, 16), (17, 16), (40, 17), (3, 1), (64, 8)]),
    (128, 16, 8, 2, [(0, 32), (32, 32), (33, 32), (95, 65), (7, 127), (5000, 100)]),
    (128, 64, 12, 4, [(50, 50), (1, 192), (31, 224), (63, 255), (12000, 43)]),
    (80, 32, 5, 1, [(20, 90), (70, 200), (0, 255), (3000, 26)]),
    (48, 16, 24, 1, [(0, 8), (9, 6), (500, 33), (31, 2), (31, 5)]),
    (32, 256, 9, 3, [(100, 60), (64, 43), (1000, 300)]),
    (64, 128, 3, 3, [(0, 127), (1, 128), (31, 160), (700, 129)]),
    (32, 16, 256, 2, [(0, 9), (31, 10), (200, 33), (5, 1)]),
])
def test_paged_fwd_shared_tiles(d, page, H, Hkv, reqs):
    check_fwd(P.make("bf16", H, Hkv, d, page, reqs, seed=d + H, stride_pad=24, pad_rows=1), 0.5, "bf16")
    check_fwd(P.make("bf16", H, Hkv, d, page, [filler(H)] + reqs, seed=d + H, stride_pad=24, pad_rows=1), 0.5, "bf16",
              skip=0)


@pytest.mark.parametrize("dt,S,H,Hkv,d,ctx_hi,new_hi,every", [
    ("bf16", 128, 4, 2, 64, 200, 1, 0), ("bf16", 129, 4, 2, 64, 200, 1, 0), ("bf16", 300, 2, 1, 64, 90, 4, 0),
    ("bf16", 260, 4, 1, 128, 300, 2, 90), ("f32", 200, 2, 2, 48, 100, 3, 0), ("bf16", 700, 1, 1, 32, 40, 2, 200),
])
def test_paged_fwd_many_requests(dt, S, H, Hkv, d, ctx_hi, new_hi, every):
    """Batches around and past the number of requests whose sums fit a work-group's memory; every so many a long chunk."""
    rng = np.random.default_rng(S)
    reqs = [(int(rng.integers(0, ctx_hi)), int(rng.integers(0 if new_hi > 1 else 1, new_hi + 1))) for _ in range(S)]
    for b in range(every // 2, S, every or S):
        if every:
            reqs[b] = (reqs[b][0], 150 + b)
    if every:
        reqs[S // 2] = filler(H)
    m = P.make(dt, H, Hkv, d, 16, reqs, seed=S, pad_rows=2)
    m["total"][S // 3] = -1
    check_fwd(m, 0.5, dt, skip=S // 2 if every else None)


@pytest.mark.parametrize("dt,H,Hkv,d,reqs", [
    ("bf16", 1, 1, 128, [(40000, 1)]), ("bf16", 16, 1, 64, [(50000, 1)]), ("bf16", 8, 1, 128, [(9000, 4), (30000, 3)]),
    ("bf16", 4, 1, 64, [(20000, 64)]), ("bf16", 2, 2, 80, [(15000, 1), (0, 1), (20, 2)]), ("f32", 16, 1, 32, [(9000, 2)]),
    ("f32", 1, 1, 48, [(12000, 1)]),
])
def test_paged_fwd_many_pieces(dt, H, Hkv, d, reqs):
    """Few rows whose histories lie in many ranges: one, four or sixteen rows to a work-group that joins them."""
    check_fwd(P.make(dt, H, Hkv, d, 16, reqs, seed=d + H), 0.5, dt)


def test_paged_fwd_many_heads():
    check_fwd(P.make("bf16", 256, 256, 32, 16, [(5, 1), (40, 3)], seed=1), 0.5, "bf16")
    check_fwd(P.make("bf16", 256, 2, 64, 16, [(5, 1), (700, 2), (20, 9)], seed=1), 0.5, "bf16")
    check_fwd(P.make("f32", 256, 1, 32, 16, [(5, 1), (90, 2)], seed=1), 0.5, "f32")


def test_paged_fwd_token_strides_past_the_chunk_tiles():
    """A token stride whose 256 rows no 31-bit offset reaches."""
    m = P.make("bf16", 2, 1, 64, 16, [(30, 140), (3, 1)], seed=3)
    d = P.to_device(m)
    wide = torch.empty((m["N"], 1 << 22), dtype=torch.bfloat16, device=DEV)
    view = wide[:, :128].unflatten(1, (2, 64))
    view.copy_(m["P1"])
    y = R.paged_fwd(view, d["cP2"], d["cV"], d["table"], d["total"], d["cu"], m["tau"], 0.5, max_new=140)
    torch.cuda.synchronize()
    ref, spread = PO.paged_fwd(P.f64(m["P1"]), np.nan_to_num(P.f64(m["cP2"])), np.nan_to_num(P.f64(m["cV"])),
                               m["table"].numpy(), m["total"].numpy(), m["cu"].numpy(), m["tau"], 0.5,
                               np.zeros(tuple(m["P1"].shape)), 140, with_spread=True)
    assert np.all(np.abs(P.f64(y) - ref) <= P.bound(ref, spread, "bf16", 1e-6))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_caches_past_32_bit_offsets(dt):
    """Pages on both sides of 2^31 and 2^32 elements: written by the append, read by single tokens and chunks."""
    H, Hkv, d, page = 4, 2, 128, 256
    per = Hkv * page * d
    n_pages = (1 << 32) // per + 40
    reqs = [(600, 1), (100, 160), (300, 5)]
    m = P.make(dt, H, Hkv, d, page, reqs, seed=7)
    held = int(m["cP2"].shape[0])
    marks = [(1 << 31) // per, (1 << 32) // per]
    where = np.array([0, n_pages - 1] + [k + j for k in marks for j in (-2, -1, 0, 1)] + list(range(50, 50 + held)))[:held]
    big = [torch.empty((n_pages, Hkv, page, d), dtype=m["cP2"].dtype, device=DEV) for _ in range(2)]
    at = torch.from_numpy(where).to(DEV)
    for b, c in zip(big, (m["cP2"], m["cV"])):
        b[at] = c.to(DEV)
    small = m["table"].numpy()
    table = torch.from_numpy(np.where(small >= 0, where[np.clip(small, 0, None)], P.BAD).astype(np.int32)).to(DEV)
    dev = P.to_device(m)
    want = R.paged_fwd(dev["P1"], dev["cP2"], dev["cV"], dev["table"], dev["total"], dev["cu"], m["tau"], 0.5, max_new=160)
    got = R.paged_fwd(dev["P1"], *big, table, dev["total"], dev["cu"], m["tau"], 0.5, max_new=160)
    assert torch.equal(got, want)
    # The same rows appended: into the last row of each page that is used.
    n = len(where)
    x = torch.from_numpy(np.random.default_rng(1).standard_normal((n, 2 * Hkv, d))).to(m["cP2"].dtype).to(DEV)
    slot = i32(where * page + page - 1)
    R.paged_append(x[:, :Hkv], x[:, Hkv:], slot, *big)
    torch.cuda.synchronize()
    assert torch.equal(big[0][at][:, :, -1], x[:, :Hkv]) and torch.equal(big[1][at][:, :, -1], x[:, Hkv:])
    for b, c in zip(big, (m["cP2"], m["cV"])):
        np.testing.assert_array_equal(b[at][:, :, :-1].cpu().float().numpy(), c[:, :, :-1].float().numpy())


@pytest.mark.parametrize("dt,reqs", [("bf16", RAGGED), ("bf16", CHUNKS), ("f32", RAGGED)])
def test_paged_fwd_large_evidence(dt, reqs):
    """Evidence far beyond the exponent range of an unshifted exponential (|U| to some hundreds): the stabiliser moves.
    The products of the evidence are summed in fp32 over d = 64: off by at most 6 sqrt(64) 2^-24 of the sum of their
    magnitudes (below 5000: 64 products of mean 25 * 2 / pi), over sqrt(64): 1.8e-3; an exponent |E| below 300 adds
    |E| 2^-22 = 7e-5. So du < 2e-3."""
    check_fwd(P.make(dt, 4, 2, 64, 16, reqs, seed=5, scale=5.0), 0.5, dt, du=2e-3)


def test_paged_fwd_leaves_other_rows():
    """Refused, empty, oversized and inconsistent requests are skipped; the rest is computed."""
    m = P.make("bf16", 4, 2, 64, 16, [(10, 3), (0, 0), (40, 4), (7, 1), (30, 20), (5, 2), (2, 2)], seed=3, pad_rows=4)
    m["total"][2] = -1                                   # refused
    m["total"][3] = 0                                    # fewer cached rows than new ones
    m["total"][5] = (m["table"].shape[1]) * 16 + 1       # past its table row
    check_fwd(m, 0.5, "bf16", max_new=8)                 # request 4 has more than 8 new tokens
    cu = m["cu"].clone()
    m["cu"][-1] = m["N"] + 1                             # past the packed rows
    check_fwd(m, 0.5, "bf16", max_new=64)
    m["cu"] = cu
    m["cu"][0] = -2
    check_fwd(m, 0.5, "bf16", max_new=64)


@pytest.mark.parametrize("dt,reqs", [("bf16", DECODE), ("bf16", CHUNKS), ("f32", RAGGED)])
def test_paged_fwd_pages_outside_the_cache_read_as_zeros(dt, reqs):
    m = P.make(dt, 4, 2, 64, 16, reqs, seed=8)
    for b in range(len(reqs)):
        m["table"][b, 0] = [P.BAD, m["cP2"].shape[0], 2**31 - 1][b % 3]
    check_fwd(m, 0.5, dt)


def test_paged_fwd_shared_pages():
    """Requests whose tables name the same pages (a common beginning) read the same rows."""
    m = P.make("bf16", 8, 2, 128, 16, [(64, 5), (64, 5), (64, 1)], seed=4)
    m["table"][1, :4] = m["table"][0, :4]
    m["table"][2, :4] = m["table"][0, :4]
    check_fwd(m, 0.5, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_paged_fwd_equals_one_pass_rows(dt):
    """A prompt in one chunk and the same prompt token by token are the same rows of the forward."""
    T = 300
    m = P.make(dt, 2, 2, 64, 32, [(0, T)], seed=6)
    whole = P.f64(check_fwd(m, 0.5, dt))
    d = P.to_device(m)
    dense = [c[m["table"][0, :-1].long()].permute(1, 0, 2, 3).reshape(2, -1, 64)[:, :T] for c in (m["cP2"], m["cV"])]
    one = R.fwd(*(t.to(DEV).contiguous()[None] for t in (m["P1"].permute(1, 0, 2), *dense)), m["tau"], 0.5)
    steps = []
    for p in (0, 1, 31, 32, 200, T - 1):
        steps.append(R.paged_fwd(d["P1"][p:p + 1], d["cP2"], d["cV"], d["table"], i32([p + 1]), i32([0, 1]), m["tau"], 0.5))
        assert np.max(np.abs(P.f64(steps[-1])[0] - whole[p])) <= (3e-2 if dt == "bf16" else 1e-5)
    np.testing.assert_allclose(P.f64(one)[0].transpose(1, 0, 2), whole, atol=3e-2 if dt == "bf16" else 1e-5)


def test_paged_fwd_same_call_same_bits_and_shared_workspace():
    """Calls of different shapes on one stream through one workspace, twice each."""
    ms = [P.make("bf16", 8, 2, 128, 16, [(9000, 1), (300, 1), (5000, 4)], seed=1),
          P.make("bf16", 8, 8, 64, 16, CHUNKS, seed=2), P.make("f32", 4, 1, 48, 32, RAGGED, seed=3),
          P.make("bf16", 8, 2, 128, 32, CHUNKS + [filler(8)], seed=4)]
    need = max(R.paged_workspace_bytes(m["N"], len(m["total"]), m["P1"].shape[1], m["cP2"].shape[1], m["P1"].shape[2])
               for m in ms)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    first = [run_fwd(m, 0.5, None, ws=ws) for m in ms]
    for m, y in zip(ms[::-1], first[::-1]):
        assert torch.equal(run_fwd(m, 0.5, None, ws=ws), y)


# ---- together --------------------------------------------------------------------

class Server:
    """A serving loop over the three calls: requests of random prompts, fed in chunks, then token by token."""

    def __init__(self, dt, H, Hkv, d, page, n_pages, S, width, seed):
        self.rng = np.random.default_rng(seed)
        self.dt, self.shape, self.page, self.n_pages = W.torch_dtype(dt), (H, Hkv, d), page, n_pages
        self.cP2, self.cV = (torch.full((n_pages, Hkv, page, d), float("nan"), dtype=self.dt, device=DEV) for _ in range(2))
        self.table = torch.full((S, width), P.BAD, dtype=torch.int32, device=DEV)
        self.free = i32(self.rng.permutation(n_pages))
        self.n_free = i32([n_pages])
        self.lens = i32([0] * S)
        self.tau = self.rng.uniform(0.5, 2.0, H).astype(np.float32)
        self.theta = self.rng.uniform(-2, 2, Hkv // 2).astype(np.float32)
        self.rows = [[] for _ in range(S)]                       # raw (P1, P2, I) of each request's tokens
        self.ys = [[] for _ in range(S)]

    def step(self, n_new, N):
        H, Hkv, d = self.shape
        x = torch.from_numpy(self.rng.standard_normal((N, H + 2 * Hkv, d))).to(self.dt).to(DEV)
        nn = i32(n_new)
        cu, total, slot, pos, _ = R.page_map(self.lens, nn, self.table, self.free, self.n_free, N, self.page,
                                             self.n_pages, out=tuple(torch.empty(k, dtype=torch.int32, device=DEV) for k in
                                                                     (len(n_new) + 1, len(n_new), N, N)) + (self.n_free,))
        q = R.paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], slot, self.cP2, self.cV, P1=x[:, :H], pos=pos, rope="half",
                           theta=self.theta, pairing="B")
        y = R.paged_fwd(q, self.cP2, self.cV, self.table, total, cu, self.tau, 0.5, max_new=max(1, max(n_new)))
        torch.cuda.synchronize()
        tot, at = total.cpu().numpy(), cu.cpu().numpy()
        for b, n in enumerate(n_new):
            if n < 0:
                self.rows[b], self.ys[b] = [], []
            if tot[b] >= 0 and n > 0:
                self.rows[b].append(P.f64(x[at[b]:at[b + 1]]))
                self.ys[b].append(P.f64(y[at[b]:at[b + 1]]))
        self.lens = torch.where(total >= 0, total, self.lens)
        return tot

    def check(self, tol):
        H, Hkv, d = self.shape
        for b, rows in enumerate(self.rows):
            if not rows:
                continue
            x, y = np.concatenate(rows), np.concatenate(self.ys[b])
            T = len(x)
            assert T == int(self.lens[b])
            pos = np.arange(T)
            p1 = PR.rope(x[:, :H].transpose(1, 0, 2), pos, 1e4, "half")
            p2 = PR.rope(x[:, H:H + Hkv].transpose(1, 0, 2), pos, 1e4, "half")
            v = PR.givens_mix(x[:, H + Hkv:].transpose(1, 0, 2)[None], self.theta, "B")[0]
            for h in range(H):
                g = h // (H // Hkv)
                ref = RO.relation_head(p1[h], p2[g], v[g], self.tau[h], 0.5)
                assert np.max(np.abs(y[:, h] - ref)) <= tol, (b, h)


@pytest.mark.parametrize("dt,tol", [("bf16", 3e-2), ("f32", 2e-5)])
def test_serving_loop(dt, tol):
    """Prompts in chunks, single tokens, a refused request that is tried again, finished requests whose pages others
    take. bf16: P1, P2, I~ and Y are each rounded once more than in the forward's 2e-2 bar: half as much again."""
    s = Server(dt, 8, 2, 64, 16, 40, 4, 20, seed=9)
    s.step([70, 5, 0, 1], 80)
    s.step([1, 130, 33, 1], 165)
    s.check(tol)
    for _ in range(3):
        s.step([1, 1, 1, 1], 6)
    tot = s.step([1, 1, 290, 20], 312)                 # request 2 does not fit in what is free
    assert tot[2] == -1
    s.step([1, -1, 0, 1], 2)                           # request 1 ends and returns its pages
    tot = s.step([1, 150, 200, 1], 352)                # and others take them
    assert tot[1] == 150 and tot[2] > 0
    s.step([2, 1, 1, 3], 7)
    s.check(tol)
    held = sum(-(-int(n) // 16) for n in s.lens.cpu())
    assert held + int(s.n_free) == 40
    used = [int(s.table[b, k]) for b in range(4) for k in range(-(-int(s.lens[b]) // 16))]
    rest = s.free[:int(s.n_free)].cpu().tolist()
    assert sorted(used + rest) == list(range(40))


@pytest.mark.parametrize("N,H,page,width,steps", [
    (700, 8, 16, 60, (([0] * 6, [300, 1, 0, 30, 2, 129]), ([300, 0, 16, 800, 2, 129], [1] * 6),
                      ([301, 5, 0, 1, 3, 700], [40, 1, 300, 1, 1, 1]), ([10, 9, 8, 7, 6, 5], [0] * 6))),
    # Chunks on query tiles, single tokens, chunks in the scan, tiles again.
    (1500, 16, 64, 60, (([2300, 0, 0, 0, 0, 0], [1200, 1, 0, 200, 2, 65]), ([3500, 1, 16, 800, 2, 129], [1] * 6),
                        ([301, 5, 0, 1, 3, 700], [40, 1, 300, 1, 1, 1]), ([2048, 9, 832, 7, 6, 5], [1000, 0, 400, 0, 0, 0]))),
])
def test_paged_calls_replay_in_a_graph(N, H, page, width, steps):
    """The three calls captured once and replayed with new lengths and inputs, against the eager calls. The captured
    call's max_new covers every replay, and the batch is padded to its capacity. Tables and free list name the same
    pages; no step gives two tokens one slot (lengths of 2000 and 800 in the last one would, 48 of 1400: whose values
    stay is then open, and eager and replay differ)."""
    S, Hkv, d, n_pages = 6, 2, 64, 200
    rng = np.random.default_rng(2)
    lens, nn = torch.zeros(S, dtype=torch.int32, device=DEV), torch.zeros(S, dtype=torch.int32, device=DEV)
    base = rng.permutation(n_pages)
    x = torch.zeros((N, H + 2 * Hkv, d), dtype=torch.bfloat16, device=DEV)
    state = {}
    for name in ("graph", "eager"):
        state[name] = dict(table=torch.zeros((S, width), dtype=torch.int32, device=DEV), free=i32(base), n_free=i32([n_pages]),
                           cP2=torch.zeros((n_pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV),
                           cV=torch.zeros((n_pages, Hkv, page, d), dtype=torch.bfloat16, device=DEV),
                           out=tuple(torch.zeros(k, dtype=torch.int32, device=DEV) for k in (S + 1, S, N, N, 1)),
                           q=torch.zeros((N, H, d), dtype=torch.bfloat16, device=DEV),
                           Y=torch.zeros((N, H, d), dtype=torch.bfloat16, device=DEV),
                           ws=torch.empty(R.paged_workspace_bytes(N, S, H, Hkv, d), dtype=torch.uint8, device=DEV))

    def work(s):
        cu, total, slot, pos, _ = R.page_map(lens, nn, s["table"], s["free"], s["n_free"], N, page, n_pages, out=s["out"])
        R.paged_append(x[:, H:H + Hkv], x[:, H + Hkv:], slot, s["cP2"], s["cV"], P1=x[:, :H], pos=pos, rope="interleaved",
                       out=s["q"])
        R.paged_fwd(s["q"], s["cP2"], s["cV"], s["table"], total, cu, 1.0, 0.5, max_new=N, out=s["Y"], workspace=s["ws"])
        return [s["Y"], s["q"], s["table"], *s["out"]]

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
    for ln, n in steps:
        lens.copy_(i32(ln))
        nn.copy_(i32(n))
        x.copy_(torch.from_numpy(rng.standard_normal(tuple(x.shape))).to(torch.bfloat16))
        for s in state.values():
            s["free"].copy_(i32(base))
            s["Y"].fill_(0.0)
            s["table"].copy_(i32(np.arange(S * width).reshape(S, width) % n_pages))
        torch.cuda.synchronize()
        want = [t.clone() for t in work(state["eager"])]
        torch.cuda.synchronize()
        slots = want[5][want[5] >= 0].cpu().numpy()
        assert len(np.unique(slots)) == len(slots)
        for s in state.values():
            s["Y"].fill_(0.0)
            s["table"].copy_(i32(np.arange(S * width).reshape(S, width) % n_pages))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), k


def test_paged_calls_allocate_on_the_stream_they_are_given():
    """What a call allocates for a stream other than the current one is not taken by the current one's next tensors."""
    m = P.make("bf16", 8, 2, 128, 16, [(20000, 1), (300, 9), (0, 400)], seed=1, pad_rows=3)
    want = run_fwd(m, 0.5, None, fill=0.0)
    d = P.to_device(m)
    n = R.paged_workspace_bytes(m["N"], 3, 8, 2, 128)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        y = R.paged_fwd(d["P1"], d["cP2"], d["cV"], d["table"], d["total"], d["cu"], m["tau"], 0.5, max_new=m["max_new"],
                        stream=side)
        others = [torch.zeros(n, dtype=torch.uint8, device=DEV), torch.ones_like(y)]
        torch.cuda.synchronize()
        assert torch.equal(y, want) and float(others[1].min()) == 1.0
        x = torch.randn((m["N"], 4, 128), device=DEV, dtype=torch.bfloat16)
        slot, c = i32(np.arange(m["N"])), [torch.zeros_like(d["cP2"]) for _ in range(2)]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        q = R.paged_append(x[:, :2], x[:, 2:], slot, *c, P1=x, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(q, x)


def test_paged_calls_on_streams_at_once():
    """Calls on three streams at once, a workspace each, against the same calls one after another."""
    ms = [P.make("bf16", 8, 2, 128, 16, [(6000, 1), (300, 9), (0, 400)], seed=1), P.make("bf16", 4, 4, 64, 16, CHUNKS, seed=2),
          P.make("bf16", 8, 2, 128, 16, CHUNKS + [filler(8)], seed=3)]
    want = [run_fwd(m, 0.5, None) for m in ms]
    ds = [P.to_device(m) for m in ms]
    streams = [torch.cuda.Stream() for _ in ms]
    outs = [torch.full_like(y, 3.0) for y in want]
    torch.cuda.synchronize()
    for _ in range(5):
        for d, s, y in zip(ds, streams, outs):
            R.paged_fwd(d["P1"], d["cP2"], d["cV"], d["table"], d["total"], d["cu"], d["tau"], 0.5, max_new=d["max_new"],
                        out=y, stream=s, workspace=d.setdefault("ws", torch.empty(R.paged_workspace_bytes(
                            d["N"], len(d["total"]), d["P1"].shape[1], d["cP2"].shape[1], d["P1"].shape[2]),
                            dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for y, w in zip(outs, want):
        assert torch.equal(y, w)
