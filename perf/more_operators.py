"""Cases of the paged Relation Cache in 8 bits and of trees of drafted tokens: the
append that quantises rows as it writes them, the forward that reads them back, the
plan of a batch of trees, the forward of a tree's tokens over what is cached, and the
cut back to the tokens that were accepted.

Each case is one call of one of these. A batch packs the new tokens of S requests one
after another; request b has len_b cached tokens and n_b new ones. Where ``own`` is
false, ``run`` computes the plain form with elementary torch operations in 32 bits;
where it is true, it calls the library's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
ROPE_BASE = 10000.0
TEMP_BYTES = 4 << 30            # of one temporary of the plain forward
LOW, HIGH = -100, 119           # exponents of the scales


# ---- cases ------------------------------------------------------------------

def _append(name, N, H, Hkv, d, page, rope, mix, pad=0, fused=True, shape=1):
    return dict(name=name, op="append", N=N, H=H, Hkv=Hkv, d=d, page=page, rope=rope, mix=mix, pad=pad, fused=fused,
                shape=shape)


def _plan(name, S, new_lo, new_hi, words, chunks=0, chunk=0, pad=0, shape=1):
    return dict(name=name, op="plan", S=S, new_lo=new_lo, new_hi=new_hi, ctx_lo=0, ctx_hi=20000, words=words,
                chunks=chunks, chunk=chunk, pad=pad, shape=shape)


def _fwd(name, S, new_lo, new_hi, ctx_lo, ctx_hi, H, Hkv, d, page, pages, words=0, chunks=0, chunk=0, lam=0.5, scale=1.0,
         shape=1):
    return dict(name=name, op="fwd", S=S, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, H=H, Hkv=Hkv,
                d=d, page=page, pages=pages, words=words, chunks=chunks, chunk=chunk, lam=lam, scale=scale, shape=shape)


def _keep(name, S, new_lo, new_hi, ctx_hi, Hkv, d, page, pages, most, shape=1):
    return dict(name=name, op="keep", S=S, new_lo=new_lo, new_hi=new_hi, ctx_lo=0, ctx_hi=ctx_hi, Hkv=Hkv, d=d,
                page=page, pages=pages, most=most, chunks=0, chunk=0, shape=shape)


def listed():
    return [
        # The new tokens of one decode step into 8-bit pages, sliced from a fused projection.
        _append("append8_decode", 64, 32, 32, 128, 64, "interleaved", True),
        # Packed prompts into 8-bit pages, grouped heads, half-split rotary pairs, a padded tail.
        _append("append8_prompts", 16384, 32, 8, 128, 16, "half", True, pad=100),
        # A few small trees of drafted tokens: the smallest plan.
        _plan("plan_few", 8, 3, 12, 1),
        # A serving batch of trees of up to 60 nodes, with two chunks of prompts among them and a padded tail.
        _plan("plan_batch", 256, 1, 60, 2, chunks=2, chunk=500, pad=33),
        # One token of a short request over 8-bit pages: the smallest forward, where latency counts.
        _fwd("fwd8_one", 1, 1, 1, 300, 300, 8, 8, 64, 16, "e4m3"),
        # The decode batch of the benchmark (64 sequences of 1,024 to 4,096 cached rows, 32 heads of 128), in 8-bit pages.
        _fwd("fwd8_batch", 64, 1, 1, 1024, 4096, 32, 32, 128, 64, "e4m3", lam=0.0),
        # Chunks of prompts of odd lengths over what is cached of them in 8 bits.
        _fwd("fwd8_chunks", 6, 100, 1500, 0, 6000, 32, 8, 128, 32, "e4m3"),
        # Trees of drafted tokens over 16-bit pages, many requests of middling length.
        _fwd("tree_drafts", 48, 2, 24, 200, 9000, 16, 4, 64, 32, "bf16", words=1),
        # Larger trees over long requests in 8-bit pages.
        _fwd("tree8_long", 16, 20, 64, 2000, 30000, 32, 8, 128, 16, "e4m3", words=2, scale=1.5),
        # 32-bit pages, small heads, trees that begin with nothing cached among them.
        _fwd("tree_f32", 6, 5, 40, 0, 2000, 8, 2, 48, 16, "f32", words=2),
        # The accepted tokens of the drafts above: few rows move, few pages go back.
        _keep("keep_drafts", 48, 2, 24, 9000, 4, 64, 32, "bf16", 6),
        # A large batch of trees in 8-bit pages, cut back to the accepted path.
        _keep("keep8_many", 512, 20, 64, 2000, 8, 128, 16, "e4m3", 16),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: {m: max(work(c)[m] for c in listed() if c["op"] == op) for m in ("bytes", "flops")}
            for op in ("append", "plan", "fwd", "keep")}
    while True:
        kind = rng.random()
        shape = rng.randrange(1 << 20)
        page = rng.choice([16, 32, 64, 128, 256])
        d = rng.choice([32, 48, 64, 80, 128])
        Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        H = Hkv * rng.choice([1, 1, 2, 3, 4, 5, 8])
        if H > 64:
            continue
        if kind < 0.2:
            c = _append("", _log_int(rng, 1, 16384), H, Hkv, d, page, rng.choice(["none", "interleaved", "half"]),
                        rng.random() < 0.6 and Hkv % 2 == 0, pad=rng.choice([0, 0, 5, 61]), fused=rng.random() < 0.6,
                        shape=shape)
        elif kind < 0.35:
            hi = _log_int(rng, 1, 200)
            words = (hi + 31) // 32
            chunks = rng.choice([0, 0, 1, 3])
            c = _plan("", max(chunks, _log_int(rng, 1, 300)), rng.choice([1, hi]), hi, words, chunks=chunks,
                      chunk=32 * words + _log_int(rng, 1, 700), pad=rng.choice([0, 0, 9, 150]), shape=shape)
        elif kind < 0.5:
            hi = _log_int(rng, 1, 64)
            c = _keep("", _log_int(rng, 1, 512), rng.choice([1, hi]), hi, _log_int(rng, 1, 9000), Hkv, d, page,
                      rng.choice(["bf16", "f32", "e4m3"]), _log_int(rng, 1, 20), shape=shape)
            if c["S"] * c["ctx_hi"] * Hkv * d > 1 << 30:                        # the size of the caches
                continue
        else:
            pages = rng.choice(["e4m3", "e4m3", "e4m3", "bf16", "f32"])
            tree = pages != "e4m3" or rng.random() < 0.4
            ctx = _log_int(rng, 1, 60000)
            new = _log_int(rng, 1, 64) if tree else rng.choice([1, 1, _log_int(rng, 1, 16), _log_int(rng, 1, 3000)])
            S = _log_int(rng, 1, 100)
            if pages == "f32":
                ctx = min(ctx, 8000)
            words = (new + 31) // 32 if tree else 0
            c = _fwd("", S, rng.choice([1, new]), new, rng.choice([0, ctx // 3, ctx]), ctx, H, Hkv, d, page, pages,
                     words=words, chunks=rng.choice([0, 0, min(S, 2)]), chunk=32 * words + _log_int(rng, 1, 500),
                     lam=rng.choice([0.0, 0.5, 1.0]), scale=rng.choice([0.5, 1.0, 1.5]), shape=shape)
        w, top = work(c), most[c["op"]]
        slow = 8 if c.get("pages") == "f32" and c["op"] == "fwd" else 1
        if w["bytes"] <= top["bytes"] and slow * w["flops"] <= max(top["flops"], 1):
            del c["name"]
            return c


# ---- lengths, which the case alone gives -------------------------------------

def _lens(c):
    """(cached tokens, new tokens) of each request."""
    r = random.Random(c["shape"])
    ln = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["S"])]
    nn = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["S"])]
    for k in range(c["chunks"]):
        nn[(k * 7 + 3) % c["S"]] = c["chunk"]
    return ln, nn


def _kept(c, nn):
    r = random.Random(c["shape"] + 1)
    return [r.randint(0, min(c["most"], n)) for n in nn]


def _pages(n, page):
    return (n + page - 1) // page


def _row_bytes(c):
    """Of one cached row of one head, P2 and V."""
    return 2 * c["d"] + 2 if c["pages"] == "e4m3" else 2 * c["d"] * (2 if c["pages"] == "bf16" else 4)


def work(c):
    if c["op"] == "append":
        # The tokens read and P1 written in 16 bits, P2 and V written in 8 with a scale each; a slot and a position.
        n = c["N"]
        return {"bytes": n * (c["d"] * (4 * c["H"] + 4 * c["Hkv"] + 2 * c["Hkv"]) + 2 * c["Hkv"]) + 8 * n,
                "flops": n * c["d"] * (3 * ((c["H"] + c["Hkv"]) * (c["rope"] != "none") + c["Hkv"] * c["mix"])
                                       + 4 * c["Hkv"])}
    ln, nn = _lens(c)
    N, S = sum(nn), c["S"]
    if c["op"] == "plan":
        # Parents read, positions and the rows of the trees written.
        trees = sum(n for n in nn if n <= 32 * c["words"])
        return {"bytes": 4 * (2 * N + c["pad"] + trees * c["words"] + 2 * S + 1), "flops": 0}
    if c["op"] == "keep":
        # Each kept row read and written, the kept tokens, the lengths, and the pages that go back.
        kept = _kept(c, nn)
        back = sum(_pages(a + n, c["page"]) - _pages(a + k, c["page"]) for a, n, k in zip(ln, nn, kept))
        return {"bytes": 2 * sum(kept) * c["Hkv"] * _row_bytes(c) + 4 * (sum(kept) + 2 * back + 4 * S + 3), "flops": 0}
    T = sum(a + n for a, n in zip(ln, nn))
    tree = [n <= 32 * c["words"] for n in nn]
    # A tree's token sees what is cached and itself at the least (its ancestors are not counted), a chunk's all before.
    rows = sum(n * (a + 1) if t else n * a + n * (n + 1) // 2 for a, n, t in zip(ln, nn, tree))
    pages = sum(_pages(a + n, c["page"]) for a, n in zip(ln, nn))
    e = 4 if c["pages"] == "f32" else 2
    return {"bytes": 2 * N * c["H"] * c["d"] * e + T * c["Hkv"] * _row_bytes(c)
            + 4 * (pages + 2 * S + 1 + c["words"] * sum(n for n, t in zip(nn, tree) if t)),
            "flops": 4 * c["d"] * c["H"] * rows}


# ---- 8-bit rows -----------------------------------------------------------------

def _quantise(x):
    """Rows of x (last axis) as e4m3 values and the exponent k of each row's scale 2^k: the least one that leaves no
    value above 448, between LOW and HIGH."""
    m, e = torch.frexp(x.abs().amax(-1, keepdim=True).double())           # m in [0.5, 1)
    k = torch.where(m > 0.875, e - 8, e - 9)
    k = torch.where(m == 0, LOW, k).clamp(LOW, HIGH)
    q = (x * torch.exp2(-k.double()).to(x.dtype)).clamp(-448.0, 448.0)
    return q.to(torch.float8_e4m3fn), k[..., 0]


def _as_scale(k):
    return (k + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _scale_values(s):
    """2^k of each stored scale."""
    return torch.exp2(s.view(torch.uint8).float() - 127.0)


# ---- what a program holds before the call -------------------------------------

def _table(s, c, held, g, dev, spare=3):
    """Pages of the requests in an order of their own, as block table; returns their count."""
    n_pages, width = sum(held) + spare, max(max(held), 1)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + held, device=dev).cumsum(0)[:-1, None]
    col = torch.arange(width, device=dev)[None, :]
    s["table"] = torch.where(col < torch.tensor(held, device=dev)[:, None], perm[(first + col).clamp(max=n_pages - 1)],
                             -1).contiguous()
    return n_pages, perm[sum(held):]


def _caches(s, n_pages, Hkv, ps, d, pages, scale, g, dev):
    for name, size in (("cP2", scale), ("cV", 1.0)):
        x = torch.randn((n_pages, Hkv, ps, d), generator=g, device=dev, dtype=torch.float32) * size
        if pages == "e4m3":
            q, k = _quantise(x)
            s[name] = q
            s.setdefault("scale", torch.empty((n_pages, Hkv, 2, ps), dtype=torch.float8_e8m0fnu, device=dev))
            s["scale"].view(torch.uint8)[:, :, 0 if name == "cP2" else 1] = _as_scale(k).view(torch.uint8)
        else:
            s[name] = x.to(DTYPES[pages])


def _parents(cu, nn, g, dev):
    """A tree over the new tokens of each request: the first is its root, others hang on one of the six before them."""
    n = torch.tensor(nn, device=dev)
    k = torch.arange(sum(nn), device=dev) - torch.repeat_interleave(cu[:-1].long(), n)
    u = torch.rand(sum(nn), generator=g, device=dev)
    return torch.where(k == 0, -1, (k - 1 - (u * torch.minimum(k, torch.full_like(k, 6))).long()).clamp(min=0)).to(torch.int32)


def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c}

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def normal(shape, dt, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dt)

    if c["op"] == "append":
        H, Hkv, d, ps = c["H"], c["Hkv"], c["d"], c["page"]
        n, rows = c["N"], c["N"] + c["pad"]
        r = random.Random(c["shape"])
        start = [r.randint(0, 5000) for _ in range(1 + n // 300)]
        pos = torch.tensor([start[t // 300] + t % 300 for t in range(n)] + [-1] * c["pad"], dtype=torch.int32)
        n_pages = _pages(n, ps) + 64
        perm = torch.randperm(n_pages, generator=g, device=dev)
        t = torch.arange(n, device=dev)
        s["slot"] = torch.cat([perm[t // ps] * ps + t % ps, torch.full((c["pad"],), -1, device=dev)]).to(torch.int32)
        s["pos"], s["n"] = pos.to(dev), n
        bf = torch.bfloat16
        if c["fused"]:
            x = normal((rows, H + 2 * Hkv, d), bf)
            s["P1"], s["P2"], s["I"] = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        else:
            s["P1"], s["P2"], s["I"] = normal((rows, H, d), bf), normal((rows, Hkv, d), bf), normal((rows, Hkv, d), bf)
        r = random.Random(seed)
        s["theta"] = [r.uniform(-math.pi, math.pi) for _ in range(Hkv // 2)] if c["mix"] else None
        s["P1o"] = torch.zeros((rows, H, d), dtype=bf, device=dev)
        _caches(s, n_pages, Hkv, ps, d, "e4m3", 1.0, g, dev)
        return s

    ln, nn = _lens(c)
    total = [a + n for a, n in zip(ln, nn)]
    s["total"], s["ln"], s["nn"], s["max_new"] = i32(total), ln, nn, max(nn)
    s["cu"] = i32([sum(nn[:b]) for b in range(c["S"] + 1)])
    N = sum(nn)
    if c["op"] == "plan":
        N += c["pad"]
        s["parent"] = torch.cat([_parents(s["cu"], nn, g, dev), i32([-1] * c["pad"])])
        s["tree"] = torch.zeros((N, c["words"]), dtype=torch.int32, device=dev)
        s["pos"] = torch.zeros(N, dtype=torch.int32, device=dev)
        return s

    Hkv, d, ps = c["Hkv"], c["d"], c["page"]
    n_pages, spare = _table(s, c, [_pages(t, ps) for t in total], g, dev, spare=3 if c["op"] == "fwd" else 17)
    if c["op"] == "keep":
        kept = _kept(c, nn)
        _caches(s, n_pages, Hkv, ps, d, c["pages"], 1.0, g, dev)
        # Each request keeps a growing choice of its new tokens: random keys, the kept ones in order.
        n, want = torch.tensor(nn, device=dev), torch.tensor(kept, device=dev)
        col = torch.arange(max(nn), device=dev)[None, :]
        key = torch.rand((c["S"], max(nn)), generator=g, device=dev).masked_fill(col >= n[:, None], 2.0)
        rank = key.argsort(1).argsort(1)
        place = torch.where(rank < want[:, None], col, max(nn)).sort(1).values
        s["keep"] = torch.where(col < want[:, None], place, -1)[col < n[:, None]].to(torch.int32)
        s["n_keep"] = i32(kept)
        s["lens"] = i32(ln)
        s["free"] = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        s["free"][:spare.numel()] = spare
        s["n_free"], s["n_free_out"] = i32([spare.numel()]), i32([0])
        return s

    H = c["H"]
    dt = torch.float32 if c["pages"] == "f32" else torch.bfloat16
    s["P1"] = normal((N, H, d), dt, c["scale"])
    _caches(s, n_pages, Hkv, ps, d, c["pages"], c["scale"], g, dev)
    r = random.Random(seed)
    s["tau"] = [r.uniform(0.5, 2.0) for _ in range(H)]
    s["tau_dev"] = torch.tensor(s["tau"], dtype=torch.float32, device=dev)
    s["Y"] = torch.zeros((N, H, d), dtype=dt, device=dev)
    s["tree"] = None
    if c["words"]:
        s["tree"] = _plain_trees(_parents(s["cu"], nn, g, dev), s["cu"], nn, c["words"])[0]
    if own:
        from causal_self_exchange_amd import relation as R
        s["ws"] = torch.empty(R.paged_workspace_bytes(N, c["S"], H, Hkv, d), dtype=torch.uint8, device=dev)
    return s


# ---- one pass ----------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    if own:
        from causal_self_exchange_amd import relation as R
        if c["op"] == "append":
            R.paged_append(s["P2"], s["I"], s["slot"], s["cP2"], s["cV"], P1=s["P1"], pos=s["pos"], rope=c["rope"],
                           rope_base=ROPE_BASE, theta=s["theta"], out=s["P1o"], scale=s["scale"])
            return {"P1": s["P1o"], "P2": s["cP2"], "V": s["cV"], "scale": s["scale"]}
        if c["op"] == "plan":
            tree, pos = R.tree_plan(s["parent"], s["total"], s["cu"], c["words"], out=(s["tree"], s["pos"]))
            return {"tree": tree, "pos": pos}
        if c["op"] == "keep":
            R.paged_keep(s["cP2"], s["cV"], s["table"], s["total"], s["cu"], s["keep"], s["n_keep"], s["lens"], s["free"],
                         s["n_free"], n_free_out=s["n_free_out"], scale=s.get("scale"))
            return _kept_state(s)
        return R.paged_fwd(s["P1"], s["cP2"], s["cV"], s["table"], s["total"], s["cu"], s["tau"], c["lam"],
                           max_new=s["max_new"], out=s["Y"], workspace=s["ws"], scale=s.get("scale"), tree=s["tree"])
    return {"append": _plain_append, "plan": _plain_plan, "fwd": _plain_fwd, "keep": _plain_keep}[c["op"]](s)


def _kept_state(s):
    out = {"P2": s["cP2"], "V": s["cV"], "len": s["lens"], "free": s["free"], "n_free": s["n_free_out"]}
    if "scale" in s:
        out["scale"] = s["scale"]
    return out


def _turn(x, pos, rope):
    """Rotary pairs of [n, heads, d] in 32 bits, the angles in 64."""
    if rope == "none":
        return x
    d = x.shape[-1]
    k = torch.arange(d // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[:, None] * ROPE_BASE ** (-2.0 * k / d)
    cs, sn = ang.cos().float()[:, None, :], ang.sin().float()[:, None, :]
    if rope == "half":
        a, b = x[..., :d // 2], x[..., d // 2:]
        return torch.cat([a * cs - b * sn, a * sn + b * cs], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cs - b * sn, a * sn + b * cs], -1).reshape(x.shape)


def _plain_append(s):
    c, n = s["c"], s["n"]
    ps = c["page"]
    pos, slot = s["pos"][:n], s["slot"][:n].long()
    page, off = slot // ps, slot % ps
    s["P1o"][:n] = _turn(s["P1"][:n].float(), pos, c["rope"]).to(s["P1o"].dtype)
    info = s["I"][:n].float()
    if s["theta"] is not None:
        th = torch.tensor(s["theta"], device=info.device, dtype=torch.float64)
        cs, sn = th.cos().float()[:, None], th.sin().float()[:, None]
        a, b = info[:, 0::2], info[:, 1::2]
        info = torch.stack([cs * a - sn * b, sn * a + cs * b], 2).reshape(info.shape)
    scale = s["scale"].view(torch.uint8)
    q, k = _quantise(_turn(s["P2"][:n].float(), pos, c["rope"]))
    s["cP2"][page, :, off] = q
    scale[page, :, 0, off] = (k + 127).to(torch.uint8)
    q, k = _quantise(info)
    s["cV"][page, :, off] = q
    scale[page, :, 1, off] = (k + 127).to(torch.uint8)
    return {"P1": s["P1o"], "P2": s["cP2"], "V": s["cV"], "scale": s["scale"]}


def _plain_trees(parent, cu, nn, words):
    """Rows of ancestor bits [N, words] and depths [N] of the packed tokens; requests of more than 32 words tokens are
    chunks: no bits, the depth of a token is its place."""
    dev, N = parent.device, parent.shape[0]
    S = len(nn)
    n = torch.tensor(nn, device=dev)
    Q = 32 * words
    k = torch.arange(Q, device=dev)
    live = (k[None, :] < n[:, None]) & (n <= Q)[:, None]                     # [S, Q]
    at = (cu[:-1].long()[:, None] + k).clamp(max=N - 1)
    p = torch.where(live, parent[at].long(), -1)
    p = torch.where((p >= 0) & (p < k), p, -1)
    reach = (p[:, :, None] == k).float()                                     # token, ancestor
    for _ in range(max(1, (Q - 1).bit_length())):                            # paths of twice the length each time
        reach = (reach + torch.matmul(reach, reach.contiguous())).clamp(max=1.0)
    bits = (reach.reshape(S, Q, words, 32).long() << torch.arange(32, device=dev)).sum(3)
    bits = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    tree = torch.zeros((N, words), dtype=torch.int32, device=dev)
    tree[at[live]] = bits[live]
    depth = torch.zeros(N, dtype=torch.long, device=dev)
    depth[:sum(nn)] = torch.arange(sum(nn), device=dev) - torch.repeat_interleave(cu[:-1].long(), n)
    depth[at[live]] = reach.sum(2).long()[live]
    return tree, depth


def _plain_plan(s):
    nn, N = s["nn"], s["parent"].shape[0]
    tree, depth = _plain_trees(s["parent"], s["cu"], nn, s["c"]["words"])
    n = torch.tensor(nn, device=tree.device)
    ctx = torch.repeat_interleave(s["total"].long() - n, n)
    s["tree"].copy_(tree)
    s["pos"].fill_(-1)
    s["pos"][:sum(nn)] = (ctx + depth[:sum(nn)]).to(torch.int32)
    return {"tree": s["tree"], "pos": s["pos"]}


def _plain_fwd(s):
    """Requests of like sizes at once, padded, as many as the temporaries allow; a long one by itself."""
    c = s["c"]
    H, Hkv, d, ps = c["H"], c["Hkv"], c["d"], c["page"]
    G, dev, b = H // Hkv, s["P1"].device, 0
    cu = [0]
    for n in s["nn"]:
        cu.append(cu[-1] + n)
    while b < c["S"]:
        e, qm, tm = b, 0, 0
        while e < c["S"]:
            q2, t2 = max(qm, s["nn"][e]), max(tm, s["ln"][e] + s["nn"][e])
            if e > b and (e + 1 - b) * t2 * max(H * q2, Hkv * d) * 4 > TEMP_BYTES:
                break
            e, qm, tm = e + 1, q2, t2
        nb = e - b
        tok = torch.arange(qm, device=dev)
        j = torch.arange(tm, device=dev)
        new = torch.tensor(s["nn"][b:e], device=dev)
        total = s["total"][b:e].long()
        ctx = total - new
        live = tok[None, :] < new[:, None]
        row = (s["cu"][b:e].long()[:, None] + tok).clamp(max=s["P1"].shape[0] - 1)
        page = s["table"][b:e].long()[:, :_pages(tm, ps)].clamp(min=0)

        def rows(cache, part):                                                  # [nb, Hkv, tm, d]
            x = cache[page].float()
            if "scale" in s:
                x *= _scale_values(s["scale"])[page][:, :, :, part, :, None]
            x = x.permute(0, 2, 1, 3, 4).reshape(nb, Hkv, -1, d)[:, :, :tm]
            return torch.where((j < total[:, None])[:, None, :, None], x, 0.0).contiguous()

        k, v = rows(s["cP2"], 0), rows(s["cV"], 1)
        own_row = (ctx[:, None] + tok).clamp(max=tm - 1)                          # [nb, qm]
        seen = j < own_row[:, :, None]
        if s["tree"] is not None:
            # Bit (row, j - ctx) of the trees; chunks see all rows before their own.
            o = (j - ctx[:, None])[:, None, :].expand(nb, qm, tm)
            w = s["tree"][row].long().gather(2, (o >> 5).clamp(0, c["words"] - 1))
            bit = ((w >> (o & 31)) & 1) == 1
            seen = seen & ((o < 0) | bit | (new > 32 * c["words"])[:, None, None])
        q = s["P1"][row].float().reshape(nb, qm, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(nb, Hkv, G * qm, d)
        u = torch.matmul(q.contiguous(), k.transpose(2, 3).contiguous()) / math.sqrt(d)
        u = u.reshape(nb, Hkv, G, qm, tm)
        at = own_row[:, None, None, :, None].expand(nb, Hkv, G, qm, 1)
        self_u = u.gather(4, at) / s["tau_dev"].reshape(1, Hkv, G, 1, 1)
        self_s = 1.0 / (1.0 + (-self_u).exp())
        r = u / (1.0 + (-u).exp())
        r -= c["lam"] * (seen.sum(2) + 1).float().log()[:, None, None, :, None]
        r = torch.where(seen[:, None, None], r, -math.inf)
        r.scatter_(4, at, self_s)
        r = (r - r.amax(4, keepdim=True)).exp_()
        z = r.sum(4, keepdim=True)
        y = torch.matmul(r.reshape(nb, Hkv, G * qm, tm), v).reshape(nb, Hkv, G, qm, d) / z
        y = y.permute(0, 3, 1, 2, 4).reshape(nb, qm, H, d).to(s["Y"].dtype)
        s["Y"][cu[b]:cu[e]] = y.reshape(nb * qm, H, d) if nb * qm == cu[e] - cu[b] else y[live]
        b = e
    return s["Y"]


def _plain_keep(s):
    c = s["c"]
    ps, F, width = c["page"], s["free"].numel(), s["table"].shape[1]
    dev = s["free"].device
    cu, total, n = s["cu"].long(), s["total"].long(), s["n_keep"].long()
    ctx = total - (cu[1:] - cu[:-1])
    col = torch.arange(c["most"], device=dev)[None, :]
    live = col < n[:, None]
    pick = s["keep"][(cu[:-1, None] + col).clamp(max=s["keep"].numel() - 1)].long()
    src, dst = (ctx[:, None] + pick)[live], (ctx[:, None] + col)[live]
    b = torch.arange(c["S"], device=dev)[:, None].expand(live.shape)[live]
    sp, dp = s["table"][b, src // ps].long(), s["table"][b, dst // ps].long()
    so, do = src % ps, dst % ps
    for cache in (s["cP2"], s["cV"]):
        cache[dp, :, do] = cache[sp, :, so]
    if "scale" in s:
        x = s["scale"].view(torch.uint8)
        x[dp, :, :, do] = x[sp, :, :, so]
    s["lens"].copy_((ctx + n).to(torch.int32))
    # Pages behind the last kept row go on top of the free list, in order.
    page = torch.arange(width, device=dev)[None, :]
    back = ((page >= ((ctx + n + ps - 1) // ps)[:, None]) & (page < ((total + ps - 1) // ps)[:, None])).reshape(-1)
    have = s["n_free"].long().clamp(0, F)
    place = have + back.cumsum(0) - 1
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free.scatter_(0, torch.where(back & (place < F), place, F), s["table"].reshape(-1))
    s["free"].copy_(free[:F])
    s["n_free_out"].copy_((have + back.sum()).clamp(max=F).to(torch.int32))
    return _kept_state(s)


# ---- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "plan":
        return _exact_plan(s)
    if c["op"] == "keep":
        return _exact_keep(s)
    H, Hkv, d, ps = c["H"], c["Hkv"], c["d"], c["page"]
    out = torch.zeros(s["Y"].shape, dtype=torch.float64, device=s["Y"].device)
    trees = s["tree"].cpu().tolist() if s["tree"] is not None else None
    t0 = 0
    for b in range(c["S"]):
        L, n = s["ln"][b], s["nn"][b]
        T = L + n
        pages = s["table"][b, :_pages(T, ps)].long()
        blind = torch.ones((n, T), dtype=torch.bool).triu(L)                     # [token, row]: rows not seen
        if trees is not None and n <= 32 * c["words"]:
            new = [[not (trees[t0 + i][a // 32] >> (a % 32)) & 1 or a >= i for a in range(n)] for i in range(n)]
            blind[:, L:] = torch.tensor(new)
        blind = blind.to(out.device)
        count = (~blind).sum(1).double() + 1.0
        for g in range(Hkv):
            p2, val = s["cP2"][pages, g].double(), s["cV"][pages, g].double()
            if "scale" in s:
                e = s["scale"][pages, g].view(torch.uint8).double() - 127.0
                p2, val = p2 * 2.0 ** e[:, 0, :, None], val * 2.0 ** e[:, 1, :, None]
            p2, val = p2.reshape(-1, d)[:T], val.reshape(-1, d)[:T]
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                p1 = s["P1"][t0:t0 + n, h].double()
                ev = p1 @ p2.t() * d ** -0.5
                own_ev = (p1 * p2[L:]).sum(1) * d ** -0.5
                logit = ev * torch.sigmoid(ev) - c["lam"] * torch.log(count)[:, None]
                logit[blind] = -math.inf
                i = torch.arange(n, device=out.device)
                logit[i, L + i] = torch.sigmoid(own_ev / s["tau_dev"][h].double())
                out[t0:t0 + n, h] = torch.softmax(logit, 1) @ val
        t0 += n
    return out


def _exact_append(s):
    c, n = s["c"], s["n"]
    d, ps = c["d"], c["page"]

    def turned(x):
        x = x[:n].double().clone()
        if c["rope"] != "none":
            for k in range(d // 2):
                a, b = (k, k + d // 2) if c["rope"] == "half" else (2 * k, 2 * k + 1)
                ang = (s["pos"][:n].double() * ROPE_BASE ** (-2.0 * k / d))[:, None]
                u, v = x[:, :, a].clone(), x[:, :, b].clone()
                x[:, :, a], x[:, :, b] = u * ang.cos() - v * ang.sin(), u * ang.sin() + v * ang.cos()
        return x

    def stored(x):
        """The nearest e4m3 value (ties to even) of each element over its row's scale, and the scales."""
        top = x.abs().amax(-1, keepdim=True)
        k = torch.ceil(torch.log2(top / 448.0))
        k = torch.where(448.0 * 2.0 ** (k - 1) >= top, k - 1, torch.where(448.0 * 2.0 ** k < top, k + 1, k))
        k = torch.where(top > 0, k.clamp(LOW, HIGH), float(LOW))
        y = x / 2.0 ** k
        step = 2.0 ** (torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
        return torch.round(y / step) * step, 2.0 ** k[..., 0]

    info = s["I"][:n].double().clone()
    for k, th in enumerate(s["theta"] or []):
        u, v = info[:, 2 * k].clone(), info[:, 2 * k + 1].clone()
        info[:, 2 * k] = math.cos(th) * u - math.sin(th) * v
        info[:, 2 * k + 1] = math.sin(th) * u + math.cos(th) * v
    at = s["slot"][:n].long()
    p1, cp2, cv = s["P1o"].double(), s["cP2"].double(), s["cV"].double()
    scale = 2.0 ** (s["scale"].view(torch.uint8).double() - 127.0)
    p1[:n] = turned(s["P1"])
    cp2[at // ps, :, at % ps], scale[at // ps, :, 0, at % ps] = stored(turned(s["P2"]))
    cv[at // ps, :, at % ps], scale[at // ps, :, 1, at % ps] = stored(info)
    return {"P1": p1, "P2": cp2, "V": cv, "scale": scale}


def _exact_plan(s):
    c, parent = s["c"], s["parent"].tolist()
    N, W = len(parent), c["words"]
    tree, pos, t0 = [[0] * W for _ in range(N)], [-1] * N, 0
    for L, n in zip(s["ln"], s["nn"]):
        for k in range(n):
            if n > 32 * W:
                pos[t0 + k] = L + k
                continue
            up, m = parent[t0 + k], 0
            bits = 0
            while 0 <= up:
                bits |= 1 << up
                m += 1
                up = parent[t0 + up]
            pos[t0 + k] = L + m
            for w in range(W):
                x = bits >> (32 * w) & 0xffffffff
                tree[t0 + k][w] = x - (1 << 32) if x >> 31 else x
        t0 += n
    return {"tree": torch.tensor(tree, dtype=torch.int32), "pos": torch.tensor(pos, dtype=torch.int32)}


def _exact_keep(s):
    c, ps = s["c"], s["c"]["page"]
    table, keep, n_keep, free, have = s["table"].tolist(), s["keep"].tolist(), s["n_keep"].tolist(), s["free"].tolist(), int(s["n_free"])
    caches = {"P2": s["cP2"].double(), "V": s["cV"].double()}
    if "scale" in s:
        caches["scale"] = 2.0 ** (s["scale"].view(torch.uint8).double() - 127.0)
        caches["scale"] = caches["scale"].transpose(2, 3)                      # rows third, as in the others
    lens, t0 = [], 0
    for b, (L, n) in enumerate(zip(s["ln"], s["nn"])):
        for k in range(n_keep[b]):
            src, dst = L + keep[t0 + k], L + k
            if src != dst:
                for x in caches.values():
                    x[table[b][dst // ps], :, dst % ps] = x[table[b][src // ps], :, src % ps]
        lens.append(L + n_keep[b])
        for p in range(_pages(lens[-1], ps), _pages(L + n, ps)):
            if have < len(free):
                free[have] = table[b][p]
                have += 1
        t0 += n
    i = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    if "scale" in caches:
        caches["scale"] = caches["scale"].transpose(2, 3).contiguous()
    return caches | {"len": i(lens), "free": i(free), "n_free": i([have])}
