"""Cases of the paged Relation Cache: the page map, the append of a packed
batch of new tokens, and the Relation forward of those tokens over the pages.

Each case is one call of one of the three. A batch packs the new tokens of S
requests one after another; request b has len_b cached tokens and n_b new ones.
Where ``own`` is false, ``run`` computes the plain form with elementary torch
operations in 32 bits; where it is true, it calls the library's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ROPE_BASE = 10000.0
TEMP_BYTES = 4 << 30            # of one temporary of the plain forward


# ---- cases ------------------------------------------------------------------

def _map(name, S, len_hi, new_lo, new_hi, page, release=0.0, pad=0, free=1.0, shape=1):
    return dict(name=name, op="map", S=S, len_hi=len_hi, new_lo=new_lo, new_hi=new_hi, page=page, release=release,
                pad=pad, free=free, shape=shape)


def _append(name, N, H, Hkv, d, page, dtype, rope, mix, pad=0, fused=True, shape=1):
    return dict(name=name, op="append", N=N, H=H, Hkv=Hkv, d=d, page=page, dtype=dtype, rope=rope, mix=mix, pad=pad,
                fused=fused, shape=shape)


def _fwd(name, S, new_lo, new_hi, ctx_lo, ctx_hi, H, Hkv, d, page, dtype="bf16", chunks=0, chunk=0, lam=0.5,
         scale=1.0, shape=1):
    return dict(name=name, op="fwd", S=S, new_lo=new_lo, new_hi=new_hi, ctx_lo=ctx_lo, ctx_hi=ctx_hi, H=H, Hkv=Hkv,
                d=d, page=page, dtype=dtype, chunks=chunks, chunk=chunk, lam=lam, scale=scale, shape=shape)


def listed():
    return [
        # One decode step of a serving batch: every request adds one token, a few need a new page.
        _map("map_decode", 256, 4096, 1, 1, 16),
        # Prompts admitted while finished requests give their pages back; the free list runs out near the end and the
        # batch is padded behind its last token.
        _map("map_prompts", 1024, 2000, 1, 130, 16, release=0.1, pad=77, free=0.9),
        # The new tokens of one decode step, sliced from a fused projection: rotary coordinates and mixed heads.
        _append("append_decode", 64, 32, 32, 128, 64, "bf16", "interleaved", True),
        # The tokens of packed prompts with grouped heads, half-split rotary pairs, a padded tail.
        _append("append_prompts", 16384, 32, 8, 128, 16, "bf16", "half", True, pad=100),
        # A single short request with small heads: the smallest call, where latency counts.
        _fwd("decode_one", 1, 1, 1, 300, 300, 8, 8, 64, 16),
        # The decode batch of the benchmark (64 sequences of 1,024 to 4,096 cached rows, 32 heads of 128), paged.
        _fwd("decode_batch", 64, 1, 1, 1024, 4096, 32, 32, 128, 64, lam=0.0),
        # Few requests with long caches and eight query heads per cached head.
        _fwd("decode_long", 8, 1, 1, 32768, 131072, 32, 4, 128, 16, scale=1.5),
        # Several tokens per request (drafted tokens to be checked), ragged, odd lengths.
        _fwd("drafts", 48, 2, 7, 200, 9000, 16, 4, 64, 32),
        # Whole prompts of different lengths, packed, nothing cached before.
        _fwd("prompts", 5, 500, 6000, 0, 0, 32, 8, 128, 64),
        # One chunk of a long prompt over what is cached of it.
        _fwd("chunk_long", 1, 2048, 2048, 30001, 30001, 32, 8, 128, 128),
        # A serving batch that mixes decode steps with two prompt chunks, in the smallest pages.
        _fwd("mixed", 40, 1, 1, 100, 8000, 8, 8, 80, 16, chunks=2, chunk=1111),
        # 32-bit caches, chunks of odd lengths, grouped heads of 48.
        _fwd("chunks_f32", 6, 1, 97, 0, 2000, 8, 2, 48, 16, dtype="f32"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {op: {m: max(work(c)[m] for c in listed() if c["op"] == op) for m in ("bytes", "flops")}
            for op in ("map", "append", "fwd")}
    while True:
        kind = rng.random()
        shape = rng.randrange(1 << 20)
        page = rng.choice([16, 32, 64, 128, 256])
        if kind < 0.2:
            hi = _log_int(rng, 1, 300)
            c = _map("", _log_int(rng, 1, 1024), _log_int(rng, 1, 6000), rng.choice([0, 1, 1]), hi, page,
                     release=rng.choice([0.0, 0.1, 0.5]), pad=rng.choice([0, 0, 13, 200]),
                     free=rng.choice([0.5, 0.95, 1.2]), shape=shape)
        else:
            d = rng.choice([32, 48, 64, 80, 128])
            Hkv = rng.choice([1, 2, 3, 4, 8, 16, 32])
            H = Hkv * rng.choice([1, 1, 2, 3, 4, 5, 8])
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            if H > 64:
                continue
            if kind < 0.4:
                c = _append("", _log_int(rng, 1, 16384), H, Hkv, d, page, dtype,
                            rng.choice(["none", "interleaved", "half"]), rng.random() < 0.6 and Hkv % 2 == 0,
                            pad=rng.choice([0, 0, 5, 61]), fused=rng.random() < 0.6, shape=shape)
            else:
                ctx = _log_int(rng, 1, 60000)
                new = rng.choice([1, 1, _log_int(rng, 1, 16), _log_int(rng, 1, 5000)])
                S = _log_int(rng, 1, 100)
                if dtype == "f32":
                    new, ctx = min(new, 700), min(ctx, 8000)
                c = _fwd("", S, rng.choice([1, new]), new, rng.choice([0, ctx // 3, ctx]), ctx, H, Hkv, d, page,
                         dtype=dtype, chunks=rng.choice([0, 0, min(S, 2)]), chunk=_log_int(rng, 1, 1500),
                         lam=rng.choice([0.0, 0.5, 1.0]), scale=rng.choice([0.5, 1.0, 1.5]), shape=shape)
                if dtype == "f32":
                    c["chunk"] = min(c["chunk"], 700)
        w, top = work(c), most[c["op"]]
        slow = 8 if c.get("dtype") == "f32" and c["op"] == "fwd" else 1
        if w["bytes"] <= top["bytes"] and slow * w["flops"] <= max(top["flops"], 1):
            del c["name"]
            return c


# ---- lengths, which the case alone gives -------------------------------------

def _lens(c):
    """(cached tokens, new tokens) of each request; new = -1 for a finished request."""
    r = random.Random(c["shape"])
    if c["op"] == "map":
        ln = [r.randint(0, c["len_hi"]) for _ in range(c["S"])]
        nn = [-1 if r.random() < c["release"] else r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["S"])]
        return ln, nn
    ln = [r.randint(c["ctx_lo"], c["ctx_hi"]) for _ in range(c["S"])]
    nn = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["S"])]
    for k in range(c["chunks"]):
        nn[(k * 7 + 3) % c["S"]] = c["chunk"]
    return ln, nn


def _pages(n, page):
    return (n + page - 1) // page


def work(c):
    if c["op"] == "map":
        ln, nn = _lens(c)
        N = sum(max(n, 0) for n in nn) + c["pad"]
        moved = sum(_pages(ln[b], c["page"]) if n < 0 else _pages(ln[b] + n, c["page"]) - _pages(ln[b], c["page"])
                    for b, n in enumerate(nn))
        # Lengths and counts read; totals and offsets written; each page moved between list and table; the partly
        # filled page of each request read; a slot and a position written per token.
        return {"bytes": 4 * (2 * c["S"] + 2 * c["S"] + 1 + 2 * moved + c["S"] + 2 * N), "flops": 0}
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        n = c["N"]
        return {"bytes": n * c["d"] * e * (2 * c["H"] + 4 * c["Hkv"]) + 8 * n,
                "flops": n * c["d"] * 3 * ((c["H"] + c["Hkv"]) * (c["rope"] != "none") + c["Hkv"] * c["mix"])}
    ln, nn = _lens(c)
    N, T = sum(nn), sum(a + b for a, b in zip(ln, nn))
    rows = sum(n * a + n * (n + 1) // 2 for a, n in zip(ln, nn))
    pages = sum(_pages(a + n, c["page"]) for a, n in zip(ln, nn))
    return {"bytes": e * c["d"] * (2 * N * c["H"] + 2 * T * c["Hkv"]) + 4 * (pages + 2 * c["S"] + 1),
            "flops": 4 * c["d"] * c["H"] * rows}


# ---- what a program holds before the call -------------------------------------

def prepare(case, seed):
    c, dev = case, torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = {"c": c}

    def i32(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def normal(shape, dt, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev, dtype=torch.float32) * scale).to(dt)

    if c["op"] == "map":
        ln, nn = _lens(c)
        ps = c["page"]
        held = [_pages(a, ps) for a in ln]
        need = sum(max(0, _pages(a + n, ps) - h) for a, n, h in zip(ln, nn, held) if n > 0)
        width = max(_pages(a + max(n, 0), ps) for a, n in zip(ln, nn)) + 2
        n_free = max(1, int(need * c["free"]))
        n_pages = sum(held) + n_free
        order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
        first = torch.tensor([0] + held, device=dev).cumsum(0)[:-1, None]
        col = torch.arange(width, device=dev)[None, :]
        at = (first + col).clamp(max=n_pages - 1)
        s["table"] = torch.where(col < torch.tensor(held, device=dev)[:, None], order[at], -1).contiguous()
        s["free"] = torch.full((n_pages,), -1, dtype=torch.int32, device=dev)
        s["free"][:n_free] = order[sum(held):]
        s["n_free"] = i32([n_free])
        s["len"], s["new"] = i32(ln), i32(nn)
        s["N"], s["n_pages"] = max(1, sum(max(n, 0) for n in nn) + c["pad"]), n_pages
        S = c["S"]
        s["out"] = (torch.zeros(S + 1, dtype=torch.int32, device=dev), torch.zeros(S, dtype=torch.int32, device=dev),
                    torch.zeros(s["N"], dtype=torch.int32, device=dev),
                    torch.zeros(s["N"], dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev))
        return s

    dt = DTYPES[c["dtype"]]
    H, Hkv, d, ps = c["H"], c["Hkv"], c["d"], c["page"]
    if c["op"] == "append":
        n, rows = c["N"], c["N"] + c["pad"]
        r = random.Random(c["shape"])
        start = [r.randint(0, 5000) for _ in range(1 + n // 300)]
        pos = torch.tensor([start[t // 300] + t % 300 for t in range(n)] + [-1] * c["pad"], dtype=torch.int32)
        n_pages = _pages(n, ps) + 64
        perm = torch.randperm(n_pages, generator=g, device=dev)
        t = torch.arange(n, device=dev)
        s["slot"] = torch.cat([perm[t // ps] * ps + t % ps, torch.full((c["pad"],), -1, device=dev)]).to(torch.int32)
        s["pos"], s["n"] = pos.to(dev), n
        if c["fused"]:
            x = normal((rows, H + 2 * Hkv, d), dt)
            s["P1"], s["P2"], s["I"] = x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:]
        else:
            s["P1"], s["P2"], s["I"] = normal((rows, H, d), dt), normal((rows, Hkv, d), dt), normal((rows, Hkv, d), dt)
        r = random.Random(seed)
        s["theta"] = [r.uniform(-math.pi, math.pi) for _ in range(Hkv // 2)] if c["mix"] else None
        s["P1o"] = torch.zeros((rows, H, d), dtype=dt, device=dev)
        s["cP2"], s["cV"] = normal((n_pages, Hkv, ps, d), dt), normal((n_pages, Hkv, ps, d), dt)
        return s

    ln, nn = _lens(c)
    total = [a + n for a, n in zip(ln, nn)]
    held = [_pages(t, ps) for t in total]
    n_pages, width, N = sum(held) + 3, max(held), sum(nn)
    perm = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    first = torch.tensor([0] + held, device=dev).cumsum(0)[:-1, None]
    col = torch.arange(width, device=dev)[None, :]
    s["table"] = torch.where(col < torch.tensor(held, device=dev)[:, None], perm[(first + col).clamp(max=n_pages - 1)],
                             -1).contiguous()
    s["total"] = i32(total)
    s["cu"] = i32([sum(nn[:b]) for b in range(c["S"] + 1)])
    s["P1"] = normal((N, H, d), dt, c["scale"])
    s["cP2"], s["cV"] = normal((n_pages, Hkv, ps, d), dt, c["scale"]), normal((n_pages, Hkv, ps, d), dt)
    r = random.Random(seed)
    s["tau"] = [r.uniform(0.5, 2.0) for _ in range(H)]
    s["tau_dev"] = torch.tensor(s["tau"], dtype=torch.float32, device=dev)
    s["Y"] = torch.zeros((N, H, d), dtype=dt, device=dev)
    s["ln"], s["nn"], s["max_new"] = ln, nn, max(nn)
    if own:
        from causal_self_exchange_amd import relation as R
        s["ws"] = torch.empty(R.paged_workspace_bytes(N, c["S"], H, Hkv, d), dtype=torch.uint8, device=dev)
    return s


# ---- one pass ----------------------------------------------------------------

def run(state):
    s, c = state, state["c"]
    if own:
        from causal_self_exchange_amd import relation as R
        if c["op"] == "map":
            cu, total, slot, pos, n_free = R.page_map(s["len"], s["new"], s["table"], s["free"], s["n_free"], s["N"],
                                                      c["page"], s["n_pages"], out=s["out"])
            return {"cu": cu, "total": total, "slot": slot, "pos": pos, "n_free": n_free, "table": s["table"],
                    "free": s["free"]}
        if c["op"] == "append":
            R.paged_append(s["P2"], s["I"], s["slot"], s["cP2"], s["cV"], P1=s["P1"], pos=s["pos"], rope=c["rope"],
                           rope_base=ROPE_BASE, theta=s["theta"], out=s["P1o"])
            return {"P1": s["P1o"], "P2": s["cP2"], "V": s["cV"]}
        return R.paged_fwd(s["P1"], s["cP2"], s["cV"], s["table"], s["total"], s["cu"], s["tau"], c["lam"],
                           max_new=s["max_new"], out=s["Y"], workspace=s["ws"])
    return {"map": _plain_map, "append": _plain_append, "fwd": _plain_fwd}[c["op"]](s)


def _plain_map(s):
    c = s["c"]
    ps, N, F, width = c["page"], s["N"], s["free"].numel(), s["table"].shape[1]
    dev = s["len"].device
    ln, nn = s["len"].long(), s["new"].long()
    q = nn.clamp(min=0)
    end = q.cumsum(0)
    cu = torch.cat([end.new_zeros(1), end])
    held = (ln + ps - 1) // ps
    fits = (ln >= 0) & (ln + q <= width * ps)
    ok = (nn >= 0) & fits & (end <= N)
    # Finished requests: their pages go on top of the free list, in order.
    gone = (nn == -1) & fits
    col = torch.arange(width, device=dev)[None, :]
    back = (gone[:, None] & (col < held[:, None])).reshape(-1)
    have = s["n_free"].long().clamp(0, F)
    place = have + back.cumsum(0) - 1
    free = torch.cat([s["free"], s["free"].new_zeros(1)])
    free.scatter_(0, torch.where(back & (place < F), place, F), s["table"].reshape(-1))
    s["free"].copy_(free[:F])
    have = (have + back.sum()).clamp(max=F)
    # Pages for the new tokens, from the top of the list, in order.
    need = torch.where(ok, (ln + q + ps - 1) // ps - held, 0)
    upto = need.cumsum(0)
    ok = ok & ((need == 0) | (upto <= have))
    take = have - 1 - (upto - need)[:, None] - (col - held[:, None])
    mine = ok[:, None] & (col >= held[:, None]) & (col < (held + need)[:, None])
    s["table"].copy_(torch.where(mine, free[take.clamp(0, F - 1)], s["table"]))
    total = torch.where(ok, ln + q, torch.where(gone, 0, -1))
    n_free = have - torch.where(ok, need, 0).sum()
    # Slots and positions of the packed tokens.
    t = torch.arange(N, device=dev)
    b = torch.searchsorted(end, t, right=True).clamp(max=c["S"] - 1)
    live = (t < end[-1]) & ok[b]
    at = ln[b] + t - cu[b]
    page = s["table"][b, (at // ps).clamp(0, width - 1)].long()
    slot = torch.where(live & (page >= 0) & (page < s["n_pages"]), page * ps + at % ps, -1)
    pos = torch.where(live, at, -1)
    i = torch.int32
    return {"cu": cu.to(i), "total": total.to(i), "slot": slot.to(i), "pos": pos.to(i), "n_free": n_free.to(i),
            "table": s["table"], "free": s["free"]}


def _turn(x, pos, rope):
    """Rotary pairs of [n, heads, d] in 32 bits, the angles in 64."""
    if rope == "none":
        return x
    n, _, d = x.shape
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
    dt = s["P1"].dtype
    ps = c["page"]
    pos, slot = s["pos"][:n], s["slot"][:n].long()
    s["P1o"][:n] = _turn(s["P1"][:n].float(), pos, c["rope"]).to(dt)
    s["cP2"][slot // ps, :, slot % ps] = _turn(s["P2"][:n].float(), pos, c["rope"]).to(dt)
    info = s["I"][:n].float()
    if s["theta"] is not None:
        th = torch.tensor(s["theta"], device=info.device, dtype=torch.float64)
        cs, sn = th.cos().float()[:, None], th.sin().float()[:, None]
        a, b = info[:, 0::2], info[:, 1::2]
        info = torch.stack([cs * a - sn * b, sn * a + cs * b], 2).reshape(info.shape)
    s["cV"][slot // ps, :, slot % ps] = info.to(dt)
    return {"P1": s["P1o"], "P2": s["cP2"], "V": s["cV"]}


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
        live = tok[None, :] < new[:, None]
        row = (s["cu"][b:e].long()[:, None] + tok).clamp(max=s["P1"].shape[0] - 1)
        pos = (total - new)[:, None] + tok                                     # [nb, qm]
        page = s["table"][b:e].long()[:, :_pages(tm, ps)].clamp(min=0)

        def rows(cache):                                                        # [nb, Hkv, tm, d]
            x = cache[page].float().permute(0, 2, 1, 3, 4).reshape(nb, Hkv, -1, d)[:, :, :tm]
            return torch.where((j < total[:, None])[:, None, :, None], x, 0.0).contiguous()

        k, v = rows(s["cP2"]), rows(s["cV"])
        q = s["P1"][row].float().reshape(nb, qm, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(nb, Hkv, G * qm, d)
        u = torch.matmul(q.contiguous(), k.transpose(2, 3).contiguous()) / math.sqrt(d)
        u = u.reshape(nb, Hkv, G, qm, tm)
        at = pos.clamp(max=tm - 1)[:, None, None, :, None].expand(nb, Hkv, G, qm, 1)
        self_u = u.gather(4, at) / s["tau_dev"].reshape(1, Hkv, G, 1, 1)
        self_s = 1.0 / (1.0 + (-self_u).exp())
        r = u / (1.0 + (-u).exp())
        r -= c["lam"] * (pos + 1).float().log()[:, None, None, :, None]
        r = torch.where(j < pos[:, None, None, :, None], r, -math.inf)
        r.scatter_(4, at, self_s)
        r = (r - r.amax(4, keepdim=True)).exp_()
        z = r.sum(4, keepdim=True)
        y = torch.matmul(r.reshape(nb, Hkv, G * qm, tm), v).reshape(nb, Hkv, G, qm, d) / z
        y = y.permute(0, 3, 1, 2, 4).reshape(nb, qm, H, d).to(s["Y"].dtype)
        s["Y"][cu[b]:cu[e]] = y.reshape(nb * qm, H, d) if nb * qm == cu[e] - cu[b] else y[live]
        b = e
    return s["Y"]


# ---- the definitions in 64 bits -------------------------------------------------

def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "map":
        return _exact_map(s)
    if c["op"] == "append":
        return _exact_append(s)
    H, Hkv, d, ps = c["H"], c["Hkv"], c["d"], c["page"]
    out = torch.zeros(s["Y"].shape, dtype=torch.float64, device=s["Y"].device)
    t0 = 0
    for b in range(c["S"]):
        L, n = s["ln"][b], s["nn"][b]
        T = L + n
        pages = s["table"][b, :_pages(T, ps)].long()
        seen = torch.arange(T, device=out.device)
        here = torch.arange(L, T, device=out.device)
        for h in range(H):
            g = h // (H // Hkv)
            p2 = s["cP2"][pages, g].reshape(-1, d)[:T].double()
            val = s["cV"][pages, g].reshape(-1, d)[:T].double()
            p1 = s["P1"][t0:t0 + n, h].double()
            ev = p1 @ p2.t() * d ** -0.5
            own_ev = (p1 * p2[L:]).sum(1) * d ** -0.5
            logit = ev * torch.sigmoid(ev) - c["lam"] * torch.log(here + 1.0)[:, None].double()
            logit[seen[None, :] >= here[:, None]] = -math.inf
            logit[torch.arange(n, device=out.device), here] = torch.sigmoid(own_ev / s["tau_dev"][h].double())
            out[t0:t0 + n, h] = torch.softmax(logit, 1) @ val
        t0 += n
    return out


def _exact_map(s):
    c, ps = s["c"], s["c"]["page"]
    ln, nn, table = s["len"].tolist(), s["new"].tolist(), s["table"].tolist()
    free, have = s["free"].tolist(), int(s["n_free"])
    width, F, N = len(table[0]), len(free), s["N"]
    for b in range(c["S"]):
        if nn[b] == -1:
            for k in range(_pages(ln[b], ps)):
                if have < F:
                    free[have] = table[b][k]
                    have += 1
    cu, total, slot, pos, spent = [0], [], [-1] * N, [-1] * N, 0
    for b in range(c["S"]):
        q = max(nn[b], 0)
        cu.append(cu[-1] + q)
        held = _pages(ln[b], ps)
        need = _pages(ln[b] + q, ps) - held
        if nn[b] < 0:
            total.append(0)
            continue
        if ln[b] + q > width * ps or cu[-1] > N:
            total.append(-1)
            continue
        if need and spent + need > have:
            spent += need                      # a request that found too few closes the list to later ones
            total.append(-1)
            continue
        for k in range(need):
            table[b][held + k] = free[have - 1 - spent - k]
        spent += need
        total.append(ln[b] + q)
        for k in range(q):
            p = ln[b] + k
            slot[cu[b] + k], pos[cu[b] + k] = table[b][p // ps] * ps + p % ps, p
    used = sum(_pages(total[b], ps) - _pages(ln[b], ps) for b in range(c["S"]) if nn[b] >= 0 and total[b] >= 0)
    i = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return {"cu": i(cu), "total": i(total), "slot": i(slot), "pos": i(pos), "n_free": i([have - used]),
            "table": i(table), "free": i(free)}


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

    info = s["I"][:n].double().clone()
    for k, th in enumerate(s["theta"] or []):
        u, v = info[:, 2 * k].clone(), info[:, 2 * k + 1].clone()
        info[:, 2 * k] = math.cos(th) * u - math.sin(th) * v
        info[:, 2 * k + 1] = math.sin(th) * u + math.cos(th) * v
    at = s["slot"][:n].long()
    p1, cp2, cv = s["P1o"].double(), s["cP2"].double(), s["cV"].double()
    p1[:n] = turned(s["P1"])
    cp2[at // ps, :, at % ps] = turned(s["P2"])
    cv[at // ps, :, at % ps] = info
    return {"P1": p1, "P2": cp2, "V": cv}
