"""What is measured of the cache's score forms, prompts and pages: attention of the newest tokens
with capped scores, distance slopes, documents and prefixes; the same for prompt chunks of any
length; sequences forked on shared pages; pages taken for growing sequences and released.

With `own` false, `run` computes them in plain torch on a paged cache of plain tensors; with
`own` true it makes the calls of int4_kivi_quantized_gb300. Both caches hold the same tokens:
16-bit keys and values drawn from the seed, quantized by the rule of their format
  int8   symmetric codes, one fp32 scale per 16-token block, kv head and tensor; the tokens of
         the unfinished block stay in 16 bits
  int4, int2   keys by channel over 32 tokens, values by token over 32 channels (scale and
         minimum), the unfinished key group and the newest `residual` values in 16 bits
  fp8    e4m3 bytes, scale 1

Attention, for a query at position p and a token t, x = q . k_t / sqrt(128):
  z = cap tanh(x / cap) - slope |p - t|      (cap 0: z = x - slope |p - t|)
  t is seen when t <= max(p, prefix - 1), and t >= its document's first token and t > p - window,
  or t < sinks
Pages: those free (named by no table entry) are given out lowest first, to the sequences in order.
"""
import math

import torch

own = False

D, P = 128, 16                      # head width, tokens of a page
LEVELS = {"int4": 15.0, "int2": 3.0}


# ---- the cases ---------------------------------------------------------------------------


def _case(name, kind, form, dtype="bf16", batch=1, q_heads=32, kv_heads=8, shortest=0, longest=0, nq=1, nq_least=0,
          cap=0.0, slopes=False, window=0, sinks=0, docs=1, prefix=False, residual=128, layers=1, times=1, scarce=False):
    """shortest, longest: tokens of a sequence, its nq_least .. nq newest ones (nq of each where
    nq_least is 0) being the queries; times: continuations of a forked sequence, or tokens that a
    growing one gets."""
    c = dict(kind=kind, form=form, dtype=dtype, batch=batch, q_heads=q_heads, kv_heads=kv_heads, shortest=shortest,
             longest=longest, nq=nq, nq_least=nq_least, cap=cap, slopes=slopes, window=window, sinks=sinks, docs=docs,
             prefix=prefix, residual=residual, layers=layers, times=times, scarce=scarce)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short conversation with a model that caps its scores: the call's latency counts
        _case("capped decode, one sequence", "attend", "int8", "fp16", 1, 4, 1, 256, 256, cap=50.0),
        # four draft tokens of a speculative step, conversations packed as documents, distance slopes
        _case("sloped drafts in documents", "attend", "int8", "bf16", 16, 32, 8, 777, 8191, nq=4, slopes=True, docs=3),
        # long contexts on the default 4-bit pages: the cache is read at the memory's rate
        _case("capped decode, 32k contexts", "attend", "int4", "fp16", 32, 28, 4, 32768, 32768, cap=30.0),
        # the first chunk of one conversation
        _case("prompt of 2048", "prompt", "int4", "bf16", 1, 32, 8, 2048, 2048, nq=2048),
        # chunked prefill of a batch behind cached contexts
        _case("chunks of 512, sloped", "prompt", "int8", "bf16", 8, 32, 8, 2048, 8192, nq=512, slopes=True),
        # ragged packed prompts: documents, a prefix that sees itself whole, odd lengths
        _case("odd prompts, documents, prefix", "prompt", "fp8", "fp16", 5, 12, 2, 1500, 4099, nq=777, nq_least=100,
              docs=4, prefix=True),
        # a long context's last chunk, capped
        _case("2048 behind 32k, capped", "prompt", "int4", "fp16", 1, 28, 4, 32768, 32768, nq=2048, cap=30.0),
        # a few tokens behind a long window: few rows, so the cache's length is what there is to split
        _case("33 tokens, window 4096", "prompt", "int2", "bf16", 4, 32, 8, 8000, 16384, nq=33, window=4096, sinks=4),
        # one prompt answered four ways
        _case("fork of one sequence", "fork", "int4", "bf16", 1, 32, 8, 1000, 1000, layers=4, times=4),
        # sampling or beams over a batch
        _case("fork of 16 prompts", "fork", "int4", "bf16", 16, 32, 8, 700, 2048, layers=4, times=4),
        # the pages of one scheduler step: every sequence grows, some leave
        _case("turnover of 32 sequences", "turn", "int4", "bf16", 32, 8, 1, 256, 2048, times=16),
        # the same for a large pool and draft tokens
        _case("turnover of 512 sequences", "turn", "fp8", "bf16", 512, 8, 1, 512, 16384, times=40),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "prompt", "prompt", "fork", "turn"])
    form = rng.choice(["int8", "int4", "int4", "int2", "fp8"])
    dtype = rng.choice(["bf16", "fp16"])
    kv = rng.choice([1, 2, 4, 8])
    residual = rng.choice([32, 128, 200])
    if kind == "turn":
        batch = _log(rng, 1, 512)
        longest = _log(rng, 1, 16384)
        return _case(None, kind, form, dtype, batch, kv, kv, rng.randint(0, longest), longest, residual=residual,
                     times=_log(rng, 1, 64), scarce=rng.random() < 0.2)
    if kind == "fork":
        longest = _log(rng, 1, 2048)
        return _case(None, kind, form, dtype, _log(rng, 1, max(1, min(16, 24000 // longest))), kv, kv,
                     rng.randint(max(1, longest // 3), longest), longest, residual=residual, layers=rng.randint(1, 4),
                     times=rng.randint(1, 4), scarce=rng.random() < 0.15)
    group = rng.choice([1, 2, 3, 4, 6, 7, 8])
    score = dict(cap=rng.choice([0.0, 5.0, 30.0, 50.0]), slopes=rng.random() < 0.4, docs=rng.choice([1, 1, 1, 3, 8]),
                 prefix=rng.random() < 0.25, residual=residual)
    if rng.random() < 0.3:
        score.update(window=_log(rng, 1, 4096), sinks=rng.choice([0, 1, 4, 16, 77]))
    if kind == "attend":
        nq = 1 if rng.random() < 0.5 else rng.randint(2, min(16, 96 // group))
        longest = max(_log(rng, 1, 32768), nq)
        batch = _log(rng, 1, max(1, min(128, 2000000 // (longest * kv))))
        return _case(None, kind, form, dtype, batch, kv * group, kv, rng.randint(max(nq, longest // 4), longest), longest,
                     nq, **score)
    nq = _log(rng, 1, 2048)
    longest = max(min(_log(rng, 1, 32768), 1700000000 // (nq * kv * group)), nq)
    batch = _log(rng, 1, max(1, min(24, 1700000000 // (nq * longest * kv * group), 300000 // longest)))
    return _case(None, kind, form, dtype, batch, kv * group, kv, rng.randint(max(nq, longest // 4), longest), longest,
                 nq, nq_least=rng.randint(1, nq), **score)


# ---- what a program has in hand -----------------------------------------------------------


def _spread(lo, hi, n):
    """n whole numbers spread evenly over lo .. hi."""
    return [hi] if n == 1 else [int(round(lo + (hi - lo) * i / (n - 1))) for i in range(n)]


def _done(form, n, residual):
    """Pages of a sequence of n tokens that nothing will be written to any more."""
    return min(n // 32 * 32, max(0, n - residual)) // P if form in LEVELS else n // P


def _inputs(case, seed):
    """Lengths (host and device), the tokens' rows, queries, page table and what the scores need."""
    g = torch.Generator().manual_seed(seed * 1000003 + 29)
    B, H, Hq, kind = case["batch"], case["kv_heads"], case["q_heads"], case["kind"]
    # lengths spread evenly over the case's range, the seed says which sequence has which
    order = torch.randperm(B, generator=g).tolist()
    lens = _spread(case["shortest"], case["longest"], B)
    queries = _spread(case["nq_least"] or case["nq"], case["nq"], B)
    n, m = [lens[i] for i in order], [queries[i] for i in torch.randperm(B, generator=g).tolist()]
    m = [min(x, y) for x, y in zip(n, m)]
    dev = torch.device("cuda")
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    gd = torch.Generator(device=dev).manual_seed(seed * 7919 + 5)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    s = dict(case=case, dt=dt, n=n, m=m, lens=i32(n), longest=max(n), total=sum(n))
    used = [-(-x // P) for x in n]
    if kind in ("fork", "turn"):
        kids = B * case["times"] if kind == "fork" else 0
        src = [b for b in range(B) for _ in range(case["times"])] if kind == "fork" else []
        if kind == "fork":
            need = [-(-n[b] // P) - _done(case["form"], n[b], case["residual"]) for b in src]
        else:
            grown = [x + case["times"] for x in n]
            need = [-(-(x + case["times"]) // P) - u for x, u in zip(n, used)]
        # a pool with room to spare, or too small for the last of them
        spare = max(0, sum(need) - 1 - sum(need) // 3) if case["scarce"] else sum(need) + 7 + sum(used) // 4
        rows, width = B + kids, max(used + [u + e for u, e in zip(used, need)]) if kind == "turn" else max(used)
    else:
        spare, rows, width = 0, B, max(used)
    pages = max(1, sum(used) + spare)
    perm = torch.randperm(pages, generator=g)[:sum(used)].to(torch.int32)
    bt = torch.full((rows, max(1, width)), -1, dtype=torch.int32)
    bt[:B][torch.arange(max(1, width)) < torch.tensor(used)[:, None]] = perm
    s.update(pages=pages, bt=bt.to(dev).clone(), zeros=i32([0] * B))
    if kind in ("fork", "turn"):
        refs = torch.zeros(pages, dtype=torch.int32)
        refs[perm.long()] = 1
        s.update(refs=refs.to(dev).clone(), refs_before=refs.to(dev).clone(), bt_before=bt.to(dev).clone())
        if kind == "fork":
            kept = [_done(case["form"], n[b], case["residual"]) * P for b in src]
            cu = [0]
            for b, k in zip(src, kept):
                cu.append(cu[-1] + n[b] - k)
            s.update(src=i32(src), dst=i32(range(B, B + kids)), kids=i32([n[b] for b in src]), host_src=src,
                     back_first=i32(kept), back_cu=i32(cu), back_rows=cu[-1])
        else:
            gone = torch.randperm(B, generator=g)[:(B + 1) // 2].tolist()
            # half of those that leave had given their first pages away before, others keep some for later
            some = [0 if i % 3 else n[b] // 2 for i, b in enumerate(gone)]
            s.update(grown=i32(grown), gone=i32(gone), gone_first=i32(some), gone_last=i32([n[b] for b in gone]),
                     host=(grown, gone, some))
    if kind == "turn":
        return s
    # keys with a few large channels, as language models have them
    big = torch.where(torch.rand(H, D, generator=gd, device=dev) < 0.02, 8.0, 1.0)
    total = s["total"]
    s["k"] = [(torch.randn(total, H, D, generator=gd, device=dev) * big).to(dt) for _ in range(case["layers"])]
    s["v"] = [torch.randn(total, H, D, generator=gd, device=dev).to(dt) for _ in range(case["layers"])]
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    s.update(cu=i32(cu), start=cu[:-1])
    if kind == "fork":
        return s
    s["q"] = torch.randn(sum(m), Hq, D, generator=gd, device=dev).to(dt)
    cu = [0]
    for x in m:
        cu.append(cu[-1] + x)
    s.update(cu_q=i32(cu), start_q=cu[:-1])
    if case["slopes"]:   # a geometric series over the heads
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (j + 1) / Hq) for j in range(Hq)], dtype=torch.float32, device=dev)
    if case["docs"] > 1:   # the first token of the document that each query is in
        first = []
        for x, y in zip(n, m):
            cuts = torch.cat([torch.zeros(1, dtype=torch.int64), torch.randint(0, x, (case["docs"] - 1,), generator=g)])
            at = torch.arange(x - y, x)
            first += torch.where(cuts <= at[:, None], cuts, 0).amax(1).tolist()
        s["first"] = i32(first)
    if case["prefix"]:
        s["host_prefix"] = [int(torch.randint(0, x + 1, (1,), generator=g)) for x in n]
        s["prefix"] = i32(s["host_prefix"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    kind = case["kind"]
    if own:
        import int4_kivi_quantized_gb300 as s4
        bits = {"int8": "int8", "int4": 4, "int2": 2, "fp8": 8}[case["form"]]
        slots = s["bt"].shape[0]
        c = s["cache"] = s4.KVCache(case["layers"], s["pages"], case["kv_heads"], case["residual"], slots, case["dtype"], bits=bits)
        if kind != "turn":
            for layer in range(case["layers"]):
                c.append(layer, s["k"][layer], s["v"][layer], s["cu"], s["zeros"], s["bt"][:case["batch"]])
        if kind in ("attend", "prompt"):
            s["scores"] = s4.Scores(cap=case["cap"], slopes=s.get("slopes"), window=case["window"], num_sinks=case["sinks"])
    elif kind != "turn":
        s["cache"] = [_filled(s, k, v) for k, v in zip(s["k"], s["v"])]
    if kind != "turn":
        del s["k"], s["v"]
    if kind == "attend":
        shape = (case["batch"], case["nq"])
        s["q"] = s["q"].view(*shape, case["q_heads"], D)
        if "first" in s:
            s["first"] = s["first"].view(*shape)
    return s


# ---- the plain forms: the cache -------------------------------------------------------------


def _by(x, n):
    """x / n as one division of tensors (by a host number the GPU multiplies by its rounded inverse)."""
    return x / torch.full_like(x, n)


def _filled(s, k, v):
    """A paged cache of plain tensors with every sequence's rows: codes by (page, token, head), what
    restores them, rings by slot."""
    c, dev, n, H, S = s["case"], k.device, s["pages"], s["case"]["kv_heads"], s["bt"].shape[0]
    f, R = c["form"], c["residual"]
    z = lambda *shape, t=torch.float32: torch.zeros(shape, dtype=t, device=dev)  # noqa: E731
    code = {"int8": torch.int8}.get(f, torch.uint8)
    a = dict(kc=z(n, P, H, D, t=code), vc=z(n, P, H, D, t=code))
    if f == "int8":
        a.update(ks=z(n, H), vs=z(n, H), kr=z(S, P, H, D, t=s["dt"]), vr=z(S, P, H, D, t=s["dt"]))
    elif f != "fp8":
        a.update(ks=z(n, H, D), km=z(n, H, D), vs=z(n, P, H, 4), vm=z(n, P, H, 4),
                 kr=z(S, 32, H, D, t=s["dt"]), vr=z(S, R, H, D, t=s["dt"]))
    for b, (x, at) in enumerate(zip(s["n"], s["start"])):
        _fill(a, f, R, s["bt"][b].long(), b, k[at:at + x], v[at:at + x])
    return a


def _fill(a, f, R, pages, slot, k, v):
    """One sequence's rows [n, H, D] into the plain cache."""
    n, H = k.shape[:2]
    t = torch.arange(n, device=k.device)
    if f == "fp8":
        for x, to in ((k, "kc"), (v, "vc")):
            a[to][pages[t // P], t % P] = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        return
    if f == "int8":
        w = n // P
        for x, to, scale, ring in ((k, "kc", "ks", "kr"), (v, "vc", "vs", "vr")):
            y = x[:w * P].float().view(w, P, H, D)
            top = y.abs().amax((1, 3)) if w else y.new_zeros(0, H)
            top = torch.where(top < 2.0 ** -100, 0.0, top)
            inv = torch.where(top > 0, torch.full_like(top, 127.0) / top, 0.0)
            a[to][pages[:w]] = torch.round(y * inv[:, None, :, None]).clamp(-127, 127).to(torch.int8)
            a[scale][pages[:w]] = _by(top, 127.0)
            a[ring][slot, t[w * P:] % P] = x[w * P:]
        return
    top = LEVELS[f]
    w = n // 32
    y = k[:w * 32].float().view(w, 32, H, D)
    if w:
        lo, hi = y.amin(1, keepdim=True), y.amax(1, keepdim=True)
        sc = _by(hi - lo, top)
        codes = torch.where(sc == 0, 0.0, torch.round((y - lo) / torch.where(sc == 0, 1.0, sc)).clamp(0, top))
        a["kc"][pages[:2 * w]] = codes.to(torch.uint8).view(2 * w, P, H, D)
        a["ks"][pages[:2 * w]] = sc[:, 0].repeat_interleave(2, 0)
        a["km"][pages[:2 * w]] = lo[:, 0].repeat_interleave(2, 0)
    a["kr"][slot, t[w * 32:] % 32] = k[w * 32:]
    old = max(0, n - R)
    if old:
        y = v[:old].float().view(old, H, 4, 32)
        lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
        sc = _by(hi - lo, top)
        codes = torch.where(sc == 0, 0.0, torch.round((y - lo) / torch.where(sc == 0, 1.0, sc)).clamp(0, top))
        at = pages[t[:old] // P], t[:old] % P
        a["vc"][at] = codes.to(torch.uint8).flatten(-2)
        a["vs"][at] = sc[..., 0]
        a["vm"][at] = lo[..., 0]
    a["vr"][slot, t[old:] % R] = v[old:]


def _restore(s, a, pages, slot, n, t):
    """Keys and values [len(t), H, D] in fp32 of tokens t of a sequence of n tokens."""
    f, R = s["case"]["form"], s["case"]["residual"]
    page, tau = pages[t // P].long(), t % P
    kc, vc = a["kc"][page, tau], a["vc"][page, tau]
    if f == "fp8":
        return kc.view(torch.float8_e4m3fn).float(), vc.view(torch.float8_e4m3fn).float()
    if f == "int8":
        k, v = kc.float() * a["ks"][page][..., None], vc.float() * a["vs"][page][..., None]
        ring = (t >= n // P * P)[:, None, None]
        return torch.where(ring, a["kr"][slot, tau].float(), k), torch.where(ring, a["vr"][slot, tau].float(), v)
    # code * scale + minimum rounded once, as a fused multiply-add gives it
    k = (kc.double() * a["ks"][page].double() + a["km"][page].double()).float()
    w = lambda x: x.double().repeat_interleave(32, -1)  # noqa: E731
    v = (vc.double() * w(a["vs"][page, tau]) + w(a["vm"][page, tau])).float()
    return (torch.where((t >= n // 32 * 32)[:, None, None], a["kr"][slot, t % 32].float(), k),
            torch.where((t >= max(0, n - R))[:, None, None], a["vr"][slot, t % R].float(), v))


# ---- the plain forms: attention -------------------------------------------------------------


def _seen(s, b, t):
    """Which of the tokens t each query of sequence b sees, and the queries' positions."""
    c, n, m = s["case"], s["n"][b], s["m"][b]
    p = torch.arange(n - m, n, device=t.device)[:, None]
    low = torch.zeros_like(p)
    if c["window"]:
        low = p - c["window"] + 1
    if "first" in s:
        low = torch.maximum(low, s["first"].view(-1)[s["start_q"][b]:s["start_q"][b] + m, None].long())
    high = p
    if "prefix" in s:
        high = torch.maximum(high, s["prefix"][b].long() - 1)
    return (t <= high) & ((t >= low) | (t < c["sinks"])), p


def _attention(s):
    """Softmax attention of every sequence's newest tokens, sequence by sequence."""
    c, Hq, H = s["case"], s["case"]["q_heads"], s["case"]["kv_heads"]
    q = s["q"].view(-1, Hq, D)
    outs = []
    for b, (n, m) in enumerate(zip(s["n"], s["m"])):
        t = torch.arange(n, device=q.device)
        k, v = _restore(s, s["cache"][0], s["bt"][b], b, n, t)
        x = q[s["start_q"][b]:s["start_q"][b] + m].float().view(m, H, -1, D).permute(1, 2, 0, 3)   # [H, g, m, D]
        z = (x.reshape(H, -1, D) @ k.permute(1, 2, 0)).view(H, -1, m, n) * (1.0 / math.sqrt(D))
        if c["cap"]:
            e = torch.exp(-2.0 * (z / c["cap"]).abs())
            z = torch.sign(z) * c["cap"] * ((1.0 - e) / (1.0 + e))
        seen, p = _seen(s, b, t)
        if c["slopes"]:
            z = z - s["slopes"].view(H, -1, 1, 1) * (p - t).abs().float()
        z = z.masked_fill(~seen, -math.inf)
        top = z.amax(-1, keepdim=True)
        w = torch.where(seen, torch.exp(z - torch.where(top == -math.inf, 0.0, top)), 0.0)
        w = w / w.sum(-1, keepdim=True).clamp(min=1e-30)
        o = w.view(H, -1, n) @ v.transpose(0, 1)
        outs.append(o.view(H, -1, m, D).permute(2, 0, 1, 3).reshape(m, Hq, D).to(s["dt"]))
    return torch.cat(outs).view(s["q"].shape)


# ---- the plain forms: pages -----------------------------------------------------------------


def _give(refs, bt, row, entry, need):
    """need[i] free pages, lowest first, into entries entry[i] .. of table row row[i]: what was given."""
    free = (refs == 0).nonzero()[:, 0]
    upto = need.cumsum(0)
    good = (need == 0) | (upto <= free.numel())
    given = torch.where(good, need, 0)
    i = torch.arange(need.numel(), device=refs.device).repeat_interleave(given)
    k = torch.arange(i.numel(), device=refs.device)
    page = free[k]
    bt[row[i], entry[i] + k - (given.cumsum(0) - given)[i]] = page.to(torch.int32)
    refs[page] = 1
    return torch.where(good, need, -1)


def _turn(s):
    refs, bt = s["refs"], s["bt"]
    have, want = (s["lens"].long() + P - 1) // P, (s["grown"].long() + P - 1) // P
    taken = _give(refs, bt, torch.arange(have.numel(), device=bt.device), have, want - have)
    e = torch.arange(bt.shape[1], device=bt.device)
    gone = s["gone"].long()
    lo, hi = (s["gone_first"].long() + P - 1) // P, (s["gone_last"].long() + P - 1) // P
    rows = bt[gone]
    drop = (e >= lo[:, None]) & (e < hi[:, None]) & (rows >= 0)
    refs.index_add_(0, rows[drop].long(), torch.full_like(rows[drop], -1))
    bt[gone] = torch.where(drop, -1, rows)
    return bt, refs, taken.to(torch.int32)


def _fork(s):
    c, refs, bt = s["case"], s["refs"], s["bt"]
    f, R = c["form"], c["residual"]
    src, dst, n = s["src"].long(), s["dst"].long(), s["kids"].long()
    done = torch.minimum(n // 32 * 32, (n - R).clamp(min=0)) // P if f in LEVELS else n // P
    have = (n + P - 1) // P
    taken = _give(refs, bt, dst, done, have - done)
    good = (taken >= 0)[:, None]
    e = torch.arange(bt.shape[1], device=bt.device)
    shared = good & (e < done[:, None])
    bt[dst] = torch.where(shared, bt[src], bt[dst])
    named = bt[dst][shared].long()
    refs.index_add_(0, named, torch.ones_like(named, dtype=torch.int32))
    private = good & (e >= done[:, None]) & (e < have[:, None])
    out = []
    slot = [int(x) for x in range(c["batch"], c["batch"] + len(s["host_src"]))]
    ok = good[:, 0]
    for a in s["cache"]:
        frm, to = bt[src][private].long(), bt[dst][private].long()
        for x in a:
            if x in ("kr", "vr"):
                a[x][dst[ok]] = a[x][src[ok]]
            else:
                a[x][to] = a[x][frm]
        k, v = [], []
        for b, d in zip(s["host_src"], slot):
            x = s["n"][b]
            t = torch.arange(_done(f, x, R) * P, x, device=bt.device)
            y = _restore(s, a, bt[d].clamp(min=0), d, x, t)
            k.append(y[0])
            v.append(y[1])
        out += [torch.cat(k).to(s["dt"]), torch.cat(v).to(s["dt"])]
    if c["scarce"]:   # rows of continuations that got no pages stand for nothing
        i = torch.arange(src.numel(), device=bt.device).repeat_interleave(n - s["back_first"].long(), output_size=s["back_rows"])
        out = [torch.where(ok[i][:, None, None], x, 0.0).to(s["dt"]) for x in out]
    return (bt, refs, taken.to(torch.int32), *out)


def run(s):
    c, kind = s["case"], s["case"]["kind"]
    if kind in ("fork", "turn"):   # repeated from the same pages
        s["refs"].copy_(s["refs_before"])
        s["bt"].copy_(s["bt_before"])
    if not own:
        return {"attend": _attention, "prompt": _attention, "fork": _fork, "turn": _turn}[kind](s)
    a = s["cache"]
    if kind == "attend":
        return a.attend(0, s["q"], s["bt"], s["lens"], s["longest"], s["scores"], first=s.get("first"),
                        prefix=s.get("prefix"), out_dtype=a.cdtype)
    if kind == "prompt":
        return a.prompt(0, s["q"], s["cu_q"], s["bt"], s["lens"], s["longest"], s["total"], s["scores"],
                        first=s.get("first"), prefix=s.get("prefix"), out_dtype=a.cdtype)
    if kind == "turn":
        taken = a.take_pages(s["refs"], s["bt"], s["lens"], s["grown"])
        a.release_pages(s["refs"], s["bt"], s["gone_first"], s["gone_last"], slot_ids=s["gone"])
        return s["bt"], s["refs"], taken
    taken = a.fork(s["refs"], s["bt"], s["src"], s["dst"], s["kids"])
    out, zero = [], c["scarce"]
    for layer in range(c["layers"]):
        rows = [torch.zeros((s["back_rows"], c["kv_heads"], D), dtype=s["dt"], device="cuda") for _ in range(2)] if zero else [None, None]
        out += a.gather(layer, s["bt"][c["batch"]:], s["kids"], s["back_cu"], s["back_rows"], first=s["back_first"],
                        slot_ids=s["dst"], out_k=rows[0], out_v=rows[1], out_dtype=a.cdtype)
    return (s["bt"], s["refs"], taken, *out)


# ---- the operators' definition in 64 bits ---------------------------------------------------


def _exact_rows(x, form, n, residual, key):
    """Rows [n, H, D] of one sequence as the cache restores them: codes by the formats' definition,
    which is in binary32 steps, and the values they stand for in 64 bits."""
    y, x = x.double(), x.float()
    H = x.shape[1]
    if form == "fp8":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).double()
    if form == "int8":
        w = n // P * P
        b = x[:w].view(w // P, P, H, D)
        if w:
            top = b.abs().amax((1, 3), keepdim=True)
            most = torch.full_like(top, 127)
            code = torch.round(b * (most / top))
            y[:w] = (code.double() * (top / most).double()).view(w, H, D)
        return y
    if key:
        w = n // 32 * 32
        b, dim = x[:w].view(w // 32, 32, H, D), 1
    else:
        w = max(0, n - residual)
        b, dim = x[:w].view(w, H, 4, 32), 3
    if w:
        lo, hi = b.amin(dim, keepdim=True), b.amax(dim, keepdim=True)
        sc = (hi - lo) / torch.full_like(lo, LEVELS[form])
        code = torch.where(sc > 0, torch.round((b - lo) / sc), 0.0)
        y[:w] = (code.double() * sc.double() + lo.double()).view(w, H, D)
    return y


def _exact_attention(case, s):
    Hq, H = case["q_heads"], case["kv_heads"]
    g, outs = Hq // H, []
    for b, (n, m) in enumerate(zip(s["n"], s["m"])):
        at, qa = s["start"][b], s["start_q"][b]
        k = _exact_rows(s["k"][0][at:at + n], case["form"], n, case["residual"], True)
        v = _exact_rows(s["v"][0][at:at + n], case["form"], n, case["residual"], False)
        q = s["q"][qa:qa + m].double()
        out = torch.zeros(m, Hq, D, dtype=torch.float64, device=q.device)
        t = torch.arange(n, device=q.device)[None]
        p = torch.arange(n - m, n, device=q.device)[:, None]
        hidden = t > p
        if case["prefix"]:
            hidden = hidden & (t >= s["host_prefix"][b])
        early = torch.zeros_like(hidden)
        if case["window"]:
            early |= p - t >= case["window"]
        if case["docs"] > 1:
            early |= t < s["first"][qa:qa + m, None]
        hidden = hidden | (early & (t >= case["sinks"]))
        empty = hidden.all(1)
        for j in range(Hq):
            z = q[:, j] @ k[:, j // g].T / math.sqrt(D)
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if case["slopes"]:
                z -= s["slopes"][j].double() * (p - t).abs()
            z[hidden] = -math.inf
            out[:, j] = torch.softmax(z, -1) @ v[:, j // g]
        out[empty] = 0.0
        outs.append(out)
    out = torch.cat(outs)
    return out.view(case["batch"], case["nq"], Hq, D) if case["kind"] == "attend" else out


def _exact_pages(case, s):
    """Table, counts and what was given, entry by entry on the host."""
    bt, refs = s["bt"].tolist(), s["refs"].tolist()
    free, given = [p for p, r in enumerate(refs) if r == 0], []
    asked, ok = 0, []
    if case["kind"] == "turn":
        jobs = [(b, range(-(-x // P), -(-y // P))) for b, (x, y) in enumerate(zip(s["n"], s["host"][0]))]
    else:
        jobs = [(case["batch"] + i, range(_done(case["form"], s["n"][b], case["residual"]), -(-s["n"][b] // P)))
                for i, b in enumerate(s["host_src"])]
    room = len(free)
    for row, entries in jobs:
        asked += len(entries)
        ok.append(len(entries) == 0 or asked <= room)
        given.append(len(entries) if ok[-1] else -1)
        if ok[-1]:
            for e in entries:
                bt[row][e] = free.pop(0)
                refs[bt[row][e]] = 1
    if case["kind"] == "turn":
        _, gone, some = s["host"]
        for b, x in zip(gone, some):
            for e in range(-(-x // P), -(-s["n"][b] // P)):
                refs[bt[b][e]] -= 1
                bt[b][e] = -1
    else:
        for (row, entries), b, good in zip(jobs, s["host_src"], ok):
            for e in range(entries.start if good else 0):
                bt[row][e] = bt[b][e]
                refs[bt[b][e]] += 1
    t = lambda x: torch.tensor(x, dtype=torch.int32, device=s["bt"].device)  # noqa: E731
    return t(bt), t(refs), t(given), ok


def exact(case, seed):
    s = _inputs(case, seed)
    if case["kind"] in ("attend", "prompt"):
        return _exact_attention(case, s)
    bt, refs, given, ok = _exact_pages(case, s)
    out = []
    for layer in range(case["layers"] if case["kind"] == "fork" else 0):
        for x, key in ((s["k"][layer], True), (s["v"][layer], False)):
            rows = [_exact_rows(x[s["start"][b]:s["start"][b] + s["n"][b]], case["form"], s["n"][b], case["residual"], key)
                    for b in range(case["batch"])]
            out.append(torch.cat([rows[b][_done(case["form"], s["n"][b], case["residual"]) * P:] * (1.0 if good else 0.0)
                                  for b, good in zip(s["host_src"], ok)]))
    return (bt, refs, given, *out)


# ---- what a pass cannot do without ----------------------------------------------------------

STORED = {"int8": 256.5, "int4": 192.0, "int2": 128.0, "fp8": 256.0}   # bytes of a token and kv head, keys and values


def _late(form, n, residual):
    """Tokens of a sequence whose (keys, values) are in 16 bits."""
    if form == "fp8":
        return 0.0
    return n % P if form == "int8" else (n % 32 + min(n, residual)) / 2


def work(case):
    B, H, Hq, kind, form = case["batch"], case["kv_heads"], case["q_heads"], case["kind"], case["form"]
    n = _spread(case["shortest"], case["longest"], B)
    wide = 4.0 * D                                  # a token's key and value in 16 bits
    if kind == "turn":
        need = sum(-(-(x + case["times"]) // P) - -(-x // P) for x in n)
        gone = sum(-(-x // P) for x in n) * 5 / 12
        pages = need + 7 + 1.25 * sum(-(-x // P) for x in n)
        # counts looked at once; entries and counts that change, written (read too where they go down)
        return {"bytes": 4.0 * (pages + 2 * need + 4 * gone), "flops": 0.0}
    if kind == "fork":
        total = 0.0
        for x in n:
            done, have = _done(form, x, case["residual"]), -(-x // P)
            late = _late(form, x, case["residual"])
            kept = (x - done * P - late) * STORED[form] + late * wide
            total += case["times"] * (case["layers"] * H * (3 * kept + (x - done * P) * wide) + 4.0 * 2 * have + 8.0 * done)
        return {"bytes": total, "flops": 0.0}
    m = [min(x, y) for x, y in zip(n, _spread(case["nq_least"] or case["nq"], case["nq"], B))]
    bytes_, pairs = 0.0, 0.0
    for x, y in zip(n, m):
        span = x                                    # what the middle query sees, its document's part or its window
        if case["window"]:
            span = min(span, case["window"] + case["sinks"])
        mid = x - (y - 1) / 2
        if case["prefix"]:
            mid = (mid + x) / 2
        if case["docs"] > 1:
            mid = mid / case["docs"]
        pairs += y * min(span, mid)
        seen = min(x, span + y - 1) if case["docs"] == 1 else min(x, x / case["docs"] + y)
        late = min(seen, _late(form, x, case["residual"]))
        bytes_ += H * ((seen - late) * STORED[form] + late * wide) + 2 * y * Hq * D * 2.0
    return {"bytes": bytes_, "flops": 4.0 * D * Hq * pairs}
