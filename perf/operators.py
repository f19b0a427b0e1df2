"""What is measured of the cache's operators: attention over 8-bit pages with a scale for each
block and head, attention with a sliding window and sinks, appends that rotate the keys on the
way, and the batched restore of cached tokens.

With `own` false, `run` computes them in plain torch on a paged cache of plain tensors; with
`own` true it makes the calls of int4_kivi_quantized_gb300. Both caches hold the same tokens:
16-bit keys and values drawn from the seed, quantized by the rule of their format
  int8   symmetric codes, one fp32 scale per 16-token block, kv head and tensor; the tokens of
         the unfinished block stay in 16 bits
  int4, int2   keys by channel over 32 tokens, values by token over 32 channels (scale and
         minimum), the unfinished key group and the newest `residual` values in 16 bits
  fp8    e4m3 bytes, scale 1
"""
import math

import torch

own = False

D, P = 128, 16                      # head width, tokens of a page
LEVELS = {"int4": 15.0, "int2": 3.0}


# ---- the cases ---------------------------------------------------------------------------


def _case(name, kind, form, dtype, batch, q_heads, kv_heads, shortest, longest, nq=1, window=0, sinks=0,
          residual=128, rotary=128, interleaved=False):
    c = dict(kind=kind, form=form, dtype=dtype, batch=batch, q_heads=q_heads, kv_heads=kv_heads,
             shortest=shortest, longest=longest, nq=nq, window=window, sinks=sinks, residual=residual,
             rotary=rotary, interleaved=interleaved)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one short conversation: the call's latency counts
        _case("int8 decode, one sequence", "attend", "int8", "fp16", 1, 4, 1, 256, 256),
        # a serving batch at mixed lengths
        _case("int8 decode, batch 32", "attend", "int8", "bf16", 32, 32, 8, 1024, 8192),
        # long contexts: the cache is read at the memory's rate
        _case("int8 decode, 32k contexts", "attend", "int8", "fp16", 32, 28, 4, 32768, 32768),
        # four draft tokens of a speculative step verified at once
        _case("int8 verify, 4 tokens", "attend", "int8", "bf16", 16, 32, 8, 777, 8191, nq=4),
        # a small window over one sequence of the default 4-bit pages
        _case("int4 window 256, one sequence", "window", "int4", "bf16", 1, 32, 8, 5001, 5001, window=256, sinks=4),
        # long conversations behind a 4096-token window
        _case("int4 window 4096, batch 64", "window", "int4", "bf16", 64, 32, 8, 4096, 16384, window=4096, sinks=4),
        # odd sizes: a window that starts inside a page, draft tokens, fp8 pages
        _case("fp8 window 1000, 5 tokens", "window", "fp8", "fp16", 24, 12, 2, 333, 4099, nq=5, window=1000, sinks=3),
        # one generated token of every sequence, its query rotated too
        _case("int8 step, batch 128", "step", "int8", "bf16", 128, 32, 8, 256, 2048),
        # a prompt chunk of each of several sequences
        _case("int8 prompts of 2048", "append", "int8", "bf16", 8, 32, 8, 1900, 2048),
        # the default 4-bit pages, partly rotated heads
        _case("int4 prompts of 2048", "append", "int4", "fp16", 8, 28, 4, 2000, 2048, rotary=64),
        # a cached prefix restored for a dense kernel
        _case("int4 restore, one sequence", "gather", "int4", "bf16", 1, 32, 8, 1500, 1500),
        # the histories of a batch
        _case("int8 restore, batch 16", "gather", "int8", "bf16", 16, 32, 8, 2048, 8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attend", "window", "step", "append", "gather"])
    form = rng.choice({"attend": ["int8"], "step": ["int8", "int8", "fp8"]}.get(kind, ["int8", "int4", "int2", "fp8"]))
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 6, 7, 8])
    nq = 1 if kind in ("step", "append", "gather") or rng.random() < 0.5 else rng.randint(2, min(16, 96 // group))
    top = {"attend": 32768, "window": 16384, "step": 2048, "append": 2048, "gather": 8192}[kind]
    longest = max(_log(rng, 1, top), nq)
    shortest = rng.randint(max(nq, longest // 4), longest)
    most = {"attend": 2000000, "window": 4000000, "step": 1000000, "append": 120000, "gather": 600000}[kind]
    batch = _log(rng, 1, max(1, min(128, most // (longest * kv))))
    window = _log(rng, 1, 4096) if kind == "window" else 0
    sinks = rng.choice([0, 1, 4, 16, 77]) if kind == "window" else 0
    rotary = rng.choice([128, 128, 64, 96, 32]) if kind in ("step", "append") else 128
    return _case(None, kind, form, rng.choice(["bf16", "fp16"]), batch, kv * group, kv, shortest, longest, nq,
                 window, sinks, rng.choice([32, 128, 200]), rotary, rng.random() < 0.3)


# ---- what a program has in hand -----------------------------------------------------------


def _inputs(case, seed):
    """Lengths (host and device), the tokens' rows, queries, page table and rotation table."""
    g = torch.Generator().manual_seed(seed * 1000003 + 17)
    B, H, Hq = case["batch"], case["kv_heads"], case["q_heads"]
    # lengths spread evenly over the case's range, the seed says which sequence has which
    n = torch.linspace(case["shortest"], case["longest"], B, dtype=torch.float64).round().long() if B > 1 else torch.tensor([case["longest"]])
    n = n[torch.randperm(B, generator=g)]
    dev = torch.device("cuda")
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float16
    gd = torch.Generator(device=dev).manual_seed(seed * 7919 + 3)
    total = int(n.sum())
    # keys with a few large channels, as language models have them
    big = torch.where(torch.rand(H, D, generator=gd, device=dev) < 0.02, 8.0, 1.0)
    k = (torch.randn(total, H, D, generator=gd, device=dev) * big).to(dt)
    v = torch.randn(total, H, D, generator=gd, device=dev).to(dt)
    rows = {"step": B, "append": total}.get(case["kind"])
    q = torch.randn(*((rows,) if rows else (B, case["nq"])), Hq, D, generator=gd, device=dev).to(dt)
    pages = (n + P - 1) // P + (1 if case["kind"] == "step" else 0)
    most = int(pages.max())
    perm = torch.randperm(int(pages.sum()), generator=g).to(torch.int32)
    bt = torch.full((B, most), -1, dtype=torch.int32)
    bt[torch.arange(most) < pages[:, None]] = perm
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), n.cumsum(0)])
    s = dict(case=case, dt=dt, k=k, v=v, q=q, bt=bt.to(dev), lens=n.to(torch.int32).to(dev),
             cu=cu.to(torch.int32).to(dev), n=n.to(dev), first=cu[:-1].to(dev), total=total, pages=int(pages.sum()),
             longest=int(n.max()), zeros=torch.zeros(B, dtype=torch.int32, device=dev))
    if case["kind"] in ("step", "append"):
        half = case["rotary"] // 2
        at = torch.arange(case["longest"] + 2, dtype=torch.float64, device=dev)[:, None]
        angle = at * 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
        s["table"] = torch.cat([angle.cos(), angle.sin()], 1).to(torch.float32).contiguous()
    if case["kind"] == "step":
        s["k1"] = torch.randn(B, H, D, generator=gd, device=dev).to(dt)
        s["v1"] = torch.randn(B, H, D, generator=gd, device=dev).to(dt)
        s["ones"] = torch.arange(B + 1, dtype=torch.int32, device=dev)
        s["grown"] = s["lens"] + 1
    if case["kind"] in ("step", "gather"):
        # what is read back: the newest 16 tokens after a step, else everything
        back = (n + 1).clamp(max=16) if case["kind"] == "step" else n
        s["back_first"] = ((n + 1 - back) if case["kind"] == "step" else n - back).to(torch.int32).to(dev)
        s["back_cu"] = torch.cat([torch.zeros(1, dtype=torch.int64), back.cumsum(0)]).to(torch.int32).to(dev)
        s["back_rows"] = int(back.sum())
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import int4_kivi_quantized_gb300 as s4
        bits = {"int8": "int8", "int4": 4, "int2": 2, "fp8": 8}[case["form"]]
        c = s["cache"] = s4.KVCache(1, s["pages"], case["kv_heads"], case["residual"], case["batch"], case["dtype"], bits=bits)
        if "table" in s:
            s["rope"] = s4.Rope(s["table"], interleaved=case["interleaved"])
        if case["kind"] != "append":
            c.append(0, s["k"], s["v"], s["cu"], s["zeros"], s["bt"])
        if case["kind"] == "step":   # a step is repeated from the same lengths
            at, size = c.layout.lens_offset, 4 * case["batch"] * case["kv_heads"]
            s["stored"] = c.pool[at:at + size]
            s["stored_before"] = s["stored"].clone()
    else:
        s["cache"] = _empty(s)
        if case["kind"] != "append":
            _fill(s, s["k"], s["v"])
    if case["kind"] != "append":
        del s["k"], s["v"]
    return s


# ---- the plain forms ----------------------------------------------------------------------


def _empty(s):
    """A paged cache of plain tensors: codes by (page, head, token), what restores them, rings."""
    c, dev, n, H, B = s["case"], s["q"].device, s["pages"], s["case"]["kv_heads"], s["case"]["batch"]
    f = c["form"]
    z = lambda *shape, t=torch.float32: torch.zeros(shape, dtype=t, device=dev)  # noqa: E731
    code = {"int8": torch.int8}.get(f, torch.uint8)
    a = dict(kc=z(n, H, P, D, t=code), vc=z(n, H, P, D, t=code))
    if f == "int8":
        a.update(ks=z(n, H), vs=z(n, H), kr=z(B, H, P, D, t=s["dt"]), vr=z(B, H, P, D, t=s["dt"]))
    elif f != "fp8":
        a.update(ks=z(n, H, D), km=z(n, H, D), vs=z(n, H, P, 4), vm=z(n, H, P, 4),
                 kr=z(B, H, 32, D, t=s["dt"]), vr=z(B, H, c["residual"], D, t=s["dt"]))
    return a


def _blocks(x, first, n, size):
    """Ragged rows [total, H, D] as padded blocks [B, blocks, size, H, D], and the token of each."""
    B, blocks = n.numel(), -(-int(n.max()) // size)
    t = torch.arange(blocks * size, device=x.device).view(1, blocks, size).expand(B, -1, -1)
    at = (first[:, None, None] + t).clamp(max=x.shape[0] - 1)
    y = x[at].float()
    return torch.where((t < n[:, None, None])[..., None, None], y, 0.0), t


def _by(x, n):
    """x / n as one division of tensors (by a host number the GPU multiplies by its rounded inverse)."""
    return x / torch.full_like(x, n)


def _div_codes(x, lo, scale, top):
    c = torch.round((x - lo) / torch.where(scale == 0, 1.0, scale)).clamp(0, top)
    return torch.where(scale == 0, 0.0, c)


def _int8(y):
    """Codes and scales of blocks [..., 16, H, D]: one scale per block and head."""
    top = y.abs().amax((-3, -1))
    top = torch.where(top < 2.0 ** -100, 0.0, top)
    inv = torch.where(top > 0, torch.full_like(top, 127.0) / top, 0.0)
    return torch.round(y * inv[..., None, :, None]).clamp(-127, 127).to(torch.int8), _by(top, 127.0)


def _fill(s, k, v):
    """Every sequence's rows from its first token on into the plain cache."""
    c, a, n = s["case"], s["cache"], s["n"]
    f, B = c["form"], c["batch"]
    if f == "int8":
        for x, code, scale, ring in ((k, "kc", "ks", "kr"), (v, "vc", "vs", "vr")):
            y, t = _blocks(x, s["first"], n, P)
            codes, sc = _int8(y)
            whole = t[..., -1] < n[:, None]
            page = s["bt"][:, :t.shape[1]][whole].long()
            a[code][page] = codes[whole].transpose(1, 2)
            a[scale][page] = sc[whole]
            _to_ring(a[ring], x, s["first"], n - n % P, n)
    elif f == "fp8":
        for x, code in ((k, "kc"), (v, "vc")):
            y, t = _blocks(x, s["first"], n, P)
            page = s["bt"][:, :t.shape[1]][t[..., 0] < n[:, None]].long()
            e = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            a[code][page] = e[t[..., 0] < n[:, None]].transpose(1, 2)
    else:
        top = LEVELS[f]
        y, t = _blocks(k, s["first"], n, 32)
        lo, hi = y.amin(2, keepdim=True), y.amax(2, keepdim=True)
        sc = _by(hi - lo, top)
        codes = _div_codes(y, lo, sc, top).to(torch.uint8)
        whole = t[..., -1] < n[:, None]
        wide = torch.nn.functional.pad(s["bt"], (0, 2 * t.shape[1] - s["bt"].shape[1])) if s["bt"].shape[1] < 2 * t.shape[1] else s["bt"]
        pair = wide[:, :2 * t.shape[1]].view(B, t.shape[1], 2)[whole].long()      # [groups, 2]
        a["kc"][pair] = codes[whole].view(-1, 2, P, c["kv_heads"], D).transpose(2, 3)
        a["ks"][pair] = sc[whole].expand(-1, 2, -1, -1)
        a["km"][pair] = lo[whole].expand(-1, 2, -1, -1)
        _to_ring(a["kr"], k, s["first"], n - n % 32, n)
        old = (n - c["residual"]).clamp(min=0)
        y, t = _blocks(v, s["first"], n, P)
        y = y.view(*y.shape[:-1], 4, 32)
        lo, hi = y.amin(-1, keepdim=True), y.amax(-1, keepdim=True)
        sc = _by(hi - lo, top)
        codes = _div_codes(y, lo, sc, top).to(torch.uint8).flatten(-2)
        gone = t < old[:, None, None]
        page = s["bt"][:, :t.shape[1], None].expand(-1, -1, P)[gone].long()
        tau = t[gone] % P
        a["vc"][page, :, tau] = codes[gone]
        a["vs"][page, :, tau] = sc[..., 0][gone]
        a["vm"][page, :, tau] = lo[..., 0][gone]
        _to_ring(a["vr"], v, s["first"], old, n)


def _to_ring(ring, x, first, lo, hi):
    """Rows of tokens [lo, hi) of every sequence to ring rows t mod the ring's length."""
    R = ring.shape[2]
    t = lo[:, None] + torch.arange(R, device=x.device)
    there = t < hi[:, None]
    slot = torch.arange(lo.numel(), device=x.device)[:, None].expand_as(t)[there]
    ring[slot, :, t[there] % R] = x[(first[:, None] + t)[there]]


def _restore(s, slot, t, lens):
    """Keys and values of tokens t of the sequences `slot` (same shape), [..., H, D] in fp32."""
    c, a = s["case"], s["cache"]
    f = c["form"]
    last = lens[slot] - 1
    t = torch.minimum(t.clamp(min=0), last.clamp(min=0))
    page, tau = s["bt"][slot, t // P].long().clamp(min=0), t % P
    kc, vc = a["kc"][page, :, tau], a["vc"][page, :, tau]
    if f == "fp8":
        return kc.view(torch.float8_e4m3fn).float(), vc.view(torch.float8_e4m3fn).float()
    if f == "int8":
        k, v = kc.float() * a["ks"][page][..., None], vc.float() * a["vs"][page][..., None]
        ring = (t >= lens[slot] - lens[slot] % P)[..., None, None]
        return torch.where(ring, a["kr"][slot, :, tau].float(), k), torch.where(ring, a["vr"][slot, :, tau].float(), v)
    # code * scale + minimum rounded once, as a fused multiply-add gives it
    k = (kc.double() * a["ks"][page].double() + a["km"][page].double()).float()
    w = lambda x: x.double().repeat_interleave(32, -1)  # noqa: E731
    v = (vc.double() * w(a["vs"][page, :, tau]) + w(a["vm"][page, :, tau])).float()
    kr = (t >= lens[slot] - lens[slot] % 32)[..., None, None]
    vr = (t >= (lens[slot] - c["residual"]).clamp(min=0))[..., None, None]
    return (torch.where(kr, a["kr"][slot, :, t % 32].float(), k),
            torch.where(vr, a["vr"][slot, :, t % c["residual"]].float(), v))


def _attention(s):
    """Softmax attention of the last nq positions; a window of 0 leaves everything visible."""
    c, n = s["case"], s["n"]
    B, H, nq, W, S = c["batch"], c["kv_heads"], c["nq"], c["window"], c["sinks"]
    dev = n.device
    if W:
        # the sinks, then the tokens that some query's window holds
        span = min(W + nq - 1, s["longest"])
        recent = (n[:, None] - span) + torch.arange(span, device=dev)
        few = min(S, s["longest"])
        t = torch.cat([torch.arange(few, device=dev).expand(B, -1), torch.where(recent < few, -1, recent)], 1)
    else:
        t = torch.arange(s["longest"], device=dev).expand(B, -1)
    slot = torch.arange(B, device=dev)[:, None].expand_as(t)
    k, v = _restore(s, slot, t, n)                                             # [B, L, H, D]
    at = n[:, None] - nq + torch.arange(nq, device=dev)                        # positions of the queries
    seen = (t[:, None] >= 0) & (t[:, None] <= at[..., None])
    if W:
        seen &= (t[:, None] > at[..., None] - W) | (t[:, None] < S)
    q = s["q"].float().view(B, nq, H, -1, D).permute(0, 2, 1, 3, 4).reshape(B, H, -1, D)
    z = q @ k.permute(0, 2, 3, 1) * (1.0 / math.sqrt(D))
    z = z.view(B, H, nq, -1, t.shape[1]).masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(z - z.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.view(B, H, -1, t.shape[1]) @ v.permute(0, 2, 1, 3)
    return o.view(B, H, nq, -1, D).permute(0, 2, 1, 3, 4).reshape(B, nq, -1, D).to(s["dt"])


def _rotate(x, row, interleaved):
    """Rows x [n, heads, D] turned by their rows of the table, in fp32, rounded to the 16-bit type."""
    half = row.shape[1] // 2
    cos, sin = row[:, None, :half], row[:, None, half:]
    y = x.float()
    if interleaved:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, y[..., 2 * half:]], -1).to(x.dtype)


def _step(s):
    """One token more of every sequence into the plain cache (8-bit forms)."""
    c, a, n = s["case"], s["cache"], s["n"]
    row = s["table"][n]
    k = _rotate(s["k1"], row, c["interleaved"])
    slot = torch.arange(c["batch"], device=n.device)
    page, tau = s["bt"][slot, n // P].long(), n % P
    if c["form"] == "fp8":
        for x, code in ((k, "kc"), (s["v1"], "vc")):
            a[code][page, :, tau] = x.float().clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        for x, code, scale, ring in ((k, "kc", "ks", "kr"), (s["v1"], "vc", "vs", "vr")):
            a[ring][slot, :, tau] = x
            codes, sc = _int8(a[ring].float().transpose(1, 2))
            whole = tau == P - 1
            a[code][page] = torch.where(whole[:, None, None, None], codes.transpose(1, 2), a[code][page])
            a[scale][page] = torch.where(whole[:, None], sc, a[scale][page])
    return _rotate(s["q"], row, c["interleaved"])


def _rows(cu, rows):
    """Sequence and place within it of each of `rows` ragged rows."""
    r = torch.arange(rows, device=cu.device)
    i = torch.searchsorted(cu.long(), r, right=True) - 1
    return i, r - cu.long()[i]


def run(s):
    c, kind = s["case"], s["case"]["kind"]
    if own:
        a = s["cache"]
        if kind == "attend" and c["nq"] == 1:
            return a.decode(0, s["q"][:, 0], s["bt"], s["lens"], s["longest"], out_dtype=a.cdtype)
        if kind == "attend":
            return a.multi_query(0, s["q"], s["bt"], s["lens"], s["longest"], out_dtype=a.cdtype)
        if kind == "window":
            return a.window(0, s["q"], s["bt"], s["lens"], s["longest"], c["window"], c["sinks"], out_dtype=a.cdtype)
        if kind == "append":
            q = a.append_rope(0, s["k"], s["v"], s["cu"], s["zeros"], s["bt"], s["rope"], q=s["q"])
            return (q, *a.gather(0, s["bt"], s["lens"], s["cu"], s["total"], out_dtype=a.cdtype))
        if kind == "step":
            s["stored"].copy_(s["stored_before"])
            q = a.append_rope(0, s["k1"], s["v1"], s["ones"], s["lens"], s["bt"], s["rope"], q=s["q"])
            return (q, *a.gather(0, s["bt"], s["grown"], s["back_cu"], s["back_rows"], first=s["back_first"], out_dtype=a.cdtype))
        return a.gather(0, s["bt"], s["lens"], s["back_cu"], s["back_rows"], first=s["back_first"], out_dtype=a.cdtype)
    if kind in ("attend", "window"):
        o = _attention(s)
        return o[:, 0] if kind == "attend" and c["nq"] == 1 else o
    q, lens, cu, rows, first = None, s["n"], s["cu"], s["total"], None
    if kind == "append":
        i, t = _rows(cu, rows)
        row = s["table"][t]
        q = _rotate(s["q"], row, c["interleaved"])
        _fill(s, _rotate(s["k"], row, c["interleaved"]), s["v"])
    else:
        if kind == "step":
            q, lens = _step(s), s["n"] + 1
        i, t = _rows(s["back_cu"], s["back_rows"])
        t = t + s["back_first"].long()[i]
    k, v = _restore(s, i, t, lens)
    return ((q,) if q is not None else ()) + (k.to(s["dt"]), v.to(s["dt"]))


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
    lo, hi = b.amin(dim, keepdim=True), b.amax(dim, keepdim=True)
    sc = (hi - lo) / torch.full_like(lo, LEVELS[form])
    code = torch.where(sc > 0, torch.round((b - lo) / sc), 0.0)
    y[:w] = (code.double() * sc.double() + lo.double()).view(w, H, D)
    return y


def _exact_turn(x, table, t, interleaved):
    half = table.shape[1] // 2
    y = x.double()
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    c, sn = table[t, None, :half].double(), table[t, None, half:].double()
    z = y.clone()
    z[..., a] = y[..., a] * c - y[..., b] * sn
    z[..., b] = y[..., a] * sn + y[..., b] * c
    return z.to(x.dtype)


def exact(case, seed):
    s = _inputs(case, seed)
    f, R, nq, W = case["form"], case["residual"], case["nq"], case["window"]
    heads = case["q_heads"] // case["kv_heads"]
    outs = []
    for b in range(case["batch"]):
        n, f0 = int(s["n"][b]), int(s["first"][b])
        k, v = s["k"][f0:f0 + n], s["v"][f0:f0 + n]
        if case["kind"] == "append":
            at = torch.arange(n, device=k.device)
            k = _exact_turn(k, s["table"], at, case["interleaved"])
            q = _exact_turn(s["q"][f0:f0 + n], s["table"], at, case["interleaved"])
            outs.append((q.double(), _exact_rows(k, f, n, R, True), _exact_rows(v, f, n, R, False)))
        elif case["kind"] == "step":
            q = _exact_turn(s["q"][b:b + 1], s["table"], n, case["interleaved"])
            k = torch.cat([k, _exact_turn(s["k1"][b:b + 1], s["table"], n, case["interleaved"])])
            v = torch.cat([v, s["v1"][b:b + 1]])
            outs.append((q.double(), _exact_rows(k, f, n + 1, R, True)[-16:], _exact_rows(v, f, n + 1, R, False)[-16:]))
        elif case["kind"] == "gather":
            outs.append((_exact_rows(k, f, n, R, True), _exact_rows(v, f, n, R, False)))
        else:
            k, v = _exact_rows(k, f, n, R, True), _exact_rows(v, f, n, R, False)
            t = torch.arange(n, device=k.device)
            rows = []
            for i in range(nq):
                at = n - nq + i
                seen = t <= at
                if W:
                    seen &= (at - t < W) | (t < case["sinks"])
                q = s["q"][b, i].double().view(-1, heads, D)                       # [H, g, D]
                p = torch.softmax((q @ k[seen].permute(1, 2, 0)) / math.sqrt(D), -1)
                rows.append((p @ v[seen].transpose(0, 1)).reshape(-1, D))
            o = torch.stack(rows)
            outs.append(o[0] if case["kind"] == "attend" and nq == 1 else o)
    if case["kind"] in ("attend", "window"):
        return torch.stack(outs)
    return tuple(torch.cat(x) for x in zip(*outs))


# ---- what a pass cannot do without ----------------------------------------------------------

STORED = {"int8": 256.5, "int4": 192.0, "int2": 128.0, "fp8": 256.0}   # bytes of a token and kv head, keys and values


def work(case):
    B, H, Hq, nq = case["batch"], case["kv_heads"], case["q_heads"], case["nq"]
    kind, stored = case["kind"], STORED[case["form"]]
    n = (case["shortest"] + case["longest"]) / 2 if B > 1 else case["longest"]
    wide = 4 * D                                    # a token's key and value in 16 bits
    if kind in ("attend", "window"):
        seen = min(n, case["window"] + nq - 1 + case["sinks"]) if kind == "window" else n
        late = {"int8": min(seen, 7.5), "fp8": 0.0}.get(case["form"], min(seen, (15.5 + case["residual"]) / 2))
        kv = B * H * ((seen - late) * stored + late * wide)
        return {"bytes": kv + 2 * B * nq * Hq * D * 2, "flops": 4.0 * D * B * nq * Hq * seen}
    if kind == "gather":
        return {"bytes": B * H * n * (stored + wide), "flops": 0.0}
    new = B * (n if kind == "append" else 1)        # rows in; stored; read back
    back = B * (n if kind == "append" else min(16, n + 1))
    held = stored if kind == "append" else wide
    turned = new * (2 * Hq * D * 2 + case["rotary"] * 4)
    return {"bytes": new * H * (wide + held) + back * H * (held + wide) + turned, "flops": 6.0 * new * (H + Hq) * D}
