"""Plain model of the caches' contents and of attention over them, for the tests: what
each page format restores (codes by the formats' binary32 definition, in torch
elementwise arithmetic), masked softmax attention in 64 bits, and how far a kernel's
output may be from it by arithmetic alone."""
from __future__ import annotations

import math

import torch

INT8 = "int8"
LOG2E = 1.4426950408889634


def int8_rows(x):
    """(codes, scales, restored) of rows [n, H, 128]; scales [blocks, H]; the unfinished block stays."""
    n, H, D = x.shape
    w = n // 16 * 16
    b = x[:w].float().view(w // 16, 16, H, D)
    top = b.abs().amax((1, 3)) if w else torch.zeros(0, H, device=x.device)
    top = torch.where(top < 2.0 ** -100, torch.zeros_like(top), top)
    # tensors over tensors: by a host number the GPU multiplies by a rounded inverse
    most = torch.full_like(top, 127.0)
    inv = torch.where(top == 0, torch.zeros_like(top), most / torch.where(top == 0, torch.ones_like(top), top))
    codes = torch.round(b * inv[:, None, :, None]).clamp(-127, 127)
    sc = top / most
    y = x.float().clone()
    y[:w] = (codes * sc[:, None, :, None]).view(w, H, D)
    return codes, sc, y


def kivi_rows(x, bits, residual, key):
    """Restored rows [n, H, 128] in fp32, fmaf(code, scale, min), and |min| per element."""
    n, H, D = x.shape
    top = 15.0 if bits == 4 else 3.0
    y, m = x.float().clone(), torch.zeros(n, H, D, device=x.device)
    if key:
        w = n // 32 * 32
        b, dim = x[:w].float().view(w // 32, 32, H, D), 1
    else:
        w = max(0, n - residual)
        b, dim = x[:w].float().view(w, H, 4, 32), 3
    if w:
        lo, hi = b.amin(dim, keepdim=True) + 0.0, b.amax(dim, keepdim=True) + 0.0
        s = (hi - lo) / torch.full_like(lo, top)
        c = torch.where(s == 0, torch.zeros_like(b), torch.round((b - lo) / torch.where(s == 0, torch.ones_like(s), s)).clamp(0, top))
        y[:w] = (c.double() * s.double() + lo.double()).float().view(w, H, D)
        m[:w] = lo.abs().expand_as(b).reshape(w, H, D)
    return y, m


def fp8_rows(x, scale):
    """Restored rows; scale [H]."""
    s = scale.to(x.device).float()[None, :, None]
    return (x.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn).float() * s


def restored(k, v, bits, residual, scales=None):
    """(K, V, |offset| of K, of V): offsets are the KIVI minima that a kernel adds apart."""
    if bits == INT8:
        K, V = int8_rows(k)[2], int8_rows(v)[2]
    elif bits == 8:
        one = torch.ones(k.shape[1])
        ks, vs = scales if scales is not None else (one, one)
        K, V = fp8_rows(k, torch.as_tensor(ks)), fp8_rows(v, torch.as_tensor(vs))
    else:
        K, mk = kivi_rows(k, bits, residual, True)
        V, mv = kivi_rows(v, bits, residual, False)
        return K, V, mk, mv
    return K, V, torch.zeros_like(K), torch.zeros_like(V)


def attention(q, K, V, positions, window=None, sinks=0, scale=1 / math.sqrt(128)):
    """q [nq, Hq, 128] at `positions` over restored K, V [T, H, 128], in 64 bits:
    (out, probabilities [nq, Hq, T])."""
    nq, Hq, D = q.shape
    T, H, _ = K.shape
    g = Hq // H
    t = torch.arange(T, device=q.device)
    p = torch.as_tensor(positions, device=q.device)[:, None]
    seen = t <= p
    if window is not None:
        seen = seen & ((t > p - window) | (t < sinks))
    kk = K.double().repeat_interleave(g, 1)
    z = torch.einsum("qhd,thd->qht", q.double(), kk) * scale
    z = torch.where(seen[:, None], z, torch.full_like(z, -math.inf))
    P = torch.softmax(z, -1)
    vv = V.double().repeat_interleave(g, 1)
    # a masked row takes no part, whatever it holds
    out = torch.stack([torch.einsum("ht,thd->hd", P[i][:, seen[i]], vv[seen[i]]) for i in range(nq)])
    return out, P, seen


def bound(q, K, V, mk, mv, P, seen, out, out_dtype, bits, scale=1 / math.sqrt(128)):
    """How far a kernel's out may be from `out`.

    Scores: products of f16 operands are exact, an 8-step fp32 MMA chain over terms of
    total size S loses at most 8 steps of 2^-23 S, the rounding of a folded (split) query
    2^-21 S, fp32 scaling a few 2^-24: dz <= 2^-19 S in all (log2 domain: times scale
    log2 e), where S = sum |q| (|k| + |min|) and on INT8 pages sum |q| (|k| + 128 step),
    step = |k|max of the row / 127 at least as large as its block's step allows; taken
    per row as the largest element of the whole head. P then is off by 2^dz - 1.
    P V: P (times its scale on KIVI pages) is rounded to f16: half a step, 2^-11
    relative, or 2^-25 of its operand below f16's normal range (codes to 255, so 255
    steps of the scale, at most 2.01 |v|max on INT8 pages, 15 scales on KIVI pages,
    |v|max on FP8 pages), against a sum of P of at least 1; fp32 sums 2^-19 of what they
    add. Output: half a step of its type."""
    H, g = K.shape[1], q.shape[1] // K.shape[1]
    fin = lambda x: torch.nan_to_num(x.double(), 0, 0, 0)  # noqa: E731
    kabs, vabs = fin(K).abs() + mk.double(), fin(V).abs() + mv.double()
    if bits == INT8:
        kabs = kabs + 1.01 * fin(K).abs().amax((0, 2), keepdim=True)
        vabs = vabs + 1.01 * fin(V).abs().amax((0, 2), keepdim=True)
    rep = lambda x: x.repeat_interleave(g, 1)  # noqa: E731
    S = torch.einsum("qhd,thd->qht", q.double().abs(), rep(kabs))
    dz = torch.where(seen[:, None], S, torch.zeros_like(S)).amax(-1) * scale * LOG2E * 2.0 ** -19   # [nq, Hq]
    A = torch.einsum("qht,thd->qhd", P, rep(vabs))
    n = seen.sum(-1)[:, None, None].double()
    M = vabs.amax()
    rel = 2.0 ** -11 + 2.0 ** -19 + 2 * (torch.exp2(dz)[..., None] - 1)
    half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[out_dtype]
    return rel * A + n * 2.0 ** -25 * M + half * out.abs() + 2.0 ** -25


def check(got, q, K, V, mk, mv, positions, bits, window=None, sinks=0, what=""):
    """got [nq, Hq, 128] against the plain attention, within the bound."""
    out, P, seen = attention(q, K, V, positions, window, sinks)
    tol = bound(q, K, V, mk, mv, P, seen, out, got.dtype, bits)
    err = (got.double() - out).abs()
    assert torch.isfinite(out).all()
    assert bool((err <= tol).all()), f"{what}: error {float(err.max()):.3e}, {float((err / tol).max()):.2f} of the bound"
    return float((err / tol).max())


class Filled:
    """A cache of one layer filled with seeded sequences, their rows, and the plain model of each."""

    def __init__(self, lens, H=2, bits=4, dtype="bf16", residual=32, seed=0, chunks=None, slots=None, spare=0,
                 fp8_scales=None, edit=None, device="cuda", loose=0):
        import int4_kivi_quantized_gb300 as s4
        import s4kv_inputs as inp
        self.lens, self.H, self.bits, self.residual = list(lens), H, bits, residual
        self.dev = torch.device(device)
        self.dtype = torch.bfloat16 if dtype == "bf16" else torch.float16
        pages = [max(1, -(-(n + spare) // 16)) for n in self.lens]
        total = sum(pages) + loose
        self.bt = inp.block_tables("permuted", len(pages), pages, total, seed + 1).to(self.dev)
        nslots = len(pages) if slots is None else max(slots) + 1
        self.slots = None if slots is None else torch.tensor(slots, dtype=torch.int32, device=self.dev)
        self.cache = s4.KVCache(1, total, H, residual, nslots, dtype, device=self.dev, bits=bits)
        self.scales = fp8_scales
        if fp8_scales is not None:
            self.cache.set_fp8_scales(0, *fp8_scales)
        outl = inp.outlier_channels(seed, 0, H, 128, 2)
        self.k, self.v = [], []
        for b, n in enumerate(self.lens):
            k, v = inp.kv_rows(inp.mix_seed(seed, b), n, H, 128, self.dtype, outl, 8.0)
            if edit is not None:
                edit(b, k, v)
            self.k.append(k.to(self.dev))
            self.v.append(v.to(self.dev))
        self.seq = self.i32(self.lens)
        at = [0] * len(pages)
        for step in (chunks or [max(self.lens + [1])]):   # chunk sizes, the last one repeated
            at = self.append_to(at, [min(n, a + step) for a, n in zip(at, self.lens)])
        while at != self.lens:
            at = self.append_to(at, [min(n, a + step) for a, n in zip(at, self.lens)])

    def i32(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device=self.dev)

    def append_to(self, at, to):
        k = torch.cat([x[a:t] for x, a, t in zip(self.k, at, to)])
        v = torch.cat([x[a:t] for x, a, t in zip(self.v, at, to)])
        cu = [0]
        for a, t in zip(at, to):
            cu.append(cu[-1] + t - a)
        self.cache.append(0, k, v, self.i32(cu), self.i32(at), self.bt, slot_ids=self.slots)
        return list(to)

    def plain(self, b):
        return restored(self.k[b], self.v[b], self.bits, self.residual, self.scales)

    def ok(self):
        rc, detail = self.cache.status()
        assert rc == 0, (rc, detail)
