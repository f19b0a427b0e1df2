"""Plain model of attention with a score form, for the tests: which tokens a query sees,
scores, softmax and output in 64 bits, and how far a kernel's output may be from it by
arithmetic alone."""
from __future__ import annotations

import math

import torch

SCALE = 1 / math.sqrt(128)
LOG2E = 1.4426950408889634


def seen_of(T, positions, window=0, sinks=0, first=None, prefix=None):
    """[nq, T]: whether the query at positions[i] sees token t."""
    rows = []
    for i, p in enumerate(positions):
        lo, hi = 0, p
        if window:
            lo = max(lo, p - window + 1)
        if first is not None:
            lo = max(lo, first[i])
        if prefix is not None:
            hi = max(hi, min(prefix, T) - 1)
        rows.append([t <= min(hi, T - 1) and (t >= lo or t < sinks) for t in range(T)])
    return torch.tensor(rows, dtype=torch.bool).view(len(positions), T)


def attention(q, K, V, positions, seen, cap=0.0, slopes=None, scale=SCALE):
    """q [nq, Hq, 128] over restored K, V [T, H, 128]: (out [nq, Hq, 128], P [nq, Hq, T])."""
    nq, Hq, D = q.shape
    T, H, _ = K.shape
    g = Hq // H
    outs, Ps = [], []
    for i in range(nq):
        t = torch.nonzero(seen[i].to(q.device))[:, 0]
        P = torch.zeros(Hq, T, dtype=torch.float64, device=q.device)
        if t.numel() == 0:
            outs.append(torch.zeros(Hq, D, dtype=torch.float64, device=q.device))
            Ps.append(P)
            continue
        k, v = K[t].double().repeat_interleave(g, 1), V[t].double().repeat_interleave(g, 1)
        z = torch.einsum("hd,thd->ht", q[i].double(), k) * scale
        if cap:
            z = cap * torch.tanh(z / cap)
        if slopes is not None:
            z = z - slopes.double()[:, None] * (positions[i] - t).abs()
        p = torch.softmax(z, -1)
        P[:, t] = p
        outs.append(torch.einsum("ht,thd->hd", p, v))
        Ps.append(P)
    return torch.stack(outs), torch.stack(Ps)


def capped(S, cap):
    """What a cap adds to the error of scores of size S (its slope is at most 1): the cubic near zero is off
    by 5.5e-7 relative and its seven roundings by 2^-22 (less than 2^-20 together); where a score of
    half the cap is about, 1 - 2 / (1 + exp(2 x)) by 2^-21 of the cap (an exponential and a reciprocal
    of 2^-22, halved by their slope, the rounding of 2 x up to 2^-23 of it, two more)."""
    near = torch.minimum(S, torch.full_like(S, cap)) * 2.0 ** -20
    return near + (cap * 2.0 ** -21 if float(S.amax()) > cap / 2 else 0.0)


def prompt_bound(q, K, V, positions, P, seen, out, out_dtype, cap=0.0, slopes=None, scale=SCALE):
    """How far a prompt kernel's out may be from `out`.

    Scores: keys restored in binary32 and rounded to f16, half a step 2^-11 of each (2^-25
    below f16's normal range); products of f16 operands exact, sums of 128 of them in binary32
    2^-19 of what they add, a bf16 query's elements below 2^-28 of its largest lost (2^-28 of the
    largest for each of 128). A cap: capped().
    A bias |p - t| slope and what it is added to round to 2^-24 of themselves, three times.
    log2 units: times log2 e.
    P V: P rounded to f16, 2^-11 (2^-25 below the normal range, against a sum of P of at least
    1), values 2^-11 (2^-25), exponentials and binary32 sums 2^-19; the output half a step of its
    type."""
    H, g = K.shape[1], q.shape[1] // K.shape[1]
    rep = lambda x: x.double().abs().repeat_interleave(g, 1)  # noqa: E731
    fin = lambda x: torch.nan_to_num(x.double(), 0, 0, 0)  # noqa: E731
    see = seen.to(q.device)
    qa = q.double().abs()
    S = torch.einsum("qhd,thd->qht", qa, rep(fin(K)))
    S = torch.where(see[:, None], S, torch.zeros_like(S)).amax(-1) * scale
    small = (qa.sum(-1) * 2.0 ** -25 + 128 * qa.amax(-1) * 2.0 ** -28 * fin(K).abs().amax()) * scale
    dz = S * (2.0 ** -11 + 2.0 ** -19) + small
    if cap:
        dz = dz + capped(S, cap)
    if slopes is not None:
        t = torch.arange(K.shape[0], device=q.device)
        far = torch.stack([torch.where(see[i], (t - p).abs(), torch.zeros_like(t)).amax() for i, p in enumerate(positions)])
        dz = dz + 3 * 2.0 ** -24 * (slopes.double().abs()[None] * far[:, None].double() + S)
    dz = dz * LOG2E
    A = torch.einsum("qht,thd->qhd", P, rep(fin(V)))
    n = see.sum(-1)[:, None, None].double()
    M = fin(V).abs().amax()
    rel = 2.0 ** -10 + 2.0 ** -18 + 2 * (torch.exp2(dz)[..., None] - 1)
    half = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}[out_dtype]
    return rel * A + n * 2.0 ** -25 * M + half * out.abs() + 2.0 ** -24


def compare(got, want, tol, what=""):
    assert torch.isfinite(want).all()
    err = (got.double() - want).abs()
    assert bool((err <= tol).all()), f"{what}: error {float(err.max()):.3e}, {float((err / tol).max()):.2f} of the bound"
    return float((err / tol).max()) if err.numel() else 0.0


def attend_bound(q, K, V, mk, mv, positions, P, seen, out, out_dtype, bits, cap=0.0, slopes=None, scale=SCALE):
    """How far attention of the newest tokens with a score form may be from `out`: plain_cache.bound
    (the arithmetic up to the scores and from the probabilities on is that of windows), with the
    form's own errors on the scores as in prompt_bound."""
    from plain_cache import bound
    base = bound(q, K, V, mk, mv, P, seen.to(q.device), out, out_dtype, bits, scale)
    H, g = K.shape[1], q.shape[1] // K.shape[1]
    rep = lambda x: x.repeat_interleave(g, 1)  # noqa: E731
    fin = lambda x: torch.nan_to_num(x.double(), 0, 0, 0).abs()  # noqa: E731
    see = seen.to(q.device)
    S = torch.einsum("qhd,thd->qht", q.double().abs(), rep(fin(K) + mk.double()))
    S = torch.where(see[:, None], S, torch.zeros_like(S)).amax(-1) * scale
    dz = torch.zeros_like(S)
    if cap:
        dz = dz + capped(S, cap)
    if slopes is not None:
        t = torch.arange(K.shape[0], device=q.device)
        far = torch.stack([torch.where(see[i], (t - p).abs(), torch.zeros_like(t)).amax() for i, p in enumerate(positions)])
        dz = dz + 3 * 2.0 ** -24 * (slopes.double().abs()[None] * far[:, None].double() + S)
    A = torch.einsum("qht,thd->qhd", P, rep(fin(V) + mv.double()))
    return base + 2 * (torch.exp2(dz * LOG2E)[..., None] - 1) * A
