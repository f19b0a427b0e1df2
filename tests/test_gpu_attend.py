"""Attention of the newest tokens with a score form (KVCache.attend) on the GPU against the
plain model in 64 bits."""
import random

import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled
from score_model import attend_bound, attention, compare, seen_of

pytestmark = pytest.mark.gpu


class Call:
    def __init__(self, lens, nq=1, H=2, g=4, bits=4, dtype="bf16", residual=32, seed=0, cap=0.0, slopes=False, window=0,
                 sinks=0, first=None, prefix=None, **filled):
        self.f = Filled(lens, H=H, bits=bits, dtype=dtype, residual=residual, seed=seed, **filled)
        f, self.nq, self.Hq, self.bits = self.f, nq, H * g, bits
        self.q = inp.queries(seed + 5, len(lens) * nq, self.Hq, 128, f.dtype).to(f.dev).view(len(lens), nq, self.Hq, 128)
        rng = random.Random(seed)
        self.cap, self.window, self.sinks = cap, window, sinks
        self.slopes = torch.tensor([rng.uniform(0.0, 0.3) * (-1) ** (j == 1) for j in range(self.Hq)], device=f.dev) if slopes else None
        self.first = None if first is None else [[first(b, p) for p in self.positions(b)] for b in range(len(lens))]
        self.prefix = None if prefix is None else list(prefix)
        self.scores = s4.Scores(cap, self.slopes, window, sinks)

    def positions(self, b):
        return list(range(self.f.lens[b] - self.nq, self.f.lens[b]))

    def run(self, out_dtype=s4.S4KV_F32, **kw):
        f = self.f
        first = None if self.first is None else torch.tensor(self.first, dtype=torch.int32, device=f.dev)
        args = dict(first=first, prefix=None if self.prefix is None else f.i32(self.prefix), out_dtype=out_dtype, slot_ids=f.slots)
        args.update(kw)
        return f.cache.attend(0, self.q, f.bt, f.seq, max(f.lens + [1]), self.scores, **args)

    def check(self, got):
        for b, n in enumerate(self.f.lens):
            if n == 0:
                assert not got[b].any()
                continue
            K, V, mk, mv = self.f.plain(b)
            pos = self.positions(b)
            seen = seen_of(n, pos, self.window, self.sinks, None if self.first is None else self.first[b],
                           None if self.prefix is None else self.prefix[b])
            want, P = attention(self.q[b], K, V, pos, seen, self.cap, self.slopes)
            tol = attend_bound(self.q[b], K, V, mk, mv, pos, P, seen, want, got.dtype, self.bits, self.cap, self.slopes)
            compare(got[b], want, tol, f"sequence {b}")
        self.f.ok()


FORMATS = [(4, "bf16"), (4, "fp16"), (2, "bf16"), (8, "fp16"), (8, "bf16"), (INT8, "bf16"), (INT8, "fp16")]
FORMS = [0, 1, 2]   # of the launch: by size, slices, clusters


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("nq", [1, 5])
@pytest.mark.parametrize("bits,dtype", FORMATS)
def test_capped_and_sloped(bits, dtype, nq, form):
    c = Call([5, 16, 33, 64, 300, 777], nq=nq, bits=bits, dtype=dtype, cap=20.0, slopes=True, seed=1)
    c.f.cache.set_option(s4.S4KV_OPT_WINDOW_FORM, form)
    c.check(c.run())


@pytest.mark.parametrize("bits", [4, 2, 8, INT8])
def test_no_form_at_all(bits):
    c = Call([1, 100, 250], bits=bits, seed=2)
    c.check(c.run())
    plain = c.f.cache.window(0, c.q, c.f.bt, c.f.seq, 250, 1 << 20)
    assert torch.equal(c.run(), plain)


@pytest.mark.parametrize("cap", [0.25, 3.0, 50.0, 1e5])
@pytest.mark.parametrize("bits", [4, 8, INT8])
def test_caps(cap, bits):
    c = Call([40, 333], nq=2, bits=bits, cap=cap, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("g,nq", [(1, 16), (3, 7), (6, 16), (7, 1), (8, 12), (5, 3)])
@pytest.mark.parametrize("bits", [4, 8, INT8])
def test_columns(g, nq, bits):
    c = Call([90, 210], nq=nq, H=1, g=g, bits=bits, cap=10.0, slopes=True, seed=4)
    c.check(c.run())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (7, 3), (64, 40), (100, 0), (3, 1000)])
@pytest.mark.parametrize("bits", [4, 2, 8, INT8])
def test_windows(window, sinks, bits, form):
    c = Call([4, 130, 401], nq=4, bits=bits, window=window, sinks=sinks, slopes=True, seed=5)
    c.f.cache.set_option(s4.S4KV_OPT_WINDOW_FORM, form)
    c.check(c.run())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (2, "fp16"), (8, "bf16"), (INT8, "fp16")])
@pytest.mark.parametrize("sinks", [0, 37])
@pytest.mark.parametrize("prefix", [False, True])
def test_documents_and_prefixes(bits, dtype, sinks, prefix, form):
    # documents: before the newest tokens, among them, a query that sees nothing, all of them beyond
    first = lambda b, p: [-5, 70, 0, 2 ** 31 - 1][b] if p % 6 else p + (b == 2)  # noqa: E731
    c = Call([40, 200, 333, 90], nq=6, g=2, bits=bits, dtype=dtype, first=first, sinks=sinks,
             prefix=[39, 198, 5, 1 << 30] if prefix else None, seed=6)
    c.f.cache.set_option(s4.S4KV_OPT_WINDOW_FORM, form)
    c.check(c.run())


@pytest.mark.parametrize("bits", [4, 2, 8, INT8])
def test_long_caches_and_slots(bits):
    c = Call([2500, 0, 4000], bits=bits, residual=128, cap=30.0, slots=[2, 7, 0], seed=7)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_outputs_in_the_cache_dtype(dtype):
    c = Call([200, 700], nq=3, dtype=dtype, cap=5.0, seed=8)
    c.check(c.run(c.f.cache.cdtype))


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [4, INT8])
@pytest.mark.parametrize("nq", [1, 4])
def test_masked_rows_that_are_not_finite(what, bits, nq):
    # INT8 blocks of 16 restore whole to values that are not finite: the documents end with blocks
    def edit(b, k, v):
        k[195], v[197] = what, what
    c = Call([212], nq=nq, bits=bits, edit=edit, first=lambda b, p: 208, cap=10.0, residual=32, seed=9)
    got = c.run()
    K, V, mk, mv = c.f.plain(0)
    pos = c.positions(0)
    seen = seen_of(212, pos, first=[208] * nq)
    want, P = attention(c.q[0], K, V, pos, seen, 10.0)
    lo = 208 - 208 % 32   # (the model's error bound looks at the visible rows only)
    clean = lambda x: torch.nan_to_num(x, 0, 0, 0)  # noqa: E731
    tol = attend_bound(c.q[0], clean(K[lo:]), clean(V[lo:]), clean(mk[lo:]), clean(mv[lo:]), [p - lo for p in pos], P[..., lo:],
                       seen[:, lo:], want, got.dtype, bits, 10.0)
    compare(got[0], want, tol)


@pytest.mark.parametrize("bits", [4, INT8])
def test_a_query_of_nothing_beside_rows_that_are_not_finite(bits):
    def edit(b, k, v):
        k[:], v[180:] = 1.0, float("nan")
    c = Call([200], nq=2, bits=bits, edit=edit, first=lambda b, p: 2 ** 31 - 1, residual=32, seed=10)
    assert not c.run().any()
    c.f.ok()
