"""Prompt attention (KVCache.prompt) on the GPU against the plain model in 64 bits."""
import random

import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled
from score_model import attention, compare, prompt_bound, seen_of

pytestmark = pytest.mark.gpu


class Call:
    """A filled cache, chunks of its sequences' newest tokens, and a score form."""

    def __init__(self, lens, chunks, H=2, g=4, bits=4, dtype="bf16", residual=32, seed=0, cap=0.0, slopes=False, window=0,
                 sinks=0, first=None, prefix=None, **filled):
        self.f = Filled(lens, H=H, bits=bits, dtype=dtype, residual=residual, seed=seed, **filled)
        f, self.chunks, self.Hq = self.f, list(chunks), H * g
        self.q = inp.queries(seed + 5, sum(chunks), self.Hq, 128, f.dtype).to(f.dev).view(-1, self.Hq, 128)
        cu = [0]
        for m in chunks:
            cu.append(cu[-1] + m)
        self.at, self.cu = cu, f.i32(cu)
        self.cap, self.window, self.sinks = cap, window, sinks
        rng = random.Random(seed)
        self.slopes = torch.tensor([rng.uniform(0.0, 0.3) * (-1) ** (j == 1) for j in range(self.Hq)], device=f.dev) if slopes else None
        # first: per query, from `first(sequence, position)`; prefix: per sequence
        self.first = None if first is None else [first(b, p) for b in range(len(lens)) for p in self.positions(b)]
        self.prefix = None if prefix is None else list(prefix)
        self.scores = s4.Scores(cap, self.slopes, window, sinks)

    def positions(self, b):
        return range(self.f.lens[b] - self.chunks[b], self.f.lens[b])

    def run(self, out_dtype=None, **kw):
        f = self.f
        args = dict(scores=self.scores, first=None if self.first is None else f.i32(self.first),
                    prefix=None if self.prefix is None else f.i32(self.prefix),
                    out_dtype=s4.S4KV_F32 if out_dtype is None else out_dtype, slot_ids=f.slots)
        args.update(kw)
        return f.cache.prompt(0, self.q, self.cu, f.bt, f.seq, max(f.lens + [1]), sum(f.lens), **args)

    def seen(self, b):
        first = None if self.first is None else self.first[self.at[b]:self.at[b + 1]]
        return seen_of(self.f.lens[b], list(self.positions(b)), self.window, self.sinks, first,
                       None if self.prefix is None else self.prefix[b])

    def check(self, got, skip=()):
        worst = 0.0
        for b, m in enumerate(self.chunks):
            if m == 0 or b in skip:
                continue
            K, V, _, _ = self.f.plain(b)
            q, pos, seen = self.q[self.at[b]:self.at[b + 1]], list(self.positions(b)), self.seen(b)
            want, P = attention(q, K, V, pos, seen, self.cap, self.slopes)
            tol = prompt_bound(q, K, V, pos, P, seen, want, got.dtype, self.cap, self.slopes)
            worst = max(worst, compare(got[self.at[b]:self.at[b + 1]], want, tol, f"sequence {b}"))
        self.f.ok()
        return worst


FORMATS = [(4, "bf16"), (4, "fp16"), (2, "bf16"), (8, "fp16"), (8, "bf16"), (INT8, "bf16"), (INT8, "fp16")]


@pytest.mark.parametrize("bits,dtype", FORMATS)
def test_one_whole_prompt(bits, dtype):
    c = Call([300], [300], bits=bits, dtype=dtype)
    c.check(c.run())


@pytest.mark.parametrize("bits,dtype", FORMATS)
def test_ragged_chunks(bits, dtype):
    # none, one token, a chunk that ends a page, whole prompts, lengths around tiles and blocks
    c = Call([77, 1, 130, 256, 129, 400], [0, 1, 16, 256, 129, 37], bits=bits, dtype=dtype, seed=3)
    c.check(c.run())


@pytest.mark.parametrize("g", [1, 2, 3, 5, 6, 7, 8])
@pytest.mark.parametrize("H", [1, 3])
def test_head_groups(g, H):
    c = Call([200, 131], [97, 131], H=H, g=g, bits=INT8, seed=g)
    c.check(c.run())


@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0, 1e4])
@pytest.mark.parametrize("bits", [4, INT8])
def test_caps(cap, bits):
    c = Call([150, 90], [150, 20], bits=bits, cap=cap, seed=7)
    c.check(c.run())


@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_slopes(cap):
    c = Call([260, 90], [130, 20], cap=cap, slopes=True, seed=8)
    c.check(c.run())


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (40, 0), (130, 4), (1000, 200)])
@pytest.mark.parametrize("bits", [4, 8])
def test_windows(window, sinks, bits):
    c = Call([500, 140, 3], [200, 33, 3], bits=bits, window=window, sinks=sinks, seed=9)
    c.check(c.run())


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("window", [0, 50])
def test_documents_and_prefixes(prefix, window):
    # documents that start inside the chunk, before it, and where a query sees nothing
    first = lambda b, p: p + 1 if p == 170 else 160 if p > 160 else 40 if p > 40 else -3  # noqa: E731
    c = Call([250, 200], [200, 120], bits=INT8, first=first, prefix=[90, 1000] if prefix else None, window=window, slopes=True,
             sinks=0, seed=10)
    got = c.run()
    c.check(got)
    if not prefix and window == 0:
        assert not got[170 - 50].any()   # nothing to see: zeros


def test_first_beyond_everything_and_sinks():
    c = Call([100], [40], first=lambda b, p: 2 ** 31 - 1, sinks=5, seed=11)
    c.check(c.run())
    d = Call([100], [40], first=lambda b, p: 2 ** 31 - 1, seed=11)
    assert not d.run().any()
    d.f.ok()


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (2, "fp16"), (8, "bf16"), (INT8, "fp16")])
@pytest.mark.parametrize("chunk", [1, 33])
def test_few_rows_behind_a_long_cache(bits, dtype, chunk):
    # the cache's length is split over CTAs
    c = Call([3000, 1500], [chunk, 5], bits=bits, dtype=dtype, residual=128, cap=30.0, seed=12)
    c.check(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_outputs_in_the_cache_dtype(dtype):
    c = Call([200, 700], [64, 9], dtype=dtype, seed=13)
    c.check(c.run(c.f.cache.cdtype))


def test_slots_in_any_order():
    c = Call([140, 90, 60], [20, 90, 1], slots=[5, 0, 3], seed=14)
    c.check(c.run())


@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("bits", [4, 8, INT8])
def test_masked_rows_that_are_not_finite(what, bits):
    # tokens of another document, and later tokens of the chunk, in the newest 16-bit rows
    def edit(b, k, v):
        k[200], v[201] = what, what
    if bits == 8:   # (e4m3 has no infinity and appends finite values only)
        def edit(b, k, v):  # noqa: F811
            k[200], v[201] = 448.0, -448.0
    c = Call([206], [26], bits=bits, residual=32, edit=edit, first=lambda b, p: 202 if p >= 202 else 0, seed=15)
    got = c.run()
    keep = [i for i, p in enumerate(c.positions(0)) if p < 200 or p >= 202]
    K, V, _, _ = c.f.plain(0)
    pos, seen = [list(c.positions(0))[i] for i in keep], c.seen(0)[keep]
    want, P = attention(c.q[keep], K, V, pos, seen)
    compare(got[keep], want, prompt_bound(c.q[keep], K, V, pos, P, seen, want, got.dtype))
    if bits != 8:
        assert torch.isnan(got[21]).all()   # position 201 sees both
    c.f.ok()


def test_large_and_small_queries():
    c = Call([130], [130], dtype="bf16", bits=INT8, seed=16)
    for factor in (2.0 ** 60, 2.0 ** -60):
        c.q = (inp.queries(21, 130, c.Hq, 128, c.f.dtype).to(c.f.dev) * factor).to(c.f.dtype).view(-1, c.Hq, 128)
        got = c.run(sm_scale=1.0 / factor / 11.3)
        K, V, _, _ = c.f.plain(0)
        pos, seen = list(range(130)), c.seen(0)
        scale = 1.0 / factor / 11.3
        want, P = attention(c.q, K, V, pos, seen, scale=scale)
        compare(got, want, prompt_bound(c.q, K, V, pos, P, seen, want, got.dtype, scale=scale))


def test_many_sequences():
    lens = [1 + (37 * i) % 90 for i in range(300)]
    c = Call(lens, [min(n, 1 + i % 7) if i % 3 else 0 for i, n in enumerate(lens)], H=1, g=2, bits=INT8, seed=17)
    c.check(c.run())
