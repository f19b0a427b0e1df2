"""Prompts of more sequences than a warp has lanes: wrong offsets, sequences that are refused, the most there may be."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from plain_cache import INT8
from test_gpu_prompt import Call

pytestmark = pytest.mark.gpu


def call(n, **kw):
    lens = [1 + (41 * i) % 150 for i in range(n)]
    return Call(lens, [min(x, (i * 7) % 23) for i, x in enumerate(lens)], H=1, g=3, bits=INT8, **kw)


@pytest.mark.parametrize("n", [33, 300])
def test_wrong_offsets(n):
    c = call(n, seed=71)
    good = c.run()
    c.check(good)
    out, cu = torch.full_like(good, 7.0), c.at

    def wrong(i, x):
        y = list(cu)
        y[i] = x
        return y
    for bad in (wrong(0, 1), wrong(0, -1), wrong(n, cu[n] - 1), wrong(n, cu[n] + 1), wrong(n // 2, -3), wrong(n // 2, cu[n] + 5),
                wrong(n - 1, cu[n] + 1), wrong(20, cu[25] + 1), wrong(1, 2 ** 31 - 1), wrong(n // 2, -2 ** 31), [0] * (n + 1)):
        c.cu = c.f.i32(bad)
        c.run(out=out)
        assert c.f.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_CU), bad
        assert bool((out == 7.0).all())
    c.cu = c.f.i32(cu)
    assert torch.equal(c.run(), good)
    c.f.ok()


def test_refused_sequences_among_many():
    c = call(200, seed=72)
    good = c.run()
    seq = list(c.f.lens)
    bad = [b for b in range(200) if c.chunks[b] and b % 9 == 0]
    for b in bad:
        seq[b] += 1
    c.f.seq = c.f.i32(seq)
    got = c.f.cache.prompt(0, c.q, c.cu, c.f.bt, c.f.seq, 200, sum(seq))
    assert c.f.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    for b in range(200):
        rows = slice(c.at[b], c.at[b + 1])
        assert not got[rows].any() if b in bad else torch.equal(got[rows], good[rows])


def test_as_many_as_there_may_be():
    c = call(4096, seed=73)
    got = c.run()
    c.check(got, skip=[b for b in range(4096) if b % 37])
