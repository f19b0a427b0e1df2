"""The launch form of window calls as the library chooses it (S4KV_OPT_WINDOW_FORM = 0), on both sides
of each bound of its rule, and the form that is asked for where the grid cannot hold it."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled, check

pytestmark = pytest.mark.gpu
FORMATS = [4, 2, 8, INT8]
SLICES, CLUSTERS = 1, 2


def _queries(seed, B, Hq, dtype):
    return torch.randn(B, 1, Hq, 128, generator=inp.gen(seed), dtype=torch.float32).to(dtype).cuda()


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _same(f, q, top, window, want, b0=0):
    """Form 0 gives the bits of the form `want`; sequences from b0 on are checked against the plain model."""
    got = {}
    for form in (0, SLICES, CLUSTERS):
        f.cache.set_option(s4.S4KV_OPT_WINDOW_FORM, form)
        got[form] = f.cache.window(0, q, f.bt, f.seq, top, window)
        f.ok()
    assert torch.equal(got[0], got[want])
    for b in range(b0, len(f.lens), max(1, len(f.lens) // 5)):
        for out in got.values():
            check(out[b], q[b], *f.plain(b), [f.lens[b] - 1], f.bits, window)


@pytest.mark.parametrize("bits", FORMATS)
def test_one_segment_more_than_sms(bits):
    """Segments: sequences, one kv head each."""
    for B, want in ((_sms(), CLUSTERS), (_sms() + 1, SLICES)):
        lens = [33 + (7 * i) % 50 for i in range(B)]
        f = Filled(lens, H=1, bits=bits, residual=16, seed=2)
        _same(f, _queries(1, B, 4, f.dtype), max(lens), 2000, want)


@pytest.mark.parametrize("bits", FORMATS)
def test_longest_segment_of_a_cluster(bits):
    """With a segment for every SM but one a cluster is one CTA, whose twelve warps take at most 384 tokens each; the
    longest length is the caller's bound, whatever the lengths are."""
    B, block = _sms() - 1, 32 if bits in (4, 2) else 16
    f = Filled([50 + i for i in range(B)], H=1, bits=bits, residual=16, seed=3)
    q = _queries(2, B, 4, f.dtype)
    at = 12 * 384 - 2 * block + block     # the first bound whose blocks, with the two cut ones, are more
    _same(f, q, at - 1, 10000, CLUSTERS)
    _same(f, q, at, 10000, SLICES)
    _same(f, q, 30000, at - 2, CLUSTERS)   # the window and its query token: as many
    _same(f, q, 30000, at - 1, SLICES)


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("extra", [-1, 0, 700])
def test_clusters_of_eight_and_sixteen(bits, extra):
    """From 193 blocks on a call of at most six segments takes clusters of 16 CTAs."""
    block = 32 if bits in (4, 2) else 16
    top = 191 * block + extra
    f = Filled([top, 700], H=2, bits=bits, residual=16, seed=4)
    _same(f, _queries(3, 2, 8, f.dtype), top, 100000, CLUSTERS)


@pytest.mark.parametrize("bits", FORMATS)
def test_cluster_sizes_between(bits):
    """Clusters of 1, 2, 4 and 8, by the segments that the SMs leave room for."""
    for B in (70, 35, 17, 9):
        f = Filled([400 + 3 * i for i in range(B)], H=1, bits=bits, residual=16, seed=B)
        _same(f, _queries(B, B, 2, f.dtype), max(f.lens), 100000, CLUSTERS)


def test_clusters_asked_for_beyond_the_grid():
    """4096 sequences of 16 kv heads are 65536 segments, one more than a grid holds: slices."""
    B, H = 4096, 16
    lens = [1 + i % 3 for i in range(B)]
    f = Filled(lens, H=H, bits=INT8, seed=5)
    q = _queries(4, B, H, f.dtype)
    _same(f, q, 3, 10, SLICES, b0=17)
    f.cache.set_option(s4.S4KV_OPT_WINDOW_FORM, CLUSTERS)
    out = f.cache.window(0, q, f.bt, f.seq, 3, 10)
    f.cache.set_option(s4.S4KV_OPT_WINDOW_FORM, SLICES)
    assert torch.equal(out, f.cache.window(0, q, f.bt, f.seq, 3, 10))
    f.ok()
