"""Forks of sources with holes among the pages that have to be copied."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from plain_cache import INT8
from test_gpu_pages import Fork, done_of, i32, ok, up

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits,R", [(4, 32), (4, 200), (2, 20), (8, 32)])
@pytest.mark.parametrize("bad", [-1, -5, 10 ** 6])
def test_forks_of_a_source_with_a_hole(bits, R, bad):
    """A page that the fork would have to copy is missing: nothing of that fork is done, the others are."""
    n = 261
    f = Fork([n, n, 70], 5, bits, R=R, layers=2, seed=3)
    done, held = done_of(bits, n, R), up(n) if bits == 8 else -(-max(n // 32 * 32, n - R) // 16)
    assert held > done
    for e in {done, held - 1}:
        keep = int(f.table[1, e])
        f.table[1, e] = bad
        table, refs, lens = f.table.clone(), f.refs.clone(), f.c.pool[f.c.layout.lens_offset:f.c.layout.layer_offset].clone()
        got = f.c.fork(f.refs, f.table, i32([1, 1]), i32([3, 5]), i32([n, n]))
        assert got.tolist() == [-1, -1]
        assert f.c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)
        assert torch.equal(f.table, table) and torch.equal(f.refs, refs)
        assert torch.equal(f.c.pool[f.c.layout.lens_offset:f.c.layout.layer_offset], lens)
        got = f.c.fork(f.refs, f.table, i32([0, 1, 2]), i32([3, 5, 6]), i32([n, n, 70]))
        assert got[1] == -1 and int(got[0]) == up(n) - done and int(got[2]) >= 0
        assert f.c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)
        for s, d, x in ((0, 3, n), (2, 6, 70)):
            for layer in range(2):
                for a, b in zip(f.restored(layer, s, x), f.restored(layer, d, x)):
                    assert torch.equal(a, b)
        ok(f.c)
        assert (f.table[5] == -1).all()
        f.c.release_pages(f.refs, f.table, i32([0, 0]), i32([n, 70]), slot_ids=i32([3, 6]))
        assert torch.equal(f.refs, refs)
        f.table[1, e] = keep
    # entries that nothing is copied from may be holes, as behind a window
    if done:
        f.c.release_pages(f.refs, f.table, i32([0]), i32([16]), slot_ids=i32([1]))
        assert int(f.c.fork(f.refs, f.table, i32([1]), i32([4]), i32([n]))[0]) == up(n) - done
        assert int(f.table[4, 0]) == -1
        ok(f.c)


def test_forks_of_int8_pages_copy_none():
    f = Fork([40], 1, INT8)
    f.table[0, 2] = -1   # the unfinished block's page, which nothing is written to yet
    assert f.c.fork(f.refs, f.table, i32([0]), i32([1]), i32([40])).tolist() == [1]
    ok(f.c)
