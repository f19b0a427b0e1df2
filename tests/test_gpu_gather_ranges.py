"""Ranges of the batched restore: a sequence without rows is not looked at."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from plain_cache import INT8, Filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 2, 8, INT8])
def test_a_sequence_without_rows_may_hold_anything(bits):
    f = Filled([100, 50, 70], H=2, bits=bits, residual=32, seed=4)
    bt = f.bt.clone()
    bt[1] = -5
    k, v = f.cache.gather(0, bt, f.i32([100, 9999, 70]), f.i32([0, 40, 40, 100]), 100, first=f.i32([60, 123456, 10]),
                          slot_ids=f.i32([0, 77, 2]))
    f.ok()
    (K0, V0, _, _), (K2, V2, _, _) = f.plain(0), f.plain(2)
    assert torch.equal(k, torch.cat([K0[60:], K2[10:]])) and torch.equal(v, torch.cat([V0[60:], V2[10:]]))
    k, v = f.cache.gather(0, bt, f.i32([-1, 3, 1 << 30]), f.i32([0, 0, 0, 0]), 0)
    f.ok()
    assert k.shape == (0, 2, 128)
    with pytest.raises(s4.S4KVError):     # rows of no sequence
        s4.s4kv_gather(f.cache.h, 0, bt, bt.shape[1], f.seq, None, None, f.i32([0]), 5, 0, f.k[0], f.v[0], f.cache.cdtype)
