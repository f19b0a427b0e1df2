"""How far a sequence's pages may be given back: not ahead of what has still to be written to them."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from plain_cache import INT8, Filled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 2, 8, INT8])
def test_appends_behind_released_pages(bits):
    """Window 40, residual 128: KIVI pages from token T - R on still get values as tokens leave the ring, so that they stay;
    8-bit pages that are full go."""
    T, R, W, m = 300, 128, 40, 90
    kivi = bits in (4, 2)
    for ahead in (False, True):
        f = Filled([T], H=2, bits=bits, residual=R, spare=200, seed=81)
        refs = torch.zeros(f.cache.cfg.num_pages, dtype=torch.int32, device="cuda")
        refs[f.bt[0].long()] = 1
        block = 32 if kivi else 16
        last = (min(T + 1 - W, T // 32 * 32, T - R) if kivi and not ahead else T + 1 - W) // block * block
        f.cache.release_pages(refs, f.bt, f.i32([0]), f.i32([last]))
        f.ok()
        k, v = (torch.randn(m, 2, 128, device="cuda").to(f.dtype) for _ in range(2))
        f.cache.append(0, k, v, f.i32([0, m]), f.i32([T]), f.bt)
        q = torch.randn(1, 1, 8, 128, device="cuda").to(f.dtype)
        if kivi and ahead:   # values of tokens 172 .. 261 have no page to go to
            assert f.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)
        else:
            out = f.cache.attend(0, q, f.bt, f.i32([T + m]), T + m, s4.Scores(window=W))
            assert torch.isfinite(out).all()
            f.ok()
