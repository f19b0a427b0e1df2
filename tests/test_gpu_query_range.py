"""bf16 queries beyond f16's range, over keys of the inverse size: attention on INT8 pages (blocks and
the unfinished one) and windows on FP8 pages."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled, check

pytestmark = pytest.mark.gpu


def _filled(bits, power, lens, flat=False):
    """Keys of kv head h times 2^-power[h] (FP8: by the head's scale); flat: channel 0 holds zeros."""
    def edit(b, k, v):
        for h, p in enumerate(power):
            k[:, h] = (k[:, h].float() * 2.0 ** -p).to(k.dtype)
        if flat:
            k[:, :, 0] = 0
    return Filled(lens, H=len(power), bits=bits, seed=9, edit=edit,
                  fp8_scales=([2.0 ** -p for p in power], [1.0] * len(power)) if bits == 8 else None)


def _all(f, q, window):
    B, nq = q.shape[:2]
    out = f.cache.window(0, q, f.bt, f.seq, max(f.lens), window, 2)
    f.ok()
    for b, n in enumerate(f.lens):
        check(out[b], q[b], *f.plain(b), range(n - nq, n), f.bits, window, 2, f"seq {b} of {n}, window {window}")
    if f.bits == INT8:
        out = f.cache.multi_query(0, q, f.bt, f.seq, max(f.lens))
        f.ok()
        for b, n in enumerate(f.lens):
            check(out[b], q[b], *f.plain(b), range(n - nq, n), INT8, what=f"seq {b} of {n}")


@pytest.mark.parametrize("bits", [INT8, 8])
@pytest.mark.parametrize("form", [0, 1, 2])
@pytest.mark.parametrize("nq", [1, 4])
@pytest.mark.parametrize("power", [(17, -20), (40, -40), (90, -90), (0, 1)])
def test_queries_of_any_size(bits, form, nq, power):
    f = _filled(bits, power, [5, 100, 333])
    f.cache.set_option(s4.S4KV_OPT_WINDOW_FORM, form)
    q = torch.randn(3, nq, 8, 128, generator=inp.gen(4))
    q[:, :, :4] *= 2.0 ** power[0]
    q[:, :, 4:] *= 2.0 ** power[1]
    q = q.to(torch.bfloat16).cuda()
    for window in (60, 1000):
        _all(f, q, window)


@pytest.mark.parametrize("bits", [INT8, 8])
@pytest.mark.parametrize("nq", [1, 4])
def test_small_elements_beside_a_large_one(bits, nq):
    """One element of 2^12, the others about 2^-16 (f16 has them as subnormals), the keys about 2^14 and
    zero at the large one's channel; a head of zeros, and columns that all differ in size."""
    f = _filled(bits, (-14, -14), [100, 200], flat=True)
    q = torch.randn(2, nq, 8, 128, generator=inp.gen(5)) * 2.0 ** -16
    q[..., 0] = 4096.0
    q[:, :, 3] = 0
    q = q.to(torch.bfloat16).cuda()
    _all(f, q, 50)
    q = torch.randn(2, nq, 8, 128, generator=inp.gen(6)) * torch.exp2(-torch.arange(8.0) - 13)[:, None]
    _all(f, q.to(torch.bfloat16).cuda(), 1000)


def test_a_query_that_is_not_finite_is_its_own_rows_loss():
    f = _filled(INT8, (0, 0), [100])
    q = torch.randn(1, 2, 8, 128, generator=inp.gen(7)).to(torch.bfloat16).cuda()
    want = f.cache.window(0, q, f.bt, f.seq, 100, 60, 2)
    bad = q.clone()
    bad[0, 0, 1, 5], bad[0, 1, 6, 7] = float("inf"), float("nan")
    out = f.cache.window(0, bad, f.bt, f.seq, 100, 60, 2)
    f.ok()
    for i in range(2):
        for h in range(8):
            if (i, h) in ((0, 1), (1, 6)):
                assert torch.isnan(out[0, i, h]).all()
            else:
                assert torch.equal(out[0, i, h], want[0, i, h])
