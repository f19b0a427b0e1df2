"""What a query does not see has no say in its row, not in the last bit either: later tokens, other documents'
and what rings and pages still hold."""
import pytest
import torch

import test_gpu_attend
import test_gpu_prompt
from plain_cache import INT8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("cap", [0.0, 3.0, 50.0])
@pytest.mark.parametrize("bits", [8, INT8, 4, 2])
def test_prompt_rows_before_other_tokens(bits, cap, slopes):
    # (8-bit floats stand alone; the others share scales in blocks of 32 tokens at most)
    cut = 167 if bits == 8 else 160

    def run(factor):
        def edit(b, k, v):
            k[cut:] *= factor
            v[cut:] *= -factor
        c = test_gpu_prompt.Call([300], [300], bits=bits, residual=32, edit=edit, cap=cap, slopes=slopes, seed=41)
        got = c.run()
        c.f.ok()
        return got
    a, b = run(1.0), run(25.0)
    assert torch.equal(a[:cut], b[:cut])
    assert not torch.equal(a[cut:], b[cut:])


@pytest.mark.parametrize("cap", [0.0, 50.0])
@pytest.mark.parametrize("bits", [4, INT8])
@pytest.mark.parametrize("what", [float("nan"), float("inf"), 30000.0])
def test_prompt_rows_before_values_that_are_not_finite(bits, cap, what):
    def run(x):
        def edit(b, k, v):
            k[293], v[294] = x, x
        c = test_gpu_prompt.Call([300], [200], bits=bits, residual=32, edit=edit, cap=cap, seed=42)
        return c.run()
    a, b = run(1.0), run(what)
    assert torch.equal(a[:193], b[:193])


@pytest.mark.parametrize("cap", [3.0, 50.0])
@pytest.mark.parametrize("bits", [4, 2, 8, INT8])
def test_newest_token_beside_another_document(bits, cap):
    # the document starts in the unfinished block, whose rows are in 16 bits
    def run(factor):
        def edit(b, k, v):
            k[288:294] *= factor
            v[288:294] *= factor
        c = test_gpu_attend.Call([300], nq=1, bits=bits, residual=32, edit=edit, cap=cap, first=lambda b, p: 294, seed=43)
        got = c.run()
        c.f.ok()
        return got
    assert torch.equal(run(1.0), run(40.0))


@pytest.mark.parametrize("cap", [3.0, 50.0])
@pytest.mark.parametrize("bits", [4, 8, INT8])
def test_newest_tokens_beside_what_the_slot_held_before(bits, cap):
    """A slot that held a longer sequence of large numbers, and one that held nothing."""
    outs = []
    for before in (False, True):
        c = test_gpu_attend.Call([203], nq=2, bits=bits, residual=32, cap=cap, spare=64, seed=44)
        f = c.f
        if before:
            big = torch.full((263, 2, 128), 300.0, dtype=f.dtype, device="cuda")
            f.cache.append(0, big, big, f.i32([0, 263]), f.i32([0]), f.bt)
            f.append_to([0], [203])
        outs.append(c.run())
        f.ok()
    assert torch.equal(*outs)


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (2, "fp16"), (8, "bf16"), (INT8, "fp16")])
def test_calls_repeat_bit_for_bit(bits, dtype):
    c = test_gpu_prompt.Call([3000, 700, 41], [70, 300, 41], bits=bits, dtype=dtype, cap=30.0, slopes=True, seed=45)
    d = test_gpu_attend.Call([3000, 700, 41], nq=4, bits=bits, dtype=dtype, cap=30.0, seed=46)
    a, b = c.run(), d.run()
    for _ in range(5):
        assert torch.equal(c.run(), a) and torch.equal(d.run(), b)
    c.f.ok(), d.f.ok()
