"""Capped scores over the whole range of caps and of queries: caps far above every score, where the form is
the scores themselves, and far below, where it is all but none; queries of zeros and of any size."""
import pytest
import torch

import test_gpu_attend
import test_gpu_prompt
from plain_cache import INT8

pytestmark = pytest.mark.gpu

CAPS = [2.0 ** -60, 1e-9, 1e-3, 4e4, 1e6, 1e8, 2.0 ** 60]
FORMATS = [(4, "bf16"), (2, "fp16"), (8, "fp16"), (INT8, "bf16")]


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("bits,dtype", FORMATS)
def test_prompts(bits, dtype, cap):
    c = test_gpu_prompt.Call([300, 90], [170, 20], bits=bits, dtype=dtype, cap=cap, seed=31)
    c.q[40:60] = 0.0           # whole warps of rows and parts of them
    c.q[100, 3] = 0.0
    c.check(c.run())


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("bits,dtype", FORMATS)
def test_sloped_prompts(bits, dtype, cap):
    c = test_gpu_prompt.Call([300, 90], [170, 20], bits=bits, dtype=dtype, cap=cap, slopes=True, seed=32)
    c.q[40:60] = 0.0
    c.check(c.run())


@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("bits,dtype", FORMATS)
def test_newest_tokens(bits, dtype, cap):
    c = test_gpu_attend.Call([40, 333], nq=3, bits=bits, dtype=dtype, cap=cap, seed=33)
    c.q[1, 1] = 0.0
    c.check(c.run())


@pytest.mark.parametrize("cap", [2.0 ** -60, 1e-9, 1e8, 2.0 ** 60])
def test_nothing_but_queries_of_zeros(cap):
    """Every score is zero, every visible token counts as much as another."""
    c = test_gpu_prompt.Call([200], [200], bits=8, cap=cap, seed=34)
    c.q.zero_()
    c.check(c.run())
    d = test_gpu_attend.Call([200], nq=2, bits=8, cap=cap, seed=34)
    d.q.zero_()
    d.check(d.run())


def test_queries_of_all_sizes_below_a_cap_far_above():
    """Rows of one warp whose queries differ by powers of two: each goes through the cap as it would alone."""
    c = test_gpu_prompt.Call([260], [130], bits=INT8, cap=2.0 ** 40, seed=35)
    c.q *= torch.tensor([1.0, 2.0 ** -9, 2.0 ** -40, 0.0], dtype=c.q.dtype, device="cuda").repeat(33)[:130, None, None]
    c.check(c.run())


@pytest.mark.parametrize("slopes", [False, True])
@pytest.mark.parametrize("cap", [0.7, 6.0, 50.0])
def test_rows_near_zero_beside_rows_beyond(cap, slopes):
    """Small and large queries in one warp: some rows' scores pass half of the cap, their neighbours' do not."""
    c = test_gpu_prompt.Call([400], [200], bits=4, dtype="bf16", cap=cap, slopes=slopes, seed=36)
    by = [1.0, 2.0 ** -14, 8.0, 2.0 ** -5, 0.0, 2.0 ** -30, 0.25]
    c.q *= torch.tensor(by, dtype=c.q.dtype, device="cuda").repeat(29)[:200, None, None]
    c.check(c.run())
