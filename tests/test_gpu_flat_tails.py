"""Prompts whose probabilities lie far below the largest: many tokens that weigh little each are not lost in the
16-bit products."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4

pytestmark = pytest.mark.gpu


def outputs(T, m, gap, first, split=False):
    """Token `first` has a score `gap` powers of two above all others and a value of zero, the others ones."""
    dev, i32 = "cuda", lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    pages = -(-T // 16)
    c = s4.KVCache(1, pages, 1, 32, 1, "fp16", bits=8)
    k, v = torch.zeros(T, 1, 128, dtype=torch.float16, device=dev), torch.ones(T, 1, 128, dtype=torch.float16, device=dev)
    k[first, 0, 0], v[first] = 8.0, 0.0
    bt = torch.arange(pages, dtype=torch.int32, device=dev)[None]
    c.append(0, k, v, i32([0, T]), i32([0]), bt)
    q = torch.zeros(m, 1, 128, dtype=torch.float16, device=dev)
    q[:, 0, 0] = 1.0
    out = c.prompt(0, q, i32([0, m]), bt, i32([T]), T, sm_scale=gap * 0.6931471805599453 / 8.0)
    assert c.status()[0] == 0
    return out


@pytest.mark.parametrize("gap", [20.0, 24.0, 25.5, 26.5, 29.0])
@pytest.mark.parametrize("T,m", [(300, 150), (5000, 3), (70000, 20)])
def test_many_small_probabilities(T, m, gap):
    """P is held in f16 against a reference 7 powers of two below the largest so far, so that what lies
    2^-gap below the largest is rounded by 2^-32 of it at most; the values are exact."""
    for first in (0, T - m - 5):
        got = outputs(T, m, gap, first).double()
        others = torch.arange(T - m, T, dtype=torch.float64, device="cuda")   # tokens seen beside the large one
        want = others * 2.0 ** -gap / (1 + others * 2.0 ** -gap)
        # scores exact but for the scale's rounding and their product's: gap (2^-24 + 2^-23), as a factor of each p
        tol = others * 2.0 ** -32 + want * (2.0 ** -11 + 2.0 ** -18 + gap * 2.0 ** -22)
        assert bool(((got - want[:, None, None]).abs() <= tol[:, None, None]).all()), float(((got - want[:, None, None]).abs() / tol[:, None, None]).amax())
