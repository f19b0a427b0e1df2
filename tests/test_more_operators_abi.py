"""Score forms, prompts, pages and forks on the CPU: refusals that need no device, structures, and
the plain model that the GPU tests compare with."""
import ctypes
import math
import os
import subprocess
import sys

import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from score_model import attention, seen_of

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_calls_without_a_cache_are_refused():
    one = torch.zeros(64, dtype=torch.int32)
    form = s4.s4kv_scores(0.0, None, 0, 0, None, None)
    for call in (lambda: s4.s4kv_score_attention(None, 0, form, one, 1, 1, one, 1, one, None, 1, 0.0, one, s4.S4KV_F32, one,
                                                 256, 1, stream=0),
                 lambda: s4.s4kv_prompt_workspace_bytes(None, 1, 1, 1, 1, 1),
                 lambda: s4.s4kv_prompt_attention(None, 0, form, one, 1, one, 1, one, 1, one, None, 1, 0.0, one, s4.S4KV_F32,
                                                  one, 256, 1, 1, stream=0),
                 lambda: s4.s4kv_take_pages(None, one, one, 1, 1, one, one, None, 1, one, stream=0),
                 lambda: s4.s4kv_release_pages(None, one, one, 1, 1, one, one, None, 1, stream=0),
                 lambda: s4.s4kv_fork(None, one, one, 1, 1, one, one, one, 1, one, stream=0)):
        with pytest.raises(s4.S4KVError) as e:
            call()
        assert e.value.code == s4.S4KV_ERR_INVALID_ARG


def test_score_forms_are_checked():
    assert ctypes.sizeof(s4.s4kv_scores) == 40
    s4.Scores(), s4.Scores(50.0, torch.ones(4), 4096, 4), s4.Scores(window=2 ** 40, num_sinks=2 ** 40)
    for kw in (dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-30), dict(window=-1),
               dict(num_sinks=-1), dict(slopes=torch.ones(4, dtype=torch.float64)), dict(slopes=torch.ones(2, 2)),
               dict(slopes=torch.ones(8)[::2])):
        with pytest.raises(ValueError):
            s4.Scores(**kw)


def test_score_forms_do_not_change():
    f = s4.Scores(50.0, torch.ones(4))
    for name in ("cap", "slopes", "window", "num_sinks"):
        with pytest.raises(AttributeError):
            setattr(f, name, None)
    assert f.cap == 50.0 and f.slopes.shape == (4,)


def test_plain_spans_are_the_documented_ones():
    see = lambda *a, **k: [r.nonzero().flatten().tolist() for r in seen_of(*a, **k)]  # noqa: E731
    assert see(6, [3, 5]) == [[0, 1, 2, 3], [0, 1, 2, 3, 4, 5]]
    assert see(6, [3, 5], window=2, sinks=1) == [[0, 2, 3], [0, 4, 5]]
    assert see(6, [2, 5], first=[2, 6]) == [[2], []]
    assert see(6, [1, 2], prefix=5) == [[0, 1, 2, 3, 4]] * 2
    assert see(6, [1, 4], prefix=99, window=2) == [[0, 1, 2, 3, 4, 5], [3, 4, 5]]
    assert see(6, [4], first=[9], sinks=2) == [[0, 1]]


def test_plain_scores_are_the_formula():
    q, K, V = torch.zeros(1, 1, 128), torch.zeros(2, 1, 128), torch.zeros(2, 1, 128)
    q[0, 0, 0], K[0, 0, 0], K[1, 0, 0], V[0, 0, 3], V[1, 0, 3] = 2.0, 3.0, -1.0, 1.0, 5.0
    out, P = attention(q, K, V, [1], seen_of(2, [1]), cap=4.0, slopes=torch.tensor([0.5]), scale=1.0)
    z0, z1 = 4 * math.tanh(6 / 4) - 0.5, 4 * math.tanh(-2 / 4)
    p0 = math.exp(z0) / (math.exp(z0) + math.exp(z1))
    assert abs(float(P[0, 0, 0]) - p0) < 1e-12 and abs(float(out[0, 0, 3]) - (p0 + 5 * (1 - p0))) < 1e-6


def test_the_binding_is_imported_without_torch():
    """Sizes and structures need the library alone."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "import int4_kivi_quantized_gb300 as s4\n"
            "print(s4.s4kv_cache_bytes(s4.make_config(1, 10, 2, 64, 4))[1], s4.Scores(50.0).cap)")
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert got.returncode == 0, got.stderr
    assert got.stdout.split()[1] == "50.0"
