"""INT8 pages, rotating appends, windowed attention and the batched restore on the CPU: ledger,
pool size, refusals that need no device, and the plain model that the GPU tests compare with."""
import ctypes

import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from plain_cache import INT8, attention, int8_rows, kivi_rows, restored


def test_int8_configuration_ledger_and_pool():
    L, P, H, S = 3, 10, 2, 4
    cfg = s4.make_config(L, P, H, 64, S, bits=s4.S4KV_BITS_INT8)
    r = s4.s4kv_kv_bytes(cfg, 5, 100)
    lbh = L * 5 * H
    assert r["code_bytes"] == lbh * 100 * 128 * 2
    assert r["meta_bytes"] == lbh * 6 * 8                 # two scales for each of 6 whole blocks
    assert r["residual_bytes"] == lbh * 2 * 16 * 128 * 2   # rings of one block
    assert r["paged_bytes"] == lbh * 7 * 4128
    pool, per = s4.s4kv_cache_bytes(cfg)
    assert per == 258
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    rings = up(S * H * 16 * 256) * 2
    header = up(up(256 + L * S * H * 4) + S * H * 4)
    assert pool == header + L * (up(P * H * 4128) + rings)
    tokens, pages = s4.s4kv_capacity_tokens(cfg, 1e9)
    fit, _ = s4.s4kv_cache_bytes(s4.make_config(L, pages, H, 64, S, bits=s4.S4KV_BITS_INT8))
    over, _ = s4.s4kv_cache_bytes(s4.make_config(L, pages + 1, H, 64, S, bits=s4.S4KV_BITS_INT8))
    assert tokens == 16 * pages and fit <= 1e9 < over
    for bad in (0x100, 0x102, 0x104, 9, 0x208, -8):
        with pytest.raises(s4.S4KVError) as e:
            s4.s4kv_cache_bytes(s4.make_config(1, 10, 2, 64, 4, bits=bad))
        assert e.value.code == s4.S4KV_ERR_UNSUPPORTED, bad


def test_calls_without_a_cache_are_refused():
    one = torch.zeros(64, dtype=torch.int32)
    rope = s4.s4kv_rope(one.data_ptr(), 1, 16, 0)
    for call in (lambda: s4.s4kv_append_rope(None, 0, rope, one, one, 1, one, None, one, one, 1, 1, stream=0),
                 lambda: s4.s4kv_window_workspace_bytes(None, 1, 1, 1, 1),
                 lambda: s4.s4kv_window_attention(None, 0, one, 1, 1, 1, 0, one, 1, one, None, 1, 0.0, one, s4.S4KV_F32,
                                                  one, 256, 1, stream=0),
                 lambda: s4.s4kv_gather(None, 0, one, 1, one, None, None, one, 1, 1, one, one, s4.S4KV_F32, stream=0)):
        with pytest.raises(s4.S4KVError) as e:
            call()
        assert e.value.code == s4.S4KV_ERR_INVALID_ARG


def test_rotation_tables_are_checked():
    s4.Rope(torch.zeros(4, 64))
    for t in (torch.zeros(4, 64, dtype=torch.float64), torch.zeros(256), torch.zeros(64, 4).t(), torch.zeros(2, 4, 64)):
        with pytest.raises(ValueError):
            s4.Rope(t)
    assert ctypes.sizeof(s4.s4kv_rope) == 24


def test_plain_int8_rule():
    x = torch.zeros(35, 2, 128)
    x[3, 0, 7], x[4, 0, 8], x[20, 1, 1] = 127.0, -63.5, 1e-31
    codes, sc, y = int8_rows(x)
    assert sc[0, 0] == 1.0 and sc[1, 1] == 0.0 and codes.shape[0] == 2
    assert codes[0, 3, 0, 7] == 127 and codes[0, 4, 0, 8] == -64     # half to even
    assert torch.equal(y[32:], x[32:]) and y[4, 0, 8] == -64.0
    g = torch.Generator().manual_seed(1)
    x = torch.randn(64, 3, 128, generator=g)
    _, sc, y = int8_rows(x)
    step = sc.repeat_interleave(16, 0)[..., None]
    assert bool(((x - y).abs() <= step * (0.5 + 2 ** -15)).all())


@pytest.mark.parametrize("bits", [4, 2])
def test_plain_kivi_rule_is_the_oracles(bits):
    import oracle
    import s4kv_inputs as inp
    k, v = inp.kv_rows(3, 100, 2, 128, torch.float16)
    seq = oracle.Seq(num_kv_heads=2, residual_v=20, dtype=oracle.F16, bits=bits)
    seq.append(inp.to_bits(k), inp.to_bits(v))
    K, V = kivi_rows(k, bits, 20, True)[0], kivi_rows(v, bits, 20, False)[0]
    for h in range(2):
        rk, rv = seq.dequant(h)
        assert torch.equal(K[:, h], torch.from_numpy(rk)) and torch.equal(V[:, h], torch.from_numpy(rv))


def test_plain_window_is_the_documented_mask():
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(20, 1, 128, generator=g).half() for _ in range(2))
    q = torch.randn(2, 1, 128, generator=g).half()
    K, V, _, _ = restored(k, v, INT8, 1)
    _, P, seen = attention(q, K, V, [18, 19], 3, 2)
    assert seen[0].nonzero().flatten().tolist() == [0, 1, 16, 17, 18]
    assert seen[1].nonzero().flatten().tolist() == [0, 1, 17, 18, 19]
    assert torch.allclose(P.sum(-1), torch.ones(2, 1, dtype=torch.float64))
