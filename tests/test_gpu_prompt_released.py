"""Prompts behind a window whose pages before it have been given back."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from plain_cache import INT8
from test_gpu_prompt import Call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,sinks", [(100, 4), (33, 0), (200, 40), (128, 130), (1, 1)])
@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (2, "fp16"), (8, "bf16"), (INT8, "fp16")])
def test_prompts_behind_a_window(bits, dtype, window, sinks):
    lens, chunks = [900, 517, 333, 1300], [40, 300, 1, 129]
    c = Call(lens, chunks, bits=bits, dtype=dtype, residual=20, window=window, sinks=sinks, seed=51)
    f = c.f
    want = c.run()
    c.check(want)
    block = 16 if bits in (8, INT8) else 32
    first = [-(-sinks // block) * block] * len(lens)
    last = [max(0, min(n - m - window + 1, n - 20)) // block * block for n, m in zip(lens, chunks)]
    refs = torch.zeros(f.cache.cfg.num_pages, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):
        refs[f.bt[b, :-(-n // 16)].long()] = 1
    held = int(refs.sum())
    f.cache.release_pages(refs, f.bt, f.i32(first), f.i32(last))
    f.ok()
    assert held - int(refs.sum()) == sum(max(0, y - x) // 16 for x, y in zip(first, last)) > 0
    got = c.run()
    f.ok()
    assert torch.equal(got, want)
    # the page of the first token that the chunk does see: reported
    f.bt[0, (lens[0] - chunks[0] - window + 1) // 16] = -1
    c.run()
    assert f.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)


@pytest.mark.parametrize("bits", [4, 8, INT8])
def test_a_window_narrower_than_the_residual(bits):
    """Pages go back as the header says, never ahead of what is still to be written to them; the sequence then grows
    through them, chunk by chunk, as one that keeps its pages."""
    H, R, W, block = 2, 128, 40, 16 if bits in (8, INT8) else 32
    kept, given = (s4.KVCache(1, 64, H, R, 1, "bf16", bits=bits) for _ in range(2))
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    g = torch.Generator().manual_seed(5)
    table = torch.full((1, 64), -1, dtype=torch.int32, device="cuda")
    whole, refs = torch.arange(64, dtype=torch.int32, device="cuda")[None], torch.zeros(64, dtype=torch.int32, device="cuda")
    scores, T, most = s4.Scores(window=W), 0, 0
    for m in (200, 3, 61, 1, 90, 130, 17, 250):
        k, v = (torch.randn(m, H, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
        q = torch.randn(m, 8, 128, generator=g).to(torch.bfloat16).cuda()
        assert given.take_pages(refs, table, i32([T]), i32([T + m])).tolist() == [-(-(T + m) // 16) - -(-T // 16)]
        for c, bt in ((kept, whole), (given, table)):
            c.append(0, k, v, i32([0, m]), i32([T]), bt)
        T += m
        a, b = (c.prompt(0, q, i32([0, m]), bt, i32([T]), T, T, scores) for c, bt in ((kept, whole), (given, table)))
        assert torch.equal(a, b)
        a, b = (c.attend(0, q[-1:, None].reshape(1, 1, 8, 128), bt, i32([T]), T, scores) for c, bt in ((kept, whole), (given, table)))
        assert torch.equal(a, b)
        assert kept.status()[0] == 0 and given.status()[0] == 0
        # the next query sees T + 1 - W and later; KIVI pages: and what has left the rings
        done = T + 1 - W if bits in (8, INT8) else min(T + 1 - W, T // 32 * 32, T - R)
        given.release_pages(refs, table, i32([0]), i32([max(0, done) // block * block]))
        most = max(most, int(refs.sum()))
    assert most < 16 and given.status()[0] == 0
