"""Calls on a stream of their own while the current stream is busy: their results are neither written
over by work that was queued before nor handed on while they are still read."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled

pytestmark = pytest.mark.gpu
CALLS = ["decode", "multi_query", "window", "gather", "append_rope", "dequant"]
BUSY = 200_000_000   # cycles, about a tenth of a second


def _call(f, which, seed):
    """A call of `which` that only the queries or token rows of `seed` change: stream -> tuple of results."""
    g = inp.gen(seed)
    q = torch.randn(2, 2, 8, 128, generator=g).to(f.dtype).cuda()
    one = q[:, 0].contiguous()
    k, v = (x.cuda() for x in inp.kv_rows(seed, 40, 2, 128, f.dtype))
    qn = torch.randn(40, 8, 128, generator=g).to(f.dtype).cuda()
    at = torch.arange(64, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    rope = s4.Rope(torch.cat([at.cos(), at.sin()], 1).float().cuda())
    cu, zero, rows = f.i32([0, 40]), f.i32([0]), f.i32([0, 300, 500])
    first, spare = f.i32([seed, 2 * seed]), f.i32([2])
    tail = f.bt[:, :40].contiguous()
    held = (q, one, k, v, qn, rope, cu, zero, rows, first, spare, tail)   # inputs outlive the calls

    def call(stream):
        c, _ = f.cache, held
        if which == "decode":
            return (c.decode(0, one, f.bt, f.seq, 600, stream=stream),)
        if which == "multi_query":
            return (c.multi_query(0, q, f.bt, f.seq, 600, stream=stream),)
        if which == "window":
            return (c.window(0, q, f.bt, f.seq, 600, 200, 3, stream=stream),)
        if which == "gather":
            return c.gather(0, f.bt, f.seq, rows, 500, first=first, stream=stream)
        if which == "append_rope":   # into the slot that no sequence has
            return (c.append_rope(0, k, v, cu, zero, tail[2:], rope, slot_ids=spare, q=qn, stream=stream),)
        return c.dequant(0, 0, f.bt[0], 600, stream=stream)
    return call


@pytest.mark.parametrize("bits", [INT8, 4])
@pytest.mark.parametrize("which", CALLS)
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_results_on_another_stream(bits, which, handle):
    f = Filled([600, 560, 40], H=2, bits=bits, residual=32, seed=3)
    f.seq, f.lens = f.seq[:2].contiguous(), f.lens[:2]
    a, b = _call(f, which, 5), _call(f, which, 6)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    a(stream)                                    # (first use of the stream's memory)
    want, other = a(None), b(None)
    want, other = [x.clone() for x in want], [x.clone() for x in other]
    torch.cuda.synchronize()
    # blocks of the results' sizes, given back while the current stream has still to write them
    blocks = [torch.empty_like(x) for x in want]
    torch.cuda._sleep(BUSY)
    for x in blocks:
        x.fill_(7.0)
    del blocks, x
    got = a(stream)
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    # results dropped while the current stream has still to read them, behind the call on the other
    got = a(stream)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = [x.clone() for x in got]
    del got, x
    again = b(stream)
    torch.cuda.synchronize()
    for x, y in zip(kept, want):
        assert torch.equal(x, y)
    for x, y in zip(again, other):
        assert torch.equal(x, y)
    f.ok()
