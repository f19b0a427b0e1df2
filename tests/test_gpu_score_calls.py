"""Calls of attend and prompt that are refused, captured, made on other streams or side by side."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled

pytestmark = pytest.mark.gpu
BUSY = 200_000_000   # cycles, about a tenth of a second


class Pair:
    """Three sequences, their newest tokens as queries of an attend and of a prompt call."""

    def __init__(self, bits=4, lens=(300, 90, 171), chunks=(40, 9, 171), seed=0, **kw):
        self.f = f = Filled(lens, H=2, bits=bits, residual=32, seed=seed, **kw)
        self.lens, self.chunks = list(lens), list(chunks)
        self.q = inp.queries(seed + 1, sum(chunks), 8, 128, f.dtype).to(f.dev).view(-1, 8, 128)
        self.q1 = inp.queries(seed + 2, 3 * 2, 8, 128, f.dtype).to(f.dev).view(3, 2, 8, 128)
        cu = [0]
        for m in chunks:
            cu.append(cu[-1] + m)
        self.cu = f.i32(cu)
        slopes = torch.linspace(0.01, 0.2, 8, device=f.dev)
        self.scores = s4.Scores(20.0, slopes, 150, 3)

    def prompt(self, **kw):
        f = self.f
        args = dict(bt=f.bt, seq=f.seq, cu=self.cu, longest=max(self.lens), total=sum(self.lens), q=self.q)
        args.update({k: kw.pop(k) for k in list(kw) if k in args})
        return f.cache.prompt(0, args["q"], args["cu"], args["bt"], args["seq"], args["longest"], args["total"], self.scores, **kw)

    def attend(self, **kw):
        f = self.f
        args = dict(bt=f.bt, seq=f.seq, longest=max(self.lens), q=self.q1)
        args.update({k: kw.pop(k) for k in list(kw) if k in args})
        return f.cache.attend(0, args["q"], args["bt"], args["seq"], args["longest"], self.scores, **kw)

    def status(self):
        return self.f.cache.status()


@pytest.mark.parametrize("bits", [4, 8, INT8])
@pytest.mark.parametrize("which", ["prompt", "attend"])
def test_one_bad_sequence_beside_good_ones(bits, which):
    p = Pair(bits, slots=[2, 0, 5])
    f = p.f
    call = getattr(p, which)
    slots = dict(slot_ids=f.slots)
    good = call(**slots)
    f.ok()
    rows = slice(40, 49) if which == "prompt" else slice(1, 2)
    keep = [i for i in range(good.shape[0]) if not rows.start <= i < rows.stop]
    for change, detail in ((dict(seq=f.i32([300, 91, 171])), s4.S4KV_DEV_BAD_LENGTH),
                           (dict(slot_ids=f.i32([2, 6, 5])), s4.S4KV_DEV_BAD_SLOT),
                           (dict(slot_ids=f.i32([2, -1, 5])), s4.S4KV_DEV_BAD_SLOT)):
        got = call(**{**slots, **change})
        assert p.status() == (s4.S4KV_ERR_DEVICE, detail)
        assert torch.equal(got[keep], good[keep]) and not got[rows].any()
    # pages outside the pool: reported, the other sequences as they were
    for bad in (-1, 10 ** 6):
        bt = f.bt.clone()
        bt[1, 1:] = bad
        got = call(**slots, bt=bt)
        assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)
        assert torch.equal(got[keep], good[keep])
    # a table too narrow for one of them
    got = call(**slots, bt=f.bt[:, :12].contiguous())
    assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_TABLE)
    rows = slice(0, 40) if which == "prompt" else slice(0, 1)
    assert not got[rows].any() and torch.equal(got[rows.stop:], good[rows.stop:])
    # a sequence longer than said
    got = call(**slots, longest=299)
    assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    assert not got[rows].any() and torch.equal(got[rows.stop:], good[rows.stop:])
    assert torch.equal(call(**slots), good)
    f.ok()


def test_prompts_with_wrong_sums_and_offsets():
    p = Pair()
    good = p.prompt()
    # fewer tokens in all than there are: the last sequences find no room
    got = p.prompt(total=0)   # (three tiles for 300 + 90 + 171 tokens' six)
    assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    for rows in (slice(0, 40), slice(40, 49), slice(49, 220)):
        assert torch.equal(got[rows], good[rows]) or not got[rows].any()
    out = torch.full_like(good, 7.0)
    for cu in ([0, 40, 30, 220], [1, 40, 49, 220], [0, 40, 49, 219], [0, 40, 300, 220], [0, -5, 49, 220]):
        p.prompt(cu=p.f.i32(cu), out=out)
        assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_CU), cu
        assert bool((out == 7.0).all())
    # a chunk longer than its sequence
    long = torch.cat([p.q, p.q])[:120 + 60]
    got = p.prompt(q=long, cu=p.f.i32([0, 40, 140, 180]))
    assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    assert torch.equal(got[:40], good[:40]) and not got[40:140].any() and got[140:].any()


def test_sequences_without_a_chunk_are_not_looked_at():
    p = Pair(chunks=(40, 0, 171))
    good = p.prompt()
    p.f.ok()
    bt = p.f.bt.clone()
    bt[1] = -3
    got = p.prompt(bt=bt, seq=p.f.i32([300, -7, 171]), slot_ids=p.f.i32([0, 99, 2]))
    assert torch.equal(got, good)
    p.f.ok()
    none = p.prompt(q=p.q[:0], cu=p.f.i32([0, 0, 0, 0]))
    assert none.shape == (0, 8, 128)
    p.f.ok()


@pytest.mark.parametrize("which", ["prompt", "attend"])
def test_inputs_written_right_before(which):
    """Queries, offsets, lengths, first tokens and prefixes that the work queued just before has still to write, other
    ones call by call: the launches that start early read none of them too soon."""
    p = Pair(chunks=(40, 9, 171))
    call = getattr(p, which)
    n = (220,) if which == "prompt" else (3, 2)
    q0 = p.q if which == "prompt" else p.q1
    g = torch.Generator().manual_seed(3)
    sets = []
    for i in range(4):
        first = torch.randint(0, 60, n, generator=g, dtype=torch.int32).cuda()
        m = torch.tensor([0, 10 + 20 * i, 30 + 20 * i, 220], dtype=torch.int32).cuda()
        sets.append(dict(q=(q0 * (0.5 + 0.25 * i)).contiguous(), first=first, prefix=p.f.i32([5 * i, 40, 3]), cu=m))
    if which == "attend":
        for s in sets:
            s.pop("cu")
    else:   # (the last chunk is longer than its sequence: reported, zeros)
        for s in sets:
            s["cu"] = p.f.i32([0, 40, 49, 220]) if s["cu"][3] - s["cu"][2] > 171 else s["cu"]
    want = [call(**s).clone() for s in sets]
    p.status()
    held = {k: torch.zeros_like(v) for k, v in sets[0].items()}
    torch.cuda.synchronize()
    got = []
    for turn in range(3):
        for s in sets:
            torch.cuda._sleep(300_000)
            for k, v in s.items():
                held[k].copy_(v)
            got.append(call(**held))
    torch.cuda.synchronize()
    p.status()
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 4]), i


def test_bounds_of_zero():
    """A call that says that no sequence has a token: the offsets are still looked at, the sequences reported."""
    p = Pair()
    got = p.prompt(longest=0, total=0)
    assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH) and not got.any()
    p.prompt(longest=0, total=0, cu=p.f.i32([0, 50, 40, 220]))
    assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_CU)
    got = p.attend(longest=0)
    assert p.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH) and not got.any()


def test_calls_of_no_sequences():
    p = Pair()
    c, none, no_rows = p.f.cache, p.f.i32([]), p.f.bt[:0]
    assert c.prompt(0, p.q[:0], p.f.i32([0]), no_rows, none, 0, 0).shape == (0, 8, 128)
    assert c.attend(0, p.q1[:0], no_rows, none, 0, p.scores).shape == (0, 2, 8, 128)
    refs = torch.zeros(c.cfg.num_pages, dtype=torch.int32, device="cuda")
    assert c.take_pages(refs, no_rows, none, none).shape == (0,)
    assert c.fork(refs, p.f.bt[:1].contiguous(), none, none, none).shape == (0,)
    c.release_pages(refs, no_rows, none, none)
    assert not refs.any()
    p.f.ok()


@pytest.mark.parametrize("which", ["prompt", "attend"])
def test_ends_of_the_integers(which):
    """first and prefix at both ends of their type: everything, nothing, and as without them."""
    p = Pair()
    call = getattr(p, which)
    n = (220,) if which == "prompt" else (3, 2)
    fill = lambda shape, x: torch.full(shape, x, dtype=torch.int32, device="cuda")  # noqa: E731
    least, most = -2 ** 31, 2 ** 31 - 1
    p.scores = s4.Scores(20.0)
    good, whole = call(), call(prefix=p.f.seq)
    assert torch.equal(call(first=fill(n, least)), good)
    assert torch.equal(call(prefix=fill((3,), least)), good)
    assert torch.equal(call(prefix=fill((3,), most)), whole) and not torch.equal(good, whole)
    assert not call(first=fill(n, most)).any()
    p.f.ok()


@pytest.mark.parametrize("which", ["prompt", "attend"])
def test_waits_that_run_out(which):
    p = Pair()
    call = getattr(p, which)
    good = call()
    p.f.cache.set_option(s4.S4KV_OPT_WAIT_NS, 0)   # the first wait gives up
    got = call()
    assert p.status() == (s4.S4KV_ERR_DEVICE_TIMEOUT, s4.S4KV_DEV_TIMEOUT)
    assert torch.isfinite(got).all()
    p.f.cache.set_option(s4.S4KV_OPT_WAIT_NS, 1000000000)
    assert torch.equal(call(), good)
    p.f.ok()


def test_refused_on_the_host():
    p = Pair()
    f, c = p.f, p.f.cache
    for bad in (dict(q=p.q.float()), dict(q=p.q[:, :, :64].contiguous()), dict(q=p.q[:, ::2]), dict(cu=f.i32([0, 220])),
                dict(cu=p.cu.long()), dict(bt=f.bt[:2].contiguous()), dict(first=f.i32([0] * 3)), dict(prefix=f.i32([0] * 4)),
                dict(out=torch.empty(220, 8, 128, dtype=torch.float64, device="cuda")), dict(out_dtype=9), dict(q=p.q.cpu())):
        with pytest.raises(ValueError):
            p.prompt(**bad)
    for bad in (dict(q=p.q1.float()), dict(first=f.i32([[0], [0], [0]])), dict(prefix=f.i32([1, 2])), dict(bt=f.bt[:2].contiguous())):
        with pytest.raises(ValueError):
            p.attend(**bad)
    wrong = s4.Scores(slopes=torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        c.prompt(0, p.q, p.cu, f.bt, f.seq, 300, 600, wrong)
    for code, call in ((s4.S4KV_ERR_INVALID_ARG, lambda: c.prompt(1, p.q, p.cu, f.bt, f.seq, 300, 600)),
                       (s4.S4KV_ERR_INVALID_ARG, lambda: c.prompt(0, p.q, p.cu, f.bt, f.seq, -1, 600)),
                       (s4.S4KV_ERR_INVALID_ARG, lambda: c.prompt(0, p.q, p.cu, f.bt, f.seq, 300, -1)),
                       (s4.S4KV_ERR_INVALID_ARG, lambda: c.prompt(0, p.q[:, :3].contiguous(), p.cu, f.bt, f.seq, 300, 600)),
                       (s4.S4KV_ERR_UNSUPPORTED, lambda: c.prompt(0, torch.cat([p.q, p.q, p.q], 1), p.cu, f.bt, f.seq, 300, 600)),
                       (s4.S4KV_ERR_UNSUPPORTED, lambda: c.attend(0, p.q1.repeat(1, 8, 2, 1), f.bt, f.seq, 300, s4.Scores())),
                       (s4.S4KV_ERR_INVALID_ARG, lambda: p.attend(q=p.q1.repeat(1, 9, 1, 1)))):
        with pytest.raises(s4.S4KVError) as e:
            call()
        assert e.value.code == code
    form = s4.s4kv_scores(20.0, None, 0, 0, None, None)
    nb = s4.s4kv_prompt_workspace_bytes(c.h, 3, 220, 8, 300, 561)
    ws, out = torch.empty(nb + 16, dtype=torch.uint8, device="cuda"), torch.empty(220, 8, 128, device="cuda")

    def raw(form=form, q=p.q.data_ptr(), ws=ws.data_ptr(), nb=nb, out=out.data_ptr(), dt=s4.S4KV_F32, cu=p.cu.data_ptr(), n=3):
        s4.s4kv_prompt_attention(c.h, 0, form, q, 220, cu, 8, f.bt, f.bt.shape[1], f.seq, None, n, 0.0, out, dt, ws, nb, 300, 561)
    raw()
    for code, kw in ((s4.S4KV_ERR_WORKSPACE_TOO_SMALL, dict(nb=nb - 1)), (s4.S4KV_ERR_INVALID_ARG, dict(ws=ws.data_ptr() + 8)),
                     (s4.S4KV_ERR_INVALID_ARG, dict(q=p.q.data_ptr() + 2)), (s4.S4KV_ERR_INVALID_ARG, dict(out=0)),
                     (s4.S4KV_ERR_INVALID_ARG, dict(cu=0)), (s4.S4KV_ERR_INVALID_ARG, dict(dt=s4.S4KV_F16)),
                     (s4.S4KV_ERR_INVALID_ARG, dict(n=4097)), (s4.S4KV_ERR_INVALID_ARG, dict(n=0)),
                     (s4.S4KV_ERR_INVALID_ARG, dict(form=s4.s4kv_scores(-1.0, None, 0, 0, None, None))),
                     (s4.S4KV_ERR_INVALID_ARG, dict(form=s4.s4kv_scores(float("nan"), None, 0, 0, None, None))),
                     (s4.S4KV_ERR_INVALID_ARG, dict(form=s4.s4kv_scores(1e-30, None, 0, 0, None, None))),
                     (s4.S4KV_ERR_INVALID_ARG, dict(form=s4.s4kv_scores(0.0, None, -1, 0, None, None)))):
        with pytest.raises(s4.S4KVError) as e:
            raw(**kw)
        assert e.value.code == code, kw
    raw(form=None)   # no form: plain causal attention
    f.ok()


@pytest.mark.parametrize("bits", [4, INT8])
@pytest.mark.parametrize("which", ["prompt", "attend"])
@pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])
def test_results_on_another_stream(bits, which, handle):
    a, b = Pair(bits, seed=3), Pair(bits, seed=4)
    b.f, b.scores = a.f, a.scores   # the same cache, other queries
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    one, two = getattr(a, which), getattr(b, which)
    one(stream=stream)
    want, other = one().clone(), two().clone()
    torch.cuda.synchronize()
    block = torch.empty_like(want)
    torch.cuda._sleep(BUSY)
    block.fill_(7.0)
    del block
    got = one(stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda._sleep(BUSY)
    kept = got.clone()
    del got
    again = two(stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(kept, want) and torch.equal(again, other)
    a.f.ok()


@pytest.mark.parametrize("bits", [4, 8, INT8])
def test_two_prompts_at_once_and_replayed(bits):
    a, b = Pair(bits, seed=5), Pair(bits, seed=6, lens=(2000, 33, 700), chunks=(3, 33, 90))
    wa, wb, wc = a.prompt().clone(), b.prompt().clone(), b.attend().clone()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append((a.prompt(stream=s1), b.prompt(stream=s2), b.attend(stream=s1)))
    torch.cuda.synchronize()
    for x, y, z in got:
        assert torch.equal(x, wa) and torch.equal(y, wb) and torch.equal(z, wc)
    # two graphs of their own, replayed in turn with other queries, lengths unchanged
    graphs = []
    for p in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = (p.prompt(), p.attend())
        graphs.append((g, out, p))
    for k in range(3):
        for g, out, p in graphs:
            p.q.copy_(inp.queries(50 + k, p.q.shape[0], 8, 128, p.f.dtype).view_as(p.q))
            g.replay()
        for g, out, p in graphs:
            assert torch.equal(out[0], p.prompt()) and torch.equal(out[1], p.attend())
    a.f.ok(), b.f.ok()


def test_a_prompt_is_its_chunks():
    # a prompt appended and attended chunk by chunk sees what the model says: the same keys once restored
    # (8-bit pages of whole blocks do not change as later tokens come)
    p = Pair(8, lens=(256, 256, 256), chunks=(256, 256, 256))
    whole = p.prompt()
    f = p.f
    g = s4.KVCache(1, f.cache.cfg.num_pages, 2, 32, 3, "bf16", bits=8)
    at = [0, 0, 0]
    for n in (100, 16, 1, 139):
        to = [x + n for x in at]
        k, v = (torch.cat([x[a:t] for x, a, t in zip(y, at, to)]) for y in (f.k, f.v))
        g.append(0, k, v, f.i32([0, n, 2 * n, 3 * n]), f.i32(at), f.bt)
        q = torch.cat([p.q[256 * b + at[b]:256 * b + to[b]] for b in range(3)])
        got = g.prompt(0, q, f.i32([0, n, 2 * n, 3 * n]), f.bt, f.i32(to), max(to), sum(to), p.scores)
        want = torch.cat([whole[256 * b + at[b]:256 * b + to[b]] for b in range(3)])
        assert (got - want).abs().max() < 1e-2
        at = to
    f.ok()


def test_attend_and_prompt_agree():
    for bits in (4, 2, 8, INT8):
        p = Pair(bits, lens=(700, 64, 171), chunks=(2, 2, 2))
        p.q1 = p.q.view(3, 2, 8, 128)
        a, b = p.attend(), p.prompt().view(3, 2, 8, 128)
        assert (a - b).abs().max() < 2e-2
        p.f.ok()
