"""Attention within a sliding window with sinks, on every page format."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled, check, restored

pytestmark = pytest.mark.gpu
FORMATS = [4, 2, 8, INT8]


def _queries(seed, B, nq, Hq, dtype):
    return torch.randn(B, nq, Hq, 128, generator=inp.gen(seed), dtype=torch.float32).to(dtype).cuda()


def _scales(bits, H):
    return ([0.5 + 0.25 * h for h in range(H)], [1.5 - 0.25 * h for h in range(H)]) if bits == 8 else None


@pytest.fixture(params=[1, 2], ids=["slices", "clusters"], autouse=True)
def form(request, monkeypatch):
    """Every test runs on both launch forms."""
    make = s4.KVCache.__init__

    def init(self, *a, **kw):
        make(self, *a, **kw)
        self.set_option(s4.S4KV_OPT_WINDOW_FORM, request.param)
    monkeypatch.setattr(s4.KVCache, "__init__", init)
    return request.param


def _all(f, q, window, sinks, what="", **kw):
    B, nq = q.shape[:2]
    out = f.cache.window(0, q, f.bt, f.seq, max(f.lens), window, sinks, slot_ids=f.slots, **kw)
    f.ok()
    worst = 0.0
    for b, n in enumerate(f.lens):
        if n == 0:
            assert not out[b].any()
        else:
            worst = max(worst, check(out[b], q[b], *f.plain(b), range(n - nq, n), f.bits, window, sinks,
                                     f"{what} seq {b} of {n}, window {window}, sinks {sinks}"))
    return out, worst


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,g", [(2, 4), (1, 7)])
def test_single_token(bits, dtype, H, g):
    lens = [1, 2, 0, 16, 31, 33, 64, 100, 257, 700, 1111]
    f = Filled(lens, H=H, bits=bits, dtype=dtype, residual=32, seed=3, slots=list(range(len(lens)))[::-1],
               fp8_scales=_scales(bits, H))
    q = _queries(1, len(lens), 1, H * g, f.dtype)
    for window, sinks in ((1, 0), (1, 4), (16, 0), (17, 3), (32, 1), (33, 33), (100, 16), (256, 5), (5000, 0), (40, 300),
                          (64, 2 ** 31 - 1), (2 ** 31 - 1, 4)):
        _all(f, q, window, sinks)
    _all(f, q, 100, 4, out_dtype=f.cache.cdtype)


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("nq,H,g", [(2, 2, 1), (3, 1, 3), (5, 2, 4), (16, 1, 6), (16, 2, 2)])
def test_several_tokens(bits, nq, H, g):
    lens = [nq, nq + 1, 40, 65, 128, 333, 900]
    lens = [max(nq, n) for n in lens]
    f = Filled(lens, H=H, bits=bits, residual=33, seed=7 + nq, fp8_scales=_scales(bits, H), chunks=[50, 13])
    q = _queries(2, len(lens), nq, H * g, f.dtype)
    for window, sinks in ((1, 0), (2, 1), (15, 0), (32, 4), (47, 18), (128, 0), (1000, 3), (30, 64)):
        _all(f, q, window, sinks)


@pytest.mark.parametrize("bits", [4, 2])
@pytest.mark.parametrize("residual", [1, 16, 128, 200, 1024])
def test_kivi_residual_lengths(bits, residual):
    """The window's start inside the residual, at its border and in the pages."""
    lens = [30, 96, 160, 420]
    f = Filled(lens, H=2, bits=bits, residual=residual, seed=residual)
    q = _queries(3, len(lens), 1, 8, f.dtype)
    for window, sinks in ((5, 2), (31, 40), (127, 4), (129, 0), (210, 33), (400, 1)):
        _all(f, q, window, sinks)


@pytest.mark.parametrize("bits", FORMATS)
def test_a_window_wider_than_the_sequence_is_full_attention(bits):
    lens = [77, 500, 1024]
    f = Filled(lens, H=2, bits=bits, residual=64, seed=4)
    q = _queries(4, 3, 1, 8, f.dtype)
    out, _ = _all(f, q, 1024, 0)
    full = f.cache.decode(0, q[:, 0].contiguous(), f.bt, f.seq, 1024)
    if bits == INT8:
        assert torch.equal(out[:, 0], full)
    else:
        assert float((out[:, 0] - full).abs().max()) < 2e-3


@pytest.mark.parametrize("bits", FORMATS)
def test_pages_outside_the_window_are_not_needed(bits):
    """Table entries between the sinks' and the window's blocks hold -1; their pages hold NaN patterns."""
    lens = [900, 640]
    f = Filled(lens, H=2, bits=bits, residual=32, seed=9)
    nq, window, sinks = 2, 100, 20
    q = _queries(5, 2, nq, 8, f.dtype)
    want, _ = _all(f, q, window, sinks)
    bt, block = f.bt.clone(), 2 if bits in (4, 2) else 1
    lay = f.cache.layout
    pages = f.cache.pool[lay.layer_offset:lay.layer_offset + f.cache.cfg.num_pages * lay.page_stride].view(f.cache.cfg.num_pages, -1)
    for b, n in enumerate(lens):
        lo = -(-sinks // 16)
        lo = -(-lo // block) * block
        hi = (n - nq - window + 1) // (16 * block) * block
        assert hi > lo + 4
        for p in range(lo, hi):
            pages[int(f.bt[b, p])] = 0xFF
        bt[b, lo:hi] = -1
    got = f.cache.window(0, q, bt, f.seq, max(lens), window, sinks)
    f.ok()
    assert torch.equal(got, want)
    bt[0, (lens[0] - 1) // 16 - 3] = -1      # a page that is needed: reported
    f.cache.window(0, q, bt, f.seq, max(lens), window, sinks)
    assert f.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), float("-inf")])
@pytest.mark.parametrize("Hq", [2, 8])
def test_masked_tokens_may_hold_anything(bits, dtype, bad, Hq):
    """Keys and values that are not finite, at tokens that no query, or only the later queries, see.

    KIVI pages: in the full-precision rows (a group's own scale belongs to all its tokens). INT8: in the
    unfinished block. FP8: any token (infinities saturate when stored; a NaN stays one)."""
    n, nq, window = 300, 4, 9
    late = 2                                    # the token of query nq - late is bad: queries before it are not

    def edit(b, k, v):
        for t in ([n - late] if b == 0 else [n - nq - window + 1, n - nq - window + 2]):   # seen by query 0 (and 1) only
            k[t] = bad
            v[t, :, 3:7] = bad
    f = Filled([n, n], H=2, bits=bits, dtype=dtype, residual=64, seed=2, edit=edit)
    q = _queries(6, 2, nq, Hq, f.dtype)
    out = f.cache.window(0, q, f.bt, f.seq, n, window, 0)
    f.ok()
    for b, clean in ((0, range(0, nq - late)), (1, range(2, nq))):
        for i in clean:
            K, V, mk, mv = f.plain(b)
            if bits == 8:
                K, V = K.clone(), V.clone()
            check(out[b, i:i + 1], q[b, i:i + 1], K, V, mk, mv, [n - nq + i], bits, window, 0, f"seq {b} query {i}")
    if bits != 8:
        assert not torch.isfinite(out[0, nq - 1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("nq,Hq", [(1, 2), (3, 8)])
def test_int8_extremes_beside_the_window(dtype, nq, Hq):
    """A token that no query sees holds the type's lowest and largest value and sets the scale of a block that
    is seen in part: the block's other tokens are restored as zeros, and count as exact zeros."""
    n, window, sinks = 300 + nq, 100, 5
    t = torch.bfloat16 if dtype == "bf16" else torch.float16

    def edit(b, k, v):
        for x in (195, 9):    # in the blocks that the window's start and the last sink cut
            k[x], v[x] = torch.finfo(t).min, torch.finfo(t).min
            k[x, :, ::2], v[x, :, 1::2] = torch.finfo(t).max, torch.finfo(t).max
    f = Filled([n], H=2, bits="int8", dtype=dtype, seed=4, edit=edit)
    q = _queries(9, 1, nq, Hq, f.dtype)
    out = f.cache.window(0, q, f.bt, f.seq, n, window, sinks)
    f.ok()
    K, V, mk, mv = f.plain(0)
    for x in (195, 9):
        K[x] = V[x] = 0
    assert not K[192:208].any() and not V[:16].any()
    check(out[0], q[0], K, V, mk, mv, range(n - nq, n), "int8", window, sinks)


def test_int8_values_of_any_size():
    """Values near the type's largest and smallest scales, all seen."""
    big = 2.0 ** 120

    def edit(b, k, v):
        v *= big if b == 0 else 2.0 ** -98
    f = Filled([70, 70], H=2, bits="int8", dtype="bf16", seed=4, edit=edit)
    assert f.v[0].float().abs().max() > 2.0 ** 121 and torch.isfinite(f.v[0].float()).all()
    q = _queries(9, 2, 1, 4, f.dtype)
    for window in (1000, 50):
        out = f.cache.window(0, q, f.bt, f.seq, 70, window, 0)
        f.ok()
        for b in range(2):
            up = 2.0 ** -120 if b == 0 else 2.0 ** 98    # (the bound's smallest terms are made for values near 1)
            K, V, mk, mv = f.plain(b)
            check(out[b] * up, q[b], K, V * up, mk, mv, [69], "int8", window, 0, f"seq {b}")


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("nq,H,g", [(1, 1, 96), (1, 2, 17), (8, 1, 12), (3, 2, 32), (16, 1, 5)])
def test_many_heads_per_kv_head(bits, nq, H, g):
    f = Filled([nq, 200, 333], H=H, bits=bits, residual=64, seed=g)
    q = _queries(7, 3, nq, H * g, f.dtype)
    _all(f, q, 90, 7)
    _all(f, q, 4000, 0)


@pytest.mark.parametrize("bits", FORMATS)
def test_scale_layers_and_a_slot_asked_for_twice(bits):
    f = Filled([150, 90], H=2, bits=bits, residual=32, seed=5)
    two = s4.KVCache(3, f.cache.cfg.num_pages, 2, 32, 2, "bf16", bits=bits)
    k, v = torch.cat(f.k), torch.cat(f.v)
    two.append(2, k, v, f.i32([0, 150, 240]), f.i32([0, 0]), f.bt)
    q = _queries(8, 2, 2, 8, f.dtype)
    want = f.cache.window(0, q, f.bt, f.seq, 150, 70, 3)
    assert torch.equal(two.window(2, q, f.bt, f.seq, 150, 70, 3), want)
    assert two.status() == (0, 0)
    two.window(1, q, f.bt, f.seq, 150, 70, 3)            # nothing was appended to layer 1
    assert two.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    bt2, q2 = torch.cat([f.bt[:1], f.bt[:1]]), torch.cat([q[:1], q[:1]])
    twice = f.cache.window(0, q2, bt2, f.i32([150, 150]), 150, 70, 3, slot_ids=f.i32([0, 0]))
    f.ok()
    for i in range(2):   # (another batch is cut into other slices: not the same bits)
        check(twice[i], q[0], *f.plain(0), range(148, 150), bits, 70, 3)
    # a softmax scale of its own: that of queries scaled by it
    out = f.cache.window(0, q, f.bt, f.seq, 150, 70, 3, sm_scale=2.0 / 128 ** 0.5)
    for b, n in enumerate(f.lens):
        check(out[b], q[b] * 2, *f.plain(b), range(n - 2, n), bits, 70, 3)


def test_lengths_slots_and_tables_are_checked():
    f = Filled([100, 50, 0], H=2, bits=4, residual=32, seed=1)
    q = _queries(1, 3, 3, 4, f.dtype)
    good = f.cache.window(0, q, f.bt, f.seq, 100, 20, 2)
    f.ok()
    assert not good[2].any()

    def bad(detail, bt=f.bt, seq=f.seq, top=100, slots=None):
        out = f.cache.window(0, q, bt, seq, top, 20, 2, slot_ids=slots)
        assert f.cache.status() == (s4.S4KV_ERR_DEVICE, detail)
        return out
    out = bad(s4.S4KV_DEV_BAD_LENGTH, seq=f.i32([100, 49, 0]))
    assert not out[1].any() and torch.equal(out[0], good[0])
    bad(s4.S4KV_DEV_BAD_LENGTH, top=99)
    bad(s4.S4KV_DEV_BAD_LENGTH, seq=f.i32([-5, 50, 0]))
    for top in (2 ** 31 - 1, 2 ** 31 - 20, -2 ** 31):     # beside a good sequence, which keeps its rows
        out = bad(s4.S4KV_DEV_BAD_LENGTH, seq=f.i32([100, top, 0]))
        assert not out[1].any() and torch.equal(out[0], good[0])
    bad(s4.S4KV_DEV_BAD_SLOT, slots=f.i32([0, 3, 2]))
    bad(s4.S4KV_DEV_BAD_TABLE, bt=f.bt[:, :5].contiguous())
    # shorter than the chunk of queries
    g = Filled([2, 50], H=2, bits=4, residual=32, seed=1)
    out = g.cache.window(0, q[:2].contiguous(), g.bt, g.seq, 50, 20)
    assert g.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH) and not out[0].any()


def test_argument_errors_launch_nothing():
    f = Filled([100], H=2, bits=4, residual=8, seed=1)
    q = _queries(1, 1, 1, 4, f.dtype)
    out = torch.full((1, 1, 4, 128), 5.0, device="cuda")
    nb = s4.s4kv_window_workspace_bytes(f.cache.h, 1, 1, 4, 100)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")

    def code(want, **kw):
        a = dict(h=f.cache.h, layer=0, q=q, num_q_tokens=1, num_q_heads=4, window=10, num_sinks=0, block_table=f.bt,
                 bt_stride=f.bt.shape[1], seq_lens=f.seq, slot_ids=None, B=1, sm_scale=0.0, out=out,
                 out_dtype=s4.S4KV_F32, workspace=ws, ws_bytes=nb, max_seq_len=100)
        a.update(kw)
        with pytest.raises(s4.S4KVError) as e:
            s4.s4kv_window_attention(**a)
        assert e.value.code == want, kw
    bad, uns = s4.S4KV_ERR_INVALID_ARG, s4.S4KV_ERR_UNSUPPORTED
    for kw in (dict(window=0), dict(window=-1), dict(num_sinks=-1), dict(layer=1), dict(q=None), dict(out=None),
               dict(block_table=None), dict(seq_lens=None), dict(q=q.data_ptr() + 2), dict(out=out.data_ptr() + 4),
               dict(num_q_heads=5), dict(num_q_tokens=0), dict(num_q_tokens=17), dict(out_dtype=s4.S4KV_F16),
               dict(bt_stride=0), dict(B=-1), dict(B=4097), dict(workspace=None), dict(max_seq_len=-1)):
        code(bad, **kw)
    for kw in (dict(num_q_tokens=9), dict(num_q_tokens=8, num_q_heads=26)):   # past R = 8; 104 columns
        code(uns, **kw)
    code(s4.S4KV_ERR_WORKSPACE_TOO_SMALL, ws_bytes=nb - 1)
    torch.cuda.synchronize()
    assert bool((out == 5.0).all())
    for kw in (dict(q=q.float()), dict(q=torch.cat([q, q], -1)[..., :128]), dict(q=q.cpu()), dict(seq_lens=f.seq.long()),
               dict(block_table=f.bt[:0]), dict(out=out[..., :64]), dict(out_dtype=s4.S4KV_F16)):
        a = dict(layer=0, q=q, block_table=f.bt, seq_lens=f.seq, max_seq_len=100, window=10)
        a.update(kw)
        with pytest.raises(ValueError):
            f.cache.window(**a)


@pytest.mark.parametrize("bits", FORMATS)
def test_bounded_wait_gives_up_and_the_next_call_is_clean(bits):
    f = Filled([3000, 2500], H=2, bits=bits, residual=32, seed=6)
    q = _queries(2, 2, 1, 8, f.dtype)
    good = f.cache.window(0, q, f.bt, f.seq, 3000, 2000, 3)
    f.cache.set_option(s4.S4KV_OPT_WAIT_NS, 0)
    f.cache.window(0, q, f.bt, f.seq, 3000, 2000, 3)
    assert f.cache.status() == (s4.S4KV_ERR_DEVICE_TIMEOUT, s4.S4KV_DEV_TIMEOUT)
    f.cache.set_option(s4.S4KV_OPT_WAIT_NS, 1_000_000_000)
    assert torch.equal(f.cache.window(0, q, f.bt, f.seq, 3000, 2000, 3), good)
    f.ok()


def test_captured_graphs_and_other_streams_share_nothing():
    """Two captured calls and eager ones on two streams at once give each its own result."""
    f = Filled([2000, 1500], H=2, bits=INT8, seed=6)
    g = Filled([1800, 300], H=2, bits=4, seed=7)
    qf, qg = _queries(2, 2, 1, 8, f.dtype), _queries(3, 2, 1, 8, g.dtype)
    want_f = f.cache.window(0, qf, f.bt, f.seq, 2000, 900, 4)
    want_g = g.cache.window(0, qg, g.bt, g.seq, 1800, 500, 4)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c, q in ((f, qf), (g, qg)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            outs.append(c.cache.window(0, q, c.bt, c.seq, 2000, 900 if c is f else 500, 4))
        graphs.append(gr)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        e1 = f.cache.window(0, qf, f.bt, f.seq, 2000, 900, 4, stream=s1)
        e2 = g.cache.window(0, qg, g.bt, g.seq, 1800, 500, 4, stream=s2.cuda_stream)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], want_f) and torch.equal(outs[1], want_g)
        assert torch.equal(e1, want_f) and torch.equal(e2, want_g)
    f.ok()
    g.ok()


def test_many_sequences_and_a_long_table():
    lens = [(37 * i) % 90 for i in range(400)]
    f = Filled(lens, H=1, bits=INT8, seed=12)
    q = _queries(2, 400, 1, 2, f.dtype)
    out = f.cache.window(0, q, f.bt, f.seq, 90, 33, 2)
    f.ok()
    for b in range(0, 400, 23):
        if lens[b]:
            check(out[b], q[b], *restored(f.k[b], f.v[b], INT8, 32), [lens[b] - 1], INT8, 33, 2)
        else:
            assert not out[b].any()
