"""Appends that rotate the keys (and the queries) on the way: the caches they leave are those of
rows rotated beforehand, byte for byte."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8

pytestmark = pytest.mark.gpu
FORMATS = [4, 2, 8, INT8]


def table(rows, dim, device="cuda"):
    half = dim // 2
    at = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    return torch.cat([at.cos(), at.sin()], 1).float().to(device)


def rotate(x, pos, tab, interleaved):
    """Rows x [n, heads, 128] at pos, in fp32 steps, rounded once."""
    half = tab.shape[1] // 2
    c, s = tab[pos][:, None, :half], tab[pos][:, None, half:]
    y = x.float()
    a, b = (y[..., 0:2 * half:2], y[..., 1:2 * half:2]) if interleaved else (y[..., :half], y[..., half:2 * half])
    u, w = a * c - b * s, b * c + a * s
    z = y.clone()
    if interleaved:
        z[..., 0:2 * half:2], z[..., 1:2 * half:2] = u, w
    else:
        z[..., :half], z[..., half:2 * half] = u, w
    return z.to(x.dtype)


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


class Pair:
    """Two equal caches: one appended to with the rotation, one with rows rotated beforehand."""

    def __init__(self, lens, bits, dtype, residual, H, seed):
        self.lens, self.H, self.seed = lens, H, seed
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        pages = [max(1, -(-n // 16)) for n in lens]
        self.bt = inp.block_tables("permuted", len(lens), pages, sum(pages), seed).cuda()
        self.caches = []
        for _ in range(2):
            c = s4.KVCache(1, sum(pages), H, residual, len(lens), dtype, bits=bits)
            c.pool.zero_()
            if bits == 8:   # a power of two, and not
                c.set_fp8_scales(0, [(0.5, 0.37)[h % 2] for h in range(H)], [(1.3, 2.0)[h % 2] for h in range(H)])
            self.caches.append(c)
        self.at = [0] * len(lens)

    def grow(self, to, rope, tab, interleaved, Hq=0, in_place=False, round_=0):
        new = [t - a for a, t in zip(self.at, to)]
        total = sum(new)
        k, v = inp.kv_rows(inp.mix_seed(self.seed, round_), total, self.H, 128, self.dt)
        k, v = k.cuda(), v.cuda()
        q = torch.randn(total, Hq, 128, generator=inp.gen(round_ + 5)).to(self.dt).cuda() if Hq else None
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        pos = torch.cat([torch.arange(a, t) for a, t in zip(self.at, to)]).cuda()
        want_q = rotate(q, pos, tab, interleaved) if Hq else None
        got = self.caches[0].append_rope(0, k, v, _i32(cu), _i32(self.at), self.bt, rope, q=q, q_out=q if in_place else None)
        self.caches[1].append(0, rotate(k, pos, tab, interleaved), v, _i32(cu), _i32(self.at), self.bt)
        if Hq:
            assert torch.equal(got, want_q)
        self.at = list(to)

    def same(self):
        for c in self.caches:
            assert c.status() == (0, 0)
        assert torch.equal(self.caches[0].pool, self.caches[1].pool)


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("dim,interleaved", [(128, False), (128, True), (64, False), (96, False), (16, False), (32, True), (112, False)])
def test_pages_rings_and_queries_are_those_of_rotated_rows(bits, dtype, dim, interleaved):
    lens = [1, 31, 32, 100, 300, 0, 77]
    tab = table(300, dim)
    rope = s4.Rope(tab, interleaved)
    p = Pair(lens, bits, dtype, 40, 3, seed=dim)
    for i, step in enumerate([0, 5, 28, 1, 33, 64, 150, 300]):
        p.grow([min(n, a + step) for a, n in zip(p.at, lens)], rope, tab, interleaved, Hq=5, in_place=i % 2 == 1, round_=i)
    assert p.at == lens
    p.same()


@pytest.mark.parametrize("bits", FORMATS)
def test_tokens_one_at_a_time(bits):
    lens = [70, 40]
    tab = table(70, 128)
    p = Pair(lens, bits, "bf16", 16, 2, seed=3)
    for i in range(70):
        p.grow([min(n, i + 1) for n in lens], s4.Rope(tab), tab, False, Hq=8 if i % 3 else 0, round_=i)
    p.same()


@pytest.mark.parametrize("bits", FORMATS)
def test_long_prompts_and_many_sequences(bits):
    tab = table(2500, 128)
    p = Pair([2500, 1999], bits, "bf16", 128, 4, seed=4)
    p.grow([1200, 700], s4.Rope(tab), tab, False, Hq=8, round_=0)
    p.grow([2500, 1999], s4.Rope(tab), tab, False, Hq=8, round_=1)
    p.same()
    lens = [(13 * i) % 37 for i in range(300)]
    tab = table(40, 64)
    p = Pair(lens, bits, "fp16", 20, 1, seed=5)
    p.grow([n // 2 for n in lens], s4.Rope(tab), tab, False, Hq=2, round_=0)
    p.grow(lens, s4.Rope(tab), tab, False, Hq=2, round_=1)
    p.same()


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("H,Hq", [(1, 1), (5, 3), (64, 64), (8, 1024), (2, 17)])
def test_head_counts(bits, H, Hq):
    lens = [3, 40, 0, 17]
    tab = table(40, 128)
    p = Pair(lens, bits, "fp16", 24, H, seed=H)
    p.grow([2, 21, 0, 16], s4.Rope(tab), tab, False, Hq=Hq, round_=0)
    p.grow(lens, s4.Rope(tab), tab, False, Hq=Hq, round_=1, in_place=True)
    p.grow(lens, s4.Rope(tab), tab, False, Hq=Hq, round_=2)   # nothing new
    p.same()


@pytest.mark.parametrize("bits", FORMATS)
def test_a_position_past_the_table_is_reported_and_stores_nothing(bits):
    tab = table(100, 128)
    cache = s4.KVCache(1, 40, 2, 16, 2, "bf16", bits=bits)
    cache.pool.zero_()
    if bits == 8:
        cache.set_fp8_scales(0, [1.0, 1.0], [1.0, 1.0])
    bt = torch.arange(40, dtype=torch.int32, device="cuda").view(2, 20)
    k, v = inp.kv_rows(1, 101 + 64, 2, 128, torch.bfloat16)
    q = torch.randn(165, 4, 128, generator=inp.gen(1)).bfloat16().cuda()
    q_out = torch.zeros_like(q)
    cache.append_rope(0, k.cuda(), v.cuda(), _i32([0, 101, 165]), _i32([0, 0]), bt, s4.Rope(tab), q=q, q_out=q_out)
    assert cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_POSITION)
    lay = cache.layout
    lens = cache.pool[lay.lens_offset:lay.lens_offset + 16].view(torch.int32)
    assert lens.tolist() == [0, 0, 64, 64]
    assert not q_out[:101].any() and torch.equal(q_out[101:], rotate(q[101:], torch.arange(64).cuda(), tab, False))
    pages = cache.pool[lay.layer_offset:lay.layer_offset + 40 * lay.page_stride].view(40, -1)
    assert not pages[:20].any() and pages[20:22].any()
    # the last row of the table is a position like any other
    cache.append_rope(0, k[:100].cuda(), v[:100].cuda(), _i32([0, 100]), _i32([0]), bt, s4.Rope(tab))
    assert cache.status() == (0, 0)


def test_argument_errors_launch_nothing():
    cache = s4.KVCache(1, 8, 2, 16, 1, "bf16")
    held = cache.pool.clone()
    tab = table(64, 128)
    bt = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    k, v = (x.cuda() for x in inp.kv_rows(1, 20, 2, 128, torch.bfloat16))
    q = torch.randn(20, 4, 128, generator=inp.gen(1)).bfloat16().cuda()
    c = lambda **kw: s4.s4kv_rope(**{**dict(table=tab.data_ptr(), max_positions=64, rotary_dim=128, interleaved=0), **kw})  # noqa: E731

    def code(want, **kw):
        a = dict(h=cache.h, layer=0, rope=c(), k=k, v=v, num_new_tokens=20, cu_new=_i32([0, 20]), slot_ids=None,
                 seq_lens_before=_i32([0]), block_table=bt, bt_stride=8, n=1, q=q, num_q_heads=4, q_out=q)
        a.update(kw)
        with pytest.raises(s4.S4KVError) as e:
            s4.s4kv_append_rope(**a)
        assert e.value.code == want, kw
    bad, uns = s4.S4KV_ERR_INVALID_ARG, s4.S4KV_ERR_UNSUPPORTED
    for kw in (dict(rope=c(table=None)), dict(rope=c(table=tab.data_ptr() + 4)), dict(rope=c(max_positions=0)),
               dict(rope=c(interleaved=2)), dict(q_out=None), dict(q=None), dict(num_q_heads=0),
               dict(q=q.data_ptr() + 2), dict(k=None), dict(layer=1), dict(cu_new=None), dict(bt_stride=0)):
        code(bad, **kw)
    for d in (0, 8, 24, 144, -16):
        code(uns, rope=c(rotary_dim=d))
    code(uns, num_q_heads=1025)
    for kw in (dict(k=k.float()), dict(k=k[:, :1]), dict(v=v[:-1]), dict(q=q[:-1]), dict(q_out=q), dict(cu_new=_i32([0])),
               dict(block_table=bt.long()), dict(k=k.cpu())):
        a = dict(layer=0, k=k, v=v, cu_new=_i32([0, 20]), seq_lens_before=_i32([0]), block_table=bt, rope=s4.Rope(tab))
        a.update(kw)
        with pytest.raises(ValueError):
            cache.append_rope(**a)
    torch.cuda.synchronize()
    assert torch.equal(held[cache.layout.lens_offset:], cache.pool[cache.layout.lens_offset:])


def test_captured_step_replays():
    """A step captured once and replayed on new rows, lengths advanced on the device."""
    tab = table(64, 128)
    p = Pair([60], INT8, "bf16", 16, 2, seed=8)
    p.grow([10], s4.Rope(tab), tab, False, round_=0)
    k, v, q = (torch.zeros(1, h, 128, dtype=torch.bfloat16, device="cuda") for h in (2, 2, 4))
    cu, before = _i32([0, 1]), _i32([10])
    rope = s4.Rope(tab)
    qo = torch.zeros_like(q)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        p.caches[0].append_rope(0, k, v, cu, before, p.bt, rope, q=q, q_out=qo)
        before.add_(1)
    for t in range(10, 45):
        a, b = inp.kv_rows(100 + t, 1, 2, 128, torch.bfloat16)
        k.copy_(a)
        v.copy_(b)
        q.copy_(torch.randn(1, 4, 128, generator=inp.gen(t)))
        gr.replay()
        at = torch.tensor([t], device="cuda")
        p.caches[1].append(0, rotate(k, at, tab, False), v, cu, _i32([t]), p.bt)
        assert torch.equal(qo, rotate(q, at, tab, False))
    p.same()
