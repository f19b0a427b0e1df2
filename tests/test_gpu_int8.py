"""INT8 block pages: the stored bytes, attention over them, and their refusals."""
import numpy as np
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled, check, int8_rows, restored

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 2], ids=["slices", "clusters"])
def form(request, monkeypatch):
    """A test runs on both launch forms."""
    make = s4.KVCache.__init__

    def init(self, *a, **kw):
        make(self, *a, **kw)
        self.set_option(s4.S4KV_OPT_WINDOW_FORM, request.param)
    monkeypatch.setattr(s4.KVCache, "__init__", init)


def _queries(seed, B, nq, Hq, dtype):
    return torch.randn(B, nq, Hq, 128, generator=inp.gen(seed), dtype=torch.float32).to(dtype).cuda()


def _record_codes(f):
    """Key and value codes [pages, H, 16, 128] and scales [pages, H, 2] as the header documents the record."""
    lay = f.cache.layout
    n = f.cache.cfg.num_pages
    raw = f.cache.pool[lay.layer_offset:lay.layer_offset + n * lay.page_stride].view(n, f.H, lay.record_bytes).cpu().numpy()
    K, V = np.zeros((n, f.H, 16, 128), int), np.zeros((n, f.H, 16, 128), int)
    for kp in range(4):
        for L in range(32):
            a, b = L // 4, L % 4
            w = raw[:, :, kp * 512 + L * 16: kp * 512 + L * 16 + 16].astype(int) - 128
            for x in range(4):
                for j in range(2):
                    K[:, :, a, 32 * b + 8 * kp + 2 * x + j] = w[:, :, 4 * x + j]
                    K[:, :, a + 8, 32 * b + 8 * kp + 2 * x + j] = w[:, :, 4 * x + 2 + j]
            w = raw[:, :, 2048 + kp * 512 + L * 16: 2048 + kp * 512 + L * 16 + 16].astype(int) - 128
            for u in range(2):
                m = 2 * kp + u
                for i, (t, c) in enumerate([(2 * b, 8 * a + m), (2 * b + 1, 8 * a + m), (2 * b, 64 + 8 * a + m),
                                            (2 * b + 1, 64 + 8 * a + m), (2 * b + 8, 8 * a + m), (2 * b + 9, 8 * a + m),
                                            (2 * b + 8, 64 + 8 * a + m), (2 * b + 9, 64 + 8 * a + m)]):
                    V[:, :, t, c] = w[:, :, 8 * u + i]
    sc = np.ascontiguousarray(raw[:, :, 4096:4104]).view(np.float32)
    return K, V, sc


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("chunks", [None, [1], [7], [16], [33, 5, 64], [15, 17]])
def test_codes_scales_and_rings_are_the_definitions(dtype, chunks):
    lens = [1, 15, 16, 17, 32, 100, 0, 131]
    f = Filled(lens, H=3, bits=INT8, dtype=dtype, chunks=chunks, slots=[3, 0, 9, 4, 5, 6, 7, 1], seed=5)
    f.ok()
    K, V, sc = _record_codes(f)
    for b, n in enumerate(lens):
        kc, ks, kr = int8_rows(f.k[b])
        vc, vs, vr = int8_rows(f.v[b])
        for p in range(n // 16):
            pp = int(f.bt[b, p])
            assert np.array_equal(K[pp].transpose(1, 0, 2), kc[p].cpu().numpy()), (b, p)
            assert np.array_equal(V[pp].transpose(1, 0, 2), vc[p].cpu().numpy()), (b, p)
            assert np.array_equal(sc[pp, :, 0], ks[p].cpu().numpy()) and np.array_equal(sc[pp, :, 1], vs[p].cpu().numpy())
        if n:
            gk, gv = f.cache.dequant(0, int(f.slots[b]), f.bt[b], n)
            assert torch.equal(gk.transpose(0, 1), kr) and torch.equal(gv.transpose(0, 1), vr)
    f.ok()


def test_small_and_zero_and_large_blocks():
    """Blocks of zeros, below 2^-100 (stored as zero), of bf16's smallest and largest magnitudes."""
    def edit(b, k, v):
        k[:16] = 0
        v[:16] *= 1e-37
        k[16:32] *= 1e-20
        v[16:32] = (v[16:32].float() * 1e37).to(v.dtype)
        k[32:48] = 3.3e38
        k[40] = -3.3e38
    f = Filled([64], H=2, bits=INT8, seed=8, edit=edit)
    K, V, _, _ = f.plain(0)
    gk, gv = f.cache.dequant(0, 0, f.bt[0], 64)
    assert torch.equal(gk.transpose(0, 1), K) and torch.equal(gv.transpose(0, 1), V)
    assert not gv[:, :16].any() and not gk[:, :16].any()


def test_a_block_that_is_not_finite_restores_to_such_values_and_no_other_does():
    def edit(b, k, v):
        k[20, 0, 5] = float("nan")
        v[37, 1, 9] = float("inf")
    f = Filled([64], H=2, bits=INT8, seed=9, edit=edit)
    gk, gv = f.cache.dequant(0, 0, f.bt[0], 64)
    assert not torch.isfinite(gk[0, 16:32]).any() and torch.isfinite(gk[1]).all()
    assert torch.isfinite(gk[0, :16]).all() and torch.isfinite(gk[0, 32:]).all()
    assert not torch.isfinite(gv[1, 32:48]).any() and torch.isfinite(gv[0]).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,g", [(1, 1), (2, 4), (3, 5), (4, 7), (1, 8)])
def test_decode(dtype, H, g, form):
    lens = [1, 15, 16, 17, 0, 255, 257, 1000, 2049]
    f = Filled(lens, H=H, bits=INT8, dtype=dtype, seed=11 + g, slots=[8, 7, 6, 5, 4, 3, 2, 1, 0])
    q = _queries(3, len(lens), 1, H * g, f.dtype)
    for od in (s4.S4KV_F32, f.cache.cdtype):
        out = f.cache.decode(0, q[:, 0], f.bt, f.seq, max(lens), out_dtype=od, slot_ids=f.slots)
        f.ok()
        for b, n in enumerate(lens):
            if n == 0:
                assert not out[b].any()
            else:
                check(out[b:b + 1], q[b], *f.plain(b), [n - 1], INT8, what=f"seq {b} of {n}")


@pytest.mark.parametrize("nq,H,g", [(2, 1, 3), (4, 2, 4), (5, 1, 2), (16, 1, 6), (16, 3, 1), (3, 2, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_multi_query(nq, H, g, dtype, form):
    lens = [nq, nq + 1, 16 + nq, 31, 64, 333, 1500]
    lens = [max(n, nq) for n in lens]
    f = Filled(lens, H=H, bits=INT8, dtype=dtype, seed=30 + nq, chunks=[7, 100])
    q = _queries(4, len(lens), nq, H * g, f.dtype)
    out = f.cache.multi_query(0, q, f.bt, f.seq, max(lens))
    f.ok()
    for b, n in enumerate(lens):
        check(out[b], q[b], *f.plain(b), range(n - nq, n), INT8, what=f"seq {b} of {n}")


def test_decode_splits_agree_with_one_worker(form):
    """The same call on one worker warp and on all: the combine changes roundings only."""
    f = Filled([4000], H=2, bits=INT8, seed=2)
    q = _queries(5, 1, 1, 8, f.dtype)
    f.cache.set_option(s4.S4KV_OPT_DECODE_WARPS, 1)
    one = f.cache.decode(0, q[:, 0], f.bt, f.seq, 4000)
    f.cache.set_option(s4.S4KV_OPT_DECODE_WARPS, 0)
    all_ = f.cache.decode(0, q[:, 0], f.bt, f.seq, 4000)
    K = f.plain(0)
    check(one, q[0], *K, [3999], INT8)
    check(all_, q[0], *K, [3999], INT8)
    assert torch.equal(all_, f.cache.decode(0, q[:, 0], f.bt, f.seq, 4000))   # no order depends on timing


def test_decode_step_and_noalloc_equal_append_and_decode(form):
    lens = [0, 14, 15, 16, 200]
    f = Filled(lens, H=2, bits=INT8, seed=21, spare=40)
    g = Filled(lens, H=2, bits=INT8, seed=21, spare=40)
    cu = f.i32(range(len(lens) + 1))
    for s in range(20):
        k, v = inp.kv_rows(inp.mix_seed(77, s), len(lens), 2, 128, f.dtype)
        k, v = k.cuda(), v.cuda()
        q = _queries(100 + s, len(lens), 1, 8, f.dtype)[:, 0].contiguous()
        before, after = f.i32([n + s for n in lens]), f.i32([n + s + 1 for n in lens])
        top = max(lens) + s + 1
        f.cache.append(0, k, v, cu, before, f.bt)
        want = f.cache.decode(0, q, f.bt, after, top)
        got, got2 = torch.empty_like(want), torch.empty_like(want)
        ws, nb = g.cache.workspace(len(lens), 8, top)
        s4.s4kv_decode_step(g.cache.h, 0, k, v, q, 8, g.bt, g.bt.shape[1], after, None, len(lens), 0.0, got,
                            s4.S4KV_F32, ws, nb, top)
        s4.s4kv_decode_attention_noalloc(g.cache.h, 0, q, 8, g.bt, g.bt.shape[1], after, None, len(lens), 0.0, got2,
                                         s4.S4KV_F32, top)
        assert torch.equal(got, want) and torch.equal(got2, want)
    f.ok()
    g.ok()
    lay = f.cache.layout   # lengths, pages and rings: the same bytes
    assert torch.equal(f.cache.pool[lay.layer_offset:], g.cache.pool[lay.layer_offset:]) or \
        all(torch.equal(a, b) for i, n in enumerate(lens)
            for a, b in zip(f.cache.dequant(0, i, f.bt[i], n + 20), g.cache.dequant(0, i, g.bt[i], n + 20)))


def test_bad_caller_data_is_reported(form):
    f = Filled([100, 50], H=2, bits=INT8, seed=1, spare=20)
    q = _queries(1, 2, 1, 4, f.dtype)[:, 0].contiguous()

    def status(code, detail):
        assert f.cache.status() == (code, detail)

    good = f.cache.decode(0, q, f.bt, f.seq, 100)
    for entry in (-1, f.cache.cfg.num_pages):
        bt = f.bt.clone()
        bt[0, 2] = entry
        out = f.cache.decode(0, q, bt, f.seq, 100)
        status(s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)
        assert torch.equal(out[1], good[1])
    out = f.cache.decode(0, q, f.bt, f.i32([100, 51]), 100)
    status(s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    assert not out[1].any() and torch.equal(out[0], good[0])
    f.cache.decode(0, q, f.bt, f.seq, 99)
    status(s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    f.cache.decode(0, q, f.bt[:, :6].contiguous(), f.seq, 100)
    status(s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_TABLE)
    f.cache.decode(0, q, f.bt, f.seq, 100, slot_ids=f.i32([0, 2]))
    status(s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_SLOT)
    # appends: a wrong length, slot, table and cu_new change nothing
    k, v = inp.kv_rows(3, 20, 2, 128, f.dtype)
    k, v, lay = k.cuda(), v.cuda(), f.cache.layout
    held = f.cache.pool[lay.lens_offset:].clone()
    one = f.bt[:1].contiguous()
    for cu, before, bt, slots, detail in (
            ([0, 20], [99], one, None, s4.S4KV_DEV_BAD_LENGTH), ([0, 20], [100], one, [2], s4.S4KV_DEV_BAD_SLOT),
            ([0, 20], [100], one[:, :7].contiguous(), None, s4.S4KV_DEV_BAD_TABLE),
            ([0, 19], [100], one, None, s4.S4KV_DEV_BAD_CU), ([1, 20], [100], one, None, s4.S4KV_DEV_BAD_CU),
            ([0, 20], [-1], one, None, s4.S4KV_DEV_BAD_CU)):
        f.cache.append(0, k, v, f.i32(cu), f.i32(before), bt, slot_ids=None if slots is None else f.i32(slots))
        status(s4.S4KV_ERR_DEVICE, detail)
        assert torch.equal(held, f.cache.pool[lay.lens_offset:])
    assert torch.equal(f.cache.decode(0, q, f.bt, f.seq, 100), good)
    f.ok()


def test_bounded_wait_gives_up_and_the_next_call_is_clean(form):
    f = Filled([3000, 2500], H=2, bits=INT8, seed=6)
    q = _queries(2, 2, 1, 8, f.dtype)[:, 0].contiguous()
    good = f.cache.decode(0, q, f.bt, f.seq, 3000)
    f.cache.set_option(s4.S4KV_OPT_WAIT_NS, 0)
    f.cache.decode(0, q, f.bt, f.seq, 3000)
    assert f.cache.status() == (s4.S4KV_ERR_DEVICE_TIMEOUT, s4.S4KV_DEV_TIMEOUT)
    f.cache.set_option(s4.S4KV_OPT_WAIT_NS, 1_000_000_000)
    assert torch.equal(f.cache.decode(0, q, f.bt, f.seq, 3000), good)
    f.ok()


def test_rows_behind_the_last_sequence_and_other_pages_are_left():
    f = Filled([70, 33], H=2, bits=INT8, seed=13, loose=3, slots=[2, 0])
    used = set(int(x) for b, n in enumerate(f.lens) for x in f.bt[b, :n // 16])
    lay, n = f.cache.layout, f.cache.cfg.num_pages
    pages = f.cache.pool[lay.layer_offset:lay.layer_offset + n * lay.page_stride].view(n, -1)
    other = [p for p in range(n) if p not in used]
    pages[other] = 0xA5
    out = torch.full((3, 4, 128), 7.0, device="cuda")
    q = _queries(2, 2, 1, 4, f.dtype)[:, 0].contiguous()
    f.cache.decode(0, q, f.bt, f.seq, 70, out=out[:2], slot_ids=f.slots)
    assert bool((out[2] == 7.0).all()) and bool((pages[other] == 0xA5).all())
    f.ok()


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB: the last pages hold the sequence."""
    H, pages = 8, 140000
    cache = s4.KVCache(1, pages, H, 32, 2, "bf16", bits="int8")
    n = 1000
    need = -(-n // 16)
    bt = torch.arange(pages - need, pages, dtype=torch.int32, device="cuda")[None]
    assert (pages - need) * H * 4128 > 2 ** 32
    k, v = inp.kv_rows(4, n, H, 128, torch.bfloat16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache.append(0, k, v, i32(0, n), i32(0), bt, slot_ids=i32(1))
    q = _queries(2, 1, 1, 32, torch.bfloat16)
    out = cache.decode(0, q[:, 0], bt, i32(n), n, slot_ids=i32(1))
    assert cache.status() == (0, 0)
    check(out, q[0], *restored(k, v, INT8, 32), [n - 1], INT8)
