"""Token ranges restored into dense rows, and the operators together as a server uses them."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8, Filled, check

pytestmark = pytest.mark.gpu
FORMATS = [4, 2, 8, INT8]


def _scales(bits, H):
    return ([0.5 + 0.25 * h for h in range(H)], [1.5 - 0.25 * h for h in range(H)]) if bits == 8 else None


def _cu(counts, f):
    cu = [0]
    for n in counts:
        cu.append(cu[-1] + n)
    return f.i32(cu), cu


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("residual", [1, 16, 50])
def test_rows_are_the_restored_tokens(bits, dtype, residual):
    lens = [1, 0, 16, 33, 64, 257, 100, 90]
    f = Filled(lens, H=3, bits=bits, dtype=dtype, residual=residual, seed=6, slots=[7, 6, 5, 4, 3, 2, 1, 0],
               fp8_scales=_scales(bits, 3), chunks=[40, 21])
    plain = [f.plain(b) for b in range(len(lens))]
    for first, counts in (([0] * 8, lens), ([0, 0, 15, 1, 31, 100, 99, 17], [1, 0, 1, 31, 2, 157, 1, 16]),
                          ([0, 0, 0, 30, 64, 255, 0, 5], [0, 0, 16, 3, 0, 2, 100, 0])):
        cu, c = _cu(counts, f)
        for od in (s4.S4KV_F32, f.cache.cdtype):
            k, v = f.cache.gather(0, f.bt, f.seq, cu, c[-1], first=f.i32(first), slot_ids=f.slots, out_dtype=od)
            f.ok()
            for b in range(len(lens)):
                for got, want in ((k, plain[b][0]), (v, plain[b][1])):
                    assert torch.equal(got[c[b]:c[b + 1]], want[first[b]:first[b] + counts[b]].to(got.dtype)), (b, first[b], counts[b])
    k, v = f.cache.gather(0, f.bt, f.seq, _cu(lens, f)[0], sum(lens), slot_ids=f.slots)
    assert torch.equal(k, torch.cat([p[0] for p in plain])) and torch.equal(v, torch.cat([p[1] for p in plain]))


@pytest.mark.parametrize("bits", FORMATS)
def test_many_short_ranges(bits):
    lens = [(29 * i) % 75 for i in range(500)]
    f = Filled(lens, H=1, bits=bits, residual=20, seed=4)
    counts = [min(n, (7 * i) % 40) for i, n in enumerate(lens)]
    first = [(n - c) // 2 for n, c in zip(lens, counts)]
    cu, c = _cu(counts, f)
    k, v = f.cache.gather(0, f.bt, f.seq, cu, c[-1], first=f.i32(first))
    f.ok()
    want = [f.plain(b) for b in range(500)]
    assert torch.equal(k, torch.cat([w[0][a:a + n] for w, a, n in zip(want, first, counts)]))
    assert torch.equal(v, torch.cat([w[1][a:a + n] for w, a, n in zip(want, first, counts)]))


@pytest.mark.parametrize("bits", FORMATS)
def test_only_the_pages_of_the_range_are_needed(bits):
    f = Filled([200], H=2, bits=bits, residual=32, seed=4)
    bt = f.bt.clone()
    bt[0, :4] = -1
    bt[0, 8:] = -7
    k, v = f.cache.gather(0, bt, f.seq, f.i32([0, 64]), 64, first=f.i32([64]))
    f.ok()
    K, V, _, _ = f.plain(0)
    assert torch.equal(k, K[64:128]) and torch.equal(v, V[64:128])
    out = torch.full((66, 2, 128), 3.0, device="cuda")
    f.cache.gather(0, bt, f.seq, f.i32([0, 66]), 66, first=f.i32([62]), out_k=out, out_v=out.clone())
    assert f.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)
    assert bool((out[:2] == 3.0).all()) and torch.equal(out[2:], K[64:128])


@pytest.mark.parametrize("bits", FORMATS)
def test_bad_caller_data_is_reported_and_its_rows_are_left(bits):
    f = Filled([100, 50], H=2, bits=bits, residual=32, seed=4)
    K, V, _, _ = f.plain(0)

    def bad(detail, seq=(100, 50), first=(0, 0), slots=None, bt=f.bt, cu=(0, 30, 50), rows=50, kept=True):
        k = torch.full((rows, 2, 128), 3.0, device="cuda")
        v = k.clone()
        f.cache.gather(0, bt, f.i32(seq), f.i32(cu), rows, first=f.i32(first), out_k=k, out_v=v,
                       slot_ids=None if slots is None else f.i32(slots))
        assert f.cache.status() == (s4.S4KV_ERR_DEVICE, detail)
        assert bool((k[30:] == 3.0).all()) and bool((v[30:] == 3.0).all())
        if kept:
            assert torch.equal(k[:30], K[first[0]:first[0] + 30]) and torch.equal(v[:30], V[first[0]:first[0] + 30])
        else:
            assert bool((k == 3.0).all()) and bool((v == 3.0).all())
    bad(s4.S4KV_DEV_BAD_LENGTH, seq=(100, 49))
    bad(s4.S4KV_DEV_BAD_LENGTH, seq=(100, -1))
    bad(s4.S4KV_DEV_BAD_POSITION, first=(7, 31))
    bad(s4.S4KV_DEV_BAD_POSITION, first=(70, 1000000))
    bad(s4.S4KV_DEV_BAD_SLOT, slots=(0, 2))
    bad(s4.S4KV_DEV_BAD_SLOT, slots=(0, -1))
    bad(s4.S4KV_DEV_BAD_TABLE, bt=f.bt[:, :2].contiguous(), first=(0, 30))
    for cu in ((0, 30, 49), (1, 30, 50), (0, 60, 50)):
        bad(s4.S4KV_DEV_BAD_CU, cu=cu, kept=False)
    bad(s4.S4KV_DEV_BAD_CU, first=(-1, 0), kept=False)


@pytest.mark.parametrize("bits", FORMATS)
def test_a_slot_asked_for_twice_and_another_layer(bits):
    f = Filled([150], H=2, bits=bits, residual=32, seed=5)
    two = s4.KVCache(2, f.cache.cfg.num_pages, 2, 32, 1, "bf16", bits=bits)
    two.append(1, f.k[0], f.v[0], f.i32([0, 150]), f.i32([0]), f.bt)
    K, V, _, _ = f.plain(0)
    k, v = two.gather(1, torch.cat([f.bt, f.bt, f.bt]), f.i32([150] * 3), f.i32([0, 100, 100, 150]), 150,
                      first=f.i32([50, 3, 17]), slot_ids=f.i32([0, 0, 0]))
    assert two.status() == (0, 0)
    assert torch.equal(k, torch.cat([K[50:], K[17:67]])) and torch.equal(v, torch.cat([V[50:], V[17:67]]))
    two.gather(0, f.bt, f.i32([150]), f.i32([0, 10]), 10)
    assert two.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)


@pytest.mark.parametrize("H", [1, 3, 5, 8, 64])
def test_head_counts(H):
    for bits in FORMATS:
        f = Filled([70, 33], H=H, bits=bits, residual=20, seed=H)
        k, v = f.cache.gather(0, f.bt, f.seq, f.i32([0, 70, 103]), 103, out_dtype=f.cache.cdtype)
        f.ok()
        for b, rows in ((0, slice(0, 70)), (1, slice(70, 103))):
            K, V, _, _ = f.plain(b)
            assert torch.equal(k[rows], K.to(k.dtype)) and torch.equal(v[rows], V.to(v.dtype))


def test_a_table_that_ends_inside_a_key_group_is_refused():
    """KIVI pages: tokens 64..79 need the metadata of pages 4 and 5; a table of five columns has not both."""
    f = Filled([96, 96], H=2, bits=4, residual=16, seed=4)
    k = torch.full((160, 2, 128), 3.0, device="cuda")
    f.cache.gather(0, f.bt[:, :5].contiguous(), f.seq, f.i32([0, 80, 160]), 160, out_k=k, out_v=k.clone())
    assert f.cache.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_TABLE) and bool((k == 3.0).all())
    f.cache.gather(0, f.bt[:, :4].contiguous(), f.seq, f.i32([0, 64, 128]), 128, out_k=k[:128], out_v=k[:128].clone())
    f.ok()
    assert torch.equal(k[:64], f.plain(0)[0][:64]) and torch.equal(k[64:128], f.plain(1)[0][:64])


def test_argument_errors_launch_nothing():
    f = Filled([100], H=2, bits=4, seed=4)
    out = torch.full((100, 2, 128), 3.0, device="cuda")

    def code(want, **kw):
        a = dict(h=f.cache.h, layer=0, block_table=f.bt, bt_stride=f.bt.shape[1], seq_lens=f.seq, slot_ids=None,
                 first_token=None, cu_rows=f.i32([0, 100]), num_rows=100, n=1, out_k=out, out_v=out,
                 out_dtype=s4.S4KV_F32)
        a.update(kw)
        with pytest.raises(s4.S4KVError) as e:
            s4.s4kv_gather(**a)
        assert e.value.code == want, kw
    for kw in (dict(layer=-1), dict(n=-1), dict(n=0), dict(n=8193), dict(num_rows=-1), dict(out_k=None),
               dict(out_v=out.data_ptr() + 4), dict(cu_rows=None), dict(seq_lens=None), dict(block_table=None),
               dict(bt_stride=0), dict(out_dtype=s4.S4KV_F16)):
        code(s4.S4KV_ERR_INVALID_ARG, **kw)
    torch.cuda.synchronize()
    assert bool((out == 3.0).all())
    for kw in (dict(cu_rows=f.i32([0])), dict(first=f.i32([0, 0])), dict(out_k=out[:50]), dict(out_k=out.half()),
               dict(seq_lens=f.seq.float()), dict(out_dtype=s4.S4KV_F16)):
        a = dict(layer=0, block_table=f.bt, seq_lens=f.seq, cu_rows=f.i32([0, 100]), num_rows=100)
        a.update(kw)
        with pytest.raises(ValueError):
            f.cache.gather(**a)
    k, v = f.cache.gather(0, f.bt[:0], f.seq[:0], f.i32([0]), 0)   # nothing asked for
    assert k.shape == v.shape == (0, 2, 128)
    f.ok()


@pytest.mark.parametrize("bits", FORMATS)
def test_a_windowed_model_served(bits):
    """Prompts appended with rotation, the prefix restored, then steps and drafts: rotated append, windowed
    attention, against the plain model of the same tokens. The pages behind the window are given to others."""
    H, Hq, window, sinks, R = 2, 8, 60, 4, 32
    lens, steps = [150, 90], 40
    total = [n + steps for n in lens]
    half = 64
    at = torch.arange(max(total), dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    rope = s4.Rope(torch.cat([at.cos(), at.sin()], 1).float().cuda())
    cos, sin = rope.table[:, None, :half], rope.table[:, None, half:]

    def turn(x, pos):
        a, b = x.float()[..., :half], x.float()[..., half:]
        return torch.cat([a * cos[pos] - b * sin[pos], b * cos[pos] + a * sin[pos]], -1).to(x.dtype)
    f = Filled([0, 0], H=H, bits=bits, residual=R, seed=3, spare=max(total))
    c = f.cache
    raw = [inp.kv_rows(50 + b, total[b], H, 128, f.dtype) for b in range(2)]
    raw = [(k.cuda(), v.cuda()) for k, v in raw]
    keys = [turn(k, torch.arange(total[b])) for b, (k, v) in enumerate(raw)]
    at_, bt = [0, 0], f.bt.clone()
    for n, nq in [(lens, 1)] + [([m + i + 1 for m in lens], 1) for i in range(0, 30)] + [([m + 35 for m in lens], 5), (total, 5)]:
        new = [y - x for x, y in zip(at_, n)]
        cu = [0, new[0], sum(new)]
        q = torch.randn(cu[-1], Hq, 128, generator=inp.gen(n[0])).to(f.dtype).cuda()
        got = c.append_rope(0, torch.cat([raw[b][0][at_[b]:n[b]] for b in range(2)]),
                            torch.cat([raw[b][1][at_[b]:n[b]] for b in range(2)]), f.i32(cu), f.i32(at_), bt, rope, q=q)
        at_ = list(n)
        qs = torch.stack([got[cu[b + 1] - nq:cu[b + 1]] for b in range(2)])
        out = c.window(0, qs, bt, f.i32(n), max(n), window, sinks)
        f.ok()
        from plain_cache import restored
        for b in range(2):
            m = restored(keys[b][:n[b]], raw[b][1][:n[b]], bits, R)
            check(out[b], qs[b], *m, range(n[b] - nq, n[b]), bits, window, sinks, f"{n}")
            if n == lens:
                k, v = c.gather(0, bt, f.i32(n), f.i32([0, n[0], sum(n)]), sum(n))
                assert torch.equal(k[[0, n[0]][b]:][:n[b]], m[0]) and torch.equal(v[[0, n[0]][b]:][:n[b]], m[1])
            # whole 32-token groups behind the window of the next calls are no longer needed
            dead = (n[b] + 1 - 5 - window + 1 - R) // 32 * 2
            if dead > 2:
                bt[b, 2:dead] = -1
