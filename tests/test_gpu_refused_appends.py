"""An append whose sequence is reported stores nothing of it: a call made again with its old lengths, where
the slot already stands at the length that the call would leave, and others. Every byte of lengths, pages
and rings is compared."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8

pytestmark = pytest.mark.gpu
FORMATS = [INT8, 4, 2, 8]


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _rope(rows):
    at = torch.arange(rows, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)
    return s4.Rope(torch.cat([at.cos(), at.sin()], 1).float().cuda())


def _cache(bits, H, pages, slots, residual=32):
    c = s4.KVCache(1, pages, H, residual, slots, "bf16", bits=bits)
    c.pool.zero_()
    if bits == 8:   # a power of two, and not
        c.set_fp8_scales(0, [(0.5, 0.37)[h % 2] for h in range(H)], [(1.3, 2.0)[h % 2] for h in range(H)])
    return c


def _rows(seed, n, H):
    return tuple(x.cuda() for x in inp.kv_rows(seed, n, H, 128, torch.bfloat16))


def _held(c):
    return c.pool[c.layout.lens_offset:].clone()


def _refused(c, held):
    assert c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    assert torch.equal(held, _held(c))


# tokens stored, then appended by the call that is made again: one token, one that completes a page, chunks
# inside a page, over a page's end, of whole pages and key groups, long ones
CALLS = [(30, 1), (31, 1), (10, 4), (10, 20), (8, 16), (16, 16), (32, 64), (33, 200), (5, 700), (1000, 1500)]


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("H", [1, 3, 8])
@pytest.mark.parametrize("T0,new", CALLS)
def test_a_call_made_again_stores_nothing(bits, rope, H, T0, new):
    most = T0 + 2 * new + 16
    pages = -(-most // 16)
    c = _cache(bits, H, pages + 5, 2)
    bt = torch.randperm(pages + 5, generator=inp.gen(H))[:pages].int().cuda()[None]
    table, slot = _rope(most), _i32(1)

    def append(before, k, v):
        if rope:
            c.append_rope(0, k, v, _i32(0, k.shape[0]), _i32(before), bt, table, slot_ids=slot)
        else:
            c.append(0, k, v, _i32(0, k.shape[0]), _i32(before), bt, slot_ids=slot)
    first, second, other = _rows(1, T0, H), _rows(2, new, H), _rows(3, new, H)
    append(0, *first)
    append(T0, *second)
    assert c.status() == (0, 0)
    held = _held(c)
    for rows in (second, other):
        append(T0, *rows)
        _refused(c, held)
    for before in (T0 - 1, T0 + new - 1, T0 + new + 1):   # lengths that the slot never stops at here
        if before > 0 and before != T0:
            append(before, *_rows(4, min(new, 64), H))
            _refused(c, held)
    append(T0 + new, *other)                               # the slot goes on where it was
    assert c.status() == (0, 0)
    lens = c.pool[c.layout.lens_offset:c.layout.lens_offset + 8 * H].view(torch.int32).tolist()
    assert lens == [0] * H + [T0 + 2 * new] * H


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("new", [1, 20, 300])
def test_sequences_beside_a_refused_one_are_appended(bits, rope, new):
    """Of seven sequences every other one is refused: the pool is that of a call with the others alone."""
    H, T0 = 2, 25
    seqs, pages = 7, -(-(25 + 2 * new) // 16)
    bt = torch.randperm(seqs * pages, generator=inp.gen(new)).int().cuda().view(seqs, pages)
    table = _rope(T0 + 2 * new)
    a, b = (_cache(bits, H, seqs * pages, seqs) for _ in range(2))

    def append(c, which, before, k, v):
        cu = [0]
        for _ in which:
            cu.append(cu[-1] + k.shape[0] // len(which))
        args = (0, k, v, _i32(*cu), _i32(*before), bt[list(which)].contiguous())
        if rope:
            c.append_rope(*args, table, slot_ids=_i32(*which))
        else:
            c.append(*args, slot_ids=_i32(*which))
    k, v = _rows(1, seqs * T0, H)
    k1, v1 = _rows(2, seqs * new, H)
    k2, v2 = _rows(3, seqs * new, H)
    ahead, level = list(range(0, seqs, 2)), list(range(1, seqs, 2))
    part = lambda x, which: torch.cat([x[new * i:new * i + new] for i in which])  # noqa: E731
    for c in (a, b):
        append(c, range(seqs), [0] * seqs, k, v)
        append(c, ahead, [T0] * len(ahead), part(k1, ahead), part(v1, ahead))
        assert c.status() == (0, 0)
    append(a, range(seqs), [T0] * seqs, k2, v2)
    assert a.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    append(b, level, [T0] * len(level), part(k2, level), part(v2, level))
    assert b.status() == (0, 0)
    assert torch.equal(_held(a), _held(b))


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("T0", [1, 15, 16, 30, 31, 100])
def test_a_decode_step_made_again_stores_nothing(bits, T0):
    H, Hq = 2, 8
    c = _cache(bits, H, 10, 1)
    bt = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    c.append(0, *_rows(1, T0, H), _i32(0, T0), _i32(0), bt)
    q = torch.randn(1, Hq, 128, generator=inp.gen(1)).bfloat16().cuda()
    out = torch.empty(1, Hq, 128, device="cuda")
    ws, nb = c.workspace(1, Hq, 160)

    def step(length, k, v):
        s4.s4kv_decode_step(c.h, 0, k, v, q, Hq, bt, 10, _i32(length), None, 1, 0.0, out, s4.S4KV_F32, ws, nb, 160)
    row, other = _rows(2, 1, H), _rows(3, 1, H)
    step(T0 + 1, *row)
    assert c.status() == (0, 0)
    held = _held(c)
    for rows in (row, other):
        step(T0 + 1, *rows)
        _refused(c, held)
    want = c.decode(0, q, bt, _i32(T0 + 1), 160)
    assert c.status() == (0, 0)
    assert torch.equal(out, want)     # the attention of the refused step is over what is stored
    step(T0 + 2, *other)
    assert c.status() == (0, 0)


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("H", [1, 3, 5, 8, 64])
def test_chunks_behind_stored_tokens(bits, H):
    """Chunks of whole pages behind stored tokens, in one call and in pieces, leave the same bytes."""
    lens = [700, 45, 333, 16]
    pages = sum(-(-n // 16) for n in lens)
    perm = torch.randperm(pages, generator=inp.gen(H)).int()
    bt = torch.zeros(len(lens), 44, dtype=torch.int32)
    at = 0
    for b, n in enumerate(lens):
        bt[b, :-(-n // 16)] = perm[at:at - (-n // 16)]
        at -= -n // 16
    bt = bt.cuda()
    k = [_rows(10 + b, n, H) for b, n in enumerate(lens)]
    pools = []
    for cuts in ([0, 700], [0, 9, 700], [0, 16, 17, 300, 700]):
        c = _cache(bits, H, pages, len(lens))
        for lo, hi in zip(cuts, cuts[1:]):
            a, z = [min(n, lo) for n in lens], [min(n, hi) for n in lens]
            cu = [0]
            for x, y in zip(a, z):
                cu.append(cu[-1] + y - x)
            c.append(0, *(torch.cat([r[i][x:y] for r, x, y in zip(k, a, z)]) for i in range(2)), _i32(*cu), _i32(*a), bt)
        assert c.status() == (0, 0)
        pools.append([c.dequant(0, b, bt[b], n) for b, n in enumerate(lens)])
        assert c.status() == (0, 0)
    for other in pools[1:]:
        for (k0, v0), (k1, v1) in zip(pools[0], other):
            assert torch.equal(k0, k1) and torch.equal(v0, v1)


@pytest.mark.parametrize("bits", FORMATS)
@pytest.mark.parametrize("rope", [False, True])
@pytest.mark.parametrize("seed", range(6))
def test_ragged_calls_with_some_sequences_refused(bits, rope, seed):
    """Random lengths, chunks, slots and refusals (lengths already reached, others, slots and tables out of range
    beside them): the pool is that of the same calls with the accepted sequences alone."""
    rng = torch.Generator().manual_seed(100 + seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=rng))  # noqa: E731
    H, n = (1, 2, 3, 4, 8, 5)[seed], pick(3, 40)
    most = 900
    pages = -(-most // 16)
    bt = torch.randperm(n * pages, generator=rng).int().cuda().view(n, pages)
    slots = torch.randperm(n, generator=rng).tolist()
    table = _rope(most)
    a, b = (_cache(bits, H, n * pages, n) for _ in range(2))

    def append(c, which, before, new, k, v, ids):
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        args = (0, k, v, _i32(*cu), _i32(*before), bt[which].contiguous())
        if rope:
            c.append_rope(*args, table, slot_ids=_i32(*ids))
        else:
            c.append(*args, slot_ids=_i32(*ids))
    at = [0] * n
    for call in range(5):
        new = [pick(0, (3, 40, 200)[pick(0, 2)]) for _ in range(n)]
        new = [min(x, most - t - 201) for x, t in zip(new, at)]
        before, ids, good = list(at), list(slots), []
        for i in range(n):
            how = pick(0, 5) if at[i] > 0 and call else 0
            if how == 1 and new[i] > 0 and at[i] > new[i]:
                before[i] = at[i] - new[i]            # the slot stands at the length that the call would leave
            elif how == 2:
                before[i] = at[i] + 1 + pick(0, 9)
            elif how == 3:
                ids[i] = n + pick(0, 3)
            else:
                good.append(i)
        rows = [_rows(1000 * seed + 100 * call + i, new[i], H) for i in range(n)]
        append(a, list(range(n)), before, new, torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]), ids)
        rc, detail = a.status()
        assert (rc == 0) == (len(good) == n)
        append(b, good, [before[i] for i in good], [new[i] for i in good], torch.cat([rows[i][0] for i in good]),
               torch.cat([rows[i][1] for i in good]), [slots[i] for i in good])
        assert b.status() == (0, 0)
        for i in good:
            at[i] += new[i]
        assert torch.equal(_held(a), _held(b)), call
    for i in range(n):
        lens = a.pool[a.layout.lens_offset:].view(torch.int32)[slots[i] * H:slots[i] * H + H].tolist()
        assert lens == [at[i]] * H


@pytest.mark.parametrize("bits", FORMATS)
def test_chunks_of_other_slots_and_layers_at_once(bits):
    """Chunks behind stored tokens on three streams, two slots of one layer and one of another, and a captured
    chunk replayed: each leaves what it leaves alone."""
    H, T0, new = 4, 40, 300
    pages = -(-(T0 + 2 * new) // 16)
    bt = torch.arange(2 * pages, dtype=torch.int32, device="cuda").view(2, pages)
    rows = [[_rows(10 * w + x, T0 if x == 0 else new, H) for x in range(3)] for w in range(3)]
    where = [(0, 0), (0, 1), (1, 0)]           # (layer, slot)
    streams = [torch.cuda.Stream() for _ in where]
    held = []
    for together in (False, True):
        c = s4.KVCache(2, 2 * pages, H, 32, 2, "bf16", bits=bits)
        c.pool[c.layout.layer_offset:].zero_()
        one = [(_i32(0, T0), _i32(0), _i32(0, new), _i32(T0), _i32(T0 + new), bt[s:s + 1].contiguous(), _i32(s)) for _, s in where]
        for (layer, _), r, o in zip(where, rows, one):
            c.append(layer, *r[0], o[0], o[1], o[5], slot_ids=o[6])
        torch.cuda.synchronize()
        for x, before in ((1, 3), (2, 4)):
            for (layer, _), r, o, st in zip(where, rows, one, streams):
                c.append(layer, *r[x], o[2], o[before], o[5], slot_ids=o[6], stream=st if together else None)
        torch.cuda.synchronize()
        assert c.status() == (0, 0)
        held.append(_held(c))
    assert torch.equal(*held)
    lens = c.pool[c.layout.lens_offset:c.layout.lens_offset + 16 * H].view(torch.int32).tolist()
    assert lens == [T0 + 2 * new] * 3 * H + [0] * H
    # the same chunk captured, its length advanced on the device
    c = s4.KVCache(1, pages, H, 32, 1, "bf16", bits=bits)
    d = s4.KVCache(1, pages, H, 32, 1, "bf16", bits=bits)
    for x in (c, d):
        x.pool[x.layout.layer_offset:].zero_()
        x.append(0, *rows[0][0], _i32(0, T0), _i32(0), bt[:1])
    k, v, cu, before, row = *(x.clone() for x in rows[0][1]), _i32(0, new), _i32(T0), bt[:1].contiguous()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        c.append(0, k, v, cu, before, row)
        before.add_(new)
    for x in (1, 2):
        k.copy_(rows[0][x][0])
        v.copy_(rows[0][x][1])
        gr.replay()
        d.append(0, *rows[0][x], _i32(0, new), _i32(T0 + (x - 1) * new), bt[:1])
    assert c.status() == (0, 0) and d.status() == (0, 0)
    assert torch.equal(_held(c), _held(d))
