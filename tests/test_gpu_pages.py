"""Pages taken, released and shared by forks on the GPU, against plain Python."""
import random

import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def pool(num_pages, layers=1, H=1, slots=8, bits=4, residual=32, dtype="bf16"):
    return s4.KVCache(layers, num_pages, H, residual, slots, dtype, bits=bits)


def up(n):
    return -(-n // 16)


def take(refs, table, lens, new, rows):
    """The rule, entry by entry, on lists; what each sequence got."""
    free = [p for p, r in enumerate(refs) if r == 0]
    room, asked, got = len(free), 0, []
    for a, b, row in zip(lens, new, rows):
        need = up(b) - up(a)
        asked += need
        if need and asked > room:
            got.append(-1)
            continue
        for e in range(up(a), up(b)):
            table[row][e] = free.pop(0)
            refs[table[row][e]] = 1
        got.append(need)
    return got


def release(refs, table, first, last, rows):
    for a, b, row in zip(first, last, rows):
        for e in range(up(a), up(b)):
            if table[row][e] >= 0:
                refs[table[row][e]] -= 1
                table[row][e] = -1


def same(refs, table, dev_refs, dev_table):
    assert dev_refs.tolist() == refs and dev_table.tolist() == table


def ok(c):
    rc, detail = c.status()
    assert rc == 0, (rc, detail)


@pytest.mark.parametrize("num_pages,slots,width,longest", [(40, 5, 12, 190), (40000, 300, 150, 2390), (33333, 4096, 9, 140), (1, 1, 1, 16)])
@pytest.mark.parametrize("by_slot", [False, True])
def test_steps_of_a_scheduler(num_pages, slots, width, longest, by_slot):
    rng = random.Random(num_pages + by_slot)
    c = pool(num_pages, slots=min(slots, 16))
    # a fragmented pool: some pages are somebody else's
    refs = [rng.choice([0, 0, 0, 1, 2]) for _ in range(num_pages)]
    table = [[-1] * width for _ in range(slots)]
    d_refs, d_table = i32(refs), i32(table)
    lens = [0] * slots
    for _ in range(6):
        rows = list(range(slots))
        if by_slot:
            rng.shuffle(rows)
            rows = rows[:max(1, slots * 3 // 4)]
        new = [min(longest, lens[r] + rng.choice([0, 1, 5, 16, 17, 100, longest])) for r in rows]
        now = [lens[r] for r in rows]
        want = take(refs, table, now, new, rows)
        got = c.take_pages(d_refs, d_table, i32(now), i32(new), slot_ids=i32(rows) if by_slot else None)
        assert got.tolist() == want
        same(refs, table, d_refs, d_table)
        for r, n, t in zip(rows, new, want):
            lens[r] = lens[r] if t < 0 else n
        gone = [r for r in rows if rng.random() < 0.4]
        if gone:
            first = [rng.choice([0, 0, lens[r] // 2, 7]) for r in gone]
            last = [lens[r] for r in gone]
            release(refs, table, first, last, gone)
            c.release_pages(d_refs, d_table, i32(first), i32(last), slot_ids=i32(gone))
            same(refs, table, d_refs, d_table)
            for r, f in zip(gone, first):   # what a sequence kept it keeps until it is gone whole
                release(refs, table, [0], [lens[r]], [r])
            c.release_pages(d_refs, d_table, i32([0] * len(gone)), i32(last), slot_ids=i32(gone))
            same(refs, table, d_refs, d_table)
            for r in gone:
                lens[r] = 0
    ok(c)


def test_too_few_pages():
    c = pool(10, slots=4)
    refs, table = i32([0, 1] * 5), i32([[-1] * 6 for _ in range(5)])
    # 2, 0, 3, 1, 0 wanted, 5 free: the last that fits, then one that does not, one that wants none
    got = c.take_pages(refs, table, i32([0, 16, 0, 30, 5]), i32([32, 16, 48, 40, 5]))
    assert got.tolist() == [2, 0, 3, -1, 0]
    assert table.tolist() == [[0, 2] + [-1] * 4, [-1] * 6, [4, 6, 8] + [-1] * 3, [-1] * 6, [-1] * 6]
    assert refs.tolist() == [1] * 10
    # one that does not fit keeps those behind it waiting, too, except where they want nothing
    c.release_pages(refs, table, i32([0]), i32([32]))
    got = c.take_pages(refs, table, i32([0, 0, 48]), i32([48, 16, 48]))
    assert got.tolist() == [-1, -1, 0] and int((refs == 0).sum()) == 2
    ok(c)


def test_refused_sequences():
    c = pool(20, slots=4)
    refs, table = i32([0] * 20), i32([[-1] * 3 for _ in range(6)])
    cases = [  # rows, lens, new, taken, detail
        ([0, 6, 1], [0, 0, 0], [16, 16, 16], [1, -1, 1], s4.S4KV_DEV_BAD_SLOT),
        ([2, -1], [0, 0], [16, 16], [1, -1], s4.S4KV_DEV_BAD_SLOT),
        ([3, 4, 3], [0, 0, 0], [16, 16, 32], [-1, 1, -1], s4.S4KV_DEV_BAD_SLOT),   # a row named twice
        ([5, 3], [20, 0], [19, 16], [-1, 1], s4.S4KV_DEV_BAD_LENGTH),
        ([5], [-16], [16], [-1], s4.S4KV_DEV_BAD_LENGTH),
        ([5], [0], [49], [-1], s4.S4KV_DEV_BAD_TABLE),
        ([5], [0], [2 ** 31 - 1], [-1], s4.S4KV_DEV_BAD_TABLE),
    ]
    taken = 0
    for rows, lens, new, want, detail in cases:
        before = table.clone()
        got = c.take_pages(refs, table, i32(lens), i32(new), slot_ids=i32(rows))
        assert got.tolist() == want, rows
        taken += sum(x for x in want if x > 0)
        assert c.status() == (s4.S4KV_ERR_DEVICE, detail)
        assert int(refs.sum()) == taken and int((table >= 0).sum()) == taken
        bad = [r for r, w in zip(rows, want) if w < 0 and 0 <= r < 6]
        assert torch.equal(table[bad], before[bad])


def test_refused_releases():
    c = pool(8, slots=4)
    refs, table = i32([1, 1, 2, 0, 0, 0, 0, 0]), i32([[0, 1, 2], [2, 9, 3], [-7, -1, -1]])
    c.release_pages(refs, table, i32([0, 0]), i32([48, 48]), slot_ids=i32([0, 1]))
    assert c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_PAGE)   # page 9, and page 3 that nobody holds
    assert refs.tolist() == [0] * 8 and table.tolist() == [[-1] * 3, [-1] * 3, [-7, -1, -1]]
    for rows, first, last, detail in (([3], [0], [16], s4.S4KV_DEV_BAD_SLOT), ([-1], [0], [16], s4.S4KV_DEV_BAD_SLOT),
                                      ([2], [-1], [16], s4.S4KV_DEV_BAD_LENGTH), ([2], [0], [49], s4.S4KV_DEV_BAD_TABLE),
                                      ([2], [0], [1], s4.S4KV_DEV_BAD_PAGE)):
        c.release_pages(refs, table, i32(first), i32(last), slot_ids=i32(rows))
        assert c.status() == (s4.S4KV_ERR_DEVICE, detail)
        assert refs.tolist() == [0] * 8
    # a row named twice gives its pages back once; an empty range and one that ends before it starts do nothing
    refs, table = i32([1, 1, 1, 0, 0, 0, 0, 0]), i32([[0, 1, 2]])
    c.release_pages(refs, table, i32([0, 0, 16, 40]), i32([32, 32, 16, 8]), slot_ids=i32([0, 0, 0, 0]))
    assert refs.tolist() == [0, 0, 1, 0, 0, 0, 0, 0] and table.tolist() == [[-1, -1, 2]]
    ok(c)


# ---- forks ------------------------------------------------------------------------------------


def done_of(bits, n, R):
    return n // 16 if bits in (8, INT8) else min(n // 32 * 32, max(0, n - R)) // 16


class Fork:
    """Sequences in the first slots, pages taken on the device, free slots behind them."""

    def __init__(self, lens, kids, bits, dtype="bf16", R=32, H=2, layers=2, seed=0, spare=600, width=None):
        self.lens, self.bits, self.R, self.H, self.layers = list(lens), bits, R, H, layers
        self.dt = torch.bfloat16 if dtype == "bf16" else torch.float16
        slots = len(lens) + kids
        self.n_pages = sum(up(n) for n in lens) + spare
        self.c = s4.KVCache(layers, self.n_pages, H, R, slots, dtype, bits=bits)
        self.c.pool[self.c.layout.layer_offset:].fill_(0x5a)   # what no call wrote is not zero
        rng = random.Random(seed)
        self.refs = i32([rng.choice([0, 0, 3]) if spare >= 600 else 0 for _ in range(self.n_pages)])
        self.table = torch.full((slots, width or max(up(n) for n in lens) + 8), -1, dtype=torch.int32, device=DEV)
        self.seq = i32(self.lens)
        zeros = i32([0] * len(lens))
        assert (self.c.take_pages(self.refs, self.table, zeros, self.seq) >= 0).all()
        self.rows = []
        for layer in range(layers):
            kv = [inp.kv_rows(inp.mix_seed(seed, layer, b), n, H, 128, self.dt) for b, n in enumerate(lens)]
            self.rows.append(kv)
            cu = [0]
            for n in lens:
                cu.append(cu[-1] + n)
            k, v = (torch.cat([x[i] for x in kv]).to(DEV) for i in (0, 1))
            self.c.append(layer, k, v, i32(cu), zeros, self.table)

    def restored(self, layer, slot, n):
        return self.c.gather(layer, self.table[slot:slot + 1].contiguous(), i32([n]), i32([0, n]), n, slot_ids=i32([slot]))


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (2, "fp16"), (8, "bf16"), (INT8, "fp16")])
@pytest.mark.parametrize("R", [1, 20, 128])
def test_a_fork_is_the_same_sequence(bits, dtype, R):
    lens = [1, 15, 16, 31, 33, 64, 100, 161, 300]
    f = Fork(lens, 2 * len(lens), bits, dtype, R, seed=R)
    refs, table = f.refs.tolist(), f.table.tolist()
    src = [b for b in range(len(lens)) for _ in range(2)]
    dst = list(range(len(lens), 3 * len(lens)))
    random.Random(1).shuffle(dst)
    n = [lens[b] for b in src]
    want = take(refs, table, [16 * done_of(bits, x, R) for x in n], n, dst)
    for s, d, x in zip(src, dst, n):
        for e in range(done_of(bits, x, R)):
            table[d][e] = table[s][e]
            refs[table[s][e]] += 1
    got = f.c.fork(f.refs, f.table, i32(src), i32(dst), i32(n))
    assert got.tolist() == want
    same(refs, table, f.refs, f.table)
    for layer in range(f.layers):
        for s, d, x in zip(src, dst, n):
            for a, b in zip(f.restored(layer, s, x), f.restored(layer, d, x)):
                assert torch.equal(a, b)
    ok(f.c)
    # all of them go on by other tokens (through pages, groups and rings): each as if it were alone
    more = 70
    slots = list(range(3 * len(lens)))
    length = lens + [0] * len(dst)
    owner = list(range(len(lens))) + [0] * len(dst)
    for s, d in zip(src, dst):
        length[d], owner[d] = lens[s], s
    grown = [x + more for x in length]
    assert (f.c.take_pages(f.refs, f.table, i32(length), i32(grown)) >= 0).all()
    cu = i32([more * i for i in range(len(slots) + 1)])
    new = [[inp.kv_rows(inp.mix_seed(77, layer, i), more, f.H, 128, f.dt) for i in slots] for layer in range(f.layers)]
    for layer in range(f.layers):
        k, v = (torch.cat([x[i] for x in new[layer]]).to(DEV) for i in (0, 1))
        f.c.append(layer, k, v, cu, i32(length), f.table)
    alone = s4.KVCache(1, 64, f.H, R, 1, dtype, bits=bits)
    for layer in range(f.layers):
        for i in slots:
            k, v = (torch.cat([f.rows[layer][owner[i]][j], new[layer][i][j]]).to(DEV) for j in (0, 1))
            bt = torch.arange(64, dtype=torch.int32, device=DEV)[None]
            alone.append(0, k, v, i32([0, grown[i]]), i32([0]), bt)
            want = alone.gather(0, bt, i32([grown[i]]), i32([0, grown[i]]), grown[i])
            for a, b in zip(f.restored(layer, i, grown[i]), want):
                assert torch.equal(a, b), (layer, i)
    ok(f.c)
    # and all of them leave
    taken = f.refs.clone()
    f.c.release_pages(f.refs, f.table, i32([0] * len(slots)), i32(grown))
    assert (f.table == -1).all()
    assert set(f.refs.tolist()) <= {0, 3} and (taken >= f.refs).all()
    ok(f.c)


def test_forks_without_room_and_forks_refused():
    f = Fork([100, 40, 0], 6, 4, R=32, layers=3, spare=9)
    # 100 tokens: 4 pages done, 3 to take; 40 tokens: none done, 3 to take
    table, refs = f.table.clone(), f.refs.clone()
    got = f.c.fork(f.refs, f.table, i32([0, 1, 0, 0, 2]), i32([3, 4, 5, 6, 7]), i32([100, 40, 100, 100, 0]))
    assert got.tolist() == [3, 3, 3, -1, 0]
    assert torch.equal(f.table[6], table[6]) and not (f.refs == 0).any()
    assert f.c.status() == (0, 0)
    for a, b in zip(f.restored(2, 0, 100), f.restored(2, 5, 100)):
        assert torch.equal(a, b)
    before = f.c.pool.clone()
    table, refs = f.table.clone(), f.refs.clone()
    for src, dst, n, detail in (([0, 0], [6, 6], [100, 100], s4.S4KV_DEV_BAD_SLOT), ([0], [0], [100], s4.S4KV_DEV_BAD_SLOT),
                                ([0, 1], [1, 0], [100, 40], s4.S4KV_DEV_BAD_SLOT), ([0], [9], [100], s4.S4KV_DEV_BAD_SLOT),
                                ([-1], [6], [100], s4.S4KV_DEV_BAD_SLOT), ([0], [6], [99], s4.S4KV_DEV_BAD_LENGTH),
                                ([0], [6], [-1], s4.S4KV_DEV_BAD_LENGTH)):
        assert f.c.fork(f.refs, f.table, i32(src), i32(dst), i32(n)).tolist() == [-1] * len(src)
        assert f.c.status() == (s4.S4KV_ERR_DEVICE, detail)
        assert torch.equal(f.table, table) and torch.equal(f.refs, refs)
    at = f.c.layout.lens_offset
    assert torch.equal(f.c.pool[at:], before[at:])
    # a layer that holds another length
    lens = f.c.pool[at:at + 4 * 3 * 9 * 2].view(torch.int32).view(3, 9, 2)
    lens[2, 1, 1] = 41
    assert f.c.fork(f.refs, f.table, i32([1]), i32([6]), i32([40])).tolist() == [-1]
    assert f.c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_LENGTH)
    # a table too narrow
    narrow = f.table[:, :6].contiguous()
    assert f.c.fork(f.refs, narrow, i32([0]), i32([6]), i32([100])).tolist() == [-1]
    assert f.c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_TABLE)


def test_forks_behind_a_window():
    # pages between the sinks' block (32 tokens) and the window given away: the fork has the same holes
    f = Fork([400], 1, 4, R=32)
    f.c.release_pages(f.refs, f.table, i32([32]), i32([160]), slot_ids=i32([0]))
    assert f.c.fork(f.refs, f.table, i32([0]), i32([1]), i32([400])).tolist() == [up(400) - done_of(4, 400, 32)]
    assert f.table[1, 2:10].tolist() == [-1] * 8 and torch.equal(f.table[1, :2], f.table[0, :2])
    q = inp.queries(3, 1, 4, 128, f.dt).to(DEV).view(1, 1, 4, 128)
    a, b = (f.c.window(0, q, f.table[i:i + 1].contiguous(), i32([400]), 400, 200, 4, slot_ids=i32([i])) for i in (0, 1))
    assert torch.equal(a, b)
    ok(f.c)


@pytest.mark.parametrize("bits", [4, INT8])
def test_a_captured_step_takes_its_own_pages(bits):
    """take, append, attend and fork captured once and replayed: pages, tables and outputs as eager
    calls leave them."""
    def make():
        return Fork([45, 80, 31], 1, bits, R=20, layers=1, seed=5)
    g = inp.gen(9)
    steps = 20
    k, v = (torch.randn(steps, 3, 2, 128, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    q = torch.randn(steps, 3, 1, 4, 128, generator=g).to(torch.bfloat16).to(DEV)
    scores = s4.Scores(cap=30.0)

    def run(f, graph):
        lens, new, cu = f.seq.clone(), f.seq + 1, i32([0, 1, 2, 3])
        kk, vv, qq = k[0].clone(), v[0].clone(), q[0].clone()
        taken = torch.empty(3, dtype=torch.int32, device=DEV)
        out = torch.empty(3, 1, 4, 128, device=DEV)
        src, dst, forked = i32([1]), i32([3]), torch.empty(1, dtype=torch.int32, device=DEV)
        bt = f.table[:3]

        def step():
            f.c.take_pages(f.refs, f.table, lens, new, taken=taken)
            f.c.append(0, kk, vv, cu, lens, bt)
            f.c.attend(0, qq, bt, new, 128, scores, out=out)
            f.c.release_pages(f.refs, f.table, i0, fork_len, slot_ids=dst)
            f.c.fork(f.refs, f.table, src, dst, new[1:2], taken=forked)
            fork_len.copy_(new[1:2])
            lens.add_(1)
            new.add_(1)
        i0, fork_len = i32([0]), i32([0])
        call = step
        if graph:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            keep = [x.clone() for x in (f.c.pool, f.refs, f.table)]
            with torch.cuda.stream(side):
                step()
            torch.cuda.current_stream().wait_stream(side)
            for x, y in zip((f.c.pool, f.refs, f.table), keep):
                x.copy_(y)
            lens.copy_(f.seq), new.copy_(f.seq + 1), fork_len.zero_()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                step()
            for x, y in zip((f.c.pool, f.refs, f.table), keep):
                x.copy_(y)
            lens.copy_(f.seq), new.copy_(f.seq + 1), fork_len.zero_()
            call = gr.replay
        outs = []
        for i in range(steps):
            kk.copy_(k[i]), vv.copy_(v[i]), qq.copy_(q[i])
            call()
            outs.append(out.clone())
        n = int(new[1]) - 1
        ok(f.c)
        return torch.stack(outs), f.refs, f.table, *f.restored(0, 3, n), *f.restored(0, 1, n)
    a, b = run(make(), False), run(make(), True)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert torch.equal(a[3], a[5]) and torch.equal(a[4], a[6])
