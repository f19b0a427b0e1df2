"""Pages, prompts, forks and score forms together, as a scheduler uses them: the outputs are bit for
bit those of a second cache whose sequences share nothing and never give a page back."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import s4kv_inputs as inp
from plain_cache import INT8

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, HQ, SLOTS, WIDTH = 2, 8, 5, 20


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


class Program:
    """A cache with its table and lengths. shared: pages come from the device and forks share them;
    otherwise slot s has pages WIDTH s .. WIDTH s + WIDTH - 1 and a fork appends the tokens again."""

    def __init__(self, shared, bits, dtype):
        self.shared, self.c = shared, s4.KVCache(1, SLOTS * WIDTH, H, 40, SLOTS, dtype, bits=bits)
        if bits == 8:
            self.c.set_fp8_scales(0, [0.02, 0.03], [0.01, 0.05])
        self.refs = torch.zeros(SLOTS * WIDTH, dtype=torch.int32, device=DEV)
        self.table = torch.full((SLOTS, WIDTH), -1, dtype=torch.int32, device=DEV)
        if not shared:
            self.table.copy_(torch.arange(SLOTS * WIDTH, dtype=torch.int32, device=DEV).view(SLOTS, WIDTH))
        self.lens, self.told = [0] * SLOTS, [[] for _ in range(SLOTS)]

    def append(self, slots, k, v, chunks):
        before = [self.lens[s] for s in slots]
        after = [a + m for a, m in zip(before, chunks)]
        if self.shared:
            assert (self.c.take_pages(self.refs, self.table, i32(before), i32(after), slot_ids=i32(slots)) >= 0).all()
        cu = [0]
        for m in chunks:
            cu.append(cu[-1] + m)
        self.c.append(0, k, v, i32(cu), i32(before), self.table[slots].contiguous(), slot_ids=i32(slots))
        for j, s in enumerate(slots):
            self.lens[s] = after[j]
            self.told[s].append((k[cu[j]:cu[j + 1]], v[cu[j]:cu[j + 1]]))
        return i32(cu), i32(after)

    def prompt(self, slots, k, v, q, chunks, **kw):
        cu, after = self.append(slots, k, v, chunks)
        return self.c.prompt(0, q, cu, self.table[slots].contiguous(), after, max(self.lens), slot_ids=i32(slots), **kw)

    def drafts(self, slots, k, v, q, **kw):
        _, after = self.append(slots, k, v, [q.shape[1]] * len(slots))
        return self.c.attend(0, q, self.table[slots].contiguous(), after, max(self.lens), slot_ids=i32(slots), **kw)

    def fork(self, src, dst):
        if self.shared:
            got = self.c.fork(self.refs, self.table, i32(src), i32(dst), i32([self.lens[s] for s in src]))
            assert (got >= 0).all()
            for s, d in zip(src, dst):
                self.lens[d] = self.lens[s]
            return
        for s, d in zip(src, dst):
            for k, v in list(self.told[s]):
                self.append([d], k, v, [k.shape[0]])

    def leave(self, slots):
        if self.shared:
            self.c.release_pages(self.refs, self.table, i32([0] * len(slots)), i32([self.lens[s] for s in slots]), slot_ids=i32(slots))
        for s in slots:
            self.lens[s], self.told[s] = 0, []


@pytest.mark.parametrize("bits,dtype", [(4, "bf16"), (2, "fp16"), (8, "bf16"), (INT8, "fp16")])
def test_a_scheduler_on_shared_pages(bits, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float16
    form = s4.Scores(15.0, torch.linspace(0.01, 0.1, HQ, device=DEV), 120, 4)

    def rows(seed, n):
        k, v = (x.to(DEV) for x in inp.kv_rows(seed, n, H, 128, dt))
        return k, v, inp.queries(seed + 50, n, HQ, 128, dt).to(DEV).view(n, HQ, 128)

    def run(shared):
        p, outs = Program(shared, bits, dtype), []
        outs.append(p.prompt([0, 1], *rows(1, 133), [100, 33], scores=form))
        outs.append(p.prompt([1, 0], *rows(2, 61), [1, 60], first=i32([0] * 10 + [90] * 51), prefix=i32([0, 50])))
        p.fork([0, 0, 1], [2, 4, 3])
        k, v, q = rows(3, 25)
        outs.append(p.drafts([4, 1, 2, 0, 3], k, v, q.view(5, 5, HQ, 128), scores=form, prefix=i32([20] * 5)))
        p.leave([0, 3])                       # the forks' shared pages stay
        p.fork([4], [3])                      # a fork of a fork, on pages given back
        outs.append(p.prompt([0, 3], *rows(4, 170), [130, 40], scores=form))
        for i in range(3):
            k, v, q = rows(5 + i, 5)
            outs.append(p.drafts([0, 1, 2, 3, 4], k, v, q.view(5, 1, HQ, 128), scores=form))
        p.leave([0, 1, 2, 3, 4])
        assert p.c.status()[0] == 0
        if shared:
            assert not p.refs.any() and (p.table == -1).all()
        return outs

    # (the second program's slots are told to start again by an append at length zero)
    for a, b in zip(run(True), run(False)):
        assert torch.isfinite(a).all() and torch.equal(a, b)
