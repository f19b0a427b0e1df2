"""Pages: entries that name a page already."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from test_gpu_pages import i32, ok, pool

pytestmark = pytest.mark.gpu


def test_pages_are_not_taken_into_entries_that_name_one():
    c = pool(40, slots=8)
    refs = i32([0, 1, 1, 0] * 10)
    table = torch.full((6, 8), -1, dtype=torch.int32, device="cuda")
    table[1, 2], table[3, 0], table[4, 7], table[5, 3] = 1, 2, 5, -9
    was = table.clone()
    lens, new = i32([0, 20, 16, 0, 0, 40]), i32([33, 60, 64, 10, 112, 64])
    got = c.take_pages(refs, table, lens, new)
    # row 1 wants entries 2 and 3 (2 names page 1), 3 wants 0, 5 wants 3 (no entry is -9); 4's page lies behind what it wants
    assert got.tolist() == [3, -1, 3, -1, 7, -1]
    assert c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_TABLE)
    assert torch.equal(table[[1, 3, 5]], was[[1, 3, 5]])
    named = torch.cat([table[0, :3], table[2, 1:4], table[4, :7]]).tolist()
    assert len(set(named)) == 13 and all(p % 4 in (0, 3) for p in named) and named == sorted(named)
    assert int(refs.sum()) == 20 + 13 and all(int(refs[p]) == 1 for p in named)
    assert int(table[4, 7]) == 5 and (table[0, 3:] == -1).all() and int(table[2, 0]) == -1
    # once the entry is free they get theirs
    table[1, 2], table[3, 0], table[5, 3] = -1, -1, -1
    assert c.take_pages(refs, table, lens[[1, 3]].contiguous(), new[[1, 3]].contiguous(), slot_ids=i32([1, 3])).tolist() == [2, 1]
    ok(c)


@pytest.mark.parametrize("n,need", [(1, 2000), (700, 3), (4096, 2)])
def test_many_of_them(n, need):
    pages = n * need + 100
    c = pool(pages, slots=4)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    table = torch.full((n, need + 1), -1, dtype=torch.int32, device="cuda")
    held = [i for i in range(n) if i % 5 == 0]
    table[held, need - 1 if n > 1 else 1234] = 0
    refs[0] = len(held)
    got = c.take_pages(refs, table, i32([0] * n), i32([16 * need] * n)).tolist()
    assert got == [-1 if i % 5 == 0 else need for i in range(n)]
    assert c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_TABLE)
    good = [i for i in range(n) if i % 5]
    named = table[good][:, :need].flatten()
    assert named.unique().numel() == named.numel() == len(good) * need and int((refs == 1).sum()) == len(good) * need + (len(held) == 1)
    assert int((table[held] >= 0).sum()) == len(held)


def test_too_few_pages_count_as_before():
    """A sequence that is refused for an entry and one that finds too few pages in one call."""
    c = pool(8, slots=4)
    refs, table = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.full((4, 8), -1, dtype=torch.int32, device="cuda")
    table[0, 1] = 7
    refs[7] = 1
    # 2 (refused, its pages counted), 4, 2 of 7 free: the third finds one page too few
    assert c.take_pages(refs, table, i32([0, 0, 0, 5]), i32([32, 64, 32, 5])).tolist() == [-1, 4, -1, 0]
    assert c.status() == (s4.S4KV_ERR_DEVICE, s4.S4KV_DEV_BAD_TABLE)
    assert int(refs.sum()) == 5 and (table[2] == -1).all()
