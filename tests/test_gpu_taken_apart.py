"""Pages: results may not lie over what the call reads."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
from test_gpu_pages import Fork, i32, ok

pytestmark = pytest.mark.gpu


def test_results_may_not_overlap_what_is_read():
    f = Fork([40, 20, 5], 3, 4)
    c, refs, table = f.c, f.refs, f.table
    x = i32([40, 20, 5, 7, 41, 21, 6, 7])
    before = [t.clone() for t in (x, refs, table)]
    for call in (lambda: c.take_pages(refs, table, x[:3], x[4:7], taken=x[:3]),
                 lambda: c.take_pages(refs, table, x[:3], x[4:7], taken=x[2:5]),
                 lambda: c.take_pages(refs, table, x[:3], x[4:7], taken=x[5:8]),
                 lambda: c.take_pages(refs, table, x[:3], x[4:7], slot_ids=x[1:4], taken=x[1:4]),
                 lambda: c.fork(refs, table, x[:1], x[4:5], x[2:3], taken=x[:1]),
                 lambda: c.fork(refs, table, x[:1], x[4:5], x[2:3], taken=x[4:5]),
                 lambda: c.fork(refs, table, x[:1], x[4:5], x[2:3], taken=x[2:3])):
        with pytest.raises(s4.S4KVError) as e:
            call()
        assert e.value.code == s4.S4KV_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(before, (x, refs, table)))
    # side by side is fine
    y = i32([40, 20, 5, 41, 21, 6, 0, 0, 0])
    assert c.take_pages(refs, table, y[:3], y[3:6], taken=y[6:]).tolist() == [0, 0, 0]
    ok(c)
