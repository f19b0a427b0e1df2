"""Score attention and prompts on 8-bit float pages whose heads have scales of their own, against the plain model in 64 bits."""
import pytest
import torch

import int4_kivi_quantized_gb300 as s4
import test_gpu_attend
import test_gpu_prompt
from score_model import LOG2E, attention, compare

pytestmark = pytest.mark.gpu

# key and value scales of two heads; restored values from 2e-9 to beyond 65504
SCALES = [([0.02, 0.03], [0.01, 0.05]), ([1e-4, 200.0], [170.0, 3e-6]), ([2.0 ** -20, 1.0], [2.0 ** -24, 1000.0])]

CASES = [(0, "bf16"), (0, "fp16"), (1, "bf16"), (2, "bf16")]   # (rows of the others' sizes are no fp16 numbers)


def bound(q, K, V, P, seen, out, scale):
    """Codes are exact in f16, so that a score's error is that of its sum: 2^-19 of the size of what is added (128 terms in
    binary32, the scales' product), and a bf16 query's elements below 2^-20 of its largest, 2^-28 of the largest each.
    P is rounded to f16, 2^-11 (2^-25 of the largest below f16's normal range, for each token); exponentials and sums 2^-18."""
    H, g = K.shape[1], q.shape[1] // K.shape[1]
    rep = lambda x: x.double().abs().repeat_interleave(g, 1)  # noqa: E731
    qa, see = q.double().abs(), seen.to(q.device)
    S = torch.einsum("qhd,thd->qht", qa, rep(K))
    S = torch.where(see[:, None], S, torch.zeros_like(S)).amax(-1)
    lost = qa.amax(-1) * 2.0 ** -28 * rep(K).sum(-1).amax(0)
    dz = (S * 2.0 ** -19 + lost) * scale * LOG2E
    A = torch.einsum("qht,thd->qhd", P, rep(V))
    n, M = see.sum(-1)[:, None, None].double(), rep(V).amax((0, 2))[None, :, None]
    return (2.0 ** -11 + 2.0 ** -18 + 2 * (torch.exp2(dz)[..., None] - 1)) * A + n * 2.0 ** -25 * M + 2.0 ** -24 * out.abs()


def edit_for(scales):
    """Rows whose codes spread over the whole range of the format."""
    def edit(b, k, v):
        for x, s in ((k, scales[0]), (v, scales[1])):
            x *= torch.tensor([8.0 * y for y in s]).to(x.dtype)[None, :, None]
            x[::7, :, :9] *= 16.0   # up to and beyond the largest code
    return edit


@pytest.mark.parametrize("which,dtype", CASES)
@pytest.mark.parametrize("chunks", [[300, 77], [33, 2]])
def test_prompts(which, dtype, chunks):
    c = test_gpu_prompt.Call([300, 1500], chunks, bits=8, dtype=dtype, fp8_scales=SCALES[which], edit=edit_for(SCALES[which]), seed=61)
    # each head of keys at its own size: queries that bring the scores back to a few units
    c.q *= torch.tensor([1 / (16 * s) for s in SCALES[which][0]], device="cuda").to(c.q.dtype).repeat_interleave(4)[None, :, None]
    got = c.run()
    for b in range(2):
        K, V, _, _ = c.f.plain(b)
        q, pos, seen = c.q[c.at[b]:c.at[b + 1]], list(c.positions(b)), c.seen(b)
        want, P = attention(q, K, V, pos, seen)
        compare(got[c.at[b]:c.at[b + 1]], want, bound(q, K, V, P, seen, want, 128 ** -0.5), f"sequence {b}")
    c.f.ok()


@pytest.mark.parametrize("which,dtype", CASES)
@pytest.mark.parametrize("nq", [1, 4])
def test_newest_tokens(which, dtype, nq):
    c = test_gpu_attend.Call([300, 1500], nq=nq, bits=8, dtype=dtype, fp8_scales=SCALES[which], edit=edit_for(SCALES[which]), seed=62)
    c.q *= torch.tensor([1 / (16 * s) for s in SCALES[which][0]], device="cuda").to(c.q.dtype).repeat_interleave(4)[None, None, :, None]
    got = c.run()
    for b in range(2):
        K, V, _, _ = c.f.plain(b)
        pos = c.positions(b)
        seen = test_gpu_attend.seen_of(c.f.lens[b], pos)
        want, P = attention(c.q[b], K, V, pos, seen)
        compare(got[b], want, bound(c.q[b], K, V, P, seen, want, 128 ** -0.5), f"sequence {b}")
    c.f.ok()


def test_scales_in_a_capped_and_sloped_form():
    c = test_gpu_prompt.Call([300, 90], [120, 90], bits=8, fp8_scales=([0.05, 2.0], [0.5, 0.01]), cap=10.0, slopes=True, seed=63)
    c.check(c.run())
    d = test_gpu_attend.Call([300, 90], nq=3, bits=8, fp8_scales=([0.05, 2.0], [0.5, 0.01]), cap=10.0, slopes=True, seed=63)
    d.check(d.run())


def test_scales_of_another_layer():
    """Each layer has its own: the call reads those of its layer."""
    dev = "cuda"
    c = s4.KVCache(2, 8, 1, 32, 1, "bf16", bits=8)
    c.set_fp8_scales(0, [0.1], [0.5])
    c.set_fp8_scales(1, [0.4], [0.125])
    g = torch.Generator().manual_seed(3)
    k, v = (torch.randn(60, 1, 128, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    q = torch.randn(60, 4, 128, generator=g).to(torch.bfloat16).to(dev)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    bt = torch.arange(4, dtype=torch.int32, device=dev)[None]
    from plain_cache import fp8_rows
    from score_model import seen_of
    for layer, (ks, vs) in enumerate(((0.1, 0.5), (0.4, 0.125))):
        c.append(layer, k, v, i32([0, 60]), i32([0]), bt)
        K, V = fp8_rows(k, torch.tensor([ks])), fp8_rows(v, torch.tensor([vs]))
        seen = seen_of(60, range(60))
        want, P = attention(q, K, V, list(range(60)), seen)
        got = c.prompt(layer, q, i32([0, 60]), bt, i32([60]), 60)
        compare(got, want, bound(q, K, V, P, seen, want, 128 ** -0.5))
        assert c.status()[0] == 0
