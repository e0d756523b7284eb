"""Attention within a chunk of short and long documents together: each one gets
what it gets alone."""
import pytest
import torch

from tests import gpu_util as U
from tests.test_chunk_gpu import call, compare, cumulative, inputs, slopes_of

pytestmark = pytest.mark.gpu

MIXES = [[5, 40], [40, 5], [5] * 64 + [2048], [33, 32, 1, 0, 500, 16, 17, 129], [(7 * i) % 70 for i in range(300)],
         [1] * 900 + [300] + [20] * 100]


def alone(lens, q, k, v, prior, prefix=None, **kw):
    """(out, lse), a call a document."""
    out = torch.empty((sum(lens), *q.shape[1:]), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(out.shape[:2], device="cuda")
    cu = cumulative(lens)
    for i, n in enumerate(lens):
        r = slice(cu[i], cu[i] + n)
        if n:
            out[r], lse[r] = call(U.lib(), [n], q[r], k[r], v[r], None if prior is None else (prior[0][r], prior[1][r]),
                                  prefix=None if prefix is None else [prefix[i]], **kw)
    return out, lse


@pytest.mark.parametrize("cap,bias,prior", [(0.0, False, False), (0.0, False, True), (20.0, True, True)])
@pytest.mark.parametrize("gqa", [4, 5])
@pytest.mark.parametrize("lens", MIXES)
def test_documents_get_what_they_get_alone(lens, gqa, cap, bias, prior):
    """Equal bits, and both within the bounds."""
    O = U.lib()
    q, k, v, p = inputs(lens, 2, gqa, seed=len(lens), extra=3, layout="fused", prior=prior)
    kw = dict(cap=cap, slopes=slopes_of(2 * gqa) if bias else None, prefix=[n // 3 for n in lens])
    out, lse = call(O, lens, q, k, v, p, **kw)
    compare(lens, q, k, v, out, lse, prior=p, **kw)
    want = alone(lens, q, k, v, p, **kw)
    n = sum(lens)
    assert torch.equal(out[:n], want[0]) and torch.equal(lse[:n], want[1])


def test_merged_in_place_captured_and_queued():
    """Behind the kernel that makes its inputs, over its own prior rows, before a kernel that reads them."""
    O = U.lib()
    lens = [5] * 20 + [700] + [32] * 20
    n = sum(lens)
    q, k, v, p = inputs(lens, 2, 4, seed=7, prior=True)
    want = call(O, lens, q, k, v, p, cap=20.0)
    keep = p[0].clone(), p[1].clone()
    cfg = O.make_rotary_config(128)
    pos = torch.zeros(n, dtype=torch.int32, device="cuda")       # at position 0 a rotation copies
    qr, kr = torch.zeros_like(q), torch.zeros_like(k)
    seen, other = torch.zeros_like(p[0]), torch.zeros_like(k)
    stream = torch.cuda.Stream()

    def enqueue(s):
        O.oscar_rotary(cfg, pos, q, k, qr, kr, stream=s)
        O.oscar_chunk_attention(cumulative(lens), qr, kr, v, p[0], p[1], cap=20.0, prior_out=p[0], prior_lse=p[1], stream=s)
        O.oscar_rotary(cfg, pos, p[0], k, seen, other, stream=s)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        enqueue(None)
    for i in range(12):
        p[0].copy_(keep[0])
        p[1].copy_(keep[1])
        for t in (qr, kr, seen):
            t.zero_()
        torch.cuda.synchronize()
        if i % 2:
            graph.replay()
        else:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(1 << 20)
                enqueue(stream)
        torch.cuda.synchronize()
        assert torch.equal(p[0], want[0]) and torch.equal(p[1], want[1]) and torch.equal(seen, want[0])


def test_a_wait_that_gives_up_leaves_the_short_documents():
    O = U.lib()
    lens = [9] * 30 + [600, 300]
    q, k, v, _ = inputs(lens, 2, 4, seed=8)
    want = call(O, lens, q, k, v)
    O.oscar_test_arm_wait_timeout()
    out, lse = call(O, lens, q, k, v)
    gone = torch.isnan(lse)
    assert gone.any() and not gone[:270].any()
    assert torch.equal(out[~gone], want[0][~gone]) and torch.equal(lse[~gone], want[1][~gone])
    again = call(O, lens, q, k, v)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
