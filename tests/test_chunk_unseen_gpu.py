"""Attention within a chunk: what a row does not see has no part in its bits, be
it hidden keys and values, other rows' queries or the other documents of the
call."""
import pytest
import torch

from tests import gpu_util as U
from tests.test_chunk_gpu import call, compare, inputs, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loud", [40.0, 3.0e38, float("inf"), float("nan")])
@pytest.mark.parametrize("gqa", [3, 4])
@pytest.mark.parametrize("cap,bias", [(5.0, False), (30.0, False), (30.0, True), (0.0, False)])
def test_hidden_tokens_under_a_cap(cap, bias, gqa, loud):
    """Later tokens, another document and the rows behind the last one, loud or not finite: the same bits."""
    O = U.lib()
    lens = [70, 150, 133]
    q, k, v, _ = inputs(lens, 2, gqa, seed=80, extra=40)
    kw = dict(cap=cap, slopes=slopes_of(2 * gqa) if bias else None)
    clean = call(O, lens, q, k, v, **kw)
    compare(lens, q, k, v, *clean, **kw)
    for name, rows in [("the rows behind the last document", slice(353, 393)), ("another document", slice(70, 220)),
                       ("later tokens", slice(60, 70)), ("a token's own query", slice(100, 101))]:
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        q2[rows] = (q2[rows].float() * loud).bfloat16()
        if name != "a token's own query":
            k2[rows] = (k2[rows].float() * loud).bfloat16()
            v2[rows] = loud
        out, lse = call(O, lens, q2, k2, v2, **kw)
        keep = torch.ones(353, dtype=torch.bool)
        keep[rows] = False
        assert torch.equal(out[:353][keep], clean[0][:353][keep]), name
        assert torch.equal(lse[:353][keep], clean[1][:353][keep]), name


@pytest.mark.parametrize("loud", [40.0, 3.0e38, float("inf"), float("nan")])
@pytest.mark.parametrize("gqa", [1, 3, 4])
@pytest.mark.parametrize("cap,prior", [(0.0, False), (0.0, True), (30.0, False)])
def test_hidden_tokens_of_short_documents(cap, prior, gqa, loud):
    """The same of documents of up to 32 tokens, 16 rows of which share their keys and values."""
    O = U.lib()
    lens = [11, 6, 32, 16]
    q, k, v, p = inputs(lens, 2, gqa, seed=81, extra=9, prior=prior)
    clean = call(O, lens, q, k, v, p, cap=cap)
    compare(lens, q, k, v, *clean, prior=p, cap=cap)
    for rows in (slice(65, 74), slice(11, 17), slice(9, 10), slice(5, 11), slice(20, 21), slice(30, 49), slice(56, 57)):
        k2, v2 = k.clone(), v.clone()
        k2[rows] = (k2[rows].float() * loud).bfloat16()
        v2[rows] = loud
        out, lse = call(O, lens, q, k2, v2, p, cap=cap)
        seen = torch.zeros(65, dtype=torch.bool)         # rows at or behind one of these tokens, in its document
        for a, n in ((0, 11), (11, 6), (17, 32), (49, 16)):
            first = max(a, rows.start)
            if first < min(a + n, rows.stop):
                seen[first:a + n] = True
        assert torch.equal(out[:65][~seen], clean[0][:65][~seen])
        assert torch.equal(lse[:65][~seen], clean[1][:65][~seen])


@pytest.mark.parametrize("n", [9, 16, 32])
def test_values_that_are_not_finite_in_several_tokens_of_a_short_document(n):
    """Rows that see some of them, in one channel each: the other channels keep their sums."""
    O = U.lib()
    q, k, v, _ = inputs([n, n], 2, 3, seed=82)
    for t in range(2, n, 3):
        v[t, t % 2, 5 * t % 128] = float("inf") if t % 2 else float("nan")
    out, lse = call(O, [n, n], q, k, v)
    compare([n, n], q, k, v, out, lse)
