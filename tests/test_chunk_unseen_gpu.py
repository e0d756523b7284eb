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
