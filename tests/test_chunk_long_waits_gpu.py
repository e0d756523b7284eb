"""Attention within a chunk: waits that last as long as a long document are not
taken for ones that nothing ends."""
import pytest
import torch

from tests import gpu_util as U
from tests.test_chunk_gpu import call, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,prefix", [(131072, 0), (131072 + 100, 0), (98304, 98304), (98304 + 77, 50000)])
def test_only_the_wait_that_nothing_ends_gives_up(n, prefix):
    """With the limit of the test hook (2^14 polls) and one copy of the first CTA left out: the value rows of the last
    steps, and the next piece, are waited for during a whole piece, about 1,000 steps, by the other CTAs as well.  Only
    rows of the first CTA may be missing."""
    O = U.lib()
    q, k, v, _ = inputs([n], 1, 1, seed=71)
    want = call(O, [n], q, k, v, prefix=[prefix])
    assert torch.isfinite(want[1]).all()
    O.oscar_test_arm_wait_timeout()
    out, lse = call(O, [n], q, k, v, prefix=[prefix])
    gone = torch.isnan(lse)
    pieces, sms = -(-n // 256), torch.cuda.get_device_properties(0).multi_processor_count
    assert 0 < int(gone.sum()) <= 256 * -(-pieces // sms)
    assert torch.equal(out[~gone], want[0][~gone]) and torch.equal(lse[~gone], want[1][~gone])
