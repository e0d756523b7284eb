"""Attention within a chunk: several documents in several rounds of pieces, in
sorted order (as many tiles as either launch holds) and without it."""
import pytest
import torch

from tests import gpu_util as U
from tests.test_chunk_gpu import call, compare, inputs
from tests.test_chunk_mixed_gpu import alone

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cap,prior", [(0.0, False), (20.0, True)])
@pytest.mark.parametrize("lens,hkv,gqa", [
    ([2500, 40, 1800, 2500, 700, 2049], 1, 16),              # 603 tiles of 256 rows, 6 documents
    ([1000, 2047, 33] * 5 + [129], 2, 8),                    # 495 tiles a KV head, 16 documents
    ([34 + 61 * i for i in range(40)], 1, 13),               # 2,505 tiles, 40 documents
    ([3333, 64, 2222, 1, 3001, 999, 2, 2500], 1, 48),        # 2,274 tiles, 8 documents, two of them short
])
def test_several_rounds(lens, hkv, gqa, cap, prior):
    O = U.lib()
    q, k, v, p = inputs(lens, hkv, gqa, seed=len(lens), extra=2, prior=prior)
    out, lse = call(O, lens, q, k, v, p, cap=cap)
    want = alone(lens, q, k, v, p, cap=cap)
    n = sum(lens)
    assert torch.equal(out[:n], want[0]) and torch.equal(lse[:n], want[1])
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)
    # the shortest tiled document against the definition
    i = min((m, j) for j, m in enumerate(lens) if m > 32)[1]
    r = slice(sum(lens[:i]), sum(lens[:i + 1]))
    compare([lens[i]], q[r], k[r], v[r], out[r], lse[r], None if p is None else (p[0][r], p[1][r]), cap=cap)
