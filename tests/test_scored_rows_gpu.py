"""Prefill over the cache and decode under a score rule: a row's bits do not
depend on the queries beside it."""
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from tests import gpu_util as U
from tests.test_scored_gpu import slopes_of
from tests.test_sparse_gpu import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("loud", [0.01, 30.0, float("inf"), float("nan")])
@pytest.mark.parametrize("cap,bias", [(5.0, False), (30.0, True), (0.0, True)])
@pytest.mark.parametrize("L,hkv,hq,n_q,meta,split", [(1000, 2, 8, 40, 32, False), (77, 1, 3, 21, 32, False),
                                                     (4096 + 5, 1, 5, 33, 16, True)])
def test_prefill_rows_by_themselves(L, hkv, hq, n_q, meta, split, cap, bias, loud):
    O = U.lib()
    cache = make([L], hkv, meta, seed=20)
    gen = torch.Generator().manual_seed(21)
    q = torch.randn((n_q, hq, 128), generator=gen).bfloat16().cuda()
    slopes = slopes_of(hq).cuda() if bias else None
    ws = None
    if split:
        ws = torch.empty(O.oscar_prefill_workspace_bytes(cache.handle, 0, n_q, hq), dtype=torch.uint8, device="cuda")

    def call(x):
        out, lse = torch.empty_like(x), torch.empty((n_q, hq), device="cuda")
        cache.scored_prefill(0, x, hq, out, lse, ws, cap=cap, slopes=slopes)
        O.oscar_cache_check(cache.handle)
        return out, lse

    clean = call(q)
    other = torch.rand((n_q, hq), generator=gen).cuda() < 0.3
    out, lse = call(torch.where(other[..., None], (q.float() * loud).bfloat16(), q))
    assert torch.equal(out[~other], clean[0][~other]) and torch.equal(lse[~other], clean[1][~other])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("cap,bias", [(5.0, False), (30.0, True)])
@pytest.mark.parametrize("hkv,hq", [(2, 8), (1, 5), (1, 13)])
def test_decode_rows_by_themselves(hkv, hq, cap, bias, dtype):
    O = U.lib()
    cache = make([3000, 77], hkv, 32, seed=22)
    q = W.make_q(2, hq, seed=23).cuda()
    slopes = slopes_of(hq).cuda() if bias else None
    ws = cache.workspace(2, hq)

    def call(x):
        out = torch.empty((2, hq, 128), dtype=dtype, device="cuda")
        cache.scored_decode([0, 1], x, hq, out, ws, cap=cap, slopes=slopes)
        O.oscar_cache_check(cache.handle)
        return out

    clean = call(q)
    for loud in (0.01, 30.0, float("inf"), float("nan")):
        other = torch.zeros((2, hq), dtype=torch.bool, device="cuda")
        other[0, 1::3] = True
        other[1, ::2] = True
        out = call(torch.where(other[..., None], (q.float() * loud).bfloat16(), q))
        assert torch.equal(out[~other], clean[~other]), loud
