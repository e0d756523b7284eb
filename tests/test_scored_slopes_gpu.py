"""Decode and prefill over the cache with scores far from zero: slopes over the
whole range that a call takes, and loud queries."""
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from tests import gpu_util as U
from tests.test_scored_gpu import check_decode
from tests.test_sparse_gpu import make

pytestmark = pytest.mark.gpu

STEEP = [2.0 ** 59, 1.5 * 2.0 ** 40, 2.0 ** 30, 1000.0]


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("lens", [[1500, 77], [1024, 129]])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_steep_slopes(lens, sign, cap, dtype, meta):
    """All weight on the newest token, or on the first one: what the cache reads back for it."""
    O = U.lib()
    cache = make(lens, 2, meta, seed=30)
    slopes = sign * torch.tensor(STEEP + STEEP)
    out = check_decode(cache, [0, 1], W.make_q(2, 8, seed=31).cuda(), cap, slopes, dtype)
    for i, n in enumerate(lens):
        at = n - 1 if sign > 0 else 0
        k, v = (torch.empty((1, 2, 128), device="cuda") for _ in range(2))
        cache.read([i], [at], [at + 1], k, v)
        O.oscar_cache_check(cache.handle)
        want = v[0].repeat_interleave(4, 0)
        # value factors in float16 (2^-11 of the largest scale times 3), outputs in bf16; next to nothing in float32
        tol = 2.0 ** -8 * want.abs() + 2.0 ** -8 * want.abs().max() if dtype == torch.bfloat16 else 2.0 ** -16 * want.abs().max()
        assert ((out[i].float() - want).abs() <= tol).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("L,split", [(1500, False), (4101, True), (77, False)])
def test_prefill_steep_slopes(L, split, sign, cap):
    O = U.lib()
    cache = make([L], 2, 32, seed=32)
    q = W.make_q(21, 8, seed=33).cuda()
    out, lse = torch.empty_like(q), torch.empty((21, 8), device="cuda")
    ws = None
    if split:
        ws = torch.empty(O.oscar_prefill_workspace_bytes(cache.handle, 0, 21, 8), dtype=torch.uint8, device="cuda")
    slopes = (sign * torch.tensor(STEEP + STEEP)).cuda()
    cache.scored_prefill(0, q, 8, out, lse, ws, cap=cap, slopes=slopes)
    O.oscar_cache_check(cache.handle)
    at = L - 1 if sign > 0 else 0
    k, v = (torch.empty((1, 2, 128), device="cuda") for _ in range(2))
    cache.read([0], [at], [at + 1], k, v)
    torch.cuda.synchronize()
    want = v[0].repeat_interleave(4, 0)[None]
    assert ((out.float() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -12 * want.abs().max()).all()
    far = L + torch.arange(21, device="cuda")[:, None] - at
    top = -slopes[None].double() * far
    # scores here: at most sqrt(128) 2^9 (queries of a few units along keys of a few tens)
    assert ((lse.double() - top).abs() <= 2.0 ** 13 + 2.0 ** -21 * top.abs()).all()


@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 24, 2.0 ** 40])
def test_loud_queries_over_the_cache(size):
    """Scores of 2^12 to 2^45: finite rows, with and without slopes."""
    O = U.lib()
    cache = make([1500, 77], 2, 32, seed=34)
    q = (W.make_q(2, 8, seed=35).float() * size).bfloat16().cuda()
    for slopes in (None, torch.tensor(STEEP[1:] + [0.0] + STEEP[1:] + [-1.0])):
        for dtype in (torch.bfloat16, torch.float32):
            assert torch.isfinite(check_decode(cache, [0, 1], q, 0.0, slopes, dtype).float()).all()
    out, lse = torch.empty_like(q), torch.empty((2, 8), device="cuda")
    cache.scored_prefill(0, q, 8, out, lse, slopes=torch.ones(8, device="cuda"))
    O.oscar_cache_check(cache.handle)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    O.oscar_prefill_attention(cache.handle, 0, q, 8, 0.0, out, lse)
    O.oscar_cache_check(cache.handle)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
