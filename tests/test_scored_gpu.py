"""Decode and chunked prefill over the cache under a score rule, against the
rule in 64 bits on the GPU's own cache.

Bound, as for the decode over listed groups (see test_sparse_gpu): scores off by
d = 2^-16 max_t A_t + 2^-20 with A_t the absolute sum behind a score, and by the
rule's own cap 2^-21 and 2^-22 of the distance term; the cap only contracts
differences.  Outputs by (e^(2 d) - 1 + 2^-16) max|v|, the value factors (float16
for bf16 decodes: 3 (2^-11 + n 2^-31) of the largest value scale, else 3 n 2^-30
of it), and half a step of the output type."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from oracle import oscar_oracle as OR
from tests import gpu_util as U
from tests.test_sparse_gpu import make

pytestmark = pytest.mark.gpu


def slopes_of(hq, sign=1.0):
    return torch.tensor([sign * 2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)])


def under_rule(q, h, pos, cap, slopes, scale):
    """q [R, 128] at positions pos [R] over a head's cache: (o, lse, d, room) with slopes [R]."""
    sc = 1 / math.sqrt(128) if not scale else scale
    s = OR.decode_scores(q, h, sc)                                     # [T, R]
    a = [0.0]
    if h.num_groups:
        size = (h.keys.codes * np.abs(h.keys.scale.astype(np.float64))[:, None] +
                np.abs(h.keys.zero.astype(np.float64))[:, None]) * h.keys.norm.astype(np.float64)[..., None]
        a.append((size.reshape(-1, 128) @ np.abs(OR.canalized_rotation(q)).T).max() * sc)
    if h.window_k.shape[0]:
        a.append((np.abs(h.window_k) @ np.abs(q).T).max() * sc)
    d = 2.0 ** -16 * max(a) + 2.0 ** -20
    if cap:
        s = cap * np.tanh(s / cap)
        d += cap * 2.0 ** -21
    if slopes is not None:
        far = np.abs(pos[None, :] - np.arange(h.length)[:, None])
        s = s - slopes[None, :] * far
        d += np.abs(slopes).max() * far.max() * 2.0 ** -22
    m = s.max(0)
    e = np.exp(s - m)
    v = OR.decode_values(h)
    return (e / e.sum(0)).T @ v, m + np.log(e.sum(0)), d, (np.expm1(2 * d) + 2.0 ** -16) * np.abs(v).max()


def check_decode(cache, ids, q, cap=0.0, slopes=None, dtype=torch.bfloat16, scale=0.0):
    O = U.lib()
    n, hq, gqa = len(ids), q.shape[1], q.shape[1] // cache.num_kv_heads
    out = torch.full((n + 1, hq, 128), 7.0, dtype=dtype, device="cuda")
    cache.scored_decode(ids, q, hq, out, cache.workspace(n, hq), cap=cap,
                        slopes=None if slopes is None else slopes.cuda(), softmax_scale=scale)
    O.oscar_cache_check(cache.handle)
    assert torch.all(out[n:] == 7.0)
    arena, qn, go = U.read_arena(cache), U.f64(q), U.f64(out)
    half = torch.finfo(dtype).eps / 2
    for i, s in enumerate(ids):
        for j in range(cache.num_kv_heads):
            rows = slice(gqa * j, gqa * (j + 1))
            h = U.gpu_head(cache, arena, s, j)
            pos = np.full(gqa, cache.length(s) - 1)
            ref, _, d, room = under_rule(qn[i, rows], h, pos, cap, None if slopes is None else slopes.double().numpy()[rows], scale)
            if h.num_groups:
                top = float(h.values.scale.max())
                room += 3 * (2.0 ** -11 + h.length * 2.0 ** -31) * top if dtype == torch.bfloat16 else 3 * h.length * 2.0 ** -30 * top
            err = np.abs(go[i, rows] - ref)
            assert np.all(err <= room + half * (np.abs(ref) + room)), (i, j, err.max(), room)
    return out[:n]


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("cap,bias", [(30.0, False), (0.0, True), (5.0, True), (0.5, False)])
@pytest.mark.parametrize("lens,hkv,hq", [([1024], 1, 4), ([2100, 128, 77], 2, 2), ([6000, 300], 2, 16), ([4000], 1, 5),
                                         ([129, 1], 3, 9), ([2560], 2, 26), ([700] * 17, 1, 8)])
def test_decode(lens, hkv, hq, cap, bias, meta):
    cache = make(lens, hkv, meta, seed=hq)
    ids = list(range(len(lens)))[::-1]
    q = W.make_q(len(lens), hq, seed=3).cuda()
    slopes = slopes_of(hq) if bias else None
    check_decode(cache, ids, q, cap, slopes)
    check_decode(cache, ids, q, cap, slopes, torch.float32, scale=0.3)


def test_decode_slopes_of_both_signs():
    """Some heads prefer the far tokens, some have no slope."""
    cache = make([1500, 130], 2, 32, seed=5)
    slopes = slopes_of(8)
    slopes[::2] *= -1.0
    slopes[3] = 0.0
    check_decode(cache, [0, 1], W.make_q(2, 8, seed=4).cuda(), 20.0, slopes, torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_decode_without_a_rule_is_the_decode(dtype):
    O = U.lib()
    cache = make([900, 140], 2, 32, seed=6)
    q = W.make_q(2, 8, seed=5).cuda()
    a, b = (torch.empty((2, 8, 128), dtype=dtype, device="cuda") for _ in range(2))
    ws = cache.workspace(2, 8)
    cache.scored_decode([0, 1], q, 8, a, ws)
    (cache.decode if dtype == torch.bfloat16 else cache.decode_f32)([0, 1], q, 8, b, ws)
    O.oscar_cache_check(cache.handle)
    assert torch.equal(a, b)


def test_decode_of_infinite_scores_under_a_cap():
    """A key that gives an infinite score counts as one at the cap."""
    O = U.lib()
    cache = make([20], 1, 32, seed=7)
    k = torch.zeros((1, 1, 128), dtype=torch.bfloat16)
    k[0, 0, 0] = float("inf")
    v = torch.ones((1, 1, 128), dtype=torch.bfloat16)
    cache.append([0], [0, 1], k.cuda(), v.cuda())
    q = W.make_q(1, 2, seed=6)
    q[0, :, 1:] = 0.0
    q[0, 0, 0], q[0, 1, 0] = 2.0, -2.0
    out = torch.empty((1, 2, 128), device="cuda")
    cache.scored_decode([0], q.cuda(), 2, out, cache.workspace(1, 2), cap=4.0)
    O.oscar_cache_check(cache.handle)
    h = U.gpu_head(cache, U.read_arena(cache), 0, 0)
    for r, sign in ((0, 1.0), (1, -1.0)):
        s = 4.0 * np.tanh(np.append(h.window_k[:-1] @ U.f64(q)[0, r] / math.sqrt(128), sign * np.inf) / 4.0)
        p = np.exp(s - s.max())
        ref = (p / p.sum()) @ h.window_v
        assert np.abs(U.f64(out)[0, r] - ref).max() <= 2.0 ** -16 * np.abs(h.window_v).max()


def check_prefill(L, hkv, hq, n_q, cap, bias, meta=32, split=False, scale=0.0, seed=1):
    O = U.lib()
    cache = make([L], hkv, meta, seed=seed)
    gen = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((n_q, hq, 128), generator=gen).bfloat16()
    slopes = slopes_of(hq) if bias else None
    out = torch.empty((n_q, hq, 128), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((n_q, hq), device="cuda")
    ws = None
    if split:
        nb = O.oscar_prefill_workspace_bytes(cache.handle, 0, n_q, hq)
        assert nb > 0
        ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    cache.scored_prefill(0, q.cuda(), hq, out, lse, ws, cap=cap, slopes=None if slopes is None else slopes.cuda(),
                         softmax_scale=scale)
    O.oscar_cache_check(cache.handle)
    arena, gqa = U.read_arena(cache), hq // hkv
    for j in range(hkv):
        h = U.gpu_head(cache, arena, 0, j)
        rows = U.f64(q)[:, gqa * j:gqa * (j + 1)].reshape(-1, 128)
        pos = L + np.repeat(np.arange(n_q), gqa)
        sl = None if slopes is None else np.tile(slopes.double().numpy()[gqa * j:gqa * (j + 1)], n_q)
        ref, rl, d, room = under_rule(rows, h, pos, cap, sl, scale)
        got = U.f64(out)[:, gqa * j:gqa * (j + 1)].reshape(-1, 128)
        gl = U.f64(lse)[:, gqa * j:gqa * (j + 1)].reshape(-1)
        err = np.abs(got - ref)
        assert np.all(err <= room + 2.0 ** -8 * (np.abs(ref) + room)), (j, err.max(), room)
        assert np.all(np.abs(gl - rl) <= d + 2.0 ** -20 * (1 + np.abs(rl))), (j, np.abs(gl - rl).max(), d)


@pytest.mark.parametrize("cap,bias", [(30.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("L,hkv,hq,n_q,meta,split", [(1024, 1, 4, 40, 32, False), (77, 2, 2, 5, 32, False),
                                                     (2100, 2, 6, 70, 16, False), (4096 + 5, 1, 5, 33, 32, True),
                                                     (128, 1, 8, 1, 16, False)])
def test_prefill(L, hkv, hq, n_q, meta, split, cap, bias):
    check_prefill(L, hkv, hq, n_q, cap, bias, meta, split)
    check_prefill(L, hkv, hq, n_q, cap, bias, meta, split, scale=0.4, seed=2)


def test_prefill_without_a_rule_is_the_prefill():
    O = U.lib()
    cache = make([700], 2, 32, seed=8)
    q = W.make_q(30, 8, seed=9).cuda()
    a, b = torch.empty_like(q), torch.empty_like(q)
    la, lb = torch.empty((30, 8), device="cuda"), torch.empty((30, 8), device="cuda")
    cache.scored_prefill(0, q, 8, a, la)
    O.oscar_prefill_attention(cache.handle, 0, q, 8, 0.0, b, lb)
    O.oscar_cache_check(cache.handle)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_the_wait_s_test_hook_reaches_the_scored_decode():
    O = U.lib()
    cache = make([600], 1, 32, seed=10)
    q, out = W.make_q(1, 4, seed=1).cuda(), torch.empty((1, 4, 128), dtype=torch.bfloat16, device="cuda")
    ws = cache.workspace(1, 4)
    O.oscar_test_arm_wait_timeout()
    cache.scored_decode([0], q, 4, out, ws, cap=30.0)
    with pytest.raises(O.OscarError) as e:
        O.oscar_cache_check(cache.handle)
    assert e.value.status == O.OSCAR_ERR_DEVICE_TIMEOUT
    check_decode(cache, [0], q, 30.0)


def test_refusals():
    O = U.lib()
    cache = make([300], 2, 32, seed=11)
    q, out = W.make_q(1, 8, seed=1).cuda(), torch.full((1, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = cache.workspace(1, 8)
    bad = [dict(cap=-1.0), dict(cap=float("nan")), dict(cap=1e6), dict(slopes=torch.zeros(8)),
           dict(slopes=torch.zeros(7, device="cuda")), dict(slopes=torch.zeros(8, device="cuda", dtype=torch.float64)),
           dict(slopes=torch.zeros(16, device="cuda")[::2])]
    for kw in bad:
        with pytest.raises((O.OscarError, ValueError)):
            cache.scored_decode([0], q, 8, out, ws, **kw)
        with pytest.raises((O.OscarError, ValueError)):
            cache.scored_prefill(0, q, 8, out, **kw)
    with pytest.raises(ValueError):
        cache.scored_decode([0], q, 8, out.half(), ws, cap=10.0)
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)
