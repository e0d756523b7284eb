"""Group summaries and the choice of groups, exactly: everything up to the
order of the scores is whole numbers (see include/oscar.h), computed here in
Python integers and exact fractions of the stored parameters."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from oracle import oscar_oracle as OR
from tests import gpu_util as U
from tests import layout

pytestmark = pytest.mark.gpu

HU = OR.hadamard_unnormalised().astype(np.int64)


def make(lens, hkv, meta=32, seed=1, chunk=4096, index=True):
    gen = torch.Generator().manual_seed(seed)
    kv = [W.make_sequence_kv(n, hkv, W.LLAMA_RECIPE, gen) for n in lens]
    cache = U.lib().OscarCache(len(lens), hkv, max(lens) + 300, meta_bits=meta)
    live = [i for i, n in enumerate(lens) if n]
    U.append_all(cache, live, [kv[i][0] for i in live], [kv[i][1] for i in live], chunk=chunk)
    if index:
        cache.enable_index()
        cache.update_index(range(len(lens)))
    return cache


def rne(x):
    """Nearest whole number, ties to even, of an exact fraction."""
    return round(Fraction(x))


def summary(scale, zero, norm):
    """lo8, hi8, w_max, w_min of one group's float32 parameters."""
    lo = np.float32(zero)
    hi = (lo.astype(np.float64) + 3.0 * np.float64(scale)).astype(np.float32)
    top = max(float(np.abs(lo).max()), float(np.abs(hi).max()))
    e = -100
    if top > 0:
        e = max(-100, math.frexp(top)[1] - 8)
        while Fraction(127) * Fraction(2) ** e < Fraction(top):
            e += 1
    unit = Fraction(2) ** e
    lo8 = np.array([rne(Fraction(float(x)) / unit) for x in lo])
    hi8 = np.array([rne(Fraction(float(x)) / unit) for x in hi])
    w = [np.float32(np.float64(f(np.float32(norm))) * 2.0 ** e) for f in (np.max, np.min)]
    return lo8, hi8, float(w[0]), float(w[1])


def summaries(cache, arena, slot, head):
    h = U.gpu_head(cache, arena, slot, head)
    return [summary(h.keys.scale[g], h.keys.zero[g], h.keys.norm[g]) for g in range(h.num_groups)]


def query8(q):
    """q [heads, 128] float64 (bf16 values) -> whole numbers in +-127."""
    q = np.where(np.isfinite(q), q, 0.0)
    top = float(np.abs(q).max())
    e = max(-100, math.frexp(top)[1]) if top else -100
    a = np.array([[rne(Fraction(float(x)) * Fraction(2) ** (22 - e)) for x in row] for row in q], dtype=np.int64)
    b = a @ HU
    shift = 0
    while int(np.abs(b).max()) > 127 << shift:
        shift += 1
    return (b + ((1 << shift) >> 1)) >> shift


def choose(q8, groups, n, first, last):
    score = []
    for lo8, hi8, wmax, wmin in groups:
        s = max(int(np.maximum(x * lo8, x * hi8).sum()) for x in q8)
        score.append(Fraction(s) * Fraction(wmax if s >= 0 else wmin))
    ng = len(groups)
    order = sorted(range(ng), key=lambda g: (not (g < first or g >= ng - last), -score[g], g))[:n]
    return sorted(order) + [-1] * (n - len(order))


def index_arrays(cache):
    S, H, M = cache.max_batch, cache.num_kv_heads, -(-cache.max_seq_len // 128)
    raw = cache.index.cpu().numpy()
    codes = raw[:256 * S * H * M].view(np.int8).reshape(S, H, M, 32, 2, 4)
    w = raw[256 * S * H * M:264 * S * H * M].view("<f4").reshape(S, H, M, 2)
    return codes[..., 0, :].reshape(S, H, M, 128), codes[..., 1, :].reshape(S, H, M, 128), w


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("lens,hkv", [([128], 1), ([1000, 64, 2500], 2), ([1300], 3)])
def test_summaries(lens, hkv, meta):
    cache = make(lens, hkv, meta, seed=2)
    arena = U.read_arena(cache)
    lo, hi, w = index_arrays(cache)
    for i, n in enumerate(lens):
        for j in range(hkv):
            for g, (a, b, wmax, wmin) in enumerate(summaries(cache, arena, i, j) if n >= 128 else []):
                assert np.array_equal(lo[i, j, g], a) and np.array_equal(hi[i, j, g], b), (i, j, g)
                assert w[i, j, g, 0] == np.float32(wmax) and w[i, j, g, 1] == np.float32(wmin)


def run(cache, ids, q, n, first, last, out=None):
    hkv = cache.num_kv_heads
    if out is None:
        out = torch.full((len(ids) + 1, hkv, n), 77, dtype=torch.int32, device="cuda")
    cache.select_groups(ids, q, q.shape[1], out, first, last)
    torch.cuda.synchronize()
    assert torch.all(out[len(ids):] == 77)
    return out[:len(ids)].cpu().numpy()


def check(cache, ids, q, n, first=0, last=0):
    got = run(cache, ids, q, n, first, last)
    arena, qn, hkv = U.read_arena(cache), U.f64(q), cache.num_kv_heads
    gqa = q.shape[1] // hkv
    for i, s in enumerate(ids):
        for j in range(hkv):
            groups = summaries(cache, arena, s, j) if cache.length(s) >= 128 else []
            want = choose(query8(qn[i, gqa * j:gqa * (j + 1)]), groups, n, first, last)
            assert got[i, j].tolist() == want, (s, j)


@pytest.mark.parametrize("lens,hkv,hq,n,first,last,meta", [
    ([2048], 1, 1, 3, 0, 0, 32), ([2048], 1, 4, 3, 1, 1, 16), ([5000, 100, 640], 2, 6, 5, 1, 2, 32),
    ([1280, 0], 2, 16, 1, 0, 0, 32), ([1280], 1, 64, 4, 4, 0, 32), ([1281], 1, 5, 4, 0, 4, 32),
    ([700], 2, 4, 5, 0, 0, 32), ([700], 2, 4, 4, 2, 2, 32), ([700], 2, 4, 9, 3, 5, 16), ([9000], 1, 20, 33, 2, 3, 32),
])
def test_choice(lens, hkv, hq, n, first, last, meta):
    cache = make(lens, hkv, meta, seed=sum(lens) + hq)
    for seed in (1, 2):
        check(cache, list(range(len(lens)))[::-1], W.make_q(len(lens), hq, seed=seed).cuda(), n, first, last)


def _write_index(cache, lo, hi, w):
    """Overwrites the index of slot 0, head 0 (its layout is in the header)."""
    S, H, M = cache.max_batch, cache.num_kv_heads, -(-cache.max_seq_len // 128)
    ng = lo.shape[0]
    c = np.stack([lo.reshape(ng, 32, 4), hi.reshape(ng, 32, 4)], 2).astype(np.int8).reshape(-1)
    cache.index[:c.size] = torch.from_numpy(c.view(np.uint8).copy()).cuda()
    at = 256 * S * H * M
    cache.index[at:at + 8 * ng] = torch.from_numpy(np.ascontiguousarray(w, "<f4").view(np.uint8).reshape(-1).copy()).cuda()


@pytest.mark.parametrize("ng,n", [(1100, 1), (1100, 64), (1100, 600), (1100, 1099), (513, 512), (40, 7), (5003, 90)])
@pytest.mark.parametrize("kind", ["ties", "two levels", "spread", "wide", "negative"])
def test_selection_of_given_summaries(ng, n, kind):
    """Index contents made for the selection: equal scores everywhere, a few
    distinct ones, magnitudes over the whole float32 range, all below zero."""
    cache = U.lib().OscarCache(1, 1, 128 * ng)
    rng = np.random.default_rng(ng + n)
    g = torch.Generator().manual_seed(1)
    k = torch.randn((128 * ng, 1, 128), generator=g).bfloat16().cuda()
    cache.append([0], [0, 128 * ng], k, k)
    cache.enable_index()
    cache.update_index([0])
    lo = rng.integers(-127, 128, (ng, 128))
    hi = np.minimum(lo + rng.integers(0, 100, lo.shape), 127)
    w = np.abs(rng.standard_normal((ng, 2))).astype(np.float32)
    w[:, 0] = w.max(1)
    if kind in ("ties", "two levels"):
        lo[:], hi[:], w[:] = lo[0], hi[0], 1.0
        if kind == "two levels":
            w[rng.integers(0, 2, ng) == 1] = 2.0
    if kind == "wide":
        w = (w * 2.0 ** rng.integers(-120, 100, (ng, 1))).astype(np.float32)
        w[rng.integers(0, ng, ng // 10)] = 0.0
    if kind == "negative":
        hi = np.minimum(hi, 0)
        lo = np.minimum(lo, hi)
    _write_index(cache, lo, hi, w)
    q = W.make_q(1, 3, seed=5).cuda()
    if kind == "negative":      # a query whose rotation is not below zero anywhere: only channel 0 of the basis
        q[:] = 0
        q[:, :, 0] = 1.0
    q8 = query8(U.f64(q)[0])
    groups = [(lo[i], hi[i], float(w[i, 0]), float(w[i, 1])) for i in range(ng)]
    for first, last in ((0, 0), (1, 0)):
        assert run(cache, [0], q, n, first, last)[0, 0].tolist() == choose(q8, groups, n, first, last)


@pytest.mark.parametrize("ng,hq", [(9001, 3), (2600, 64), (12000, 64)])
def test_long_sequences(ng, hq):
    """Slices that turn their stages over, with one stage and with two."""
    cache = U.lib().OscarCache(1, 1, 128 * ng)
    k = torch.randn((128 * ng, 1, 128), device="cuda").bfloat16()
    cache.append([0], [0, 128 * ng], k, k)
    del k
    cache.enable_index()
    cache.update_index([0])
    rng = np.random.default_rng(ng)
    lo = rng.integers(-127, 128, (ng, 128))
    hi = np.minimum(lo + rng.integers(0, 100, lo.shape), 127)
    w = np.abs(rng.standard_normal((ng, 2))).astype(np.float32)
    _write_index(cache, lo, hi, w)
    q = W.make_q(1, hq, seed=5).cuda()
    q8 = query8(U.f64(q)[0])
    pos, neg = np.maximum(q8, 0), np.minimum(q8, 0)
    s = (pos @ hi.T + neg @ lo.T).max(0).astype(np.float64)      # whole numbers below 2^22
    score = s * np.where(s >= 0, w[:, 0], w[:, 1]).astype(np.float64)     # 22 x 24 bits: exact
    order = sorted(range(ng), key=lambda g: (-score[g], g))
    for n in (1, 100, ng - 1):
        assert run(cache, [0], q, n, 0, 0)[0, 0].tolist() == sorted(order[:n])


def test_a_sequence_too_long_is_refused():
    O = U.lib()
    cache = O.OscarCache(1, 1, 128 * 12001)
    k = torch.zeros((128 * 12001, 1, 128), dtype=torch.bfloat16, device="cuda")
    cache.append([0], [0, 128 * 12001], k, k)
    cache.enable_index()
    cache.update_index([0])
    out = torch.zeros((1, 1, 5), dtype=torch.int32, device="cuda")
    q = W.make_q(1, 1, seed=5).cuda()
    with pytest.raises(O.OscarError) as e:
        cache.select_groups([0], q, 1, out)
    assert e.value.status == O.OSCAR_ERR_UNSUPPORTED
    out = torch.zeros((1, 1, 12001), dtype=torch.int32, device="cuda")
    cache.select_groups([0], q, 1, out)                          # all of them: nothing to choose
    assert out[0, 0].tolist() == list(range(12001))


def test_queries_at_the_edges():
    """Zero, tiny, huge and non-finite queries choose what the definition says."""
    cache = make([1920], 2, seed=8)
    base = W.make_q(1, 4, seed=3).cuda()
    for f in (0.0, 1e-38, 1e-30, 1e30, 3e38):
        q = (base.float() / base.float().abs().max() * f).bfloat16()
        check(cache, [0], q, 4)
    q = base.clone()
    q[0, 0, 3], q[0, 1, 5], q[0, 2, 7] = float("nan"), float("inf"), -float("inf")
    check(cache, [0], q, 4)


def test_a_planted_group_is_found():
    """A key far along the query's direction puts its group in front."""
    gen = torch.Generator().manual_seed(4)
    k, v = W.make_sequence_kv(4096, 1, W.KVRecipe(), gen)
    q = W.make_q(1, 1, seed=6)
    k[128 * 19 + 5, 0] = (20 * q[0, 0].float() / q[0, 0].float().norm()).bfloat16()
    cache = U.lib().OscarCache(1, 1, 4096)
    U.append_all(cache, [0], [k], [v])
    cache.enable_index()
    cache.update_index([0])
    assert run(cache, [0], q.cuda(), 1, 0, 0)[0, 0].tolist() == [19]


def test_update_follows_appends_and_resets():
    """The index is refused while stale, brought up to date group by group, and
    the same as a rebuild."""
    O = U.lib()
    cache = make([500, 260], 2, seed=9)
    q = W.make_q(2, 4, seed=1).cuda()
    run(cache, [0, 1], q, 2, 0, 0)
    gen = torch.Generator().manual_seed(10)
    k, v = W.make_sequence_kv(200, 2, W.LLAMA_RECIPE, gen)
    cache.append([0], [0, 5], k[:5].cuda(), v[:5].cuda())     # no group closes
    run(cache, [0, 1], q, 2, 0, 0)
    cache.append([0], [0, 195], k[5:].contiguous().cuda(), v[5:].contiguous().cuda())
    with pytest.raises(O.OscarError, match="index"):
        run(cache, [0, 1], q, 2, 0, 0)
    run(cache, [1], q[:1], 2, 0, 0)
    cache.update_index([0, 1])
    check(cache, [0, 1], q, 2)
    def live():
        lo, hi, w = index_arrays(cache)
        return [x[i, :, :cache.length(i) // 128].copy() for i in (0, 1) for x in (lo, hi, w)]
    step = live()
    cache.index.fill_(0x55)
    cache.update_index([0, 1], rebuild=True)
    for a, b in zip(step, live()):
        assert np.array_equal(a, b)
    O.oscar_cache_reset(cache.handle, 0)
    cache.append([0], [0, 200], k.cuda(), v.cuda())
    with pytest.raises(O.OscarError, match="index"):
        run(cache, [0], q[:1], 2, 0, 0)
    cache.update_index([0])
    check(cache, [0], q[:1], 2)


def test_stream_graph_and_many_sequences():
    cache = make([640 + 128 * (i % 3) for i in range(40)], 1, seed=14)
    ids = list(range(40))
    q = W.make_q(40, 2, seed=2).cuda()
    check(cache, ids, q, 3, 1, 1)
    out = torch.zeros((40, 1, 3), dtype=torch.int32, device="cuda")
    want = run(cache, ids, q, 3, 1, 1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    cache.select_groups(ids, q, 2, out, 1, 1, stream=s)
    s.synchronize()
    assert np.array_equal(out.cpu().numpy(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.update_index(ids, rebuild=True)
        cache.select_groups(ids, q, 2, out, 1, 1)
    out.zero_()
    cache.index.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(out.cpu().numpy(), want)


def test_queries_in_page_locked_memory_and_a_single_group():
    cache = make([300, 128], 2, seed=21)
    q = W.make_q(2, 4, seed=3)
    want = run(cache, [0, 1], q.cuda(), 1, 0, 0)
    assert np.array_equal(run(cache, [0, 1], q.pin_memory(), 1, 0, 0), want)
    check(cache, [0, 1], q.cuda(), 1)


def test_an_imported_sequence_is_indexed_anew():
    O = U.lib()
    cache = make([1400, 1500], 2, seed=22)
    q = W.make_q(1, 4, seed=4).cuda()
    state = cache.export_sequence(1)
    cache.import_sequence(0, *state)
    with pytest.raises(O.OscarError, match="index"):
        run(cache, [0], q, 3, 0, 0)
    cache.update_index([0])
    check(cache, [0], q, 3)
    assert np.array_equal(run(cache, [0], q, 3, 0, 0), run(cache, [1], q, 3, 0, 0))


def test_two_streams_at_once():
    cache = make([128 * 150, 128 * 40], 2, seed=23)
    q = [W.make_q(2, 8, seed=30 + i).cuda() for i in range(2)]
    want = [run(cache, [0, 1], q[i], 7, 1, 1) for i in range(2)]
    outs = [torch.zeros((20, 2, 2, 7), dtype=torch.int32, device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(20):
        for i in range(2):
            cache.select_groups([0, 1], q[i], 8, outs[i][k], 1, 1, stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(np.array_equal(outs[i][k].cpu().numpy(), want[i]) for k in range(20))


def test_refusals():
    O = U.lib()
    cache = make([600, 0], 2, index=False)
    q = W.make_q(1, 4, seed=2).cuda()
    out = torch.zeros((1, 2, 3), dtype=torch.int32, device="cuda")

    def refused(fn, status=O.OSCAR_ERR_INVALID_ARG):
        with pytest.raises(O.OscarError) as e:
            fn()
        assert e.value.status == status
    refused(lambda: cache.select_groups([0], q, 4, out))          # no index
    refused(lambda: cache.update_index([0]))
    small = torch.empty(O.oscar_index_required_bytes(cache.handle) - 1, dtype=torch.uint8, device="cuda")
    refused(lambda: O.oscar_index_attach(cache.handle, small), O.OSCAR_ERR_CAPACITY)
    big = torch.empty(small.numel() + 256, dtype=torch.uint8, device="cuda")
    refused(lambda: O.oscar_index_attach(cache.handle, big[16:]))
    refused(lambda: O.oscar_index_attach(cache.handle, torch.empty(small.numel() + 1, dtype=torch.uint8)))
    cache.enable_index()
    refused(lambda: cache.select_groups([0], q, 4, out))          # not up to date
    cache.update_index([0, 1])
    refused(lambda: cache.update_index([0, 0]))
    refused(lambda: cache.update_index([2]))
    refused(lambda: cache.select_groups([2], q, 4, out))
    refused(lambda: cache.select_groups([0], q, 4, out, 2, 2))
    refused(lambda: cache.select_groups([0], q, 4, out, -1, 0))
    refused(lambda: cache.select_groups([0], q, 4, out.cpu()))
    refused(lambda: cache.select_groups([0], torch.zeros((1, 5, 128), dtype=torch.bfloat16, device="cuda"), 5, out))
    refused(lambda: cache.select_groups([0], torch.zeros((1, 130, 128), dtype=torch.bfloat16, device="cuda"), 130,
                                        out), O.OSCAR_ERR_UNSUPPORTED)
    refused(lambda: cache.select_groups([0], q, 4, out[..., :0].contiguous()))
    with pytest.raises(ValueError):
        cache.select_groups([0], q, 4, out[:, :1].contiguous())
    cache.select_groups([1], q, 4, out)
    assert torch.all(out == -1)
    O.oscar_index_attach(cache.handle, None)
    refused(lambda: cache.select_groups([0], q, 4, out))


@pytest.mark.parametrize("ng,hkv,n", [(64, 1, 16), (5000, 1, 90), (5003, 2, 64), (11900, 1, 30)])
def test_wait_that_runs_out(ng, hkv, n):
    """A copy left unissued (the library's own hook): the bounded wait gives
    up, the call reports it, later calls are unaffected.  Slices of one chunk,
    of three with two stages (the copy of the second is in flight when the wait
    for the first gives up), and of more."""
    O = U.lib()
    cache = O.OscarCache(1, hkv, 128 * ng + 128)
    blocks = torch.randint(0, 60, (hkv, ng, cache.block_bytes), dtype=torch.uint8, device="cuda")   # finite parameters
    cache.import_sequence(0, 128 * ng, blocks, None, torch.ones((2, hkv), device="cuda"))
    del blocks
    cache.enable_index()
    cache.update_index([0])
    q = W.make_q(1, 4 * hkv, seed=42).cuda()
    want, got = (torch.full((1, hkv, n), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    cache.select_groups([0], q, 4 * hkv, want, 1, 1)
    O.oscar_cache_check(cache.handle)
    assert torch.all(want >= 0) and torch.all(want[..., 1:] > want[..., :-1])
    O.oscar_test_arm_wait_timeout()
    cache.select_groups([0], q, 4 * hkv, got, 1, 1)
    with pytest.raises(O.OscarError) as e:
        O.oscar_cache_check(cache.handle)
    assert e.value.status == O.OSCAR_ERR_DEVICE_TIMEOUT
    O.oscar_cache_check(cache.handle)
    for _ in range(2):
        cache.select_groups([0], q, 4 * hkv, got, 1, 1)
    O.oscar_cache_check(cache.handle)
    assert torch.equal(got, want)


def test_enabling_the_index_again_keeps_its_memory():
    """Queued updates and selections may still use it: nothing is valid in it
    any more, but it is not handed out to others."""
    cache = make([1300], 2)
    q = W.make_q(1, 8, seed=45).cuda()
    want, got = (torch.empty((1, 2, 4), dtype=torch.int32, device="cuda") for _ in range(2))
    cache.select_groups([0], q, 8, want)
    at = cache.index.data_ptr()
    cache.enable_index()
    assert cache.index.data_ptr() == at
    with pytest.raises(U.lib().OscarError):
        cache.select_groups([0], q, 8, got)
    cache.update_index([0])
    cache.select_groups([0], q, 8, got)
    assert torch.equal(got, want)
