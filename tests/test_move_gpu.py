"""Forks, cuts and compactions: the destination's bytes against the source's,
and what the other calls then see."""
import numpy as np
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from tests import gpu_util as U

pytestmark = pytest.mark.gpu


def make(lens, hkv, slots, meta=32, seed=1, room=300):
    gen = torch.Generator().manual_seed(seed)
    kv = [W.make_sequence_kv(n, hkv, W.LLAMA_RECIPE, gen) for n in lens]
    cache = U.lib().OscarCache(slots, hkv, max(lens) + room, meta_bits=meta)
    U.append_all(cache, list(range(len(lens))), [k for k, _ in kv], [v for _, v in kv], chunk=4096)
    return cache


def state(cache, slot):
    """(blocks [hkv, groups, bytes], window rows [hkv, 2, w, 128], maxima [2, hkv]) on the host."""
    n, blocks, window, maxima = cache.export_sequence(slot)
    torch.cuda.synchronize()
    return blocks.cpu(), window[:, :, :n % 128].cpu(), maxima.cpu()


def equal(a, b):
    return all(x.shape == y.shape and torch.equal(x.view(torch.uint8), y.view(torch.uint8))
               for x, y in zip((t.contiguous() for t in a), (t.contiguous() for t in b)))


def prefix(cache, slot, n):
    """What a fork of the first n tokens has to hold: blocks and maxima as they are, and the window."""
    have = cache.length(slot)
    blocks, window, maxima = state(cache, slot)
    g = n // 128
    if n % 128 and g < have // 128:
        k, v = (torch.empty((n % 128, cache.num_kv_heads, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        cache.read([slot], [128 * g], [n], k, v)
        torch.cuda.synchronize()
        rows = torch.stack([k, v], 1).permute(2, 1, 0, 3).cpu()
    else:
        rows = window[:, :, :n % 128] if g == have // 128 else window[:, :, :0]
    return blocks[:, :g], rows, maxima


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("lens,take,hkv", [
    ([1000], [1000], 1), ([1000], [900], 2), ([1000], [896], 2), ([1000], [1], 3), ([77], [77], 2), ([77], [40], 2),
    ([128], [128], 1), ([128], [127], 5), ([129], [128], 2), ([700, 3, 2000], [500, 3, 1999], 2), ([300], [0], 2)])
def test_fork(lens, take, hkv, meta):
    n = len(lens)
    cache = make(lens, hkv, 2 * n, meta)
    want = [prefix(cache, i, t) for i, t in enumerate(take)]
    before = [state(cache, i) for i in range(n)]
    dst = [n + i for i in range(n)]
    cache.fork(list(range(n)), dst, take)
    for d, t, w in zip(dst, take, want):
        assert cache.length(d) == t
        assert equal(state(cache, d), w)
    for i in range(n):
        assert equal(state(cache, i), before[i])


@pytest.mark.parametrize("meta", [32, 16])
def test_many_forks_of_one_sequence(meta):
    """Forks of different lengths of one source, beside forks of another, more than a small launch takes."""
    cache = make([1500, 390], 2, 62, meta)
    rng = np.random.default_rng(3)
    take = [int(x) for x in rng.integers(0, 1501, 40)] + [int(x) for x in rng.integers(0, 391, 20)]
    src, dst = [0] * 40 + [1] * 20, [int(x) for x in 2 + rng.permutation(60)]
    order = rng.permutation(60)
    want = [prefix(cache, s, t) for s, t in zip(src, take)]
    cache.fork([src[i] for i in order], [dst[i] for i in order], [take[i] for i in order])
    for d, t, w in zip(dst, take, want):
        assert cache.length(d) == t and equal(state(cache, d), w)


def test_as_many_forks_as_a_call_takes():
    cache = make([260, 100], 1, 1026, room=10)
    take = [(i * 37) % 261 for i in range(1024)]
    want = {t: prefix(cache, 0, t) for t in (0, 1, 100, 128, 200, 256, 260)}
    cache.fork([0] * 1024, list(range(2, 1026)), take)
    for i, t in enumerate(take):
        assert cache.length(2 + i) == t
        if t in want:
            assert equal(state(cache, 2 + i), want[t])


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("n", [1000, 999, 896, 850, 128, 127, 5, 0])
def test_truncate(n, meta):
    cache = make([1000, 400], 2, 2, meta)
    want, other = prefix(cache, 0, n), state(cache, 1)
    cache.truncate([0], [n])
    assert cache.length(0) == n and cache.length(1) == 400
    assert equal(state(cache, 0), want) and equal(state(cache, 1), other)


def kept(cache, slot, groups):
    blocks, window, maxima = state(cache, slot)
    return blocks[:, groups], window, maxima


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("how", ["none", "first", "last", "recent", "even", "all", "but one", "random"])
@pytest.mark.parametrize("lens,hkv", [([1000, 300], 2), ([128 * 300 + 77], 1), ([100, 128 * 7], 3)])
def test_keep_groups(lens, hkv, how, inplace, meta):
    n = len(lens)
    cache = make(lens, hkv, 2 * n, meta)
    rng = np.random.default_rng(4)
    lists = []
    for m in lens:
        ng = m // 128
        every = list(range(ng))
        lists.append({"none": [], "first": every[:1], "last": every[-1:], "recent": every[:2] + every[max(2, ng // 2):],
                      "even": every[::2], "all": every, "but one": every[:ng // 3] + every[ng // 3 + 1:],
                      "random": sorted(int(x) for x in rng.permutation(ng)[:ng // 2])}[how])
    want = [kept(cache, i, g) for i, g in enumerate(lists)]
    before = [state(cache, i) for i in range(n)]
    src = list(range(n))
    dst = None if inplace else [n + i for i in src]
    cache.keep_groups(src, lists, dst)
    for i in src:
        d = i if inplace else n + i
        assert cache.length(d) == 128 * len(lists[i]) + lens[i] % 128
        assert equal(state(cache, d), want[i])
        if not inplace:
            assert equal(state(cache, i), before[i])


@pytest.mark.parametrize("inplace", [False, True])
def test_keep_more_runs_than_a_launch_takes(inplace):
    lens = [128 * 5201, 128 * 900 + 5]
    cache = U.lib().OscarCache(4, 1, lens[0])
    for i, n in enumerate(lens):
        blocks = torch.randint(0, 256, (1, n // 128, cache.block_bytes), dtype=torch.uint8, device="cuda")
        window = torch.randn((1, 2, 128, 128), device="cuda").bfloat16()
        cache.import_sequence(i, n, blocks, window, torch.ones((2, 1), device="cuda"))
    lists = [list(range(1, 5201, 2)), list(range(0, 900, 3))]
    want = [kept(cache, i, g) for i, g in enumerate(lists)]
    cache.keep_groups([0, 1], lists, None if inplace else [2, 3])
    for i in range(2):
        assert equal(state(cache, i if inplace else 2 + i), want[i])


def test_pairs_in_place_and_not_in_one_call():
    cache = make([1000, 700, 500], 2, 5)
    lists = [[1, 3, 6], [0, 4], []]
    want = [kept(cache, i, g) for i, g in enumerate(lists)]
    cache.keep_groups([0, 1, 2], lists, [0, 4, 2])
    for slot, w in ((0, want[0]), (4, want[1]), (2, want[2])):
        assert equal(state(cache, slot), w)


def decoded(cache, slot, q, ws):
    out = torch.empty((1, q.shape[1], 128), device="cuda")
    cache.decode_f32([slot], q, q.shape[1], out, ws)
    return out


def test_a_fork_goes_on_like_its_source():
    """Appends, decodes, index and listed decodes of a fork give the bits that the source gives."""
    O = U.lib()
    cache = make([900], 2, 2, seed=5)
    cache.enable_index()
    cache.update_index([0])
    cache.fork([0], [1])
    gen = torch.Generator().manual_seed(6)
    ws, q = cache.workspace(2, 8), W.make_q(2, 8, seed=7).cuda()
    q[1] = q[0]
    with pytest.raises(O.OscarError):           # the fork's groups are not in the index yet
        cache.select_groups([1], q[:1], 8, torch.empty((1, 2, 3), dtype=torch.int32, device="cuda"))
    for n in (1, 130, 77):
        k, v = W.make_sequence_kv(n, 2, W.LLAMA_RECIPE, gen)
        cache.append([0, 1], [0, n, 2 * n], torch.cat([k, k]).cuda(), torch.cat([v, v]).cuda())
        cache.update_index([0, 1])
        out = torch.empty((2, 8, 128), device="cuda")
        cache.decode_f32([0, 1], q, 8, out, ws)
        groups = torch.empty((2, 2, 3), dtype=torch.int32, device="cuda")
        cache.select_groups([0, 1], q, 8, groups)
        some = torch.empty((2, 8, 128), device="cuda")
        cache.sparse_decode([0, 1], q, 8, groups, some, ws)
        O.oscar_cache_check(cache.handle)
        assert torch.equal(groups[0], groups[1])
        assert (out[0] - out[1]).abs().max() <= 2e-5 and (some[0] - some[1]).abs().max() <= 2e-5   # (other CTA splits)
        assert equal(state(cache, 0), state(cache, 1))


def test_index_after_a_cut_and_a_compaction():
    O = U.lib()
    cache = make([1500], 2, 2, seed=8)
    cache.enable_index()
    cache.update_index([0])
    q, groups = W.make_q(1, 8, seed=9).cuda(), torch.empty((1, 2, 4), dtype=torch.int32, device="cuda")
    cache.truncate([0], [1200])                 # the entries of the groups left are kept
    cache.select_groups([0], q, 8, groups)
    first = groups.clone()
    cache.update_index([0], rebuild=True)
    cache.select_groups([0], q, 8, groups)
    torch.cuda.synchronize()
    assert torch.equal(first, groups) and int(first.max()) < 9
    cache.keep_groups([0], [[0, 1, 4, 6, 7, 8]])
    with pytest.raises(O.OscarError):
        cache.select_groups([0], q, 8, groups)
    cache.update_index([0])                     # groups 2 .. 5 are summarised again
    cache.select_groups([0], q, 8, groups)
    first = groups.clone()
    cache.update_index([0], rebuild=True)
    cache.select_groups([0], q, 8, groups)
    torch.cuda.synchronize()
    assert torch.equal(first, groups)


def test_decode_after_a_move_waits_for_it():
    """Decodes queued behind a move see the moved blocks, although the library copies settled blocks early."""
    O = U.lib()
    hq = 8
    cache = make([3000, 2600], 2, 3, seed=10)
    q, ws = W.make_q(1, hq, seed=11).cuda(), cache.workspace(1, hq)
    first, last = list(range(0, 23, 2)), list(range(11, 20))
    want = []
    for queued in (False, True):
        a = make([3000, 2600], 2, 3, seed=10)
        outs = []
        for _ in range(3):                      # the library knows the stream and that groups are settled
            decoded(a, 0, q, ws)
            decoded(a, 2, q, ws) if a.length(2) else None
        torch.cuda.synchronize()
        if queued:
            torch.cuda._sleep(1 << 22)

        def step(call):
            r = call()
            if not queued:
                torch.cuda.synchronize()
            return r

        step(lambda: a.fork([0], [2]))
        outs.append(step(lambda: decoded(a, 2, q, ws)))
        outs.append(step(lambda: decoded(a, 2, q, ws)))
        step(lambda: a.keep_groups([2], [first]))
        outs.append(step(lambda: decoded(a, 2, q, ws)))
        step(lambda: a.fork([1], [2], [2500]))
        outs.append(step(lambda: decoded(a, 2, q, ws)))
        step(lambda: a.keep_groups([1], [last], [2]))
        outs.append(step(lambda: decoded(a, 2, q, ws)))
        step(lambda: a.truncate([2], [1000]))
        outs.append(step(lambda: decoded(a, 2, q, ws)))
        torch.cuda.synchronize()
        O.oscar_cache_check(a.handle)
        want.append(outs)
    for x, y in zip(*want):
        assert torch.equal(x, y)


def test_captured():
    cache = make([900], 2, 2, seed=12)
    ws, q = cache.workspace(1, 8), W.make_q(1, 8, seed=13).cuda()
    want = prefix(cache, 0, 700)
    out = torch.empty((1, 8, 128), device="cuda")
    decoded(cache, 0, q, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.fork([0], [1], [700])
        cache.decode_f32([1], q, 8, out, ws)
    graph.replay()
    torch.cuda.synchronize()
    assert equal(state(cache, 1), want)
    again = decoded(cache, 1, q, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, again)


def test_refusals_change_nothing():
    O = U.lib()
    cache = make([500, 300], 2, 4, seed=14)
    before = [state(cache, i) for i in range(2)]
    for call in [lambda: cache.fork([0], [4]), lambda: cache.fork([-1], [2], [0]), lambda: cache.fork([0, 1], [2, 2]),
                 lambda: cache.fork([0], [2], [501]), lambda: cache.fork([0], [2], [-1]),
                 lambda: cache.fork([0, 1], [1, 2]),                     # slot 1 read and written
                 lambda: cache.fork([0, 0], [0, 2], [200, 500]),         # slot 0 cut and read
                 lambda: cache.fork([0, 1], [2]), lambda: cache.fork([0], [2], [1, 2]),
                 lambda: cache.keep_groups([0], [[0, 0]]), lambda: cache.keep_groups([0], [[2, 1]]),
                 lambda: cache.keep_groups([0], [[3]]), lambda: cache.keep_groups([0], [[-1]]),
                 lambda: cache.keep_groups([0], [[0]], [9]), lambda: cache.keep_groups([0, 1], [[0], [0]], [1, 0]),
                 lambda: cache.keep_groups([0], [[0], [1]]), lambda: cache.keep_groups([0], [[0.5]]),
                 lambda: cache.keep_groups([0], 3)]:
        with pytest.raises((O.OscarError, ValueError, TypeError)):
            call()
    torch.cuda.synchronize()
    assert [cache.length(i) for i in range(4)] == [500, 300, 0, 0]
    for i in range(2):
        assert equal(state(cache, i), before[i])
    cache.fork([], [])
    cache.keep_groups([], [])
