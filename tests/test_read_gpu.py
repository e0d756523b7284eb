"""Tokens read back against the stored cache dequantised in float64, and
sequences moved out and in.

Bounds.  A value is one multiply-add of the stored float32 parameters (half a
step of float32) rounded once more to the output type.  A key is 128 such
values (each within 2^-24 of |code s| + |z|) through seven additions and a
multiply (each within 2^-24 of the running sum, which the sum of magnitudes
bounds): 10 * 2^-24 * n / sqrt(128) * sum_c (|code s| + |z|), then the output
rounding."""
import numpy as np
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from oracle import oscar_oracle as OR
from tests import gpu_util as U

pytestmark = pytest.mark.gpu


def make(lens, hkv, meta=32, seed=1, capacity=None, chunk=1000):
    gen = torch.Generator().manual_seed(seed)
    kv = [W.make_sequence_kv(n, hkv, W.LLAMA_RECIPE, gen) for n in lens]
    cache = U.lib().OscarCache(len(lens), hkv, capacity or max(lens) + 1, meta_bits=meta)
    live = [i for i, n in enumerate(lens) if n]
    U.append_all(cache, live, [kv[i][0] for i in live], [kv[i][1] for i in live], chunk=chunk)
    return cache, kv


def stored(cache, arena, slot, head):
    """(keys, values, key bound) of a slot's tokens in float64."""
    h = U.gpu_head(cache, arena, slot, head)
    k, v, b = [h.window_k], [h.window_v], [np.zeros_like(h.window_k)]
    if h.num_groups:
        n = h.keys.norm.astype(np.float64)[..., None]
        rot = OR.dequant_keys(h.keys) * n
        size = (h.keys.codes * np.abs(h.keys.scale.astype(np.float64))[:, None] +
                np.abs(h.keys.zero.astype(np.float64))[:, None]) * n
        k.insert(0, (rot @ OR.hadamard()).reshape(-1, 128))
        b.insert(0, np.broadcast_to(size.sum(-1, keepdims=True) / np.sqrt(128) * 10 * 2.0 ** -24,
                                    rot.shape).reshape(-1, 128))
        v.insert(0, OR.dequant_values(h.values).reshape(-1, 128))
    return np.concatenate(k), np.concatenate(v), np.concatenate(b)


def check(cache, ids, start, end, dtype, kw=True, vw=True, offset=0):
    rows = sum(e - s for s, e in zip(start, end))
    hkv = cache.num_kv_heads

    def out():
        flat = torch.full(((rows + 2) * hkv * 128 + 16,), 7.0, dtype=dtype, device="cuda")
        return flat, flat[offset:offset + rows * hkv * 128].view(rows, hkv, 128)
    (kf, k), (vf, v) = out(), out()
    cache.read(ids, start, end, k if kw else None, v if vw else None)
    U.lib().oscar_cache_check(cache.handle)
    for f in (kf, vf):   # nothing behind (or before) the rows is written
        assert torch.all(f[:offset] == 7.0) and torch.all(f[offset + rows * hkv * 128:] == 7.0)
    arena = U.read_arena(cache)
    half = torch.finfo(dtype).eps / 2
    gk, gv = U.f64(k), U.f64(v)
    row = 0
    for i, s, e in zip(ids, start, end):
        for j in range(hkv):
            rk, rv, bk = (x[s:e] for x in stored(cache, arena, i, j))
            if kw:
                err = np.abs(gk[row:row + e - s, j] - rk)
                assert np.all(err <= bk + half * (np.abs(rk) + bk)), (i, j, "k")
            if vw:
                err = np.abs(gv[row:row + e - s, j] - rv)
                room = 2.0 ** -24 * np.abs(rv)
                assert np.all(err <= room + half * (np.abs(rv) + room)), (i, j, "v")
        row += e - s
    if not kw:
        assert torch.all(kf == 7.0)
    if not vw:
        assert torch.all(vf == 7.0)


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lens,hkv", [([1], 1), ([127], 2), ([128], 1), ([129], 3), ([1061], 1),
                                      ([300, 1, 517, 128, 90], 2), ([2047], 8)])
def test_whole_sequences(lens, hkv, dtype, meta):
    cache, _ = make(lens, hkv, meta)
    check(cache, list(range(len(lens))), [0] * len(lens), lens, dtype)


@pytest.mark.parametrize("dtype,offset", [(torch.bfloat16, 0), (torch.bfloat16, 8), (torch.float32, 4)])
def test_ranges(dtype, offset):
    """Parts that start and end inside groups, in the window, across both; the
    same slot twice; empty ranges; outputs that are 16- but not 32-byte
    aligned."""
    cache, _ = make([700, 260, 64], 2, seed=4)
    ids = [0, 1, 2, 0, 0, 1, 0, 2]
    start = [5, 250, 10, 128, 699, 0, 40, 64]
    end = [6, 260, 11, 256, 700, 0, 655, 64]
    check(cache, ids, start, end, dtype, offset=offset)
    check(cache, ids, start, end, dtype, kw=False)
    check(cache, ids, start, end, dtype, vw=False)


def test_many_ranges():
    """More ranges than one launch takes."""
    cache, _ = make([500], 1, seed=6)
    n = 1100
    start = [(37 * i) % 400 for i in range(n)]
    check(cache, [0] * n, start, [s + 1 + i % 3 for i, s in enumerate(start)], torch.bfloat16)


def test_read_back_is_close_to_what_was_appended():
    """Every key channel in the rotated basis is within half a code step (plus
    rounding) of the appended one: read rows are in the appended basis."""
    cache, kv = make([512], 2, seed=8)
    k = torch.empty((512, 2, 128), device="cuda")
    v = torch.empty_like(k)
    cache.read([0], [0], [512], k, v)
    arena = U.read_arena(cache)
    for j in range(2):
        h = U.gpu_head(cache, arena, 0, j)
        step = (h.keys.scale.astype(np.float64)[:, None] * h.keys.norm.astype(np.float64)[..., None]).reshape(-1, 128)
        diff = (U.f64(k)[:, j] - U.f64(kv[0][0])[:, j]) @ OR.hadamard()
        assert np.all(np.abs(diff) <= 0.5 * step * (1 + 1e-4) + 1e-5 * np.abs(U.f64(k)[:, j]).max())
        vs = np.repeat(h.values.scale.astype(np.float64), 32, -1).reshape(-1, 128)
        assert np.all(np.abs(U.f64(v)[:, j] - U.f64(kv[0][1])[:, j]) <= 0.5 * vs * (1 + 1e-4) + 1e-6)


def test_stream_graph_and_repeats():
    cache, _ = make([900], 4, seed=3)
    k, v = (torch.empty((900, 4, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.read([0], [0], [900], k, v)
    rk, rv = k.clone(), v.clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    k.zero_(), v.zero_()
    torch.cuda.synchronize()
    cache.read([0], [0], [900], k, v, stream=s)
    s.synchronize()
    assert torch.equal(k, rk) and torch.equal(v, rv)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.read([0], [0], [900], k, v)
    k.zero_(), v.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(k, rk) and torch.equal(v, rv)


@pytest.mark.parametrize("pinned", [False, True])
@pytest.mark.parametrize("meta", [32, 16])
def test_export_import(meta, pinned):
    """A sequence moved to another slot of another cache decodes, continues and
    reads back as before."""
    lens = [1061, 64, 256]
    cache, kv = make(lens, 2, meta, seed=11, capacity=2000)
    O = U.lib()
    other = O.OscarCache(4, 2, 2000, meta_bits=meta)
    # the destination held something else before
    U.append_all(other, [3], [kv[0][0][:300]], [kv[0][1][:300]])
    slots = [3, 1, 0]
    for i, s in enumerate(slots):
        state = cache.export_sequence(i, pinned=pinned)
        assert state[0] == lens[i]
        torch.cuda.synchronize()
        other.import_sequence(s, *state)
        assert other.length(s) == lens[i]
    a, b = U.read_arena(cache), U.read_arena(other)
    for i, s in enumerate(slots):
        assert np.array_equal(U.live_bytes(cache, a, i), U.live_bytes(other, b, s))
    # both go on the same way
    gen = torch.Generator().manual_seed(12)
    more = [W.make_sequence_kv(200, 2, W.LLAMA_RECIPE, gen) for _ in lens]
    U.append_all(cache, [0, 1, 2], [m[0] for m in more], [m[1] for m in more])
    U.append_all(other, slots, [m[0] for m in more], [m[1] for m in more])
    q = W.make_q(3, 8, seed=13).cuda()
    x, y = (torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cache.decode([0, 1, 2], q, 8, x, cache.workspace(3, 8))
    other.decode(slots, q, 8, y, other.workspace(3, 8))
    O.oscar_cache_check(other.handle)
    assert torch.equal(x, y)


def test_export_import_of_slices():
    """Buffers that start anywhere: rows of a batch's tensors, one KV head."""
    cache, _ = make([700, 390], 1, seed=14, capacity=900)
    n, blocks, window, maxima = cache.export_sequence(0)
    batch = torch.zeros((3, 2, 1), device="cuda")
    flat = torch.zeros(blocks.numel() + 1, dtype=torch.uint8, device="cuda")
    win = torch.zeros(window.numel() + 1, dtype=torch.bfloat16, device="cuda")
    batch[1], flat[1:], win[1:] = maxima, blocks.view(-1), window.view(-1)
    cache.import_sequence(1, n, flat[1:].view(blocks.shape), win[1:].view(window.shape), batch[1])
    a = U.read_arena(cache)
    assert np.array_equal(U.live_bytes(cache, a, 0), U.live_bytes(cache, a, 1))


def test_import_after_a_decode_is_attended():
    """A decode that follows an import on the stream of earlier decodes sees
    the new blocks (none of the slot's old ones copied early)."""
    O = U.lib()
    cache, _ = make([2048, 2048], 2, seed=21)
    q = W.make_q(1, 8, seed=22).cuda()
    ws = cache.workspace(1, 8)
    want, got = (torch.empty((1, 8, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for _ in range(2):
        cache.decode([1], q, 8, want, ws)
        cache.decode([0], q, 8, got, ws)
    state = cache.export_sequence(1)
    assert O.oscar_test_settled_groups(cache, [0])[0] > 0
    cache.import_sequence(0, *state)
    assert O.oscar_test_settled_groups(cache, [0]) == [0]
    cache.decode([0], q, 8, got, ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_refusals():
    O = U.lib()
    cache, _ = make([300, 0], 2)
    k = torch.zeros((300, 2, 128), device="cuda")
    v = torch.zeros_like(k)

    def refused(status, ids, s, e, kk=k, vv=v):
        with pytest.raises(O.OscarError) as err:
            cache.read(ids, s, e, kk, vv)
        assert err.value.status == status
    bad = O.OSCAR_ERR_INVALID_ARG
    refused(bad, [0], [0], [301], torch.zeros((301, 2, 128), device="cuda"), None)
    refused(bad, [0], [-1], [10])
    refused(bad, [0], [20], [10])
    refused(bad, [2], [0], [0])
    refused(bad, [-1], [0], [0])
    refused(bad, [1], [0], [1])
    refused(bad, [0], [0], [300], k, k)
    both = torch.zeros((301, 2, 128), dtype=torch.bfloat16, device="cuda")
    refused(bad, [0], [0], [300], both[:300], both[1:])      # the buffers overlap
    refused(bad, [0], [0], [300], k.cpu(), v)
    flat = torch.zeros(300 * 256 + 8, device="cuda")
    refused(bad, [0], [0], [300], flat[2:2 + 300 * 256].view(300, 2, 128), v)
    with pytest.raises(ValueError):
        cache.read([0], [0], [300], k[:, :1].contiguous(), None)
    cache.read([], [], [], None, None)
    cache.read([0], [7], [7], k, v)
    n, blocks, window, maxima = cache.export_sequence(0)
    for args, status in [((0, 100000, blocks, window, maxima), None), ((0, -1, blocks, window, maxima), None),
                         ((5, 300, blocks, window, maxima), bad), ((0, 300, blocks, None, maxima), bad),
                         ((0, 301, blocks, window, maxima), O.OSCAR_OK),
                         ((0, 300, None, window, maxima), bad)]:
        if status == O.OSCAR_OK:
            cache.import_sequence(*args)
            continue
        with pytest.raises((O.OscarError, ValueError)) as err:
            cache.import_sequence(*args)
        if status is not None:
            assert err.value.status == status
    with pytest.raises(O.OscarError):
        O.oscar_cache_import(cache.handle, 0, 100000, blocks, window, maxima)
    assert cache.length(0) == 301


@pytest.mark.parametrize("meta", [32, 16])
def test_state_buffers_too_small_are_refused(meta):
    """Buffers for fewer heads or tokens than the copies would take, in the
    functions as in the methods; the slot keeps what it holds."""
    O = U.lib()
    cache, _ = make([700, 640], 4, meta, seed=33, capacity=1000)
    n, blocks, window, maxima = cache.export_sequence(0)
    before = U.read_arena(cache)
    for state in [(blocks[:3], window, maxima), (blocks[:, :4].contiguous(), window, maxima),
                  (blocks.view(-1)[:-1], window, maxima), (blocks, window[:2], maxima),
                  (blocks, window, maxima[:, :1].contiguous()), (blocks, window, maxima[:1])]:
        with pytest.raises(ValueError):
            O.oscar_cache_export(cache.handle, 0, *state)
        with pytest.raises(ValueError):
            O.oscar_cache_import(cache.handle, 1, n, *state)
    with pytest.raises(ValueError):
        O.oscar_cache_import(cache.handle, 1, n + 128 - n % 128, blocks, None, maxima)     # one group more
    assert cache.length(1) == 640
    after = U.read_arena(cache)
    assert np.array_equal(U.live_bytes(cache, before, 1), U.live_bytes(cache, after, 1))
    # larger ones, and none where nothing is copied
    more = torch.zeros(blocks.numel() + 5, dtype=torch.uint8, device="cuda")
    O.oscar_cache_export(cache.handle, 0, more, window, maxima)
    assert torch.equal(more[:-5], blocks.view(-1)) and torch.all(more[-5:] == 0)
    O.oscar_cache_export(cache.handle, 1, more, None, maxima)
    O.oscar_cache_import(cache.handle, 0, 640, more, None, maxima)
    torch.cuda.synchronize()
    after = U.read_arena(cache)
    assert np.array_equal(U.live_bytes(cache, before, 1), U.live_bytes(cache, after, 0))


@pytest.mark.parametrize("pinned", [False, True])
@pytest.mark.parametrize("raw", [False, True])
def test_a_state_dropped_before_its_copies_ran(pinned, raw):
    """Export and import queued behind a busy stream that is not the current
    one, and the state dropped at once: its memory is not handed out again
    before the copies have run, and they carry the right bytes."""
    cache, _ = make([1061, 1061], 2, seed=31)
    torch.cuda.synchronize()
    before = U.read_arena(cache)
    s = torch.cuda.Stream()
    stream = s.cuda_stream if raw else s
    where = dict(pin_memory=True) if pinned else dict(device="cuda")

    def others(like):      # what an allocation of the same sizes gets
        return [torch.empty(t.shape, dtype=t.dtype, **where) for t in like]
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    state = cache.export_sequence(0, pinned=pinned, stream=stream)
    at = [t.data_ptr() for t in state[1:]]
    like = [torch.empty_like(t, device="meta") for t in state[1:]]
    del state
    held = others(like)
    assert not s.query()                                       # the copies are still queued
    assert not set(at) & {t.data_ptr() for t in held}
    torch.cuda.synchronize()
    del held
    state = cache.export_sequence(0, pinned=pinned)            # complete, on the current stream
    torch.cuda.synchronize()
    U.lib().oscar_cache_reset(cache.handle, 1)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(200_000_000)
    cache.import_sequence(1, *state, stream=stream)
    at = [t.data_ptr() for t in state[1:]]
    del state
    held = others(like)
    assert not s.query()
    assert not set(at) & {t.data_ptr() for t in held}
    for t in held:
        t.fill_(0)
    torch.cuda.synchronize()
    after = U.read_arena(cache)
    assert np.array_equal(U.live_bytes(cache, before, 0), U.live_bytes(cache, after, 1))
    assert cache.length(1) == 1061


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_wait_that_runs_out(dtype, meta):
    """A copy left unissued (the library's own hook): the bounded wait gives
    up, the call reports it, later calls are unaffected.  With more tiles than
    blocks, so that the block that gives up has a further tile."""
    O = U.lib()
    cache, _ = make([128 * 60 + 5], 8, meta, seed=41, chunk=4096)
    assert 61 * 8 > 3 * torch.cuda.get_device_properties(0).multi_processor_count
    n = cache.length(0)
    want, got = (torch.empty((2, n, 8, 128), dtype=dtype, device="cuda") for _ in range(2))
    cache.read([0], [0], [n], want[0], want[1])
    O.oscar_cache_check(cache.handle)
    O.oscar_test_arm_wait_timeout()
    cache.read([0], [0], [n], got[0], got[1])
    with pytest.raises(O.OscarError) as e:
        O.oscar_cache_check(cache.handle)
    assert e.value.status == O.OSCAR_ERR_DEVICE_TIMEOUT
    O.oscar_cache_check(cache.handle)
    cache.read([0], [0], [n], got[0], got[1])
    O.oscar_cache_check(cache.handle)
    assert torch.equal(got, want)


def test_export_import_of_registered_host_memory():
    """Page-locked memory that is not torch's (the caller keeps it)."""
    cache, _ = make([700, 0], 2, seed=35, capacity=900)
    n, blocks, window, maxima = cache.export_sequence(0)
    host = [torch.zeros(t.shape, dtype=t.dtype) for t in (blocks, window, maxima)]
    rt = torch.cuda.cudart()
    for t in host:
        assert int(rt.cudaHostRegister(t.data_ptr(), t.numel() * t.element_size(), 0)) == 0
    try:
        U.lib().oscar_cache_export(cache.handle, 0, *host)
        cache.import_sequence(1, n, *host)
        torch.cuda.synchronize()
    finally:
        for t in host:
            rt.cudaHostUnregister(t.data_ptr())
    assert torch.equal(host[0], blocks.cpu()) and torch.equal(host[2], maxima.cpu())
    a = U.read_arena(cache)
    assert np.array_equal(U.live_bytes(cache, a, 0), U.live_bytes(cache, a, 1))
