"""Decode attention over listed groups against the oracle's attention over the
same groups of the GPU's own cache, in float64.

Bound.  With the listed tokens' scores s_t and A_t = scale n_t sum_c |q_rot_c|
(|code s| + |z|) (window: scale sum_c |q_c k_c|), the score arithmetic (fp16
hi + lo factors good to 2^-22, float32 sums over 128 terms: 128 roundings at
most, far fewer in a row) is off by at most d = 2^-16 max_t A_t + 2^-20; the
weights then by a factor e^(2 d) at most, and the value sums (2^-22 factors,
float32 sums, ex2.approx 2^-22) by 2^-16 of the largest |v|.  So
|out - ref| <= (e^(2 d) - 1 + 2^-16) max|v|, then the output rounding, and
|lse - ref| <= d + 2^-20 (1 + |ref|).

bf16 outputs take the factors p_t s_t of the value codes (0 to 3) in fp16, as
x_t = p_t s_t 2^(F - p) with 2^14 <= 2^F S < 2^15 for the head's largest value
scale S, and p <= 8.  Normal x_t are off by 2^-11 x_t at most, subnormal ones by
2^-25, which is at most 2^-25 2^8 2^-14 S = 2^-31 S of p_t s_t.  The weights
p_t / l sum to 1 and l >= 1, so n tokens' value sums are off by
3 (2^-11 + n 2^-31) S at most, S in the first term the largest scale attended.
float32 outputs take them as fp16 hi + lo, p <= 9: where the remainder is
subnormal it is off by 2^-25, 2^-30 S of p_t s_t (this counts where S, the largest
of the whole sequence, is far above the scales attended): 3 n 2^-30 S."""
import numpy as np
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from oracle import oscar_oracle as OR
from tests import gpu_util as U

pytestmark = pytest.mark.gpu


def make(lens, hkv, meta=32, seed=1):
    gen = torch.Generator().manual_seed(seed)
    kv = [W.make_sequence_kv(n, hkv, W.LLAMA_RECIPE, gen) for n in lens]
    cache = U.lib().OscarCache(len(lens), hkv, max(lens) + 300, meta_bits=meta)
    U.append_all(cache, list(range(len(lens))), [k for k, _ in kv], [v for _, v in kv], chunk=4096)
    return cache


def listed(h, idx):
    """The head's cache restricted to the listed groups (repeats kept) and the window."""
    keys = values = None
    if len(idx):
        keys = OR.KeyGroup(h.keys.codes[idx], h.keys.scale[idx], h.keys.zero[idx], h.keys.norm[idx], None)
        values = OR.ValueGroup(h.values.codes[idx], h.values.scale[idx], h.values.zero[idx], None)
    return OR.HeadCache(keys, values, h.window_k, h.window_v)


def check_head(q, h, got, lse, scale, half, largest):
    if h.length == 0:
        assert np.all(got == 0) and np.all(lse == -np.inf)
        return
    ref, rl = OR.history_attention(q, h, scale)
    sc = 1 / np.sqrt(128) if scale is None else scale
    a = [0.0]
    if h.num_groups:
        size = (h.keys.codes * np.abs(h.keys.scale.astype(np.float64))[:, None] +
                np.abs(h.keys.zero.astype(np.float64))[:, None]) * h.keys.norm.astype(np.float64)[..., None]
        a.append((size.reshape(-1, 128) @ np.abs(OR.canalized_rotation(q)).T).max() * sc)
    if h.window_k.shape[0]:
        a.append((np.abs(h.window_k) @ np.abs(q).T).max() * sc)
    d = 2.0 ** -16 * max(a) + 2.0 ** -20
    room = (np.expm1(2 * d) + 2.0 ** -16) * np.abs(OR.decode_values(h)).max()
    if h.num_groups:
        if half == 2.0 ** -8:
            room += 3 * (2.0 ** -11 * h.values.scale.max() + h.length * 2.0 ** -31 * largest)
        else:
            room += 3 * h.length * 2.0 ** -30 * largest
    err = np.abs(got - ref)
    assert np.all(err <= room + half * (np.abs(ref) + room)), f"{err.max():.3e} > {room:.3e}"
    assert np.all(np.abs(lse - rl) <= d + 2.0 ** -20 * (1 + np.abs(rl)))


def check(cache, ids, q, groups, dtype=torch.float32, scale=0.0):
    O = U.lib()
    n, hq, hkv = len(ids), q.shape[1], cache.num_kv_heads
    out = torch.full((n + 1, hq, 128), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((n + 1, hq), 7.0, device="cuda")
    cache.sparse_decode(ids, q, hq, groups, out, cache.workspace(n, hq), lse, softmax_scale=scale)
    O.oscar_cache_check(cache.handle)
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)
    arena, qn, go, gl, gi = U.read_arena(cache), U.f64(q), U.f64(out), U.f64(lse), groups.cpu().numpy()
    assert np.all(np.isfinite(go))
    gqa = hq // hkv
    for i, s in enumerate(ids):
        for j in range(hkv):
            idx = [int(g) for g in gi[i, j] if 0 <= g < cache.length(s) // 128]
            heads = slice(gqa * j, gqa * (j + 1))
            full = U.gpu_head(cache, arena, s, j)
            check_head(qn[i, heads], listed(full, idx), go[i, heads], gl[i, heads], None if scale == 0.0 else scale,
                       torch.finfo(dtype).eps / 2, full.values.scale.max() if full.num_groups else 0.0)
    return out[:n], lse[:n]


def lists(cache, ids, n, seed, empty=0.0):
    rng = np.random.default_rng(seed)
    out = np.full((len(ids), cache.num_kv_heads, n), -1, np.int32)
    for i, s in enumerate(ids):
        for j in range(cache.num_kv_heads):
            pick = rng.permutation(cache.length(s) // 128)[:n]
            keep = rng.random(pick.size) >= empty
            out[i, j, :pick.size] = np.where(keep, pick, rng.choice([-1, -2 ** 31, 2 ** 31 - 1, 10 ** 6], pick.size))
            out[i, j] = rng.permutation(out[i, j])
    return torch.from_numpy(out).cuda()


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("lens,hkv,hq,n,empty", [
    ([1024], 1, 4, 1, 0.0), ([2100, 128, 77], 2, 2, 5, 0.0), ([6000, 300], 2, 16, 9, 0.3), ([4000], 1, 5, 40, 0.5),
    ([129, 1], 3, 9, 2, 0.0), ([2560], 2, 24, 7, 0.2), ([5000, 5001, 4999], 1, 1, 33, 0.9)])
def test_against_the_oracle(lens, hkv, hq, n, empty, meta):
    cache = make(lens, hkv, meta, seed=hq + n)
    ids = list(range(len(lens)))[::-1]
    q = W.make_q(len(lens), hq, seed=3).cuda()
    check(cache, ids, q, lists(cache, ids, n, 7, empty))
    check(cache, ids, q, lists(cache, ids, n, 8, empty), torch.bfloat16, scale=0.03)


@pytest.mark.parametrize("lens,hkv,hq,n,meta", [
    ([128 * (1 + i % 5) + 3 * i for i in range(40)], 2, 8, 3, 32),      # windows of every length, more rows than SMs
    ([128 * (1 + i % 4) for i in range(40)], 2, 8, 2, 16),              # no windows
    ([30 + 17 * i for i in range(33)], 1, 8, 2, 32),                    # some without a group, 8 heads
    ([140 + 9 * i for i in range(41)], 2, 6, 5, 16),                    # 3 heads
    ([16, 32, 48, 127, 128, 255, 256, 257] * 32, 1, 1, 1, 32),          # whole tiles of 16 window tokens
    ([1000] * 20, 1, 13, 6, 32),                                        # two passes: 8 and 5 heads
    ([260 + i for i in range(36)], 1, 7, 2, 32)])
def test_many_rows(lens, hkv, hq, n, meta):
    """More query heads than 1.5 per SM: the combine with a CTA per KV head."""
    cache = make(lens, hkv, meta, seed=hq + n)
    ids = list(range(len(lens)))
    q = W.make_q(len(lens), hq, seed=4).cuda()
    check(cache, ids, q, lists(cache, ids, n, 11, 0.2))


def test_wait_that_runs_out():
    """A copy left unissued (the library's own hook): the bounded waits give
    up, the call reports it, later calls are unaffected."""
    O = U.lib()
    cache = make([2000], 1, seed=15)
    q = W.make_q(1, 4, seed=16).cuda()
    groups = torch.arange(8, dtype=torch.int32).view(1, 1, 8).cuda()
    want = check(cache, [0], q, groups)
    out, ws = torch.empty((1, 4, 128), device="cuda"), cache.workspace(1, 4)
    O.oscar_test_arm_wait_timeout()
    cache.sparse_decode([0], q, 4, groups, out, ws)
    with pytest.raises(O.OscarError) as e:
        O.oscar_cache_check(cache.handle)
    assert e.value.status == O.OSCAR_ERR_DEVICE_TIMEOUT
    again = check(cache, [0], q, groups)
    assert torch.equal(want[0], again[0]) and torch.equal(want[1], again[1])


def test_two_streams_at_once():
    """Calls on two streams with their own workspaces, lists and outputs."""
    cache = make([3000, 2900], 2, seed=17)
    q = [W.make_q(2, 8, seed=18 + i).cuda() for i in range(2)]
    g = [lists(cache, [0, 1], 9, 20 + i, 0.1) for i in range(2)]
    want = [check(cache, [0, 1], q[i], g[i]) for i in range(2)]
    ws = [cache.workspace(2, 8) for _ in range(2)]
    outs = [torch.empty((20, 2, 8, 128), device="cuda") for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(20):
        for i in range(2):
            cache.sparse_decode([0, 1], q[i], 8, g[i], outs[i][k], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    U.lib().oscar_cache_check(cache.handle)
    for i in range(2):
        assert all(torch.equal(outs[i][k], want[i][0]) for k in range(20))


def test_many_entries_per_block():
    """More entries than a block's ring and than one look-up of 32."""
    cache = make([128 * 500 + 3], 1, seed=31)
    ids = [0]
    q = W.make_q(1, 4, seed=4).cuda()
    rng = np.random.default_rng(5)
    g = rng.integers(-3, 500, (1, 1, 30000)).astype(np.int32)       # repeats and empty entries
    want_idx = [int(x) for x in g[0, 0] if x >= 0]
    groups = torch.from_numpy(g).cuda()
    out = torch.empty((1, 4, 128), device="cuda")
    lse = torch.empty((1, 4), device="cuda")
    cache.sparse_decode(ids, q, 4, groups, out, cache.workspace(1, 4), lse)
    U.lib().oscar_cache_check(cache.handle)
    # a group listed c times weighs c times: the oracle with weights
    h = U.gpu_head(cache, U.read_arena(cache), 0, 0)
    count = np.bincount(want_idx, minlength=500).astype(np.float64)
    s = OR.decode_scores(U.f64(q)[0], h)
    wts = np.concatenate([np.repeat(count, 128), np.ones(3)])[:, None]
    m = s.max(0)
    p = np.exp(s - m) * wts
    ref = (p / p.sum(0)).T @ OR.decode_values(h)
    top = np.abs(OR.decode_values(h)).max()
    # the bound of the other tests with max_t A_t below 64 and sums over 1e5 tokens in 2^-14
    assert np.abs(U.f64(out)[0] - ref).max() <= (np.expm1(2 * 64 * 2.0 ** -16) + 2.0 ** -14) * top
    assert np.abs(U.f64(lse)[0] - (m + np.log(p.sum(0)))).max() <= 64 * 2.0 ** -16 + 2.0 ** -14


def test_rows_with_nothing():
    """Empty lists with and without a window, in a batch with full ones."""
    cache = make([1024, 1030, 60, 2048], 2, seed=5)
    q = W.make_q(4, 8, seed=6).cuda()
    groups = lists(cache, [0, 1, 2, 3], 4, 9)
    groups[0] = -1
    groups[1] = 99
    groups[3, 1] = -7
    out, lse = check(cache, [0, 1, 2, 3], q, groups)
    assert torch.all(out[0] == 0) and torch.all(lse[0] == -float("inf"))
    assert torch.all(out[3, 4:] == 0) and torch.all(lse[3, :4].isfinite())
    # every row of the call empty
    out, lse = check(cache, [0, 3], q[:2], torch.full((2, 2, 3), -1, dtype=torch.int32, device="cuda"), torch.bfloat16)
    assert torch.all(out == 0)


@pytest.mark.parametrize("factor", [300.0, 1e4])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_token_of_large_values(factor, dtype):
    """One token's values far above the others': the value factors are scaled
    by the sequence's largest, also where its group is not listed."""
    gen = torch.Generator().manual_seed(51)
    k, v = W.make_sequence_kv(1100, 2, W.LLAMA_RECIPE, gen)
    v[300] *= factor
    cache = U.lib().OscarCache(1, 2, 1300)
    U.append_all(cache, [0], [k], [v], chunk=4096)
    q = W.make_q(1, 8, seed=52).cuda()
    for idx in ([0, 2, 5], [0, 1, 4, 7], [1, 3, 6], [7]):
        check(cache, [0], q, torch.tensor(idx, dtype=torch.int32).repeat(1, 2, 1).cuda(), dtype)


def test_all_groups_listed_is_the_full_decode():
    """Every group in order, each once, against the full decode: each is
    within 2e-3 of the oracle (the full decode's own bound; the sparse one's is
    tighter, see check)."""
    for lens, hkv, hq in ([[5000], 2, 8], [[3000, 3000], 1, 7]):
        cache = make(lens, hkv, seed=41)
        n, ng = len(lens), lens[0] // 128
        q = W.make_q(n, hq, seed=2).cuda()
        groups = torch.arange(ng, dtype=torch.int32).expand(n, hkv, ng).contiguous().cuda()
        ids = list(range(n))
        a = torch.empty((n, hq, 128), device="cuda")
        cache.decode_f32(ids, q, hq, a, cache.workspace(n, hq))
        b, _ = check(cache, ids, q, groups)
        check(cache, ids, q, groups, torch.bfloat16)
        assert (a - b).abs().max().item() <= 4e-3


def test_lse_merges_two_parts():
    """Two calls over the halves of the groups merge into the whole (the
    window goes with the first; the second sequence has none)."""
    cache = make([2048], 1, seed=6)
    q = W.make_q(1, 4, seed=7).cuda()
    ws = cache.workspace(1, 4)
    parts = []
    for g in (range(0, 9), range(9, 16)):
        idx = torch.tensor(list(g), dtype=torch.int32).view(1, 1, -1).cuda()
        out, lse = check(cache, [0], q, idx)
        parts.append((U.f64(out)[0], U.f64(lse)[0]))
    o, _ = OR.merge_attention(*parts[0], *parts[1])
    full = torch.empty((1, 4, 128), device="cuda")
    cache.decode_f32([0], q, 4, full, ws)
    assert np.abs(o - U.f64(full)[0]).max() <= 4e-3        # two sides of 2e-3, as the decode's own tests have


def test_interleaved_with_other_decodes():
    """Sparse and full decodes, appends and selections in turn on one stream,
    twice, against each alone after a synchronise."""
    O = U.lib()
    cache = make([3000, 1500], 2, seed=51)
    cache.enable_index()
    gen = torch.Generator().manual_seed(52)
    k, v = W.make_sequence_kv(300, 2, W.LLAMA_RECIPE, gen)
    k, v = k.cuda(), v.cuda()
    twin = make([3000, 1500], 2, seed=51)
    twin.enable_index()
    q = W.make_q(2, 8, seed=53).cuda()
    ws, ws2 = cache.workspace(2, 8), twin.workspace(2, 8)
    at = 0

    def step(c, w, o, l, d, wait):
        c.append([0, 1], [0, 7, 14], k[at:at + 14], v[at:at + 14])
        if wait:
            torch.cuda.synchronize()
        c.update_index([0, 1])
        g = torch.empty((2, 2, 6), dtype=torch.int32, device="cuda")
        c.select_groups([0, 1], q, 8, g, 1, 1)
        if wait:
            torch.cuda.synchronize()
        c.sparse_decode([0, 1], q, 8, g, o, w, l)
        if wait:
            torch.cuda.synchronize()
        c.decode([0, 1], q, 8, d, w)
        if wait:
            torch.cuda.synchronize()
    outs = [[torch.empty((2, 8, 128), device="cuda"), torch.empty((2, 8), device="cuda"),
             torch.empty((2, 8, 128), dtype=torch.bfloat16, device="cuda")] for _ in range(42)]
    for i in range(21):
        step(cache, ws, *outs[i], False)
        at += 14
    at = 0
    for i in range(21):
        step(twin, ws2, *outs[21 + i], True)
        at += 14
    torch.cuda.synchronize()
    O.oscar_cache_check(cache.handle)
    for a, b in zip(outs[:21], outs[21:]):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_graph_replay_reads_new_lists():
    cache = make([4000], 2, seed=61)
    q = W.make_q(1, 8, seed=62).cuda()
    groups = lists(cache, [0], 5, 1)
    ws, out, lse = cache.workspace(1, 8), torch.empty((1, 8, 128), device="cuda"), torch.empty((1, 8), device="cuda")
    cache.sparse_decode([0], q, 8, groups, out, ws, lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.sparse_decode([0], q, 8, groups, out, ws, lse)
    for seed in (2, 3):
        groups.copy_(lists(cache, [0], 5, seed, 0.2))
        g.replay()
        torch.cuda.synchronize()
        got = out.clone(), lse.clone()
        want = check(cache, [0], q, groups)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_host_buffers_and_offsets():
    """q, out and lse in page-locked memory; a list that starts 4 bytes into a buffer."""
    cache = make([2000, 700], 2, seed=71)
    q = W.make_q(2, 8, seed=72)
    groups = lists(cache, [0, 1], 3, 4)
    want, wl = check(cache, [0, 1], q.cuda(), groups)
    flat = torch.zeros(groups.numel() + 1, dtype=torch.int32, device="cuda")
    flat[1:] = groups.view(-1)
    out, lse = torch.zeros((2, 8, 128)).pin_memory(), torch.zeros((2, 8)).pin_memory()
    cache.sparse_decode([0, 1], q.pin_memory(), 8, flat[1:].view(2, 2, 3), out, cache.workspace(2, 8), lse)
    torch.cuda.synchronize()
    assert torch.equal(out, want.cpu()) and torch.equal(lse, wl.cpu())


def test_refusals():
    O = U.lib()
    cache = make([600], 2, seed=3)
    q = W.make_q(1, 4, seed=2).cuda()
    ws, out = cache.workspace(1, 4), torch.empty((1, 4, 128), device="cuda")
    groups = torch.zeros((1, 2, 3), dtype=torch.int32, device="cuda")

    def refused(fn, status=O.OSCAR_ERR_INVALID_ARG):
        with pytest.raises(O.OscarError) as e:
            fn()
        assert e.value.status == status
    refused(lambda: cache.sparse_decode([0], q, 4, groups.cpu(), out, ws))
    refused(lambda: O.oscar_sparse_decode_attention(cache.handle, [0, 0], q.expand(2, 4, 128).contiguous(), 4, 0.0,
                                                    groups.expand(2, 2, 3).contiguous(),
                                                    out.expand(2, 4, 128).contiguous(), ws))
    refused(lambda: cache.sparse_decode([0], q, 4, groups[..., :0].contiguous(), out, ws))
    refused(lambda: cache.sparse_decode([1], q, 4, groups, out, ws))
    refused(lambda: cache.sparse_decode([0], q, 4, groups, out, ws[:64]), O.OSCAR_ERR_CAPACITY)
    refused(lambda: cache.sparse_decode([0], q, 4, groups, out, ws, softmax_scale=-1.0))
    refused(lambda: cache.sparse_decode([0], q, 4, groups, out.cpu(), ws))
    O.oscar_cache_reset(cache.handle, 0)
    refused(lambda: cache.sparse_decode([0], q, 4, groups, out, ws))
    with pytest.raises(ValueError):
        cache.sparse_decode([0], q, 4, groups[:, :1].contiguous(), out, ws)


NAN_SHAPES = [([1000], 1, 4, 3), ([1030, 900], 2, 6, 4), ([2048, 400], 1, 8, 5),      # the combine per query head
              ([300 + i for i in range(40)], 2, 8, 2), ([256 + i % 2 for i in range(35)], 1, 7, 2)]   # per KV head


@pytest.mark.parametrize("lens,hkv,hq,n", NAN_SHAPES)
@pytest.mark.parametrize("attend", ["groups", "window", "both"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_query_that_is_not_finite(lens, hkv, hq, n, attend, value, dtype):
    """NaN outputs and log-sum-exp for that query head wherever it has a token
    to attend (its scores are NaN, as are the full decode's outputs), zeros and
    -inf where it has none; the other heads' bits do not change."""
    cache = make([x // 128 * 128 for x in lens] if attend == "groups" else lens, hkv, seed=hq + n)
    ids, gqa = list(range(len(lens))), hq // hkv
    groups = lists(cache, ids, n, 21, 0.2)
    if attend == "window":
        groups.fill_(-1)
    q = W.make_q(len(lens), hq, seed=8).cuda()
    ws = cache.workspace(len(lens), hq)

    def call(x):
        out, lse = torch.empty((len(lens), hq, 128), dtype=dtype, device="cuda"), torch.empty((len(lens), hq), device="cuda")
        cache.sparse_decode(ids, x, hq, groups, out, ws, lse)
        U.lib().oscar_cache_check(cache.handle)
        return out, lse
    out, lse = call(q)
    bad = torch.zeros((len(lens), hq), dtype=torch.bool, device="cuda")
    bad[0, 1] = bad[-1, -1] = bad[len(lens) // 2, 0] = True
    qb = q.clone()
    qb[..., 37] = torch.where(bad, torch.full_like(q[..., 37], value), q[..., 37])
    got, got_lse = call(qb)
    used = torch.tensor([[any(0 <= g < cache.length(s) // 128 for g in groups[i, h // gqa].tolist()) or
                          cache.length(s) % 128 > 0 for h in range(hq)] for i, s in enumerate(ids)], device="cuda")
    nan = bad & used
    assert nan.any()
    assert torch.all(got[nan].isnan()) and torch.all(got_lse[nan].isnan())
    assert torch.equal(got[~nan], out[~nan]) and torch.equal(got_lse[~nan], lse[~nan])
    assert torch.all(got[bad & ~used] == 0) and torch.all(got_lse[bad & ~used] == -float("inf"))
    full = torch.empty((len(lens), hq, 128), device="cuda")
    cache.decode_f32(ids, qb, hq, full, ws)
    assert torch.all(full[bad].isnan())


@pytest.mark.parametrize("lens,hkv,hq", [([5 + i % 120 for i in range(200)], 2, 4), ([127] * 40, 1, 8)])
def test_window_wait_that_runs_out(lens, hkv, hq):
    """Sequences without a group, so many that a block per KV head stages the
    window: its copies left unissued (the library's own hook)."""
    O = U.lib()
    cache = make(lens, hkv, seed=81)
    ids = list(range(len(lens)))
    assert len(lens) * hq > 1.5 * torch.cuda.get_device_properties(0).multi_processor_count
    q = W.make_q(len(lens), hq, seed=82).cuda()
    groups = torch.zeros((len(lens), hkv, 2), dtype=torch.int32, device="cuda")
    want = check(cache, ids, q, groups)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = cache.workspace(len(lens), hq)
    O.oscar_test_arm_wait_timeout()
    cache.sparse_decode(ids, q, hq, groups, out, ws, lse)
    with pytest.raises(O.OscarError) as e:
        O.oscar_cache_check(cache.handle)
    assert e.value.status == O.OSCAR_ERR_DEVICE_TIMEOUT
    # only the first block's row was given up
    gqa = hq // hkv
    assert torch.equal(out[1:], want[0][1:]) and torch.equal(out[0, gqa:], want[0][0, gqa:])
    assert torch.equal(lse[1:], want[1][1:])
    cache.sparse_decode(ids, q, hq, groups, out, ws, lse)
    O.oscar_cache_check(cache.handle)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("value", [float("inf"), -float("inf"), float("nan")])
def test_a_value_that_is_not_finite(value, dtype, meta):
    """One channel of one token is not finite.  Lists without its group are not
    touched by it (the value factors are scaled by the largest finite value
    scale); with it an infinity costs its 32 channels only.  (A NaN leaves the
    quantiser's minimum and maximum alone and is stored as some code.)"""
    gen = torch.Generator().manual_seed(53)
    k, v = W.make_sequence_kv(1100, 2, W.LLAMA_RECIPE, gen)
    v = (8 * v.float()).bfloat16()
    v[300, 0, 37] = value
    cache = U.lib().OscarCache(1, 2, 1300, meta_bits=meta)
    U.append_all(cache, [0], [k], [v], chunk=4096)
    q = W.make_q(1, 8, seed=54).cuda()
    ws, arena = cache.workspace(1, 8), U.read_arena(cache)
    for idx in ([0, 1, 4, 7], [0, 2, 5], [2])[:1 if np.isnan(value) else 3]:
        groups = torch.tensor(idx, dtype=torch.int32).repeat(1, 2, 1).cuda()
        out, lse = torch.empty((1, 8, 128), dtype=dtype, device="cuda"), torch.empty((1, 8), device="cuda")
        cache.sparse_decode([0], q, 8, groups, out, ws, lse)
        U.lib().oscar_cache_check(cache.handle)
        got, gl = U.f64(out)[0], U.f64(lse)[0]
        for j in range(2):
            heads = slice(4 * j, 4 * j + 4)
            full = U.gpu_head(cache, arena, 0, j)
            if j == 0 and np.isinf(value):      # the token's second value group as zeros: 32 channels of no account
                assert not np.isfinite(full.values.scale * full.values.zero).all()
                full.values.scale[2, 44, 1] = full.values.zero[2, 44, 1] = 0
                assert np.isfinite(full.values.scale).all() and np.isfinite(full.values.zero).all()
            h, g = listed(full, idx), got[heads].copy()
            if j == 0 and 2 in idx:
                assert not np.isfinite(g[:, 32:64]).any()
                g[:, 32:64] = OR.history_attention(U.f64(q)[0, heads], h, None)[0][:, 32:64]
            check_head(U.f64(q)[0, heads], h, g, gl[heads], None, torch.finfo(dtype).eps / 2, full.values.scale.max())
