"""The operators as a serving loop uses them: rotate the step's queries and
keys, append, bring the index up to date, choose groups, attend over them, and
read the sequence back; against the same steps in float64 on the library's own
intermediate results."""
import numpy as np
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from oracle import oscar_oracle as OR
from tests import gpu_util as U
from tests import test_read_gpu as R
from tests import test_rotary_gpu as ROT
from tests import test_select_gpu as SEL
from tests import test_sparse_gpu as SP

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("meta", [32, 16])
def test_serving_loop(meta):
    O = U.lib()
    hkv, hq, keep = 2, 8, 6
    lens = [1500, 383, 90]
    gen = torch.Generator().manual_seed(81)
    cfg = O.make_rotary_config(128, base=500000.0, scaling="banded", factor=8.0, original_length=8192)
    cache = O.OscarCache(3, hkv, 2000, meta_bits=meta)
    cache.enable_index()
    for i, n in enumerate(lens):           # prefill: rotated keys, appended
        k, v = W.make_sequence_kv(n, hkv, W.LLAMA_RECIPE, gen)
        k = k.cuda()
        O.oscar_rotary(cfg, torch.arange(n, dtype=torch.int32).cuda(), k)
        cache.append([i], [0, n], k, v.cuda())
    ids = [0, 1, 2]
    ws = cache.workspace(3, hq)
    for step in range(3):                  # the second sequence closes a group at the first step
        qkv = torch.randn((3, hq + 2 * hkv, 128), generator=gen).bfloat16().cuda()
        raw = qkv.clone()
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        pos = torch.tensor([cache.length(i) for i in ids], dtype=torch.int32).cuda()
        qr = torch.empty((3, hq, 128), dtype=torch.bfloat16, device="cuda")
        kr = torch.empty((3, hkv, 128), dtype=torch.bfloat16, device="cuda")
        O.oscar_rotary(cfg, pos, q, k, qr, kr)
        ROT.check(cfg, pos, raw[:, :hq], qr)
        ROT.check(cfg, pos, raw[:, hq:hq + hkv], kr)
        cache.append(ids, [0, 1, 2, 3], kr, v.contiguous())
        cache.update_index(ids)
        groups = torch.empty((3, hkv, keep), dtype=torch.int32, device="cuda")
        cache.select_groups(ids, qr, hq, groups, keep_first=1, keep_last=1)
        out = torch.empty((3, hq, 128), dtype=torch.bfloat16, device="cuda")
        cache.sparse_decode(ids, qr, hq, groups, out, ws)
        torch.cuda.synchronize()
        SEL.check(cache, ids, qr, keep, 1, 1)
        again, _ = SP.check(cache, ids, qr, groups, torch.bfloat16)
        assert torch.equal(again, out)
    R.check(cache, ids, [0, 100, 0], [cache.length(i) for i in ids], torch.bfloat16)
    # attention over the read-back rows is the attention over the packed cache
    n = cache.length(0)
    k, v = (torch.empty((n, hkv, 128), device="cuda") for _ in range(2))
    cache.read([0], [0], [n], k, v)
    full = torch.empty((1, hq, 128), device="cuda")
    cache.decode_f32([0], qr[:1].contiguous(), hq, full, ws)
    for j in range(hkv):
        s = U.f64(qr)[0, 4 * j:4 * j + 4] @ U.f64(k)[:, j].T / np.sqrt(128)
        ref = OR.softmax_attend(s.T, U.f64(v)[:, j])
        assert np.abs(ref - U.f64(full)[0, 4 * j:4 * j + 4]).max() <= 2e-3     # the decode's own bound


@pytest.mark.parametrize("how", ["all", "listed", "fused"])
def test_short_sequences_right_after_rotation(how):
    """Sequences without a group: the window is attended by the only kernel of
    the decode, which must not read queries (or a new token) before the rotation
    has written them."""
    O = U.lib()
    n, hkv, hq, steps = 16, 8, 32, 24
    gen = torch.Generator().manual_seed(82)
    cfg = O.make_rotary_config(128)
    k, v = (torch.randn((n * 90, hkv, 128), generator=gen).bfloat16().cuda() for _ in range(2))
    cu, ids = [90 * i for i in range(n + 1)], list(range(n))
    caches = [O.OscarCache(n, hkv, 128) for _ in range(2)]
    for c in caches:
        c.append(ids, cu, k, v)
    ws = caches[0].workspace(n, hq)
    groups = torch.zeros((n, hkv, 1), dtype=torch.int32, device="cuda")
    v_new = torch.randn((n, hkv, 128), generator=gen).bfloat16().cuda()

    def step(cache, q, k_new, wait):
        qr, kr = torch.zeros_like(q), torch.zeros_like(k_new)
        out = torch.zeros_like(q)
        torch.cuda.synchronize()
        torch.cuda._sleep(1 << 20)         # both launches are enqueued before the first one runs
        O.oscar_rotary(cfg, pos, q, k_new, qr, kr)
        if wait:
            torch.cuda.synchronize()
        if how == "all":
            cache.decode(ids, qr, hq, out, ws)
        elif how == "listed":
            cache.sparse_decode(ids, qr, hq, groups, out, ws)
        else:
            cache.append_decode(ids, kr, v_new, qr, hq, out, ws)
        torch.cuda.synchronize()
        return out

    for i in range(steps):
        pos = torch.full((n,), 7 * i, dtype=torch.int32, device="cuda")
        q = torch.randn((n, hq, 128), generator=gen).bfloat16().cuda()
        k_new = torch.randn((n, hkv, 128), generator=gen).bfloat16().cuda()
        assert torch.equal(step(caches[0], q, k_new, False), step(caches[1], q, k_new, True)), i


@pytest.mark.parametrize("meta", [32, 16])
def test_queued_calls_match_waited_ones(meta):
    """Every call of the loop enqueued behind a busy stream, so that each kernel
    may start while the one before it finishes, against the same calls with a
    wait after each: the same bits."""
    O = U.lib()
    hkv, hq, keep = 2, 8, 3
    lens = [700, 383, 90, 127, 255]
    n, ids = len(lens), list(range(len(lens)))
    gen = torch.Generator().manual_seed(83)
    cfg = O.make_rotary_config(96, interleaved=True, scaling="yarn", factor=4.0, original_length=4096)
    kv = [W.make_sequence_kv(m, hkv, W.LLAMA_RECIPE, gen) for m in lens]
    steps = [torch.randn((n, hq + 2 * hkv, 128), generator=gen).bfloat16().cuda() for _ in range(6)]

    def run(queued):
        cache = O.OscarCache(n, hkv, 1200, meta_bits=meta)
        cache.enable_index()
        for i, (k, v) in enumerate(kv):
            cache.append([i], [0, lens[i]], k.cuda(), v.cuda())
        cache.update_index(ids)
        ws, made = cache.workspace(n, hq), []
        for step, x in enumerate(steps):
            pos = torch.tensor([cache.length(i) for i in ids], dtype=torch.int32).cuda()
            q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:].contiguous()
            new = lambda *shape, dtype=torch.bfloat16: torch.zeros(shape, dtype=dtype, device="cuda")
            qr, kr, out, dense, fused = new(n, hq, 128), new(n, hkv, 128), new(n, hq, 128), new(n, hq, 128), new(n, hq, 128)
            groups, lse = new(n, hkv, keep, dtype=torch.int32), new(n, hq, dtype=torch.float32)
            tail = [cache.length(i) - 50 for i in ids]
            rows = [new(50 * n + n, hkv, 128, dtype=torch.float32) for _ in range(2)]
            calls = [lambda: O.oscar_rotary(cfg, pos, q, k, qr, kr),
                     lambda: cache.append(ids, list(range(n + 1)), kr, v),
                     lambda: cache.update_index(ids),
                     lambda: cache.select_groups(ids, qr, hq, groups, keep_last=1),
                     lambda: cache.sparse_decode(ids, qr, hq, groups, out, ws, lse=lse),
                     lambda: O.oscar_rotary(cfg, pos, qr, transpose=True),
                     lambda: cache.decode(ids, qr, hq, dense, ws),
                     lambda: O.oscar_rotary(cfg, pos, kr),
                     lambda: cache.append_decode(ids, kr, v, qr, hq, fused, ws),
                     lambda: cache.read(ids, tail, [t + 51 for t in tail], *rows),
                     lambda: cache.update_index(ids)]
            torch.cuda.synchronize()
            if queued:
                torch.cuda._sleep(1 << 22)
            for call in calls:
                call()
                if not queued:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            O.oscar_cache_check(cache.handle)
            made += [qr, kr, groups, out, lse, dense, fused, *rows]
        return made

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)


def test_the_cache_s_kv_heads_are_checked_by_every_form_of_a_call():
    """Buffers for another number of KV heads are refused by the functions and
    by the methods (the kernels would run past them): nothing is enqueued."""
    O = U.lib()
    gen = torch.Generator().manual_seed(71)
    k, v = W.make_sequence_kv(700, 4, W.LLAMA_RECIPE, gen)
    cache = O.OscarCache(1, 4, 1000)
    U.append_all(cache, [0], [k], [v])
    cache.enable_index()
    cache.update_index([0])
    assert O.oscar_cache_get_config(cache.handle).num_kv_heads == 4
    q, out = W.make_q(1, 8, seed=72).cuda(), torch.full((1, 8, 128), 7.0, device="cuda")
    ws = cache.workspace(1, 8)
    for heads in (1, 2, 3, 5, 8):
        rows = torch.full((700, heads, 128), 7.0, device="cuda")
        groups = torch.full((1, heads, 3), 7, dtype=torch.int32, device="cuda")
        right = torch.empty((700, 4, 128), device="cuda")
        for call in [lambda: O.oscar_cache_read(cache.handle, [0], [0], [700], rows, None),
                     lambda: O.oscar_cache_read(cache.handle, [0], [0], [700], right, rows),
                     lambda: O.oscar_cache_read(cache.handle, [0], [0], [700], rows, None, num_kv_heads=heads),
                     lambda: cache.read([0], [0], [700], None, rows),
                     lambda: O.oscar_select_groups(cache.handle, [0], q, 8, groups),
                     lambda: O.oscar_select_groups(cache.handle, [0], q, 8, groups, num_kv_heads=heads),
                     lambda: cache.select_groups([0], q, 8, groups),
                     lambda: O.oscar_sparse_decode_attention(cache.handle, [0], q, 8, 0.0, groups, out, ws),
                     lambda: O.oscar_sparse_decode_attention(cache.handle, [0], q, 8, 0.0, groups, out, ws,
                                                             num_kv_heads=heads),
                     lambda: cache.sparse_decode([0], q, 8, groups, out, ws)]:
            with pytest.raises(ValueError, match="KV heads"):
                call()
        torch.cuda.synchronize()
        assert torch.all(rows == 7.0) and torch.all(groups == 7) and torch.all(out == 7.0)
    O.oscar_cache_read(cache.handle, [0], [0], [700], right, None)
    groups = torch.zeros((1, 4, 3), dtype=torch.int32, device="cuda")
    O.oscar_select_groups(cache.handle, [0], q, 8, groups, num_kv_heads=4)
    O.oscar_cache_check(cache.handle)
