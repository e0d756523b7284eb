"""The operators as a serving loop uses them together, against 64 bits: a prompt
taken over by forks, a chunk of new tokens (its queries over the cache, its own
attention, merged), its tokens appended, steps decoded under the same rule, the
cache pruned."""
import math

import numpy as np
import pytest
import torch

from int2_kv_cache_oscar_gb300 import workloads as W
from oracle import oscar_oracle as OR
from tests import chunk_ref as C
from tests import gpu_util as U
from tests import test_scored_gpu as SC

pytestmark = pytest.mark.gpu


def cached_rows(cache, slot):
    """The slot's keys and values as float64 rows [tokens, hkv, 128] (keys in their own basis)."""
    O, n = U.lib(), cache.length(slot)
    arena = U.read_arena(cache)
    ks, vs = [], []
    for j in range(cache.num_kv_heads):
        h = U.gpu_head(cache, arena, slot, j)
        parts = []
        if h.num_groups:
            unit = OR.dequant_keys(h.keys) * h.keys.norm.astype(np.float64)[..., None]
            parts.append(OR.canalized_rotation(unit.reshape(-1, 128)))       # its own inverse
        parts.append(h.window_k)
        ks.append(np.concatenate(parts))
        vs.append(OR.decode_values(h))
    assert ks[0].shape[0] == n
    return torch.from_numpy(np.stack(ks, 1)), torch.from_numpy(np.stack(vs, 1))


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (25.0, False), (0.0, True), (25.0, True)])
@pytest.mark.parametrize("new", [5, 150])
def test_forked_prompts_chunks_and_steps(meta, cap, bias, new):
    O = U.lib()
    hkv, gqa, prompt = 2, 4, 700
    hq = hkv * gqa
    gen = torch.Generator().manual_seed(21 + new)
    k, v = W.make_sequence_kv(prompt, hkv, W.LLAMA_RECIPE, gen)
    cache = O.OscarCache(4, hkv, 1200, meta_bits=meta)
    cache.append([0], [0, prompt], k.cuda(), v.cuda())
    take = [700, 650, 128]                  # the whole prompt, one cut in a group, one at a group's end
    cache.fork([0, 0, 0], [1, 2, 3], take)
    slopes = SC.slopes_of(hq).cuda() if bias else None
    rule = dict(cap=cap, slopes=slopes)
    lens = [new, new - 2, new - 4]
    cu = [0, lens[0], lens[0] + lens[1], sum(lens)]
    n = cu[-1]
    x = torch.randn((n, hq + 2 * hkv, 128), generator=gen).bfloat16().cuda()
    q, kn, vn = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    qd = q.contiguous()
    out, lse = torch.empty((n, hq, 128), dtype=torch.bfloat16, device="cuda"), torch.empty((n, hq), device="cuda")
    before = [cached_rows(cache, s) for s in (1, 2, 3)]
    for i, s in enumerate((1, 2, 3)):
        cache.scored_prefill(s, qd[cu[i]:cu[i + 1]], hq, out[cu[i]:cu[i + 1]], lse[cu[i]:cu[i + 1]], **rule)
    O.oscar_chunk_attention(cu, q, kn, vn, out, lse, prior_out=out, prior_lse=lse, **rule)
    torch.cuda.synchronize()
    O.oscar_cache_check(cache.handle)
    scale = 1 / math.sqrt(128)
    for i in range(3):
        a, e = cu[i], cu[i + 1]
        kk = torch.cat([before[i][0], kn[a:e].double().cpu()]).repeat_interleave(gqa, 1)
        vv = torch.cat([before[i][1], vn[a:e].double().cpu()]).repeat_interleave(gqa, 1)
        L, m = take[i], e - a
        s = torch.einsum("ihc,thc->hit", q[a:e].double().cpu(), kk) * scale
        at, pos = torch.arange(L + m), L + torch.arange(m)
        s = C.rule(s, (pos[:, None] - at[None]).abs().double(), cap, None if slopes is None else slopes.cpu())
        s = s.masked_fill(at[None, None] > pos[None, :, None], -math.inf)
        p = torch.softmax(s, -1)
        want, size = torch.einsum("hit,thc->ihc", p, vv), torch.einsum("hit,thc->ihc", p, vv.abs())
        es = C.score_error(q[a:e], torch.cat([before[i][0].cuda(), kn[a:e].double()]), scale, cap, slopes, L + m)
        # the history's rows are rounded to bf16 once more before they are merged, and
        # its scores are off by 2^-16 of their absolute sums at most
        es += 2.0 ** -16 * float(q.abs().double().amax()) * float(kk.abs().sum(-1).amax()) * scale
        tol = 2.0 ** -8 * want.abs() + (2.1 * 2.0 ** -8 + 2 * es + 2.0 ** -16) * size
        err = (out[a:e].double().cpu() - want).abs()
        assert bool((err <= tol).all()), float((err / tol).max())
        total = torch.logsumexp(s, -1).T
        assert bool(((lse[a:e].double().cpu() - total).abs() <= es + 2.0 ** -19 * (1 + total.abs())).all())
    cache.append([1, 2, 3], cu, kn.contiguous(), vn.contiguous())
    for i, s in enumerate((1, 2, 3)):
        assert cache.length(s) == take[i] + lens[i]
    SC.check_decode(cache, [3, 1, 2], W.make_q(3, hq, seed=30).cuda(), cap, None if slopes is None else slopes.cpu())
    # drafted tokens are taken back, the oldest groups but the first go
    cache.truncate([1, 2, 3], [take[i] + max(1, lens[i] - 3) for i in range(3)])
    cache.keep_groups([1], [[0] + list(range(3, cache.length(1) // 128))])
    SC.check_decode(cache, [1, 2, 3], W.make_q(3, hq, seed=31).cuda(), cap, None if slopes is None else slopes.cpu())
    SC.check_decode(cache, [0], W.make_q(1, hq, seed=32).cuda())


def test_queued_calls_match_waited_ones():
    """Every call enqueued behind a busy stream against the same calls with a wait
    after each: the same bits."""
    O = U.lib()
    hkv, hq = 2, 8
    gen = torch.Generator().manual_seed(41)
    k, v = W.make_sequence_kv(900, hkv, W.LLAMA_RECIPE, gen)
    steps = [torch.randn((3 * 7, hq + 2 * hkv, 128), generator=gen).bfloat16().cuda() for _ in range(4)]
    slopes = SC.slopes_of(hq).cuda()

    def run(queued):
        cache = O.OscarCache(5, hkv, 1500)
        cache.append([0], [0, 900], k.cuda(), v.cuda())
        ids, made = [1, 2, 3], []
        ws = cache.workspace(3, hq)
        torch.cuda.synchronize()
        if queued:
            torch.cuda._sleep(1 << 22)

        def call(f):
            f()
            if not queued:
                torch.cuda.synchronize()

        call(lambda: cache.fork([0, 0, 0], ids, [900, 800, 256]))
        for x in steps:
            q, kn, vn = x[:, :hq].contiguous(), x[:, hq:hq + hkv].contiguous(), x[:, hq + hkv:].contiguous()
            new = lambda dtype=torch.bfloat16, *s: torch.zeros(s, dtype=dtype, device="cuda")  # noqa: E731
            out, lse, one = new(torch.bfloat16, 21, hq, 128), new(torch.float32, 21, hq), new(torch.float32, 3, hq, 128)
            for i, s in enumerate(ids):
                call(lambda: cache.scored_prefill(s, q[7 * i:7 * i + 7], hq, out[7 * i:7 * i + 7], lse[7 * i:7 * i + 7],
                                                  cap=20.0, slopes=slopes))
            call(lambda: O.oscar_chunk_attention([0, 7, 14, 21], q, kn, vn, out, lse, prior_out=out, prior_lse=lse, cap=20.0,
                                                 slopes=slopes))
            call(lambda: cache.append(ids, [0, 7, 14, 21], kn, vn))
            call(lambda: cache.scored_decode(ids, q[:3].contiguous(), hq, one, ws, cap=20.0, slopes=slopes))
            call(lambda: cache.truncate([2], [cache.length(2) - 5]))
            call(lambda: cache.keep_groups([1], [[0] + list(range(2, cache.length(1) // 128))]))
            call(lambda: cache.fork([3], [4]))
            call(lambda: cache.scored_decode([4, 1, 2], q[3:6].contiguous(), hq, one, ws, slopes=slopes))
            made += [out, lse, one]
        torch.cuda.synchronize()
        O.oscar_cache_check(cache.handle)
        return made

    for a, b in zip(run(True), run(False)):
        assert torch.equal(a, b)
