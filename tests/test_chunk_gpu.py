"""Attention within a chunk against the definition in 64 bits: documents,
prefixes, caps, distance biases, merged rows, layouts, and what hidden tokens
must not do."""
import math

import pytest
import torch

from tests import chunk_ref as C
from tests import gpu_util as U

pytestmark = pytest.mark.gpu

SLOPES = "slopes"


def cumulative(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def inputs(lens, hkv, gqa, seed, extra=0, layout="dense", prior=False):
    gen = torch.Generator().manual_seed(seed)
    n, hq = sum(lens) + extra, hkv * gqa
    q = torch.randn((n, hq, 128), generator=gen)
    k = torch.randn((n, hkv, 128), generator=gen) + 0.5 * torch.randn((1, hkv, 128), generator=gen)
    k[..., 5] *= 6.0
    v = torch.randn((n, hkv, 128), generator=gen)
    q, k, v = q.bfloat16().cuda(), k.bfloat16().cuda(), v.bfloat16().cuda()
    if layout == "fused":
        x = torch.cat([q, k, v], 1)
        q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    elif layout == "heads":          # [heads][tokens][128]
        q, k, v = (t.transpose(0, 1).contiguous().transpose(0, 1) for t in (q, k, v))
    p = None
    if prior:
        p = (torch.randn((n, hq, 128), generator=gen).mul(0.3).bfloat16().cuda(),
             (torch.randn((n, hq), generator=gen) + math.log(1 + n)).cuda())
        p[1][::3] = -math.inf
        p[0][::3] = float("nan")     # nothing before these rows: not read
    return q, k, v, p


def slopes_of(hq):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)]).cuda()


def call(O, lens, q, k, v, prior=None, stream=None, **kw):
    out = torch.full(tuple(q.shape), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(tuple(q.shape[:2]), 7.0, device="cuda")
    po, pl = prior if prior is not None else (None, None)
    O.oscar_chunk_attention(cumulative(lens), q, k, v, out, lse, prior_out=po, prior_lse=pl, stream=stream, **kw)
    torch.cuda.synchronize()
    return out, lse


def compare(lens, q, k, v, out, lse, prior=None, prefix=None, cap=0.0, slopes=None, softmax_scale=0.0):
    n = sum(lens)
    scale = softmax_scale or 1.0 / math.sqrt(128)
    want, wl, size = C.chunk(cumulative(lens), q[:n], k[:n], v[:n], prefix, cap, slopes,
                             None if prior is None else (prior[0][:n], prior[1][:n]), scale)
    fin = lambda t: torch.where(torch.isfinite(t), t, torch.zeros_like(t))  # noqa: E731
    es = C.score_error(fin(q[:n]), fin(k[:n]), scale, cap, slopes, max(lens))
    r = C.check(out[:n], lse[:n], want, wl, size, es)
    assert torch.all(out[n:] == 7.0) and torch.all(lse[n:] == 7.0)      # rows behind the last document
    return r


@pytest.mark.parametrize("lens", [[1], [5], [2, 1, 3], [31], [32], [33], [127], [128], [129], [0, 7, 0], [5] * 8,
                                  [255, 256, 257], [300, 1, 64, 700], [1000]])
def test_causal(lens):
    O = U.lib()
    q, k, v, _ = inputs(lens, 2, 4, seed=sum(lens))
    compare(lens, q, k, v, *call(O, lens, q, k, v))


@pytest.mark.parametrize("gqa", [1, 2, 3, 5, 6, 8, 12, 16, 130])
@pytest.mark.parametrize("hkv", [1, 3])
def test_head_groups(gqa, hkv):
    O = U.lib()
    lens = [77, 200] if gqa < 100 else [9, 4]
    q, k, v, prior = inputs(lens, hkv, gqa, seed=gqa, prior=True)
    compare(lens, q, k, v, *call(O, lens, q, k, v, prior), prior=prior)


@pytest.mark.parametrize("cap", [0.0, 30.0, 1.0])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("how", ["none", "some", "all"])
@pytest.mark.parametrize("prior", [False, True])
def test_rules(cap, bias, how, prior):
    O = U.lib()
    lens = [40, 513, 1, 0, 260]
    prefix = {"none": None, "some": [13, 129, 0, 0, 128], "all": list(lens)}[how]
    q, k, v, p = inputs(lens, 2, 4, seed=3, extra=5, layout="fused", prior=prior)
    slopes = slopes_of(8) if bias else None
    compare(lens, q, k, v, *call(O, lens, q, k, v, p, prefix=prefix, cap=cap, slopes=slopes), prior=p, prefix=prefix,
            cap=cap, slopes=slopes)


@pytest.mark.parametrize("layout", ["dense", "fused", "heads"])
@pytest.mark.parametrize("scale", [0.0, 0.25, 1e-3])
def test_layouts_and_scales(layout, scale):
    O = U.lib()
    lens = [150, 90]
    q, k, v, _ = inputs(lens, 4, 2, seed=5, extra=3, layout=layout)
    compare(lens, q, k, v, *call(O, lens, q, k, v, softmax_scale=scale), softmax_scale=scale)


def test_many_documents():
    """More documents than the small launch holds, empty ones among them, and as many as a call takes."""
    O = U.lib()
    lens = [(7 * i) % 23 for i in range(1024)]
    q, k, v, _ = inputs(lens, 1, 3, seed=6)
    compare(lens, q, k, v, *call(O, lens, q, k, v))


@pytest.mark.parametrize("cap", [2.0, 5.0, 8.0, 12.0, 18.0, 30.0, 60.0, 1000.0])
@pytest.mark.parametrize("lens", [[21], [333]])
def test_caps_near_and_far(cap, lens):
    """Scores of a few units under caps that they reach, come near and stay far from."""
    O = U.lib()
    q, k, v, _ = inputs(lens, 2, 4, seed=int(cap))
    compare(lens, q, k, v, *call(O, lens, q, k, v, cap=cap), cap=cap)
    q[::7] = (q[::7].float() * 4.0).bfloat16()          # rows of a warp in different ranges
    compare(lens, q, k, v, *call(O, lens, q, k, v, cap=cap), cap=cap)


@pytest.mark.parametrize("gqa", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_several_pieces_a_block(gqa, cap):
    """More pieces of work than SMs, of all lengths: each one's queries replace the last one's."""
    O = U.lib()
    lens = [33 + (37 * i) % 290 for i in range(40)]
    q, k, v, p = inputs(lens, 4, gqa, seed=20 + gqa, layout="fused", prior=True, extra=2)
    compare(lens, q, k, v, *call(O, lens, q, k, v, p, cap=cap), prior=p, cap=cap)


@pytest.mark.parametrize("gqa", [32, 64, 127, 128])
def test_many_heads_a_group(gqa):
    O = U.lib()
    lens = [40, 3, 71]
    q, k, v, _ = inputs(lens, 2, gqa, seed=gqa, layout="heads", extra=1)
    compare(lens, q, k, v, *call(O, lens, q, k, v))


def test_long_document():
    O = U.lib()
    lens = [5001]
    q, k, v, _ = inputs(lens, 1, 2, seed=7)
    compare(lens, q, k, v, *call(O, lens, q, k, v))


def test_growing_maxima():
    """Keys that grow along the document: the maxima in use are replaced in many steps."""
    O = U.lib()
    lens = [1500]
    q, k, v, _ = inputs(lens, 1, 4, seed=8)
    k = (k.float() * torch.linspace(0.1, 6.0, 1500, device="cuda")[:, None, None]).bfloat16()
    compare(lens, q, k, v, *call(O, lens, q, k, v))
    q = q.abs()
    k = (k.abs() * 0.2).bfloat16()      # every score larger than those before
    compare(lens, q, k, v, *call(O, lens, q, k, v, cap=50.0), cap=50.0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_hidden_tokens_have_no_part(value):
    """Whatever keys and values hold that a token does not see: later tokens, other documents, rows behind."""
    O = U.lib()
    lens = [70, 150, 33]
    q, k, v, _ = inputs(lens, 2, 4, seed=9, extra=40)
    clean = call(O, lens, q, k, v)
    for name, rows in [("the rows behind the last document", slice(253, 293)), ("another document", slice(70, 220)),
                       ("later tokens", slice(60, 70))]:
        k2, v2 = k.clone(), v.clone()
        k2[rows] = value
        v2[rows] = value
        out, lse = call(O, lens, q, k2, v2)
        keep = torch.ones(253, dtype=torch.bool)
        keep[rows] = False
        assert torch.equal(out[:253][keep], clean[0][:253][keep]), name
        assert torch.equal(lse[:253][keep], clean[1][:253][keep]), name


@pytest.mark.parametrize("where", [0, 3, 64, 127, 128, 200])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_visible_values_that_are_not_finite(where, value):
    """A value that is not finite spoils its channel of the rows that see it, no other."""
    O = U.lib()
    lens = [260]
    q, k, v, _ = inputs(lens, 2, 3, seed=10)
    v[where, 1, 7] = value
    v[min(where + 1, 259), 1, 9] = -value
    out, lse = call(O, lens, q, k, v)
    compare(lens, q, k, v, out, lse)
    assert torch.isfinite(out[:, :3].float()).all() and torch.isfinite(out[:where].float()).all()


def test_a_key_that_is_not_finite():
    O = U.lib()
    lens = [200]
    q, k, v, _ = inputs(lens, 1, 2, seed=11)
    clean = call(O, lens, q, k, v)
    k[150, 0, 3] = float("nan")
    out, lse = call(O, lens, q, k, v)
    assert torch.equal(out[:150], clean[0][:150]) and torch.equal(lse[:150], clean[1][:150])
    assert torch.isnan(out[150:].float()).all() and torch.isnan(lse[150:]).all()


def test_large_scores():
    """Scores of thousands: one key has all the weight."""
    O = U.lib()
    lens = [300]
    q, k, v, _ = inputs(lens, 1, 4, seed=12)
    q = (q.float() * 60).bfloat16()
    out, lse = call(O, lens, q, k, v)
    compare(lens, q, k, v, out, lse)


def test_merge_in_place():
    O = U.lib()
    lens = [100, 29]
    q, k, v, p = inputs(lens, 2, 4, seed=13, prior=True)
    out, lse = call(O, lens, q, k, v, p)
    O.oscar_chunk_attention(cumulative(lens), q, k, v, p[0], p[1], prior_out=p[0], prior_lse=p[1])
    torch.cuda.synchronize()
    assert torch.equal(p[0], out) and torch.equal(p[1], lse)


def test_without_lse_and_repeated():
    """The same bits every time, with and without the log-sum-exp."""
    O = U.lib()
    lens = [700, 300]
    q, k, v, _ = inputs(lens, 2, 4, seed=14)
    first = call(O, lens, q, k, v)
    out = torch.empty_like(q)
    for _ in range(5):
        O.oscar_chunk_attention(cumulative(lens), q, k, v, out)
        torch.cuda.synchronize()
        assert torch.equal(out, first[0])


def test_captured_and_on_another_stream():
    O = U.lib()
    lens = [90, 260]
    q, k, v, p = inputs(lens, 2, 4, seed=15, prior=True)
    want = call(O, lens, q, k, v, p, cap=20.0)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], device="cuda")
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        O.oscar_chunk_attention(cumulative(lens), q, k, v, out, lse, cap=20.0, prior_out=p[0], prior_lse=p[1])
    q2 = (q.float() * 0.5).bfloat16()
    want2 = call(O, lens, q2, k, v, p, cap=20.0, stream=s)
    for x, w in ((q.clone(), want), (q2, want2)):
        q.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_two_streams_at_once():
    O = U.lib()
    jobs = []
    for i in range(4):
        lens = [600 + 10 * i, 40]
        q, k, v, _ = inputs(lens, 4, 4, seed=20 + i)
        jobs.append((lens, q, k, v, call(O, lens, q, k, v), torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for lens, q, k, v, _, out, s in jobs:
        O.oscar_chunk_attention(cumulative(lens), q, k, v, out, stream=s)
    torch.cuda.synchronize()
    for _, _, _, _, want, out, _ in jobs:
        assert torch.equal(out, want[0])


def test_right_after_the_kernel_that_makes_its_inputs():
    """Enqueued behind a busy stream: the launch may start early, its reads must not."""
    O = U.lib()
    cfg = O.make_rotary_config(128)
    lens = [300]
    q, k, v, _ = inputs(lens, 2, 4, seed=16)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    qr, kr, out = torch.zeros_like(q), torch.zeros_like(k), torch.empty_like(q)
    O.oscar_rotary(cfg, pos, q, k, qr, kr)
    torch.cuda.synchronize()
    want = call(O, lens, qr, kr, v)[0]
    for _ in range(10):
        qr.zero_()
        kr.zero_()
        torch.cuda.synchronize()
        torch.cuda._sleep(1 << 20)
        O.oscar_rotary(cfg, pos, q, k, qr, kr)
        O.oscar_chunk_attention([0, 300], qr, kr, v, out)
        O.oscar_rotary(cfg, pos, q, k, kr.new_empty(q.shape), kr.new_empty(k.shape))
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals_on_the_device():
    O = U.lib()
    q, k, v, p = inputs([20], 2, 4, seed=17, prior=True)
    out = torch.full_like(q, 7.0)

    def refused(status, **kw):
        args = dict(cu=[0, 20], q=q, k=k, v=v, out=out, lse=None, prior=(None, None), slopes=None, cap=0.0, scale=0.0,
                    prefix=None)
        args.update(kw)
        with pytest.raises((O.OscarError, ValueError)) as e:
            O.oscar_chunk_attention(args["cu"], args["q"], args["k"], args["v"], args["out"], args["lse"],
                                    prefix=args["prefix"], cap=args["cap"], slopes=args["slopes"],
                                    prior_out=args["prior"][0], prior_lse=args["prior"][1], softmax_scale=args["scale"])
        if status is not None:
            assert e.value.status == status
        torch.cuda.synchronize()
        assert torch.all(out == 7.0)

    refused(1, out=q)                                       # out over q
    both = torch.empty((40, 8, 128), dtype=torch.bfloat16, device="cuda")
    refused(1, out=both[:20], prior=(both[1:21], p[1]))     # out over a shifted prior
    refused(1, q=q.cpu())                                   # pageable host memory
    refused(1, k=k[:, :1].expand(20, 2, 128))               # a stride of 0
    odd = torch.empty(20 * 2 * 128 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(20, 2, 128)
    refused(1, k=odd)                                       # 8-byte aligned
    host = torch.empty((20, 8, 128), dtype=torch.bfloat16)
    refused(1, out=host)
    refused(1, slopes=torch.zeros(8))                       # pageable
    refused(None, slopes=torch.zeros(7, device="cuda"))
    ok = torch.empty((20, 8, 128), dtype=torch.bfloat16).pin_memory()
    O.oscar_chunk_attention([0, 20], q, k, v, ok)
    torch.cuda.synchronize()
    assert torch.equal(ok.cuda(), call(O, [20], q, k, v)[0])


@pytest.mark.parametrize("n", [20, 40])
def test_overlapping_buffers_are_refused(n):
    O = U.lib()
    q, k, v, p = inputs([n], 2, 4, seed=18, prior=True)
    out = torch.full_like(q, 7.0)

    def refused(**kw):
        with pytest.raises(O.OscarError, match="overlap"):
            O.oscar_chunk_attention(**{**dict(cu_seqlens=[0, n], q=q, k=k, v=v, out=out), **kw})

    inside = lambda t: t.view(-1).view(torch.float32)[:n * 8].view(n, 8)  # noqa: E731
    for t in (q, k, v, out):
        refused(lse=inside(t))
    refused(prior_out=p[0], prior_lse=p[1], lse=inside(p[0]))
    refused(prior_out=p[0], prior_lse=inside(out))
    both = torch.empty((n + 1, 8), device="cuda")
    refused(prior_out=p[0], prior_lse=both[1:], lse=both[:n])
    torch.cuda.synchronize()
    assert torch.all(out == 7.0)


# ---- documents of at most 32 tokens have a kernel of their own

@pytest.mark.parametrize("cap,bias", [(0.0, False), (30.0, True), (1.0, False)])
@pytest.mark.parametrize("gqa", [1, 4, 5, 16, 33])
@pytest.mark.parametrize("prior", [False, True])
def test_short_documents(gqa, cap, bias, prior):
    O = U.lib()
    lens = [5, 32, 1, 0, 17, 8, 9, 16, 31, 24]
    prefix = [0, 32, 1, 0, 16, 3, 9, 15, 0, 20]
    q, k, v, p = inputs(lens, 3, gqa, seed=40 + gqa, extra=2, layout="fused", prior=prior)
    slopes = slopes_of(3 * gqa) if bias else None
    compare(lens, q, k, v, *call(O, lens, q, k, v, p, cap=cap, slopes=slopes), prior=p, cap=cap, slopes=slopes)
    compare(lens, q, k, v, *call(O, lens, q, k, v, p, prefix=prefix, cap=cap, slopes=slopes), prior=p, prefix=prefix,
            cap=cap, slopes=slopes)


def test_short_documents_beside_a_longer_one():
    """The longest document chooses the kernel: the same rows either way, within both bounds."""
    O = U.lib()
    lens = [5, 20, 32]
    q, k, v, _ = inputs(lens + [40], 2, 4, seed=60)
    compare(lens, q[:57], k[:57], v[:57], *call(O, lens, q[:57], k[:57], v[:57]))
    compare(lens + [40], q, k, v, *call(O, lens + [40], q, k, v))


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_short_hidden_tokens_have_no_part(value):
    O = U.lib()
    lens = [11, 6, 32]
    q, k, v, _ = inputs(lens, 2, 4, seed=61, extra=9)
    clean = call(O, lens, q, k, v)
    for rows in (slice(49, 58), slice(11, 17), slice(5, 11), slice(30, 49)):
        k2, v2 = k.clone(), v.clone()
        k2[rows] = value
        v2[rows] = value
        out, lse = call(O, lens, q, k2, v2)
        keep = torch.ones(49, dtype=torch.bool)
        keep[rows] = False
        # (the rows of a document with such a token are summed in another order)
        assert (out[:49][keep].float() - clean[0][:49][keep].float()).abs().max() <= 2.0 ** -7 * 4
        assert torch.equal(lse[:49][keep], clean[1][:49][keep])


@pytest.mark.parametrize("where", [0, 7, 8, 31])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_short_visible_values_that_are_not_finite(where, value):
    O = U.lib()
    lens = [32, 3]
    q, k, v, _ = inputs(lens, 2, 3, seed=62)
    v[where, 1, 7] = value
    out, lse = call(O, lens, q, k, v)
    compare(lens, q, k, v, out, lse)
    assert torch.isfinite(out[:, :3].float()).all() and torch.isfinite(out[:where].float()).all()


def test_short_merge_in_place_captured():
    O = U.lib()
    lens = [5] * 8
    q, k, v, p = inputs(lens, 2, 4, seed=63, prior=True)
    want = call(O, lens, q, k, v, p)
    keep = p[0].clone(), p[1].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O.oscar_chunk_attention(cumulative(lens), q, k, v, p[0], p[1], prior_out=p[0], prior_lse=p[1])
    for _ in range(2):
        p[0].copy_(keep[0])
        p[1].copy_(keep[1])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(p[0], want[0]) and torch.equal(p[1], want[1])


@pytest.mark.parametrize("lens", [[33], [700, 300], [5000], [64] * 500])
@pytest.mark.parametrize("gqa", [3, 4])
def test_a_wait_that_gives_up(lens, gqa):
    """One copy of the first CTA left out: the call ends, rows that were not computed are NaN, the others are right,
    and the next call is unaffected."""
    O = U.lib()
    q, k, v, _ = inputs(lens, 2, gqa, seed=70)
    want = call(O, lens, q, k, v)
    O.oscar_test_arm_wait_timeout()
    out, lse = call(O, lens, q, k, v)
    gone = torch.isnan(lse)
    assert gone.any() and torch.equal(gone, torch.isnan(out.float()).all(-1))
    assert torch.equal(gone, torch.isnan(out.float()).any(-1))
    assert torch.equal(out[~gone], want[0][~gone]) and torch.equal(lse[~gone], want[1][~gone])
    again = call(O, lens, q, k, v)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
