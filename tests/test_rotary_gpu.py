"""Rotary positions against the formula in 64 bits.

Error of one output (float32 arithmetic): cosine and sine 2 ulp (2^-22 of at
most 1, twice 2^-24 more for the phase's rounding to float32 and the attention
factor), two products and a sum: together at most 9 * 2^-24 (|x_a| + |x_b|) m;
the output type rounds by half a step of the result."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import gpu_util as U

pytestmark = pytest.mark.gpu

PI = Fraction(31415926535897932384626433832795028841971693993751058209749445923, 10 ** 64)
F32 = 9 * 2.0 ** -24


def wave(cfg, pos, transpose):
    """cos, sin [n, pairs] with the angle reduced exactly (rational arithmetic)."""
    f, m = U.lib().oscar_rotary_frequencies(cfg)
    turns = [Fraction(x) / (2 * PI) for x in f]
    a = np.array([[float((int(p) * t) % 1) for t in turns] for p in pos]).reshape(len(pos), len(f)) * 2 * math.pi
    return np.cos(a) * m, np.sin(a) * (-m if transpose else m), m


def reference(cfg, pos, x, transpose):
    """(y, bound of the float32 arithmetic) of x [n, heads, 128] in float64."""
    c, s, m = wave(cfg, pos, transpose)
    dim = cfg.rotary_dim
    a, b = (slice(0, dim, 2), slice(1, dim, 2)) if cfg.interleaved else (slice(0, dim // 2), slice(dim // 2, dim))
    y, bound = x.copy(), np.zeros_like(x)
    c, s = c[:, None], s[:, None]
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    e = F32 * m * (np.abs(x[..., a]) + np.abs(x[..., b]))
    bound[..., a], bound[..., b] = e, e
    return y, bound


def check(cfg, pos, x, got, transpose=False, what=""):
    ref, bound = reference(cfg, pos.cpu().numpy(), U.f64(x), transpose)
    half = torch.finfo(got.dtype).eps / 2
    bound = bound + half * (np.abs(ref) + bound)
    err = np.abs(U.f64(got) - ref)
    assert np.all(err <= bound), f"{what}: {np.max(err / np.maximum(bound, 1e-300)):.2f} of the bound"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,n,hq,hkv", [(128, 1, 32, 8), (128, 17, 4, 1), (64, 130, 3, 1), (16, 5, 1, 1),
                                          (96, 33, 8, 2), (112, 700, 2, 2), (128, 1, 130, 3), (32, 3000, 1, 1)])
def test_matches_the_formula(dtype, interleaved, dim, n, hq, hkv):
    O = U.lib()
    g = torch.Generator().manual_seed(dim + n)
    q = torch.randn((n, hq, 128), generator=g).to(dtype).cuda()
    k = torch.randn((n, hkv, 128), generator=g).to(dtype).cuda()
    pos = torch.randint(0, 131072, (n,), generator=g, dtype=torch.int32).cuda()
    cfg = O.make_rotary_config(dim, base=500000.0, interleaved=interleaved, scaling="banded", factor=8.0,
                               original_length=8192)
    for transpose in (False, True):
        qo, ko = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
        O.oscar_rotary(cfg, pos, q, k, qo, ko, transpose=transpose)
        check(cfg, pos, q, qo, transpose, "q")
        check(cfg, pos, k, ko, transpose, "k")
    if dim < 128:   # the channels behind the rotated ones are copied
        assert torch.equal(qo[..., dim:], q[..., dim:])


@pytest.mark.parametrize("scaling", ["none", "linear", "yarn"])
def test_scalings_and_far_positions(scaling):
    """Positions up to the ends of int32, negative ones too."""
    O = U.lib()
    pos = torch.tensor([0, 1, -1, 131071, -131072, 2 ** 31 - 1, -2 ** 31, 1 << 30, 12345678], dtype=torch.int32).cuda()
    x = torch.randn((9, 2, 128), generator=torch.Generator().manual_seed(3)).cuda()
    cfg = O.make_rotary_config(128, scaling=scaling, factor=4.0, original_length=4096)
    y = torch.empty_like(x)
    O.oscar_rotary(cfg, pos, x, None, y)
    check(cfg, pos, x, y, what=scaling)


def test_strides_in_place_and_broadcast():
    O = U.lib()
    g = torch.Generator().manual_seed(9)
    cfg = O.make_rotary_config(128)
    n = 37
    pos = torch.arange(100, 100 + n, dtype=torch.int32).cuda()
    # q and k inside a fused projection, in place; v keeps its bytes
    qkv = torch.randn((n, 12, 128), generator=g).bfloat16().cuda()
    before = qkv.clone()
    O.oscar_rotary(cfg, pos, qkv[:, :8], qkv[:, 8:10])
    check(cfg, pos, before[:, :8], qkv[:, :8], what="in place q")
    check(cfg, pos, before[:, 8:10], qkv[:, 8:10], what="in place k")
    assert torch.equal(qkv[:, 10:], before[:, 10:])
    # heads outside tokens, in and out, and tokens in reverse
    x = torch.randn((5, n, 128), generator=g).cuda()
    y = torch.empty_like(x)
    O.oscar_rotary(cfg, pos, x.transpose(0, 1), None, y.transpose(0, 1))
    check(cfg, pos, x.transpose(0, 1), y.transpose(0, 1), what="head-major")
    # the same row for every token and head
    one = torch.randn((1, 1, 128), generator=g).cuda()
    y = torch.empty((n, 3, 128), device="cuda")
    O.oscar_rotary(cfg, pos, one.expand(n, 3, 128), None, y)
    check(cfg, pos, one.expand(n, 3, 128), y, what="broadcast")
    # rows that are neighbours only after the padding between them
    x = torch.randn((n, 2, 136), generator=g).bfloat16().cuda()
    O.oscar_rotary(cfg, pos, x[..., 8:], None, y2 := torch.empty((n, 2, 128), dtype=torch.bfloat16, device="cuda"))
    check(cfg, pos, x[..., 8:], y2, what="padded")


def test_rows_past_the_tokens_stay():
    O = U.lib()
    cfg = O.make_rotary_config(128)
    pos = torch.arange(64, dtype=torch.int32).cuda()
    x = torch.randn((64, 2, 128), device="cuda")
    y = torch.full((64, 2, 128), 7.0, device="cuda")
    O.oscar_rotary(cfg, pos, x[:13], None, y[:13])
    assert torch.all(y[13:] == 7.0)
    O.oscar_rotary(cfg, pos, x[:0], None, y[:0])
    assert torch.all(y[13:] == 7.0)


def test_gradient_by_differences_and_inverse():
    """d/dx <w, R x> = R^T w, by differences in the float32 kernel (R is
    linear: a difference is exact up to the rounding of two float32 sums), and
    the transpose undoes the rotation when m = 1."""
    O = U.lib()
    g = torch.Generator().manual_seed(5)
    cfg = O.make_rotary_config(64, interleaved=True, scaling="yarn", factor=4.0, original_length=4096)
    pos = torch.tensor([7, 70000], dtype=torch.int32).cuda()
    x, w = (torch.randn((2, 1, 128), generator=g).cuda() for _ in range(2))
    grad = torch.empty_like(w)
    O.oscar_rotary(cfg, pos, w, None, grad, transpose=True)
    for c in (0, 1, 33, 63, 64, 127):
        step = torch.zeros_like(x)
        step[..., c] = 1.0
        hi, lo = torch.empty_like(x), torch.empty_like(x)
        O.oscar_rotary(cfg, pos, x + step, None, hi)
        O.oscar_rotary(cfg, pos, x - step, None, lo)
        diff = ((hi - lo).double() * w.double()).sum(-1) / 2
        # each of hi, lo is off by at most 9 2^-24 m (|x_a| + |x_b| + 1) and rounds once more; two channels count
        room = 2 * 12 * 2.0 ** -24 * 1.2 * (2 * x.abs().max().item() + 2) * w.abs().max().item()
        assert (diff - grad[..., c].double()).abs().max().item() <= room
    cfg = O.make_rotary_config(128, base=500000.0)
    y, back = torch.empty_like(x), torch.empty_like(x)
    O.oscar_rotary(cfg, pos, x, None, y)
    O.oscar_rotary(cfg, pos, y, None, back, transpose=True)
    top = x.abs().max().item()
    assert (back - x).abs().max().item() <= 2 * 2 * 10 * 2.0 ** -24 * 2 * top


def test_nan_and_inf_stay_in_their_pairs():
    O = U.lib()
    cfg = O.make_rotary_config(128)
    pos = torch.tensor([3], dtype=torch.int32).cuda()
    x = torch.ones((1, 2, 128), device="cuda")
    x[0, 0, 5] = float("nan")
    x[0, 1, 70] = float("inf")
    y = torch.empty_like(x)
    O.oscar_rotary(cfg, pos, x, None, y)
    bad = ~torch.isfinite(y)
    want = torch.zeros_like(bad)
    want[0, 0, [5, 69]] = True
    want[0, 1, [6, 70]] = True
    assert torch.equal(bad, want)


def test_stream_and_graph():
    O = U.lib()
    cfg = O.make_rotary_config(128)
    pos = torch.arange(9, dtype=torch.int32).cuda()
    x = torch.randn((9, 4, 128), device="cuda").bfloat16()
    ref, y = torch.empty_like(x), torch.empty_like(x)
    O.oscar_rotary(cfg, pos, x, None, ref)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    O.oscar_rotary(cfg, pos, x, None, y, stream=s)
    s.synchronize()
    assert torch.equal(y, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O.oscar_rotary(cfg, pos, x, None, y)
    pos += 5
    graph.replay()
    O.oscar_rotary(cfg, pos, x, None, ref)
    torch.cuda.synchronize()
    assert torch.equal(y, ref)


def test_refusals():
    O = U.lib()
    cfg = O.make_rotary_config(128)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.zeros((4, 2, 128), device="cuda", dtype=torch.bfloat16)
    flat = torch.zeros(4 * 2 * 160, device="cuda", dtype=torch.bfloat16)

    def refused(*a, **kw):
        with pytest.raises(O.OscarError) as e:
            O.oscar_rotary(*a, **kw)
        assert e.value.status == O.OSCAR_ERR_INVALID_ARG
    refused(cfg, pos, x.cpu())                                               # host rows
    refused(cfg, pos.cpu(), x)                                               # pageable positions
    refused(cfg, pos, flat[4:4 + 1024].view(4, 2, 128))                      # 8-byte aligned
    refused(cfg, pos, flat.as_strided((4, 2, 128), (264, 132, 1)))           # stride of 264 bytes
    refused(cfg, pos, x, None, x[:1].expand(4, 2, 128))                      # one output row for all tokens
    refused(cfg, pos, x, None, flat.as_strided((4, 2, 128), (128, 64, 1)))   # overlapping output rows
    refused(cfg, pos, x, None, x.as_strided((4, 2, 128), (128, 512, 1)))     # "in place" with other strides


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_stride_of_a_single_token_or_head_does_not_matter(dtype):
    """One token, or one head, taken out of a tensor whose pitch along that
    dimension is no multiple of 16 bytes."""
    cfg = U.lib().make_rotary_config(128, base=500000.0)
    x = torch.randn((6, 128), device="cuda").to(dtype)
    for shape, strides in [((1, 6, 128), (771, 128, 1)), ((6, 1, 128), (128, 5, 1)), ((1, 6, 128), (1, 128, 1))]:
        odd = x.as_strided(shape, strides)
        pos = torch.arange(9, 9 + shape[0], dtype=torch.int32, device="cuda")
        want, got = torch.empty(shape, dtype=dtype, device="cuda"), torch.empty(shape, dtype=dtype, device="cuda")
        U.lib().oscar_rotary(cfg, pos, odd.clone(memory_format=torch.contiguous_format), None, want)
        U.lib().oscar_rotary(cfg, pos, odd, None, got)
        assert torch.equal(got, want)
        y = x.clone().as_strided(shape, strides)
        U.lib().oscar_rotary(cfg, pos, y)                      # in place
        assert torch.equal(y, want)
