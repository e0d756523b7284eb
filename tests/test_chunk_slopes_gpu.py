"""Attention within a chunk: scores far from zero, by queries and keys or by slopes
over the whole range that a call takes."""
import pytest
import torch

from tests import gpu_util as U
from tests.test_chunk_gpu import call, compare, inputs, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens", [[20], [300, 33], [700]])
@pytest.mark.parametrize("size", [2.0 ** 8, 2.0 ** 12, 2.0 ** 20, 2.0 ** 30])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_far_from_zero(lens, size, sign):
    """Keys along the queries' direction: scores of 2^16 to 2^60, the last ones or the first ones the largest."""
    O = U.lib()
    q, k, v, _ = inputs(lens, 2, 2, seed=92)
    q, k = torch.zeros_like(q), torch.zeros_like(k)
    at = 0
    for n in lens:
        q[at:at + n, :, 3] = sign * size
        k[at:at + n, :, 3] = (size * (1 + torch.arange(n, device="cuda")[:, None] // 4 * 2.0 ** -7)).bfloat16()
        k[at:at + n, :, 4] = (size * 2.0 ** -16 * (torch.arange(n, device="cuda")[:, None] % 4)).bfloat16()
        q[at:at + n, :, 4] = sign * size
        at += n
    out, lse = call(O, lens, q, k, v, softmax_scale=1.0)
    compare(lens, q, k, v, out, lse, softmax_scale=1.0)
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    at = 0
    for n in lens:
        for i in (0, n // 2, n - 1):
            s = (q[at + i, 0].double() * k[at:at + i + 1, 0].double()).sum(-1)
            # (exact in float32: size^2 times a number of 18 bits)
            p = torch.softmax(s, 0)
            want = p @ v[at:at + i + 1, 0].double()
            assert ((out[at + i, 0].double() - want).abs() <= 2.0 ** -6 * v.abs().max()).all()
            assert abs(float(lse[at + i, 0]) - float(torch.logsumexp(s, 0))) <= 2.0 ** -21 * abs(float(s.abs().max())) + 2.0 ** -20
        at += n


@pytest.mark.parametrize("lens", [[20], [300, 33], [700]])
@pytest.mark.parametrize("scale", [2.0 ** -30, 2.0 ** -20, 0.0, 1.0])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_steep_slopes(lens, scale, sign):
    """All weight on the token itself, or (slopes below 0) on the first one, whatever the scale."""
    O = U.lib()
    q, k, v, _ = inputs(lens, 2, 2, seed=90)
    slopes = sign * torch.tensor([2.0 ** 59, 1.5 * 2.0 ** 40, 2.0 ** 30, 1000.0]).cuda()
    out, lse = call(O, lens, q, k, v, slopes=slopes, softmax_scale=scale)
    compare(lens, q, k, v, out, lse, slopes=slopes, softmax_scale=scale)
    at = 0
    for n in lens:
        own = torch.arange(n, device="cuda")
        want = v[at:at + n] if sign > 0 else v[at:at + 1].expand(n, 2, 128)
        # the one weight left is 2^x for the x by which its base is rounded (the sum of the weights too), which bf16 rounds
        # by half a step, 2^-8, at most; the output by another
        want = want.repeat_interleave(2, 1).float()
        assert ((out[at:at + n].float() - want).abs() <= 2.0 ** -7 * want.abs()).all()
        top = torch.zeros_like(lse[at:at + n]) if sign > 0 else slopes.abs()[None] * own[:, None]
        # the score itself (below 2^15.7 times the scale: 128 products of at most 8 x 50) beside the distance's, in float32
        assert ((lse[at:at + n] - top).abs() <= 2.0 ** 15.7 * (scale or 128 ** -0.5) + 2.0 ** -21 * top).all()
        at += n


@pytest.mark.parametrize("lens", [[20], [300, 33], [700]])
@pytest.mark.parametrize("scale", [2.0 ** -60, 1.3 * 2.0 ** -45, 2.0 ** -31])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_steep_slopes_and_small_scales(lens, scale, sign):
    """The same where a slope over the scale leaves float32's range at a distance of a few hundred tokens."""
    test_steep_slopes(lens, scale, sign)


@pytest.mark.parametrize("scale", [1.7 * 2.0 ** -40, 2.0 ** -31])
@pytest.mark.parametrize("prior", [False, True])
def test_ordinary_slopes_and_small_scales(scale, prior):
    """Scores that hardly differ: distances alone weigh the values."""
    O = U.lib()
    lens = [130, 40, 257]
    q, k, v, p = inputs(lens, 2, 4, seed=91, prior=prior)
    slopes = slopes_of(8)
    slopes[::2] *= -0.1
    compare(lens, q, k, v, *call(O, lens, q, k, v, p, slopes=slopes, softmax_scale=scale), prior=p, slopes=slopes,
            softmax_scale=scale)
