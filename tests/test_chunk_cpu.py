"""Chunk attention: the refusals that need no GPU, and the reference itself."""
import ctypes
import math

import pytest
import torch

from tests import chunk_ref as C
from tests.test_rotary_cpu import O  # noqa: F401  (the library, built where it is missing)


def rows(n=4, heads=2, dtype=torch.bfloat16):
    return torch.zeros((n, heads, 128), dtype=dtype)


def test_refusals_before_any_gpu_call(O):  # noqa: F811
    lib = O.raw_library()
    r = ctypes.byref(O.oscar_rows(4096, 256, 128))
    cu = lambda *x: (ctypes.c_int32 * len(x))(*x)  # noqa: E731

    def call(n=1, c=cu(0, 4), prefix=None, q=r, hq=4, hkv=2, scale=0.0, rule=None, po=None, pl=None, out=4096, lse=None):
        return lib.oscar_chunk_attention(n, c, prefix, q, r, r, hq, hkv, scale, rule, po, pl, out, lse, None)

    bad, cap = O.OSCAR_ERR_INVALID_ARG, O.OSCAR_ERR_CAPACITY
    assert call(n=-1) == bad
    assert call(n=1025) == cap
    assert call(n=0) == O.OSCAR_OK
    assert call(c=cu(0, 0)) == O.OSCAR_OK                  # nothing to do
    assert call(c=None) == bad
    assert call(c=cu(1, 4)) == bad
    assert call(n=2, c=cu(0, 4, 3)) == bad
    assert call(prefix=cu(5)) == bad
    assert call(prefix=cu(-1)) == bad
    assert call(hq=3) == bad
    assert call(hq=0) == bad
    assert call(hkv=0) == bad
    assert call(hq=1 << 16) == bad
    assert call(c=cu(0, 2 ** 31 - 1)) == cap
    assert call(scale=-1.0) == bad
    assert call(scale=float("nan")) == bad
    assert call(scale=float("inf")) == bad
    assert call(po=4096) == bad                            # a prior without its log-sum-exp
    assert call(pl=4096) == bad
    assert call(out=None) == bad
    assert call(out=4100) == bad
    assert call(lse=4098) == bad
    for c in (-1.0, 1e-4, 2000.0, float("nan"), float("inf")):
        assert call(rule=ctypes.byref(O.oscar_score_rule(c, 0, None))) == bad
    assert call(rule=ctypes.byref(O.oscar_score_rule(0.0, 1, None))) == bad
    assert call(rule=ctypes.byref(O.oscar_score_rule(0.0, 0, 4098))) == bad


def test_binding_refusals(O):  # noqa: F811
    q, k = rows(heads=4), rows()
    ok = dict(cu_seqlens=[0, 4], q=q, k=k, v=k, out=q)

    def refused(match, kind=ValueError, **kw):
        with pytest.raises(kind, match=match):
            O.oscar_chunk_attention(**{**ok, **kw})

    refused("bfloat16", q=rows(heads=4, dtype=torch.float32))
    refused("shape", q=rows(n=3, heads=4))
    refused("shape", v=rows(heads=3))
    refused("shape", k=torch.zeros((4, 2, 64), dtype=torch.bfloat16))
    refused("contiguous channels", k=torch.zeros((4, 2, 256), dtype=torch.bfloat16)[..., ::2])
    refused("shape", out=rows(n=3, heads=4))
    refused("contiguous", out=rows(heads=8)[:, :4])
    refused("out must be", kind=TypeError, out=None)
    refused("float32", lse=torch.zeros((4, 4), dtype=torch.float64))
    refused("shape", lse=torch.zeros((4, 3)))
    refused("prefix", prefix=[1, 2])
    refused("entry more", cu_seqlens=[])
    refused("shape", slopes=torch.zeros(3))
    refused("float32", slopes=torch.zeros(4, dtype=torch.float64))
    refused("out of range", cu_seqlens=[0, 2 ** 40])
    refused("integer", kind=TypeError, cu_seqlens=[0, 4.5])
    refused("number", kind=TypeError, cap="wide")
    with pytest.raises(O.OscarError):                      # num_q_heads not a multiple
        O.oscar_chunk_attention(**{**ok, "q": rows(heads=3), "out": rows(heads=3), "stream": 0})


def test_reference():
    """The 64-bit reference by hand: two tokens, and rows merged with what precedes them."""
    q = torch.zeros((2, 1, 128), dtype=torch.float64)
    q[:, 0, 0] = math.sqrt(128)
    k, v = torch.zeros((2, 1, 128), dtype=torch.float64), torch.zeros((2, 1, 128), dtype=torch.float64)
    k[0, 0, 0], k[1, 0, 0] = 1.0, 3.0
    v[0, 0, 1], v[1, 0, 1] = 2.0, -4.0
    o, lse, _ = C.chunk([0, 2], q, k, v)
    w = 1.0 / (1.0 + math.exp(2.0))
    assert float(o[0, 0, 1]) == pytest.approx(2.0) and float(lse[0, 0]) == pytest.approx(1.0)
    assert float(o[1, 0, 1]) == pytest.approx(2.0 * w - 4.0 * (1 - w))
    o, _, _ = C.chunk([0, 2], q, k, v, prefix=[2], slopes=torch.tensor([0.5]))
    w = 1.0 / (1.0 + math.exp(1.5))                        # token 0 sees token 1 at distance 1
    assert float(o[0, 0, 1]) == pytest.approx(2.0 * w - 4.0 * (1 - w))
    o, _, _ = C.chunk([0, 2], q, k, v, cap=2.0)
    a, b = 2 * math.tanh(0.5), 2 * math.tanh(1.5)
    w = 1.0 / (1.0 + math.exp(b - a))
    assert float(o[1, 0, 1]) == pytest.approx(2.0 * w - 4.0 * (1 - w))
    po, pl = torch.full((2, 1, 128), 10.0, dtype=torch.float64), torch.full((2, 1), 1.0, dtype=torch.float64)
    o, lse, _ = C.chunk([0, 2], q, k, v, prior=(po, pl))
    assert float(o[0, 0, 1]) == pytest.approx(6.0) and float(lse[0, 0]) == pytest.approx(1.0 + math.log(2.0))
