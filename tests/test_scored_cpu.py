"""Decode and prefill under a score rule, forks and compaction: the refusals
that need no GPU."""
import ctypes

import pytest
import torch

from tests.test_rotary_cpu import O  # noqa: F401  (the library, built where it is missing)


def test_refusals_before_any_gpu_call(O):  # noqa: F811
    lib, p = O.raw_library(), ctypes.c_void_p(4096)
    ids = (ctypes.c_int32 * 1)(0)
    rule = lambda cap=0.0, reserved=0, slopes=None: ctypes.byref(O.oscar_score_rule(cap, reserved, slopes))  # noqa: E731

    def decode(r=None, t=0, c=None):
        return lib.oscar_scored_decode_attention(c, 1, ids, p, 8, 0.0, r, t, p, p, 1 << 20, None)

    def prefill(r=None, c=None):
        return lib.oscar_scored_prefill_attention(c, 0, 1, p, 8, 0.0, r, p, None, None, 0, None)

    assert decode(t=2) == O.OSCAR_ERR_UNSUPPORTED
    for bad in (rule(-1.0), rule(float("nan")), rule(float("inf")), rule(1e-5), rule(1025.0), rule(reserved=1),
                rule(slopes=4098)):
        assert decode(bad) == O.OSCAR_ERR_INVALID_ARG and "rule" in O.oscar_last_error()
        assert prefill(bad) == O.OSCAR_ERR_INVALID_ARG and "rule" in O.oscar_last_error()
    for call in (decode, prefill):                          # a good rule, no cache
        for r in (None, rule(), rule(30.0), rule(0.0009765625), rule(1024.0)):
            assert call(r) == O.OSCAR_ERR_INVALID_ARG and "cache" in O.oscar_last_error()
    assert lib.oscar_cache_fork(None, 0, None, None, None, None) == O.OSCAR_ERR_INVALID_ARG
    assert lib.oscar_cache_keep_groups(None, 0, None, None, None, None, None) == O.OSCAR_ERR_INVALID_ARG


def test_binding_refusals(O):  # noqa: F811
    q, ws = torch.zeros((1, 8, 128), dtype=torch.bfloat16), torch.zeros(64, dtype=torch.uint8)
    decode = lambda q=q, out=q, ws=ws, **kw: O.oscar_scored_decode_attention(None, [0], q, 8, 0.0, out, ws, **kw)  # noqa: E731
    prefill = lambda q=q, out=q, **kw: O.oscar_scored_prefill_attention(None, 0, q, 8, 0.0, out, **kw)  # noqa: E731
    for call in (decode, prefill):
        with pytest.raises(ValueError, match="bfloat16"):
            call(q=q.float())
        with pytest.raises(ValueError, match="shape"):
            call(q=torch.zeros((1, 7, 128), dtype=torch.bfloat16))
        with pytest.raises(ValueError, match="shape"):
            call(slopes=torch.zeros(7))
        with pytest.raises(ValueError, match="float32"):
            call(slopes=torch.zeros(8, dtype=torch.float64))
        with pytest.raises(TypeError):
            call(cap="x")
        with pytest.raises(ValueError, match="out must be"):
            call(out=q.half())
    with pytest.raises(ValueError, match="shape"):
        prefill(lse=torch.zeros((1, 7)))
    with pytest.raises(ValueError, match="uint8"):
        prefill(workspace=torch.zeros(4))
    for call in [lambda: O.oscar_cache_fork(None, [0], [1, 2], [1]), lambda: O.oscar_cache_fork(None, [0], [1], []),
                 lambda: O.oscar_cache_keep_groups(None, [0], [], [[]]),
                 lambda: O.oscar_cache_keep_groups(None, [0], [1], []),
                 lambda: O.oscar_cache_fork(None, [2 ** 40], [1], [1])]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        O.oscar_cache_keep_groups(None, [0], [1], [1])
    with pytest.raises(O.OscarError, match="cache"):
        O.oscar_cache_fork(None, [], [], [], stream=0)
