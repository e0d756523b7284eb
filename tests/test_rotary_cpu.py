"""Rotary configuration on the host: frequencies against the formulas in
Python floats, and the refusals that need no GPU."""
import copy
import ctypes
import math
import pickle

import pytest
import torch


@pytest.fixture(scope="module")
def O():
    import os

    from int2_kv_cache_oscar_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from int2_kv_cache_oscar_gb300 import oscar
    return oscar


def frequencies(dim, base, scaling, factor, original, low, high):
    """The header's formulas (float64)."""
    f = [base ** (-2.0 * i / dim) for i in range(dim // 2)]
    if scaling == "none":
        return f
    if scaling == "linear":
        return [x / factor for x in f]
    if scaling == "banded":
        out = []
        for x in f:
            t = original * x / (2 * math.pi)
            if t < low:
                out.append(x / factor)
            elif t > high:
                out.append(x)
            else:
                r = (t - low) / (high - low)
                out.append((1 - r) * x / factor + r * x)
        return out
    c = lambda t: dim * math.log(original / (2 * math.pi * t)) / (2 * math.log(base))  # noqa: E731
    lo, hi = max(math.floor(c(high)), 0), min(math.ceil(c(low)), dim - 1)
    hi = lo + 0.001 if lo == hi else hi
    out = []
    for i, x in enumerate(f):
        r = min(1.0, max(0.0, (i - lo) / (hi - lo)))
        out.append(x / factor * r + x * (1 - r))
    return out


@pytest.mark.parametrize("dim", [16, 64, 112, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1.5])
@pytest.mark.parametrize("scaling,low,high", [("none", 0, 0), ("linear", 0, 0), ("banded", 0, 0), ("banded", 2, 9),
                                              ("yarn", 0, 0), ("yarn", 0.5, 40)])
def test_frequencies(O, dim, base, scaling, low, high):
    cfg = O.make_rotary_config(dim, base=base, scaling=scaling, factor=8.0, original_length=8192, low=low, high=high)
    f, m = O.oscar_rotary_frequencies(cfg)
    default = {"banded": (1.0, 4.0), "yarn": (1.0, 32.0)}.get(scaling, (0, 0))
    low, high = (low, high) if high else default
    want = frequencies(dim, base, scaling, 8.0, 8192, low, high)
    # pow is good to an ulp or so, and the ramp's differences keep a few more
    assert len(f) == dim // 2
    for a, b in zip(f, want):
        assert abs(a - b) <= 1e-13 * b
    assert m == pytest.approx(0.1 * math.log(8.0) + 1.0 if scaling == "yarn" else 1.0, rel=1e-15)


def test_attention_factor_given(O):
    assert O.oscar_rotary_frequencies(O.make_rotary_config(64, scaling="yarn", factor=4.0, original_length=4096,
                                                           attention_factor=1.25))[1] == 1.25


@pytest.mark.parametrize("change,status", [
    (dict(rotary_dim=0), 4), (dict(rotary_dim=24), 4), (dict(rotary_dim=144), 4), (dict(rotary_dim=-16), 4),
    (dict(head_dim=64), 4), (dict(base=1.0), 1), (dict(base=float("inf")), 1), (dict(base=float("nan")), 1),
    (dict(scaling="linear", factor=0.5), 1), (dict(scaling="linear", factor=float("nan")), 1),
    (dict(scaling="banded", factor=2.0, original_length=0.0), 1),
    (dict(scaling="banded", factor=2.0, original_length=4096.0, low=4.0, high=4.0), 1),
    (dict(scaling="yarn", factor=2.0, original_length=4096.0, low=-1.0, high=4.0), 1),
    (dict(attention_factor=float("inf")), 1)])
def test_bad_configurations(O, change, status):
    with pytest.raises(O.OscarError) as e:
        O.make_rotary_config(**change)
    assert e.value.status == status


def test_refusals_before_any_gpu_call(O):
    lib = O.raw_library()
    cfg = O.make_rotary_config()
    rows = ctypes.byref(O.oscar_rotary_rows(4096, 4096, 128, 128, 128, 128, 1))
    pos = ctypes.c_void_p(4096)
    call = lambda n=1, p=pos, t=0, tr=0: lib.oscar_rotary(cfg.address, n, p, t, rows, None, tr, None)  # noqa: E731
    assert call(n=-1) == O.OSCAR_ERR_INVALID_ARG
    assert call(p=None) == O.OSCAR_ERR_INVALID_ARG
    assert call(p=ctypes.c_void_p(4097)) == O.OSCAR_ERR_INVALID_ARG
    assert call(t=2) == O.OSCAR_ERR_UNSUPPORTED
    assert call(tr=2) == O.OSCAR_ERR_INVALID_ARG
    assert call(n=0) == O.OSCAR_OK
    assert lib.oscar_rotary(None, 1, pos, 0, rows, None, 0, None) == O.OSCAR_ERR_INVALID_ARG
    assert lib.oscar_rotary(ctypes.addressof(O.oscar_rotary_table()), 1, pos, 0, rows, None, 0,
                            None) == O.OSCAR_ERR_INVALID_ARG          # never prepared
    assert lib.oscar_rotary_prepare(ctypes.byref(cfg.cfg), None) == O.OSCAR_ERR_INVALID_ARG
    for fn, args in [("oscar_cache_read", (None, 0, None, None, None, 0, None, None, None)),
                     ("oscar_cache_export", (None, 0, None, None, None, None)),
                     ("oscar_cache_import", (None, 0, 0, None, None, None, None)),
                     ("oscar_index_required_bytes", (None, None)),
                     ("oscar_index_attach", (None, None, 0)),
                     ("oscar_index_update", (None, 0, None, 0, None)),
                     ("oscar_select_groups", (None, 0, None, None, 1, 1, 0, 0, None, None)),
                     ("oscar_sparse_decode_attention", (None, 1, None, None, 1, 0.0, pos, 1, 0, None, None, None, 0,
                                                        None))]:
        assert getattr(lib, fn)(*args) == O.OSCAR_ERR_INVALID_ARG, fn
    assert lib.oscar_sparse_decode_attention(None, 1, None, None, 1, 0.0, None, 1, 0, None, None, None, 0,
                                             None) == O.OSCAR_ERR_INVALID_ARG


def test_binding_refusals(O):
    cfg = O.make_rotary_config()
    pos = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros((4, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bfloat16 or torch.float32"):
        O.oscar_rotary(cfg, pos, q.half())
    with pytest.raises(ValueError, match="shape"):
        O.oscar_rotary(cfg, pos[:3], q)
    with pytest.raises(ValueError, match="int32"):
        O.oscar_rotary(cfg, pos.long(), q)
    with pytest.raises(ValueError, match="shape"):
        O.oscar_rotary(cfg, pos, q, k=torch.zeros((3, 1, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="shape"):
        O.oscar_rotary(cfg, pos, q, q_out=torch.zeros((4, 1, 128), dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous channels"):
        O.oscar_rotary(cfg, pos, torch.zeros((4, 2, 256), dtype=torch.bfloat16)[..., ::2])
    with pytest.raises(ValueError, match="bfloat16"):
        O.oscar_rotary(cfg, pos, q, k=q.float())
    with pytest.raises(ValueError, match="scaling"):
        O.make_rotary_config(scaling="other")
    groups = torch.zeros((1, 1, 4), dtype=torch.int32)
    q1 = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="int32"):
        O.oscar_select_groups(None, [0], q1, 4, groups.long())
    with pytest.raises(ValueError, match="shape"):
        O.oscar_select_groups(None, [0, 1], q1, 4, groups)
    with pytest.raises(ValueError, match="shape"):
        O.oscar_sparse_decode_attention(None, [0], q1, 4, 0.0, groups[0], q1, torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(ValueError, match="out must be"):
        O.oscar_sparse_decode_attention(None, [0], q1, 4, 0.0, groups, q1.half(), torch.zeros(64, dtype=torch.uint8))
    with pytest.raises(TypeError, match="q must be a torch.Tensor"):
        O.oscar_rotary(cfg, pos, [1.0])
    with pytest.raises(TypeError):
        O.oscar_cache_read(None, [0.5], [0], [1], None, None)
    with pytest.raises(ValueError, match="out of range"):
        O.oscar_cache_read(None, [2 ** 40], [0], [1], None, None)
    with pytest.raises(ValueError, match="KV heads"):
        O.oscar_select_groups(None, [0], q1, 4, groups, num_kv_heads=2)
    with pytest.raises(ValueError, match="same length"):
        O.oscar_cache_read(None, [0], [0, 1], [2], None, None)
    with pytest.raises(ValueError, match="shape"):
        O.oscar_cache_read(None, [0], [0], [5], torch.zeros((4, 1, 128)), None)
    with pytest.raises(ValueError, match="float32"):
        O.oscar_cache_read(None, [0], [0], [4], torch.zeros((4, 1, 128)),
                           torch.zeros((4, 1, 128), dtype=torch.bfloat16))


def test_copies_have_their_own_table(O):
    """A copied or unpickled configuration does not point into the original."""
    cfg = O.make_rotary_config(rotary_dim=64, base=500.0)
    table = bytes(cfg._table)
    deep, back, shallow = copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), copy.copy(cfg)
    assert deep.address != cfg.address and back.address != cfg.address
    del cfg
    for c in (deep, back, shallow):
        assert c.address == ctypes.addressof(c._table)
        assert bytes((ctypes.c_char * ctypes.sizeof(c._table)).from_address(c.address)) == table
