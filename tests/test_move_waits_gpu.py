"""Forks that end inside a group: a copy of the read-back of that group left
unissued (the library's own hook).  The bounded wait gives up, the call's end is
reported, groups and other slots hold what they should, later calls are
unaffected."""
import pytest
import torch

from tests import gpu_util as U
from tests.test_move_gpu import equal, make, prefix, state

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("meta", [32, 16])
@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("n", [1, 20])
def test_wait_of_a_cut_that_runs_out(n, inplace, meta):
    """In place, and in a fork, where the read-back runs beside the copies."""
    O = U.lib()
    cache = make([700, 900], 3, 2 + n, meta)
    src = [i % 2 for i in range(n)]
    dst = list(range(2, 2 + n))
    take = [300 + i for i in range(n)]
    want = [prefix(cache, s, t) for s, t in zip(src, take)]
    before = [state(cache, s) for s in (0, 1)]
    if inplace:                                      # slots that hold all of their source, then are cut
        cache.fork(src, dst)
        src = dst
    O.oscar_cache_check(cache.handle)
    O.oscar_test_arm_wait_timeout()
    cache.fork(src, dst, take)
    with pytest.raises(O.OscarError) as e:
        O.oscar_cache_check(cache.handle)            # synchronises: the call returned
    assert e.value.status == O.OSCAR_ERR_DEVICE_TIMEOUT
    O.oscar_cache_check(cache.handle)
    for d, t, w in zip(dst, take, want):             # groups and maxima came all the same
        assert cache.length(d) == t
        got = state(cache, d)
        assert equal((got[0], got[2]), (w[0], w[2]))
    assert all(equal(state(cache, s), b) for s, b in zip((0, 1), before))
    # the same forks once more
    src = [i % 2 for i in range(n)]
    cache.fork(src, dst, take)
    O.oscar_cache_check(cache.handle)
    for d, t, w in zip(dst, take, want):
        assert cache.length(d) == t and equal(state(cache, d), w)
