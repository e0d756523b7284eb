import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


def half_built(lib, calls):
    """The C library is there, the compiled Python calls beside it are not (a
    tree built before they existed): the tests that build do so only without
    the library."""
    return os.path.exists(lib) and not os.path.exists(calls)


def pytest_sessionstart(session):
    from int2_kv_cache_oscar_gb300 import build
    if not hasattr(session.config, "workerinput") and half_built(build.LIB, build.CALLS):
        build.build()
