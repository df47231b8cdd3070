"""Shared pytest configuration.

Tests marked ``gpu`` need an MI355X (gfx950) and the built HIP library; every
other test runs on the CPU only.
"""
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)
TESTS = os.path.dirname(os.path.abspath(__file__))
if TESTS not in sys.path:
    sys.path.insert(0, TESTS)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: a longer CPU test (still minutes at most)")


@pytest.fixture(autouse=True)
def _announce_gpu_case(request):
    """Name each GPU case on stderr (uncaptured, flushed) before it runs, so a
    run that dies on the GPU still says which case it was in."""
    if request.node.get_closest_marker("gpu") is not None:
        sys.__stderr__.write("\n[gpu case] %s\n" % request.node.nodeid)
        sys.__stderr__.flush()
    yield


@pytest.fixture(scope="session", autouse=True)
def _built_libraries():
    """Build the HIP libraries (hipcc, no GPU needed), the module over the layer
    library and the oracle where one is missing, so a fresh tree can run the
    suite; nothing is rebuilt otherwise.  A module that does not build fails the
    tests that call it, and those alone."""
    import dequantize_reduce_transfer_amd as fq
    import oracle
    from dequantize_reduce_transfer_amd import layer

    if not os.path.exists(fq.LIB_PATH) and not os.environ.get("FP8Q_LIB"):
        from dequantize_reduce_transfer_amd import build as hip_build
        sys.__stderr__.write("[conftest] building %s\n" % fq.LIB_PATH)
        hip_build.build()
    if os.path.exists(layer.LIB_PATH) and not os.path.exists(layer.BINDING_PATH):
        from dequantize_reduce_transfer_amd import build as hip_build
        sys.__stderr__.write("[conftest] building %s\n" % layer.BINDING_PATH)
        try:
            hip_build.build_binding()
        except (RuntimeError, OSError) as e:
            sys.__stderr__.write("[conftest] %s\n" % e)
    oracle.build(force=False)
    yield
