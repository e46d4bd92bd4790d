import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a B200 (sm_100a) GPU")


# Lines that tests add to the end-of-run summary (the parity statistics of the
# full-size workloads), printed even in quiet mode.
_SUMMARY = []


@pytest.fixture(scope="session")
def summary_lines():
    return _SUMMARY


def pytest_terminal_summary(terminalreporter):
    if _SUMMARY:
        terminalreporter.write_sep("-", "parity statistics")
        for line in _SUMMARY:
            terminalreporter.write_line(line)


@pytest.fixture(scope="session")
def orc():
    """The C oracle, built if needed."""
    import oracle
    return oracle.load()


def _cuda_ok():
    try:
        import torch
        return torch.cuda.is_available()
    except Exception:
        return False


# Modules that call the C ABI with made-up addresses.  Their calls must find no
# device: one that passes the argument checks (some are meant to) would launch a
# kernel on memory that is not there.
FAKE_ADDRESSES = ("test_abi_host.py", "test_abi_fuzz.py", "test_mx_abi_host.py")


def pytest_collection_modifyitems(config, items):
    if _cuda_ok():
        host_only = pytest.mark.skip(reason="made-up addresses must not reach a device")
        for it in items:
            if os.path.basename(str(it.fspath)) in FAKE_ADDRESSES:
                it.add_marker(host_only)
        return
    skip = pytest.mark.skip(reason="no CUDA device")
    for it in items:
        if "gpu" in it.keywords:
            it.add_marker(skip)
