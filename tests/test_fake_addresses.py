"""Tests that hand made-up addresses to the C ABI run only where no device is
visible.  Collected (never run) in a child process that believes it has one."""
import glob
import os
import re
import subprocess
import sys

from tests import conftest

HERE = os.path.dirname(os.path.abspath(__file__))

COLLECT = """
import os, sys
import torch
torch.cuda.is_available = lambda: True
import pytest

class Report:
    def pytest_collection_finish(self, session):
        for it in session.items:
            print("ITEM", os.path.basename(str(it.fspath)), it.name.replace(" ", "_"),
                  any(m.name == "skip" for m in it.iter_markers()))

sys.exit(pytest.main(["--collect-only", "-q", "-p", "no:cacheprovider", *sys.argv[1:]],
                     plugins=[Report()]))
"""


def collect(*names):
    r = subprocess.run([sys.executable, "-c", COLLECT, *(os.path.join(HERE, n) for n in names)],
                       cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    return [line.split()[1:] for line in r.stdout.splitlines() if line.startswith("ITEM ")]


def test_skipped_where_a_device_is_visible():
    items = collect(*conftest.FAKE_ADDRESSES, "test_mx_ref.py")
    seen = {}
    for module, name, skipped in items:
        seen[module] = seen.get(module, 0) + 1
        assert skipped == str(module != "test_mx_ref.py"), (module, name)
    assert set(seen) == {*conftest.FAKE_ADDRESSES, "test_mx_ref.py"}
    assert min(seen.values()) > 2
    assert any(name == "test_workspace_rules" for _, name, _ in items)


def test_every_such_module_is_listed():
    """Their made-up addresses are large constants: 0x7f... bases or 2^36 steps."""
    found = set()
    for path in glob.glob(os.path.join(HERE, "test_*.py")):
        if path != os.path.abspath(__file__) and \
                re.search(r"0x7F0{6,}|= 1 << 36|0x1000_?0{4,}", open(path).read()):
            found.add(os.path.basename(path))
    assert found == set(conftest.FAKE_ADDRESSES)
