"""The cached operators in the checked build: no index check fires on valid calls, and
every output is bit-identical to libdd.so's. Each library runs in a process of its own."""
import os
import subprocess
import sys

import pytest
import torch

from speculative_verification_cover_b200 import build, dd

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def _child(path, checked):
    build.build()
    env = dict(os.environ, DD_CHECK_BOUNDS="1" if checked else "0")
    subprocess.run([sys.executable, os.path.join(HERE, "cached_checked_child.py"), str(path)], env=env, check=True,
                   timeout=600)
    return torch.load(path)


def test_checked_outputs_bit_identical(tmp_path):
    checked, plain = _child(tmp_path / "checked.pt", True), _child(tmp_path / "plain.pt", False)
    assert checked["checked"] and not plain["checked"]
    for op in ("attention", "evict", "beam"):
        for name, want in plain[op].items():
            got = checked[op][name]
            assert int(got["status"]) == dd.DD_OK and int(want["status"]) == dd.DD_OK, (op, name)
            for key in want:
                assert torch.equal(got[key], want[key]), (op, name, key)
