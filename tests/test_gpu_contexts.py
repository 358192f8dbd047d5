"""The library in two contexts of one device: kernel attributes belong to a
context, so each one has to opt in to large shared memory."""

import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu


def test_a_second_context_runs_every_kernel():
    case = os.path.join(os.path.dirname(os.path.abspath(__file__)), "context_case.py")
    got = subprocess.run([sys.executable, case], capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "contexts ok" in got.stdout, got.stdout + got.stderr
