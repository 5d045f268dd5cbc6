"""The checked library's routed-field calls (tests/checked_run_routed.py, in a
process of its own)."""
import os
import subprocess
import sys

import pytest

from tests.gpu_util import say

pytestmark = pytest.mark.gpu

HERE = os.path.dirname(os.path.abspath(__file__))


def test_checked_library_records_no_failed_check():
    say("checked library run, routed fields")
    r = subprocess.run([sys.executable, "-u", os.path.join(HERE, "checked_run_routed.py")], capture_output=True,
                       text=True, timeout=100)
    print(r.stdout[-4000:], r.stderr[-2000:])
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-2000:]
