"""The paged attention's bounded waits: with a limit that runs out at once the call reports
FP8_ERR_TIMEOUT, nothing stays in flight, and the next call is right.  In a process of its own."""
import os
import subprocess
import sys

import pytest


@pytest.mark.gpu
def test_attention_abort_path_drains_and_recovers(cuda_device):
    child = os.path.join(os.path.dirname(os.path.abspath(__file__)), "abort_attention_child.py")
    r = subprocess.run([sys.executable, child], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("OK"), r.stdout[-2000:] + r.stderr[-4000:]
