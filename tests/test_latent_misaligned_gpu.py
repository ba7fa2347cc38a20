"""The latent decodes' check of their shared memory's alignment, in a build that takes every block for misaligned."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_misaligned_blocks_leave_the_join_nothing():
    done = subprocess.run([sys.executable, os.path.join(ROOT, "tests", "latent_misaligned_run.py")], cwd=ROOT,
                          capture_output=True, text=True, timeout=900)
    assert done.returncode == 0 and done.stdout.strip().endswith("left alone"), done.stdout[-2000:] + done.stderr[-2000:]
