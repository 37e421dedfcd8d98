"""The operators around the mixer through the bounds-checked build (libkda_debug.so): every one of their GPU
tests but those that only take long, with no out-of-bounds access flagged (calls there end in
check_device_status, which raises on the bit)."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_block_suites_pass_through_the_checked_build():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", "not random_shapes and not offsets",
                        "tests/test_gpu_block.py", "tests/test_gpu_ssm_values.py", "tests/test_gpu_ssm_cuts.py"],
                       cwd=ROOT, env=dict(os.environ, KDA_DEBUG_BUILD="1"), capture_output=True, text=True, timeout=900)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 480, r.stdout[-2000:]  # the suites in full (500 when written), not a part of them
