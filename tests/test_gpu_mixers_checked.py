"""The mixers beside KDA through the bounds-checked build (libkda_debug.so): their GPU tests with no out-of-bounds access
flagged (calls there end in check_device_status, which raises on the bit)."""
import os
import re
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mixer_suites_pass_through_the_checked_build():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "-k", "not far_offsets",
                        "tests/test_gpu_gdn.py", "tests/test_gpu_paged.py"],
                       cwd=ROOT, env=dict(os.environ, KDA_DEBUG_BUILD="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    m = re.search(r"(\d+) passed", r.stdout)
    assert m and int(m.group(1)) >= 360, r.stdout[-2000:]  # the suites in full, not a part of them
