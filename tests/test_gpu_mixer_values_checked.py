"""The values of the mixers beside KDA (short sequences, keys with a common part, angles, infinite scores) through the
bounds-checked build (libkda_debug.so), with no out-of-bounds access flagged."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_mixer_values_pass_through_the_checked_build():
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-x", "-m", "gpu", "-p", "no:cacheprovider", "tests/test_gpu_gdn_short.py",
                        "tests/test_gpu_gdn_values.py", "tests/test_gpu_rope_angles.py", "tests/test_gpu_attn_values.py"],
                       cwd=ROOT, env=dict(os.environ, KDA_DEBUG_BUILD="1"), capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
