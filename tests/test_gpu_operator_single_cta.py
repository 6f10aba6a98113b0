"""Distillation through the head on single-CTA tiles (LMHEAD_CTA_PAIR=0, read once per
process): the cases of the CTA pairs' test, in a child process."""
import os
import subprocess
import sys

import pytest

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_distillation_on_single_cta_tiles():
    ensure_built()
    r = subprocess.run([sys.executable, "-m", "pytest", "tests/test_gpu_distill.py", "-q", "-x", "-m",
                        "gpu", "-k", "test_through_the_head or test_head"], cwd=ROOT,
                       env=dict(os.environ, LMHEAD_CTA_PAIR="0"), capture_output=True, text=True,
                       timeout=600)
    print(r.stdout[-3000:], r.stderr[-3000:])
    assert r.returncode == 0 and " passed" in r.stdout
