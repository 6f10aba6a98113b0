"""The on-policy distillation example: layer norm, the head's distillation, logit
processing and scoring together, as a trainer uses them."""
import importlib.util
import math
import os

import pytest

from conftest import ROOT
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu


def test_on_policy_distillation_learns():
    ensure_built()
    path = os.path.join(ROOT, "examples", "on_policy_distillation.py")
    spec = importlib.util.spec_from_file_location("on_policy_distillation", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    losses = module.main(steps=6)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < losses[0]
