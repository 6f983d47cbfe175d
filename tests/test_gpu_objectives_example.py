"""The example that trains with all objectives: every stage's loss falls."""
import gc
import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu


def test_every_stage_learns():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "objectives.py")
    spec = importlib.util.spec_from_file_location("objectives_example", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    stages = module.main(steps=10)
    gc.collect()  # leave no device memory to be freed inside another test
    assert len(stages) == 4
    for stage, (before, after) in stages.items():
        assert math.isfinite(before) and math.isfinite(after) and after < before, (stage, before, after)
