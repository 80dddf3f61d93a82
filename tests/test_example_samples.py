"""The example's serving loop runs and meets the definition."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("steps", [2, 24, 90])
def test_parallel_samples(steps, capsys):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mla_paged_decode_gb300 import build
    build.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import parallel_samples
    assert parallel_samples.main(["--steps", str(steps), "--check"]) == 0
    assert "pages live" in capsys.readouterr().out
