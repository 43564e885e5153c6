"""The example runs with each type of weights, and in training."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMALL = ["--tokens", "100", "--hidden", "256", "--inner", "128", "--experts", "8", "--topk", "2"]


@pytest.mark.parametrize("more", [["--weights", "int8"], ["--weights", "fp8"], ["--weights", "bf16"], ["--train"]])
def test_expert_layer(more):
    out = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "expert_layer.py"), *SMALL, *more], cwd=ROOT,
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = out.stdout.strip().splitlines()
    assert len(lines) == (1 if "--train" in more else 3) and all("status 0" in line and "nan" not in line for line in lines)
