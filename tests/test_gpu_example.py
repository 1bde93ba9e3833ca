"""The example that runs the operators together: the decoding keeps its promises
(it checks the banned ids itself) and the student's loss falls."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_decode_and_distill():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    spec = importlib.util.spec_from_file_location("decode_and_distill",
                                                  os.path.join(ROOT, "examples", "decode_and_distill.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses = m.main(["--requests", "8", "--steps", "6", "--epochs", "30", "--vocab", "5000"])
    assert losses[-1] < 0.7 * losses[0]
