"""The Python of README.md runs as written, in order; a student that is the teacher
has no loss in its distillation lines (so both sides are at one temperature)."""
import os
import re

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Names(dict):
    """The examples' variables: the student's logits are the teacher's, and every loss is kept."""

    def __init__(self):
        super().__init__()
        self.losses = []

    def __missing__(self, name):
        if name == "student_logits":
            return self["x"]
        raise KeyError(name)

    def __setitem__(self, name, value):
        super().__setitem__(name, value)
        if name == "loss":
            self.losses.append(value)


def test_readme_examples():
    import torch
    if not torch.cuda.is_available():
        pytest.fail("the -m gpu tests need a CUDA device")
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    names = Names()
    for block in blocks:
        exec(compile(block, "README.md", "exec"), {}, names)
    assert len(names.losses) >= 2
    for loss in names.losses:
        # exact values give 0; the log-probs' own rounding is below 1e-5 (tests of top_log_probs), weighed by a mass of 1
        assert loss.shape == (256,) and float(loss.abs().max()) < 1e-4
