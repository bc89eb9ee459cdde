"""The README's recurrent layer runs as written on the GPU, and its results are finite."""
import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_readme_recurrent_layer_runs():
    text = open(os.path.join(ROOT, "README.md")).read()
    code = next(c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "RecurrentStep" in c)
    scope = {}
    exec(compile(code, "README.md", "exec"), scope)
    torch.cuda.synchronize()
    for name in ("y", "final", "dx", "da", "db", "d_initial", "dA_log", "ddt_bias", "d_hidden", "d_norm_w", "scales"):
        assert torch.isfinite(scope[name].float()).all(), name
    assert scope["rows"].shape == (3, 16, 128) and scope["scales"].shape == (3, 16)
