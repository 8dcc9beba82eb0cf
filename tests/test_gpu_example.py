"""The serving example runs, and its own checks hold."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("samples,prompt,steps", [(6, 75, 5), (40, 130, 3), (2, 1, 1)])
def test_serve_samples(samples, prompt, steps):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serve_samples.py")
    spec = importlib.util.spec_from_file_location("serve_samples", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.main(samples, prompt, steps) > 0
