"""The example of serving steps runs, for every cache format, and its last step is right."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_steps.py")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "i8"])
def test_serving_steps(fmt, capsys):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    spec = importlib.util.spec_from_file_location("serving_steps", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    assert m.main(["--cache", fmt, "--steps", "6"]) == 0
    assert "sequence 2" in capsys.readouterr().out
