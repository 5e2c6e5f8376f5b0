"""CPU tests of the example of serving steps: its check sees outputs that are not numbers, and its arguments."""
import importlib.util
import os
import types

import pytest
import torch

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "serving_steps.py")


@pytest.fixture()
def example():
    spec = importlib.util.spec_from_file_location("serving_steps", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _step(example):
    """Two sequences of 2 and 1 new tokens over 5 and 3, in plain torch."""
    m, g = example, torch.Generator().manual_seed(0)
    lens, start = [5, 3], [0, 2, 3]
    k, v = (torch.randn(8, m.KV_HEADS, m.DIM, generator=g) for _ in range(2))
    q = torch.randn(3, m.HEADS, m.DIM, generator=g)
    out = torch.zeros(3, m.HEADS, m.DIM)
    for row, (b, end) in enumerate(((0, 4), (0, 5), (1, 3))):
        lo = sum(lens[:b])
        for h in range(m.HEADS):
            j = h // (m.HEADS // m.KV_HEADS)
            p = torch.softmax(k[lo:lo + end, j] @ q[row, h] * m.DIM ** -0.5, 0)
            out[row, h] = p @ v[lo:lo + end, j]
    batch = types.SimpleNamespace(q_start=torch.tensor(start, dtype=torch.int32))
    return q, out, batch, lens, k, v


@pytest.mark.parametrize("at", [0, 1, 2])
def test_the_check_sees_outputs_that_are_not_numbers(example, monkeypatch, at):
    q, out, batch, lens, k, v = _step(example)
    monkeypatch.setattr(example.sg, "sgmv_kv_read", lambda *a, **kw: (k, v))
    cache = types.SimpleNamespace(dtype=torch.int8)
    assert example.check(q, out, batch, lens, cache) <= 1e-5
    for x in (float("nan"), float("inf")):
        bad = out.clone()
        bad[at, 3, 7] = x
        assert not example.check(q, bad, batch, lens, cache) <= 1e-5
    bad = out.clone()
    bad[at, 3, 7] += 0.5
    assert abs(float(example.check(q, bad, batch, lens, cache)) - 0.5) < 1e-4


def test_steps_are_at_least_one(example, capsys):
    for steps in ("0", "-3"):
        with pytest.raises(SystemExit):
            example.main(["--steps", steps])
        assert "--steps" in capsys.readouterr().err
