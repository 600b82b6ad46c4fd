"""The example that trains a block, quantises it and serves it runs, learns, and
its 4-bit form stays near the 16-bit one."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_example_learns_and_serves():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    spec = importlib.util.spec_from_file_location(
        "feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    weights, losses = example.train(steps=60)
    assert losses[-1] < 0.7 * losses[0]
    # 15 steps over a group's range, errors uniform within half a step: 4 sigma / 15
    # / sqrt(12) of a weight's sigma each, about 0.1, through three matrices.
    assert example.serve(weights) < 0.35
