"""The example's block in eight bits runs and stays near the 16-bit one."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.gpu
def test_a_prompt_in_eight_bits():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    spec = importlib.util.spec_from_file_location(
        "feed_forward", os.path.join(ROOT, "examples", "feed_forward.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    weights = example.block_weights(256, 768, torch.Generator("cuda").manual_seed(1), torch.bfloat16)
    # Codes are off by half a step, top / 254: of rows of normal values, whose top is at most 5
    # deviations, 5 / 254 / root 3 of a deviation in the root mean square, at four places of the
    # way (norm, its weights, gate, its weights; the first two count for g and u), the 16-bit
    # block's roundings beside them: below 5 %.
    assert example.serve_prompt(weights) < 0.05
