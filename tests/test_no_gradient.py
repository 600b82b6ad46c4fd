"""Calls through which no gradient goes refuse inputs that require one; no derivative stops
without a word.  (On the CPU the refusal comes before the one of the device.)"""
import pytest

torch = pytest.importorskip("torch")
from torch.autograd import forward_ad

import dense_fp32_sgemm_gb300 as sg

gpu = pytest.mark.gpu


def on(where):
    if where == "cuda" and not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return where


DEVICES = ["cpu", pytest.param("cuda", marks=gpu)]


@pytest.mark.parametrize("where", DEVICES)
@pytest.mark.parametrize("which", range(5))
def test_gradient_of_the_norms_gradient(where, which):
    dev = on(where)
    x, r, dy, dh = (torch.randn(4, 8, device=dev) for _ in range(4))
    inputs = [dy, x, torch.ones(8, device=dev), r, dh]
    inputs[which].requires_grad_()
    dy, x, w, r, dh = inputs
    for more in ({}, {"need_dx": False}, {"dx": torch.empty(4, 8, device=dev)}):
        with pytest.raises(ValueError, match="has no gradient"):
            sg.rms_norm_backward(dy, x, w, residual=r, dh=dh, **more)
    if where == "cuda":
        with torch.no_grad():
            dx, dw = sg.rms_norm_backward(dy, x, w, residual=r, dh=dh)
        assert not dx.requires_grad and not dw.requires_grad


@gpu
def test_gradient_of_a_matrix_scales():
    on("cuda")
    q = torch.ones(16, 64, dtype=torch.int8, device="cuda")
    x, xs = torch.ones(3, 64, dtype=torch.int8, device="cuda"), torch.ones(3, device="cuda")
    scales = torch.ones(16, device="cuda")
    m = sg.Q8Matrix(q, scales)
    scales.requires_grad_()
    for stream in (None, torch.cuda.current_stream()):
        for y in (None, torch.empty(3, 16, dtype=torch.bfloat16, device="cuda")):
            with pytest.raises(ValueError, match="has no gradient"):
                m.matmul(x, xs, y, stream=stream)
    with torch.no_grad():
        assert bool((m.matmul(x, xs) == 64).all())


@pytest.mark.parametrize("where", DEVICES)
def test_gradient_of_quantised_weights(where):
    dev = on(where)
    w = torch.randn(8, 6, device=dev, requires_grad=True)
    with pytest.raises(ValueError, match="has no gradient"):
        sg.q8_quantize(w)
    if where == "cuda":
        with torch.no_grad():
            sg.q8_quantize(w)
        sg.q8_quantize(w.detach())


@pytest.mark.parametrize("where", DEVICES)
def test_given_outputs_that_require_a_gradient(where):
    dev = on(where)
    x, w = torch.randn(4, 8, device=dev), torch.ones(8, device=dev)
    out = torch.zeros(4, 8, device=dev, requires_grad=True)
    row = torch.zeros(8, device=dev, requires_grad=True)
    streams = [None] if where == "cpu" else [None, torch.cuda.current_stream()]
    for s in streams:
        for refused in (lambda: sg.rms_norm(x, w, y=out, stream=s), lambda: sg.rms_norm(x, w, h=out, stream=s),
                        lambda: sg.rms_norm(x, w, residual=x, h=out * 1, stream=s),
                        lambda: sg.rms_norm_q8(x, w, h=out, stream=s),
                        lambda: sg.gate_q8(x, x, scales=row[:4], stream=s),
                        lambda: sg.rows_q8(x, scales=row[:4], stream=s),
                        lambda: sg.rms_norm_backward(x, x, w, dx=out, stream=s),
                        lambda: sg.rms_norm_backward(x, x, w, dweight=row, stream=s)):
            with pytest.raises(ValueError, match="given"):
                refused()
    assert bool((out == 0).all()) and bool((row == 0).all())
    if where == "cuda":
        with torch.no_grad():
            assert sg.rms_norm(x, w, y=out) is out
