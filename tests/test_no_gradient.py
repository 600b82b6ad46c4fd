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


def tangents(dev):
    """name -> a call with a tensor that carries a tangent, and the same without one."""
    x, w = torch.randn(4, 8, device=dev), torch.ones(8, device=dev)
    calls = {}
    for which in range(3):
        def norm(call, which=which):
            def run(wrap):
                t = [x, w, x.clone()]
                t[which] = wrap(t[which])
                return call(*t)
            return run
        calls[f"norm {which}"] = norm(lambda a, b, r: sg.rms_norm(a, b, residual=r))
        calls[f"norm_q8 {which}"] = norm(lambda a, b, r: sg.rms_norm_q8(a, b, residual=r))
        calls[f"backward {which}"] = norm(lambda a, b, r: sg.rms_norm_backward(x, a, b, residual=r))
    calls["backward dy"] = lambda wrap: sg.rms_norm_backward(wrap(x), x, w)
    calls["backward dh"] = lambda wrap: sg.rms_norm_backward(x, x, w, dh=wrap(x))
    calls["gate g"] = lambda wrap: sg.gate_q8(wrap(x), x)
    calls["gate u"] = lambda wrap: sg.gate_q8(x, wrap(x))
    calls["rows"] = lambda wrap: sg.rows_q8(wrap(x))
    calls["quantize"] = lambda wrap: sg.q8_quantize(wrap(x))
    calls["given y"] = lambda wrap: sg.rms_norm(x, w, y=wrap(torch.empty_like(x)))
    if dev == "cuda":
        q, s = sg.rows_q8(x)
        ws = torch.ones(4, device=dev)
        m = sg.Q8Matrix(q, ws)
        calls["product"] = lambda wrap: m.matmul(q, wrap(s))
        calls["product, scales"] = lambda wrap: sg.Q8Matrix(q, wrap(ws)).matmul(q, s)
    return calls


@pytest.mark.parametrize("where", DEVICES)
def test_tangents_of_forward_mode(where):
    dev = on(where)
    for name, call in tangents(dev).items():
        for grad in (True, False):
            with forward_ad.dual_level(), torch.set_grad_enabled(grad):
                with pytest.raises(ValueError, match="forward-mode"):
                    call(lambda t: forward_ad.make_dual(t, torch.ones_like(t)))
                if where == "cuda":
                    call(lambda t: t)  # (a level alone is no tangent)


@pytest.mark.parametrize("where", DEVICES)
@pytest.mark.parametrize("which", range(5))
def test_tangents_through_the_gated_block(where, which):
    dev = on(where)
    t = [torch.randn(3, 8, device=dev), torch.randn(8, 16, device=dev), torch.randn(8, 16, device=dev),
         torch.randn(16, 8, device=dev), torch.empty(3, 8, device=dev)]
    with forward_ad.dual_level():
        if where == "cuda":
            sg.ffn_forward(*t)
        t[which] = forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        with pytest.raises(ValueError, match="forward-mode"):
            sg.ffn_forward(*t)


@gpu
@pytest.mark.parametrize("which", range(3))
def test_tangents_through_products_with_4_bit_weights(which):
    on("cuda")
    x, y = torch.randn(2, 64, device="cuda"), torch.empty(2, 16, device="cuda")
    m = sg.w4_quantize(torch.randn(64, 16, device="cuda"), group=32)
    with forward_ad.dual_level():
        m.matvec(x, y)
        t = [x, y, m.scales]
        t[which] = forward_ad.make_dual(t[which], torch.ones_like(t[which]))
        m = sg.W4Matrix(m.qweight, t[2], 64, 32, zeros=m.zeros)
        with pytest.raises(ValueError, match="forward-mode"):
            m.matvec(*t[:2])
