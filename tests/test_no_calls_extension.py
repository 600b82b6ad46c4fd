"""The calls on torch tensors where the extension for the usual ones was not built: all of
them take the way through Python."""
import os

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg
from dense_fp32_sgemm_gb300 import _build, q8


@pytest.fixture
def no_extension(monkeypatch, tmp_path):
    sg.build()
    monkeypatch.setattr(_build, "CALLS_PATH", os.path.join(tmp_path, "_torch_calls.so"))
    monkeypatch.setattr(q8, "_calls", None)


def test_checks_are_made(no_extension):
    x, w = torch.ones(3, 8), torch.ones(8)
    for call in (lambda: sg.rms_norm(x, w), lambda: sg.rms_norm_backward(x, x, w), lambda: sg.rms_norm_q8(x, w),
                 lambda: sg.gate_q8(x, x), lambda: sg.rows_q8(x)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()


@pytest.mark.gpu
def test_results_are_the_same(monkeypatch, tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    x, r, dy = (torch.randn(40, 264, device="cuda") for _ in range(3))
    w = torch.rand(264, device="cuda") + 0.5

    def calls():
        q, s = sg.rows_q8(x)
        m = sg.q8_quantize(r.t().contiguous())
        return [*sg.rms_norm(x, w, residual=r), *sg.rms_norm_backward(dy, x, w), *sg.rms_norm_q8(x, w),
                *sg.gate_q8(x, r), q, s, m.matmul(q, s)]

    want = calls()
    monkeypatch.setattr(_build, "CALLS_PATH", os.path.join(tmp_path, "_torch_calls.so"))
    monkeypatch.setattr(q8, "_calls", None)
    assert all(torch.equal(a, b) for a, b in zip(want, calls()))


def test_a_build_without_it_is_made_whole(monkeypatch, tmp_path):
    # (the compilers are not run)
    if not _build._torch():
        pytest.skip("torch without CUDA")
    sg.build()
    made = []
    monkeypatch.setattr(_build, "CALLS_PATH", os.path.join(tmp_path, "_torch_calls.so"))
    monkeypatch.setattr(_build, "_compile_calls", lambda: made.append("compiled") or "object")
    monkeypatch.setattr(_build, "_link_calls", lambda obj: made.append(obj))
    _build.build()
    assert made == ["compiled", "object"]
