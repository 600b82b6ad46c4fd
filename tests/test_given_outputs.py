"""Outputs that are given to the operators in 8 bits: graphs that hold one learn that it was
overwritten."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg


@pytest.mark.gpu
def test_codes_and_scales_count_as_written():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    x, w = torch.randn(5, 32, device="cuda"), torch.ones(32, device="cuda")
    for call in (lambda q, s: sg.rms_norm_q8(x, w, q=q, scales=s), lambda q, s: sg.gate_q8(x, x, q=q, scales=s),
                 lambda q, s: sg.rows_q8(x, q=q, scales=s)):
        q, s = torch.empty(5, 32, dtype=torch.int8, device="cuda"), torch.ones(5, device="cuda")
        a = torch.ones(5, device="cuda", requires_grad=True)
        loss = (a * s).sum()  # holds s
        before = q._version
        call(q, s)
        assert q._version == before + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()
