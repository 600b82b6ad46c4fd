"""Memory that the norm's gradient takes beside its operands."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


@pytest.mark.gpu
@pytest.mark.parametrize("need_dw", [True, False])
def test_rows_that_fit_registers_take_none_for_themselves(device, need_dw):
    T, D = 1 << 24, 4
    x, dy, dx = (torch.randn(T, D, device="cuda") for _ in range(3))
    w, dw = torch.ones(D, device="cuda"), torch.empty(D, device="cuda")
    sg.rms_norm_backward(dy[:9], x[:9], w, dx=dx[:9], dweight=dw)  # (kernels are loaded)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    sg.rms_norm_backward(dy, x, w, dx=dx, dweight=dw, need_dw=need_dw, stream=side)
    torch.cuda.synchronize()
    # (partial rows: four values for each SM; the allocator gives 2 MB at least)
    assert before - torch.cuda.mem_get_info()[0] <= 8 << 20
    n = dy.double()
    r = 1 / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()
    want = r * (n - x.double() * r * r * (n * x.double()).mean(1, keepdim=True))
    assert float((dx.double() - want).abs().max()) <= 1e-5 * float(want.abs().max())


@pytest.mark.gpu
def test_rows_that_are_read_again_without_a_weights_gradient(device):
    # Needs no workspace either: the first call on a stream can be captured.
    x, dy = (torch.randn(6, 20000, device="cuda") for _ in range(2))
    w = torch.ones(20000, device="cuda")
    want = sg.rms_norm_backward(dy, x, w, need_dw=False)[0]
    dx = torch.zeros_like(x)
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sg.rms_norm_backward(dy, x, w, dx=dx, need_dw=False)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(dx, want)
