"""The gated block in torch's graph: gradients reach x and the weights, bit for
bit those of ffn_backward; what cannot be differentiated says so."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


def make(T, kind=torch.bfloat16, D=72, F=104, seed=6):
    gen = torch.Generator("cuda").manual_seed(seed)
    x, wg, wu, wd, dy = (torch.randn(a, b, generator=gen, device="cuda").to(kind)
                         for a, b in ((T, D), (D, F), (D, F), (F, D), (T, D)))
    return [t.requires_grad_() for t in (x, wg, wu, wd)], dy


@gpu
@pytest.mark.parametrize("kind", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("T", [3, 70])
def test_gradients_are_those_of_the_backward_call(device, T, keep, kind):
    leaves, dy = make(T, kind)
    saved = sg.ffn_saved(T, 104, dtype=kind) if keep else None
    with torch.no_grad():
        plain = sg.ffn_forward(*leaves, activation=sg.GATE_GELU, saved=saved)
        want = sg.ffn_backward(dy, *leaves, activation=sg.GATE_GELU, saved=saved)
    assert plain.grad_fn is None
    y = sg.ffn_forward(*leaves, activation=sg.GATE_GELU, saved=saved)
    assert torch.equal(y, plain)
    y.backward(dy)
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, want))


@gpu
def test_a_residual_and_broadcast_gradients(device):
    # x + block(x), summed over rows or over everything: dy comes with strides (0, 1)
    # or (0, 0).
    for total in (lambda y: y.sum(0).square().sum(), lambda y: y.sum()):
        leaves, _ = make(40, torch.float32)
        total(leaves[0] + sg.ffn_forward(*leaves)).backward()
        ref = [t.detach().double().requires_grad_() for t in leaves]
        x, wg, wu, wd = ref
        total(x + torch.nn.functional.silu(x @ wg) * (x @ wu) @ wd).backward()
        for got, want in zip(leaves, ref):
            # (FP32 sums of 40 to 208 products: below 1e-5 of the norm)
            assert float((got.grad.double() - want.grad).norm()) <= 1e-5 * float(want.grad.norm())


@gpu
def test_only_what_requires_a_gradient_gets_one(device):
    leaves, dy = make(33)
    full = [g for g in sg.ffn_backward(dy, *[t.detach() for t in leaves])]
    for on in ((0,), (2,), (1, 3)):
        parts = [t.detach().clone().requires_grad_(i in on) for i, t in enumerate(leaves)]
        sg.ffn_forward(*parts).backward(dy)
        for i, t in enumerate(parts):
            assert torch.equal(t.grad, full[i]) if i in on else t.grad is None


@gpu
def test_a_kept_buffer_that_another_pass_has_filled_is_noticed(device):
    leaves, dy = make(70)
    saved = sg.ffn_saved(70, 104, dtype=torch.bfloat16)
    y = sg.ffn_forward(*leaves, saved=saved)
    with torch.no_grad():
        sg.ffn_forward(2 * leaves[0], *leaves[1:], saved=saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward(dy)


@gpu
def test_on_another_stream(device):
    leaves, dy = make(70)
    want = sg.ffn_backward(dy, *[t.detach() for t in leaves])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y = sg.ffn_forward(*leaves, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    y.backward(dy)
    torch.cuda.synchronize()
    assert all(torch.equal(t.grad, g) for t, g in zip(leaves, want))


@gpu
def test_products_with_4_bit_weights_say_that_they_have_no_gradient(device):
    w = sg.w4_quantize(torch.randn(64, 32, device="cuda"), 32)
    x = torch.randn(2, 64, device="cuda", requires_grad=True)
    y = w.matvec(x)
    assert torch.equal(y, w.matvec(x.detach()))
    with pytest.raises(NotImplementedError):
        y.sum().backward()
    out = torch.empty(2, 32, device="cuda")
    with pytest.raises(ValueError):
        w.matvec(x, out)
    with torch.no_grad():
        assert torch.equal(w.matvec(x, out), y)


def test_a_given_output_is_refused():
    x, w, d = torch.ones(4, 8), torch.ones(8, 16), torch.ones(16, 8, requires_grad=True)
    with pytest.raises(ValueError, match="a given y has no gradient"):
        sg.ffn_forward(x, w, w, d, y=torch.empty(4, 8))
