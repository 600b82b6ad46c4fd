"""Copies of a matrix of 8-bit weights use tensors of their own, not the memory of the one
that they were made from."""
import copy
import io
import pickle

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg


def saved(m):
    file = io.BytesIO()
    torch.save(m, file)
    file.seek(0)
    return torch.load(file, weights_only=False)


@pytest.mark.gpu
@pytest.mark.parametrize("make", [copy.copy, copy.deepcopy, lambda m: pickle.loads(pickle.dumps(m)), saved])
def test_copies(make):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    for K in (64, 70):  # (70: rows off 16 bytes were laid out anew)
        gen = torch.Generator("cuda").manual_seed(K)
        w = torch.randint(-127, 128, (33, K), generator=gen, device="cuda").to(torch.int8)
        x = torch.randint(-127, 128, (20, K), generator=gen, device="cuda").to(torch.int8)
        xs = torch.ones(20, device="cuda")
        m = sg.Q8Matrix(w, torch.rand(33, generator=gen, device="cuda"), dtype=torch.float32)
        m.name = "down"
        n = make(m)
        assert type(n) is type(m) and n.name == "down"
        # (what the calls read, before one is made: nothing, or the copy's own)
        assert n._weights[3] in (-1, n.qweight.data_ptr()) and n._weights[5] in (-1, n.scales.data_ptr())
        assert (n.N, n.K, n.dtype, n.device) == (m.N, m.K, m.dtype, m.device)
        want = m.matmul(x, xs)
        assert torch.equal(n.matmul(x, xs), want)
        n.scales.mul_(2)
        assert torch.equal(n.matmul(x, xs), 2 * want)


@pytest.mark.gpu
def test_tensors_that_move_and_tensors_put_in_their_place():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    x, xs = torch.ones(20, 64, dtype=torch.int8, device="cuda"), torch.ones(20, device="cuda")
    weight = torch.nn.Parameter(torch.ones(33, 64, dtype=torch.int8, device="cuda"), requires_grad=False)
    scales = torch.nn.Parameter(torch.ones(33, device="cuda"), requires_grad=False)
    m = sg.Q8Matrix(weight, scales, dtype=torch.float32)
    keep = [weight.data, scales.data]  # (what was read before is there still)
    for stream in (None, torch.cuda.current_stream()):
        weight.data = torch.full_like(keep[0], 2)  # as a module's to() does
        assert bool((m.matmul(x, xs, stream=stream) == 128).all())
        scales.data = torch.full_like(keep[1], 0.5)
        assert bool((m.matmul(x, xs, stream=stream) == 64).all())
        m.scales = torch.full_like(keep[1], 3)
        assert bool((m.matmul(x, xs, stream=stream) == 384).all())
        m.qweight, m.scales = weight, scales
        weight.data, scales.data = keep
        assert bool((m.matmul(x, xs, stream=stream) == 64).all())
    m.scales = m.scales[:5]
    with pytest.raises(ValueError, match="scales"):
        m.matmul(x, xs)
    m.scales = scales
    assert bool((m.matmul(x, xs) == 64).all())
    m.dtype = torch.bfloat16
    assert m.matmul(x, xs).dtype == torch.bfloat16
    m.scales = torch.ones(33)
    with pytest.raises(ValueError, match="CUDA device"):
        m.matmul(x, xs)
