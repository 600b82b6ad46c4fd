"""The extension through which the usual calls of the norm and of the operators in 8 bits
go: it does what the calls with checks in Python do, and hands on what is not usual."""
import gc
import sys

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


@pytest.fixture(scope="module")
def extension():
    from dense_fp32_sgemm_gb300 import q8
    sg.build()
    return q8._calls or q8._load_calls()


def test_what_is_not_usual_is_handed_on(extension):
    x, w, q, s = torch.ones(3, 8), torch.ones(8), torch.ones(3, 8, dtype=torch.int8), torch.ones(3)
    handle = (5, 8, 0, 4096, 16, 4096, 0)
    assert extension.rms_norm(x, w, None, 1e-6, None, None) is None
    assert extension.rms_norm([1], w, None, 1e-6, None, None) is None
    assert extension.rms_norm_q8(x, w, x, 1e-6, None) is None
    assert extension.rms_norm_backward(x, w, None, 1e-6, x, None, None, None, True, True) is None
    assert extension.gate_q8(x, x, 0) is None
    assert extension.gate_q8(x, x, 2**80) is None
    assert extension.gate_q8(x, x, "silu") is None
    assert extension.q8_matmul(q, s, None, handle) is None
    assert extension.q8_matmul(q, s, None, handle[:3]) is None
    assert extension.q8_matmul(q, s, None, ("a",) * 7) is None


@pytest.mark.parametrize("name", ["rms_norm", "rms_norm_q8", "rms_norm_backward", "gate_q8",
                                  "q8_matmul"])
def test_wrong_numbers_of_arguments(extension, name):
    with pytest.raises(TypeError, match="arguments"):
        getattr(extension, name)(torch.ones(1))
    with pytest.raises(TypeError):
        getattr(extension, name)(x=torch.ones(1))


def view(rows, cols, dtype, pad=0, offset=0):
    """A matrix whose rows are cols + pad apart."""
    t = torch.empty(rows * (cols + pad) + offset, dtype=dtype, device="cuda")
    return t[offset:].view(rows, cols + pad)[:, :cols]


CASES = [(1, 1, 0, 0), (1, 64, 0, 0), (5, 64, 8, 0), (40, 33, 3, 1), (7, 1, 0, 0), (7, 1, 5, 0),
         (300, 1000, 1, 3), (0, 16, 0, 0), (4, 0, 0, 0)]


def operands(rows, cols, pad, offset, dtype):
    gen = torch.Generator("cuda").manual_seed(rows * 1000 + cols)

    def matrix():
        m = view(rows, cols, dtype, pad, offset)
        return m.copy_(torch.randn(rows, cols, generator=gen, device="cuda"))

    return [matrix() for _ in range(4)], torch.rand(cols, generator=gen, device="cuda") + 0.5


def bits(result):
    result = result if isinstance(result, tuple) else (result,)
    return [None if t is None else (t.dtype, t.shape, t.contiguous().view(torch.uint8).cpu())
            for t in result]


def same(a, b):
    assert len(a) == len(b)
    for s, t in zip(bits(tuple(a)), bits(tuple(b))):
        assert (s is None) == (t is None)
        if s is not None:
            assert s[:2] == t[:2] and torch.equal(s[2], t[2])


def as_tuple(r):
    return r if isinstance(r, tuple) else (r,)


def calls(x, r, dy, dh, w, stream):
    n = x.shape[1]
    xq, xs = sg.rows_q8(x, stream=stream)
    m = sg.Q8Matrix(torch.ones(13, n, dtype=torch.int8, device="cuda"),
                    torch.ones(13, device="cuda"), dtype=x.dtype)
    return [sg.rms_norm(x, w, stream=stream), *sg.rms_norm(x, w, residual=r, stream=stream),
            *sg.rms_norm_backward(dy, x, w, stream=stream),
            *sg.rms_norm_backward(dy, x, w, residual=r, dh=dh, stream=stream),
            *sg.rms_norm_backward(dy, x, w, need_dw=False, stream=stream),
            *sg.rms_norm_backward(dy, x, w, need_dx=False, stream=stream),
            *sg.rms_norm_q8(x, w, stream=stream), *sg.rms_norm_q8(x, w, residual=r, stream=stream),
            *sg.gate_q8(x, r, stream=stream), *sg.gate_q8(x, r, sg.GATE_GELU, stream=stream), xq, xs,
            m.matmul(xq, xs, stream=stream)]


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols,pad,offset", CASES)
def test_both_ways_agree(device, rows, cols, pad, offset, dtype):
    (x, r, dy, dh), w = operands(rows, cols, pad, offset, dtype)
    direct = calls(x, r, dy, dh, w, None)
    torch.cuda.synchronize()
    same(direct, calls(x, r, dy, dh, w, torch.cuda.current_stream()))


@gpu
def test_the_usual_calls_are_taken(device, extension):
    (x, r, dy, dh), w = operands(5, 64, 8, 0, torch.bfloat16)
    xq, xs = extension.gate_q8(x, None, 0)
    m = sg.Q8Matrix(torch.ones(16, 64, dtype=torch.int8, device="cuda"),
                    torch.ones(16, device="cuda"))
    weight = torch.nn.Parameter(w, requires_grad=False)
    assert extension.rms_norm(x, weight, None, 1e-6, None, None) is not None
    assert extension.rms_norm_q8(x, w, r, 1e-6, None) is not None
    assert extension.rms_norm_backward(x, w, r, 1e-6, dy, dh, None, None, True, True) is not None
    assert extension.gate_q8(x, r, 1) is not None
    assert extension.q8_matmul(xq, xs, None, m._weights) is not None


@gpu
def test_no_reference_and_no_memory_is_lost(device):
    (x, r, dy, dh), w = operands(64, 256, 0, 0, torch.float32)
    m = sg.Q8Matrix(torch.ones(16, 256, dtype=torch.int8, device="cuda"),
                    torch.ones(16, device="cuda"), dtype=torch.float32)
    xq, xs = sg.rows_q8(x)
    y, h, dx, dw, p = (torch.empty_like(x), torch.empty_like(x), torch.empty_like(x),
                       torch.empty_like(w), torch.empty(64, 16, device="cuda"))
    held = [x, r, dy, dh, w, xq, xs, y, h, dx, dw, p]

    def run():
        sg.rms_norm(x, w), sg.rms_norm(x, w, residual=r), sg.rms_norm(x, w, residual=r, y=y, h=h)
        sg.rms_norm_q8(x, w), sg.rms_norm_q8(x, w, residual=r), sg.rms_norm_q8(x, w, residual=r, h=h)
        sg.rms_norm_backward(dy, x, w), sg.rms_norm_backward(dy, x, w, dx=dx, dweight=dw)
        sg.rms_norm_backward(dy, x, w, need_dx=False), sg.rms_norm_backward(dy, x, w, need_dw=False)
        sg.gate_q8(x, r), sg.rows_q8(x), m.matmul(xq, xs), m.matmul(xq, xs, y=p)

    run()
    gc.collect()
    counts, bytes_ = [sys.getrefcount(t) for t in held], torch.cuda.memory_allocated()
    objects = sum(issubclass(type(o), torch.Tensor) for o in gc.get_objects())
    for _ in range(50):
        run()
    gc.collect()
    assert [sys.getrefcount(t) for t in held] == counts
    assert torch.cuda.memory_allocated() == bytes_
    assert sum(issubclass(type(o), torch.Tensor) for o in gc.get_objects()) == objects


@gpu
def test_given_outputs_come_back_and_count_as_written(device):
    (x, r, dy, dh), w = operands(9, 128, 0, 0, torch.float32)
    y, h, dx, dw = (torch.empty_like(x), torch.empty_like(x), torch.empty_like(x),
                    torch.empty_like(w))
    before = [t._version for t in (y, h, dx, dw)]
    a = sg.rms_norm(x, w, residual=r, y=y, h=h)
    b = sg.rms_norm_backward(dy, x, w, dx=dx, dweight=dw)
    assert a[0] is y and a[1] is h and b[0] is dx and b[1] is dw
    assert [t._version for t in (y, h, dx, dw)] == [v + 1 for v in before]


@gpu
@pytest.mark.parametrize("side", [False, True])
def test_inference_tensors(device, side):
    with torch.inference_mode():
        (x, r, dy, dh), w = operands(9, 128, 0, 0, torch.float32)
        stream = torch.cuda.current_stream() if side else None
        y, h = torch.empty_like(x), torch.empty_like(x)
        sg.rms_norm(x, w, residual=r, y=y, h=h, stream=stream)
        q, s, h2 = sg.rms_norm_q8(x, w, residual=r, h=torch.empty_like(x), stream=stream)
        m = sg.q8_quantize(torch.randn(128, 32, device="cuda"))
        m.matmul(q, s, y=torch.empty(9, 32, device="cuda"), stream=stream)
    same([h], [h2])
    same([y, h], sg.rms_norm(x, w, residual=r))


@gpu
def test_a_subclass_of_tensor_takes_the_other_way(device):
    class Named(torch.Tensor):
        pass

    (x, r, dy, dh), w = operands(9, 128, 0, 0, torch.float32)
    y, h = sg.rms_norm(x.as_subclass(Named), w, residual=r)
    same([y.as_subclass(torch.Tensor), h.as_subclass(torch.Tensor)],
         sg.rms_norm(x, w, residual=r))


@gpu
def test_a_status_of_the_library_is_an_error(device):
    (x, r, dy, dh), w = operands(9, 128, 0, 0, torch.float32)
    with pytest.raises(sg.SgemmError, match="sgemm_q8_gate"):
        sg.gate_q8(x, r, 77)
    with pytest.raises(sg.SgemmError, match="sgemm_rms_norm"):
        sg.rms_norm(x, w, eps=-1.0)
