"""The norm and the operators in 8 bits on other streams, in captured graphs, from two
host threads, and with matrices whose rows lie beyond 2^31 elements."""
import contextlib
import threading

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


EMPTY, EMPTY_STRIDED = torch.empty, torch.empty_strided


class OnDevice:
    """What the wrappers read of a CUDA tensor, without one."""

    end = 0

    def __init__(self, *shape, dtype=torch.float32, strides=None):
        t = EMPTY(*shape, dtype=dtype) if strides is None else \
            EMPTY_STRIDED(shape, strides, dtype=dtype)
        self.dtype, self.shape, self.device = dtype, t.shape, torch.device("cuda", 0)
        self.dim, self.stride, self.numel = t.dim, t.stride, t.numel
        self.is_contiguous, self.requires_grad = t.is_contiguous, False
        OnDevice.end += 4096
        self.data_ptr = lambda at=OnDevice.end: at

    def get_device(self):
        return 0


def calls(make, vector):
    """name -> a call on `stream` that makes its outputs, with make(rows, cols, dtype)."""
    x, w = make(40, 64, torch.float32), make(64, 96, torch.float32)
    codes, weight, scales = make(96, 64, torch.int8), vector(64), vector(96)
    xq, xs = make(40, 64, torch.int8), vector(40)
    m = sg.Q8Matrix(codes, scales, dtype=torch.float32)
    return {
        "norm": lambda stream: sg.rms_norm(x, weight, residual=x, stream=stream),
        "backward": lambda stream: sg.rms_norm_backward(x, x, weight, dh=x, stream=stream),
        "norm_q8": lambda stream: sg.rms_norm_q8(x, weight, residual=x, stream=stream),
        "gate": lambda stream: sg.gate_q8(x, x, stream=stream),
        "rows": lambda stream: sg.rows_q8(x, stream=stream),
        "product": lambda stream: m.matmul(xq, xs, stream=stream),
        "quantize": lambda stream: sg.q8_quantize(w, stream=stream),
    }


NAMES = ("norm", "backward", "norm_q8", "gate", "rows", "product", "quantize")


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_allocated_under_their_stream(monkeypatch, name):
    from dense_fp32_sgemm_gb300 import q8
    sg.build()
    call = calls(lambda rows, cols, dtype: OnDevice(rows, cols, dtype=dtype), OnDevice)[name]
    current, made = ["current"], []

    @contextlib.contextmanager
    def under(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*shape, dtype=None, device=None):
        made.append(current[-1])
        return OnDevice(*shape, dtype=dtype)

    def empty_strided(shape, strides, dtype=None, device=None):
        made.append(current[-1])
        return OnDevice(*shape, dtype=dtype, strides=strides)

    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "stream", under)
        m.setattr(q8, "_call", lambda *a: None)
        m.setattr(torch, "empty", empty)
        m.setattr(torch, "empty_like", lambda t: empty(*t.shape, dtype=t.dtype))
        m.setattr(torch, "empty_strided", empty_strided)
        call("side")
        assert made and set(made) == {"side"}
        made.clear()
        call(None)
        assert made and set(made) == {"current"}


def outputs(result):
    if isinstance(result, sg.Q8Matrix):
        return [result.qweight, result.scales]
    return list(result) if isinstance(result, tuple) else [result]


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def meet(a, b):
    return any(p < v and u < q for p, q in a for u, v in b)


def gpu_calls():
    gen = torch.Generator("cuda").manual_seed(8)

    def make(rows, cols, dtype):
        t = torch.randn(rows, cols, generator=gen, device="cuda")
        return (t * 40).to(torch.int8) if dtype == torch.int8 else t

    return calls(make, lambda n: torch.rand(n, generator=gen, device="cuda") + 0.5)


@gpu
@pytest.mark.parametrize("name", NAMES)
def test_no_memory_in_use_on_another_stream_is_taken(device, name):
    call, side = gpu_calls()[name], torch.cuda.Stream()
    want = [t.clone() for t in outputs(call(None))]
    torch.cuda.synchronize()
    call(side)  # workspace first: what follows does not wait for the device
    torch.cuda.synchronize()
    sizes = [(t.numel(), t.dtype) for t in want]

    def others():
        return [torch.empty(n, dtype=dtype, device="cuda") for n, dtype in sizes for _ in range(3)]

    # Memory that the current stream has freed but still works on is not the other's.
    sg.probe_hold(100_000_000, torch.cuda.current_stream())
    freed = spans(others())
    got = outputs(call(side))
    assert not torch.cuda.current_stream().query()
    assert not meet(freed, spans(got))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("name", NAMES)
def test_another_stream_waits_for_nothing_and_computes_the_same(device, name):
    call, side = gpu_calls()[name], torch.cuda.Stream()
    want = [t.clone() for t in outputs(call(None))]
    torch.cuda.synchronize()
    for _ in range(3):
        got = outputs(call(side))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def block(T, dtype=torch.bfloat16, D=256, F=600, seed=4):
    """A training step's norm and a prompt's way through 8 bits, and its outputs."""
    gen = torch.Generator("cuda").manual_seed(seed)
    x, r, dy, dh = (torch.randn(T, D, generator=gen, device="cuda").to(dtype) for _ in range(4))
    weight = torch.rand(D, generator=gen, device="cuda") + 0.5
    wide, down = (torch.randn(a, b, generator=gen, device="cuda").to(dtype)
                  for a, b in ((D, 2 * F), (F, D)))
    first, second = sg.q8_quantize(wide), sg.q8_quantize(down)

    def run():
        y, h = sg.rms_norm(x, weight, residual=r)
        dx, dw = sg.rms_norm_backward(dy, x, weight, residual=r, dh=dh)
        q, s, h8 = sg.rms_norm_q8(x, weight, residual=r)
        gu = first.matmul(q, s)
        q2, s2 = sg.gate_q8(gu[:, :F], gu[:, F:])
        return [y, h, dx, dw, q, s, h8, gu, q2, s2, second.matmul(q2, s2)]

    return run, x


@gpu
@pytest.mark.parametrize("T", [1, 40, 300])
def test_a_block_captured_and_replayed(device, T):
    run, x = block(T)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        run()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator("cuda").manual_seed(seed),
                            device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, run()))


@gpu
def test_a_graph_keeps_its_workspace_when_a_larger_call_outgrows_it(device):
    run, _ = block(150)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    sg.release_workspace()
    with torch.cuda.stream(side):
        want = [t.clone() for t in run()]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = run()
    large, _ = block(6000)
    with torch.cuda.stream(side):
        large()
        dirty = [torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
    graph.replay()
    torch.cuda.synchronize()
    del dirty
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_graphs_of_two_streams_replayed_at_once(device):
    # Each is captured on a stream of its own, whose workspace is its own.
    graphs = []
    for seed, T in ((4, 200), (5, 90)):
        run, _ = block(T, seed=seed)
        side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            got = run()
        graphs.append((side, graph, got, want))
    for _ in range(20):
        for side, graph, _, _ in graphs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, got, want in graphs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
def test_two_host_threads(device):
    cases = [block(T, seed=T) for T in (70, 260)]
    wants = [[t.clone() for t in run()] for run, _ in cases]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            for _ in range(15):
                got = cases[k][0]()
            side.synchronize()
        if not all(torch.equal(a, b) for a, b in zip(got, wants[k])):
            wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@gpu
def test_a_backward_pass_through_the_norm_in_a_graph(device):
    gen = torch.Generator("cuda").manual_seed(1)
    x, r, w = (torch.randn(*s, generator=gen, device="cuda") for s in ((50, 96), (50, 96), (96,)))

    def step(leaves):
        y, h = sg.rms_norm(leaves[0], leaves[2], residual=leaves[1])
        return torch.autograd.grad((y * h).sum(), leaves)

    want = step([t.clone().requires_grad_() for t in (x, r, w)])
    leaves = [t.clone().requires_grad_() for t in (x, r, w)]
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaves)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        got = step(leaves)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


# ---- matrices beyond 2^31 elements ---------------------------------------------------

@gpu
def test_rows_beyond_2_31_elements(device):
    T, D = 270_000, 8192  # 2.2e9 elements
    gen = torch.Generator("cuda").manual_seed(2)
    x = torch.empty(T, D, device="cuda", dtype=torch.bfloat16).normal_(generator=gen)
    w = torch.rand(D, generator=gen, device="cuda") + 0.5
    part = slice(T - 700, T)
    q, s = sg.rows_q8(x)
    one = sg.rows_q8(x[part])
    assert torch.equal(q[part], one[0]) and torch.equal(s[part], one[1])
    y = sg.rms_norm(x, w)
    assert torch.equal(y[part], sg.rms_norm(x[part], w))
    # (rows off 16 bytes: another order of the sum, off by 2^-18 at most, and half a step of BF16)
    odd = sg.rms_norm(x[:, 1:], w[1:])
    want = x[part, 1:].double()
    want = want / (want.square().mean(1, keepdim=True) + 1e-6).sqrt() * w[1:].double()
    assert bool(((odd[part].double() - want).abs() <= (2.0 ** -8 + 2.0 ** -17) * want.abs()).all())
    dx, dw = sg.rms_norm_backward(x[:, 1:], x[:, 1:], w[1:], dx=odd)
    one = sg.rms_norm_backward(x[part, 1:], x[part, 1:], w[1:], need_dw=False)[0]
    assert bool(((odd[part].double() - one.double()).abs() <= 2.0 ** -6 * one.double().abs() + 2.0 ** -10).all())
    del odd, dx, want, one
    q, s, h = sg.rms_norm_q8(x, w, residual=y, h=y)
    assert torch.equal(h[part], (x[part].float() + sg.rms_norm(x[part], w).float()).bfloat16())
    del q, s, h
    dx, _ = sg.rms_norm_backward(x, x, w, dx=y)
    assert torch.equal(dx[part], sg.rms_norm_backward(x[part], x[part], w)[0])


@gpu
@pytest.mark.parametrize("M", [3, 30, 150])
def test_weights_beyond_2_31_elements(device, M):
    N, K = 70_000, 32768
    w = torch.empty(N, K, device="cuda", dtype=torch.int8).random_(-128, 128)
    ws = torch.rand(N, device="cuda") + 0.5
    x = torch.empty(M, K, device="cuda", dtype=torch.int8).random_(-128, 128)
    xs = torch.rand(M, device="cuda") + 0.5
    y = sg.Q8Matrix(w, ws, dtype=torch.float32).matmul(x, xs)
    last = sg.Q8Matrix(w[-300:], ws[-300:], dtype=torch.float32).matmul(x, xs)
    assert torch.equal(y[:, -300:], last)
    # (a sum over 2^15 products is below 2^29; exact in 64 bits)
    want = (x.double() @ w[-300:].double().t()) * xs.double()[:, None] * ws[-300:].double()
    assert ((last.double() - want).abs() <= 4.2 * 2.0 ** -24 * want.abs() + 2.0 ** -149).all()


@gpu
def test_results_beyond_2_31_elements(device):
    M, N, K = 70_000, 32768, 48
    w = torch.empty(N, K, device="cuda", dtype=torch.int8).random_(-128, 128)
    x = torch.empty(M, K, device="cuda", dtype=torch.int8).random_(-128, 128)
    ws, xs = torch.rand(N, device="cuda") + 0.5, torch.rand(M, device="cuda") + 0.5
    m = sg.Q8Matrix(w, ws)
    y = m.matmul(x, xs)
    assert torch.equal(y[-300:], m.matmul(x[-300:], xs[-300:]))
