"""Memory and order where the feed-forward operators run on another stream than
the current one: outputs made by a call come from the memory of the stream that
writes them, an optimizer's states are zero before the first step on any, and the
workspace that a captured graph holds outlives larger calls.
"""
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


class OnDevice:
    """What the wrappers read of a CUDA tensor, without one."""

    def __init__(self, *shape, dtype=torch.float32, empty=torch.empty):
        t = empty(*shape, dtype=dtype)
        self.dtype, self.shape, self.device = dtype, t.shape, torch.device("cuda", 0)
        self.dim, self.stride, self.numel = t.dim, t.stride, t.numel
        self.is_contiguous, self.requires_grad = t.is_contiguous, False

    def data_ptr(self):
        return 4096

    def get_device(self):
        return 0


def calls(make):
    """name -> a call on `stream` that makes its outputs, with tensors from make(rows, cols, dtype)."""
    x, w, d = make(40, 64, torch.float32), make(64, 96, torch.float32), make(96, 64, torch.float32)
    q, s = make(8, 96, torch.int32), make(2, 96, torch.float32)
    w4 = sg.W4Matrix(q, s, 64, 32)
    return {
        "forward": lambda stream: sg.ffn_forward(x, w, w, d, stream=stream),
        "backward": lambda stream: sg.ffn_backward(x, x, w, w, d, stream=stream),
        "matvec": lambda stream: w4.matvec(x, stream=stream),
        "quantize": lambda stream: sg.w4_quantize(w, 32, stream=stream),
    }


NAMES = ("forward", "backward", "matvec", "quantize")


@pytest.mark.parametrize("name", NAMES)
def test_outputs_are_allocated_under_their_stream(monkeypatch, name):
    from dense_fp32_sgemm_gb300 import ffn
    sg.build()
    call = calls(lambda rows, cols, dtype: OnDevice(rows, cols, dtype=dtype))[name]
    current, made = ["current"], []

    @contextlib.contextmanager
    def under(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*shape, dtype=None, device=None):
        made.append(current[-1])
        return OnDevice(*shape, dtype=dtype)

    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "stream", under)
        m.setattr(ffn, "_call", lambda *a: None)
        m.setattr(torch, "empty", empty)
        call("side")
        assert made and set(made) == {"side"}
        made.clear()
        call(None)
        assert made and set(made) == {"current"}


def outputs(result):
    if isinstance(result, sg.W4Matrix):
        return [result.qweight, result.scales, result.zeros]
    return list(result) if isinstance(result, tuple) else [result]


def spans(tensors):
    return [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors]


def meet(a, b):
    return any(p < v and u < q for p, q in a for u, v in b)


@gpu
@pytest.mark.parametrize("name", NAMES)
def test_no_memory_in_use_on_another_stream_is_taken(device, name):
    gen = torch.Generator("cuda").manual_seed(8)

    def make(rows, cols, dtype):
        if dtype == torch.int32:
            return torch.zeros(rows, cols, dtype=dtype, device="cuda")
        return torch.randn(rows, cols, generator=gen, device="cuda")

    call, side = calls(make)[name], torch.cuda.Stream()
    want = [t.clone() for t in outputs(call(None))]
    torch.cuda.synchronize()
    call(side)  # workspace first: what follows does not wait for the device
    torch.cuda.synchronize()
    sizes = [(t.numel(), t.dtype) for t in want]

    def others():
        return [torch.empty(n, dtype=dtype, device="cuda") for n, dtype in sizes for _ in range(3)]

    # A result dropped before its stream has come to write it: its memory is not
    # the current stream's to use.
    sg.probe_hold(100_000_000, side)
    held = spans(outputs(call(side)))
    assert not side.query()
    assert not meet(held, spans(others()))
    torch.cuda.synchronize()
    # Memory that the current stream has freed but still works on is not the other's.
    sg.probe_hold(100_000_000, torch.cuda.current_stream())
    freed = spans(others())
    got = outputs(call(side))
    assert not torch.cuda.current_stream().query()
    assert not meet(freed, spans(got))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_states_are_zero_before_a_step_on_any_stream(device, bits):
    # The memory that the states get held ones before; the fill is queued behind work
    # that keeps the current stream busy while the step runs on another.
    n, side = 100_000, torch.cuda.Stream()
    p, g = (torch.ones(n, device="cuda") for _ in range(2))
    want = sg.AdamW([p.clone()], [g], state_bits=bits, lr=0.5)
    want.step()
    dirty = [torch.ones(n, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    del dirty
    sg.probe_hold(100_000_000, torch.cuda.current_stream())
    opt = sg.AdamW([p], [g], state_bits=bits, lr=0.5)
    opt.step(stream=side)
    torch.cuda.synchronize()
    for a, b in zip(opt.params + opt.m + opt.v, want.params + want.m + want.v):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_states_wait_for_their_fill(monkeypatch):
    # Without a device: the handle waits for the stream that fills them.
    from dense_fp32_sgemm_gb300 import ffn
    sg.build()
    log = []

    class Stream:
        def synchronize(self):
            log.append("wait")

    def zeros(n, dtype=torch.float32, device=None):
        log.append("fill")
        t = OnDevice(n, dtype=dtype)
        t.view = lambda kind: OnDevice(n, dtype=kind)
        return t

    with monkeypatch.context() as m:
        m.setattr(torch, "zeros", zeros)
        m.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
        ffn.AdamW([OnDevice(300)], [OnDevice(300)], state_bits=8)
    assert log == ["fill"] * 4 + ["wait"]


def ffn_case(T, D=64, F=500):
    gen = torch.Generator("cuda").manual_seed(T)
    x, wg, wu, wd = (torch.randn(a, b, generator=gen, device="cuda").bfloat16()
                     for a, b in ((T, D), (D, F), (D, F), (F, D)))
    y = torch.empty_like(x)
    return lambda: sg.ffn_forward(x, wg, wu, wd, y=y), y


def product_case(run, M, N, K):
    gen = torch.Generator("cuda").manual_seed(M)
    a, b = (torch.randn(n, m, generator=gen, device="cuda") for n, m in ((M, K), (K, N)))
    c = torch.empty(M, N, device="cuda")
    return lambda: run(a, b, c), c


# A small call, a larger one of the same kind on the same stream, and megabytes that the
# larger one's workspace and the two together have at least: the block's partial tiles (152
# of 256 KB and more each), stream-K tiles (two 128 KB slots a CTA, 147 and 152), split
# operands of the 3xTF32 form (two of 4 bytes an element: 33 and 67 MB).
GROWING = {
    "block": (lambda: ffn_case(150), lambda: ffn_case(3000), 39, 78),
    "stream-K": (lambda: product_case(sg.run, 2048, 1024, 1024),
                 lambda: product_case(sg.run, 2048, 2048, 2048), 39, 76),
    "counters": (lambda: product_case(sg.run, 2048, 1024, 1024),
                 lambda: product_case(sg.run, 20, 200_000, 500), 0, 0),
    "3xTF32": (lambda: product_case(sg.run_3xtf32, 1024, 1024, 2048),
               lambda: product_case(sg.run_3xtf32, 2048, 2048, 2048), 60, 95),
}


@gpu
@pytest.mark.parametrize("name", GROWING)
def test_a_graph_outlives_a_larger_call_on_its_stream(device, name):
    small, large, grown, both = GROWING[name]
    sg.release_workspace()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call, y = small()
    other, z = large()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    want = y.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    with torch.cuda.stream(side):
        other()
    torch.cuda.synchronize()
    # The larger workspace came beside the one that the graph holds.
    assert free - torch.cuda.mem_get_info()[0] >= grown * 1_000_000
    first = z.clone()
    for _ in range(2):
        y.zero_()
        z.zero_()
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            other()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, first)
    assert sg.device_status(side) == 0
    del graph
    before = torch.cuda.mem_get_info()[0]
    sg.release_workspace()
    assert torch.cuda.mem_get_info()[0] - before >= both * 1_000_000


@gpu
@pytest.mark.parametrize("name", ["block", "stream-K"])
def test_the_first_call_on_a_stream_while_the_default_one_is_busy(device, name):
    # The call's new counters have to be zero, whatever stands in the default stream.
    # Memory that held ones is freed first, so that new counters are not zero by chance.
    call, y = GROWING[name][0]()
    call()
    torch.cuda.synchronize()
    want = y.clone()
    dirty = torch.full((1 << 24,), -1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    sg.release_workspace()
    del dirty
    torch.cuda.empty_cache()
    side = torch.cuda.Stream()
    sg.probe_hold(100_000_000)  # on the default stream
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and sg.device_status(side) == 0


def work(seed):
    """Calls of every kind on tensors of their own, and what they leave (each call writes
    the same again, but for the parameters)."""
    gen = torch.Generator("cuda").manual_seed(seed)
    T, D, F = 130 + seed, 72, 3000
    x, wg, wu, wd, dy = ((torch.randn(a, b, generator=gen, device="cuda") * b ** -0.5).bfloat16()
                         for a, b in ((T, D), (D, F), (D, F), (F, D), (T, D)))
    y, few = torch.empty_like(x), torch.empty_like(x[:3])
    grads = [torch.empty_like(t) for t in (x, wg, wu, wd)]
    packed = sg.w4_quantize(wd, 64)
    tokens = torch.randn(2, F, generator=gen, device="cuda").bfloat16()
    out = torch.empty(2, D, device="cuda", dtype=torch.bfloat16)
    master = wg.float()
    opt = sg.AdamW([master], grads[1:2], state_bits=8)

    def run():
        sg.ffn_forward(x, wg, wu, wd, y=y)
        sg.ffn_forward(x[:3], wg, wu, wd, y=few)
        sg.ffn_backward(dy, x, wg, wu, wd, *grads)
        packed.matvec(tokens, out)
        opt.step()

    return run, [y, few, *grads, out, master, opt.m[0].view(torch.uint8)]


ROUNDS = 12


def alone(seed):
    run, left = work(seed)
    for _ in range(ROUNDS):
        run()
    torch.cuda.synchronize()
    return [t.clone() for t in left]


@gpu
def test_two_streams_at_once(device):
    want = [alone(seed) for seed in (0, 1)]
    both = [work(seed) for seed in (0, 1)]
    streams = [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    for _ in range(ROUNDS):
        for (run, _), stream in zip(both, streams):
            with torch.cuda.stream(stream):
                run()
    torch.cuda.synchronize()
    for (_, left), expected in zip(both, want):
        assert all(torch.equal(a, b) for a, b in zip(left, expected))
    assert all(sg.device_status(s) == 0 for s in streams)


@gpu
@pytest.mark.parametrize("shared", [False, True])
def test_two_host_threads(device, shared):
    # On streams of their own, and on one stream: a call's launches stay together.
    want = [alone(seed) for seed in (0, 1)]
    both = [work(seed) for seed in (0, 1)]
    one = torch.cuda.Stream()
    streams = [one, one] if shared else [torch.cuda.Stream() for _ in both]
    torch.cuda.synchronize()
    failed = []

    def thread(run, stream):
        try:
            with torch.cuda.stream(stream):
                for _ in range(ROUNDS):
                    run()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=thread, args=(run, s)) for (run, _), s in zip(both, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for (_, left), expected in zip(both, want):
        assert all(torch.equal(a, b) for a, b in zip(left, expected))
    assert all(sg.device_status(s) == 0 for s in streams)
