"""The root-mean-square norm: against the formula in 64 bits, element by element; its
gradients against the formula's and against differences; refusals.

Bounds.  A thread adds at most n = 32 squares (rows of up to 16384 elements, 256 for
the longer ones here) and ten more additions join the threads, all of
terms above zero: the mean is off by at most (n + 12) 2^-24 of itself, the root by half of that,
and the sum h, the products and the division add five roundings.  That is
below 2^-18 of y (2^-16 for the longer rows); y's own rounding is half a unit.
The gradients' second sum has terms of both signs: its error is that share of the sum of
their magnitudes.  dweight adds at most 2^-24 per row that a thread has taken and
that joins it, at most T + 40 in all, of the sum of its terms' magnitudes.
"""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
EPS = 1e-5
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


def spread(t, pad, offset=0, fill=float("nan")):
    """The same values with rows `pad` elements further apart, `offset` elements
    into a larger buffer of `fill`."""
    n, m = t.shape
    flat = torch.full((n * (m + pad) + offset + 8,), fill, device=t.device, dtype=t.dtype)
    view = flat[offset:offset + n * (m + pad)].view(n, m + pad)[:, :m]
    view.copy_(t)
    return view


def make(T, D, kind, wkind, pad=0, offset=0, count=4, seed=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    rows = [torch.randn(T, D, generator=gen, device="cuda") *
            torch.exp(torch.randn(T, 1, generator=gen, device="cuda")) for _ in range(count)]
    w = 1 + 0.5 * torch.randn(D, generator=gen, device="cuda")
    return [spread(r.to(TYPES[kind]), pad, offset) for r in rows], w.to(TYPES[wkind])


def tiny(dtype):
    return {torch.float16: 2.0 ** -25}.get(dtype, 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149)


def within(got, want, share, mass=None):
    """|got - want| at most `share` of mass (the result's own size if not given), and
    half a unit of the result."""
    unit, want = UNIT[got.dtype], want.double()
    slack = share * (want.abs() if mass is None else mass)
    limit = slack + unit * (want.abs() + slack) + tiny(got.dtype)
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= limit).all(), f"worst {float((err / limit).max()):.3g}"


def slack_of(D):
    return 2.0 ** -18 if D <= 8192 else 2.0 ** -16


def forward(x, w, r, kind):
    D = x.shape[1]
    got = sg.rms_norm(x, w, residual=r, eps=EPS)
    y, h = (got, None) if r is None else got
    hd = x.double() if r is None else x.double() + r.double()
    assert y.dtype == x.dtype
    within(y, hd / (hd.square().mean(1, keepdim=True) + EPS).sqrt() * w.double(), slack_of(D))
    if r is not None:
        within(h, hd, 2.0 ** -24)
    assert sg.device_status(torch.cuda.current_stream()) == 0
    return y, h


SIZES = [(1, 1), (1, 7), (1, 4096), (2, 8), (3, 31), (5, 129), (7, 256), (33, 1000), (4, 2047), (310, 520),
         (400, 1025), (9, 4104), (2, 8191), (3, 16384), (2, 16392), (2, 40001)]


@gpu
@pytest.mark.parametrize("kind,wkind", [("fp32", "fp32"), ("fp16", "fp16"), ("fp16", "fp32"),
                                        ("bf16", "bf16"), ("bf16", "fp32")])
@pytest.mark.parametrize("T,D", SIZES)
def test_forward(device, T, D, kind, wkind):
    (x, r), w = make(T, D, kind, wkind, count=2)
    forward(x, w, None, kind)
    forward(x, w, r, kind)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (4, 4), (1, 0), (3, 5)])
@pytest.mark.parametrize("T,D", [(3, 264), (305, 1032), (3, 1029), (2, 20000)])
def test_strides_and_alignment(device, T, D, pad, offset, kind):
    (x, r), w = make(T, D, kind, kind, pad, offset, count=2)
    y, h = forward(x, w, r, kind)
    out_y, out_h = spread(torch.zeros_like(y), 3, 1, 7.0), spread(torch.zeros_like(y), 8, 0, 7.0)
    sg.rms_norm(x, w, residual=r, eps=EPS, y=out_y, h=out_h)
    # (element by element or in vectors: the sums differ in order, not in what they bound)
    hd = x.double() + r.double()
    within(out_y, hd / (hd.square().mean(1, keepdim=True) + EPS).sqrt() * w.double(), slack_of(D))
    assert torch.equal(out_h, h)
    base = out_y._base
    assert bool((base[1 + T * (D + 3):] == 7.0).all()) and float(base[0]) == 7.0
    assert bool((base[1:1 + T * (D + 3)].view(T, D + 3)[:, D:] == 7.0).all())


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (3, 5), (4, 2)])
@pytest.mark.parametrize("T,D", [(40, 1), (5, 3), (17, 7), (6, 127), (400, 129), (311, 257), (310, 4099),
                                 (330, 12287), (310, 16383), (310, 16385)])
def test_rows_off_16_bytes(device, T, D, pad, offset, kind):
    # Outputs that start with either half of a word, h's not as y's.
    (x, r), w = make(T, D, kind, kind, pad, offset, count=2)
    y, h = forward(x, w, r, kind)
    forward(x, w, None, kind)
    for at_y, at_h in ((0, 1), (1, 1), (1, 0), (0, 8)):
        out_y, out_h = (spread(torch.zeros_like(y), 1, at, 7.0) for at in (at_y, at_h))
        sg.rms_norm(x, w, residual=r, eps=EPS, y=out_y, h=out_h)
        hd = x.double() + r.double()
        within(out_y, hd / (hd.square().mean(1, keepdim=True) + EPS).sqrt() * w.double(), slack_of(D))
        assert torch.equal(out_h, h)
        for out, at in ((out_y, at_y), (out_h, at_h)):
            base = out._base
            assert bool((base[:at] == 7.0).all()) and bool((base[at + T * (D + 1):] == 7.0).all())
            assert bool((base[at:at + T * (D + 1)].view(T, D + 1)[:, D:] == 7.0).all())


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D", [(4, 520), (400, 257), (2, 40001)])
def test_in_place(device, T, D, kind):
    (x, r, dy, dh), w = make(T, D, kind, kind)
    y, h = sg.rms_norm(x, w, residual=r, eps=EPS)
    a, b = x.clone(), r.clone()
    got = sg.rms_norm(a, w, residual=b, eps=EPS, y=a, h=b)
    assert got[0] is a and got[1] is b
    assert torch.equal(a, y) and torch.equal(b, h)
    a, b = x.clone(), r.clone()
    sg.rms_norm(a, w, residual=b, eps=EPS, h=a, y=b)
    assert torch.equal(b, y) and torch.equal(a, h)
    dx, dw = sg.rms_norm_backward(dy, h, w, dh=dh, eps=EPS)
    for which in (0, 1):
        c = [dy.clone(), dh.clone()]
        dx2, dw2 = sg.rms_norm_backward(c[0], h, w, dh=c[1], eps=EPS, dx=c[which])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


@gpu
def test_rows_of_zeros_infinities_and_far_values(device):
    w = torch.ones(64, device="cuda")
    x = torch.randn(6, 64, device="cuda")
    x[1] = 0
    x[2, 5] = float("inf")
    x[3, 7] = float("nan")
    x[4] *= 1e18
    x[5] *= 1e-25
    y = sg.rms_norm(x, w, eps=EPS)
    assert bool((y[1] == 0).all())
    # 1 / sqrt(infinity) is 0: zeros, and NaN where it meets the infinity.
    assert bool(torch.isnan(y[2, 5])) and bool((y[2].nan_to_num() == 0).all())
    assert bool(torch.isnan(y[3]).all())
    rest = x[[0, 4, 5]].double()
    within(y[[0, 4, 5]], rest / (rest.square().mean(1, keepdim=True) + EPS).sqrt(), 2.0 ** -18)


@gpu
def test_rows_do_not_depend_on_their_neighbours(device):
    (x, r), w = make(400, 1000, "bf16", "bf16", count=2)
    y, h = sg.rms_norm(x, w, residual=r)
    again = sg.rms_norm(x[7:320].contiguous(), w, residual=r[7:320].contiguous())
    assert torch.equal(again[0], y[7:320]) and torch.equal(again[1], h[7:320])


def gradients(h, dy, dh, w):
    hd, dyd, wd = h.double(), dy.double(), w.double()
    r = 1 / (hd.square().mean(1, keepdim=True) + EPS).sqrt()
    n = dyd * wd
    dx = r * (n - hd * r * r * (n * hd).mean(1, keepdim=True))
    mass = r * (n.abs() + hd.abs() * r * r * (n * hd).abs().mean(1, keepdim=True))
    if dh is not None:
        dx, mass = dx + dh.double(), mass + dh.double().abs()
    return dx, mass, (dyd * hd * r).sum(0), (dyd * hd * r).abs().sum(0)


def backward(h, dy, dh, w):
    T, D = h.shape
    dx, dw = sg.rms_norm_backward(dy, h, w, dh=dh, eps=EPS)
    want, mass, want_w, mass_w = gradients(h, dy, dh, w)
    assert dx.dtype == h.dtype and dw.dtype == w.dtype
    within(dx, want, slack_of(D), mass)
    within(dw, want_w, slack_of(D) + (T + 40) * 2.0 ** -24, mass_w)
    assert sg.device_status(torch.cuda.current_stream()) == 0
    return dx, dw


@gpu
@pytest.mark.parametrize("kind,wkind", [("fp32", "fp32"), ("fp16", "fp16"), ("bf16", "fp32"),
                                        ("bf16", "bf16")])
@pytest.mark.parametrize("T,D", [*SIZES, (1500, 64), (3000, 33), (700, 12288), (100, 12296), (310, 9001),
                                 (200, 16384), (155, 16377)])
def test_backward(device, T, D, kind, wkind):
    (h, dy, dh), w = make(T, D, kind, wkind, count=3)
    dx, dw = backward(h, dy, dh, w)
    backward(h, dy, None, w)
    only_x = sg.rms_norm_backward(dy, h, w, dh=dh, eps=EPS, need_dw=False)
    only_w = sg.rms_norm_backward(dy, h, w, dh=dh, eps=EPS, need_dx=False)
    assert only_x[1] is None and only_w[0] is None
    assert torch.equal(only_x[0], dx) and torch.equal(only_w[1], dw)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D", [(3, 31), (300, 520), (50, 1025), (40, 8192), (320, 9001), (200, 10504), (3, 40001)])
def test_backward_at_the_sum_in_32_bits(device, T, D, kind):
    (x, r, dy, dh), w = make(T, D, kind, "fp32")
    dx, dw = sg.rms_norm_backward(dy, x, w, residual=r, dh=dh, eps=EPS)
    want, mass, want_w, mass_w = gradients(x.double() + r.double(), dy, dh, w)
    within(dx, want, slack_of(D), mass)
    within(dw, want_w, slack_of(D) + (T + 40) * 2.0 ** -24, mass_w)
    only = sg.rms_norm_backward(dy, x, w, residual=r, eps=EPS, need_dx=False)[1]
    assert torch.equal(only, dw)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (1, 0), (3, 5)])
def test_backward_strides(device, pad, offset, kind):
    for T, D in ((70, 520), (40, 1029)):
        (h, dy, dh), w = make(T, D, kind, "fp32", pad, offset, count=3)
        backward(h, dy, dh, w)


@gpu
def test_gradients_against_differences(device):
    (x, r, dy, dh), w = make(5, 70, "fp32", "fp32")
    h = x + r
    dx, dw = sg.rms_norm_backward(dy, h, w, dh=dh, eps=EPS)

    def loss(hd, wd):
        y = hd / (hd.square().mean(1, keepdim=True) + EPS).sqrt() * wd
        return (y * dy.double()).sum() + (hd * dh.double()).sum()

    # Central differences in 64 bits: off by step^2 times the third derivative (below 1e3
    # here, as rows are of size one) and 2^-52 of the loss (below 1e4) over the step.
    step, hd, wd = 1e-5, h.double(), w.double()
    for row, col in ((0, 0), (1, 69), (4, 33)):
        up, down = hd.clone(), hd.clone()
        up[row, col] += step
        down[row, col] -= step
        slope = float((loss(up, wd) - loss(down, wd)) / (2 * step))
        assert abs(slope - float(dx[row, col])) <= 1e-6 + 1e-5 * abs(slope)
    for col in (0, 41):
        up, down = wd.clone(), wd.clone()
        up[col] += step
        down[col] -= step
        slope = float((loss(hd, up) - loss(hd, down)) / (2 * step))
        assert abs(slope - float(dw[col])) <= 1e-6 + 1e-5 * abs(slope)


@gpu
def test_no_rows(device):
    w = torch.ones(8, device="cuda")
    x = torch.empty(0, 8, device="cuda")
    y, h = sg.rms_norm(x, w, residual=x)
    assert y.shape == h.shape == (0, 8)
    dx, dw = sg.rms_norm_backward(x, x, w, dweight=torch.full((8,), 3.0, device="cuda"))
    assert dx.shape == (0, 8) and bool((dw == 0).all())
    e = torch.empty(5, 0, device="cuda")
    assert sg.rms_norm(e, w[:0]).shape == (5, 0)
    assert sg.rms_norm_backward(e, e, w[:0])[1].shape == (0,)


# ---- the graph --------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kind", TYPES)
def test_part_of_the_graph(device, kind):
    (x, r, dy, dh), w = make(30, 136, kind, "fp32")
    leaves = [t.clone().requires_grad_() for t in (x, w, r)]
    y, h = sg.rms_norm(leaves[0], leaves[1], residual=leaves[2], eps=EPS)
    torch.autograd.backward([y, h], [dy, dh])
    dx, dw = sg.rms_norm_backward(dy, h.detach(), w, dh=dh, eps=EPS)
    assert torch.equal(leaves[0].grad, dx) and torch.equal(leaves[2].grad, dx)
    assert torch.equal(leaves[1].grad, dw)
    a = x.clone().requires_grad_()
    sg.rms_norm(a, w, eps=EPS).backward(dy)
    assert torch.equal(a.grad, sg.rms_norm_backward(dy, x, w, eps=EPS)[0])


@gpu
def test_graph_with_one_output_used_and_broadcast_gradients(device):
    (x, r), w = make(12, 40, "fp32", "fp32", count=2)
    for use in (lambda y, h: y.sum(), lambda y, h: (2 * h).sum(), lambda y, h: (y + h).sum(0).square().sum()):
        leaves = [t.clone().requires_grad_() for t in (x, w, r)]
        use(*sg.rms_norm(leaves[0], leaves[1], residual=leaves[2], eps=EPS)).backward()
        ref = [t.double().requires_grad_() for t in (x, w, r)]
        h = ref[0] + ref[2]
        use(h / (h.square().mean(1, keepdim=True) + EPS).sqrt() * ref[1], h).backward()
        for got, want in zip(leaves, ref):
            want = torch.zeros_like(want) if want.grad is None else want.grad
            # (FP32 sums of 40 terms: below 1e-5 of the norm)
            assert float((got.grad.double() - want).norm()) <= 1e-5 * float(want.norm())


@gpu
def test_frozen_inputs_get_no_gradient(device):
    (x, r), w = make(6, 40, "fp32", "fp32", count=2)
    a = x.clone().requires_grad_()
    y, h = sg.rms_norm(a, w, residual=r)
    (y.sum() + h.sum()).backward()
    assert a.grad is not None and w.grad is None and r.grad is None
    v = w.clone().requires_grad_()
    sg.rms_norm(x, v).sum().backward()
    assert v.grad is not None
    with pytest.raises(ValueError, match="given y or h"):
        sg.rms_norm(a, w, y=torch.empty_like(x))
    with torch.no_grad():
        sg.rms_norm(a, w, y=torch.empty_like(x))


@gpu
def test_a_tensor_overwritten_in_place_is_known_to_graphs_that_hold_it(device):
    (x, r), w = make(6, 40, "fp32", "fp32", count=2)
    a = x.clone().requires_grad_()
    b = a * 2
    loss = (b * b).sum()  # holds b
    with torch.no_grad():
        sg.rms_norm(r, w, residual=b, h=b)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


# ---- refusals ---------------------------------------------------------------------

def call(name, **change):
    """An entry point's status for plausible host-side arguments with some changed (no
    memory is touched: each of these is refused, or has nothing to do)."""
    lib = sg.library()
    args = dict(T=4, D=8, type=0, x=4096, ldx=8, residual=8192, ldr=8, weight=12288, wtype=0, eps=1e-6,
                h=16384, ldh=8, y=20480, ldy=8, q=24576, ldq=8, scales=28672, dy=32768, lddy=8,
                dh=36864, lddh=8, dx=40960, lddx=8, dw=45056)
    args.update(change)
    a = args
    lead = (a["T"], a["D"], a["type"], a["x"], a["ldx"], a["residual"], a["ldr"], a["weight"],
            a["wtype"], a["eps"], a["h"], a["ldh"])
    if name == "norm":
        return lib.sgemm_rms_norm(*lead, a["y"], a["ldy"], None)
    if name == "q8":
        return lib.sgemm_rms_norm_q8(*lead, a["q"], a["ldq"], a["scales"], None)
    return lib.sgemm_rms_norm_backward(*lead[:10], a["dy"], a["lddy"], a["dh"], a["lddh"], a["dx"],
                                       a["lddx"], a["dw"], None)


@pytest.mark.parametrize("name", ["norm", "q8", "backward"])
@pytest.mark.parametrize("change", [
    dict(T=-1), dict(D=-1), dict(type=3), dict(type=1, wtype=2), dict(wtype=5), dict(eps=-1.0),
    dict(eps=float("nan")), dict(ldx=7), dict(x=None), dict(x=4098), dict(weight=None), dict(weight=12290)])
def test_invalid_arguments(name, change):
    sg.build()
    assert call(name, **change) == 1


@pytest.mark.parametrize("name,change", [
    ("norm", dict(ldr=7)), ("norm", dict(ldh=7)), ("norm", dict(ldy=7)), ("norm", dict(y=None)),
    ("norm", dict(y=20482)), ("norm", dict(residual=8194)), ("norm", dict(h=16386)), ("q8", dict(ldq=7)),
    ("q8", dict(q=None)), ("q8", dict(scales=None)), ("q8", dict(scales=28673)), ("backward", dict(lddy=7)),
    ("backward", dict(dy=None)), ("backward", dict(ldr=7)), ("backward", dict(residual=8194)), ("backward", dict(dy=32770)), ("backward", dict(lddh=7)),
    ("backward", dict(dh=36866)), ("backward", dict(lddx=7)), ("backward", dict(dx=40962)),
    ("backward", dict(dw=45058))])
def test_invalid_arguments_of_one_call(name, change):
    sg.build()
    assert call(name, **change) == 1


def test_sizes_that_are_too_large_or_empty():
    sg.build()
    for name in ("norm", "q8", "backward"):
        assert call(name, D=2 ** 26 + 1, **{k: 2 ** 27 for k in ("ldx", "ldr", "ldh", "ldy", "ldq", "lddy",
                                                                  "lddh", "lddx")}) == 7
        assert call(name, T=2 ** 31) == 7
    assert call("norm", T=0, x=None, y=None, h=None, residual=None) == 0
    assert call("norm", D=0) == 0
    assert call("q8", T=0) == 0
    assert call("backward", D=0) == 0
    assert call("backward", dx=None, dw=None) == 0


@gpu
def test_wrapper_refusals(device):
    x, w = torch.randn(4, 8, device="cuda"), torch.ones(8, device="cuda")
    bad = [
        (TypeError, lambda: sg.rms_norm(x.double(), w)), (TypeError, lambda: sg.rms_norm(x, w.half())),
        (TypeError, lambda: sg.rms_norm(x.half(), w.bfloat16())), (ValueError, lambda: sg.rms_norm(x[0], w)),
        (ValueError, lambda: sg.rms_norm(x, w[:7])), (ValueError, lambda: sg.rms_norm(x, w, residual=x[:3])),
        (TypeError, lambda: sg.rms_norm(x, w, residual=x.half())), (ValueError, lambda: sg.rms_norm(x.t(), w[:4])),
        (ValueError, lambda: sg.rms_norm(x[:1].expand(4, 8), w)), (ValueError, lambda: sg.rms_norm(x, w.cpu())),
        (ValueError, lambda: sg.rms_norm(x, torch.ones(16, device="cuda")[::2])),
        (ValueError, lambda: sg.rms_norm(x, w, residual=x, y=x, h=x)),
        (ValueError, lambda: sg.rms_norm(x, w, y=x[:, :7])),
        (ValueError, lambda: sg.rms_norm_backward(x[:3], x, w)),
        (TypeError, lambda: sg.rms_norm_backward(x, x, w, dweight=torch.empty(8, device="cuda").half())),
        (ValueError, lambda: sg.rms_norm_backward(x, x, w, dx=torch.empty(1, 8, device="cuda").expand(4, 8))),
        (sg.SgemmError, lambda: sg.rms_norm(x, w, eps=-1.0))]
    for kind, refused in bad:
        with pytest.raises(kind):
            refused()
