"""The norm's gradient over the range of its rows: the formula in 64 bits, element by
element, with rows whose r^3 (r = 1 / sqrt(mean(h^2) + eps)) FP32 does not hold.

Bounds as test_norm.py derives them: `slack` of a share for the sums and roundings, of
the sum of the terms' magnitudes (its bound is relative, so the rows' size does not enter
while squares, n h and the results are in FP32's range), half a unit of the result, and
half a unit of the smallest values."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
UNIT = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


def within(got, want, share, mass):
    slack = share * mass
    limit = slack + UNIT[got.dtype] * (want.abs() + slack) + 2.0 ** (-133 if got.dtype == torch.bfloat16 else -149)
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (err <= limit).all(), f"worst {float((err / limit).max()):.3g}"


def operands(T, D, kind, size, seed=1):
    """h of this size, dy partly along it (so that the second term of dx counts), dh of the
    size that dx has, and the weight."""
    gen = torch.Generator("cuda").manual_seed(seed)
    h, dy, dh = (torch.randn(T, D, generator=gen, device="cuda") for _ in range(3))
    w = 1 + 0.3 * torch.randn(D, generator=gen, device="cuda")
    dy = dy + h
    return [t.to(TYPES[kind]) for t in (h * size, dy, dh / size)] + [w]


def compare(h, dy, dh, w, eps, residual=None):
    T, D = h.shape
    hd = h.double() if residual is None else h.double() + residual.double()
    n = dy.double() * w.double()
    r = 1 / (hd.square().mean(1, keepdim=True) + eps).sqrt()
    unit = hd * r
    want = r * (n - unit * (n * unit).mean(1, keepdim=True)) + dh.double()
    mass = r * (n.abs() + unit.abs() * (n * unit).abs().mean(1, keepdim=True)) + dh.double().abs()
    dx, dw = sg.rms_norm_backward(dy, h, w, residual=residual, dh=dh, eps=eps)
    share = 2.0 ** -18 if D <= 8192 else 2.0 ** -16
    within(dx, want, share, mass)
    terms = dy.double() * unit
    within(dw, terms.sum(0), share + (T + 40) * 2.0 ** -24, terms.abs().sum(0))


# Rows of one piece a thread, of more (FP32: up to four), with the weight's gradient in shared
# memory (16 bits), and read again; on 16 bytes and off.
SIZES = [(3, 264), (400, 1029), (160, 8192), (20, 7001), (155, 10504), (160, 9001), (3, 20008), (2, 16401)]


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D", SIZES)
def test_large_rows(device, T, D, kind):
    # (their squares add up to 2 10^38 at most)
    for size in (1e12, 1e14, 1e15, 5e16):
        compare(*operands(T, D, kind, size), 1e-5)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D", SIZES)
def test_small_rows_without_eps(device, T, D, kind):
    for size in (1e-11, 1e-13, 1e-14, 1e-16):
        compare(*operands(T, D, kind, size), 0.0)


@gpu
@pytest.mark.parametrize("size,eps", [(1e18, 1e-5), (1e-18, 0.0), (1e-16, 1e-30), (1e-13, 1e-28)])
def test_the_ends_of_the_range(device, size, eps):
    for T, D in ((5, 200), (200, 67)):
        h, dy, dh, w = operands(T, D, "fp32", size)
        compare(h, dy, dh, w, eps)
        compare(h, dy, dh, w, eps, residual=(h * 0.5).roll(1, 1))


@gpu
def test_small_gradients_of_large_rows(device):
    # dy r leaves FP32's normal range, dy (h r) does not.
    h, dy, dh, w = operands(300, 520, "fp32", 1e17)
    dy = dy * 1e-25
    unit = h.double() / (h.double().square().mean(1, keepdim=True) + 1e-5).sqrt()
    terms = dy.double() * unit
    dw = sg.rms_norm_backward(dy, h, w, eps=1e-5, need_dx=False)[1]
    within(dw, terms.sum(0), 2.0 ** -18 + 340 * 2.0 ** -24, terms.abs().sum(0))


@gpu
@pytest.mark.parametrize("D", [264, 1029, 20001])
def test_rows_whose_squares_pass_the_range(device, D):
    # r counts as zero there: dx is dh, and the row adds nothing to dweight.
    h, dy, dh, w = operands(4, D, "fp32", 1.0)
    h[1] *= 1e21
    dx, dw = sg.rms_norm_backward(dy, h, w, dh=dh, eps=1e-5)
    assert torch.equal(dx[1], dh[1])
    keep = [0, 2, 3]
    other = sg.rms_norm_backward(dy[keep], h[keep], w, dh=dh[keep], eps=1e-5)
    assert torch.equal(dx[keep], other[0])
    terms = dy[keep].double() * h[keep].double() / (h[keep].double().square().mean(1, keepdim=True) + 1e-5).sqrt()
    within(dw, terms.sum(0), 2.0 ** -16, terms.abs().sum(0))
