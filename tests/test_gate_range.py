"""The gate in 8 bits where FP32 does not hold what lies between its inputs and
act(g) u: far gates, and factors whose product with the gate passes its range.

Codes are compared for equality, scales within the roundings that test_q8.py derives
(the formula in 64 bits holds every value here)."""
import math

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}
TINY = 2.0 ** -96
# Rows of few threads, in registers (several pieces a thread), and read again; on 16 bytes and off.
SIZES = [(2, 256), (3, 257), (400, 1032), (330, 1029), (3, 20008), (2, 20001)]
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


def normal(T, D, kind, seed, scale=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(T, D, generator=gen, device="cuda") * scale).to(TYPES[kind])


def act64(g, act):
    g = g.double()
    if act == sg.GATE_SILU:
        return g / (1 + torch.exp(-g))
    if act == sg.GATE_GELU:
        return g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return torch.where(g > 0, g, 0.0)


def check(got, s, u, act, share=2.0 ** -22):
    """Codes and scales of rows s * u; an element with the s of the row's largest has the
    quotient of the two u, which may lie exactly between two codes (ReLU: the products
    are exact, and so is 127 times their quotient where it is short)."""
    q, scales = got
    a, u = s * u.double(), u.double()
    top = a.abs().amax(1, keepdim=True)
    want = torch.round(a * 127 / top.clamp(min=TINY))
    if act != sg.GATE_RELU:
        at = a.abs().argmax(1, keepdim=True)
        t = (u * 127 / u.gather(1, at).abs()) * (s / s.gather(1, at).abs())
        want = torch.where(top > TINY, torch.round(t), want)
    want = want.to(torch.int8)
    assert torch.equal(q, want), f"{int((q != want).sum())} of {q.numel()} codes differ"
    limit = (top.clamp(min=TINY) / 127).view(-1)
    assert ((scales.double() - limit).abs() <= share * limit).all()


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("T,F", SIZES)
def test_far_gates_below_zero(device, T, F, act, kind):
    # act(g) u is zero there, whatever the cube of g is in FP32; the other elements are of size one.
    for far in (-1e4, -2e13, -1e14, -1e20, -1e30, -3e38):
        g, u = normal(T, F, kind, 1, 2.0), normal(T, F, kind, 2)
        for column in (0, F // 2 + 3, F - 1):
            g[:, column] = far
        u[:, F - 1] = 1e8
        check(sg.gate_q8(g, u, activation=act), act64(g, act), u, act)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("T,F", SIZES)
def test_far_gates_above_zero(device, T, F, act, kind):
    # act(g) u is g u: of size one with a small u, of the gate's size with one of one.
    for far, small in ((1e4, 1e-4), (2e13, 1e-13), (1e20, 1e-20), (1e30, 1e-30), (3e38, 1e-37)):
        for factor in (small, 0.75):
            g, u = normal(T, F, kind, 3, 2.0), normal(T, F, kind, 4)
            for column in (1, F // 2 + 3, F - 2):
                g[:, column] = far
                u[:, column] *= factor
            u[0, 1] = 0.0
            a = act64(g, act)
            top = (a * u.double()).abs().amax(1)
            fine, beyond = top < 3.40e38, top > 3.41e38  # (FP32 ends at 3.4028e38)
            q, scales = sg.gate_q8(g, u, activation=act)
            check((q[fine], scales[fine]), a[fine], u[fine], act)
            assert bool(torch.isnan(scales[beyond]).all()) and bool((q[beyond] == 0).all())


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("T,F", SIZES)
def test_products_with_the_gate_beyond_the_range(device, T, F, act, kind):
    # g u passes FP32, act(g) u does not: -2 and 3e38 in SiLU are -7e37.
    for low in (-90.0, -60.0, -30.0, -12.0):
        g = torch.linspace(low, low + 9.5, F, device="cuda").to(TYPES[kind]).expand(T, F).contiguous()
        u = ((1 + 0.2 * normal(T, F, "fp32", 5).clamp(-3, 3)) * 1.5e38).to(TYPES[kind])
        u[0] *= 1e-3
        check(sg.gate_q8(g, u, activation=act), act64(g, act), u, act)
    g, u = normal(T, F, kind, 6, 2.0).abs().neg(), normal(T, F, kind, 7)
    g[:, F - 3], u[:, F - 3] = -2.0, 3e38
    check(sg.gate_q8(g, u, activation=act), act64(g, act), u, act)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("F", [257, 1032, 20008])
def test_what_is_not_finite_stays_so(device, F, act, kind):
    inf, nan = float("inf"), float("nan")
    # The last row's product is beyond FP32; zero gates of infinite factors are NaN.
    pairs = [(inf, 1.0), (inf, -1e-30), (-inf, 1.0), (nan, 1.0), (1.0, nan), (1.0, inf), (-50.0, inf),
             (0.0, inf), (-1e20, inf), (-1e20, nan), (nan, inf), (1e30, 1e30)]
    for T in (len(pairs) + 1, 400):
        g, u = normal(T, F, kind, 8, 2.0), normal(T, F, kind, 9)
        for row, (a, b) in enumerate(pairs):
            g[row, (37 * row + 5) % F], u[row, (37 * row + 5) % F] = a, b
        if act == sg.GATE_RELU:
            g[2, (37 * 2 + 5) % F] = inf  # (ReLU of minus infinity is zero)
        q, scales = sg.gate_q8(g, u, activation=act)
        n = len(pairs)
        assert bool(torch.isnan(scales[:n]).all()) and bool((q[:n] == 0).all())
        check((q[n:], scales[n:]), act64(g[n:], act), u[n:], act)
