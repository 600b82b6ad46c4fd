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
