"""Scales of rows in 8 bits: the row's largest magnitude over 127, rounded once where that
is a value of the input, twice where it is a product."""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D", [(3000, 40), (5000, 33), (200, 20001)])
def test_rows_and_weights_have_the_same(device, T, D, kind):
    x = torch.randn(T, D, generator=torch.Generator("cuda").manual_seed(T), device="cuda").to(TYPES[kind])
    scales = sg.rows_q8(x)[1]
    want = x.double().abs().amax(1) / 127
    # Half a unit of the last place, 2^-24 of the value.
    assert ((scales.double() - want).abs() <= 2.0 ** -24 * want).all()
    assert torch.equal(sg.q8_quantize(x.t().contiguous()).scales, scales)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("T,D", [(3000, 40), (5000, 33), (200, 20001)])
def test_gate(device, T, D, act, kind):
    gen = torch.Generator("cuda").manual_seed(D + act)
    g, u = (torch.randn(T, D, generator=gen, device="cuda").to(TYPES[kind]) for _ in range(2))
    s = g.double()
    if act == sg.GATE_SILU:
        s = s / (1 + torch.exp(-s))
    elif act == sg.GATE_GELU:
        s = s / (1 + torch.exp(-2 * (2 / torch.pi) ** 0.5 * (s + 0.044715 * s ** 3)))
    else:
        s = s.clamp(min=0)
    want = (s * u.double()).abs().amax(1) / 127
    # The product's rounding and the quotient's (the gate has some 46 bits).
    assert ((sg.gate_q8(g, u, activation=act)[1].double() - want).abs() <= (2.0 ** -23 + 2.0 ** -40) * want).all()
