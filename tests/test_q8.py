"""Operators in 8 bits: codes equal to the formula's in 64 bits, scales and products
within their roundings, products of any size exact before they are scaled; refusals.

Bounds.  A scale is top (a product of two FP32 values, rounded), times the norm's root
(off by at most 2^-18, see the norm's tests), over 127: below 2^-22 without the
norm, below 2^-17.5 with it.  A product's sum is exact; its rounding to FP32 and two
scalings are off by at most 3 2^-24 (and 2^-47), y's rounding by half a unit.
"""
import math

import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

TYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
UNIT = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -133}
EPS = 1e-5
TINY = 2.0 ** -96
ZERO = float(torch.tensor(TINY) / 127)  # the scale of a row of zeros, FP32
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


def spread(t, pad, offset=0, fill=None):
    """The same values with rows `pad` elements further apart, `offset` elements
    into a larger buffer of `fill`."""
    n, m = t.shape
    fill = (float("nan") if t.is_floating_point() else 99) if fill is None else fill
    flat = torch.full((n * (m + pad) + offset + 8,), fill, device=t.device, dtype=t.dtype)
    view = flat[offset:offset + n * (m + pad)].view(n, m + pad)[:, :m]
    view.copy_(t)
    return view


def normal(T, D, kind, seed=1, scale=1.0):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.randn(T, D, generator=gen, device="cuda") * scale).to(TYPES[kind])


def codes(a):
    """Codes of rows of doubles, and their largest magnitudes."""
    top = a.abs().amax(1, keepdim=True).clamp(min=TINY) if a.shape[1] else \
        torch.full((a.shape[0], 1), TINY, device=a.device, dtype=torch.float64)
    return torch.round(a * 127 / top).to(torch.int8), top


def gate_codes(s, u):
    """Codes of rows s * u, s rounded to 64 bits: where an element has the s of the row's
    largest, their quotient is that of the two u, and may lie exactly between two codes."""
    a = s * u
    q, top = codes(a)
    if not a.shape[1]:
        return q, top
    at = a.abs().argmax(1, keepdim=True)
    t = (u * 127 / u.gather(1, at).abs()) * (s / s.gather(1, at).abs())
    return torch.where(top > TINY, torch.round(t).to(torch.int8), q), top


def check(got, a, root=None, share=2.0 ** -22, u=None):
    q, scales = got[:2]
    want, top = codes(a) if u is None else gate_codes(a, u)
    assert q.dtype == torch.int8 and scales.dtype == torch.float32
    assert torch.equal(q, want), f"{int((q != want).sum())} of {q.numel()} codes differ"
    limit = top / 127 if root is None else top / 127 * root
    assert ((scales.double() - limit.view(-1)).abs() <= share * limit.view(-1) + 2.0 ** -149).all()
    assert sg.device_status(torch.cuda.current_stream()) == 0


SIZES = [(1, 1), (1, 7), (1, 4096), (2, 8), (3, 31), (5, 129), (33, 1000), (4, 2047), (310, 520),
         (400, 1025), (9, 4104), (2, 8191), (3, 16384), (2, 16392), (2, 40001), (700, 5336)]


# ---- rows, the norm and the gate in 8 bits -----------------------------------------

@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D", SIZES)
def test_rows(device, T, D, kind):
    x = normal(T, D, kind)
    check(sg.rows_q8(x), x.double())


@gpu
@pytest.mark.parametrize("kind,wkind", [("fp32", "fp32"), ("fp16", "fp16"), ("bf16", "fp32"),
                                        ("bf16", "bf16")])
@pytest.mark.parametrize("T,D", SIZES)
def test_norm(device, T, D, kind, wkind):
    x, r = normal(T, D, kind), normal(T, D, kind, 2, 3.0)
    w = (1 + 0.3 * normal(1, D, "fp32", 3)).view(D).to(TYPES[wkind])
    for res in (None, r):
        got = sg.rms_norm_q8(x, w, residual=res, eps=EPS)
        h = x.double() if res is None else x.double() + r.double()
        check(got, h * w.double(), 1 / (h.square().mean(1, keepdim=True) + EPS).sqrt(), 2.0 ** -15.5)
        if res is not None:
            assert torch.equal(got[2], sg.rms_norm(x, w, residual=res, eps=EPS)[1])


def act64(g, act):
    if act == sg.GATE_SILU:
        return g / (1 + torch.exp(-g))
    if act == sg.GATE_GELU:
        return g / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    return torch.where(g > 0, g, 0.0)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", [0, 1, 2])
@pytest.mark.parametrize("T,F", SIZES)
def test_gate(device, T, F, act, kind):
    both = normal(T, 2 * F, kind, 4, 2.0)
    g, u = both[:, :F], both[:, F:]
    a, b = act64(g.double(), act), u.double()
    # (ReLU: the products are exact, and so is 127 times the quotient where it is short)
    check(sg.gate_q8(g, u, activation=act), *((a * b,) if act == sg.GATE_RELU else (a,)),
          u=None if act == sg.GATE_RELU else b)


@gpu
@pytest.mark.parametrize("act", [0, 1])
def test_gate_over_its_whole_range(device, act):
    # Gates from -100 to 100 beside factors that make every one of them count in some row.
    g = torch.linspace(-100, 100, 4001, device="cuda")
    for scale in (1e-6, 1.0, 1e4, 1e20, 1e32):
        lo = [g[a:a + 500] for a in range(0, 4000, 250)]
        rows = torch.stack([t[:500] for t in lo if len(t) == 500])
        u = scale * (1 + 0.3 * normal(rows.shape[0], 500, "fp32", 5))
        check(sg.gate_q8(rows, u, activation=act), act64(rows.double(), act), u=u.double())


@gpu
def test_ties_go_to_even(device):
    # top = 127 2^-7: every odd multiple of 2^-8 lies in the middle of two codes.
    for kind in TYPES:
        x = torch.arange(-127, 128, 2, device="cuda").float().mul(2.0 ** -8)
        x = torch.cat([x, torch.tensor([127 * 2.0 ** -7], device="cuda")]).view(1, -1).to(TYPES[kind])
        check(sg.rows_q8(x), x.double())
        check(sg.rms_norm_q8(x, torch.ones(x.shape[1], device="cuda"), eps=EPS), x.double(),
              1 / (x.double().square().mean() + EPS).sqrt(), 2.0 ** -17.5)
        check(sg.gate_q8(torch.ones_like(x), x, activation=sg.GATE_RELU), x.double())


@gpu
@pytest.mark.parametrize("act", [0, 1, 2])
def test_ties_of_elements_with_the_same_gate(device, act):
    # The quotients of the u alone decide: 127 times 1, 63.5 / 127 and so on.
    gen = torch.Generator("cuda").manual_seed(3)
    g = torch.rand(40, 1, generator=gen, device="cuda").mul(6).add(0.1).bfloat16().expand(40, 254).contiguous()
    u = (torch.arange(-126, 128, device="cuda").float() / 2 * 2.0 ** -6).bfloat16().expand(40, 254).contiguous()
    u[:, 0] = 127 * 2.0 ** -6
    q, _ = sg.gate_q8(g, u, activation=act)
    assert torch.equal(q.double(), torch.round(u.double() * 64))


@gpu
def test_borders_between_codes(device):
    # Elements within a unit of the last place of a border, on both sides.
    gen = torch.Generator("cuda").manual_seed(6)
    T, D = 64, 1000
    top = torch.rand(T, 1, generator=gen, device="cuda", dtype=torch.float64).add(0.5).float()
    k = torch.randint(-126, 126, (T, D), generator=gen, device="cuda").double() + 0.5
    x = (k * top.double() / 127).float()
    step = torch.randint(-1, 2, (T, D), generator=gen, device="cuda")
    x = (x.view(torch.int32) + step.to(torch.int32)).view(torch.float32)
    x[:, 17] = top[:, 0]
    check(sg.rows_q8(x), x.double())
    w = (1 + 0.3 * normal(1, D, "fp32", 3)).view(D)
    x = (x.double() / w.double()).float()
    h = x.double()
    check(sg.rms_norm_q8(x, w, eps=EPS), h * w.double(), 1 / (h.square().mean(1, keepdim=True) + EPS).sqrt(),
          2.0 ** -17.5)


@gpu
@pytest.mark.parametrize("D", [96, 1001])
def test_rows_of_zeros_infinities_and_small_values(device, D):
    x = normal(6, D, "fp32")
    x[1] = 0
    x[2, 3] = float("inf")
    x[3, 4] = float("nan")
    x[4] *= 1e-35
    x[5] *= 1e30
    fine = [0, 1, 4, 5]
    w, one = torch.ones(D, device="cuda"), torch.ones_like(x)
    for q, scales in (sg.rows_q8(x), sg.rms_norm_q8(x, w, eps=EPS), sg.gate_q8(one, x, activation=sg.GATE_RELU)):
        want, top = codes(x[fine].double())
        assert torch.equal(q[fine], want)
        assert bool(torch.isnan(scales[[2, 3]]).all()) and bool((q[[2, 3]] == 0).all())
    q, scales = sg.rows_q8(x)
    assert float(scales[1]) == ZERO and bool((q[1] == 0).all())
    # A NaN stays in its own row of the product.
    m = sg.q8_quantize(normal(D, 24, "fp32", 9))
    y = m.matmul(q, scales)
    assert bool(torch.isnan(y[[2, 3]]).all()) and bool(torch.isfinite(y[fine]).all())


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (1, 0), (3, 5)])
@pytest.mark.parametrize("T,D", [(3, 264), (310, 1032), (3, 1029), (2, 20000)])
def test_strides_and_alignment(device, T, D, pad, offset, kind):
    x, u = (spread(normal(T, D, kind, s, 2.0), pad, offset) for s in (1, 2))
    w = torch.ones(D, device="cuda", dtype=TYPES[kind])
    q, h = spread(torch.zeros(T, D, device="cuda", dtype=torch.int8), pad, offset, 77), torch.empty_like(x)
    scales = torch.empty(T, device="cuda")
    check(sg.rows_q8(x, q=q, scales=scales), x.double())
    check(sg.gate_q8(x, u, q=q, scales=scales), act64(x.double(), 0), u=u.double())
    got = sg.rms_norm_q8(x, w, residual=u, eps=EPS, q=q, scales=scales, h=h)
    hd = x.double() + u.double()
    check(got, hd, 1 / (hd.square().mean(1, keepdim=True) + EPS).sqrt(), 2.0 ** -15.5)
    assert got[0] is q and got[1] is scales and got[2] is h
    base = q._base
    assert bool((base[:offset] == 77).all()) and bool((base[offset + T * (D + pad):] == 77).all())
    assert bool((base[offset:offset + T * (D + pad)].view(T, D + pad)[:, D:] == 77).all())


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D", [(4, 520), (400, 257), (2, 40001)])
def test_residual_updated_in_place(device, T, D, kind):
    x, r = normal(T, D, kind), normal(T, D, kind, 2, 3.0)
    w = (1 + 0.3 * normal(1, D, "fp32", 3)).view(D)
    want = sg.rms_norm_q8(x, w, residual=r)
    a, b = x.clone(), r.clone()
    got = sg.rms_norm_q8(x, w, residual=b, h=b)
    assert got[2] is b and all(torch.equal(p, q) for p, q in zip(got, want))
    got = sg.rms_norm_q8(a, w, residual=r, h=a)
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("K,N", [(1, 1), (3, 5), (128, 32), (257, 100), (1000, 1025), (4096, 96)])
def test_quantize(device, K, N, kind):
    for pad in (0, 5):
        w = spread(normal(K, N, kind, 7), pad)
        m = sg.q8_quantize(w)
        want, top = codes(w.double().t())
        assert torch.equal(m.qweight, want) and m.dtype == w.dtype
        within = top.view(-1) / 127
        assert ((m.scales.double() - within).abs() <= 2.0 ** -22 * within).all()


@gpu
def test_quantize_keeps_what_is_not_finite_in_its_channel(device):
    w = normal(70, 9, "fp32")
    w[3, 1], w[4, 2] = float("inf"), float("nan")
    w[:, 3] = 0
    m = sg.q8_quantize(w)
    assert bool(torch.isnan(m.scales[[1, 2]]).all()) and bool((m.qweight[[1, 2, 3]] == 0).all())
    y = m.matmul(*sg.rows_q8(normal(20, 70, "fp32", 2)))
    assert bool(torch.isnan(y[:, [1, 2]]).all())
    assert bool(torch.isfinite(y[:, [0, 3, 4, 5, 6, 7, 8]]).all()) and bool((y[:, 3] == 0).all())


# ---- products ---------------------------------------------------------------------

def random_codes(rows, K, seed, low=-128, high=128):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.randint(low, high, (rows, K), generator=gen, device="cuda").to(torch.int8)


def product(x, w, xs, ws, dtype, y=None):
    m = sg.Q8Matrix(w, ws, dtype=dtype)
    y = m.matmul(x, xs, y)
    # Whole numbers below 2^53: exact in 64 bits.
    want = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    limit = (3.1 * 2.0 ** -24 + UNIT[dtype]) * want.abs() * (1 + 2.0 ** -8) + LEAST[dtype]
    assert y.dtype == dtype and torch.isfinite(y).all()
    err = (y.double() - want).abs()
    assert (err <= limit).all(), f"worst {float((err / limit).max()):.3g}"
    assert sg.device_status(torch.cuda.current_stream()) == 0
    return y


def scales(n, seed, K=1):
    gen = torch.Generator("cuda").manual_seed(seed)
    return (torch.rand(n, generator=gen, device="cuda") + 0.5) * 0.01 / math.sqrt(max(K, 1))


MANY = [(9, 128, 128), (9, 1, 1), (10, 17, 300), (16, 1000, 520), (33, 130, 257), (64, 2048, 384), (96, 64, 5461),
        (97, 64, 256), (97, 1025, 700), (192, 4096, 256), (193, 257, 1000), (333, 2047, 1365), (500, 3000, 130),
        (1000, 96, 3001), (700, 1500, 5000)]
FEW = [(1, 1, 1), (1, 15, 3), (1, 16, 4), (1, 4096, 1025), (2, 513, 300), (3, 1000, 640), (4, 2047, 77),
       (5, 2050, 260), (7, 64, 40000), (8, 12288, 96), (8, 30000, 24),
       (4, 8192, 4096), (5, 5001, 5300), (8, 8192, 4096)]


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("M,K,N", MANY + FEW)
def test_product(device, M, K, N, kind):
    product(random_codes(M, K, 1), random_codes(N, K, 2), scales(M, 3, K), scales(N, 4), TYPES[kind])


@gpu
@pytest.mark.parametrize("M", [1, 8, 9, 96, 200])
@pytest.mark.parametrize("K", [1023, 1024, 1025, 2048, 5000, 131071])
def test_sums_are_exact_at_the_ends_of_the_range(device, M, K):
    # With scales of one and codes that all have the same magnitude, FP32 y is the sum
    # rounded once; -128 times -128 at every k is the largest there is.
    one = torch.ones(300, device="cuda")
    for a, b in ((-128, -128), (127, -128), (127, 127)):
        x = torch.full((M, K), a, device="cuda", dtype=torch.int8)
        w = torch.full((300, K), b, device="cuda", dtype=torch.int8)
        w[::7, ::3] = 1  # some channels with another sum
        y = sg.Q8Matrix(w, one, dtype=torch.float32).matmul(x, one[:M])
        want = (x.double() @ w.double().t()).float()
        assert torch.equal(y, want)


@gpu
@pytest.mark.parametrize("M", [8, 64, 300])
def test_products_do_not_depend_on_the_rows_beside_them(device, M):
    x, w = random_codes(M, 3000, 1), random_codes(500, 3000, 2)
    m = sg.Q8Matrix(w, scales(500, 4), dtype=torch.float32)
    xs = scales(M, 3)
    y = m.matmul(x, xs)
    for a, b in ((0, 1), (M // 2, M), (3, 8)):
        assert torch.equal(m.matmul(x[a:b].contiguous(), xs[a:b].contiguous()), y[a:b])
    assert torch.equal(m.matmul(x, xs), y)


@gpu
@pytest.mark.parametrize("M", [1, 5, 60, 250])
@pytest.mark.parametrize("pad,offset", [(16, 0), (16, 16), (1, 0), (8, 8), (3, 5)])
def test_product_strides(device, M, pad, offset):
    K, N = 1040, 333
    for dtype in TYPES.values():
        x, w = spread(random_codes(M, K, 1), pad, offset), spread(random_codes(N, K, 2), pad, offset)
        y = spread(torch.zeros(M, N, device="cuda", dtype=dtype), pad, offset, 7.0)
        product(x, w, scales(M, 3, K), scales(N, 4), dtype, y)
        base = y._base
        assert bool((base[:offset] == 7.0).all()) and bool((base[offset + M * (N + pad):] == 7.0).all())
        assert bool((base[offset:offset + M * (N + pad)].view(M, N + pad)[:, N:] == 7.0).all())


@gpu
@pytest.mark.parametrize("M", [3, 40, 200])
def test_unaligned_weights_through_the_c_call(device, M):
    # (the handle would copy them once; the call copies them itself)
    K, N = 515, 130
    x, w = random_codes(M, K, 1), spread(random_codes(N, K, 2), 2, 3)
    xs, ws, y = scales(M, 3), scales(N, 4), torch.empty(M, N, device="cuda")
    status = sg.library().sgemm_q8_matmul(
        M, N, K, 0, x.data_ptr(), K, xs.data_ptr(), w.data_ptr(), K + 2, ws.data_ptr(), y.data_ptr(), N,
        torch.cuda.current_stream().cuda_stream)
    assert status == 0
    assert torch.equal(y, sg.Q8Matrix(w, ws, dtype=torch.float32).matmul(x, xs))


@gpu
def test_empty_products(device):
    m = sg.Q8Matrix(random_codes(5, 8, 1), scales(5, 2))
    assert m.matmul(random_codes(0, 8, 1), scales(0, 1)).shape == (0, 5)
    e = sg.Q8Matrix(random_codes(5, 0, 1), scales(5, 2))
    for M in (2, 40):
        y = torch.full((M, 5), 3.0, device="cuda", dtype=torch.bfloat16)
        assert bool((e.matmul(random_codes(M, 0, 1), scales(M, 1), y) == 0).all())
    q, s = sg.rows_q8(torch.empty(3, 0, device="cuda"))
    assert q.shape == (3, 0) and bool((s == ZERO).all())
    assert sg.rows_q8(torch.empty(0, 7, device="cuda"))[0].shape == (0, 7)
    x, s = torch.empty(3, 0, device="cuda"), torch.full((3,), 5.0, device="cuda")
    q, s = sg.rms_norm_q8(x, x[0], scales=s)
    assert q.shape == (3, 0) and bool((s == ZERO).all())


@gpu
@pytest.mark.parametrize("M", [40, 200])
def test_a_wait_that_runs_out_is_reported(device, M):
    # The loads stop after two stages (of 512, which at most 152 CTAs share): every role's
    # wait ends, the call is flagged, and the next one is right again.
    x, w = random_codes(M, 65536, 1), random_codes(512, 65536, 2)
    m = sg.Q8Matrix(w, scales(512, 4), dtype=torch.float32)
    xs = scales(M, 3)
    want = m.matmul(x, xs)
    assert sg.device_status(torch.cuda.current_stream()) == 0
    try:
        sg.set_wait_timeout_ns(2_000_000, 2)
        m.matmul(x, xs)
        torch.cuda.synchronize()
        assert sg.device_status(torch.cuda.current_stream()) != 0
    finally:
        sg.set_wait_timeout_ns()
    assert torch.equal(m.matmul(x, xs), want)
    assert sg.device_status(torch.cuda.current_stream()) == 0


@gpu
@pytest.mark.parametrize("T", [4, 150])
def test_a_block_served_in_eight_bits(device, T):
    """Norm, gate and up, gate, down: each step is that of its formula on what the one
    before returned, and the whole is near the block in 64 bits."""
    D, F = 264, 1000
    x, r = normal(T, D, "bf16"), normal(T, D, "bf16", 2, 2.0)
    norm = (1 + 0.2 * normal(1, D, "fp32", 3)).view(D)
    wide, down = normal(D, 2 * F, "bf16", 4, D ** -0.5), normal(F, D, "bf16", 5, F ** -0.5)
    first, second = sg.q8_quantize(wide), sg.q8_quantize(down)
    q, s, h = sg.rms_norm_q8(x, norm, residual=r)
    gu = first.matmul(q, s)
    want = (q.double() @ first.qweight.double().t()) * s.double()[:, None] * first.scales.double()
    assert ((gu.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -21) * want.abs() + 2.0 ** -133).all()
    q2, s2 = sg.gate_q8(gu[:, :F], gu[:, F:])
    check((q2, s2), act64(gu[:, :F].double(), 0), u=gu[:, F:].double())
    y = second.matmul(q2, s2)
    hd = x.double() + r.double()
    n = hd / (hd.square().mean(1, keepdim=True) + 1e-6).sqrt() * norm.double()
    g, u = (n @ wide.double()).chunk(2, 1)
    exact = (act64(g, 0) * u) @ down.double()
    # Codes are off by half a step, top / 254 each: of a row of normal values, whose top is
    # at most 5 deviations, 1/88 of a deviation in the root mean square (a third of
    # 5/254 times root 3), at five places (norm, two weights, gate, and g and u both
    # feel the first two): below 5 %.
    assert float((y.double() - exact).norm()) <= 0.05 * float(exact.norm())


# ---- streams and graphs -------------------------------------------------------------

@gpu
@pytest.mark.parametrize("M", [3, 50, 300])
def test_captured_and_replayed(device, M):
    x, w = random_codes(M, 2000, 1), random_codes(600, 2000, 2)
    m, xs = sg.Q8Matrix(w, scales(600, 4)), scales(M, 3)
    y = torch.empty(M, 600, device="cuda", dtype=torch.bfloat16)
    m.matmul(x, xs, y)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(side):
        m.matmul(x, xs, y)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side):
        m.matmul(x, xs, y)
    for seed in (5, 6):
        x.copy_(random_codes(M, 2000, seed))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, m.matmul(x, xs))


@gpu
def test_two_streams_at_once(device):
    x, w = random_codes(200, 3000, 1), random_codes(700, 3000, 2)
    m, xs = sg.Q8Matrix(w, scales(700, 4)), scales(200, 3)
    h = normal(200, 3000, "bf16")
    norm = torch.ones(3000, device="cuda")
    dy = normal(200, 3000, "bf16", 2)
    want, grads = m.matmul(x, xs), sg.rms_norm_backward(dy, h, norm)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[(m.matmul(x, xs, stream=s), *sg.rms_norm_backward(dy, h, norm, stream=s)) for s in streams]
           for _ in range(10)]
    torch.cuda.synchronize()
    for y, dx, dw in (t for pair in got for t in pair):
        assert torch.equal(y, want) and torch.equal(dx, grads[0]) and torch.equal(dw, grads[1])


# ---- refusals ---------------------------------------------------------------------

def matmul_call(**change):
    a = dict(M=4, N=6, K=8, type=0, x=4096, ldx=8, xs=8192, w=12288, ldw=8, ws=16384, y=20480, ldy=6)
    a.update(change)
    return sg.library().sgemm_q8_matmul(a["M"], a["N"], a["K"], a["type"], a["x"], a["ldx"], a["xs"],
                                        a["w"], a["ldw"], a["ws"], a["y"], a["ldy"], None)


def gate_call(**change):
    a = dict(T=4, F=8, type=0, act=0, g=4096, ldg=8, u=8192, ldu=8, q=12288, ldq=8, s=16384)
    a.update(change)
    return sg.library().sgemm_q8_gate(a["T"], a["F"], a["type"], a["act"], a["g"], a["ldg"], a["u"],
                                      a["ldu"], a["q"], a["ldq"], a["s"], None)


def quantize_call(**change):
    a = dict(N=6, K=8, type=0, W=4096, ldw=6, q=8192, ldq=8, s=12288)
    a.update(change)
    return sg.library().sgemm_q8_quantize(a["N"], a["K"], a["type"], a["W"], a["ldw"], a["q"], a["ldq"],
                                          a["s"], None)


def test_invalid_arguments():
    sg.build()
    for change in (dict(M=-1), dict(N=-1), dict(K=-1), dict(type=3), dict(ldx=7), dict(ldw=7), dict(ldy=5),
                   dict(x=None), dict(w=None), dict(xs=None), dict(ws=None), dict(y=None), dict(y=20482),
                   dict(xs=8193), dict(ws=16386)):
        assert matmul_call(**change) == 1, change
    for change in (dict(T=-1), dict(F=-1), dict(type=-1), dict(act=3), dict(ldg=7), dict(ldu=7), dict(ldq=7),
                   dict(g=None), dict(g=4097), dict(u=8193), dict(q=None), dict(s=None), dict(s=16385)):
        assert gate_call(**change) == 1, change
    for change in (dict(N=-1), dict(K=-1), dict(type=9), dict(ldw=5), dict(ldq=7), dict(W=None), dict(W=4098),
                   dict(q=None), dict(s=None), dict(s=12290)):
        assert quantize_call(**change) == 1, change
    big = 2 ** 27
    assert matmul_call(K=131072, ldx=131072, ldw=131072) == 7
    assert matmul_call(M=2 ** 26 + 1) == 7 and matmul_call(N=2 ** 26 + 1, ldy=big) == 7
    assert gate_call(T=2 ** 31) == 7 and gate_call(F=2 ** 26 + 1, ldg=big, ldu=big, ldq=big) == 7
    assert quantize_call(N=2 ** 26 + 1, ldw=big) == 7 and quantize_call(K=2 ** 26 + 1, ldq=big) == 7
    assert matmul_call(M=0) == 0 and matmul_call(N=0) == 0 and gate_call(T=0) == 0 and quantize_call(N=0) == 0


@gpu
def test_wrapper_refusals(device):
    x, w, xs, ws = random_codes(3, 16, 1), random_codes(4, 16, 2), scales(3, 1), scales(4, 2)
    m = sg.Q8Matrix(w, ws)
    f = torch.randn(3, 16, device="cuda")
    one = torch.ones(16, device="cuda")
    bad = [
        (TypeError, lambda: sg.Q8Matrix(w.float(), ws)), (ValueError, lambda: sg.Q8Matrix(w[0], ws)),
        (ValueError, lambda: sg.Q8Matrix(w, ws[:3])), (TypeError, lambda: sg.Q8Matrix(w, ws.half())),
        (TypeError, lambda: sg.Q8Matrix(w, ws, dtype=torch.float64)),
        (ValueError, lambda: sg.Q8Matrix(w[:1].expand(4, 16), ws)), (ValueError, lambda: sg.Q8Matrix(w.cpu(), ws)),
        (ValueError, lambda: m.matmul(x[:, :15], xs)), (TypeError, lambda: m.matmul(x.float(), xs)),
        (ValueError, lambda: m.matmul(x, xs[:2])), (TypeError, lambda: m.matmul(x, xs.double())),
        (ValueError, lambda: m.matmul(x, xs.cpu())), (ValueError, lambda: m.matmul(x[0], xs)),
        (TypeError, lambda: m.matmul(x, xs, torch.empty(3, 4, device="cuda"))),
        (ValueError, lambda: m.matmul(x, xs, torch.empty(3, 5, device="cuda", dtype=torch.bfloat16))),
        (ValueError, lambda: sg.rows_q8(f[0])), (TypeError, lambda: sg.rows_q8(f.double())),
        (TypeError, lambda: sg.rows_q8(f, q=torch.empty(3, 16, device="cuda", dtype=torch.uint8))),
        (ValueError, lambda: sg.gate_q8(f, f[:2])), (TypeError, lambda: sg.gate_q8(f, f.half())),
        (sg.SgemmError, lambda: sg.gate_q8(f, f, activation=3)), (ValueError, lambda: sg.q8_quantize(f[0])),
        (ValueError, lambda: sg.rms_norm_q8(f, one, scales=torch.empty(2, device="cuda"))),
        (ValueError, lambda: sg.rows_q8(f.clone().requires_grad_())),
        (ValueError, lambda: sg.rms_norm_q8(f, one.clone().requires_grad_())),
        (ValueError, lambda: m.matmul(x, xs.clone().requires_grad_()))]
    for kind, refused in bad:
        with pytest.raises(kind):
            refused()
    with torch.no_grad():
        sg.rms_norm_q8(f, one.clone().requires_grad_())
