"""Products with 4-bit weights: against the formula in 64 bits, element by
element; quantisation against its definition; refusals.

The bound.  A group's sum runs over products x (q - z), or with 16-bit x over
x q or x (128 + q) with z or 128 + z times the sum of x taken off afterwards:
its G / 16 additions and a few roundings around it lose at most
(G / 16 + 8) 2^-23 of the sum of |x| times the largest factor, W = 15 (FP32),
32 (fp16) or 288 (bf16: 143 + 143, and room).  The groups' scaled sums and those
of the warps and CTAs add at most (K / G + 64) 2^-24 of the sum of
|x| |s (q - z)|.  The output is rounded once.
"""
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

TYPES = {"fp32": (torch.float32, 2.0 ** -24, 15.0), "fp16": (torch.float16, 2.0 ** -11, 32.0),
         "bf16": (torch.bfloat16, 2.0 ** -8, 288.0)}
gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


def nibbles(words, K):
    w = words.to(torch.int64) & 0xFFFFFFFF
    return torch.stack([(w >> (4 * i)) & 15 for i in range(8)], 1).reshape(-1, words.shape[1])[:K]


def spread(t, pad, offset, fill):
    """The same values with rows `pad` elements further apart, `offset` elements
    into a larger buffer of `fill`."""
    n, m = t.shape
    flat = torch.full((n * (m + pad) + offset + 8,), fill, device=t.device, dtype=t.dtype)
    view = flat[offset:offset + n * (m + pad)].view(n, m + pad)[:, :m]
    view.copy_(t)
    return view


def make(M, K, N, G, kind, zeros, pad=0, offset=0, seed=11):
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype = TYPES[kind][0]
    groups = -(-K // G)
    q = torch.randint(-2 ** 31, 2 ** 31, (-(-K // 8), N), generator=gen, device="cuda").to(torch.int32)
    s = ((torch.rand(groups, N, generator=gen, device="cuda") + 0.25) * 0.05).to(dtype)
    z = torch.randint(0, 16, (groups, N), generator=gen, device="cuda").to(torch.uint8) if zeros else None
    x = torch.randn(M, K, generator=gen, device="cuda").to(dtype)
    if pad or offset:
        q, s = spread(q, pad, offset, -1), spread(s, pad, offset, float("nan"))
        x = spread(x, pad, offset, float("nan"))
        z = spread(z, pad, offset, 255) if zeros else None
    return x, q, s, z


def formula(x, q, s, z, G):
    K = x.shape[1]
    group = torch.arange(K, device=x.device) // G
    w = nibbles(q, K).double() - (z.double()[group] if z is not None else 8.0)
    w = w * s.double()[group]
    return x.double() @ w, x.double().abs() @ w.abs(), x.double().abs() @ s.double()[group]


def check(x, q, s, z, G, kind):
    dtype, unit, widest = TYPES[kind]
    M, K = x.shape
    y = sg.W4Matrix(q, s, K, G, zeros=z).matvec(x)
    want, mass, scaled = formula(x, q, s, z, G)
    slack = (G / 16 + 8) * 2.0 ** -23 * widest * scaled + (K / G + 64) * 2.0 ** -24 * mass
    limit = slack + unit * (want.abs() + slack) + (2.0 ** -24 if kind == "fp16" else 0.0)
    err = (y.double() - want).abs()
    assert y.dtype == dtype and torch.isfinite(y).all()
    assert (err <= limit).all(), f"worst {float((err / limit).max()):.3g}"
    assert sg.device_status(torch.cuda.current_stream()) == 0
    return y


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M,K,N,G", [
    (1, 1, 1, 32), (1, 7, 3, 32), (1, 8, 16, 32), (1, 128, 64, 128), (1, 129, 65, 32), (1, 1000, 1025, 32),
    (1, 4096, 512, 128), (1, 2050, 96, 64), (2, 300, 48, 96), (3, 520, 130, 160), (5, 640, 208, 64),
    (8, 333, 77, 32), (9, 512, 128, 128), (16, 1024, 272, 64), (17, 96, 40, 32), (33, 256, 256, 256)])
def test_matvec(device, M, K, N, G, zeros, kind):
    check(*make(M, K, N, G, kind, zeros), G, kind)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("pad,offset", [(16, 0), (16, 16), (4, 0), (1, 0), (16, 1), (3, 5)])
def test_strides_and_alignment(device, pad, offset, kind):
    check(*make(3, 520, 96, 64, kind, True, pad, offset), 64, kind)
    check(*make(1, 256, 64, 32, kind, True, pad, offset), 32, kind)


@gpu
@pytest.mark.parametrize("kind", TYPES)
def test_x_larger_than_its_staging(device, kind):
    check(*make(16, 24000, 64, 128, kind, True), 128, kind)


@gpu
@pytest.mark.parametrize("kind", TYPES)
def test_whole_numbers_are_exact(device, kind):
    # Small whole x and scale 1: every partial sum is a whole number below 2^24,
    # and the outputs here fit the type (|y| <= 128).
    gen = torch.Generator("cuda").manual_seed(2)
    dtype = TYPES[kind][0]
    K, N, G = 512, 80, 64
    _, q, s, z = make(1, K, N, G, kind, True)
    x = torch.zeros(3, K, device="cuda", dtype=dtype)
    for m in range(3):
        at = torch.randperm(K, generator=gen, device="cuda")[:4]
        x[m, at] = torch.randint(-2, 3, (4,), generator=gen, device="cuda").to(dtype)
    y = sg.W4Matrix(q, torch.ones_like(s), K, G, zeros=z).matvec(x)
    assert torch.equal(y.double(), formula(x, q, torch.ones_like(s), z, G)[0])


@gpu
def test_unused_nibbles_and_columns_do_not_matter(device):
    x, q, s, z = make(2, 75, 40, 32, "bf16", True)
    first = sg.W4Matrix(q, s, 75, 32, zeros=z).matvec(x)
    other = q.clone()
    other[-1] ^= torch.tensor(-1 << 12, device="cuda", dtype=torch.int32)  # values 3 to 7 of the last row
    assert torch.equal(sg.W4Matrix(other, s, 75, 32, zeros=z).matvec(x), first)
    wide = torch.full((2, 50), 7.0, device="cuda", dtype=torch.bfloat16)
    sg.W4Matrix(q, s, 75, 32, zeros=z).matvec(x, wide[:, 3:43])
    assert torch.equal(wide[:, 3:43], first)
    wide[:, 3:43] = 7.0
    assert bool((wide == 7.0).all())


@gpu
def test_rows_are_independent(device):
    x, q, s, z = make(4, 256, 48, 64, "fp16", True)
    w = sg.W4Matrix(q, s, 256, 64, zeros=z)
    clean = w.matvec(x)
    x[1, 3], x[2, 9] = float("nan"), float("inf")
    y = w.matvec(x)
    assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
    assert torch.equal(y[[0, 3]], clean[[0, 3]])


@gpu
@pytest.mark.parametrize("kind", TYPES)
def test_the_range_of_x(device, kind):
    # The largest x that the stated ranges allow, against the same bound; an infinity
    # is an infinity or NaN with FP32 as q - z has it, else not finite.
    K, N, G = 256, 80, 64
    x, q, s, z = make(2, K, N, G, kind, True)
    s.fill_(2.0 ** -20)
    x = (x / x.abs().max() * {"fp32": 2.0 ** 113, "fp16": 65504.0, "bf16": 2.0 ** 113}[kind]).to(x.dtype)
    check(x, q, s, z, G, kind)
    w = sg.W4Matrix(q, s, K, G, zeros=z)
    x = torch.zeros_like(x)
    x[0, 70], x[1, 3] = float("inf"), 1.0
    y = w.matvec(x)
    step = nibbles(q, K)[70].long() - z[70 // G].long()
    if kind == "fp32":
        assert torch.equal(torch.isnan(y[0]), step == 0)
        assert torch.equal(y[0][step != 0], step[step != 0] * float("inf"))
    else:
        assert not torch.isfinite(y[0]).any()
    assert torch.isfinite(y[1]).all()


@gpu
def test_same_bits_every_time_and_on_any_stream(device):
    x, q, s, z = make(1, 8192, 96, 64, "bf16", True)
    w = sg.W4Matrix(q, s, 8192, 64, zeros=z)
    first = w.matvec(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        y = w.matvec(x, stream=side)
        side.synchronize()
        assert torch.equal(y, first)


@gpu
def test_offsets_beyond_32_bits(device):
    # 4096 rows of 2^20 + 16 words: more than 2^32 of them.
    K, N, G = 32768, 2 ** 20 + 16, 128
    q = torch.zeros(K // 8, N, device="cuda", dtype=torch.int32)
    gen = torch.Generator("cuda").manual_seed(4)
    q[-2:] = torch.randint(-2 ** 31, 2 ** 31, (2, N), generator=gen, device="cuda").to(torch.int32)
    s = torch.ones(K // G, N, device="cuda", dtype=torch.float16)
    x = torch.zeros(1, K, device="cuda", dtype=torch.float16)
    x[0, -16:] = torch.randint(-3, 4, (16,), generator=gen, device="cuda").half()
    y = sg.W4Matrix(q, s, K, G).matvec(x)
    want = x[:, -16:].double() @ (nibbles(q[-2:], 16).double() - 8)
    assert torch.equal(y.double(), want)


@gpu
def test_nothing_to_do(device):
    e = lambda *shape, **k: torch.empty(*shape, device="cuda", **k)  # noqa: E731
    w = sg.W4Matrix(e(0, 16, dtype=torch.int32), e(0, 16), 0, 32)
    assert bool((w.matvec(e(3, 0)) == 0).all())
    w = sg.W4Matrix(e(2, 0, dtype=torch.int32), e(1, 0), 16, 32)
    assert w.matvec(e(3, 16)).shape == (3, 0)
    w = sg.W4Matrix(e(2, 8, dtype=torch.int32), e(1, 8), 16, 32)
    assert w.matvec(e(0, 16)).shape == (0, 8)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("K,N,G", [(64, 40, 32), (300, 33, 128), (1, 5, 32), (1000, 257, 64)])
def test_quantize(device, K, N, G, zeros, kind):
    gen = torch.Generator("cuda").manual_seed(9)
    w = torch.randn(K, N, generator=gen, device="cuda").to(TYPES[kind][0])
    w[: min(K, G), 0] = 0
    got = sg.w4_quantize(w, G, zeros=zeros)
    groups = -(-K // G)
    pad = torch.zeros(groups * G, N, device="cuda")
    pad[:K] = w.float()
    pad = pad.view(groups, G, N)
    lo, hi = pad.amin(1).clamp(max=0), pad.amax(1).clamp(min=0)
    span = (hi - lo) / 15 if zeros else torch.maximum(hi, -lo) / 7
    scale = span.to(w.dtype)
    # (a division may round the other way in the last bit of a type's rounding)
    assert torch.allclose(got.scales.float(), scale.float(), rtol=TYPES[kind][1] * 4, atol=0)
    scale = got.scales.float()
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    if zeros:
        z = torch.where(scale > 0, (-lo / safe).round().clamp(0, 15), torch.zeros_like(scale))
        assert torch.equal(got.zeros.float(), z)
    else:
        z = torch.full_like(scale, 8)
    q = ((pad / safe.unsqueeze(1)).round() + z.unsqueeze(1)).clamp(0, 15)
    q = torch.where((scale > 0).unsqueeze(1), q, z.unsqueeze(1)).view(-1, N)[:K]
    assert torch.equal(nibbles(got.qweight, K).float(), q)
    # A weight is at most half a step off, or what clamping and rounding the
    # scale take at the ends (a step).
    back = (nibbles(got.qweight, K).float() - z.repeat_interleave(G, 0)[:K]) * \
        scale.repeat_interleave(G, 0)[:K]
    assert bool(((back - w.float()).abs() <= 1.01 * scale.repeat_interleave(G, 0)[:K] + 1e-30).all())


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_does_not_hide_infinities_and_nan(device, zeros, kind):
    gen = torch.Generator("cuda").manual_seed(10)
    w = torch.randn(96, 40, generator=gen, device="cuda").to(TYPES[kind][0])
    clean = sg.w4_quantize(w, 32, zeros=zeros)
    w[40, 3], w[41, 5], w[70, 3], w[71, 9] = float("nan"), float("inf"), -float("inf"), float("nan")
    got = sg.w4_quantize(w, 32, zeros=zeros)
    spoilt = torch.zeros(3, 40, dtype=torch.bool, device="cuda")
    for g, n in ((1, 3), (1, 5), (2, 3), (2, 9)):
        spoilt[g, n] = True
    assert torch.equal(~torch.isfinite(got.scales), spoilt)
    assert torch.equal(got.scales[~spoilt], clean.scales[~spoilt])
    y = got.matvec(torch.ones(2, 96, device="cuda", dtype=w.dtype))
    assert torch.equal(torch.isnan(y).any(0), spoilt.any(0))


# ---- refusals (no device needed) ------------------------------------------------

def call(**over):
    a = dict(M=2, N=32, K=64, group=32, type=2, x=4096, ldx=64, q=8192, ldq=32, s=16384, lds=32,
             z=32768, ldz=32, y=65536, ldy=32)
    a.update(over)
    sg.build()
    return sg.library().sgemm_w4_matvec(*(a[k] for k in (
        "M", "N", "K", "group", "type", "x", "ldx", "q", "ldq", "s", "lds", "z", "ldz", "y", "ldy")), None)


@pytest.mark.parametrize("over", [
    dict(M=-1), dict(N=-1), dict(K=-1), dict(group=0), dict(group=-32), dict(group=48), dict(type=3),
    dict(ldx=63), dict(ldq=31), dict(lds=31), dict(ldz=31), dict(ldy=31), dict(x=None), dict(q=None),
    dict(s=None), dict(y=None), dict(x=4097), dict(q=8194), dict(s=16385), dict(y=65537)])
def test_matvec_refuses(over):
    assert call(**over) == 1


def test_sizes_beyond_the_limit_are_unsupported():
    assert call(M=2 ** 20 + 1) == 7
    big = 2 ** 30 + 1
    assert call(N=big, ldq=big, lds=big, ldz=big, ldy=big) == 7


def test_empty_products_need_no_device():
    assert call(M=0) == 0 and call(N=0) == 0


@pytest.mark.parametrize("args", [
    (-1, 64, 32, 0, 4096, 32, 8192, 32, 16384, 32, None, 32), (32, 64, 33, 0, 4096, 32, 8192, 32, 16384, 32, None, 32),
    (32, 64, 32, 5, 4096, 32, 8192, 32, 16384, 32, None, 32), (32, 64, 32, 0, None, 32, 8192, 32, 16384, 32, None, 32),
    (32, 64, 32, 0, 4096, 31, 8192, 32, 16384, 32, None, 32), (32, 64, 32, 0, 4096, 32, None, 32, 16384, 32, None, 32),
    (32, 64, 32, 0, 4096, 32, 8192, 32, None, 32, None, 32), (32, 64, 32, 0, 4096, 32, 8192, 32, 16384, 32, 4096, 31)])
def test_quantize_refuses(args):
    sg.build()
    assert sg.library().sgemm_w4_quantize(*args, None) == 1


@gpu
def test_wrapper_refuses(device):
    x, q, s, z = make(2, 64, 32, 32, "bf16", True)
    for kw in (dict(group=30), dict(K=80), dict(K=48)):
        a = dict(K=64, group=32)
        a.update(kw)
        with pytest.raises(ValueError):
            sg.W4Matrix(q, s, a["K"], a["group"], zeros=z)
    with pytest.raises(TypeError):
        sg.W4Matrix(q.long(), s, 64, 32)
    with pytest.raises(TypeError):
        sg.W4Matrix(q, s.double(), 64, 32)
    with pytest.raises(TypeError):
        sg.W4Matrix(q, s, 64, 32, zeros=z.to(torch.int32))
    w = sg.W4Matrix(q, s, 64, 32, zeros=z)
    with pytest.raises(TypeError):
        w.matvec(x.float())
    with pytest.raises(ValueError):
        w.matvec(x[:, :63])
    with pytest.raises(ValueError):
        w.matvec(x, torch.empty(2, 31, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        w.matvec(x.cpu())


@gpu
def test_broadcast_tensors_are_refused(device):
    x, q, s, z = make(2, 64, 32, 32, "bf16", True)
    for a in ((q[:1].expand(8, 32), s, z), (q, s[:1].expand(2, 32), z), (q, s, z[:1].expand(2, 32))):
        with pytest.raises(ValueError):
            sg.W4Matrix(a[0], a[1], 64, 32, zeros=a[2])
    w = sg.W4Matrix(q, s, 64, 32, zeros=z)
    with pytest.raises(ValueError):
        w.matvec(x[:1].expand(2, 64))
    with pytest.raises(ValueError):
        w.matvec(x, torch.empty(1, 32, device="cuda", dtype=torch.bfloat16).expand(2, 32))
    with pytest.raises(ValueError):
        sg.w4_quantize(x[:1].expand(64, 64), 32)
