"""The AdamW step: parameters against the formula in 64 bits; 32-bit states bit
for bit against the formula's FP32 operations one by one; 8-bit states code for
code; many tensors, odd sizes, any alignment; refusals.

The bound on a parameter: the update's operations (two of them approximate, 2^-22
each) lose less than 2^-19 of it, its factors and the sum 2^-22 of the parameter.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

gpu = pytest.mark.gpu
DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
BLOCK = 256


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    return torch.device("cuda", 0)


def moments32(m, v, g, grad_scale):
    """m and v after a step, by single FP32 operations (numpy: each rounded)."""
    b1, b2 = HYPER["betas"]
    f = np.float32
    g = g.float().cpu().numpy() * f(grad_scale)
    m = m * f(b1) + g * f(1 - b1)
    v = v * f(b2) + (g * g) * f(1 - b2)
    return m, v


def decode(codes, scales):
    n = codes.numel()
    unit = (scales.cpu().numpy() * np.float32(1 / np.float32(448))).repeat(BLOCK)[:n]
    return codes.cpu().float().numpy() * unit


def encode(t, least=False):
    """Codes and scales of the 8-bit states, by single FP32 operations."""
    n = t.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK, np.float32)
    pad[:n] = t
    blocks = pad.reshape(-1, BLOCK)
    top = np.maximum(np.abs(blocks).max(1), np.float32(2.0 ** -96))
    q = blocks * ((np.float32(1) / top) * np.float32(448))[:, None]
    if least:
        q = np.where((blocks > 0) & (q < 2.0 ** -9), np.float32(2.0 ** -9), q)
    codes = torch.from_numpy(q.reshape(-1)[:n].copy()).to(torch.float8_e4m3fn)
    return codes, torch.from_numpy(top)


def new_param(p, m, v, step):
    """The parameter after a step, in 64 bits, from the new m and v."""
    b1, b2 = HYPER["betas"]
    m_hat, v_hat = m.astype(np.float64) / (1 - b1 ** step), v.astype(np.float64) / (1 - b2 ** step)
    update = HYPER["lr"] * m_hat / (np.sqrt(v_hat) + HYPER["eps"])
    p = p.double().cpu().numpy()
    return p * (1 - HYPER["lr"] * HYPER["weight_decay"]) - update, update


def make(sizes, p_kind, g_kind, bits, offset=0, seed=7):
    gen = torch.Generator("cuda").manual_seed(seed)

    def cut(n, dtype):
        return torch.zeros(n + offset, device="cuda", dtype=dtype)[offset:]

    out = dict(p=[], g=[], m=[], v=[], ms=[], vs=[])
    for n in sizes:
        p, g = cut(n, DTYPES[p_kind]), cut(n, DTYPES[g_kind])
        p.copy_(torch.randn(n, generator=gen, device="cuda"))
        g.copy_(torch.randn(n, generator=gen, device="cuda") *
                torch.exp(2 * torch.randn(n, generator=gen, device="cuda")) * 0.01)
        m = (0.5 * g.float() + 0.003 * torch.randn(n, generator=gen, device="cuda")).cpu().numpy()
        r = (g.float().abs() + 0.002).cpu().numpy()
        if bits == 32:
            tm, tv = cut(n, torch.float32), cut(n, torch.float32)
            tm.copy_(torch.from_numpy(m))
            tv.copy_(torch.from_numpy(r * r))
        else:
            tm, tv = (cut(n, torch.uint8).view(torch.float8_e4m3fn) for _ in range(2))
            for to, values, scales in ((tm, m, "ms"), (tv, r, "vs")):
                codes, top = encode(values, least=scales == "vs")
                to.view(torch.uint8).copy_(codes.view(torch.uint8))
                out[scales].append(top.cuda())
        for k, t in zip(("p", "g", "m", "v"), (p, g, tm, tv)):
            out[k].append(t)
    return out


def check(s, bits, p_kind, step=3, grad_scale=1.0, copies=None):
    before = [p.clone() for p in s["p"]]
    if bits == 32:
        states = [(m.cpu().numpy().copy(), v.cpu().numpy().copy()) for m, v in zip(s["m"], s["v"])]
        scales = {}
    else:
        states = []
        for m, v, ms, vs in zip(s["m"], s["v"], s["ms"], s["vs"]):
            r = decode(v, vs)
            states.append((decode(m, ms), r * r))
        scales = dict(m_scales=s["ms"], v_scales=s["vs"])
    opt = sg.AdamW(s["p"], s["g"], s["m"], s["v"], copies=copies, **scales, **HYPER)
    opt.step(step=step, grad_scale=grad_scale)
    torch.cuda.synchronize()
    unit = {"fp32": 2.0 ** -24, "fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[p_kind]
    for i, p0 in enumerate(before):
        m, v = moments32(*states[i], s["g"][i], grad_scale)
        if bits == 32:
            assert np.array_equal(s["m"][i].cpu().numpy(), m) and np.array_equal(s["v"][i].cpu().numpy(), v)
        else:
            for t, top, values, least in ((s["m"][i], s["ms"][i], m, False),
                                          (s["v"][i], s["vs"][i], np.sqrt(v), True)):
                codes, want = encode(values, least)
                assert torch.equal(top.cpu(), want)
                assert torch.equal(t.cpu().view(torch.uint8), codes.view(torch.uint8))
        want, update = new_param(p0, m, v, step)
        limit = 2.0 ** -19 * np.abs(update) + 2.0 ** -22 * np.abs(p0.double().cpu().numpy())
        limit = limit + (unit * (np.abs(want) + limit) + 2.0 ** -25 if p_kind != "fp32" else 0)
        err = np.abs(s["p"][i].double().cpu().numpy() - want)
        assert (err <= limit).all(), f"tensor {i}: worst {np.max(err / np.maximum(limit, 1e-300)):.3g}"
        if copies is not None:
            assert torch.equal(copies[i], s["p"][i].to(copies[i].dtype))
    return opt


@gpu
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("sizes", [[1], [7], [255], [256], [257], [2048], [2049], [16384], [16385, 1, 300],
                                   [5, 100003, 64, 4097, 1]])
def test_sizes(device, sizes, bits):
    check(make(sizes, "fp32", "bf16", bits), bits, "fp32")


@gpu
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("p_kind", DTYPES)
@pytest.mark.parametrize("g_kind", DTYPES)
@pytest.mark.parametrize("offset", [0, 1])
def test_types_and_alignment(device, offset, g_kind, p_kind, bits):
    check(make([3000, 513], p_kind, g_kind, bits, offset), bits, p_kind, grad_scale=0.37)


@gpu
@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("kind", DTYPES)
def test_copies(device, kind, bits):
    s = make([1000, 256, 33], "fp32", "bf16", bits)
    copies = [torch.full_like(p, 9.0, dtype=DTYPES[kind]) for p in s["p"]]
    check(s, bits, "fp32", copies=copies)


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_more_tensors_than_one_launch_takes(device, bits):
    check(make([1 + 37 * i % 700 for i in range(900)], "fp32", "fp32", bits), bits, "fp32")


@gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_states_from_nothing(device, bits):
    # First steps from zero states; some gradients are zero for good: those
    # parameters only decay.
    gen = torch.Generator("cuda").manual_seed(1)
    p = torch.randn(700, generator=gen, device="cuda")
    p0 = p.clone()
    g = torch.zeros(700, device="cuda")
    g[300:] = torch.randn(400, generator=gen, device="cuda")
    opt = sg.AdamW([p], [g], state_bits=bits, **HYPER)
    for _ in range(3):
        opt.step()
    assert opt.steps == 3
    decay = (1 - HYPER["lr"] * HYPER["weight_decay"]) ** 3
    assert torch.allclose(p[:300], p0[:300] * decay, rtol=1e-6, atol=0)
    # a constant gradient: every step moves by lr, whatever its size
    moved = (p0[300:] * decay - p[300:]) / (3 * HYPER["lr"])
    assert torch.allclose(moved.abs(), torch.ones(400, device="cuda"), rtol=0.15 if bits == 8 else 2e-3)
    assert torch.isfinite(p).all()


@gpu
def test_small_second_moments_never_become_zero(device):
    # One large gradient in the block: the others' sqrt(v) is far below the
    # smallest code, and must not turn into a division by eps.
    p = torch.zeros(256, device="cuda")
    g = torch.full((256,), 1e-7, device="cuda")
    g[0] = 100.0
    opt = sg.AdamW([p], [g], state_bits=8, **HYPER)
    for _ in range(5):
        opt.step()
    assert bool((opt.v[0].view(torch.uint8) > 0).all())
    assert float(p.abs().max()) < 10 * 5 * HYPER["lr"]


@gpu
def test_an_infinite_gradient_spoils_its_block_alone(device):
    s = make([1024], "fp32", "fp32", 8)
    clean = make([1024], "fp32", "fp32", 8)
    s["g"][0][300] = float("inf")
    for t in (s, clean):
        sg.AdamW(t["p"], t["g"], t["m"], t["v"], m_scales=t["ms"], v_scales=t["vs"], **HYPER).step(step=2)
    keep = torch.ones(1024, dtype=torch.bool)
    keep[256:512] = False
    assert torch.equal(s["m"][0].cpu().view(torch.uint8)[keep], clean["m"][0].cpu().view(torch.uint8)[keep])
    assert torch.equal(s["p"][0].cpu()[keep], clean["p"][0].cpu()[keep])
    assert torch.isinf(s["ms"][0][1]) or torch.isnan(s["ms"][0][1])


@gpu
def test_gaps_between_tensors_are_not_written(device):
    flat = torch.full((4000,), 5.0, device="cuda")
    parts = [flat[10:1000], flat[1003:1100], flat[2000:3999]]
    g = [torch.ones_like(t) for t in parts]
    sg.AdamW(parts, g, state_bits=8, **HYPER).step()
    mask = torch.ones(4000, dtype=torch.bool, device="cuda")
    for a, b in ((10, 1000), (1003, 1100), (2000, 3999)):
        mask[a:b] = False
    assert bool((flat[mask] == 5.0).all()) and bool((flat[~mask] != 5.0).all())


@gpu
def test_a_tensor_of_more_than_2_to_31_elements(device):
    n = 2 ** 31 + 777
    p, g = (torch.zeros(n, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    g[-5:] = torch.tensor([1.0, -1.0, 0.5, 2.0, -3.0], device="cuda").bfloat16()
    g[0] = 1.0
    opt = sg.AdamW([p], [g], state_bits=8, lr=0.25, weight_decay=0.0)
    opt.step()
    # a first step moves by lr against the gradient's sign
    assert p[-5:].float().cpu().tolist() == [-0.25, 0.25, -0.25, -0.25, 0.25] and float(p[0]) == -0.25
    assert int((p != 0).sum()) == 6


@gpu
def test_streams_and_new_gradients(device):
    s = make([5000], "fp32", "bf16", 32)
    other = make([5000], "fp32", "bf16", 32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    opt = sg.AdamW(s["p"], [torch.zeros_like(s["g"][0])], s["m"], s["v"], **HYPER)
    opt.set_grads(s["g"])
    torch.cuda.synchronize()
    opt.step(step=4, stream=side)
    side.synchronize()
    sg.AdamW(other["p"], other["g"], other["m"], other["v"], **HYPER).step(step=4)
    assert torch.equal(s["p"][0], other["p"][0]) and torch.equal(s["m"][0], other["m"][0])


# ---- refusals (no device needed) ------------------------------------------------

def call(entry=None, **over):
    from dense_fp32_sgemm_gb300.ffn import _AdamTensor
    t = dict(param=4096, grad=8192, m=16384, v=32768, m_scale=65536, v_scale=131072, copy=None, numel=10)
    t.update(entry or {})
    a = dict(count=1, pt=0, gt=2, ct=0, bits=8, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, wd=0.1, step=1, gs=1.0)
    a.update(over)
    sg.build()
    table = (_AdamTensor * 1)(_AdamTensor(**t))
    return sg.library().sgemm_adamw_step(table, a["count"], a["pt"], a["gt"], a["ct"], a["bits"], a["lr"],
                                         a["b1"], a["b2"], a["eps"], a["wd"], a["step"], a["gs"], None)


@pytest.mark.parametrize("entry,over", [
    (None, dict(count=-1)), (None, dict(pt=3)), (None, dict(gt=-1)), (None, dict(ct=7)), (None, dict(bits=16)),
    (None, dict(step=0)), (None, dict(b1=1.0)), (None, dict(b1=-0.1)), (None, dict(b2=1.5)),
    (None, dict(eps=-1e-9)), (None, dict(b1=float("nan"))), (dict(numel=-1), {}), (dict(param=None), {}),
    (dict(grad=None), {}), (dict(m=None), {}), (dict(v=None), {}), (dict(m_scale=None), {}),
    (dict(v_scale=None), {}), (dict(param=4097), {}), (dict(grad=8193), {}), (dict(m_scale=65537), {}),
    (dict(m=16385), dict(bits=32)), (dict(copy=4098), {})])
def test_refuses(entry, over):
    assert call(entry, **over) == 1


def test_too_many_elements_are_unsupported():
    assert call(dict(numel=2 ** 42 + 1)) == 7


def test_no_tensors_need_no_device():
    assert call(count=0) == 0


@gpu
def test_wrapper_refuses(device):
    p, g = torch.zeros(10, device="cuda"), torch.zeros(10, device="cuda")
    with pytest.raises(ValueError):
        sg.AdamW([], [])
    with pytest.raises(ValueError):
        sg.AdamW([p], [g], state_bits=16)
    with pytest.raises(ValueError):
        sg.AdamW([p], [g[:9]])
    with pytest.raises(ValueError):
        sg.AdamW([p], [g, g])
    with pytest.raises(ValueError):
        sg.AdamW([p], [g.cpu()])
    with pytest.raises(TypeError):
        sg.AdamW([p], [g.double()])
    with pytest.raises(ValueError):
        sg.AdamW([p.view(2, 5).t()], [g])
    with pytest.raises(ValueError):
        f8 = torch.zeros(10, device="cuda", dtype=torch.uint8).view(torch.float8_e4m3fn)
        sg.AdamW([p], [g], [f8], [f8])
    with pytest.raises(sg.SgemmError):
        sg.AdamW([p], [g]).step(step=0)


@gpu
def test_refused_gradients_leave_the_handle_as_it_was(device):
    def made():
        return make([700, 33, 4096], "fp32", "fp32", 32, seed=21)

    s, clean = made(), made()
    opt, want = (sg.AdamW(t["p"], t["g"], t["m"], t["v"], **HYPER) for t in (s, clean))
    before = [bytes(e) for e in opt._table]
    others = [torch.full_like(g, 3.0) for g in s["g"]]
    for bad in (others[:2] + [others[2][:-1]], others[:2] + [others[2].cpu()], others[:2] + [others[2].bfloat16()],
                [g.bfloat16() for g in others[:2]] + [others[2]], others[:2]):
        with pytest.raises((TypeError, ValueError)):
            opt.set_grads(bad)
        assert [bytes(e) for e in opt._table] == before
        assert all(a is b for a, b in zip(opt.grads, s["g"]))
    for o in (opt, want):
        o.step(step=5)
    for k in ("p", "m", "v"):
        assert all(torch.equal(a, b) for a, b in zip(s[k], clean[k]))


@gpu
def test_states_do_not_go_by_the_default_type(device):
    p, g = torch.ones(300, device="cuda"), torch.ones(300, device="cuda")
    torch.set_default_dtype(torch.float64)
    try:
        opt = sg.AdamW([p], [g], state_bits=8, lr=0.5, weight_decay=0.0)
    finally:
        torch.set_default_dtype(torch.float32)
    opt.step()
    assert opt.m_scales[0].dtype == torch.float32 and bool(((p - 0.5).abs() < 1e-6).all())
