"""The gated feed-forward block: forward and backward pass against the formula
in 64 bits, element by element within a bound built from the roundings the
operator makes, at sizes around its tiles and with rows that lie apart; its
refusals; and the report of a wait that runs out.

The bound.  u is the type's unit roundoff.  A sum of K products carries at most
c(K) = (32 + K) 2^-23 of the sum of their magnitudes: each of K additions, and
each of the roundings of a 64-deep block of split FP32 products, loses at most
2^-23.  The activation loses at most 2^-20 of its value.  h, dg and du are
rounded to the type.  Everything else follows by propagation (below), with the
activations' slopes at most 1.13 and their second derivatives at most 1.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import dense_fp32_sgemm_gb300 as sg

TYPES = {"fp32": (torch.float32, 2.0 ** -24), "fp16": (torch.float16, 2.0 ** -11),
         "bf16": (torch.bfloat16, 2.0 ** -8)}
TINY = {"fp32": 0.0, "fp16": 2.0 ** -24, "bf16": 0.0}  # half the least subnormal, and room
ACTS = {"silu": 0, "gelu": 1, "relu": 2}
EPS_ACT, SLOPE, BEND = 2.0 ** -20, 1.13, 1.0


def c(K):
    return (32 + K) * 2.0 ** -23


def act64(g, act):
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        k = (2 / np.pi) ** 0.5
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k * (1 + 3 * 0.044715 * g * g)
    return g.clamp(min=0), (g > 0).double()


def formula(x, wg, wu, wd, act, dy=None):
    """Values and bounds of the outputs, in 64 bits, for one type's roundoff u."""
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    g, u = x @ wg, x @ wu
    a, s = act64(g, act)
    h = a * u
    out = {"y": h @ wd}
    if dy is not None:
        dy = dy.double()
        dh = dy @ wd.T
        dg, du = dh * u * s, dh * a
        out.update(dx=dg @ wg.T + du @ wu.T, dwg=x.T @ dg, dwu=x.T @ du, dwd=h.T @ dy)
    return out


def bounds(x, wg, wu, wd, act, unit, tiny, dy=None):
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    T, D = x.shape
    F = wg.shape[1]
    g, u = x @ wg, x @ wu
    a, s = act64(g, act)
    h = a * u
    ax, ag, au, ad = x.abs(), wg.abs(), wu.abs(), wd.abs()
    eg, eu = c(D) * (ax @ ag), c(D) * (ax @ au)
    ea = SLOPE * eg + EPS_ACT * a.abs()
    eh = ea * (u.abs() + eu) + a.abs() * eu
    eh = eh + unit * (h.abs() + eh) + tiny
    out = {"y": (eh @ ad + c(F) * ((h.abs() + eh) @ ad)) + 0 * (h @ wd)}
    if dy is not None:
        dy = dy.double()
        ay = dy.abs()
        dh = dy @ wd.T
        edh = c(D) * (ay @ ad.T)
        # ReLU's slope jumps where g may have either sign.
        es = (g.abs() <= eg).double() if act == "relu" else BEND * eg + 4 * EPS_ACT
        dg, du = dh * u * s, dh * a
        edg = (dh.abs() + edh) * (u.abs() + eu) * (s.abs() + es) - dg.abs()
        edu = (dh.abs() + edh) * (a.abs() + ea) - du.abs()
        edg, edu = (e + unit * (v.abs() + e) + tiny + 2.0 ** -21 * v.abs()
                    for e, v in ((edg, dg), (edu, du)))
        out["dx"] = edg @ ag.T + edu @ au.T + c(2 * F) * ((dg.abs() + edg) @ ag.T + (du.abs() + edu) @ au.T)
        out["dwg"] = ax.T @ edg + c(T) * (ax.T @ (dg.abs() + edg))
        out["dwu"] = ax.T @ edu + c(T) * (ax.T @ (du.abs() + edu))
        out["dwd"] = eh.T @ ay + c(T) * ((h.abs() + eh).T @ ay)
    return out


def rows(gen, n, m, dtype, pad=0, offset=0, scale=1.0):
    """n x m normal values whose rows lie m + pad elements apart, `offset`
    elements into a buffer that is NaN everywhere else."""
    flat = torch.full((n * (m + pad) + offset + 8,), float("nan"), device="cuda", dtype=dtype)
    view = flat[offset:offset + n * (m + pad)].view(n, m + pad)[:, :m]
    view.copy_(torch.randn(n, m, generator=gen, device="cuda") * scale)
    return view


def make(T, D, F, kind, pad=0, offset=0, seed=3):
    gen = torch.Generator("cuda").manual_seed(seed)
    dtype = TYPES[kind][0]
    r = lambda n, m, s: rows(gen, n, m, dtype, pad, offset, s)  # noqa: E731
    return dict(x=r(T, D, 1.0), wg=r(D, F, D ** -0.5), wu=r(D, F, D ** -0.5), wd=r(F, D, F ** -0.5),
                dy=r(T, D, 1.0))


def assert_close(got, want, slack, unit, tiny, what):
    err = (got.double() - want).abs()
    limit = slack + unit * (want.abs() + slack) + tiny
    assert torch.isfinite(got).all(), what
    bad = err > limit
    assert not bad.any(), f"{what}: {int(bad.sum())} beyond the bound, worst {float((err / limit).max()):.3g}"


def check(m, kind, act, saved=None, need=True):
    unit, tiny = TYPES[kind][1], TINY[kind]
    w = (m["wg"], m["wu"], m["wd"])
    if saved == "kept":
        T, F = m["x"].shape[0], m["wg"].shape[1]
        saved = sg.ffn_saved(T, F, dtype=m["x"].dtype)
        saved.fill_(float("nan"))
    y = sg.ffn_forward(m["x"], *w, activation=ACTS[act], saved=saved)
    want = formula(m["x"], *w, act, m["dy"] if need else None)
    slack = bounds(m["x"], *w, act, unit, tiny, m["dy"] if need else None)
    assert_close(y, want["y"], slack["y"], unit, tiny, "y")
    if need:
        got = dict(zip(("dx", "dwg", "dwu", "dwd"),
                       sg.ffn_backward(m["dy"], m["x"], *w, activation=ACTS[act], saved=saved)))
        for k, v in got.items():
            assert_close(v, want[k], slack[k], unit, tiny, k)
    assert sg.device_status(torch.cuda.current_stream()) == 0


gpu = pytest.mark.gpu


@pytest.fixture(scope="module")
def device():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    sg.build()
    torch.backends.cuda.matmul.allow_tf32 = False
    return torch.device("cuda", 0)


# Forward pass: one row to several tiles; sizes one off the tiles' 64, 128 and 256
# and off every vector; few-row and tensor-core forms.
@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,D,F", [(1, 1, 1), (1, 64, 96), (2, 129, 257), (3, 200, 72), (4, 33, 500),
                                   (5, 256, 384), (8, 65, 129), (9, 40, 24), (127, 63, 65),
                                   (128, 128, 128), (129, 96, 200), (256, 64, 256), (257, 257, 129),
                                   (300, 520, 264), (513, 72, 1000)])
def test_forward(device, T, D, F, kind):
    check(make(T, D, F, kind), kind, "silu", need=False)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("T", [2, 100])
def test_activations(device, T, act, kind):
    m = make(T, 96, 136, kind)
    m["x"][0] *= 30  # saturated gates, both signs
    check(m, kind, act)


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("saved", [None, "kept"])
@pytest.mark.parametrize("T,D,F", [(1, 1, 1), (1, 72, 40), (7, 130, 66), (64, 64, 64), (129, 127, 193),
                                   (256, 256, 384), (300, 96, 1032), (515, 261, 131)])
def test_training_step(device, T, D, F, saved, kind):
    check(make(T, D, F, kind), kind, "silu", saved)


# Rows that lie apart, bases off 16 bytes, and gate and up as halves of one matrix.
@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (8, 1), (5, 3)])
def test_strides_and_alignment(device, T, pad, offset, kind):
    check(make(T, 72, 104, kind, pad, offset), kind, "gelu", "kept" if T > 8 else None)
    m = make(T, 64, 48, kind)
    both = torch.cat([m["wg"], m["wu"]], dim=1)
    m["wg"], m["wu"] = both[:, :48], both[:, 48:]
    check(m, kind, "silu")


@gpu
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_deep_sums_are_cut_and_joined(device, kind):
    # Few tiles, long sums: K is shared out over the SMs.
    check(make(130, 72, 6000, kind), kind, "silu", need=False)
    check(make(3000, 96, 72, kind), kind, "silu", "kept")


@gpu
def test_norm_of_fp32_error(device):
    # A block's sums lose some 24 truncations of 2^-24 of their size, two products
    # one after the other: 2^-18 of the outputs' norm with room to spare.
    m = make(300, 640, 1100, "fp32")
    w = (m["wg"], m["wu"], m["wd"])
    want = formula(m["x"], *w, "silu", m["dy"])
    got = {"y": sg.ffn_forward(m["x"], *w)}
    got.update(zip(("dx", "dwg", "dwu", "dwd"), sg.ffn_backward(m["dy"], m["x"], *w)))
    for k, v in got.items():
        assert float((v.double() - want[k]).norm() / want[k].norm()) < 2.0 ** -18, k


@gpu
def test_gradient_against_differences(device):
    # f(w) = <dy, ffn(w)>: the derivative along a direction d against a central
    # difference of the formula in 64 bits (step 1e-4: its own error is below
    # 1e-6 of the sums here); FP32 gradients lose less than 1e-5.
    gen = torch.Generator("cuda").manual_seed(5)
    m = make(20, 24, 40, "fp32")
    dx, dwg, dwu, dwd = sg.ffn_backward(m["dy"], m["x"], m["wg"], m["wu"], m["wd"],
                                        activation=ACTS["gelu"])
    base = {k: m[k].double() for k in ("x", "wg", "wu", "wd")}
    for name, grad in (("x", dx), ("wg", dwg), ("wu", dwu), ("wd", dwd)):
        d = torch.randn(base[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        f = []
        for sign in (1, -1):
            at = dict(base)
            at[name] = base[name] + sign * 1e-4 * d
            f.append((formula(at["x"], at["wg"], at["wu"], at["wd"], "gelu")["y"] * m["dy"].double()).sum())
        slope = float((f[0] - f[1]) / 2e-4)
        mine = float((grad.double() * d).sum())
        size = float((grad.double() * d).abs().sum())
        assert abs(mine - slope) <= 1e-5 * size, name


@gpu
def test_parts_of_the_gradient(device):
    m = make(90, 64, 80, "bf16")
    args = (m["dy"], m["x"], m["wg"], m["wu"], m["wd"])
    dx, dwg, dwu, dwd = sg.ffn_backward(*args)
    only_dx = sg.ffn_backward(*args, need_dw=False)
    only_dw = sg.ffn_backward(*args, need_dx=False)
    assert torch.equal(only_dx[0], dx) and only_dx[1:] == (None, None, None)
    assert only_dw[0] is None and all(torch.equal(a, b) for a, b in zip(only_dw[1:], (dwg, dwu, dwd)))


@gpu
def test_outputs_in_place_and_nothing_else_written(device):
    m = make(70, 40, 56, "bf16")
    wide = torch.full((72, 48), 7.0, device="cuda", dtype=torch.bfloat16)
    y = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"], y=wide[1:71, 3:43])
    assert torch.equal(y, sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"]))
    wide[1:71, 3:43] = 7.0
    assert bool((wide == 7.0).all())


@gpu
@pytest.mark.parametrize("T", [3, 200])
def test_same_bits_every_time_and_on_any_stream(device, T):
    m = make(T, 96, 3000, "bf16")
    first = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        y = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"], stream=side)
        side.synchronize()
        assert torch.equal(y, first)
    with torch.cuda.stream(side):
        y = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"])
    side.synchronize()
    assert torch.equal(y, first)


@gpu
def test_nothing_to_do(device):
    for T, D, F in ((0, 8, 16), (5, 0, 16), (5, 8, 0), (200, 8, 0)):
        x, dy = torch.ones(T, D, device="cuda"), torch.ones(T, D, device="cuda")
        wg, wd = torch.ones(D, F, device="cuda"), torch.ones(F, D, device="cuda")
        y = sg.ffn_forward(x, wg, wg, wd)
        assert y.shape == (T, D) and bool((y == 0).all())
        for g in sg.ffn_backward(dy, x, wg, wg, wd):
            assert bool((g == 0).all())


@gpu
def test_infinities_and_nan_stay_in_their_rows(device):
    for T in (4, 40):
        m = make(T, 64, 72, "bf16")
        clean = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"])
        m["x"][1, 5], m["x"][2, 7] = float("nan"), float("inf")
        y = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"])
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[2]).any()
        keep = [i for i in range(T) if i not in (1, 2)]
        assert torch.equal(y[keep], clean[keep])


@gpu
@pytest.mark.parametrize("kind", ["fp32", "bf16"])
@pytest.mark.parametrize("act", ACTS)
def test_slopes_of_huge_gates(device, act, kind):
    # Gates of 10^20, whose square is beyond FP32: slope 0 or 1, and finite gradients.
    T, dtype = 30, TYPES[kind][0]
    m = make(T, 1, 6, kind)
    m["x"].fill_(1)
    m["dy"].fill_(1)
    m["wg"][0] = torch.tensor([1e20, -1e20, 1e10, -1e10, 70.0, -70.0], device="cuda", dtype=dtype)
    m["wu"].fill_(1)
    m["wd"][:, 0] = torch.tensor([1e-20, 1e-20, 1e-10, 1e-10, 1.0, 1.0], device="cuda", dtype=dtype)
    check(m, kind, act, "kept")


@gpu
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("T,saved", [(4, None), (4, "kept"), (40, None), (140, "kept")])
def test_infinities_and_nan_in_every_form(device, T, saved, kind):
    # Where the formula has no finite value there is none (an infinity may come out as
    # NaN), and everything else keeps its bits: x in rows, weights and dy by what they
    # enter.
    act = "silu"
    m = make(T, 64, 72, kind)
    keep = sg.ffn_saved(T, 72, dtype=m["x"].dtype) if saved else None

    def run(m):
        w = (m["wg"], m["wu"], m["wd"])
        y = sg.ffn_forward(m["x"], *w, activation=ACTS[act], saved=keep)
        return dict(zip(("y", "dx", "dwg", "dwu", "dwd"),
                        (y, *sg.ffn_backward(m["dy"], m["x"], *w, activation=ACTS[act], saved=keep))))

    clean = run(m)
    for name, at in (("x", (1, 5)), ("wd", (7, 3)), ("dy", (2, 9))):
        for value in (float("nan"), float("inf"), -float("inf")):
            bad = {k: v.clone() for k, v in m.items()}
            bad[name][at] = value
            want = formula(bad["x"], bad["wg"], bad["wu"], bad["wd"], act, bad["dy"])
            for k, v in run(bad).items():
                fine = torch.isfinite(want[k])
                assert torch.equal(torch.isfinite(v), fine), (name, value, k)
                untouched = fine & (want[k] == formula(m["x"], m["wg"], m["wu"], m["wd"], act, m["dy"])[k])
                assert torch.equal(v[untouched], clean[k][untouched]), (name, value, k)
    assert sg.device_status(torch.cuda.current_stream()) == 0


@gpu
def test_the_range_of_fp16_between_the_products(device):
    # h of some 10^5 in row 1 (times weights of 10^-3): a number in the form for few
    # rows, infinite where it is held in FP16; no other row minds.
    for T, saved in ((8, None), (9, None), (3, "kept")):
        m = make(T, 64, 96, "fp16")
        m["wd"] *= 2.0 ** -10
        m["x"][1] *= 500
        w = (m["wg"], m["wu"], m["wd"])
        want = formula(m["x"], *w, "relu")["y"]
        assert float((formula(m["x"], m["wg"], m["wu"], torch.eye(96, device="cuda"), "relu")["y"][1]).max()) > 7e4
        slack = bounds(m["x"], *w, "relu", TYPES["fp16"][1], TINY["fp16"])["y"]
        keep = sg.ffn_saved(T, 96, dtype=torch.float16) if saved else None
        y = sg.ffn_forward(m["x"], *w, activation=ACTS["relu"], saved=keep)
        rows = [t for t in range(T) if t != 1 or (T <= 8 and not saved)]
        assert_close(y[rows], want[rows], slack[rows], TYPES["fp16"][1], TINY["fp16"], f"{T} rows")
        if 1 not in rows:
            assert not torch.isfinite(y[1]).any()


@gpu
def test_small_fp16_gradients_by_scaling(device):
    # dy of 10^-6, whose products are FP16 subnormals: scaled by 2^14 and back, all
    # gradients have h, dg, du and their own rounding: 3 roundings of 2^-11 at most.
    m = make(300, 96, 160, "fp16")
    w = (m["wg"], m["wu"], m["wd"])
    dy = (m["dy"].double() * 1e-6 * 2.0 ** 14).half()
    want = formula(m["x"], *w, "silu", dy.double() * 2.0 ** -14)
    got = sg.ffn_backward(dy, m["x"], *w)
    for k, v in zip(("dx", "dwg", "dwu", "dwd"), got):
        v = v.double() * 2.0 ** -14
        assert float((v - want[k]).norm()) <= 3 * 2.0 ** -11 * float(want[k].norm()), k


@gpu
def test_offsets_beyond_32_bits(device):
    # h and the kept values have 2^32 elements.
    T, D, F = 131072, 16, 32768
    m = make(T, D, F, "bf16")
    saved = sg.ffn_saved(T, F, dtype=torch.bfloat16)
    y = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"], saved=saved)
    dx = sg.ffn_backward(m["dy"], m["x"], m["wg"], m["wu"], m["wd"], saved=saved, need_dw=False)[0]
    del saved
    unit = TYPES["bf16"][1]
    for at in (0, T // 2 - 4, T - 8):
        part = {k: m[k][at:at + 8] for k in ("x", "dy")}
        w = (m["wg"], m["wu"], m["wd"])
        want = formula(part["x"], *w, "silu", part["dy"])
        slack = bounds(part["x"], *w, "silu", unit, 0.0, part["dy"])
        assert_close(y[at:at + 8], want["y"], slack["y"], unit, 0.0, f"y at {at}")
        assert_close(dx[at:at + 8], want["dx"], slack["dx"], unit, 0.0, f"dx at {at}")
    sg.release_workspace()


@gpu
@pytest.mark.parametrize("kind,offset", [("bf16", 0), ("bf16", 1), ("fp32", 0), ("fp32", 1)])
def test_rows_beyond_32_bits(device, kind, offset):
    # All matrices are columns of one buffer whose 300 rows lie 2^24 elements apart:
    # their last rows start behind 2^32 elements. Few rows, and the tensor cores.
    D, F, ld, dtype = 296, 288, 2 ** 24, TYPES[kind][0]
    wide = torch.zeros(300 * ld, device="cuda", dtype=dtype)[: 300 * ld].view(300, ld)
    for T in (3, 40):
        small = make(T, D, F, kind)
        m, at = {}, offset
        for k, v in small.items():
            m[k] = wide[300 - v.shape[0]:, at:at + v.shape[1]]
            m[k].copy_(v)
            at += 512
        assert m["wg"].storage_offset() + (D - 1) * ld > 2 ** 32
        check(m, kind, "silu", None if T == 3 else "kept", need=T > 3)


@gpu
def test_graph_capture(device):
    m = make(150, 64, 500, "bf16")
    side = torch.cuda.Stream()
    want = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"])
    y = torch.empty_like(want)
    with torch.cuda.stream(side):
        sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"], y=y)  # workspace first
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"], y=y)
    y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@gpu
@pytest.mark.parametrize("T", [100, 300])
def test_a_wait_that_runs_out_is_reported(device, T):
    m = make(T, 256, 512, "bf16")
    want = sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"])
    assert sg.device_status(torch.cuda.current_stream()) == 0
    sg.set_wait_timeout_ns(5_000_000, 2)
    try:
        sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"])
        assert sg.device_status(torch.cuda.current_stream()) == 5
    finally:
        sg.set_wait_timeout_ns(0, -1)
    assert torch.equal(sg.ffn_forward(m["x"], m["wg"], m["wu"], m["wd"]), want)
    assert sg.device_status(torch.cuda.current_stream()) == 0


# ---- refusals (no device needed) ------------------------------------------------

def forward_call(**over):
    a = dict(T=4, D=8, F=16, type=0, act=0, x=4096, ldx=8, wg=8192, ldg=16, wu=16384, ldu=16, wd=32768,
             ldd=8, y=65536, ldy=8, saved=None)
    a.update(over)
    sg.build()
    return sg.library().sgemm_ffn_forward(*(a[k] for k in (
        "T", "D", "F", "type", "act", "x", "ldx", "wg", "ldg", "wu", "ldu", "wd", "ldd", "y", "ldy",
        "saved")), None)


def backward_call(**over):
    a = dict(T=4, D=8, F=16, type=0, act=0, x=4096, ldx=8, wg=8192, ldg=16, wu=16384, ldu=16, wd=32768,
             ldd=8, dy=65536, lddy=8, saved=None, dx=131072, lddx=8, dwg=262144, lddg=16, dwu=524288,
             lddu=16, dwd=1048576, lddd=8)
    a.update(over)
    sg.build()
    return sg.library().sgemm_ffn_backward(*(a[k] for k in (
        "T", "D", "F", "type", "act", "x", "ldx", "wg", "ldg", "wu", "ldu", "wd", "ldd", "dy", "lddy",
        "saved", "dx", "lddx", "dwg", "lddg", "dwu", "lddu", "dwd", "lddd")), None)


BAD = [dict(T=-1), dict(D=-1), dict(F=-1), dict(type=3), dict(type=-1), dict(act=3), dict(act=-1),
       dict(x=None), dict(wg=None), dict(wu=None), dict(wd=None), dict(x=4098), dict(type=2, wg=8193),
       dict(ldx=7), dict(ldg=15), dict(ldu=15), dict(ldd=7), dict(saved=4100)]


@pytest.mark.parametrize("over", BAD + [dict(y=None), dict(y=65537), dict(ldy=7)])
def test_forward_refuses(over):
    assert forward_call(**over) == 1


@pytest.mark.parametrize("over", BAD + [dict(dy=None), dict(lddy=7), dict(lddx=7), dict(dx=131073),
                                        dict(dwg=None), dict(dwu=None), dict(dwd=None), dict(lddg=15),
                                        dict(lddu=15), dict(lddd=7), dict(dwd=1048577)])
def test_backward_refuses(over):
    assert backward_call(**over) == 1


def test_sizes_beyond_the_limit_are_unsupported():
    big = 2 ** 26 + 1
    assert forward_call(T=big) == 7
    assert forward_call(D=big, ldx=big, ldd=big, ldy=big) == 7


def test_saved_size():
    sg.build()
    f = sg.library().sgemm_ffn_saved_floats
    assert f(-1, 4, 0) == 0 and f(4, 4, 9) == 0 and f(0, 8, 0) == 0
    # two blocks of 32 x 32 floats, and h: one or three planes of 16 bits
    assert f(1, 1, 2) == 2048 + 4 and f(1, 1, 0) == 2048 + 12
    assert f(33, 40, 2) == 2 * 4 * 1024 + 33 * 40 // 2


def test_wrapper_refuses_what_is_not_a_cuda_matrix():
    sg.build()
    x, w = torch.ones(4, 8), torch.ones(8, 16)
    with pytest.raises(ValueError):
        sg.ffn_forward(x, w, w, w.t().contiguous())  # not on a GPU
    with pytest.raises(TypeError):
        sg.ffn_forward(x.double(), w.double(), w.double(), w.double())
    with pytest.raises(ValueError):
        sg.ffn_forward(x[0], w, w, w)


class OnDevice:
    """What the wrapper reads of a CUDA tensor, without one."""

    def __init__(self, t):
        self.dtype, self.shape, self.device = t.dtype, t.shape, torch.device("cuda", 0)
        self.dim, self.stride, self.data_ptr = t.dim, t.stride, lambda: 4096


def test_overlapping_rows_are_refused():
    # Rows with less than their length between them (a broadcast gradient's, say)
    # end outside the memory that the tensor has.
    from dense_fp32_sgemm_gb300.ffn import _matrix
    f32, dev = torch.float32, torch.device("cuda", 0)

    def ld(t):
        return _matrix(OnDevice(t), "dy", *t.shape, f32, dev)[1]

    one = torch.ones(1, 8)
    for t in (one.expand(4, 8), torch.ones(64).as_strided((4, 8), (7, 1)), torch.ones(1, 1).expand(3, 1)):
        with pytest.raises(ValueError, match="dy has overlapping rows"):
            ld(t)
    assert ld(one) == 8 and ld(torch.ones(4, 8)) == 8 and ld(torch.ones(4, 12)[:, :8]) == 12
    assert ld(one.expand(1, 8)) == 8 and ld(one[:, :0].expand(4, 0)) >= 1
    assert ld(torch.ones(64).as_strided((1, 8), (3, 1))) == 8  # one row: its stride means nothing


@gpu
def test_broadcast_tensors_are_refused(device):
    T, D, F = 6, 16, 24
    x, w, d = (torch.ones(s, device="cuda") for s in ((T, D), (D, F), (F, D)))
    for bad in ((x[:1].expand(T, D), w, w, d), (x, w[:1].expand(D, F), w, d), (x, w, w, d[:1].expand(F, D))):
        with pytest.raises(ValueError):
            sg.ffn_forward(*bad)
    with pytest.raises(ValueError):
        sg.ffn_forward(x, w, w, d, y=torch.empty(1, D, device="cuda").expand(T, D))
    for over in (dict(dy=x[:1].expand(T, D)), dict(dx=x[:1].expand(T, D)), dict(dw_gate=w[:1].expand(D, F)),
                 dict(dw_down=d[:1].expand(F, D))):
        dy = over.pop("dy", x)
        with pytest.raises(ValueError):
            sg.ffn_backward(dy, x, w, w, d, **over)


@gpu
def test_wrapper_refuses_wrong_shapes_and_types(device):
    x, w, d = (torch.ones(s, device="cuda") for s in ((4, 8), (8, 16), (16, 8)))
    for bad in ((x, w[:, :15], w, d), (x, w, w[:7], d), (x, w, w, w), (x[:, :7], w, w, d)):
        with pytest.raises(ValueError):
            sg.ffn_forward(*bad)
    with pytest.raises(TypeError):
        sg.ffn_forward(x, w, w.half(), d)
    with pytest.raises(ValueError):
        sg.ffn_forward(x, w, w, w.t())  # columns apart
    with pytest.raises(ValueError):
        sg.ffn_forward(x, w, w, d, saved=torch.ones(5, device="cuda"))
    with pytest.raises(sg.SgemmError):
        sg.ffn_forward(x, w, w, d, activation=7)
