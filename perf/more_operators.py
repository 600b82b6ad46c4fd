"""Measured cases of the operators around the feed-forward block: the
root-mean-square norm before it (with the residual's addition, in a training
step, and with an output of 8 bits), the gate with an output of 8 bits, and
products of 8-bit integers with a scale for each token and channel.

Each case runs either in plain form (elementary torch operations in 32 bits,
rounded once at the end; the 8-bit codes in 64 bits, as a value next to a border
between two codes needs) or, with ``own`` set, through this package's calls.
"""
import math

import torch

own = False

torch.backends.cuda.matmul.allow_tf32 = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
ACTIVATIONS = ("silu", "gelu", "relu")
EPS = 1e-6
TINY = 2.0 ** -96  # a row's largest magnitude counts as at least this


def listed():
    return [
        # One token of one sequence before a large block: latency alone.
        {"name": "norm 1x4096 bf16", "op": "norm", "T": 1, "D": 4096, "dtype": "bf16",
         "weight": "bf16", "residual": True, "pad": 0},
        # A long prompt whose rows start nowhere near a vector: bandwidth.
        {"name": "norm 8192x8191 fp16 odd", "op": "norm", "T": 8192, "D": 8191, "dtype": "fp16",
         "weight": "fp16", "residual": False, "pad": 0},
        # A training step's share of one norm, weights kept in FP32: forward and
        # backward with the residual stream's own gradient.
        {"name": "norm train 8192x2048 bf16", "op": "train", "T": 8192, "D": 2048, "dtype": "bf16",
         "weight": "fp32", "residual": True, "pad": 0},
        # The same in FP32, odd sizes in a wider buffer, without a residual.
        {"name": "norm train 1023x1025 fp32 odd", "op": "train", "T": 1023, "D": 1025,
         "dtype": "fp32", "weight": "fp32", "residual": False, "pad": 3},
        # The norm before an 8-bit product, of a long prompt.
        {"name": "norm8 4096x4096 bf16", "op": "norm8", "T": 4096, "D": 4096, "dtype": "bf16",
         "weight": "bf16", "residual": True, "pad": 0},
        # The same for a few sequences of an FP32 model of odd width.
        {"name": "norm8 5x2047 fp32 odd", "op": "norm8", "T": 5, "D": 2047, "dtype": "fp32",
         "weight": "fp32", "residual": True, "pad": 0},
        # The gate between two 8-bit products: a short ragged prompt.
        {"name": "gate8 333x5336 fp16", "op": "gate8", "T": 333, "F": 5336, "dtype": "fp16",
         "act": "gelu", "joined": False},
        # The same of a long prompt; gate and up are halves of one product.
        {"name": "gate8 4096x12288 bf16", "op": "gate8", "T": 4096, "F": 12288, "dtype": "bf16",
         "act": "silu", "joined": True},
        # One token against a large matrix: bandwidth of 8-bit weights.
        {"name": "q8 1x4096x12288 bf16", "op": "q8", "M": 1, "K": 4096, "N": 12288, "dtype": "bf16"},
        # A batch of sequences, one token each, against the down matrix.
        {"name": "q8 64x12288x4096 bf16", "op": "q8", "M": 64, "K": 12288, "N": 4096,
         "dtype": "bf16"},
        # A short prompt, every size odd, results in FP32.
        {"name": "q8 333x2047x5461 fp32 odd", "op": "q8", "M": 333, "K": 2047, "N": 5461,
         "dtype": "fp32"},
        # A long prompt: bound by the tensor cores.
        {"name": "q8 4096x4096x12288 bf16", "op": "q8", "M": 4096, "K": 4096, "N": 12288,
         "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "train", "norm8", "gate8", "q8", "q8", "q8"))
    step = rng.choice((1, 8, 64))
    round_up = lambda v: -(-v // step) * step  # noqa: E731
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "q8":
        c = {"op": op, "M": _log(rng, 1, 8192), "K": round_up(_log(rng, 256, 16384)),
             "N": round_up(_log(rng, 256, 24576)), "dtype": dtype}
        while c["M"] * c["K"] * c["N"] > 4096 * 4096 * 12288:
            c["M"] //= 2
        return c
    if op == "gate8":
        c = {"op": op, "T": _log(rng, 1, 8192), "F": round_up(_log(rng, 256, 16384)),
             "dtype": dtype, "act": rng.choice(ACTIVATIONS), "joined": rng.random() < 0.5}
        while c["T"] * c["F"] * (2 * SIZE[dtype] + 1) > 4096 * 12288 * 5:
            c["T"] //= 2
        return c
    c = {"op": op, "T": _log(rng, 64 if op == "train" else 1, 16384),
         "D": round_up(_log(rng, 128, 16384)), "dtype": dtype,
         "weight": rng.choice((dtype, "fp32")), "residual": rng.random() < 0.6,
         "pad": rng.choice((0, 0, 8, 3))}
    while c["T"] * c["D"] * SIZE[dtype] > {"norm": 8192 * 8192, "train": 8192 * 4096,
                                           "norm8": 8192 * 4096}[op]:
        c["T"] //= 2
    return c


def work(case):
    """Bytes: each input once, each output once.  Flops: the products' and, where
    they count, the elementwise operations'."""
    e = SIZE[case["dtype"]]
    if case["op"] == "q8":
        M, K, N = case["M"], case["K"], case["N"]
        return {"bytes": N * K + M * K + 4 * (M + N) + e * M * N, "flops": 2 * M * N * K}
    if case["op"] == "gate8":
        return {"bytes": case["T"] * (case["F"] * (2 * e + 1) + 4), "flops": 10 * case["T"] * case["F"]}
    T, D, w, res = case["T"], case["D"], SIZE[case["weight"]], case["residual"]
    if case["op"] == "train":  # x (residual), dy (dh), y (h), dx; weight and its gradient
        return {"bytes": e * T * D * (7 if res else 4) + 2 * w * D, "flops": 13 * T * D}
    if case["op"] == "norm8":
        return {"bytes": T * D * (e * (3 if res else 1) + 1) + 4 * T + w * D, "flops": 6 * T * D}
    return {"bytes": e * T * D * (4 if res else 2) + w * D, "flops": 4 * T * D}


# ---- inputs -------------------------------------------------------------------

def _rows(shape, pad, dtype, gen, scale=1.0):
    """A normal matrix whose rows lie `pad` elements apart in a wider buffer."""
    wide = torch.randn(shape[0], shape[1] + pad, generator=gen, device="cuda") * scale
    return wide.to(dtype)[:, :shape[1]]


def _norm_inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, D, pad, dtype = case["T"], case["D"], case["pad"], DTYPES[case["dtype"]]
    # A residual stream: tokens of different sizes, a few channels far above the others.
    size = torch.exp(0.5 * torch.randn(T, 1, generator=gen, device="cuda"))
    channel = torch.exp(2 * (torch.rand(D, generator=gen, device="cuda") > 0.99))
    s = {}
    for name in ("x", "residual") if case["residual"] else ("x",):
        wide = _rows((T, D), pad, torch.float32, gen)
        s[name] = torch.empty(T, D + pad, device="cuda", dtype=dtype)[:, :D].copy_(
            wide * size * channel)
    s["weight"] = (1 + 0.2 * torch.randn(D, generator=gen, device="cuda")).to(DTYPES[case["weight"]])
    if case["op"] == "train":
        s["dy"] = _rows((T, D), pad, dtype, gen)
        if case["residual"]:
            s["dh"] = _rows((T, D), pad, dtype, gen)
    return s


def _gate_inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, F, dtype = case["T"], case["F"], DTYPES[case["dtype"]]
    if case["joined"]:
        both = _rows((T, 2 * F), 0, dtype, gen, 1.5)
        return {"g": both[:, :F], "u": both[:, F:]}
    return {"g": _rows((T, F), 0, dtype, gen, 1.5), "u": _rows((T, F), 0, dtype, gen, 1.5)}


def _q8_inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    M, K, N = case["M"], case["K"], case["N"]

    def codes(rows):
        # A row of normal values whose largest, some 3.5 to 4.5 deviations out, is 127.
        t = torch.randn(rows, K, generator=gen, device="cuda")
        t *= 127 / t.abs().amax(dim=1, keepdim=True)
        return t.round_().to(torch.int8)

    return {"x": codes(M), "x_scales": torch.rand(M, generator=gen, device="cuda") * 0.05 + 0.005,
            "w": codes(N), "w_scales": (torch.rand(N, generator=gen, device="cuda") + 0.5) *
            (K ** -0.5 / 32)}


def prepare(case, seed):
    if case["op"] == "q8":
        s = _q8_inputs(case, seed)
        s["y"] = torch.empty(case["M"], case["N"], device="cuda", dtype=DTYPES[case["dtype"]])
        if own:
            import dense_fp32_sgemm_gb300 as sg
            s["matrix"] = sg.Q8Matrix(s["w"], s["w_scales"], dtype=DTYPES[case["dtype"]])
    elif case["op"] == "gate8":
        s = _gate_inputs(case, seed)
    else:
        s = _norm_inputs(case, seed)
    s["case"] = case
    return s


# ---- plain forms --------------------------------------------------------------

def _codes(a):
    """The 8-bit codes of rows `a` in 64 bits, and the rows' largest magnitudes."""
    top = a.abs().amax(dim=1, keepdim=True).clamp(min=TINY)
    return torch.round(a * 127 / top).to(torch.int8), top


def _norm_plain(s, case):
    x, w = s["x"], s["weight"]
    out = {}
    h = x.float()
    if case["residual"]:
        h = h + s["residual"].float()
        out["h"] = h.to(x.dtype)
    rstd = 1 / torch.sqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    if case["op"] == "norm8":
        wide = x.double() + s["residual"].double() if case["residual"] else x.double()
        out["q"], top = _codes(wide * w.double())
        out["scales"] = (top.float() * rstd / 127).view(-1)
        return out
    out["y"] = (h * rstd * w.float()).to(x.dtype)
    if case["op"] == "train":
        dy = s["dy"].float()
        unit = h * rstd
        out["dweight"] = (dy * unit).sum(dim=0).to(w.dtype)
        dn = dy * w.float()
        dx = rstd * (dn - unit * (dn * unit).mean(dim=1, keepdim=True))
        out["dx"] = (dx + s["dh"].float() if case["residual"] else dx).to(x.dtype)
    return out


def _gate_plain(s, case):
    g, u = s["g"].double(), s["u"].double()
    if case["act"] == "silu":
        a = g / (1 + torch.exp(-g))
    elif case["act"] == "gelu":
        z = math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)
        a = g / (1 + torch.exp(-2 * z))  # = g/2 (1 + tanh z)
    else:
        a = torch.where(g > 0, g, 0.0)
    v = a * u
    q, top = _codes(v)
    if case["act"] != "relu":
        # An element whose gate is that of the row's largest may lie exactly between two
        # codes (127 times the quotient of two u); the gate's rounding must not decide.
        at = v.abs().argmax(dim=1, keepdim=True)
        t = (u * 127 / u.gather(1, at).abs()) * (a / a.gather(1, at).abs())
        q = torch.where(top > TINY, torch.round(t).to(torch.int8), q)
    return {"q": q, "scales": (top / 127).float().view(-1)}


def _q8_plain(s, case):
    y = s["x"].float() @ s["w"].float().t()
    return {"y": (y * s["x_scales"][:, None] * s["w_scales"]).to(DTYPES[case["dtype"]])}


# ---- one pass -----------------------------------------------------------------

def _own(s, case):
    import dense_fp32_sgemm_gb300 as sg
    if case["op"] == "q8":
        return {"y": s["matrix"].matmul(s["x"], s["x_scales"], s["y"])}
    if case["op"] == "gate8":
        act = {"silu": sg.GATE_SILU, "gelu": sg.GATE_GELU, "relu": sg.GATE_RELU}[case["act"]]
        q, scales = sg.gate_q8(s["g"], s["u"], activation=act)
        return {"q": q, "scales": scales}
    residual = s["residual"] if case["residual"] else None
    if case["op"] == "norm8":
        got = sg.rms_norm_q8(s["x"], s["weight"], residual=residual, eps=EPS)
        return dict(zip(("q", "scales", "h"), got))
    got = sg.rms_norm(s["x"], s["weight"], residual=residual, eps=EPS)
    out = dict(zip(("y", "h"), got)) if case["residual"] else {"y": got}
    if case["op"] == "train":
        out["dx"], out["dweight"] = sg.rms_norm_backward(
            s["dy"], s["x"], s["weight"], residual=residual,
            dh=s["dh"] if case["residual"] else None, eps=EPS)
    return out


def run(s):
    case = s["case"]
    if own:
        return _own(s, case)
    return {"q8": _q8_plain, "gate8": _gate_plain}.get(case["op"], _norm_plain)(s, case)


# ---- the definition in 64 bits --------------------------------------------------

def _exact_codes(a):
    top = a.abs().max(dim=1).values.clamp(min=TINY)
    return (127 * a / top[:, None]).round().to(torch.int8), top / 127


def _exact_norm(case, seed):
    s = {k: v.double() for k, v in _norm_inputs(case, seed).items()}
    out = {}
    x = s["x"] + s["residual"] if case["residual"] else s["x"]
    if case["residual"]:
        out["h"] = x
    leaves = [x.requires_grad_(), s["weight"].requires_grad_()]
    norm = torch.linalg.vector_norm(x, dim=1, keepdim=True)
    unit = x / (norm ** 2 / case["D"] + EPS) ** 0.5
    if case["op"] == "norm8":
        out["q"], scales = _exact_codes((x * s["weight"]).detach())
        length = (x.detach() ** 2).sum(1) / case["D"] + EPS
        out["scales"] = scales / length ** 0.5
        return out
    y = unit * s["weight"]
    if case["op"] == "train":
        dx, out["dweight"] = torch.autograd.grad(y, leaves, s["dy"])
        out["dx"] = dx + s["dh"] if case["residual"] else dx
    if case["residual"]:
        out["h"] = x.detach()
    out["y"] = y.detach()
    return out


def _exact_gate(case, seed):
    s = _gate_inputs(case, seed)
    g, u = s["g"].double(), s["u"].double()
    if case["act"] == "silu":
        a = g * torch.sigmoid(g)
    elif case["act"] == "gelu":
        a = g * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3))
    else:
        a = g.clamp(min=0)
    q, scales = _exact_codes(a * u)
    if case["act"] != "relu":  # (ties exactly: a factor that both have is not rounded twice)
        best = (a * u).abs().max(dim=1, keepdim=True).indices
        ratio = (127 * u / u.gather(1, best).abs()) * (a / a.gather(1, best).abs())
        q = torch.where((scales * 127 > TINY)[:, None], ratio.round().to(torch.int8), q)
    return {"q": q, "scales": scales}


def _exact_q8(case, seed):
    s = _q8_inputs(case, seed)
    sums = torch.mm(s["x"].double(), s["w"].double().T)  # whole numbers below 2^53
    return {"y": sums * torch.outer(s["x_scales"].double(), s["w_scales"].double())}


def exact(case, seed):
    return {"q8": _exact_q8, "gate8": _exact_gate}.get(case["op"], _exact_norm)(case, seed)
