"""Measured cases of the feed-forward operators: the gated block (forward, and
a training step), products with 4-bit weights, and the AdamW step.

Each case runs either in plain form (elementary torch operations in 32 bits,
rounded once at the end) or, with ``own`` set, through this package's calls.
"""
import math

import torch

own = False

torch.backends.cuda.matmul.allow_tf32 = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}
ACTIVATIONS = ("silu", "gelu", "relu")
BLOCK = 256  # values of one tensor that share a scale of the 8-bit states


def listed():
    return [
        # One token of one sequence through a large block: latency and the
        # bandwidth of three weight matrices; gate and up are halves of one matrix.
        {"name": "ffn decode 1 bf16", "op": "ffn", "T": 1, "D": 4096, "F": 12288, "dtype": "bf16",
         "act": "silu", "joined": True, "pad": 0},
        # A few sequences at once, weights kept in FP32, no size a multiple of
        # a vector and rows inside a wider buffer.
        {"name": "ffn decode 5 fp32 odd", "op": "ffn", "T": 5, "D": 2047, "F": 5461,
         "dtype": "fp32", "act": "gelu", "joined": False, "pad": 3},
        # A short prompt, ragged against every tile.
        {"name": "ffn prompt 333 fp16", "op": "ffn", "T": 333, "D": 2000, "F": 5336,
         "dtype": "fp16", "act": "gelu", "joined": False, "pad": 0},
        # A long prompt: bound by the tensor cores.
        {"name": "ffn prompt 4096 bf16", "op": "ffn", "T": 4096, "D": 4096, "F": 12288,
         "dtype": "bf16", "act": "silu", "joined": True, "pad": 0},
        # A training step's share of one block, activations saved.
        {"name": "ffn train 8192 bf16", "op": "train", "T": 8192, "D": 2048, "F": 8192,
         "dtype": "bf16", "act": "silu", "joined": False, "pad": 0, "saved": True},
        # The same in FP32 with odd sizes, activations computed again.
        {"name": "ffn train 1023 fp32 odd", "op": "train", "T": 1023, "D": 1025, "F": 2731,
         "dtype": "fp32", "act": "silu", "joined": False, "pad": 0, "saved": False},
        # One token against a large quantised matrix: bandwidth of 4-bit weights.
        {"name": "w4 1x4096x12288 bf16", "op": "w4", "M": 1, "K": 4096, "N": 12288, "group": 128,
         "zeros": False, "dtype": "bf16"},
        # The smallest product that a small model makes, odd in N: latency alone.
        {"name": "w4 1x1000x1025 fp16", "op": "w4", "M": 1, "K": 1000, "N": 1025, "group": 32,
         "zeros": True, "dtype": "fp16"},
        # A batch of sixteen sequences.
        {"name": "w4 16x12288x4096 bf16", "op": "w4", "M": 16, "K": 12288, "N": 4096, "group": 64,
         "zeros": True, "dtype": "bf16"},
        # FP32 activations, odd sizes on both sides.
        {"name": "w4 3x8191x8191 fp32", "op": "w4", "M": 3, "K": 8191, "N": 8191, "group": 128,
         "zeros": True, "dtype": "fp32"},
        # The step over a large model's matrices with 8-bit states.
        {"name": "adamw 8-bit large", "op": "adamw", "tensors": 24, "numel": 134000000, "bits": 8,
         "dtype": "bf16"},
        # The step over many small tensors with 32-bit states.
        {"name": "adamw 32-bit many", "op": "adamw", "tensors": 300, "numel": 3000001, "bits": 32,
         "dtype": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("ffn", "ffn", "train", "train", "w4", "w4", "adamw"))
    if op in ("ffn", "train"):
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        step = rng.choice((1, 8, 64))
        round_up = lambda v: -(-v // step) * step  # noqa: E731
        c = {"op": op, "T": _log(rng, 1 if op == "ffn" else 64, 8192),
             "D": round_up(_log(rng, 256, 4096)), "F": round_up(_log(rng, 512, 12288)),
             "dtype": dtype, "act": rng.choice(ACTIVATIONS),
             "joined": rng.random() < 0.5, "pad": rng.choice((0, 0, 8, 3))}
        if op == "train":
            c["saved"] = rng.random() < 0.5
        most = 1.2e12 if dtype != "fp32" else 3e11
        while work(c)["flops"] > most:
            c["T"] = max(1, c["T"] // 2)
            c["F"] = max(512, round_up(c["F"] * 3 // 4))
        return c
    if op == "w4":
        group = rng.choice((32, 64, 128))
        return {"op": op, "M": _log(rng, 1, 16), "K": _log(rng, 256, 16384),
                "N": _log(rng, 256, 24576), "group": group, "zeros": rng.random() < 0.5,
                "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
    tensors = _log(rng, 1, 400)
    return {"op": op, "tensors": tensors, "numel": max(300 * tensors, _log(rng, 100000, 120000000)),
            "bits": rng.choice((8, 32)), "dtype": rng.choice(("bf16", "fp16", "fp32"))}


def work(case):
    """Bytes: each input once, each output once.  Flops: the products' and, where
    they count (AdamW), the elementwise operations'."""
    e = SIZE[case["dtype"]]
    if case["op"] in ("ffn", "train"):
        T, D, F = case["T"], case["D"], case["F"]
        if case["op"] == "ffn":
            return {"bytes": e * (3 * D * F + 2 * T * D), "flops": 6 * T * D * F}
        return {"bytes": e * (6 * D * F + 4 * T * D), "flops": 18 * T * D * F}
    if case["op"] == "w4":
        M, K, N = case["M"], case["K"], case["N"]
        groups = -(-K // case["group"])
        return {"bytes": 4 * -(-K // 8) * N + groups * N * (e + (1 if case["zeros"] else 0)) +
                e * M * (K + N), "flops": 2 * M * N * K}
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    return {"bytes": case["numel"] * (8 + e + state), "flops": 15 * case["numel"]}


# ---- inputs -------------------------------------------------------------------

def _rows(shape, pad, dtype, gen, scale=1.0):
    """A normal matrix whose rows lie `pad` elements apart in a wider buffer."""
    wide = torch.randn(shape[0], shape[1] + pad, generator=gen, device="cuda") * scale
    return wide.to(dtype)[:, :shape[1]]


def _ffn_inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, D, F, dtype, pad = case["T"], case["D"], case["F"], DTYPES[case["dtype"]], case["pad"]
    s = {"x": _rows((T, D), pad, dtype, gen)}
    if case["joined"]:
        both = _rows((D, 2 * F), pad, dtype, gen, D ** -0.5)
        s["wg"], s["wu"] = both[:, :F], both[:, F:]
    else:
        s["wg"] = _rows((D, F), pad, dtype, gen, D ** -0.5)
        s["wu"] = _rows((D, F), pad, dtype, gen, D ** -0.5)
    s["wd"] = _rows((F, D), pad, dtype, gen, F ** -0.5)
    if case["op"] == "train":
        s["dy"] = _rows((T, D), pad, dtype, gen)
    return s


def _w4_inputs(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    M, K, N, dtype = case["M"], case["K"], case["N"], DTYPES[case["dtype"]]
    groups = -(-K // case["group"])
    words = torch.randint(-2 ** 31, 2 ** 31, (-(-K // 8), N), generator=gen, device="cuda",
                          dtype=torch.int64).to(torch.int32)
    scales = (torch.rand(groups, N, generator=gen, device="cuda") + 0.5) * (K ** -0.5 / 4)
    zeros = torch.randint(4, 12, (groups, N), generator=gen, device="cuda", dtype=torch.uint8)
    return {"x": torch.randn(M, K, generator=gen, device="cuda").to(dtype), "q": words,
            "scales": scales.to(dtype), "zeros": zeros if case["zeros"] else None,
            "y": torch.empty(M, N, device="cuda", dtype=dtype)}


def _sizes(case):
    """Element counts of the tensors: a few large, the rest smaller, odd ones among them."""
    n, total = case["tensors"], case["numel"]
    weights = [1.0 / (1 + i % 7) ** 2 for i in range(n)]
    scale = (total - n) / sum(weights)
    sizes = [1 + int(w * scale) for w in weights]
    sizes[0] += total - sum(sizes)
    return sizes


ADAMW = {"lr": 1e-3, "beta1": 0.9, "beta2": 0.95, "eps": 1e-8, "weight_decay": 0.1, "step": 1000}


def _adamw_inputs(case, seed):
    """Flat buffers, as a training program keeps them, and one view of each per
    tensor.  With 8-bit states the tensors start on whole blocks."""
    gen = torch.Generator("cuda").manual_seed(seed)
    sizes = _sizes(case)
    unit = BLOCK if case["bits"] == 8 else 1
    starts, end = [], 0
    for n in sizes:
        starts.append(end)
        end += -(-n // unit) * unit
    live = torch.ones(end, dtype=torch.bool, device="cuda")
    for n, at in zip(sizes, starts):
        live[at + n:at + -(-n // unit) * unit] = False
    live = live.float()
    normal = lambda: torch.randn(end, generator=gen, device="cuda") * live  # noqa: E731
    # Gradients of very different sizes next to each other, as in training.
    g = normal() * torch.exp(2 * normal()) * 1e-3
    m, v = 0.3 * g + 3e-4 * normal(), (normal() * 1e-3 + g) ** 2
    s = {"p": normal() * 0.02, "g": g.to(DTYPES[case["dtype"]]), "bits": case["bits"],
         "sizes": sizes, "starts": starts}
    if case["bits"] == 8:
        s["m"], s["ms"] = _encode_m(m)
        s["v"], s["vs"] = _encode_v(torch.sqrt(v))
    else:
        s["m"], s["v"], s["ms"], s["vs"] = m, v, None, None
    return s


def prepare(case, seed):
    if case["op"] == "w4":
        s = _w4_inputs(case, seed)
        if own:
            import dense_fp32_sgemm_gb300 as sg
            s["w"] = sg.W4Matrix(s["q"], s["scales"], case["K"], case["group"], zeros=s["zeros"])
    elif case["op"] == "adamw":
        s = _adamw_inputs(case, seed)
        cut = lambda t: [t[a:a + n] for a, n in zip(s["starts"], s["sizes"])]  # noqa: E731
        cut_scales = lambda t: None if t is None else [  # noqa: E731
            t[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(s["starts"], s["sizes"])]
        if own:
            import dense_fp32_sgemm_gb300 as sg
            s["opt"] = sg.AdamW(cut(s["p"]), cut(s["g"]), cut(s["m"]), cut(s["v"]),
                                m_scales=cut_scales(s["ms"]), v_scales=cut_scales(s["vs"]), lr=ADAMW["lr"],
                                betas=(ADAMW["beta1"], ADAMW["beta2"]), eps=ADAMW["eps"],
                                weight_decay=ADAMW["weight_decay"])
    else:
        s = _ffn_inputs(case, seed)
    s["case"] = case
    return s


# ---- plain forms --------------------------------------------------------------

def _act(g, act):
    """The activation and its derivative."""
    if act == "silu":
        s = 1 / (1 + torch.exp(-g))
        return g * s, s * (1 + g * (1 - s))
    if act == "gelu":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (g + 0.044715 * g * g * g))
        return 0.5 * g * (1 + t), \
            0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)
    on = (g > 0).to(g.dtype)
    return g * on, on


def _ffn_plain(s, case):
    dtype = s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
    g, u = x @ wg, x @ wu
    a, da = _act(g, case["act"])
    h = a * u
    out = {"y": (h @ wd).to(dtype)}
    if case["op"] == "train":
        dy = s["dy"].float()
        dh = dy @ wd.t()
        dg, du = dh * u * da, dh * a
        out["dx"] = (dg @ wg.t() + du @ wu.t()).to(dtype)
        out["dwg"], out["dwu"] = (x.t() @ dg).to(dtype), (x.t() @ du).to(dtype)
        out["dwd"] = (h.t() @ dy).to(dtype)
    return out


def _unpack(q, K):
    """[ceil(K/8), N] words of eight 4-bit values along K to [K, N] floats."""
    shift = torch.arange(0, 32, 4, device=q.device, dtype=torch.int32).view(1, 8, 1)
    return ((q.unsqueeze(1) >> shift) & 15).reshape(-1, q.shape[1])[:K].float()


def _w4_plain(s, case):
    K, G = case["K"], case["group"]
    group = torch.arange(K, device="cuda") // G
    zero = s["zeros"].float()[group] if case["zeros"] else 8.0
    w = s["scales"].float()[group] * (_unpack(s["q"], K) - zero)
    return (s["x"].float() @ w).to(s["x"].dtype)


# The 8-bit states: e4m3 codes, m in units of the block's largest |m| / 448 and
# sqrt(v) in units of the block's largest sqrt(v) / 448.  A sqrt(v) above zero never
# takes the code of zero.  Scales below 2^-96 are taken as 2^-96.
TINY = 2.0 ** -96
LEAST = 2.0 ** -9  # the smallest e4m3 value above zero


def _encode(t):
    """The codes and the blocks' largest magnitudes."""
    blocks = t.view(-1, BLOCK)
    top = blocks.abs().amax(dim=1, keepdim=True).clamp(min=TINY)
    return (blocks * (448.0 / top)).view(-1), top.view(-1)


def _encode_m(m):
    t, top = _encode(m)
    return t.to(torch.float8_e4m3fn), top


def _encode_v(r):
    t, top = _encode(r)
    return torch.where(r > 0, t.clamp(min=LEAST), t).to(torch.float8_e4m3fn), top


def _decode(codes, top):
    return (codes.view(-1, BLOCK).float() * (top / 448.0).view(-1, 1)).view(-1)


def _adamw_outputs(s):
    out = {"p": s["p"], "m": s["m"], "v": s["v"]}
    if s["bits"] == 8:
        out["m_scales"], out["v_scales"] = s["ms"], s["vs"]
    return out


def _adamw_plain(s):
    a = ADAMW
    g = s["g"].float()
    if s["bits"] == 8:
        m, r = _decode(s["m"], s["ms"]), _decode(s["v"], s["vs"])
        v = r * r
    else:
        m, v = s["m"], s["v"]
    m = m * a["beta1"] + g * (1 - a["beta1"])
    v = v * a["beta2"] + (g * g) * (1 - a["beta2"])
    r = torch.sqrt(v)
    size = a["lr"] / (1 - a["beta1"] ** a["step"])
    denom = r * (1 / math.sqrt(1 - a["beta2"] ** a["step"])) + a["eps"]
    s["p"] = s["p"] * (1 - a["lr"] * a["weight_decay"]) - size * (m / denom)
    if s["bits"] == 8:
        s["m"], s["ms"] = _encode_m(m)
        s["v"], s["vs"] = _encode_v(r)
    else:
        s["m"], s["v"] = m, v
    return _adamw_outputs(s)


# ---- one pass -----------------------------------------------------------------

def _ffn_own(s, case):
    import dense_fp32_sgemm_gb300 as sg
    act = {"silu": sg.GATE_SILU, "gelu": sg.GATE_GELU, "relu": sg.GATE_RELU}[case["act"]]
    x, wg, wu, wd = s["x"], s["wg"], s["wu"], s["wd"]
    if case["op"] == "ffn":
        return {"y": sg.ffn_forward(x, wg, wu, wd, activation=act)}
    saved = sg.ffn_saved(x.shape[0], wg.shape[1]) if case["saved"] else None
    y = sg.ffn_forward(x, wg, wu, wd, activation=act, saved=saved)
    dx, dwg, dwu, dwd = sg.ffn_backward(s["dy"], x, wg, wu, wd, activation=act, saved=saved)
    return {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}


def run(s):
    case = s["case"]
    if case["op"] == "w4":
        return {"y": s["w"].matvec(s["x"], s["y"]) if own else _w4_plain(s, case)}
    if case["op"] == "adamw":
        if not own:
            return _adamw_plain(s)
        s["opt"].step(step=ADAMW["step"])
        return _adamw_outputs(s)
    return _ffn_own(s, case) if own else _ffn_plain(s, case)


# ---- the definition in 64 bits --------------------------------------------------

def _exact_ffn(case, seed):
    s = {k: v.double() for k, v in _ffn_inputs(case, seed).items()}
    x, wg, wu, wd = s["x"], s["wg"], s["wu"], s["wd"]
    g, u = torch.mm(x, wg), torch.mm(x, wu)
    if case["act"] == "silu":
        a = g * torch.sigmoid(g)
        da = torch.sigmoid(g) + a * (1 - torch.sigmoid(g))
    elif case["act"] == "gelu":
        k = (2 / math.pi) ** 0.5
        arg, slope = k * g + k * 0.044715 * g ** 3, k + 3 * k * 0.044715 * g ** 2
        a = g / (1 + torch.exp(-2 * arg))
        da = 1 / (1 + torch.exp(-2 * arg)) + g * slope / (2 * torch.cosh(arg) ** 2)
    else:
        a, da = g.clamp(min=0), (g > 0).double()
    out = {"y": torch.mm(a * u, wd)}
    if case["op"] == "train":
        dh = torch.mm(s["dy"], wd.T)
        dg, du = dh * da * u, dh * a
        out["dx"] = torch.mm(dg, wg.T).addmm_(du, wu.T)
        out["dwg"], out["dwu"] = torch.mm(x.T, dg), torch.mm(x.T, du)
        out["dwd"] = torch.mm((a * u).T, s["dy"])
    return out


def _exact_w4(case, seed):
    s = _w4_inputs(case, seed)
    K, G, N = case["K"], case["group"], case["N"]
    pad = -K % G
    words = s["q"].to(torch.int64) & 0xFFFFFFFF
    nib = torch.stack([(words // 16 ** i) % 16 for i in range(8)], 1).reshape(-1, N)[:K].double()
    nib = torch.cat([nib, nib.new_zeros(pad, N)]).view(-1, G, N)
    zero = s["zeros"].double().unsqueeze(1) if case["zeros"] else 8.0
    w = ((nib - zero) * s["scales"].double().unsqueeze(1)).view(-1, N)[:K]
    return {"y": s["x"].double() @ w}


def _exact_adamw(case, seed):
    s = _adamw_inputs(case, seed)
    a = ADAMW
    g, p = s["g"].double(), s["p"].double()
    if case["bits"] == 8:
        # The states' codes are part of the inputs: what they stand for, in 64 bits.
        m, r = (s[k].double().view(-1, BLOCK) * (s[k + "s"].double() / 448)[:, None]
                for k in ("m", "v"))
        m, v = m.view(-1), r.view(-1) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = a["beta1"] * m + (1 - a["beta1"]) * g
    v = a["beta2"] * v + (1 - a["beta2"]) * g ** 2
    m_hat, v_hat = m / (1 - a["beta1"] ** a["step"]), v / (1 - a["beta2"] ** a["step"])
    p = p - a["lr"] * a["weight_decay"] * p - a["lr"] * m_hat / (v_hat.sqrt() + a["eps"])
    if case["bits"] == 32:
        return {"p": p, "m": m, "v": v}
    r = v.sqrt()
    out = {"p": p}
    for name, t in (("m", m), ("v", r)):
        top = t.abs().view(-1, BLOCK).amax(1).clamp(min=TINY)
        code = (t.view(-1, BLOCK) * (448 / top)[:, None]).view(-1)
        if name == "v":
            code = torch.where(r > 0, code.clamp(min=LEAST), code)
        out[name], out[name + "_scales"] = code.to(torch.float8_e4m3fn).double(), top
    return out


def exact(case, seed):
    return {"ffn": _exact_ffn, "train": _exact_ffn, "w4": _exact_w4,
            "adamw": _exact_adamw}[case["op"]](case, seed)
