"""The feed-forward operators on torch tensors: the gated block with its
backward pass, products with 4-bit weights, and the AdamW step.

Argument checks and marshalling only; all arithmetic runs in the library's
CUDA kernels (include/sgemm_ffn.h).  Work is queued on ``stream`` (a
torch.cuda.Stream) or the current stream; no call that queues work waits for it.  Outputs that
are made here are allocated on the stream that writes them, as torch does under
``torch.cuda.stream(stream)``: to use one on another stream, let that stream wait
for ``stream`` and tell the allocator by ``record_stream``.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

import dense_fp32_sgemm_gb300 as _sg

_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
ADAMW_BLOCK = 256


def _matrix(t, name, rows, cols, dtype, device):
    """Address and leading dimension of a row-major rows x cols tensor."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} must be on the same CUDA device as the other tensors")
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} must be {rows} x {cols}, got {tuple(t.shape)}")
    step, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit column stride (row-major)")
    return t.data_ptr(), _sg._leading(name, rows, cols, step)


def _empty(rows, cols, dtype, device, stream):
    """A new rows x cols tensor from the memory of the stream that will write it.
    (From the current stream's, the allocator could hand out memory that work queued
    there still uses, and give it away again while `stream` still writes.)"""
    if stream is None:
        return torch.empty(rows, cols, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(rows, cols, dtype=dtype, device=device)


def _type_of(t, name):
    try:
        return _TYPES[t.dtype]
    except KeyError:
        raise TypeError(f"{name} must be float32, float16 or bfloat16") from None


def _call(fn, device, stream, *args):
    """One C-ABI call with `device` current and the stream as last argument."""
    index = device.index
    # The raw handle: torch.cuda.current_stream() makes an object first, which
    # takes as long as the whole C call.
    raw = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == torch.cuda.current_device():
        status = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            status = fn(*args, raw)
    if status != 0:
        raise _sg.SgemmError(status, fn.__name__)


def _tangents(*tensors):
    """Whether one of the tensors (or None) carries a tangent of forward-mode differentiation."""
    if getattr(forward_ad, "_current_level", 0) < 0:  # (outside of all its levels)
        return False
    return any(t is not None and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _no_tangent(what, *tensors):
    if _tangents(*tensors):
        raise ValueError(f"{what} has no forward-mode derivative, and a tensor carries a tangent")


def _raw_stream(index):
    return torch._C._cuda_getCurrentRawStream(index)


def _block(x, w_gate, w_up, w_down):
    """Sizes, type and the leading arguments of the block's calls."""
    if x.dim() != 2 or w_gate.dim() != 2:
        raise ValueError("x and w_gate must be 2-D")
    T, D = x.shape
    F = w_gate.shape[1]
    kind, dev = _type_of(x, "x"), x.device
    args = (*_matrix(x, "x", T, D, x.dtype, dev), *_matrix(w_gate, "w_gate", D, F, x.dtype, dev),
            *_matrix(w_up, "w_up", D, F, x.dtype, dev),
            *_matrix(w_down, "w_down", F, D, x.dtype, dev))
    return T, D, F, kind, args


def _saved_address(saved, T, F, kind, device):
    if saved is None:
        return None
    need = _sg.library().sgemm_ffn_saved_floats(T, F, kind)
    if (saved.dtype != torch.float32 or saved.device != device or not saved.is_contiguous()
            or saved.numel() < need):
        raise ValueError(f"saved must be a contiguous float32 tensor of {need} elements on {device}")
    return saved.data_ptr()


def ffn_saved(T: int, F: int, device="cuda", dtype=torch.float32):
    """A buffer for what the forward pass of ``dtype`` matrices keeps for the
    backward pass (without ``dtype`` one that is large enough for any)."""
    need = _sg.library().sgemm_ffn_saved_floats(int(T), int(F), _TYPES[dtype])
    return torch.empty(need, dtype=torch.float32, device=device)


def ffn_forward(x, w_gate, w_up, w_down, y=None, activation: int = 0, saved=None, stream=None):
    """y = (act(x @ w_gate) * (x @ w_up)) @ w_down, on CUDA tensors of one type
    (float32, float16 or bfloat16).

    x: T x D, w_gate and w_up: D x F (they may be halves of one matrix),
    w_down: F x D; rows may lie apart, columns not.  ``activation`` is
    GATE_SILU, GATE_GELU or GATE_RELU.  ``saved``: a buffer from ffn_saved()
    for ffn_backward().  Returns y (allocated when not given).  With 16-bit types h is
    rounded to the type between the products, but for a few rows without ``saved``: an
    FP16 h above 65504 becomes infinite.

    Where one of the matrices requires a gradient, y is part of the graph: its
    gradient goes through ffn_backward(), with ``saved`` if given (one for each
    forward pass that waits for its gradient), else from the inputs anew.  A given
    y is refused then, and so are tensors with a tangent of forward-mode differentiation.
    """
    _no_tangent("ffn_forward", x, w_gate, w_up, w_down, y)
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad
                                    or w_down.requires_grad):
        if y is not None:
            raise ValueError("a given y has no gradient, and x or a weight requires one: "
                             "leave y out, or call under torch.no_grad()")
        # (the gradient runs on the stream that is current here)
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            return _Block.apply(x, w_gate, w_up, w_down, int(activation), saved)
    T, D, F, kind, args = _block(x, w_gate, w_up, w_down)
    if y is None:
        y = _empty(T, D, x.dtype, x.device, stream)
    _call(_sg.library().sgemm_ffn_forward, x.device, stream, T, D, F, kind, int(activation), *args,
          *_matrix(y, "y", T, D, x.dtype, x.device), _saved_address(saved, T, F, kind, x.device))
    if saved is not None:
        torch.autograd.graph.increment_version(saved)  # graphs that hold it will know
    return y


class _Block(torch.autograd.Function):
    """ffn_forward as a node of the graph."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, w_down, activation, saved):
        y = ffn_forward(x, w_gate, w_up, w_down, activation=activation, saved=saved)
        ctx.save_for_backward(x, w_gate, w_up, w_down, saved)
        ctx.activation = activation
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, w_gate, w_up, w_down, saved = ctx.saved_tensors
        need = ctx.needs_input_grad
        # (a sum's gradient comes with rows or columns that share memory)
        grads = ffn_backward(dy.contiguous(), x, w_gate, w_up, w_down, activation=ctx.activation,
                             saved=saved, need_dx=need[0], need_dw=any(need[1:4]))
        return (*grads, None, None)


def ffn_backward(dy, x, w_gate, w_up, w_down, dx=None, dw_gate=None, dw_up=None, dw_down=None,
                 activation: int = 0, saved=None, need_dx: bool = True, need_dw: bool = True,
                 stream=None):
    """Gradients (dx, dw_gate, dw_up, dw_down) of ffn_forward for dy.

    ``saved``: the buffer the forward pass filled, or None to compute its
    contents again.  Outputs not given are allocated; ``need_dx`` and
    ``need_dw`` leave out the input's or the weights' gradients (None is
    returned in their place).  With FP16 the gradients inside the block are FP16 too:
    scale a small dy up by a power of two, and the results (or AdamW's grad_scale) down.
    """
    T, D, F, kind, args = _block(x, w_gate, w_up, w_down)
    dev, dtype = x.device, x.dtype
    dya = _matrix(dy, "dy", T, D, dtype, dev)
    keep = _saved_address(saved, T, F, kind, dev)

    def out(t, name, rows, cols, wanted):
        if not wanted:
            return None, (None, max(cols, 1))
        if t is None:
            t = _empty(rows, cols, dtype, dev, stream)
        return t, _matrix(t, name, rows, cols, dtype, dev)

    dx, a = out(dx, "dx", T, D, need_dx)
    dw_gate, b = out(dw_gate, "dw_gate", D, F, need_dw)
    dw_up, c = out(dw_up, "dw_up", D, F, need_dw)
    dw_down, d = out(dw_down, "dw_down", F, D, need_dw)
    _call(_sg.library().sgemm_ffn_backward, dev, stream, T, D, F, kind, int(activation), *args,
          *dya, keep, *a, *b, *c, *d)
    return dx, dw_gate, dw_up, dw_down


class W4Matrix:
    """A K x N matrix of 4-bit weights, W[k][n] = scales[k // group][n] *
    (q[k][n] - zeros[k // group][n]), zeros 8 where none are given.

    qweight: ceil(K / 8) x N int32 words, eight values along K in a word, the
    first in the lowest bits.  scales: ceil(K / group) x N of the type x will
    have.  zeros: None, or uint8 of the scales' shape (values 0 to 15).  group:
    a multiple of 32.  The tensors are checked once and kept.
    """

    def __init__(self, qweight, scales, K: int, group: int, zeros=None):
        K, group = int(K), int(group)
        if group < 32 or group % 32:
            raise ValueError("group must be a positive multiple of 32")
        if qweight.dim() != 2:
            raise ValueError("qweight must be 2-D")
        N, dev = qweight.shape[1], qweight.device
        groups = -(-K // group)
        self.type = _type_of(scales, "scales")
        q, ldq = _matrix(qweight, "qweight", -(-K // 8), N, torch.int32, dev)
        s, lds = _matrix(scales, "scales", groups, N, scales.dtype, dev)
        z, ldz = (None, max(N, 1)) if zeros is None else _matrix(zeros, "zeros", groups, N,
                                                                 torch.uint8, dev)
        self.K, self.N, self.group, self.device, self.dtype = K, N, group, dev, scales.dtype
        self.qweight, self.scales, self.zeros = qweight, scales, zeros
        self._weights = (q, ldq, s, lds, z, ldz)
        self._index = dev.index
        self._fn = _sg.library().sgemm_w4_matvec

    def matvec(self, x, y=None, stream=None):
        """y = x @ W for M x K rows x (M is meant to be small: the weights are
        read once per 16 rows, 8 with float32).  Returns y (allocated when not given).
        No gradient goes through it: where x requires one, a backward pass through y
        raises NotImplementedError, and a given y is refused."""
        _no_tangent("W4Matrix.matvec", x, y, self.scales)
        if x.requires_grad and torch.is_grad_enabled():
            if y is not None:
                raise ValueError("a given y has no gradient, and x requires one: "
                                 "leave y out, or call under torch.no_grad()")
            with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
                return _Matvec.apply(x, self)
        M = x.shape[0]
        if y is None:
            y = _empty(M, self.N, self.dtype, self.device, stream)
        if (x.shape == (M, self.K) and y.shape == (M, self.N) and x.dtype is self.dtype
                and y.dtype is self.dtype and x.get_device() == y.get_device() == self._index
                and x.is_contiguous() and y.is_contiguous()):
            # The usual call, a few microseconds long on the device.
            xa, ldx, ya, ldy = x.data_ptr(), max(self.K, 1), y.data_ptr(), max(self.N, 1)
        else:
            xa, ldx = _matrix(x, "x", M, self.K, self.dtype, self.device)
            ya, ldy = _matrix(y, "y", M, self.N, self.dtype, self.device)
        _call(self._fn, self.device, stream, M, self.N, self.K, self.group, self.type, xa, ldx,
              *self._weights, ya, ldy)
        return y


class _Matvec(torch.autograd.Function):
    """W4Matrix.matvec as a node of the graph that has no gradient, and says so."""

    @staticmethod
    def forward(ctx, x, matrix):
        return matrix.matvec(x)

    @staticmethod
    def backward(ctx, dy):
        raise NotImplementedError("products with 4-bit weights have no gradient")


def w4_quantize(w, group: int = 128, zeros: bool = True, stream=None) -> W4Matrix:
    """The 4-bit form of a K x N CUDA tensor: per group of a column a scale
    (of w's type) and, with ``zeros``, a zero point."""
    if w.dim() != 2:
        raise ValueError("w must be 2-D")
    K, N = w.shape
    group = int(group)
    if group < 32 or group % 32:
        raise ValueError("group must be a positive multiple of 32")
    kind, dev = _type_of(w, "w"), w.device
    a = _matrix(w, "w", K, N, w.dtype, dev)
    groups = -(-K // group)
    q = _empty(-(-K // 8), N, torch.int32, dev, stream)
    s = _empty(groups, N, w.dtype, dev, stream)
    z = _empty(groups, N, torch.uint8, dev, stream) if zeros else None
    _call(_sg.library().sgemm_w4_quantize, dev, stream, N, K, group, kind, *a, q.data_ptr(),
          max(N, 1), s.data_ptr(), max(N, 1), z.data_ptr() if zeros else None, max(N, 1))
    return W4Matrix(q, s, K, group, zeros=z)


class _AdamTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("copy", ctypes.c_void_p),
                ("numel", ctypes.c_int64)]


class AdamW:
    """The AdamW step over a list of contiguous CUDA tensors.

    params: of one type (float32, float16 or bfloat16), updated in place.
    grads: buffers of one type, read by every step (set_grads() replaces
    them).  m, v: the states, float32, or float8_e4m3fn together with m_scales
    and v_scales (float32, one value per 256 elements of a tensor) for states
    of 8 bits; left out, they are made here with ``state_bits`` (which waits for the
    current stream: their zeros are there for a step on any stream).  copies:
    None, or tensors of one type that receive the updated parameters (16-bit
    weights beside FP32 parameters).  The tensors are kept: their storage must
    stay where it is.  ``steps`` counts the steps taken.
    """

    def __init__(self, params, grads, m=None, v=None, m_scales=None, v_scales=None, copies=None,
                 lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, state_bits: int = 32):
        self.params = list(params)
        if not self.params:
            raise ValueError("no parameters")
        self.device = self.params[0].device
        if m is None:
            if state_bits not in (8, 32):
                raise ValueError("state_bits must be 8 or 32")
            kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn

            def states():
                return [torch.zeros(p.numel(), dtype=torch.uint8 if state_bits == 8 else kind,
                                    device=p.device).view(kind) for p in self.params]

            m, v = states(), states()
            if state_bits == 8:
                m_scales, v_scales = ([torch.zeros(-(-p.numel() // ADAMW_BLOCK), dtype=torch.float32,
                                                   device=p.device)
                                       for p in self.params] for _ in range(2))
            if self.device.type == "cuda":
                # Steps may run on any stream: the zeros are there before the first.
                torch.cuda.current_stream(self.device).synchronize()
        self.m, self.v = list(m), list(v)
        self.state_bits = 32 if self.m[0].dtype == torch.float32 else 8
        state = torch.float32 if self.state_bits == 32 else torch.float8_e4m3fn
        if self.state_bits == 8 and (m_scales is None or v_scales is None):
            raise ValueError("8-bit states need m_scales and v_scales")
        self.m_scales = list(m_scales) if self.state_bits == 8 else None
        self.v_scales = list(v_scales) if self.state_bits == 8 else None
        self.copies = None if copies is None else list(copies)
        self.lr, self.betas, self.eps, self.weight_decay = lr, tuple(betas), eps, weight_decay
        self.steps = 0
        self._type = _type_of(self.params[0], "params")
        self._copy_type = _type_of(self.copies[0], "copies") if self.copies else 0
        self._table = (_AdamTensor * len(self.params))()
        blocks = [-(-p.numel() // ADAMW_BLOCK) for p in self.params]
        sizes = [p.numel() for p in self.params]
        for field, tensors, dtype, counts in (
                ("param", self.params, self.params[0].dtype, sizes), ("m", self.m, state, sizes),
                ("v", self.v, state, sizes), ("m_scale", self.m_scales, torch.float32, blocks),
                ("v_scale", self.v_scales, torch.float32, blocks),
                ("copy", self.copies, self.copies[0].dtype if self.copies else None, sizes)):
            if tensors is not None:
                self._fill(field, tensors, dtype, counts)
        for entry, n in zip(self._table, sizes):
            entry.numel = n
        self.set_grads(grads)

    def _fill(self, field, tensors, dtype, counts):
        """Puts the tensors' addresses into the table: all of them, or none where one is
        refused."""
        if len(tensors) != len(self._table):
            raise ValueError(f"{field}: {len(tensors)} tensors for {len(self._table)} parameters")
        index = self.device.index if self.device.type == "cuda" else None
        for t, n in zip(tensors, counts):
            if t.dtype is not dtype:
                raise TypeError(f"every {field} must be {dtype}")
            if t.get_device() != index or not t.is_contiguous() or t.numel() != n:
                raise ValueError(f"every {field} must be a contiguous tensor of its parameter's "
                                 f"size on {self.device}")
        for entry, t in zip(self._table, tensors):
            setattr(entry, field, t.data_ptr())

    def set_grads(self, grads):
        """Take the gradients from these buffers from now on.  Where one of them is refused,
        the handle stays as it was."""
        grads = list(grads)
        kind = _type_of(grads[0], "grads") if grads else 0
        self._fill("grad", grads, grads[0].dtype if grads else None,
                   [e.numel for e in self._table])
        self.grads, self._grad_type = grads, kind

    def step(self, step: int | None = None, grad_scale: float = 1.0, stream=None) -> None:
        """One step; ``step`` (from 1 on) sets the count that the bias
        corrections use, ``grad_scale`` multiplies the gradients."""
        count = self.steps + 1 if step is None else int(step)
        _call(_sg.library().sgemm_adamw_step, self.device, stream, self._table, len(self._table),
              self._type, self._grad_type, self._copy_type, self.state_bits, self.lr,
              self.betas[0], self.betas[1], self.eps, self.weight_decay, count, float(grad_scale))
        self.steps = count
