"""The operators around the feed-forward block on torch tensors: the
root-mean-square norm with the residual's addition and its gradient, and
serving in 8 bits (the norm, the gate and the weights in 8 bits, and the products
of 8-bit integers).

Argument checks and marshalling only; all arithmetic runs in the library's
CUDA kernels (include/sgemm_q8.h).  Streams, new outputs and errors are as in
ffn.py.  Graphs captured on one stream share that stream's workspace: they may be
replayed one after the other, not at once, nor beside other calls on that stream.
"""
from __future__ import annotations

import contextlib
import importlib.util
import os

import torch
from torch.autograd.function import once_differentiable

import dense_fp32_sgemm_gb300 as _sg

from . import _build
from .ffn import _TYPES, _call, _empty, _matrix, _no_tangent, _tangents, _type_of

_Q8_MOST_K = 131071


def _vector(t, name, n, dtype, device):
    """Address of a contiguous vector of n elements."""
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.device != device or device.type != "cuda":
        raise ValueError(f"{name} must be on the same CUDA device as the other tensors")
    if t.shape != (n,) or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous vector of {n} elements, got {tuple(t.shape)}")
    return t.data_ptr()


def _empty_vector(n, dtype, device, stream):
    if stream is None:
        return torch.empty(n, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=dtype, device=device)


def _empty_codes(rows, cols, device, stream):
    """A new matrix of codes whose rows start on 16 bytes."""
    shape, strides = (rows, cols), (max(-(-cols // 16) * 16, 1), 1)
    if stream is None:
        return torch.empty_strided(shape, strides, dtype=torch.int8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty_strided(shape, strides, dtype=torch.int8, device=device)


# A call takes a few microseconds on the device and its checks several times as long here.
# So the usual call, matrices of one type on the current device and its current stream, goes
# through csrc/torch_calls.cpp, which answers None where there is more to it; all others,
# and all refusals, go the way of this file.
_calls = None


class _NoCalls:
    """In place of the extension where the library was built without it: no call is usual."""

    def _more(*args):
        return None

    rms_norm = rms_norm_q8 = rms_norm_backward = gate_q8 = q8_matmul = staticmethod(_more)


def _load_calls():
    """The extension, once the library is there."""
    global _calls
    _sg.library()
    if not os.path.exists(_build.CALLS_PATH):
        _calls = _NoCalls
        return _calls
    spec = importlib.util.spec_from_file_location("_torch_calls", _build.CALLS_PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    _calls = module
    return module


def _done(result, name):
    """What a call returned, or the error that its status stands for."""
    if type(result) is int:
        raise _sg.SgemmError(result, name)
    return result


def _written(*tensors):
    """Given outputs: one that requires a gradient is refused (what is written has none), and
    graphs that hold one will know that it was overwritten."""
    _no_tangent("a given output", *tensors)
    if _graph(*tensors):
        raise ValueError("a given output has no gradient, and it requires one: leave it out, "
                         "or call under torch.no_grad()")
    for t in tensors:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _address(t, name, rows, cols, dtype, device):
    """Address and leading dimension, of None too."""
    return (None, max(cols, 1)) if t is None else _matrix(t, name, rows, cols, dtype, device)


def _graph(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


def _no_gradient(what, *tensors):
    _no_tangent(what, *tensors)
    if _graph(*tensors):
        raise ValueError(f"{what} has no gradient, and an input requires one: call it under "
                         "torch.no_grad()")


def _norm_args(x, weight, residual, eps, h, stream, want_h, h_name="h"):
    """The leading arguments of the norm's calls, and h (allocated where it is wanted and
    not given)."""
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    T, D = x.shape
    kind, dev = _type_of(x, "x"), x.device
    if weight.dtype is not x.dtype and weight.dtype is not torch.float32:
        raise TypeError(f"weight must be {x.dtype} or torch.float32")
    args = (T, D, kind, *_address(x, "x", T, D, x.dtype, dev),
            *_address(residual, "residual", T, D, x.dtype, dev),
            _vector(weight, "weight", D, weight.dtype, dev), _TYPES[weight.dtype], float(eps))
    if h is None and want_h:
        h = _empty(T, D, x.dtype, dev, stream)
    return T, D, dev, args, h, _address(h, h_name, T, D, x.dtype, dev)


def rms_norm(x, weight, residual=None, eps: float = 1e-6, y=None, h=None, stream=None):
    """y = h * weight / sqrt(mean(h^2) + eps) over the rows of h = x + residual (h = x
    without a residual), on CUDA tensors.

    x, residual: T x D of one type (float32, float16 or bfloat16); weight: D elements of
    that type or float32.  Returns y, and with a residual (y, h), h rounded to
    the type; the norm is taken of the sum before that rounding.  y and h are allocated
    when not given; one of them may be x, one the residual (updated in place).

    Where one of the inputs requires a gradient, y and h are part of the graph:
    their gradients go through rms_norm_backward() with h, which the graph keeps (the rounded
    sum alone, not x and the residual).  A given y or h is refused then.  A backward pass may
    be captured where no eager graph of the same leaves is alive: torch waits for
    the stream of such a graph, which a capture cannot.
    """
    if stream is None:
        got = (_calls or _load_calls()).rms_norm(x, weight, residual, eps, y, h)
        if got is not None:
            return _done(got, "sgemm_rms_norm")
    _no_tangent("rms_norm", x, weight, residual)
    if _graph(x, weight, residual):
        if y is not None or h is not None:
            raise ValueError("a given y or h has no gradient, and an input requires one: "
                             "leave them out, or call under torch.no_grad()")
        # (the gradient runs on the stream that is current here)
        with contextlib.nullcontext() if stream is None else torch.cuda.stream(stream):
            return _Norm.apply(x, weight, residual, float(eps))
    _written(y, h)
    T, D, dev, args, h, ha = _norm_args(x, weight, residual, eps, h, stream, residual is not None)
    if y is None:
        y = _empty(T, D, x.dtype, dev, stream)
    ya = _address(y, "y", T, D, x.dtype, dev)
    if h is not None and T and D and ya[0] == ha[0]:
        raise ValueError("y and h must not be the same tensor")
    _call(_sg.library().sgemm_rms_norm, dev, stream, *args, *ha, *ya)
    return y if residual is None else (y, h)


class _Norm(torch.autograd.Function):
    """rms_norm as a node of the graph."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        ctx.set_materialize_grads(False)
        ctx.eps = eps
        if residual is None:
            y = rms_norm(x, weight, eps=eps)
            ctx.save_for_backward(x, weight)
            return y
        y, h = rms_norm(x, weight, residual, eps)
        ctx.save_for_backward(h, weight)
        return y, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        h, weight = ctx.saved_tensors
        need_x, need_w, need_r = ctx.needs_input_grad[:3]
        if dy is None:
            return (dh if need_x else None, torch.zeros_like(weight) if need_w else None,
                    dh if need_r else None, None)
        # (a sum's gradient comes with rows or columns that share memory)
        dx, dw = rms_norm_backward(dy.contiguous(), h, weight, eps=ctx.eps,
                                   dh=None if dh is None else dh.contiguous(),
                                   need_dx=need_x or need_r, need_dw=need_w)
        return dx if need_x else None, dw, dx if need_r else None, None


def rms_norm_backward(dy, x, weight, residual=None, dh=None, eps: float = 1e-6, dx=None,
                      dweight=None, need_dx: bool = True, need_dw: bool = True, stream=None):
    """Gradients (dx, dweight) of rms_norm for dy.

    x, residual: rms_norm's, for the gradients at their sum in 32 bits; or x the h that it
    returned and no residual, which reads one matrix less, for those at the rounded
    sum.  dh: None, or the gradient that reaches h otherwise, which is added.  dx is the gradient of x
    and of the residual alike.  Outputs not given are allocated (dx may be dy or dh
    itself); ``need_dx`` and ``need_dw`` leave one out (None is returned in its place).  No
    gradient goes through it: inputs that require one are refused (call it under
    torch.no_grad(), or let torch call it: rms_norm is part of its graph).
    """
    if stream is None:
        got = (_calls or _load_calls()).rms_norm_backward(x, weight, residual, eps, dy, dh, dx, dweight,
                                                          need_dx, need_dw)
        if got is not None:
            return _done(got, "sgemm_rms_norm_backward")
    _no_gradient("rms_norm_backward", dy, x, weight, residual, dh)
    _written(dx if need_dx else None, dweight if need_dw else None)
    T, D, dev, args, _, dha = _norm_args(x, weight, residual, eps, dh, stream, False, "dh")
    dya = _address(dy, "dy", T, D, x.dtype, dev)
    dxa, dwa = (None, max(D, 1)), None
    if not need_dx:
        dx = None
    else:
        if dx is None:
            dx = _empty(T, D, x.dtype, dev, stream)
        dxa = _address(dx, "dx", T, D, x.dtype, dev)
    if not need_dw:
        dweight = None
    else:
        if dweight is None:
            dweight = _empty_vector(D, weight.dtype, dev, stream)
        dwa = _vector(dweight, "dweight", D, weight.dtype, dev)
    _call(_sg.library().sgemm_rms_norm_backward, dev, stream, *args, *dya, *dha, *dxa, dwa)
    return dx, dweight


def _codes(q, scales, T, D, dev, stream):
    """q and scales, allocated where not given, and their arguments."""
    if q is None:
        q = _empty_codes(T, D, dev, stream)
    if scales is None:
        scales = _empty_vector(T, torch.float32, dev, stream)
    return q, scales, (*_address(q, "q", T, D, torch.int8, dev),
                       _vector(scales, "scales", T, torch.float32, dev))


def rms_norm_q8(x, weight, residual=None, eps: float = 1e-6, h=None, q=None, scales=None,
                stream=None):
    """rms_norm with y in 8 bits: (q, scales), or (q, scales, h) with a residual.

    y[t] is about q[t] * scales[t]; q: T x D int8, scales: T float32.  Outputs not
    given are allocated (new codes lie in rows that start on 16 bytes); h may be x or the
    residual.  A row with an infinity or NaN has the scale NaN.  No gradient goes
    through it: inputs that require one are refused.
    """
    if stream is None and q is None and scales is None:
        got = (_calls or _load_calls()).rms_norm_q8(x, weight, residual, eps, h)
        if got is not None:
            return _done(got, "sgemm_rms_norm_q8")
    _no_gradient("rms_norm_q8", x, weight, residual)
    _written(h, q, scales)
    T, D, dev, args, h, ha = _norm_args(x, weight, residual, eps, h, stream, residual is not None)
    q, scales, qa = _codes(q, scales, T, D, dev, stream)
    _call(_sg.library().sgemm_rms_norm_q8, dev, stream, *args, *ha, *qa)
    return (q, scales) if residual is None else (q, scales, h)


def gate_q8(g, u, activation: int = 0, q=None, scales=None, stream=None):
    """act(g) * u in 8 bits: (q, scales), what the down product of a block reads.

    g, u: T x F of one type (they may be halves of one matrix).  ``activation`` is
    GATE_SILU, GATE_GELU or GATE_RELU.  Otherwise as rms_norm_q8.
    """
    if stream is None and q is None and scales is None and u is not None:
        got = (_calls or _load_calls()).gate_q8(g, u, activation)
        if got is not None:
            return _done(got, "sgemm_q8_gate")
    _no_gradient("gate_q8", g, u)
    _written(q, scales)
    if g.dim() != 2:
        raise ValueError("g must be 2-D")
    T, F = g.shape
    dev = g.device
    kind = _type_of(g, "g")
    ga = _address(g, "g", T, F, g.dtype, dev)
    ua = _matrix(u, "u", T, F, g.dtype, dev)
    q, scales, qa = _codes(q, scales, T, F, dev, stream)
    _call(_sg.library().sgemm_q8_gate, dev, stream, T, F, kind, int(activation), *ga, *ua, *qa)
    return q, scales


def rows_q8(x, q=None, scales=None, stream=None):
    """The rows of x in 8 bits: (q, scales).  Otherwise as rms_norm_q8."""
    if stream is None and q is None and scales is None:
        got = (_calls or _load_calls()).gate_q8(x, None, 0)
        if got is not None:
            return _done(got, "sgemm_q8_gate")
    _no_gradient("rows_q8", x)
    _written(q, scales)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    T, D = x.shape
    dev = x.device
    kind = _type_of(x, "x")
    xa = _address(x, "x", T, D, x.dtype, dev)
    q, scales, qa = _codes(q, scales, T, D, dev, stream)
    _call(_sg.library().sgemm_q8_gate, dev, stream, T, D, kind, 0, *xa, None, max(D, 1), *qa)
    return q, scales


_UNCHECKED = (0, 0, 0, -1, 0, -1, 0)  # in place of a Q8Matrix's addresses: no tensor's


class Q8Matrix:
    """A K x N matrix of 8-bit weights, W[k][n] = scales[n] * qweight[n][k].

    qweight: N x K int8, a row the weights of one channel (output column).  scales: N
    float32.  ``dtype`` is the type of the products.  The tensors are checked once and
    kept (again where their memory is another than it was); a qweight whose rows do not start on 16 bytes is copied into rows that do
    (the copy is waited for, so that products may run on any stream).
    """

    def __init__(self, qweight, scales, dtype=torch.bfloat16):
        if qweight.dim() != 2:
            raise ValueError("qweight must be 2-D")
        self.N, self.K = qweight.shape
        if self.K > _Q8_MOST_K:
            raise ValueError(f"K must be at most {_Q8_MOST_K}: beyond it a sum could pass 32 bits")
        if dtype not in _TYPES:
            raise TypeError("dtype must be float32, float16 or bfloat16")
        dev = qweight.device
        w, ldw = _matrix(qweight, "qweight", self.N, self.K, torch.int8, dev)
        s = _vector(scales, "scales", self.N, torch.float32, dev)
        if w % 16 or (self.N > 1 and ldw % 16):
            with torch.cuda.device(dev):
                qweight = _empty_codes(self.N, self.K, dev, None).copy_(qweight)
                torch.cuda.current_stream(dev).synchronize()
            w, ldw = _matrix(qweight, "qweight", self.N, self.K, torch.int8, dev)
        self.qweight, self.scales, self.dtype, self.device = qweight, scales, dtype, dev
        self._weights = (self.N, self.K, _TYPES[dtype], w, ldw, s, dev.index)

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name in ("qweight", "scales", "dtype"):
            super().__setattr__("_weights", _UNCHECKED)

    def __getstate__(self):
        # A copy (copy.deepcopy, pickle) has tensors of its own: its first product checks them.
        return {**self.__dict__, "_weights": _UNCHECKED}

    def matmul(self, x, x_scales, y=None, stream=None):
        """y[m] = x_scales[m] * (x[m] @ W) for M x K codes x (int8) and M scales, as
        rms_norm_q8, gate_q8 and rows_q8 return them.  The sums are exact.  Returns y
        (allocated when not given).  No gradient goes through it: scales that require one,
        the matrix's own too, are refused."""
        if self.scales.requires_grad or _tangents(self.scales):
            _no_gradient("Q8Matrix.matmul", self.scales)
        all_weights = self._weights  # (once: another thread may replace a tensor)
        if all_weights[3] != self.qweight.data_ptr() or all_weights[5] != self.scales.data_ptr():
            # (tensors put in the place of these, or a module's that was moved)
            Q8Matrix.__init__(self, self.qweight, self.scales, self.dtype)
            all_weights = self._weights
        if stream is None:
            got = (_calls or _load_calls()).q8_matmul(x, x_scales, y, all_weights)
            if got is not None:
                return _done(got, "sgemm_q8_matmul")
        _no_gradient("Q8Matrix.matmul", x_scales, y)
        if x.dim() != 2:
            raise ValueError("x must be 2-D")
        M = x.shape[0]
        N, K, kind, *weights, _ = all_weights
        if y is None:
            y = _empty(M, N, self.dtype, self.device, stream)
        else:
            _written(y)
        xa = _address(x, "x", M, K, torch.int8, self.device)
        sa = _vector(x_scales, "x_scales", M, torch.float32, self.device)
        _call(_sg.library().sgemm_q8_matmul, self.device, stream, M, N, K, kind, *xa, sa, *weights,
              *_address(y, "y", M, N, self.dtype, self.device))
        return y


def q8_quantize(w, stream=None) -> Q8Matrix:
    """The 8-bit form of a K x N CUDA tensor: a scale for each column; products of w's
    type.  No gradient goes through it: a w that requires one is refused."""
    _no_gradient("q8_quantize", w)
    if w.dim() != 2:
        raise ValueError("w must be 2-D")
    K, N = w.shape
    if K > _Q8_MOST_K:
        raise ValueError(f"K must be at most {_Q8_MOST_K}: beyond it a sum could pass 32 bits")
    kind, dev = _type_of(w, "w"), w.device
    a = _matrix(w, "w", K, N, w.dtype, dev)
    q = _empty_codes(N, K, dev, stream)
    scales = _empty_vector(N, torch.float32, dev, stream)
    _call(_sg.library().sgemm_q8_quantize, dev, stream, N, K, kind, *a, q.data_ptr(),
          max(q.stride(0), K, 1), scales.data_ptr())
    return Q8Matrix(q, scales, dtype=w.dtype)
