"""The plaintext side of an encrypted decoder (include/ckks_plain.h): residual
stream and norms around a block, products of 8-bit rows, and token sampling.

Argument checks and marshalling only: every step of the computation runs in
the HIP library.  Matrices are 2-D device tensors with unit column stride (any
row stride of at least their columns); calls are enqueued on the current torch stream of the tensors'
device, outputs and scratch come from torch's allocator.

residual_norm has a gradient.  Results of the other calls have none: where autograd
follows an operand, asking for a derivative through them raises.  Operands with a
tangent of forward-mode differentiation are refused by all of them.
"""
from __future__ import annotations

import ctypes as C
import functools
from collections import namedtuple

import torch
from torch.autograd import forward_ad

from . import _native as nat

TYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
KINDS = {"rms": 0, "layer": 1}
I8_ROW = 128        # CKKS_PLAIN_I8_ROW
MAX_COLS = 16384    # CKKS_PLAIN_MAX_COLS

ResidualNormGrads = namedtuple("ResidualNormGrads",
                               "dx dy next_weight next_bias block_weight block_bias gate")


_entry = {}


def _call(name, device, *args):
    """One C call on `device` and its current stream."""
    f = _entry.get(name)
    if f is None:
        f = _entry[name] = getattr(nat.lib(), name)
    index = device.index
    if _current_device() == index:
        code = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(device):
            code = f(*args, _raw_stream(index))
    if code:
        raise nat.CkksError(code, name)


# The addresses of the current device and stream without the objects around them, which take longer than a small
# kernel does.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


@functools.lru_cache(maxsize=4096)
def _workspace(name, *sizes):
    """Bytes of scratch that the C call of these sizes takes."""
    out = C.c_size_t()
    nat.check(getattr(nat.lib(), name)(*sizes, C.byref(out)), name)
    return out.value


@functools.lru_cache(maxsize=4096)
def _norm_grad_workspace(rows, cols, groups, next_bias, block_weight, block_bias):
    """The same for the norm's gradient: it goes by sizes and by which operands there are (16: there is one)."""
    p = nat.PlainNorm(0, 0, rows, cols, groups, 16, 16, cols, cols, 16, 16 if next_bias else None,
                      16 if block_weight else None, 16 if block_bias else None, 16 if groups else None, 1.0, 0.0)
    out = C.c_size_t()
    nat.check(nat.lib().ckks_plain_norm_grad_workspace_size(C.byref(p), C.byref(out)),
              "ckks_plain_norm_grad_workspace_size")
    return out.value


def _scratch(nbytes, device):
    """(tensor kept alive, address, size)"""
    if not nbytes:
        return None, None, 0
    t = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), nbytes


def _matrix(t, what, rows=None, cols=None, dtype=None, device=None):
    """Row stride of a matrix argument (torch leaves that of a matrix with at most one row open)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{what}: expected a device tensor")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{what}: expected a matrix with unit column stride")
    T, D = shape
    down, across = t.stride()
    if D > 1 and across != 1:
        raise ValueError(f"{what}: expected a matrix with unit column stride")
    if (rows is not None and T != rows) or (cols is not None and D != cols):
        raise ValueError(f"{what}: expected {rows} x {cols}, got {tuple(shape)}")
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{what} is on {t.device}, not on {device}")
    return down if T > 1 else max(down, D)


def _vector(t, what, n, dtype, device):
    """Address of a contiguous vector of n elements (None: null)."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.device != device:
        raise ValueError(f"{what}: expected {dtype} on {device}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{what}: expected a contiguous vector of {n}, got {tuple(t.shape)}")
    return t.data_ptr()


def _like(x):
    """A new contiguous matrix of the shape and type of x."""
    return torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)


class _NoGradient(torch.autograd.Function):
    """Hands results on as they are; a gradient through them, which nothing here computes, is an error."""
    @staticmethod
    def forward(ctx, name, results, *operands):
        ctx.name = name
        return results

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no gradient")


def _tracked(*operands):
    """Whether autograd may follow one of the operands (None: no such operand).  Tangents of forward mode do not
    show in requires_grad; a Function refuses them, as none here has a rule for them."""
    if forward_ad._current_level >= 0:
        return True
    if torch.is_grad_enabled():
        try:
            for t in operands:
                if t is not None and t.requires_grad:
                    return True
        except AttributeError:  # no tensor: the checks name it
            pass
    return False


def _type(t, what):
    code = TYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{what}: expected bfloat16, float16 or float32, got {t.dtype}")
    return code


class Int8Rows:
    """8-bit rows: row t stands for scale[t] * q[t, :cols].

    q: int8 [rows, >= cols rounded up to I8_ROW] with rows that start at multiples of I8_ROW bytes
    is kept as it is; any other layout is copied into such rows once, here.  scale: float32 [rows].

    Kernels multiply whole pieces of I8_ROW bytes, so one operand of a product has to hold zeros behind
    the columns.  Rows made here do.  What lies there in rows kept as they are is not looked at (that
    would wait for the GPU): a product of two such operands takes a copy of the smaller."""

    __slots__ = ("q", "scale", "cols", "_ends_in_zeros")

    def __init__(self, q: torch.Tensor, scale: torch.Tensor, cols: int | None = None):
        if not isinstance(q, torch.Tensor) or not q.is_cuda or q.dtype != torch.int8 or q.dim() != 2:
            raise ValueError("q: expected an int8 matrix on the device")
        cols = q.shape[1] if cols is None else cols
        if not 1 <= cols <= q.shape[1]:
            raise ValueError(f"cols: {cols} of {q.shape[1]}")
        _vector(scale, "scale", q.shape[0], torch.float32, q.device)
        padded = -(-cols // I8_ROW) * I8_ROW
        self.q, self.scale, self.cols, self._ends_in_zeros = q, scale, cols, cols == padded
        down, across = q.stride()
        if q.shape[1] < padded or across != 1 or down % I8_ROW or down < padded or q.data_ptr() % 16:
            self.q, self._ends_in_zeros = self._copy(), True

    def _copy(self) -> torch.Tensor:
        """The columns in rows of whole pieces, zeros behind them."""
        rows = torch.zeros((self.q.shape[0], -(-self.cols // I8_ROW) * I8_ROW), dtype=torch.int8, device=self.q.device)
        rows[:, :self.cols] = self.q[:, :self.cols]
        return rows

    @staticmethod
    def empty(rows: int, cols: int, device) -> "Int8Rows":
        """For a call that writes whole rows, zeros behind the columns included."""
        self = object.__new__(Int8Rows)
        self.q = torch.empty((rows, -(-cols // I8_ROW) * I8_ROW), dtype=torch.int8, device=device)
        self.scale = torch.empty(rows, dtype=torch.float32, device=device)
        self.cols, self._ends_in_zeros = cols, True
        return self

    @property
    def rows(self) -> int:
        return self.q.shape[0]

    def dequantize(self, dtype=torch.float32) -> torch.Tensor:
        return (self.q[:, :self.cols].float() * self.scale[:, None]).to(dtype)


def _norm(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind):
    """ckks_plain_norm of the arguments."""
    x_stride = _matrix(x, "x")
    T, D = x.shape
    dev, dt = x.device, x.dtype
    y_stride = _matrix(y, "y", T, D, dt, dev)
    if kind not in KINDS:
        raise ValueError(f"kind: expected 'rms' or 'layer', got {kind!r}")
    groups, gp = 0, None
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise ValueError("gate: expected a device tensor")
        if gate.dim() == 1:
            groups, gp = 1, _vector(gate, "gate", D, dt, dev)
        else:
            _matrix(gate, "gate", None, D, dt, dev)
            if not gate.is_contiguous() or gate.shape[0] < 1 or T % gate.shape[0]:
                raise ValueError(f"gate: expected contiguous rows, a divisor of {T}, got {tuple(gate.shape)}")
            groups, gp = gate.shape[0], gate.data_ptr()
    return nat.PlainNorm(_type(x, "x"), KINDS[kind], T, D, groups, x.data_ptr(), y.data_ptr(), x_stride, y_stride,
                         _vector(next_weight, "next_weight", D, dt, dev), _vector(next_bias, "next_bias", D, dt, dev),
                         _vector(block_weight, "block_weight", D, dt, dev),
                         _vector(block_bias, "block_bias", D, dt, dev), gp, scale, eps)


def _norm_forward(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind):
    p = _norm(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind)
    h, u = _like(x), _like(x)
    D = x.shape[1]
    _call("ckks_plain_residual_norm", x.device, C.byref(p), h.data_ptr(), D, u.data_ptr(), D)
    return h, u


class _ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind):
        ctx.save_for_backward(x, y, next_weight, next_bias, block_weight, block_bias, gate)
        ctx.rest = (scale, eps, kind)
        return _norm_forward(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind)

    @staticmethod
    def backward(ctx, dh, du):
        x, y, nw, nb, bw, bb, gate = ctx.saved_tensors
        scale, eps, kind = ctx.rest
        g = residual_norm_grad(x, y, dh.contiguous(), du.contiguous(), nw, nb, bw, bb, gate, scale, eps, kind)
        like = lambda v, p: None if p is None else v.view(p.shape).to(p.dtype)  # noqa: E731
        return (g.dx, g.dy, like(g.next_weight, nw), like(g.next_bias, nb), like(g.block_weight, bw),
                like(g.block_bias, bb), like(g.gate, gate), None, None, None)


def residual_norm(x, y, next_weight, next_bias=None, block_weight=None, block_bias=None, gate=None,
                  scale: float = 1.0, eps: float = 1e-6, kind: str = "rms"):
    """(h, u): the residual stream x takes the block output y, and its norm for the next block
    (ckks_plain_residual_norm).  n = y, or block_weight norm(y) + block_bias; h = x + scale gate n;
    u = next_weight norm(h) + next_bias.  x, y [T, D]; weights and biases [D]; gate [D] or [G, D]
    (a row for T / G tokens each); one type for all.  Differentiable once through torch.autograd (gradients of weights
    are summed in 32 bits, then rounded to their type; a second derivative raises)."""
    if _tracked(x, y, next_weight, next_bias, block_weight, block_bias, gate):
        return _ResidualNorm.apply(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind)
    return _norm_forward(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind)


def residual_norm_i8(x, y, next_weight, next_bias=None, block_weight=None, block_bias=None, gate=None,
                     scale: float = 1.0, eps: float = 1e-6, kind: str = "rms"):
    """(h, rows): residual_norm with u as 8-bit rows, quantised before any other rounding."""
    p = _norm(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind)
    h, u = _like(x), Int8Rows.empty(*x.shape, x.device)
    _call("ckks_plain_residual_norm_i8", x.device, C.byref(p), h.data_ptr(), x.shape[1], u.q.data_ptr(),
          u.q.shape[1], u.scale.data_ptr())
    operands = (x, y, next_weight, next_bias, block_weight, block_bias, gate)
    if _tracked(*operands):
        h, u.q, u.scale = _NoGradient.apply("residual_norm_i8", (h, u.q, u.scale), *operands)
    return h, u


def residual_norm_grad(x, y, dh, du, next_weight, next_bias=None, block_weight=None, block_bias=None, gate=None,
                       scale: float = 1.0, eps: float = 1e-6, kind: str = "rms") -> ResidualNormGrads:
    """Gradients of residual_norm's operands from those of h and u: dx and dy in the type of x, those
    of weights, biases and gate (of the gate's shape) in float32, None where there is no such operand.
    They have no gradient of their own: a second derivative raises."""
    p = _norm(x, y, next_weight, next_bias, block_weight, block_bias, gate, scale, eps, kind)
    T, D = x.shape
    dh_stride = _matrix(dh, "dh", T, D, x.dtype, x.device)
    du_stride = _matrix(du, "du", T, D, x.dtype, x.device)
    new = lambda v: None if v is None else torch.empty(v.shape, dtype=torch.float32, device=x.device)  # noqa: E731
    r = ResidualNormGrads(_like(x), _like(x), new(next_weight), new(next_bias), new(block_weight), new(block_bias),
                          new(gate))
    at = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    g = nat.PlainNormGrads(dh.data_ptr(), du.data_ptr(), dh_stride, du_stride, r.dx.data_ptr(), r.dy.data_ptr(),
                           D, D, at(r.next_weight), at(r.next_bias), at(r.block_weight), at(r.block_bias), at(r.gate))
    _keep, ws, size = _scratch(_norm_grad_workspace(T, D, p.groups, next_bias is not None, block_weight is not None,
                                                    block_bias is not None), x.device)
    _call("ckks_plain_residual_norm_grad", x.device, C.byref(p), C.byref(g), ws, size)
    operands = (x, y, dh, du, next_weight, next_bias, block_weight, block_bias, gate)
    if _tracked(*operands):
        some = iter(_NoGradient.apply("residual_norm_grad", tuple(v for v in r if v is not None), *operands))
        r = ResidualNormGrads(*(v if v is None else next(some) for v in r))
    return r


def quantize_rows(x) -> Int8Rows:
    """8-bit rows of x [T, D] (ckks_plain_quantize_rows): scale = max |x| times 1/127 of the row."""
    stride = _matrix(x, "x")
    r = Int8Rows.empty(x.shape[0], x.shape[1], x.device)
    _call("ckks_plain_quantize_rows", x.device, _type(x, "x"), x.data_ptr(), stride, x.shape[0], x.shape[1],
          r.q.data_ptr(), r.q.shape[1], r.scale.data_ptr())
    if _tracked(x):
        r.q, r.scale = _NoGradient.apply("quantize_rows", (r.q, r.scale), x)
    return r


def _product(cols, device, w, bias, dtype):
    """Checks what both products check; the address of the bias."""
    if not isinstance(w, Int8Rows):
        raise ValueError("w: expected Int8Rows")
    if cols != w.cols or device != w.q.device:
        raise ValueError(f"{cols} columns on {device}, w has {w.cols} on {w.q.device}")
    if dtype not in TYPES:
        raise ValueError(f"dtype: expected bfloat16, float16 or float32, got {dtype}")
    return _vector(bias, "bias", w.rows, torch.float32, device)


def matmul_i8(a: Int8Rows, w: Int8Rows, bias=None, dtype=torch.bfloat16) -> torch.Tensor:
    """out[t, c] = a.scale[t] w.scale[c] sum_k a.q[t, k] w.q[c, k] + bias[c] (ckks_plain_matmul_i8),
    sums exact in 32-bit integers.  bias: float32 [channels]."""
    if not isinstance(a, Int8Rows):
        raise ValueError("a: expected Int8Rows")
    dev = a.q.device
    bp = _product(a.cols, dev, w, bias, dtype)
    M, N = a.rows, w.rows
    out = torch.empty((M, N), dtype=dtype, device=dev)
    _keep, ws, size = _scratch(_workspace("ckks_plain_matmul_i8_workspace_size", M, N, a.cols), dev)
    aq, wq = a.q, w.q
    if not (a._ends_in_zeros or w._ends_in_zeros):
        aq, wq = (a._copy(), wq) if M <= N else (aq, w._copy())
    _call("ckks_plain_matmul_i8", dev, aq.data_ptr(), aq.stride(0), a.scale.data_ptr(), wq.data_ptr(), wq.stride(0),
          w.scale.data_ptr(), bp, TYPES[dtype], out.data_ptr(), N, M, N, a.cols, ws, size)
    if _tracked(a.scale, w.scale, bias):
        out, = _NoGradient.apply("matmul_i8", (out,), a.scale, w.scale, bias)
    return out


def linear_i8(x, w: Int8Rows, bias=None, dtype=None) -> torch.Tensor:
    """matmul_i8 of x [T, D] quantised row by row (ckks_plain_linear_i8); dtype defaults to that of x."""
    stride = _matrix(x, "x")
    dtype = x.dtype if dtype is None else dtype
    dev, (M, K) = x.device, x.shape
    bp = _product(K, dev, w, bias, dtype)
    N = w.rows
    out = torch.empty((M, N), dtype=dtype, device=dev)
    _keep, ws, size = _scratch(_workspace("ckks_plain_linear_i8_workspace_size", M, N, K), dev)
    _call("ckks_plain_linear_i8", dev, _type(x, "x"), x.data_ptr(), stride, w.q.data_ptr(), w.q.stride(0),
          w.scale.data_ptr(), bp, TYPES[dtype], out.data_ptr(), N, M, N, K, ws, size)
    if _tracked(x, w.scale, bias):
        out, = _NoGradient.apply("linear_i8", (out,), x, w.scale, bias)
    return out


def sample(logits, gumbel, temperature, top_k=None, top_p=None, min_p=None, allowed=None):
    """(token int64 [B], logprob float32 [B]) from logits [B, V] (ckks_plain_sample).  gumbel: float32
    [B, V], -log(-log u) of uniform numbers; temperature, top_p, min_p: float32 [B]; top_k: int32 [B];
    allowed: bool [B, V].  temperature <= 0: the largest logit.  A row without a possible token:
    token -1, logprob -infinity."""
    z_stride = _matrix(logits, "logits")
    B, V = logits.shape
    dev = logits.device
    g_stride = _matrix(gumbel, "gumbel", B, V, torch.float32, dev)
    if temperature is None:
        raise ValueError("temperature: expected float32 of every row")
    a_stride = 0
    if allowed is not None:
        a_stride = _matrix(allowed, "allowed", B, V, torch.bool, dev)
    token = torch.empty(B, dtype=torch.int64, device=dev)
    logprob = torch.empty(B, dtype=torch.float32, device=dev)
    _keep, ws, size = _scratch(_workspace("ckks_plain_sample_workspace_size", B, V), dev)
    _call("ckks_plain_sample", dev, _type(logits, "logits"), logits.data_ptr(), z_stride, gumbel.data_ptr(),
          g_stride, _vector(temperature, "temperature", B, torch.float32, dev),
          _vector(top_k, "top_k", B, torch.int32, dev), _vector(top_p, "top_p", B, torch.float32, dev),
          _vector(min_p, "min_p", B, torch.float32, dev), None if allowed is None else allowed.data_ptr(),
          a_stride, B, V, token.data_ptr(), logprob.data_ptr(),
          ws, size)
    if _tracked(logits, gumbel, temperature, top_p, min_p):
        token, logprob = _NoGradient.apply("sample", (token, logprob), logits, gumbel, temperature, top_p, min_p)
    return token, logprob
