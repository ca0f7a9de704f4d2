"""The plaintext side of an encrypted decoder (include/ckks_plain.h): embedding,
residual stream and norms around a block, norms and rotation of heads, products
of 8-bit rows, token sampling and the log probabilities of given tokens.

Argument checks and marshalling only: every step of the computation runs in
the HIP library.  Matrices are 2-D device tensors with unit column stride (any
row stride of at least their columns); calls are enqueued on the current torch stream of the tensors'
device, outputs and scratch come from torch's allocator.

embed, residual_norm, head_norm_rotate and token_logprobs have a gradient.  Results of the other calls have none:
where autograd follows an operand, asking for a derivative through them raises.  Operands with a
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
MAX_HEAD = 512      # CKKS_PLAIN_MAX_HEAD
MAX_TOP = 64        # CKKS_PLAIN_MAX_TOP

ResidualNormGrads = namedtuple("ResidualNormGrads",
                               "dx dy next_weight next_bias block_weight block_bias gate")
HeadNormRotateGrads = namedtuple("HeadNormRotateGrads", "dq dk q_weight k_weight")
TokenLogprobs = namedtuple("TokenLogprobs", "logprob entropy top_token top_logprob largest log_mass")


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


# ------------------------------------------------------------------ embedding

def _embed(tokens, table, scale, dtype):
    is_i8 = isinstance(table, Int8Rows)
    t = table.q if is_i8 else table
    if is_i8:
        (V, D), stride, code = (table.rows, table.cols), t.stride(0), None
    else:
        stride = _matrix(t, "table")
        (V, D), code = t.shape, _type(t, "table")
    dtype = (torch.bfloat16 if is_i8 else t.dtype) if dtype is None else dtype
    if dtype not in TYPES:
        raise ValueError(f"dtype: expected bfloat16, float16 or float32, got {dtype}")
    dev, T = t.device, _count(tokens, "tokens")
    tp = _vector(tokens, "tokens", T, torch.int64, dev)
    out = t.new_empty((T, D), dtype=dtype)
    if is_i8:
        _call("ckks_plain_embed_i8", dev, t.data_ptr(), stride, table.scale.data_ptr(), V, D, tp, T, scale,
              TYPES[dtype], out.data_ptr(), D)
    else:
        _call("ckks_plain_embed", dev, code, t.data_ptr(), stride, V, D, tp, T, scale, TYPES[dtype], out.data_ptr(), D)
    return out


def _count(t, what):
    """Elements of a vector argument."""
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{what}: expected a device vector")
    return t.shape[0]


class _Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale, dtype):
        ctx.save_for_backward(tokens)
        ctx.rest = (table.shape[0], scale, table.dtype)
        return _embed(tokens, table, scale, dtype)

    @staticmethod
    def backward(ctx, drows):
        tokens, = ctx.saved_tensors
        vocab, scale, dtype = ctx.rest
        return None, embed_grad(drows.contiguous(), tokens, vocab, scale, dtype), None, None


def embed(tokens, table, scale: float = 1.0, dtype=None) -> torch.Tensor:
    """[T, D]: scale times the table's row of each token (ckks_plain_embed).  tokens: int64 [T]; a token outside
    [0, V) (padding, or the -1 of sample) gives zeros.  table: [V, D], or Int8Rows (the weights of the vocabulary
    product, whose scales then multiply too).  dtype defaults to that of the table, bfloat16 for Int8Rows.
    Differentiable once through torch.autograd for a table of numbers: its gradient is summed in 32 bits, in a fixed
    order, and rounded to its type."""
    if isinstance(table, Int8Rows):
        out = _embed(tokens, table, scale, dtype)
        if _tracked(table.scale):
            out, = _NoGradient.apply("embed of Int8Rows", (out,), table.scale)
        return out
    if _tracked(table):
        return _Embed.apply(tokens, table, scale, dtype)
    return _embed(tokens, table, scale, dtype)


def embed_grad(drows, tokens, vocab: int, scale: float = 1.0, dtype=torch.float32, into=None) -> torch.Tensor:
    """[vocab, D]: gradient of embed's table from that of its rows (ckks_plain_embed_grad): row v is scale times the
    sum of drows over the tokens v.  into: a matrix [vocab, D] (of any of the three types) that the sums are added to
    and that is returned; only rows of the tokens are touched, where a new matrix is written whole.  The gradient has
    none of its own: a second derivative raises."""
    stride = _matrix(drows, "drows")
    T, D = drows.shape
    dev = drows.device
    if _count(tokens, "tokens") != T:
        raise ValueError(f"tokens: expected {T}, got {tokens.shape[0]}")
    tp = _vector(tokens, "tokens", T, torch.int64, dev)
    if into is None:
        if dtype not in TYPES:
            raise ValueError(f"dtype: expected bfloat16, float16 or float32, got {dtype}")
        out, out_stride = torch.empty((vocab, D), dtype=dtype, device=dev), D
    else:
        out, out_stride = into, _matrix(into, "into", vocab, D, None, dev)
        if into.requires_grad or _tracked(drows):
            raise ValueError("into: sums that autograd follows cannot be added to a matrix")
    _keep, ws, size = _scratch(_workspace("ckks_plain_embed_grad_workspace_size", T, vocab, D), dev)
    _call("ckks_plain_embed_grad", dev, _type(drows, "drows"), drows.data_ptr(), stride, tp, T, vocab, D, scale,
          _type(out, "into"), out.data_ptr(), out_stride, into is not None, ws, size)
    if into is not None:
        if not into.is_inference():
            torch.autograd.graph.increment_version(into)
    elif _tracked(drows):
        out, = _NoGradient.apply("embed_grad", (out,), drows)
    return out


# ------------------------------------------------------------------ heads

def _heads(t, what, tokens=None, dim=None, dtype=None, device=None):
    """(address, token stride, head stride) of a tensor of heads."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{what}: expected a device tensor [tokens, heads, head_dim]")
    if tokens is not None:
        T, _, d = t.shape
        if T != tokens or d != dim:
            raise ValueError(f"{what}: expected [{tokens}, heads, {dim}], got {tuple(t.shape)}")
        if t.dtype is not dtype:
            raise ValueError(f"{what}: expected {dtype}, got {t.dtype}")
        if t.device != device:
            raise ValueError(f"{what} is on {t.device}, not on {device}")
    token, head, across = t.stride()
    if across != 1 and t.shape[2] > 1:
        raise ValueError(f"{what}: expected unit stride within a head")
    return t.data_ptr(), token, head


def _heads_apart(t):
    """Whether the strides are what the kernels take: one within a head, and heads that share no memory."""
    (T, H, d), (token, head, across) = t.shape, t.stride()
    return across == 1 and (T < 2 or token >= d) and (H < 2 or head >= d)


def _head_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved):
    """ckks_plain_heads of the arguments."""
    qp, q_token, q_head = _heads(q, "q")
    T, H, d = q.shape
    dev, dt = q.device, q.dtype
    kp, k_token, k_head, k_heads = None, 0, 0, 0
    if k is not None:
        kp, k_token, k_head = _heads(k, "k", T, d, dt, dev)
        k_heads = k.shape[1]
        if k_heads < 1:
            raise ValueError("k: expected at least one head")
    elif k_weight is not None:
        raise ValueError("k_weight: there is no k")
    rotary, pp, fp = 0, None, None
    if (positions is None) != (inv_freq is None):
        raise ValueError("positions and inv_freq: expected both or none")
    if positions is not None:
        pp = _vector(positions, "positions", T, torch.int64, dev)
        n = _count(inv_freq, "inv_freq")
        fp, rotary = _vector(inv_freq, "inv_freq", n, torch.float32, dev), 2 * n
    return nat.PlainHeads(_type(q, "q"), 1 if interleaved else 0, T, H, k_heads, d, rotary, qp, kp, q_token, q_head,
                          k_token, k_head, _vector(q_weight, "q_weight", d, dt, dev),
                          _vector(k_weight, "k_weight", d, dt, dev), pp, fp, eps)


@functools.lru_cache(maxsize=4096)
def _head_grad_workspace(ty, tokens, q_heads, k_heads, dim, rotary, q_weight, k_weight):
    """Bytes of scratch of the gradient: it goes by sizes and by which weights there are (16: there is one)."""
    p = nat.PlainHeads(ty, 0, tokens, q_heads, k_heads, dim, rotary, 16, 16 if k_heads else None, dim, dim, dim, dim,
                       16 if q_weight else None, 16 if k_weight else None, 16, 16, 0.0)
    out = C.c_size_t()
    nat.check(nat.lib().ckks_plain_head_grad_workspace_size(C.byref(p), C.byref(out)),
              "ckks_plain_head_grad_workspace_size")
    return out.value


def _head_forward(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved):
    p = _head_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved)
    d = p.head_dim
    q_out = q.new_empty(q.shape)
    k_out = None if k is None else k.new_empty(k.shape)
    _call("ckks_plain_head_norm_rotate", q.device, C.byref(p), q_out.data_ptr(), p.q_heads * d, d,
          None if k is None else k_out.data_ptr(), p.k_heads * d, d)
    return q_out, k_out


class _HeadNormRotate(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved):
        ctx.save_for_backward(q, k, positions, inv_freq, q_weight, k_weight)
        ctx.rest = (eps, interleaved)
        return _head_forward(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, positions, inv_freq, qw, kw = ctx.saved_tensors
        if ctx.needs_input_grad[3]:
            raise RuntimeError("head_norm_rotate has no gradient of inv_freq")
        eps, interleaved = ctx.rest
        dq, dk = (v if v is None or _heads_apart(v) else v.contiguous() for v in (dq, dk))
        q_needed, k_needed = (any(ctx.needs_input_grad[i] for i in side) for side in ((0, 4), (1, 5)))
        like = lambda v, p: None if p is None else v.to(p.dtype)  # noqa: E731
        if q_needed and k_needed:
            g = head_norm_rotate_grad(q, k, dq, dk, positions, inv_freq, qw, kw, eps, interleaved)
            return g.dq, g.dk, None, None, like(g.q_weight, qw), like(g.k_weight, kw), None, None
        if q_needed:  # of one side alone
            g = head_norm_rotate_grad(q, None, dq, None, positions, inv_freq, qw, None, eps, interleaved)
            return g.dq, None, None, None, like(g.q_weight, qw), None, None, None
        g = head_norm_rotate_grad(k, None, dk, None, positions, inv_freq, kw, None, eps, interleaved)
        return None, g.dq, None, None, None, like(g.q_weight, kw), None, None


def head_norm_rotate(q, k, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                     interleaved: bool = False):
    """(q, k) [T, heads, d], each head normalised (x / sqrt(mean x^2 + eps) weight) and then rotated by position
    (ckks_plain_head_norm_rotate): pair i of its dimensions, (i, i + r) or (2 i, 2 i + 1) if interleaved, turns by
    positions[t] inv_freq[i]; dimensions from 2 r on stay.  q, k: unit stride within a head, heads and tokens at least a
    head apart (views of a joint projection, heads before tokens; an expanded tensor has to be copied), k may be None.
    The results' gradients may have any strides.  positions: int64 [T]; inv_freq: float32 [r], 2 r <= d; both
    None: no rotation.  q_weight, k_weight: [d], of the type of q; None: no norm.  d is even, at most MAX_HEAD.
    Differentiable once through torch.autograd (gradients of weights are summed in 32 bits, then rounded to their
    type; a second derivative raises, as does one by inv_freq)."""
    if _tracked(q, k, inv_freq, q_weight, k_weight):
        return _HeadNormRotate.apply(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved)
    return _head_forward(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved)


def head_norm_rotate_grad(q, k, dq, dk, positions, inv_freq, q_weight=None, k_weight=None, eps: float = 1e-6,
                          interleaved: bool = False) -> HeadNormRotateGrads:
    """Gradients of head_norm_rotate's q, k and weights from those of its results dq, dk: of q and k in their type,
    of the weights in float32, None where there is no such operand.  They have no gradient of their own: a second
    derivative raises."""
    p = _head_args(q, k, positions, inv_freq, q_weight, k_weight, eps, interleaved)
    T, d, dev = p.tokens, p.head_dim, q.device
    side = []
    for x, g, what in ((q, dq, "dq"), (k, dk, "dk")):
        if (x is None) != (g is None):
            raise ValueError(f"{what}: expected the gradient of each result")
        if x is None:
            side.append((None, 0, 0))
            continue
        side.append(_heads(g, what, T, d, x.dtype, dev))
        if g.shape[1] != x.shape[1]:
            raise ValueError(f"{what}: expected {x.shape[1]} heads, got {g.shape[1]}")
    new = lambda v, dt: None if v is None else v.new_empty(v.shape, dtype=dt)  # noqa: E731
    r = HeadNormRotateGrads(new(q, q.dtype), new(k, q.dtype), new(q_weight, torch.float32),
                            new(k_weight, torch.float32))
    at = lambda v: None if v is None else v.data_ptr()  # noqa: E731
    (dqp, dq_token, dq_head), (dkp, dk_token, dk_head) = side
    g = nat.PlainHeadGrads(dqp, dkp, dq_token, dq_head, dk_token, dk_head, at(r.dq), at(r.dk), p.q_heads * d, d,
                           p.k_heads * d, d, at(r.q_weight), at(r.k_weight))
    _keep, ws, size = _scratch(_head_grad_workspace(p.type, T, p.q_heads, p.k_heads, d, p.rotary,
                                                    q_weight is not None, k_weight is not None), dev)
    _call("ckks_plain_head_norm_rotate_grad", dev, C.byref(p), C.byref(g), ws, size)
    operands = (q, k, dq, dk, inv_freq, q_weight, k_weight)
    if _tracked(*operands):
        some = iter(_NoGradient.apply("head_norm_rotate_grad", tuple(v for v in r if v is not None), *operands))
        r = HeadNormRotateGrads(*(v if v is None else next(some) for v in r))
    return r


# ------------------------------------------------------------------ log probabilities

def _score_args(logits, tokens, temperature, allowed):
    """What both calls begin with, up to the number of columns."""
    stride = _matrix(logits, "logits")
    B, V = logits.shape
    dev = logits.device
    if tokens is None:
        raise ValueError("tokens: expected int64 of every row")
    a_stride = 0
    if allowed is not None:
        a_stride = _matrix(allowed, "allowed", B, V, torch.bool, dev)
    return (_type(logits, "logits"), logits.data_ptr(), stride, _vector(tokens, "tokens", B, torch.int64, dev),
            _vector(temperature, "temperature", B, torch.float32, dev),
            None if allowed is None else allowed.data_ptr(), a_stride, B, V)


def _score(logits, tokens, top, temperature, allowed):
    args = _score_args(logits, tokens, temperature, allowed)
    B, V = logits.shape
    dev = logits.device
    new = lambda dt, *shape: logits.new_empty(shape, dtype=dt)  # noqa: E731
    if not 0 <= top <= MAX_TOP:
        raise ValueError(f"top: expected 0 to {MAX_TOP}, got {top}")
    f32 = torch.float32
    # an allocation for each: views of one would share a version, and a write to one be taken for a write to all
    r = TokenLogprobs(new(f32, B), new(f32, B), new(torch.int64, B, top), new(f32, B, top), new(f32, B), new(f32, B))
    _keep, ws, size = _scratch(_workspace("ckks_plain_token_logprobs_workspace_size", B, V, top), dev)
    _call("ckks_plain_token_logprobs", dev, *args, top, r.logprob.data_ptr(), r.entropy.data_ptr(),
          r.largest.data_ptr(), r.log_mass.data_ptr(), r.top_token.data_ptr() if top else None,
          r.top_logprob.data_ptr() if top else None, ws, size)
    return r


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, top, temperature, allowed):
        ctx.set_materialize_grads(False)
        r = _score(logits, tokens, top, temperature, allowed)
        ctx.save_for_backward(logits, tokens, temperature, allowed, r.entropy, r.largest, r.log_mass)
        ctx.mark_non_differentiable(r.top_token)
        return tuple(r)

    @staticmethod
    def backward(ctx, dlogprob, dentropy, _token, *others):
        if ctx.needs_input_grad[3]:
            raise RuntimeError("token_logprobs has no gradient of the temperature")
        if any(g is not None for g in others):
            raise RuntimeError("token_logprobs has a gradient of logprob and entropy alone")
        logits, tokens, temperature, allowed, entropy, largest, log_mass = ctx.saved_tensors
        scores = TokenLogprobs(None, entropy, None, None, largest, log_mass)
        whole = lambda g: None if g is None else g.contiguous()  # noqa: E731
        return token_logprobs_grad(logits, tokens, scores, whole(dlogprob), whole(dentropy), temperature,
                                   allowed), None, None, None, None


def token_logprobs(logits, tokens, top: int = 0, temperature=None, allowed=None) -> TokenLogprobs:
    """Log probabilities of given tokens under logits [B, V] (ckks_plain_token_logprobs), as sample has them: a token is
    possible if allowed (bool [B, V]) and its logit neither NaN nor -infinity; x = (logit - largest) / temperature
    (float32 [B]; None or <= 0: 1) of those, and
      logprob [B]                of tokens (int64 [B]): x - log_mass; -infinity if it is not possible, 0 if it is
                                 outside [0, V) (a padded row);
      entropy [B]                in natural units;
      top_token, top_logprob     [B, top]: the largest, lower index first among equals; -1 and -infinity behind the
                                 last possible one;
      largest, log_mass [B]      the largest logit and log sum exp x.
    A row without a possible token: entropy 0, largest and log_mass -infinity.  Differentiable once through
    torch.autograd, by the logits, for logprob and entropy; any other derivative raises."""
    if _tracked(logits, temperature):
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, top, temperature, allowed))
    return _score(logits, tokens, top, temperature, allowed)


def token_logprobs_grad(logits, tokens, scores: TokenLogprobs, dlogprob=None, dentropy=None, temperature=None,
                        allowed=None) -> torch.Tensor:
    """Gradient of the logits, in their type, from those of logprob and entropy (float32 [B], None: zero;
    ckks_plain_token_logprobs_grad).  scores: what token_logprobs returned for the same operands.  Tokens that are not
    possible get 0.  The gradient has none of its own: a second derivative raises."""
    args = _score_args(logits, tokens, temperature, allowed)
    B, V = logits.shape
    dev = logits.device
    f32 = lambda v, what: _vector(v, what, B, torch.float32, dev)  # noqa: E731
    stats = [getattr(scores, n, None) for n in ("entropy", "largest", "log_mass")]
    if any(v is None for v in stats):
        raise ValueError("scores: expected what token_logprobs returned")
    out = _like(logits)
    _call("ckks_plain_token_logprobs_grad", dev, *args, *(f32(v, "scores") for v in stats), f32(dlogprob, "dlogprob"),
          f32(dentropy, "dentropy"), out.data_ptr(), V)
    operands = (logits, *stats, dlogprob, dentropy, temperature)
    if _tracked(*operands):
        out, = _NoGradient.apply("token_logprobs_grad", (out,), *operands)
    return out
