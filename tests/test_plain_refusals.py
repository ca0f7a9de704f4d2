"""The plaintext-side C entry points refuse what they do not take, with the
documented code and before any launch (so this runs without a GPU: the
addresses below are never followed)."""
import ctypes as C

import pytest

from rns_ckks_polynomial_amd import _native as nat

INV, ALIGN, UNSUP, WS = nat.EINVAL, nat.EALIGN, nat.EUNSUPPORTED, nat.EWORKSPACE
X, Y, H, U, W, G, Q, S, WSP = (0x10000000 * (i + 1) for i in range(9))
T, D = 8, 64


def norm(**kw):
    f = dict(type=0, kind=0, rows=T, cols=D, groups=0, x=X, y=Y, x_stride=D, y_stride=D, next_weight=W, next_bias=None,
             block_weight=None, block_bias=None, gate=None, scale=1.0, eps=1e-6)
    f.update(kw)
    return nat.PlainNorm(**f)


BAD_NORM = [
    (dict(type=3), INV), (dict(type=-1), INV), (dict(kind=2), INV), (dict(rows=-1), INV), (dict(cols=0), INV),
    (dict(cols=16385, x_stride=16385, y_stride=16385), UNSUP), (dict(x=None), INV), (dict(y=None), INV),
    (dict(x_stride=D - 1), INV), (dict(y_stride=D - 1), INV), (dict(next_weight=None), INV),
    (dict(block_bias=W), INV), (dict(gate=G), INV), (dict(groups=1), INV), (dict(gate=G, groups=3), INV),
    (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(x=X + 1), ALIGN), (dict(y=Y + 1), ALIGN),
    (dict(type=2, next_weight=W + 2), ALIGN), (dict(gate=G + 1, groups=1), ALIGN), (dict(rows=1 << 31), INV),
]


@pytest.mark.parametrize("kw,code", BAD_NORM)
def test_norm_arguments(kw, code):
    lib, p = nat.lib(), norm(**kw)
    assert lib.ckks_plain_residual_norm(C.byref(p), H, 1 << 15, U, 1 << 15, None) == code
    assert lib.ckks_plain_residual_norm_i8(C.byref(p), H, 1 << 15, Q, 1 << 15, S, None) == code
    g = nat.PlainNormGrads(dh=H, du=U, dh_stride=1 << 15, du_stride=1 << 15, dx=Q, dy=S, dx_stride=1 << 15,
                           dy_stride=1 << 15, next_weight=WSP)
    assert lib.ckks_plain_residual_norm_grad(C.byref(p), C.byref(g), G + (1 << 27), 1 << 20, None) == code


@pytest.mark.parametrize("h,hs,u,us,code", [
    (None, D, U, D, INV), (H, D, None, D, INV), (H, D - 1, U, D, INV), (H, D, U, D - 1, INV), (H + 1, D, U, D, ALIGN),
    (H, D, U + 1, D, ALIGN), (H, D, H, D, INV), (H, D, H + 2 * D, D, INV), (Y, D, U, D, INV), (H, D, X, D, INV),
    (X + 2 * D, D, U, D, INV), (X, D + 1, U, D, INV), (H, D, W, D, INV),
])
def test_norm_outputs(h, hs, u, us, code):
    p = norm()
    assert nat.lib().ckks_plain_residual_norm(C.byref(p), h, hs, u, us, None) == code


@pytest.mark.parametrize("q,qs,s,code", [
    (None, 128, S, INV), (Q, 128, None, INV), (Q, 64, S, INV), (Q, 192, S, INV), (Q + 8, 128, S, ALIGN),
    (Q, 128, S + 2, ALIGN), (Q, 128, Q + 128, INV), (X, 128, S, INV), (Q, 128, Y, INV), (H, 128, S, INV),
])
def test_i8_outputs(q, qs, s, code):
    p, lib = norm(), nat.lib()
    assert lib.ckks_plain_residual_norm_i8(C.byref(p), H, D, q, qs, s, None) == code
    if q != H:  # no residual stream there
        assert lib.ckks_plain_quantize_rows(0, Y if s == Y else X, D, T, D, q, qs, s, None) == code


def test_null_norm():
    lib, n = nat.lib(), C.c_size_t()
    assert lib.ckks_plain_residual_norm(None, H, D, U, D, None) == INV
    assert lib.ckks_plain_norm_grad_workspace_size(None, C.byref(n)) == INV
    assert lib.ckks_plain_norm_grad_workspace_size(C.byref(norm()), None) == INV


GRAD = dict(dh=H, du=U, dh_stride=D, du_stride=D, dx=Q, dy=S, dx_stride=D, dy_stride=D, next_weight=G)


@pytest.mark.parametrize("kw,ws,code", [
    (dict(dh=None), WSP, INV), (dict(du_stride=D - 1), WSP, INV), (dict(dx=None), WSP, INV), (dict(dy=Q), WSP, INV),
    (dict(dx=X), WSP, INV), (dict(dx=H), WSP, INV), (dict(next_weight=None), WSP, INV), (dict(next_bias=W), WSP, INV),
    (dict(gate=W), WSP, INV), (dict(next_weight=G + 2), WSP, ALIGN), (dict(dy=S + 1), WSP, ALIGN), ({}, None, WS),
    ({}, WSP + 4, ALIGN), ({}, Q, INV), ({}, X, INV),
])
def test_grad_arguments(kw, ws, code):
    p, g, lib = norm(), nat.PlainNormGrads(**{**GRAD, **kw}), nat.lib()
    assert lib.ckks_plain_residual_norm_grad(C.byref(p), C.byref(g), ws, 1 << 20, None) == code


def test_grad_workspace():
    p, g, lib, n = norm(), nat.PlainNormGrads(**GRAD), nat.lib(), C.c_size_t()
    assert lib.ckks_plain_norm_grad_workspace_size(C.byref(p), C.byref(n)) == 0 and n.value > 0
    assert lib.ckks_plain_residual_norm_grad(C.byref(p), C.byref(g), WSP, n.value - 1, None) == WS
    assert lib.ckks_plain_residual_norm_grad(C.byref(p), None, WSP, n.value, None) == INV


@pytest.mark.parametrize("args,code", [
    ((3, X, D, T, D, Q, 128, S), INV), ((0, X, D, -1, D, Q, 128, S), INV), ((0, X, D, T, 0, Q, 128, S), INV),
    ((0, X, 1 << 20, T, 16385, Q, 1 << 20, S), UNSUP), ((0, None, D, T, D, Q, 128, S), INV),
    ((2, X + 2, D, T, D, Q, 128, S), ALIGN), ((0, X, D - 1, T, D, Q, 128, S), INV),
])
def test_quantize_arguments(args, code):
    assert nat.lib().ckks_plain_quantize_rows(*args, None) == code


MM = dict(a=X, a_stride=128, a_scale=Y, w=W, w_stride=128, w_scale=G, bias=None, out_type=0, out=H, out_stride=32,
          rows=T, channels=32, cols=100, ws=WSP, ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,code", [
    (dict(a=None), INV), (dict(w=None), INV), (dict(a_scale=None), INV), (dict(w_scale=None), INV),
    (dict(out=None), INV), (dict(a_stride=64), INV), (dict(w_stride=192), INV), (dict(out_stride=31), INV),
    (dict(out_type=3), INV), (dict(rows=-1), INV), (dict(channels=-1), INV), (dict(cols=0), INV),
    (dict(cols=131072, a_stride=1 << 20, w_stride=1 << 20), INV), (dict(a=X + 8), ALIGN), (dict(w=W + 4), ALIGN),
    (dict(a_scale=Y + 1), ALIGN), (dict(bias=S + 2), ALIGN), (dict(out=H + 1), ALIGN), (dict(out=X), INV),
    (dict(out=W + 128), INV), (dict(out=Y), INV), (dict(out=G), INV), (dict(bias=S, out=S), INV),
    (dict(rows=1 << 31), INV),
])
def test_matmul_arguments(kw, code):
    assert nat.lib().ckks_plain_matmul_i8(*{**MM, **kw}.values(), None) == code


LIN = dict(type=0, x=X, x_stride=D, w=W, w_stride=128, w_scale=G, bias=None, out_type=0, out=H, out_stride=32,
           rows=T, channels=32, cols=D, ws=WSP, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INV), (dict(out_type=-1), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(w_scale=None), INV),
    (dict(out=None), INV), (dict(x_stride=D - 1), INV), (dict(w_stride=64), INV), (dict(out_stride=31), INV),
    (dict(rows=-1), INV), (dict(channels=-1), INV), (dict(cols=0), INV), (dict(rows=1 << 31), INV),
    (dict(cols=16385, x_stride=16385, w_stride=1 << 15), UNSUP), (dict(x=X + 1), ALIGN), (dict(w=W + 8), ALIGN),
    (dict(out=H + 1), ALIGN), (dict(bias=S + 2), ALIGN), (dict(ws=WSP + 8), ALIGN), (dict(ws=None), WS),
    (dict(ws_bytes=T * 128), WS), (dict(out=X), INV), (dict(out=W + 128), INV), (dict(out=G), INV),
    (dict(bias=S, out=S), INV), (dict(ws=X), INV), (dict(ws=H), INV), (dict(ws=W), INV), (dict(ws=G), INV),
    (dict(bias=S, ws=S), INV),
])
def test_linear_arguments(kw, code):
    assert nat.lib().ckks_plain_linear_i8(*{**LIN, **kw}.values(), None) == code


def test_linear_workspace():
    lib, n = nat.lib(), C.c_size_t()
    assert lib.ckks_plain_linear_i8_workspace_size(T, 32, D, C.byref(n)) == 0 and n.value >= T * 128 + T * 4
    assert lib.ckks_plain_linear_i8(*{**LIN, "ws_bytes": n.value - 1}.values(), None) == WS
    assert lib.ckks_plain_linear_i8_workspace_size(T, 32, 16385, C.byref(n)) == UNSUP
    assert lib.ckks_plain_linear_i8_workspace_size(T, 32, D, None) == INV
    assert lib.ckks_plain_linear_i8(*{**LIN, "rows": 0}.values(), None) == 0


SMP = dict(type=0, logits=X, logits_stride=D, gumbel=Y, gumbel_stride=D, temperature=W, top_k=None, top_p=None,
           min_p=None, allowed=None, allowed_stride=0, rows=T, vocab=D, token=H, logprob=U, ws=WSP, ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,code", [
    (dict(type=5), INV), (dict(logits=None), INV), (dict(gumbel=None), INV), (dict(temperature=None), INV),
    (dict(token=None), INV), (dict(logprob=None), INV), (dict(logits_stride=D - 1), INV),
    (dict(gumbel_stride=D - 1), INV), (dict(allowed=G), INV), (dict(rows=-1), INV), (dict(vocab=0), INV),
    (dict(vocab=(1 << 24) + 1), INV), (dict(logits=X + 1), ALIGN), (dict(gumbel=Y + 2), ALIGN),
    (dict(token=H + 4), ALIGN), (dict(logprob=U + 2), ALIGN), (dict(temperature=W + 2), ALIGN),
    (dict(top_k=G + 1), ALIGN), (dict(token=X), INV), (dict(logprob=Y + 8), INV), (dict(logprob=H + 8), INV),
])
def test_sample_arguments(kw, code):
    assert nat.lib().ckks_plain_sample(*{**SMP, **kw}.values(), None) == code


def test_no_rows_is_valid():
    lib = nat.lib()
    assert lib.ckks_plain_residual_norm(C.byref(norm(rows=0, x=None, y=None)), None, 0, None, 0, None) == 0
    assert lib.ckks_plain_quantize_rows(0, None, 0, 0, D, None, 0, None, None) == 0
    assert lib.ckks_plain_matmul_i8(*{**MM, "rows": 0}.values(), None) == 0
    assert lib.ckks_plain_matmul_i8(*{**MM, "channels": 0}.values(), None) == 0
    assert lib.ckks_plain_sample(*{**SMP, "rows": 0}.values(), None) == 0


def test_binding_wants_device_matrices():
    torch = pytest.importorskip("torch")
    from rns_ckks_polynomial_amd import plain
    x = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="device tensor"):
        plain.residual_norm(x, x, torch.ones(8))
    with pytest.raises(ValueError, match="device tensor"):
        plain.quantize_rows(x)
    with pytest.raises(ValueError, match="on the device"):
        plain.Int8Rows(torch.zeros(2, 128, dtype=torch.int8), torch.ones(2))
    with pytest.raises(ValueError, match="device tensor"):
        plain.sample(x, x, torch.ones(2))
    with pytest.raises(ValueError, match="Int8Rows"):
        plain.matmul_i8(x, x)
    with pytest.raises(ValueError, match="device tensor|Int8Rows"):
        plain.linear_i8(x, x)


@pytest.mark.parametrize("kw", [dict(rows=(1 << 31) - 255), dict(channels=(1 << 31) - 255, out_stride=1 << 31)])
def test_products_whose_indexes_pass_32_bits(kw):
    far = {"out": 1 << 60, "a": 1 << 50, "w": 1 << 52}  # nothing overlaps at any size
    assert nat.lib().ckks_plain_matmul_i8(*{**MM, **far, **kw}.values(), None) == INV
    far = {"out": 1 << 60, "x": 1 << 50, "w": 1 << 52, "ws": 1 << 55, "ws_bytes": 1 << 54}
    assert nat.lib().ckks_plain_linear_i8(*{**LIN, **far, **kw}.values(), None) == INV
