"""The plaintext-side kernels (include/ckks_plain.h) against their definitions
in 64 bits (plain_ref), at sizes, layouts and masks where they can go wrong.

Bounds, eps = 2^-24: a row's sums add at most 16 terms in a thread, 6 shuffles
and 16 waves, so a mean or mean square is within 38 eps of the sum of its
absolute terms; its root, the quotient and up to 6 further roundings stay under
64 eps of the largest term of the row, and each of two norms in a row adds as
much again.  A sum over rows adds at most `depth` terms in order, each within
that bound.  Storing in 16 bits adds half a step: 2^-9 (bfloat16) or 2^-11
(float16) of the value."""
import numpy as np
import pytest

import plain_ref
from gpu_util import require_gpu, say, torch
from rns_ckks_polynomial_amd import plain

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
TYPE = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def f64(t):
    return None if t is None else t.detach().cpu().to(torch.float64).numpy()


def rnd(seed, *shape, scale=1.0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal(shape) * scale)


def wide(v, dtype, pad, offset=0):
    """v on the GPU as rows of a buffer `pad` columns wider, `offset` columns in."""
    buf = torch.full((v.shape[0], v.shape[1] + pad), float("nan"), dtype=dtype, device="cuda")
    buf[:, offset:offset + v.shape[1]] = v.to(dtype)
    return buf[:, offset:offset + v.shape[1]]


def inputs(seed, T, D, ty, block, bias, groups, pad=0, offset=0):
    dt = TYPE[ty]
    x = wide(rnd(seed, T, D, scale=2) + rnd(seed + 1, 1, D), dt, pad, offset)
    y = wide(rnd(seed + 2, T, D) + 0.3, dt, pad, offset)
    v = lambda k, m, s: (rnd(seed + k, D, scale=s) + m).to(dt).cuda()  # noqa: E731
    p = {"next_weight": v(3, 1, 0.1)}
    if bias:
        p["next_bias"] = v(4, 0, 0.5)
    if block:
        p["block_weight"] = v(5, 0.5, 0.1)
        if bias:
            p["block_bias"] = v(6, 0, 0.5)
    if groups is not None:
        p["gate"] = (rnd(seed + 7, groups, D) if groups else rnd(seed + 7, D)).to(dt).cuda()
    return x, y, p


def ref_args(p):
    short = {"next_weight": "nw", "next_bias": "nb", "block_weight": "bw", "block_bias": "bb", "gate": "gate"}
    return {short[k]: f64(v) for k, v in p.items()}


def close(got, ref, size, terms, ty, what):
    tol = np.broadcast_to(terms * EPS * size, ref.shape)
    low, high = (f64(torch.from_numpy(v).float().to(TYPE[ty])) for v in (ref - tol, ref + tol))
    v = f64(got)
    bad = ~((v >= low) & (v <= high))
    assert not bad.any(), f"{what}: {bad.sum()} outside, first at {np.argwhere(bad)[0]}: {v[bad][0]} for {ref[bad][0]} +- {tol[bad][0]}"


def top(v):
    return np.abs(v).max(1, keepdims=True)


def forward_sizes(f, x, y, a, scale):
    n = top(y) if "bw" not in a else top(f["yhat"]) * np.abs(a["bw"]).max() + (np.abs(a["bb"]).max() if "bb" in a else 0)
    h = top(x) + abs(scale) * top(f["g"]) * n
    return h, f["rh"] * h * np.abs(a["nw"]).max() * (1 + top(f["hhat"])) + (np.abs(a["nb"]).max() if "nb" in a else 0)


SHAPES = [(1, 1), (3, 2), (5, 63), (4, 512), (7, 513), (2, 1000), (3, 1024), (2, 2048), (65, 1032), (3, 4096), (2, 5003),
          (2, 8192), (2, 8200), (1, 16384)]


@pytest.mark.parametrize("T,D", SHAPES)
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind,block,bias,groups", [("rms", False, False, None), ("rms", True, False, 0),
                                                    ("layer", True, True, 1), ("layer", False, True, None)])
def test_residual_norm(T, D, ty, kind, block, bias, groups):
    say(f"residual_norm {T}x{D} {ty} {kind} block={block} bias={bias} groups={groups}")
    x, y, p = inputs(T * 31 + D, T, D, ty, block, bias, groups)
    h, u = plain.residual_norm(x, y, scale=0.7, eps=1e-5, kind=kind, **p)
    assert h.dtype == u.dtype == TYPE[ty] and h.shape == u.shape == (T, D)
    s = float(np.float32(0.7))
    f = plain_ref.norm_forward(f64(x), f64(y), **ref_args(p), scale=s, eps=float(np.float32(1e-5)), kind=kind)
    sh, su = forward_sizes(f, f64(x), f64(y), ref_args(p), s)
    close(h, f["h"], sh, 64, ty, "h")
    close(u, f["u"], su, 192, ty, "u")


@pytest.mark.parametrize("pad,offset", [(8, 0), (8, 8), (1, 0), (9, 3)])
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_residual_norm_layouts(pad, offset, ty):
    """Aligned and unaligned rows give the same values; other rows and the gaps are untouched."""
    x, y, p = inputs(5, 6, 1000, ty, True, True, 3, pad, offset)
    h, u = plain.residual_norm(x, y, kind="layer", **p)
    h2, u2 = plain.residual_norm(x.contiguous(), y.contiguous(), kind="layer", **p)
    f = plain_ref.norm_forward(f64(x), f64(y), **ref_args(p), kind="layer", eps=float(np.float32(1e-6)))
    sh, su = forward_sizes(f, f64(x), f64(y), ref_args(p), 1.0)
    for a, b in ((h, u), (h2, u2)):
        close(a, f["h"], sh, 64, ty, "h")
        close(b, f["u"], su, 192, ty, "u")


def test_residual_norm_per_token_gate_and_in_place():
    x, y, p = inputs(9, 6, 256, "bf16", False, False, 6)
    h, u = plain.residual_norm(x, y, **p)
    import ctypes as C
    from rns_ckks_polynomial_amd import _native as nat
    a = plain._norm(x, y, p["next_weight"], None, None, None, p["gate"], 1.0, 1e-6, "rms")
    u2 = torch.empty_like(u)
    assert nat.lib().ckks_plain_residual_norm(C.byref(a), x.data_ptr(), 256, u2.data_ptr(), 256,
                                              torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(x, h) and torch.equal(u, u2)


def test_norm_rows_do_not_mix_what_is_not_finite():
    x, y, p = inputs(11, 5, 700, "f32", True, False, None)
    clean = plain.residual_norm(x, y, **p)
    i8 = plain.residual_norm_i8(x, y, **p)
    x[1, 3], y[3, 699] = float("inf"), float("nan")
    h, u = plain.residual_norm(x, y, **p)
    _, rows = plain.residual_norm_i8(x, y, **p)
    for r in (0, 2, 4):
        assert torch.equal(h[r], clean[0][r]) and torch.equal(u[r], clean[1][r])
        assert torch.equal(rows.q[r], i8[1].q[r]) and rows.scale[r] == i8[1].scale[r]
    assert torch.isnan(u[1]).any() and torch.isnan(u[3]).all()
    assert torch.isnan(rows.scale[[1, 3]]).all() and not rows.q[[1, 3]].any()


def test_norm_of_zeros_and_large_values():
    z = torch.zeros(2, 300, device="cuda")
    h, u = plain.residual_norm(z, z, torch.ones(300, device="cuda"))
    assert not h.any() and not u.any()
    big = torch.full((2, 300), 1e4, dtype=torch.float16, device="cuda")  # squares pass float16
    h, u = plain.residual_norm(big, big, torch.ones(300, dtype=torch.float16, device="cuda"))
    assert (u == 1).all() and (h == 20000).all()


@pytest.mark.parametrize("T,D", [(1, 1), (3, 127), (4, 128), (2, 129), (5, 2048), (3, 5003), (2, 16384)])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_quantize_rows(T, D, ty):
    say(f"quantize_rows {T}x{D} {ty}")
    x = (rnd(T + D, T, D) * 3).to(TYPE[ty]).cuda()
    r = plain.quantize_rows(x)
    q, s = plain_ref.quantise(f64(x))
    assert np.array_equal(r.scale.cpu().numpy(), s)
    assert np.array_equal(r.q[:, :D].cpu().numpy(), q) and not r.q[:, D:].any()


def test_quantize_rows_special():
    x = torch.zeros(6, 200, device="cuda")
    x[1, 5], x[2, 7], x[3, :] = float("nan"), float("-inf"), 1e-44
    x[4, :] = torch.arange(200, device="cuda") - 63.5      # ties
    x[5, 0] = 127.0
    x[5, 1:] = torch.arange(199, device="cuda") / 2 - 49.5
    r = plain.quantize_rows(x)
    q, s = plain_ref.quantise(f64(x))
    assert np.array_equal(r.scale.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(r.q[:, :200].cpu().numpy(), q)


@pytest.mark.parametrize("T,D,ty,kind", [(4, 2048, "bf16", "rms"), (3, 1001, "f32", "layer"), (9, 500, "f16", "rms")])
def test_residual_norm_i8(T, D, ty, kind):
    """h as without it; a step of u's 8-bit form is s, so with half a step and u's own error:"""
    x, y, p = inputs(17, T, D, ty, True, kind == "layer", 0)
    h, rows = plain.residual_norm_i8(x, y, kind=kind, **p)
    h2, _ = plain.residual_norm(x, y, kind=kind, **p)
    assert torch.equal(h, h2)
    f = plain_ref.norm_forward(f64(x), f64(y), **ref_args(p), kind=kind, eps=float(np.float32(1e-6)))
    _, su = forward_sizes(f, f64(x), f64(y), ref_args(p), 1.0)
    s = f64(rows.scale)[:, None]
    assert (np.abs(s - top(f["u"]) / 127) <= 192 * EPS * su / 127 + EPS * s).all()
    err = np.abs(f64(rows.q[:, :D]) * s - f["u"])
    assert (err <= 0.5 * s * (1 + 4 * EPS * 127) + 256 * EPS * su).all()
    assert not rows.q[:, D:].any()


GRADS = [(1, 1, "f32", "rms", False, False, None), (3, 65, "f32", "layer", True, True, 0),
         (37, 1000, "f16", "layer", True, True, 1), (64, 512, "bf16", "rms", True, False, 4),
         (2100, 130, "f32", "rms", True, False, 3), (2050, 72, "bf16", "rms", False, True, 2050),
         (3000, 40, "f32", "layer", True, True, 1500), (5, 5003, "bf16", "rms", True, False, 1),
         (6, 8192, "bf16", "layer", True, True, 2), (3, 16384, "f32", "rms", True, True, 0),
         (1025, 2048, "bf16", "rms", True, False, 5)]


@pytest.mark.parametrize("T,D,ty,kind,block,bias,groups", GRADS)
@pytest.mark.parametrize("pad", [0, 3])
def test_residual_norm_grad(T, D, ty, kind, block, bias, groups, pad):
    say(f"residual_norm_grad {T}x{D} {ty} {kind} block={block} bias={bias} groups={groups} pad={pad}")
    x, y, p = inputs(T + D, T, D, ty, block, bias, groups, pad)
    dh, du = (wide(rnd(k, T, D), TYPE[ty], pad) for k in (21, 22))
    g = plain.residual_norm_grad(x, y, dh, du, scale=0.5, kind=kind, **p)
    ref, size = plain_ref.norm_grad(f64(x), f64(y), f64(dh), f64(du), **ref_args(p), scale=0.5, kind=kind,
                                    eps=float(np.float32(1e-6)))
    got = {k: v for k, v in g._asdict().items() if v is not None}
    assert set(got) == set(ref)
    close(g.dx, ref["dx"], size["dx"], 384, ty, "dx")
    close(g.dy, ref["dy"], size["dy"], 768, ty, "dy")
    depth = T // 512 + 128 + 384  # terms added in order, and what each is off
    for k in sorted(set(ref) - {"dx", "dy"}):
        assert got[k].dtype == torch.float32
        close(got[k], ref[k], size[k], depth, "f32", k)


def test_norm_grad_is_the_same_on_every_run():
    x, y, p = inputs(3, 3000, 640, "bf16", True, True, 2)
    dh, du = (rnd(k, 3000, 640).to(torch.bfloat16).cuda() for k in (1, 2))
    a = plain.residual_norm_grad(x, y, dh, du, kind="layer", **p)
    for _ in range(3):
        b = plain.residual_norm_grad(x, y, dh, du, kind="layer", **p)
        assert all(torch.equal(u, v) for u, v in zip(a, b))


def test_norm_grad_without_rows():
    x, p = torch.empty(0, 96, device="cuda"), {}
    for k in ("next_weight", "next_bias", "block_weight", "block_bias"):
        p[k] = torch.ones(96, device="cuda")
    torch.full((100000,), 7.0, device="cuda")  # what the allocator hands out next holds sevens
    g = plain.residual_norm_grad(x, x, x, x, gate=torch.ones(3, 96, device="cuda"), **p)
    for v in g[2:]:
        assert v is not None and not v.any()
    h, u = plain.residual_norm(x, x, p["next_weight"])
    assert h.shape == u.shape == (0, 96)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_grad_against_differences(kind):
    """Along random directions, against central differences of the 64-bit forward.  With step t the
    differences are off by t^2 times a third derivative (1e-8 of the sum of absolute terms with
    t = 1e-4) and by 2^-53 / t of the values; float32 gradients by 1e-5 of that sum."""
    T, D = 12, 96
    x, y, p = inputs(41, T, D, "f32", True, True, 3)
    dh, du = (rnd(k, T, D).float().cuda() for k in (51, 52))
    g = plain.residual_norm_grad(x, y, dh, du, scale=0.5, kind=kind, eps=1e-5, **p)
    base = {"x": f64(x), "y": f64(y), **ref_args(p)}
    mine = {"x": g.dx, "y": g.dy, "nw": g.next_weight, "nb": g.next_bias, "bw": g.block_weight, "bb": g.block_bias,
            "gate": g.gate}
    up_h, up_u = f64(dh), f64(du)

    def loss(v):
        f = plain_ref.norm_forward(**v, scale=0.5, kind=kind, eps=float(np.float32(1e-5)))
        return (f["h"] * up_h).sum() + (f["u"] * up_u).sum()

    for n, k in enumerate(base):
        d = np.random.default_rng(60 + n).standard_normal(base[k].shape)
        t = 1e-4
        slope = (loss({**base, k: base[k] + t * d}) - loss({**base, k: base[k] - t * d})) / (2 * t)
        want = (f64(mine[k]).reshape(d.shape) * d).sum()
        size = np.abs(f64(mine[k]).reshape(d.shape) * d).sum()
        assert abs(slope - want) <= 2e-5 * size, (k, slope, want, size)


def test_residual_norm_autograd():
    x, y, p = inputs(71, 8, 256, "bf16", True, False, 2)
    leaves = [t.detach().clone().requires_grad_() for t in (x, y, p["next_weight"], p["block_weight"], p["gate"])]
    h, u = plain.residual_norm(leaves[0], leaves[1], leaves[2], block_weight=leaves[3], gate=leaves[4], scale=0.5)
    dh, du = (rnd(k, 8, 256).to(torch.bfloat16).cuda() for k in (81, 82))
    torch.autograd.backward([h, u], [dh, du])
    g = plain.residual_norm_grad(x, y, dh, du, scale=0.5, **p)
    for leaf, want in zip(leaves, (g.dx, g.dy, g.next_weight, g.block_weight, g.gate)):
        assert torch.equal(leaf.grad, want.to(torch.bfloat16))


@pytest.mark.parametrize("outer", ["linear", "square"])
def test_residual_norm_has_first_derivatives_only(outer):
    """A second derivative through the norm raises, also next to a path that has one: its terms would be missing."""
    x, y, p = inputs(72, 4, 128, "f32", True, True, 0)
    leaf = x.detach().clone().requires_grad_()
    h, u = plain.residual_norm(leaf, y, kind="layer", **p)
    loss = u.sum() + h.sum() if outer == "linear" else (u * u).sum()
    g, = torch.autograd.grad(loss, leaf, create_graph=True)
    first = plain.residual_norm_grad(x, y, *((torch.ones_like(x),) * 2 if outer == "linear" else
                                             (torch.zeros_like(x), 2 * u.detach())), kind="layer", **p)
    assert torch.equal(g.detach(), first.dx)
    with pytest.raises(RuntimeError, match="no gradient"):
        ((g * g).sum() + (leaf ** 3).sum()).backward()
    g = plain.residual_norm_grad(leaf, y, x, x, kind="layer", **p)
    with pytest.raises(RuntimeError, match="no gradient"):
        g.next_bias.sum().backward()
    with torch.no_grad():
        assert not plain.residual_norm_grad(leaf, y, x, x, kind="layer", **p).dx.requires_grad


# ------------------------------------------------------------------ products

def i8(seed, rows, cols, full=False):
    r = np.random.default_rng(seed)
    q = r.integers(-128 if full else -127, 128, (rows, cols), dtype=np.int64).astype(np.int8)
    return q, (r.random(rows) + 0.5).astype(np.float32) / 100


def product_ref(qa, sa, qw, sw, bias):
    sums = (qa.astype(np.float64) @ qw.astype(np.float64).T)  # exact: below 2^53
    out = sums * sa.astype(np.float64)[:, None] * sw.astype(np.float64)[None]
    return out if bias is None else out + bias.astype(np.float64)


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 5003, 2048), (2, 64, 127), (3, 17, 129), (4, 1024, 640), (15, 100, 1000), (16, 256, 256),
    (17, 333, 4096), (31, 48, 8192), (32, 2048, 384), (33, 130, 1152), (63, 255, 65), (64, 512, 3000), (65, 64, 2051), (100, 700, 900),
    (127, 129, 130), (128, 128, 128), (129, 257, 1280), (200, 1000, 513), (256, 256, 2048), (257, 511, 700),
    (513, 300, 256), (700, 1029, 390), (1024, 1024, 512), (1100, 2100, 200)])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_matmul_i8(M, N, K, ty):
    say(f"matmul_i8 {M}x{N}x{K} {ty}")
    qa, sa = i8(M + N, M, K, True)
    qw, sw = i8(N + K, N, K, True)
    bias = np.random.default_rng(K).standard_normal(N).astype(np.float32) if (M + N) % 2 else None
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    out = plain.matmul_i8(plain.Int8Rows(dev(qa), dev(sa)), plain.Int8Rows(dev(qw), dev(sw)),
                          None if bias is None else dev(bias), TYPE[ty])
    assert out.shape == (M, N) and out.dtype == TYPE[ty]
    ref = product_ref(qa, sa, qw, sw, bias)
    # the sum, the two scales, the product and the bias each round once
    size = np.abs(ref if bias is None else ref - bias) + (0 if bias is None else np.abs(bias))
    close(out, ref, size, 4, ty, "out")


def test_matmul_i8_largest_sums():
    """131071 products of (-128)^2: just inside 32 bits."""
    K = 131071
    a = torch.full((3, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((5, K), -128, dtype=torch.int8, device="cuda")
    w[1] = 127
    one = lambda n: torch.ones(n, device="cuda")  # noqa: E731
    out = plain.matmul_i8(plain.Int8Rows(a, one(3)), plain.Int8Rows(w, one(5)), dtype=torch.float32)
    want = torch.full((3, 5), float(np.float32(K * 16384)), device="cuda")
    want[:, 1] = float(np.float32(-K * 128 * 127))
    assert torch.equal(out, want)


def test_matmul_i8_layouts():
    """Rows of a wider buffer are taken in place, any other layout is copied; an output row is not
    written past its channels; infinite scales stay in their row."""
    qa, sa = i8(1, 20, 300)
    qw, sw = i8(2, 50, 300)
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    buf = torch.zeros(50, 640, dtype=torch.int8, device="cuda")
    buf[:, :300] = dev(qw)
    w = plain.Int8Rows(buf, dev(sw), 300)
    assert w.q.data_ptr() == buf.data_ptr()
    t = plain.Int8Rows(dev(np.ascontiguousarray(qa.T)).t(), dev(sa))
    out = plain.matmul_i8(t, w, dtype=torch.float32)
    ref = product_ref(qa, sa, qw, sw, None)
    close(out, ref, np.abs(ref), 4, "f32", "out")
    s = dev(sa)
    s[3], s[4] = float("nan"), float("inf")
    bad = plain.matmul_i8(plain.Int8Rows(t.q, s, 300), w, dtype=torch.float32)
    assert torch.isnan(bad[3]).all() and not torch.isfinite(bad[4]).any()
    keep = [r for r in range(20) if r not in (3, 4)]
    assert torch.equal(bad[keep], out[keep])
    assert plain.matmul_i8(plain.Int8Rows(t.q[:0], s[:0], 300), w).shape == (0, 50)


def test_int8_rows_of_any_stride():
    """Rows that lie over each other (a row repeated), and a single row whose stride says nothing."""
    qa, sa = i8(31, 1, 300)
    qw, sw = i8(32, 40, 300)
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    w = plain.Int8Rows(dev(qw), dev(sw))
    ref = product_ref(qa, sa, qw, sw, None)
    buf = torch.zeros(1024, dtype=torch.int8, device="cuda")
    buf[:300] = dev(qa)[0]
    for rows, width, stride in ((5, 384, 0), (5, 400, 0), (1, 400, 0), (1, 384, 128), (1, 400, 128), (1, 400, 384), (1, 400, 7)):
        a = plain.Int8Rows(buf.as_strided((rows, width), (stride, 1)), dev(np.repeat(sa, rows)), 300)
        for out in (plain.matmul_i8(a, w, dtype=torch.float32), plain.matmul_i8(w, a, dtype=torch.float32).t()):
            close(out, np.repeat(ref, rows, 0), np.repeat(np.abs(ref), rows, 0), 4, "f32", f"{rows} x {width} by {stride}")


@pytest.mark.parametrize("M,N,K", [(3, 70, 300), (40, 70, 129), (300, 200, 1)])
def test_product_of_rows_with_something_behind_the_columns(M, N, K):
    qa, sa = i8(41, M, K)
    qw, sw = i8(42, N, K)
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    ref = product_ref(qa, sa, qw, sw, None)
    wide = [torch.full((n, 512), 77, dtype=torch.int8, device="cuda") for n in (M, N)]
    for buf, q in zip(wide, (qa, qw)):
        buf[:, :K] = dev(q)
    a, w = plain.Int8Rows(wide[0], dev(sa), K), plain.Int8Rows(wide[1], dev(sw), K)
    assert a.q.data_ptr() == wide[0].data_ptr() and w.q.data_ptr() == wide[1].data_ptr()
    clean = plain.Int8Rows(dev(qa), dev(sa)), plain.Int8Rows(dev(qw), dev(sw))
    for one, other in ((a, w), (a, clean[1]), (clean[0], w)):
        close(plain.matmul_i8(one, other, dtype=torch.float32), ref, np.abs(ref), 4, "f32", "out")
    x = rnd(43, M, K).cuda().float()
    assert torch.equal(plain.linear_i8(x, w), plain.linear_i8(x, clean[1]))


def test_matmul_i8_offsets_past_32_bits():
    """Weights of 2.3 GB and an output of 4.4 GB: the last rows, and the last token's channels."""
    N, K = 1 << 16, 35000
    w = torch.zeros((N, 35072), dtype=torch.int8, device="cuda")
    w[-5:, :K] = torch.from_numpy(i8(5, 5, K)[0]).cuda()
    qa, sa = i8(6, 3, K)
    sw = torch.ones(N, device="cuda")
    out = plain.matmul_i8(plain.Int8Rows(torch.from_numpy(qa).cuda(), torch.from_numpy(sa).cuda()),
                          plain.Int8Rows(w, sw, K), dtype=torch.float32)
    ref = product_ref(qa, sa, w[-5:, :K].cpu().numpy(), np.ones(5, np.float32), None)
    close(out[:, -5:], ref, np.abs(ref), 4, "f32", "out")
    assert not out[:, :-5].any()
    del w, out
    M, N, K = 33000, 33280, 128
    qa, sa = i8(7, 64, K)
    qw, sw = i8(8, N, K)
    a = torch.zeros((M, K), dtype=torch.int8, device="cuda")
    a[-64:] = torch.from_numpy(qa).cuda()
    s = torch.ones(M, device="cuda")
    s[-64:] = torch.from_numpy(sa).cuda()
    out = plain.matmul_i8(plain.Int8Rows(a, s), plain.Int8Rows(torch.from_numpy(qw).cuda(), torch.from_numpy(sw).cuda()),
                          dtype=torch.float32)
    ref = product_ref(qa, sa, qw, sw, None)
    close(out[-64:], ref, np.abs(ref), 4, "f32", "out")
    assert not out[:1000].any()


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_i8_is_quantise_and_product(M):
    x = rnd(M, M, 1500).to(torch.bfloat16).cuda()
    qw, sw = i8(4, 600, 1500)
    w = plain.Int8Rows(torch.from_numpy(qw).cuda(), torch.from_numpy(sw).cuda())
    out = plain.linear_i8(x, w)
    assert out.dtype == torch.bfloat16
    assert torch.equal(out, plain.matmul_i8(plain.quantize_rows(x), w))
    q, s = plain_ref.quantise(f64(x))
    ref = product_ref(q, s, qw, sw, None)
    close(out, ref, np.abs(ref), 4, "bf16", "out")


# ------------------------------------------------------------------ sampling

def noise(seed, *shape):
    u = np.random.default_rng(seed).random(shape)
    return torch.from_numpy(-np.log(-np.log(u * 0.999999 + 5e-7))).float().cuda()


def check_sample(z, g, t, k=None, p=None, m=None, allowed=None):
    """Tokens equal; logprob within 2^-22 of one and the values it is made of (a difference, a quotient, an
    exponential and a logarithm of a few roundings each)."""
    token, logprob = plain.sample(z, g, t, k, p, m, allowed)
    host = lambda v: None if v is None else v.cpu().float().numpy()  # noqa: E731
    rt, rl = plain_ref.sample(z.float().cpu().numpy(), g.cpu().numpy(), host(t), host(k), host(p), host(m),
                              None if allowed is None else allowed.cpu().numpy())
    assert token.dtype == torch.int64 and logprob.dtype == torch.float32
    assert np.array_equal(token.cpu().numpy(), rt)
    got = f64(logprob)
    fine = np.isfinite(rl)
    assert np.array_equal(got[~fine], rl[~fine])
    off = np.abs(got[fine] - rl[fine])
    assert (off <= 2.0 ** -22 * (2 + 2 * np.abs(rl[fine]))).all(), off.max()
    return token


def full(B, v, dtype=torch.float32):
    return torch.full((B,), v, dtype=dtype, device="cuda")


@pytest.mark.parametrize("B,V", [(1, 1), (2, 2), (5, 63), (3, 64), (4, 257), (7, 1000), (2, 4096), (3, 5003), (1, 32768),
                                 (9, 50021), (2, 131073), (300, 128)])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k,p,m", [(0, 1.0, 0.0), (1, 1.0, 0.0), (50, 0.95, 0.0), (0, 0.9, 0.0), (0, 1.0, 0.05),
                                   (1000, 0.99, 0.001)])
def test_sample(B, V, ty, k, p, m):
    say(f"sample {B}x{V} {ty} top_k={k} top_p={p} min_p={m}")
    z = (rnd(B + V, B, V) * 2.5).to(TYPE[ty]).cuda()
    t = torch.from_numpy(np.random.default_rng(V).uniform(0.5, 1.5, B)).float().cuda()
    t[B // 2::5] = 0
    check_sample(z, noise(V, B, V), t, full(B, k, torch.int32), full(B, p), full(B, m))


def test_sample_optional_filters():
    z, g, t = (rnd(1, 4, 999) * 2).cuda().float(), noise(2, 4, 999), full(4, 1.0)
    a = check_sample(z, g, t)
    assert torch.equal(a, check_sample(z, g, t, full(4, 0, torch.int32), full(4, 1.0), full(4, 0.0)))
    assert torch.equal(a, check_sample(z, g, t, full(4, -3, torch.int32), full(4, 2.0), full(4, -1.0)))
    assert torch.equal(a, check_sample(z, g, t, full(4, 5000, torch.int32)))


@pytest.mark.parametrize("levels", [1, 2, 7])
@pytest.mark.parametrize("V", [100, 3000, 40000])
def test_sample_ties(levels, V):
    """Equal logits: the order goes by index, through the middle of a run of equals."""
    r = np.random.default_rng(levels)
    z = torch.from_numpy(r.integers(0, levels, (12, V)).astype(np.float32)).cuda()
    z[5] = -z[5]          # zeros of both signs are equal
    z[6, ::2] *= -0.0 if levels == 1 else 1.0
    k = torch.tensor([1, 2, 3, 10, 63, 64, 65, 99, V - 1, V, 0, 7], dtype=torch.int32, device="cuda")
    p = torch.tensor([1, 1, .5, .7, .9, .31, 1, .77, .999, .1, .25, .013], device="cuda")
    check_sample(z, noise(V, 12, V), full(12, 0.9), k, p)
    check_sample(z, torch.zeros(12, V, device="cuda"), full(12, 0.9), k, p)  # equal scores as well
    check_sample(z, noise(V + 1, 12, V), full(12, 0.0), k, p)


@pytest.mark.parametrize("n", [4095, 4096, 4097])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V,k,t", [(0, 0, 1.0), (0, 0, 1e9), (5000, 4500, 1.0), (5000, 4999, 1.0), (60000, 0, 1.0)])
def test_sample_as_many_equals_as_a_list_holds(n, ty, V, k, t):
    """n tokens that all weigh one: the whole row (V = 0), the allowed ones of V, or the top of V with a tail.  Row
    by row all the noise is on one token around the end of the nucleus, then it is spread."""
    say(f"sample {n} equals of {V} {ty} top_k={k} T={t}")
    B, width, r = 8, max(V, n), np.random.default_rng(n + V)
    z = np.full((B, width), -9.0) if V == 60000 else np.zeros((B, width))
    ids = np.sort(r.permutation(width)[:n])
    z[:, ids] = 0
    if t > 1:
        z = z + r.standard_normal((B, width))  # nearly flat at that temperature: each weighs one in 32 bits
    allowed = torch.zeros(B, width, dtype=torch.bool, device="cuda")
    allowed[:, torch.from_numpy(ids).cuda()] = True
    z = torch.from_numpy(z).to(TYPE[ty]).cuda()
    g = noise(n, B, width)
    p = np.float32([0.5, 0.5, 0.3, 0.3, 0.9, 0.9, 0.7, 0.999])
    mass = n + (width - n) * np.exp(-9.0) * (V == 60000)
    possible = z.masked_fill(~allowed, -np.inf) if V == 5000 else z
    ranked = np.argsort(-possible.float().cpu().numpy(), axis=1, kind="stable")
    for row, d in ((0, 0), (1, -1), (2, 1), (3, -2), (4, 1), (5, -1)):
        g[row, ranked[row, int(np.ceil(p[row].astype(np.float64) * mass)) + d]] = 50.0
    check_sample(z, g, full(B, t), full(B, k, torch.int32) if k else None, torch.from_numpy(p).cuda(), None,
                 allowed if V == 5000 else None)


@pytest.mark.parametrize("V", [5000, 20011, 70000])
@pytest.mark.parametrize("k,p", [(50, 1.0), (4500, 1.0), (4999, 0.9), (0, 0.5), (0, 0.9999), (3000, 0.8)])
def test_sample_shapes_of_distributions(V, k, p):
    """Long and flat, peaked, with outliers and infinities: the kept tokens are more than fit any list,
    or crowd into a sliver of the range."""
    r = np.random.default_rng(V + k)
    z = np.stack([
        r.standard_normal(V) * 0.01,                       # all alike
        r.standard_normal(V) * 12,                         # peaked
        np.where(np.arange(V) == 77, 1e30, r.standard_normal(V)),   # one far above
        np.where(np.arange(V) % 2 == 0, np.inf, r.standard_normal(V)),
        np.where(np.arange(V) < 3, np.inf, -np.inf),
        1.0 + r.integers(0, 40, V) * 2.0 ** -23,           # neighbouring numbers
        -np.exp(r.uniform(-60, 60, V)),                    # many octaves below zero
        r.choice([-3e38, 0.0, 3e38], V),
        np.where(r.random(V) < 0.9, -1e4, r.standard_normal(V)),    # a long flat tail
        np.round(r.standard_normal(V) * 4) / 4,            # runs of equals
    ])
    z = torch.from_numpy(z).float().cuda()
    B = z.shape[0]
    check_sample(z, noise(V, B, V), full(B, 0.8), full(B, k, torch.int32), full(B, p))


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("p,m,t", [(0.95, 0.0, 0.8), (0.95, 0.001, 1.3), (0.999, 0.0, 30.0), (0.5, 0.0, 1.0),
                                   (0.9, 0.0, 1e-30), (0.9, 0.0, 1e32)])
def test_sample_large_nuclei(ty, p, m, t):
    """Nuclei of many thousands of tokens, at the ends of the temperature's range too; half of what
    min_p is tested with is masked."""
    V = 40003
    say(f"sample nucleus {ty} top_p={p} min_p={m} T={t}")
    spread = t if ty != "f16" and t in (1e-30, 1e32) else 2.5
    z = rnd(V, 3, V) * spread
    z[1] -= 20 * spread
    allowed = torch.from_numpy(np.random.default_rng(V).random((3, V)) < 0.5).cuda() if m else None
    check_sample(z.to(TYPE[ty]).cuda(), noise(V + 3, 3, V), full(3, t), None, full(3, p), full(3, m) if m else None, allowed)


def test_sample_nucleus_that_ends_where_two_threads_bins_meet():
    """A large nucleus is counted in bins, some for each thread, and the running sums on both sides of a thread's
    border round apart.  Rows (seed, index of its top_p) whose nucleus ends within such a difference; all the noise
    is on the fourth token before the end."""
    V = 40003
    pairs = [(19, 1957), (20, 1737), (40, 677), (56, 239), (56, 1810), (94, 1260), (109, 779), (141, 1417), (151, 640),
             (170, 287), (176, 1592), (207, 1745), (229, 1636), (247, 1307), (260, 314), (274, 1734), (291, 246),
             (299, 2011), (315, 868), (327, 1743), (329, 750), (337, 1166), (339, 269), (375, 1774), (383, 531),
             (387, 1259), (391, 533)]
    z, p = np.empty((len(pairs), V), np.float32), np.empty(len(pairs), np.float32)
    g = torch.zeros(len(pairs), V)
    for row, (seed, at) in enumerate(pairs):
        r = np.random.default_rng(seed)
        z[row] = (r.standard_normal(V) * 2.5).astype(np.float32)
        p[row] = r.uniform(0.6, 0.99, 2048).astype(np.float32)[at]
        order = np.argsort(-z[row], kind="stable")
        e = np.exp(z[row][order].astype(np.float64) - np.float64(z[row].max()))
        before = np.cumsum(e) - e
        g[row, order[np.searchsorted(before, np.float64(p[row]) * e.sum()) - 4]] = 50.0
    B = len(pairs)
    check_sample(torch.from_numpy(z).cuda(), g.cuda(), full(B, 1.0), None, torch.from_numpy(p).cuda())


@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_sample_masks(ty):
    B, V = 16, 3001
    r = np.random.default_rng(3)
    z = (rnd(4, B, V) * 3).to(TYPE[ty]).cuda()
    allowed = torch.from_numpy(r.random((B, V)) < 0.2).cuda()
    allowed[2] = False
    allowed[3] = False
    allowed[3, 3000] = True
    allowed[4] = False
    allowed[4, 0] = True
    z[5][~allowed[5]] = float("nan")      # what is masked may hold anything
    z[6][~allowed[6]] = float("inf")
    z[7] = float("-inf")                  # nothing possible
    z[8, 100:] = float("nan")
    z[9, 7] = float("inf")
    allowed[9, 7] = True
    z[10, ::3] = float("inf")
    z[11] = float("-inf")
    z[11, 17], allowed[11, 17] = -5.0, True
    z[12][~allowed[12]] = torch.finfo(TYPE[ty]).max
    z[13] = torch.finfo(TYPE[ty]).min     # the lowest value is a value
    z[14] = torch.finfo(TYPE[ty]).min
    z[14, 5] = torch.finfo(TYPE[ty]).max
    t = full(B, 0.8)
    for k, p, m in [(0, 1.0, 0.0), (5, 1.0, 0.0), (0, 0.6, 0.0), (0, 1.0, 0.3), (40, 0.9, 0.01), (1, 0.0, 2.0)]:
        token = check_sample(z, noise(9, B, V), t, full(B, k, torch.int32), full(B, p), full(B, m), allowed)
        assert token[2] == -1 and token[7] == -1 and token[3] == 3000 and token[4] == 0 and token[11] == 17
        check_sample(z, noise(8, B, V), t, full(B, k, torch.int32), full(B, p), full(B, m))


def test_sample_extreme_parameters():
    B, V = 12, 700
    z = (rnd(6, B, V) * 3).float().cuda()
    t = torch.tensor([0.0, -1.0, float("nan"), 1e-30, 1e-45, 1e30, float("inf"), 1, 1, 1, 1, 1], device="cuda")
    p = torch.tensor([.5] * 7 + [0.0, -1.0, float("nan"), 1e-30, 1 - 2.0 ** -24], device="cuda")
    m = torch.tensor([.1] * 7 + [0, 0, 0, float("nan"), 1.0], device="cuda")
    token, logprob = plain.sample(z, noise(7, B, V), t, full(B, 0, torch.int32), p, m)
    first = z.argmax(1)
    assert torch.equal(token[[0, 1, 2, 3, 4, 7, 8, 10, 11]], first[[0, 1, 2, 3, 4, 7, 8, 10, 11]])
    assert torch.isfinite(logprob).all() and ((token >= 0) & (token < V)).all()
    assert abs(float(logprob[6]) + np.log(V)) < 1e-5   # every token alike


def test_sample_layouts():
    B, V = 6, 2000
    for ty in ("bf16", "f16", "f32"):
        for pad, offset in ((0, 0), (8, 8), (5, 3)):
            z, g = wide(rnd(1, B, V) * 2, TYPE[ty], pad, offset), wide(noise(2, B, V), torch.float32, pad, offset)
            mask = torch.zeros(B, V + pad, dtype=torch.bool, device="cuda")
            mask[:, offset:offset + V] = torch.from_numpy(np.random.default_rng(4).random((B, V)) < 0.5).cuda()
            check_sample(z, g, full(B, 1.0), full(B, 30, torch.int32), full(B, 0.9), None, mask[:, offset:offset + V])


def test_sample_offsets_past_32_bits():
    """Rows more than 2^32 bytes apart."""
    buf = torch.zeros(3 * (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (4, 1000), (1 << 30, 1))
    z.copy_((rnd(5, 4, 1000) * 2).to(torch.bfloat16))
    check_sample(z, noise(3, 4, 1000), full(4, 0.7), full(4, 20, torch.int32), full(4, 0.8))


def test_sample_follows_the_distribution():
    """40000 draws of 5 tokens: a count is within 5 standard deviations of its mean."""
    n = 40000
    z = torch.tensor([[1.0, 0.5, 0.0, -1.0, 2.0]], device="cuda").expand(n, 5).contiguous()
    g = noise(77, n, 5)
    token, _ = plain.sample(z, g, full(n, 0.7), full(n, 4, torch.int32))
    e = np.exp(np.array([1.0, 0.5, 0.0, -np.inf, 2.0]) / np.float32(0.7))
    p = e / e.sum()
    got = np.bincount(token.cpu().numpy(), minlength=5)
    assert (np.abs(got - n * p) <= 5 * np.sqrt(n * p * (1 - p)) + 1e-9).all(), (got, n * p)


# ------------------------------------------------------------------ more rows than a grid has threads for

@pytest.fixture
def memory_back():
    yield
    torch.cuda.empty_cache()


def same_in_parts(call, rows, border):
    """call(slice) of all rows against calls of the rows around `border` and at both ends, bit for bit."""
    whole = call(slice(0, rows))
    for at in (slice(0, 1000), slice(border - 500, border + 500), slice(rows - 1000, rows)):
        for a, b in zip(whole, call(at)):
            assert torch.equal(a[at], b)


def test_sample_of_millions_of_rows(memory_back):
    B, V = (1 << 22) + 37, 3
    z, g = torch.randn(B, V, device="cuda"), torch.rand(B, V, device="cuda")
    t, k, p, m = torch.rand(B, device="cuda"), full(B, 2, torch.int32), torch.rand(B, device="cuda"), full(B, 0.1)
    allowed = torch.rand(B, V, device="cuda") < 0.7
    same_in_parts(lambda r: plain.sample(z[r], g[r], t[r], k[r], p[r], m[r], allowed[r]), B, 1 << 21)
    same_in_parts(lambda r: plain.sample(z[r], g[r], t[r]), B, 1 << 22)


def test_norms_of_millions_of_rows(memory_back):
    T, D, border = (1 << 26) + 37, 2, 1 << 25
    x, y, gate = (torch.randn(T, D, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    w = torch.ones(D, device="cuda", dtype=torch.bfloat16)
    rows = lambda r: (r.q, r.scale)  # noqa: E731
    same_in_parts(lambda r: plain.residual_norm(x[r], y[r], w, gate=gate[r]), T, border)
    same_in_parts(lambda r: rows(plain.quantize_rows(x[r])), T, border)
    same_in_parts(lambda r: rows(plain.residual_norm_i8(x[r], y[r], w, gate=gate[r])[1]), T, border)


def test_product_of_a_billion_channels(memory_back):
    """One token; 137 GB of weights, all zero but the last."""
    N = 1 << 30
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GiB free")
    w, s = torch.zeros((N, 128), dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
    q, _ = i8(100, 1000, 128)
    w[-1000:] = torch.from_numpy(q).cuda()
    a, sa = i8(101, 1, 128)
    out = plain.matmul_i8(plain.Int8Rows(torch.from_numpy(a).cuda(), torch.from_numpy(sa).cuda()), plain.Int8Rows(w, s))
    ref = product_ref(a, sa, q, np.ones(1000, np.float32), None)
    close(out[:, -1000:], ref, np.abs(ref), 4, "bf16", "out")
    assert not out[:, :-1000].any()


# ------------------------------------------------------------------ use

def test_results_without_a_gradient_say_so():
    """Where autograd follows an operand the values are the same, and a derivative through them raises; elsewhere
    nothing is attached."""
    x, y, p = inputs(95, 4, 256, "f32", True, False, 0)
    q, s = i8(96, 300, 256)
    w = plain.Int8Rows(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    g = noise(97, 4, 300)

    def results(x, nw, bias, temperature):
        h, rows = plain.residual_norm_i8(x, y, **{**p, "next_weight": nw})
        direct = plain.quantize_rows(x)
        logits = plain.matmul_i8(rows, w, bias, torch.float32)
        line = plain.linear_i8(x, w)
        token, logprob = plain.sample(logits, g, temperature)
        floats = {"residual_norm_i8": h, "residual_norm_i8 ": rows.scale, "quantize_rows": direct.dequantize(),
                  "matmul_i8": logits, "linear_i8": line, "sample": logprob}
        return floats, [rows.q, direct.q, token]

    operands = (x, p["next_weight"], torch.ones(300, device="cuda"), full(4, 0.9))
    want, whole = results(*operands)
    assert not any(v.requires_grad for v in want.values())
    for followed in range(4):
        leaves = [v.clone().requires_grad_(i == followed) for i, v in enumerate(operands)]
        with torch.no_grad():
            got, _ = results(*leaves)
            assert not any(v.requires_grad for v in got.values())
        got, ints = results(*leaves)
        assert all(torch.equal(a, b) and not a.requires_grad for a, b in zip(ints, whole))
        reached = {0: want, 1: ["residual_norm_i8", "residual_norm_i8 ", "matmul_i8", "sample"], 2: ["matmul_i8", "sample"],
                   3: ["sample"]}[followed]
        for name, v in got.items():
            assert torch.equal(v.detach(), want[name]) and v.requires_grad == (name in reached), (name, followed)
            if v.requires_grad:
                with pytest.raises(RuntimeError, match=f"{name.strip()} has no gradient"):
                    v.sum().backward()


def test_forward_mode_is_refused():
    """A tangent would be lost; next to none in the same level the values are as ever, under no_grad too."""
    from torch.autograd import forward_ad
    x, y, p = inputs(98, 4, 256, "f32", True, False, 0)
    q, s = i8(99, 300, 256)
    w = plain.Int8Rows(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda())
    g, t = noise(97, 4, 256), full(4, 0.9)
    calls = [lambda v: plain.residual_norm(v, y, **p)[1], lambda v: plain.residual_norm_i8(v, y, **p)[0],
             lambda v: plain.residual_norm_grad(v, y, x, x, **p).dx, lambda v: plain.residual_norm(x, y, **{**p, "next_weight": v[0]})[1],
             lambda v: plain.quantize_rows(v).scale, lambda v: plain.linear_i8(v, w), lambda v: plain.sample(v, g, t)[1],
             lambda v: plain.matmul_i8(plain.Int8Rows(w.q[:4], v[:, 0].contiguous(), 256), w)]
    want = [f(x) for f in calls]
    with forward_ad.dual_level():
        dual = forward_ad.make_dual(x, torch.ones_like(x))
        for f, v in zip(calls, want):
            assert torch.equal(f(x), v)
            with pytest.raises((RuntimeError, NotImplementedError), match="forward"):
                f(dual)
            with torch.no_grad(), pytest.raises((RuntimeError, NotImplementedError), match="forward"):
                f(dual)
    assert all(torch.equal(f(x), v) for f, v in zip(calls, want))


def test_on_another_stream_and_in_a_graph():
    x, y, p = inputs(90, 4, 2048, "bf16", True, False, 0)
    qw, sw = i8(91, 4096, 2048)
    w = plain.Int8Rows(torch.from_numpy(qw).cuda(), torch.from_numpy(sw).cuda())
    g, t, k, pp = noise(92, 4, 4096), full(4, 0.8), full(4, 40, torch.int32), full(4, 0.9)

    def step():
        h, rows = plain.residual_norm_i8(x, y, **p)
        logits = plain.matmul_i8(rows, w, dtype=torch.float32)
        return (h, logits) + plain.sample(logits, g, t, k, pp)

    want = [v.clone() for v in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = step()
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for n in range(4):
        y.mul_(1.5)
        want = [v.clone() for v in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), n


def test_binding_refusals():
    x = torch.zeros(4, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    for bad, what in [(lambda: plain.residual_norm(x, x[:, :32], w), "y"), (lambda: plain.residual_norm(x, x, w[:32]), "next_weight"),
                      (lambda: plain.residual_norm(x, x.half(), w), "y"), (lambda: plain.residual_norm(x.t(), x.t(), w), "x"),
                      (lambda: plain.residual_norm(x, x, w, gate=torch.ones(3, 64, device="cuda")), "gate"),
                      (lambda: plain.residual_norm(x, x, w, kind="group"), "kind"),
                      (lambda: plain.residual_norm(x.double(), x.double(), w.double()), "x"),
                      (lambda: plain.quantize_rows(x[0]), "x"),
                      (lambda: plain.Int8Rows(torch.zeros(4, 64, dtype=torch.int8, device="cuda"), w), "scale"),
                      (lambda: plain.linear_i8(x, plain.quantize_rows(x), dtype=torch.float64), "dtype"),
                      (lambda: plain.linear_i8(x, plain.quantize_rows(x[:, :32])), "columns"),
                      (lambda: plain.sample(x, x, w), "temperature"),
                      (lambda: plain.sample(x, x, w[:4], allowed=x), "allowed"),
                      (lambda: plain.sample(x, x, w[:4], top_k=w[:4]), "top_k")]:
        with pytest.raises(ValueError, match=what):
            bad()


def test_binding_refuses_what_is_no_tensor():
    x, w = torch.zeros(4, 64, device="cuda"), torch.ones(64, device="cuda")
    rows = plain.quantize_rows(x)
    for bad, what in [(lambda: plain.residual_norm([1.0], x, w), "x"), (lambda: plain.residual_norm(x, 1.0, w), "y"),
                      (lambda: plain.residual_norm(x, x, [1.0] * 64), "next_weight"),
                      (lambda: plain.residual_norm(x, x, w, gate=[1.0] * 64), "gate"),
                      (lambda: plain.residual_norm_i8(x, x, w, gate=0.5), "gate"),
                      (lambda: plain.residual_norm_grad(x, x, None, x, w), "dh"),
                      (lambda: plain.quantize_rows([1.0]), "x"), (lambda: plain.linear_i8(None, rows), "x"),
                      (lambda: plain.matmul_i8(rows, x), "w"), (lambda: plain.matmul_i8(rows, rows, bias=[0.0] * 4), "bias"),
                      (lambda: plain.sample(None, x, w), "logits"), (lambda: plain.sample(x, None, w), "gumbel"),
                      (lambda: plain.sample(x, x, [1.0] * 4), "temperature")]:
        with pytest.raises(ValueError, match=what):
            bad()
