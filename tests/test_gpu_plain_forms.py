"""Every form of the plaintext-side kernels that the dispatch picks, at sizes
that pick it (test_gpu_plain has the small ones): rows of each number of waves
with 16 elements a thread, gradients with several rows a workgroup, each tile
of the 8-bit product with more steps than its ring holds; outputs as rows of a
wider buffer, of which nothing else may be written.

Large results are compared in part: all of the sampled rows and of the sampled
columns, first and last among them.  Bounds as in test_gpu_plain."""
import ctypes as C

import numpy as np
import pytest

import plain_ref
from gpu_util import require_gpu, say, torch
from rns_ckks_polynomial_amd import _native as nat
from rns_ckks_polynomial_amd import plain
from test_gpu_plain import EPS, TYPE, check_sample, close, f64, forward_sizes, full, i8, inputs, noise, product_ref, ref_args, rnd, top, wide

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def some(n, count, seed):
    """Sorted indexes below n: the ends, and `count` others."""
    ends = [i for i in (0, 1, n // 2, n - 2, n - 1) if 0 <= i < n]
    return np.unique(np.concatenate([ends, np.random.default_rng(seed).integers(0, n, count)]))


# ------------------------------------------------------------------ norms, more than 1024 rows

# one wave (four rows a workgroup), 2, 4, 8, 12 and 16 waves; rows no multiple of four
WIDE = [(1031, 7), (1026, 515), (1025, 1024), (1027, 1029), (1026, 2048), (1029, 3001), (1025, 4096), (1025, 5003), (1026, 8192),
        (1025, 9001), (1027, 12288), (1025, 12301), (1026, 16384)]


def rows_of(x, y, p, rows, groups):
    """References' operands of the sampled rows: a gate's row for each."""
    a = ref_args(p)
    T = x.shape[0]
    if groups:
        a["gate"] = a["gate"].reshape(groups, -1)[rows // (T // groups)]
    at = torch.from_numpy(rows).cuda()
    return f64(x[at]), f64(y[at]), a


@pytest.mark.parametrize("T,D", WIDE)
@pytest.mark.parametrize("ty,kind,block,bias,per_token", [("bf16", "rms", True, False, False), ("f32", "layer", True, True, True),
                                                          ("f16", "layer", False, True, False)])
def test_norms_of_many_rows(T, D, ty, kind, block, bias, per_token):
    say(f"norms {T}x{D} {ty} {kind}")
    groups = T if per_token else 1
    x, y, p = inputs(T + D, T, D, ty, block, bias, groups, pad=5 if per_token else 0)
    h, u = plain.residual_norm(x, y, kind=kind, scale=0.5, **p)
    h8, rows = plain.residual_norm_i8(x, y, kind=kind, scale=0.5, **p)
    assert torch.equal(h, h8)
    r = some(T, 60, D)
    at = torch.from_numpy(r).cuda()
    rx, ry, a = rows_of(x, y, p, r, groups)
    f = plain_ref.norm_forward(rx, ry, **a, scale=0.5, kind=kind, eps=float(np.float32(1e-6)))
    sh, su = forward_sizes(f, rx, ry, a, 0.5)
    close(h[at], f["h"], sh, 64, ty, "h")
    close(u[at], f["u"], su, 192, ty, "u")
    s = f64(rows.scale[at])[:, None]
    assert (np.abs(s - top(f["u"]) / 127) <= 192 * EPS * su / 127 + EPS * s).all()
    err = np.abs(f64(rows.q[at, :D]) * s - f["u"])
    assert (err <= 0.5 * s * (1 + 4 * EPS * 127) + 256 * EPS * su).all()
    assert not rows.q[:, D:].any()


@pytest.mark.parametrize("T,D", WIDE)
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_quantize_many_rows(T, D, ty):
    x = wide(rnd(T + D, T, D) * 3, TYPE[ty], 3 if ty == "f16" else 0)
    x[5], x[7, D - 1], x[9, 0] = 0, float("nan"), float("inf")
    r = plain.quantize_rows(x)
    q, s = plain_ref.quantise(f64(x))
    assert np.array_equal(r.scale.cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(r.q[:, :D].cpu().numpy(), q) and not r.q[:, D:].any()


# ------------------------------------------------------------------ gradients, several rows a workgroup

GRADS = [(9000, 100, "bf16", "layer", True, True, 1), (6100, 700, "f16", "rms", True, False, 4),
         (3100, 1500, "bf16", "layer", True, True, 2), (2600, 1500, "f32", "rms", False, False, None),
         (1700, 2500, "bf16", "layer", True, True, 1), (1700, 4096, "f32", "layer", True, True, 2),
         (1530, 3001, "f16", "rms", True, False, 1), (1100, 4096, "f32", "rms", True, False, 0),
         (1024, 5000, "bf16", "layer", True, True, 1), (900, 6144, "f32", "layer", False, True, None),
         (1000, 6001, "bf16", "rms", True, False, 5), (777, 4500, "f32", "rms", True, False, 1),
         (900, 8192, "bf16", "layer", True, True, 1), (700, 7001, "f32", "layer", True, True, 700),
         (900, 8192, "f16", "rms", True, False, 1), (700, 7001, "f32", "rms", True, False, 2),
         (600, 9001, "bf16", "layer", True, True, 1), (600, 16384, "bf16", "rms", True, False, 1),
         (520, 12301, "f32", "layer", True, True, 2), (520, 12301, "f16", "rms", False, False, 1)]


@pytest.mark.parametrize("T,D,ty,kind,block,bias,groups", GRADS)
def test_gradients_of_several_rows_a_workgroup(T, D, ty, kind, block, bias, groups):
    say(f"gradient {T}x{D} {ty} {kind} block={block} bias={bias} groups={groups}")
    pad = 3 if T % 3 == 0 else 0
    x, y, p = inputs(T + D, T, D, ty, block, bias, groups, pad)
    dh, du = (wide(rnd(k, T, D), TYPE[ty], pad) for k in (21, 22))
    g = plain.residual_norm_grad(x, y, dh, du, scale=0.5, kind=kind, **p)
    ref, size = plain_ref.norm_grad(f64(x), f64(y), f64(dh), f64(du), **ref_args(p), scale=0.5, kind=kind,
                                    eps=float(np.float32(1e-6)))
    got = {k: v for k, v in g._asdict().items() if v is not None}
    assert set(got) == set(ref)
    close(g.dx, ref["dx"], size["dx"], 384, ty, "dx")
    close(g.dy, ref["dy"], size["dy"], 768, ty, "dy")
    # at most 2048 workgroups add T / 256 rows or fewer each in order, then 16 slices of their sums are added
    depth = T // 256 + 2048 // 16 + 16 + 384
    for k in sorted(set(ref) - {"dx", "dy"}):
        close(got[k], ref[k], size[k], depth, "f32", k)


# ------------------------------------------------------------------ products by every tile

TILES = [(256, 256), (128, 256), (128, 128), (128, 64), (64, 64), (64, 32)]  # tokens x channels


def tile_of(M, N):
    """The tile of the least rounds on 256 compute units times its edges, the first of equals."""
    cost = [-(-(-(-M // m) * -(-N // n)) // 256) * (m + n) for m, n in TILES]
    return TILES[cost.index(min(cost))]


PRODUCTS = [((256, 256), 1031, 8001), ((256, 256), 1501, 6003), ((128, 256), 901, 4507), ((128, 256), 409, 10007),
            ((128, 128), 401, 4503), ((128, 128), 1201, 2307), ((128, 64), 71, 10001), ((128, 64), 301, 4501),
            ((64, 64), 131, 3001), ((64, 64), 903, 777), ((64, 32), 301, 501), ((64, 32), 1009, 403), ((64, 32), 47, 203)]


@pytest.mark.parametrize("tile,M,N", PRODUCTS)
@pytest.mark.parametrize("K,ty,with_bias", [(1, "bf16", True), (1091, "bf16", True), (1091, "f16", False), (577, "f32", True),
                                            (1300, "f32", False), (2051, "f16", True)])
def test_products_by_every_tile(tile, M, N, K, ty, with_bias):
    """2 to 34 steps of 64 bytes: odd and even numbers of stages of 1, 2 or 4 of them, and more than a ring of four
    holds.  A buffer 13 channels wider than the product keeps what is behind them."""
    say(f"product {M}x{N}x{K} {ty} bias={with_bias} tile {tile}")
    assert tile_of(M, N) == tile
    qa, sa = i8(M + K, M, K, True)
    qw, sw = i8(N + K, N, K, True)
    bias = np.random.default_rng(K).standard_normal(N).astype(np.float32) if with_bias else None
    dev = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    a, w, b = plain.Int8Rows(dev(qa), dev(sa)), plain.Int8Rows(dev(qw), dev(sw)), None if bias is None else dev(bias)
    out = torch.full((M, N + 13), 7.0, dtype=TYPE[ty], device="cuda")
    code = nat.lib().ckks_plain_matmul_i8(
        a.q.data_ptr(), a.q.stride(0), a.scale.data_ptr(), w.q.data_ptr(), w.q.stride(0), w.scale.data_ptr(),
        None if b is None else b.data_ptr(), plain.TYPES[TYPE[ty]], out.data_ptr(), N + 13, M, N, K, None, 0,
        torch.cuda.current_stream().cuda_stream)
    assert code == 0
    assert (out[:, N:] == 7).all()
    assert torch.equal(out[:, :N], plain.matmul_i8(a, w, b, TYPE[ty]))
    for rows, cols in ((some(M, 40, K), np.arange(N)), (np.arange(M), some(N, 40, K))):
        ref = product_ref(qa[rows], sa[rows], qw[cols], sw[cols], None if bias is None else bias[cols])
        size = np.abs(ref if bias is None else ref - bias[cols]) + (0 if bias is None else np.abs(bias[cols]))
        close(out[torch.from_numpy(rows).cuda()][:, torch.from_numpy(cols).cuda()], ref, size, 4, ty, "out")


def test_linear_i8_of_a_prompt():
    """More than 1024 rows: the quantiser's wide form and a large tile in one call."""
    M, N, K = 1101, 7001, 1500
    x = rnd(M, M, K).to(torch.bfloat16).cuda()
    qw, sw = i8(4, N, K)
    w = plain.Int8Rows(torch.from_numpy(qw).cuda(), torch.from_numpy(sw).cuda())
    out = plain.linear_i8(x, w)
    q, s = plain_ref.quantise(f64(x))
    r = some(M, 40, 1)
    ref = product_ref(q[r], s[r], qw, sw, None)
    close(out[torch.from_numpy(r).cuda()], ref, np.abs(ref), 4, "bf16", "out")


# ------------------------------------------------------------------ nothing else is written

def gaps(T, D, pad, dtype, value):
    return torch.full((T + 2, D + pad), value, dtype=dtype, device="cuda")


def untouched(buf, T, D, value):
    """One row in front, one behind, and what is behind the columns."""
    return bool((buf[0] == value).all() and (buf[T + 1] == value).all() and (buf[1:T + 1, D:] == value).all())


@pytest.mark.parametrize("T,D,pad", [(5, 63, 1), (3, 1000, 9), (6, 2049, 7), (2, 5003, 5), (3, 16384, 3), (1030, 63, 1), (1030, 1001, 7),
                                     (1025, 9001, 13)])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_norms_write_their_columns_only(T, D, pad, ty):
    x, y, p = inputs(3, T, D, ty, True, True, 1, pad)
    lib, dt = nat.lib(), TYPE[ty]
    a = plain._norm(x, y, p["next_weight"], p["next_bias"], p["block_weight"], p["block_bias"], p["gate"], 1.0, 1e-6, "layer")
    stream = torch.cuda.current_stream().cuda_stream
    h, u = plain.residual_norm(x, y, kind="layer", **p)
    bh, bu = gaps(T, D, pad, dt, 7.0), gaps(T, D, pad + 2, dt, 7.0)
    first = lambda b: b[1].data_ptr()  # noqa: E731
    assert lib.ckks_plain_residual_norm(C.byref(a), first(bh), D + pad, first(bu), D + pad + 2, stream) == 0
    assert untouched(bh, T, D, 7) and untouched(bu, T, D, 7)
    assert torch.equal(bh[1:T + 1, :D], h) and torch.equal(bu[1:T + 1, :D], u)
    padded = -(-D // 128) * 128
    _, rows = plain.residual_norm_i8(x, y, kind="layer", **p)
    bh, bq, bs = gaps(T, D, pad, dt, 7.0), gaps(T, padded, 128, torch.int8, 7), torch.full((T + 2,), 7.0, device="cuda")
    assert lib.ckks_plain_residual_norm_i8(C.byref(a), first(bh), D + pad, first(bq), padded + 128, bs[1:].data_ptr(), stream) == 0
    assert untouched(bh, T, D, 7) and untouched(bq, T, padded, 7) and bs[0] == 7 and bs[T + 1] == 7
    assert torch.equal(bh[1:T + 1, :D], h) and torch.equal(bq[1:T + 1, :padded], rows.q) and torch.equal(bs[1:T + 1], rows.scale)
    rows = plain.quantize_rows(x)
    bq, bs = gaps(T, padded, 128, torch.int8, 7), torch.full((T + 2,), 7.0, device="cuda")
    assert lib.ckks_plain_quantize_rows(plain.TYPES[dt], x.data_ptr(), D + pad, T, D, first(bq), padded + 128, bs[1:].data_ptr(),
                                        stream) == 0
    assert untouched(bq, T, padded, 7) and bs[0] == 7 and bs[T + 1] == 7
    assert torch.equal(bq[1:T + 1, :padded], rows.q) and torch.equal(bs[1:T + 1], rows.scale)
    want = plain.residual_norm_grad(x, y, x, y, kind="layer", **p)
    bx, by = gaps(T, D, pad, dt, 7.0), gaps(T, D, pad + 2, dt, 7.0)
    sums = torch.full((5, D + 1), 7.0, device="cuda")
    ws = torch.empty(plain._norm_grad_workspace(T, D, 1, True, True, True), dtype=torch.uint8, device="cuda")
    g = nat.PlainNormGrads(x.data_ptr(), y.data_ptr(), D + pad, D + pad, first(bx), first(by), D + pad, D + pad + 2,
                           *(sums[i].data_ptr() for i in range(5)))
    assert lib.ckks_plain_residual_norm_grad(C.byref(a), C.byref(g), ws.data_ptr(), ws.numel(), stream) == 0
    assert untouched(bx, T, D, 7) and untouched(by, T, D, 7) and (sums[:, D] == 7).all()
    assert torch.equal(bx[1:T + 1, :D], want.dx) and torch.equal(by[1:T + 1, :D], want.dy)
    for i, k in enumerate(("next_weight", "next_bias", "block_weight", "block_bias", "gate")):
        assert torch.equal(sums[i, :D], want[2 + i].view(-1)), k


@pytest.mark.parametrize("M", [1, 3, 8, 9, 70])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("N,pad", [(17, 1), (1001, 7), (1024, 4)])
def test_products_write_their_channels_only(M, ty, N, pad):
    a, w = (plain.Int8Rows(torch.from_numpy(q).cuda(), torch.from_numpy(s).cuda()) for q, s in (i8(5, M, 300), i8(6, N, 300)))
    out = gaps(M, N, pad, TYPE[ty], 7.0)
    assert nat.lib().ckks_plain_matmul_i8(a.q.data_ptr(), a.q.stride(0), a.scale.data_ptr(), w.q.data_ptr(), w.q.stride(0),
                                          w.scale.data_ptr(), None, plain.TYPES[TYPE[ty]], out[1].data_ptr(), N + pad, M, N, 300,
                                          None, 0, torch.cuda.current_stream().cuda_stream) == 0
    assert untouched(out, M, N, 7)
    assert torch.equal(out[1:M + 1, :N], plain.matmul_i8(a, w, dtype=TYPE[ty]))


# ------------------------------------------------------------------ sampling

@pytest.mark.parametrize("ty,bits", [("bf16", 0x7f81), ("f16", 0x7c01), ("f32", 0x7f800001)])
def test_sample_signalling_nan(ty, bits):
    """A NaN of either kind and sign is not possible, masked or not."""
    B, V = 4, 5003
    whole = torch.int32 if ty == "f32" else torch.int16
    z = (rnd(7, B, V) * 2).to(TYPE[ty]).cuda()
    sign = -(1 << 31) if ty == "f32" else -(1 << 15)
    z.view(whole)[:, ::3] = bits
    z.view(whole)[:, 1::7] = bits + sign
    z.view(whole)[3] = bits
    t = torch.tensor([0.0, 0.8, 0.8, 0.8], device="cuda")
    for k, p, m in ((0, 1.0, 0.0), (40, 0.9, 0.0), (0, 0.95, 0.01)):
        token = check_sample(z, noise(8, B, V), t, full(B, k, torch.int32), full(B, p), full(B, m))
        assert token[3] == -1


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [50, 3000, 60001])
@pytest.mark.parametrize("k,p", [(0, 1.0), (0, 0.9), (40, 1.0), (2500, 0.9)])
def test_sample_min_p_of_one(ty, V, k, p):
    """Only equals of the largest logit stay, also where a temperature of thousands leaves e less than 2^-24 below 1;
    the noise is on the second largest value, then on the last of the equals, then spread."""
    B, r = 9, np.random.default_rng(V)
    z = np.round(-r.exponential(1, (B, V)) * 512) / 4096 - 1 / 4096   # many near the top, in every type's steps
    z[:, r.permutation(V)[:6]] = 0
    z = torch.from_numpy(z).to(TYPE[ty]).cuda()
    ranked = np.argsort(-z.float().cpu().numpy(), axis=1, kind="stable")
    g = noise(V, B, V)
    for row in range(6):
        g[row, ranked[row, 6 if row < 3 else 5]] = 50.0
    t = torch.tensor([1.0, 1e3, 1e6] * 3, device="cuda")
    token = check_sample(z, g, t, full(B, k, torch.int32), full(B, p), full(B, 1.0))
    assert (z.gather(1, token[:, None]) == 0).all()


@pytest.mark.parametrize("ty,k,p", [("f32", 0, 0.5), ("bf16", 3000, 0.9)])
def test_sample_largest_vocabulary(ty, k, p):
    """2^24 tokens, the most there may be: a greedy row, a peaked one, one whose noise is on the last token."""
    B, V = 3, 1 << 24
    say(f"sample {B}x{V} {ty} top_k={k} top_p={p}")
    z = (rnd(5, 1, V) * 2.5).to(TYPE[ty]).cuda().repeat(B, 1)
    z[2, V - 1] = z[2].max()
    g = noise(6, 1, V).repeat(B, 1)
    g[2, V - 1] = 60.0
    t = torch.tensor([0.0, 0.3, 0.5], device="cuda")
    k, p = full(B, k, torch.int32) if k else None, full(B, p)
    token, logprob = plain.sample(z, g, t, k, p)
    host = lambda v: None if v is None else v.cpu().float().numpy()  # noqa: E731
    want, ref = plain_ref.sample(host(z), host(g), host(t), host(k), host(p))
    assert np.array_equal(token.cpu().numpy(), want) and want[2] == V - 1
    # as everywhere, and a thread's sum of V / 1024 terms in order: each addition rounds
    assert (np.abs(f64(logprob) - ref) <= 2.0 ** -22 * (2 + 2 * np.abs(ref)) + V / 1024 * EPS).all()


@pytest.mark.parametrize("unit", [2.0 ** -149, 2.0 ** -140, 2.0 ** -126, 2.0 ** -118, 2.0 ** -100, 2.0 ** 100])
@pytest.mark.parametrize("V", [3000, 20011])
def test_sample_top_k_of_tiny_and_huge_steps(unit, V):
    """The first k are found by the order alone, whatever the logits' scale (the bounds' arithmetic loses digits in
    subnormal numbers).  The noise is on the k-th token, then on the next, then spread."""
    B, r = 9, np.random.default_rng(V)
    z = (r.integers(-200, 201, (B, V)) * unit).astype(np.float32)
    k = np.array([5, 50, 500] * 3, np.int32)
    g = noise(V, B, V)
    ranked = np.argsort(-z, axis=1, kind="stable")
    for row in range(6):
        g[row, ranked[row, k[row] - (row < 3)]] = 50.0
    check_sample(torch.from_numpy(z).cuda(), g, full(B, unit if unit > 1e-35 else 1.0), torch.from_numpy(k).cuda())


def test_sample_nucleus_over_a_range_too_narrow_for_bins():
    """3000 equals and the first token behind them, at a temperature of 10^-37: that token's noise decides."""
    V, n, r = 40003, 3000, np.random.default_rng(3)
    t = np.float32(1e-37)
    z = np.float32(-1) * (r.exponential(6, V).astype(np.float32) + np.float32(0.5)) * t
    z[r.permutation(V)[:n]] = 0
    e = np.exp(z.astype(np.float64) / np.float64(t))
    behind = np.argsort(-z, kind="stable")[n]
    p = np.float32([n * (1 + 5e-5) / e.sum(), (n + 0.5 + e[behind]) / e.sum(), 0.9 * n / e.sum()])
    g = torch.zeros(3, V)
    g[:, behind] = 50.0
    z = torch.from_numpy(np.repeat(z[None], 3, 0)).cuda()
    token = check_sample(z, g.cuda(), full(3, float(t)), None, torch.from_numpy(p).cuda())
    assert token[0] == behind and token[1] == behind and token[2] != behind


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("t", [1e36, 1e37, 1e38, 3e38])
@pytest.mark.parametrize("k,p,m", [(0, 0.7, 0.0), (0, 1.0, 0.5), (500, 0.8, 0.1), (200, 1.0, 0.0)])
def test_sample_temperatures_up_to_the_largest_number(ty, t, k, p, m):
    """Logits of the temperature's size (differences within 32 bits)."""
    B, V = 3, 9001
    z = (torch.rand(B, V, generator=torch.Generator().manual_seed(V), dtype=torch.float64) - 0.5) * min(6 * t, 3e38)
    check_sample(z.to(TYPE[ty]).cuda(), noise(V, B, V), full(B, t), full(B, k, torch.int32), full(B, p), full(B, m))
