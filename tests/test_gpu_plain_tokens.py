"""Embedding, norm and rotation of heads and token log probabilities
(include/ckks_plain.h) against their definitions in 64 bits (plain_token_ref).

Bounds, eps = 2^-24 (half a step of 32 bits).
 - Embedding: each product is rounded as the definition says, so results are equal bit for bit.  A sum of n
   rows adds n terms in some order: n eps of the sum of their sizes, one more for the factor, one for `into`.
 - Heads: a square sum of d <= 512 adds at most 16 terms in a thread and 6 between lanes, its root halves the
   relative error: 12 eps, and 4 for mean, root, quotient, product with the weight.  Half turns are rounded to
   32 bits (pi / 2 eps of angle), sine and cosine to 2 steps (4 eps), a position below 2^23 leaves less than an eps
   of its 64-bit product; product and sum add 2.  Together under 32 eps of |n_a| + |n_b|.  The gradient has the
   same angles and norm twice (hat, and the mean of a hat with d terms): under 96 eps of the sizes of its terms.
   The weight's adds up N = tokens heads terms in some order: 32 + N.
 - Log probabilities: x is rounded three times (3 |x| eps), exp2 to a step (2 eps), a sum over V adds at most
   V / 256 + 32 terms in order; so log mass and logprob are off by (V / 256 + 64 + 4 far + 4 |x| + 4 log mass) eps
   with `far` the mean of |x|, and the entropy by (V / 256 + 64) eps (1 + 2 far + log mass) + 8 far eps.  p of the
   gradient is exp of a number that is known to the error of log mass and a step of itself (|lp| + log mass); below
   2^-126 exp2 gives 0, which the gradient has times |dl| + |dh| (|lp| + entropy), about 100 there, over t.
Storing in 16 bits adds half a step, by rounding the ends of the range."""
import ctypes as C

import numpy as np
import pytest

import plain_token_ref as ref
from gpu_util import require_gpu, say, torch
from rns_ckks_polynomial_amd import _native as nat
from rns_ckks_polynomial_amd import plain
from test_gpu_plain import EPS, TYPE, f64, rnd, wide

pytestmark = pytest.mark.gpu
TINY = 2.0 ** -126  # results below may be flushed


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


def near(got, want, tol, what):
    """Each value between the roundings of want - tol and want + tol; infinities equal."""
    want, tol = np.asarray(want, np.float64), np.broadcast_to(np.asarray(tol, np.float64), np.shape(want)) + TINY
    cast = lambda v: f64(torch.from_numpy(np.ascontiguousarray(v)).float().to(got.dtype))  # noqa: E731
    v = f64(got)
    assert v.shape == want.shape, (what, v.shape, want.shape)
    fine = np.isfinite(want)
    low, high = cast(np.where(fine, want - tol, 0)), cast(np.where(fine, want + tol, 0))
    bad = np.where(fine, ~((v >= low) & (v <= high)), v != want)
    assert not bad.any(), f"{what}: {bad.sum()} outside, first at {np.argwhere(bad)[0]}: {v[bad][0]} for {want[bad][0]} +- {tol[bad][0]}"


def ints(seed, n, low, high):
    return np.random.default_rng(seed).integers(low, high, n)


def on_gpu(v, dt):
    return torch.from_numpy(np.ascontiguousarray(v)).to(dt).cuda()


# ------------------------------------------------------------------ embedding

@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (3, 2, 7), (4, 1000, 2048), (5, 77, 8), (130, 300, 64), (33, 5003, 2051),
                                   (9, 40, 4096), (2, 9, 16392)])
@pytest.mark.parametrize("ty,out", [("bf16", "bf16"), ("f16", "f32"), ("f32", "f32"), ("f32", "bf16"), ("bf16", "f16")])
def test_embed(T, V, D, ty, out):
    say(f"embed {T} of {V}x{D} {ty} to {out}")
    table = wide(rnd(1, V, D), TYPE[ty], 5, 3)
    t = ints(2, T, -1, V + 1)
    got = plain.embed(on_gpu(t, torch.int64), table, scale=0.3, dtype=TYPE[out])
    rows = table.cpu().float() * torch.tensor(0.3, dtype=torch.float32)
    want = torch.stack([rows[v] if 0 <= v < V else torch.zeros(D) for v in t]).to(TYPE[out])
    assert got.dtype == TYPE[out] and torch.equal(got.cpu(), want)
    assert plain.embed(on_gpu(t, torch.int64), table).dtype == TYPE[ty]


@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (4, 100, 2048), (7, 50, 129), (3, 9, 5003)])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
def test_embed_of_8_bit_rows(T, V, D, out):
    r = plain.quantize_rows(rnd(3, V, D).float().cuda())
    t = ints(4, T, -1, V)
    got = plain.embed(on_gpu(t, torch.int64), r, scale=3.0, dtype=TYPE[out])
    s = torch.tensor(3.0) * r.scale.cpu()
    rows = r.q.cpu()[:, :D].float() * s[:, None]
    want = torch.stack([rows[v] if 0 <= v < V else torch.zeros(D) for v in t]).to(TYPE[out])
    assert torch.equal(got.cpu(), want)
    assert plain.embed(on_gpu(t, torch.int64), r).dtype == torch.bfloat16


@pytest.mark.parametrize("D", [2048, 2051])
def test_embed_of_a_prompt(D):
    """More than 64 MB, past the caches."""
    table = rnd(5, 300, D).to(torch.bfloat16).cuda()
    t = on_gpu(ints(6, 17000, 0, 300), torch.int64)
    assert torch.equal(plain.embed(t, table), table[t])
    assert torch.equal(plain.embed(t, table, 0.5, torch.float32), table[t].float() * 0.5)


def test_embed_of_tokens_far_outside_and_none():
    table = torch.ones(10, 64, device="cuda")
    t = torch.tensor([-1, 10, -2 ** 63, 2 ** 63 - 1, 2 ** 32, 9], device="cuda")
    got = plain.embed(t, table)
    assert not got[:5].any() and got[5].all()
    table[3] = float("nan")
    assert not torch.isnan(plain.embed(t, table)).any()
    assert plain.embed(t[:0], table).shape == (0, 64)


def test_embed_offsets_past_32_bits():
    """Rows more than 2^32 bytes apart."""
    buf = torch.zeros(3 * (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    table = torch.as_strided(buf, (4, 1000), (1 << 30, 1))
    table.copy_(rnd(5, 4, 1000).to(torch.bfloat16))
    t = torch.tensor([3, 0, 2], device="cuda")
    assert torch.equal(plain.embed(t, table), table[t])
    drows = torch.as_strided(buf, (4, 1000), (1 << 30, 1))
    got = plain.embed_grad(drows, torch.tensor([1, 0, 1, 1], device="cuda"), 2)
    d = f64(drows)
    near(got, [d[1], d[0] + d[2] + d[3]], 4 * EPS * (np.abs(d).sum(0)), "gradient")


def tokens_of(kind, T, V, seed=7):
    rng = np.random.default_rng(seed)
    if kind == "uniform":
        return rng.integers(-1, V + 1, T)
    if kind == "one":
        return np.full(T, V - 1)
    if kind == "none":
        return np.where(rng.random(T) < 0.5, -1, V)
    if kind == "two":  # long runs that meet inside a chunk
        return np.where(rng.random(T) < 0.37, 0, V // 2)
    if kind == "falling":
        return V - 1 - np.arange(T) * V // T
    return np.minimum(V - 1, np.exp(rng.random(T) * np.log(V)).astype(np.int64))  # most frequent first


def check_embed_grad(T, V, D, ty, out, kind, scale=0.7, pad=0, into=False):
    t = tokens_of(kind, T, V)
    drows = wide(rnd(8, T, D), TYPE[ty], pad, pad // 2) if T else torch.zeros(0, D, dtype=TYPE[ty], device="cuda")
    tg = on_gpu(t, torch.int64)
    want, size, n = ref.embed_grad(f64(drows), t, V, float(np.float32(scale)))
    if not into:
        got = plain.embed_grad(drows, tg, V, scale=scale, dtype=TYPE[out])
        assert got.dtype == TYPE[out] and got.shape == (V, D)
    else:
        buf = wide(rnd(9, V, D), TYPE[out], 3, 1)
        old = f64(buf)
        before = buf.clone()
        got = plain.embed_grad(drows, tg, V, scale=scale, into=buf)
        assert got is buf
        absent = torch.from_numpy(n[:, 0] == 0).cuda()
        assert torch.equal(buf[absent], before[absent])
        want, size = want + old, size + np.abs(old)
    near(got, want, (n + 2) * EPS * size, f"{kind} {T} of {V} x {D}")
    return drows, tg


@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (5, 3, 9), (4, 1000, 2048), (700, 37, 64), (1500, 5003, 130),
                                   (3000, 1025, 72), (40, 70000, 16), (200, 50, 2051)])
@pytest.mark.parametrize("kind", ["uniform", "one", "none", "two", "falling", "text"])
def test_embed_grad(T, V, D, kind):
    say(f"embed_grad {T} of {V}x{D} {kind}")
    check_embed_grad(T, V, D, "f32", "f32", kind)
    check_embed_grad(T, V, D, "bf16", "bf16", kind, pad=3, into=True)


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("into", [False, True])
def test_embed_grad_types(ty, out, into):
    check_embed_grad(300, 40, 200, ty, out, "text", pad=5, into=into)


def test_embed_grad_of_no_rows_and_the_same_bits():
    check_embed_grad(0, 33, 40, "f32", "f32", "one")
    keep = torch.ones(33, 40, device="cuda")
    assert plain.embed_grad(torch.zeros(0, 40, device="cuda"), torch.zeros(0, dtype=torch.int64, device="cuda"), 33,
                            into=keep).eq(1).all()
    drows, t = check_embed_grad(4000, 500, 256, "bf16", "f32", "text")
    first = plain.embed_grad(drows, t, 500)
    assert all(torch.equal(first, plain.embed_grad(drows, t, 500)) for _ in range(3))


@pytest.mark.parametrize("kind", ["text", "one", "two"])
def test_embed_grad_of_many_tokens(kind):
    """More than 2048 chunks of 32 rows; a vocabulary of more than 256 workgroups' bins."""
    check_embed_grad(70001, 140001, 8, "f32", "f32", kind)


def test_embed_grad_of_the_widest_rows():
    """A long run of rows of more than 65536 * 512 columns; sums of small integers are exact."""
    D = 65536 * 512 + 5
    d = (torch.arange(D, dtype=torch.int32, device="cuda") % 5)[None] + torch.arange(33, dtype=torch.int32, device="cuda")[:, None]
    got = plain.embed_grad(d.half(), torch.ones(33, dtype=torch.int64, device="cuda"), 2)
    assert not got[0].any() and torch.equal(got[1].int(), d.sum(0, dtype=torch.int32))


def test_embed_grad_does_not_mix_what_is_not_finite():
    T, V, D = 600, 20, 64
    t = on_gpu(tokens_of("uniform", T, V), torch.int64)
    d = rnd(11, T, D).float().cuda()
    clean = plain.embed_grad(d, t, V)
    d[t == 7] = float("nan")
    d[t < 0] = float("inf")
    got = plain.embed_grad(d, t, V)
    assert torch.isnan(got[7]).all()
    got[7] = clean[7]
    assert torch.equal(got, clean)


def test_embed_autograd():
    table = rnd(12, 50, 96).to(torch.bfloat16).cuda().requires_grad_()
    t = on_gpu(tokens_of("uniform", 300, 50), torch.int64)
    w = rnd(13, 300, 96).to(torch.bfloat16).cuda()
    rows = plain.embed(t, table, scale=2.0)
    rows.backward(w)
    assert torch.equal(table.grad, plain.embed_grad(w, t, 50, 2.0, torch.bfloat16))
    table.grad = None
    plain.embed(t, table).sum().backward()  # an expanded gradient
    assert torch.equal(table.grad, plain.embed_grad(torch.ones_like(w), t, 50, 1.0, torch.bfloat16))
    g, = torch.autograd.grad(plain.embed(t, table).square().sum(), table, create_graph=True)
    with pytest.raises(RuntimeError, match="embed_grad has no gradient"):
        g.sum().backward()
    r = plain.quantize_rows(table.detach())
    r.scale.requires_grad_()
    with pytest.raises(RuntimeError, match="embed of Int8Rows has no gradient"):
        plain.embed(t, r).sum().backward()
    with pytest.raises(ValueError, match="into"):
        plain.embed_grad(w, t, 50, into=table)


# ------------------------------------------------------------------ heads

def head_inputs(seed, T, Q, K, d, r, ty, weights=True, far=1000):
    dt = TYPE[ty]
    joint = (rnd(seed, T, (Q + 2 * K) * d) * 2).to(dt).cuda()  # queries, keys, values
    q, k = joint[:, :Q * d].view(T, Q, d), joint[:, Q * d:(Q + K) * d].view(T, K, d) if K else None
    w = [(rnd(seed + 1 + i, d) * 0.3 + 1).to(dt).cuda() if weights else None for i in range(2)]
    pos = on_gpu(ints(seed + 3, T, -far, far), torch.int64) if r else None
    freq = (10000.0 ** (-torch.arange(r, dtype=torch.float64) / r)).float().cuda() if r else None
    return q, k, pos, freq, w[0], w[1] if K else None


def host(v):
    return None if v is None else v.cpu().numpy()


HEADS = [(1, 1, 0, 2, 1), (3, 2, 2, 72, 36), (2, 1, 1, 504, 252), (3, 2, 1, 64, 32), (5, 16, 8, 128, 64), (2, 3, 1, 80, 20), (7, 5, 5, 72, 9), (4, 2, 2, 96, 48),
         (3, 1, 1, 256, 128), (2, 2, 1, 512, 256), (2, 1, 1, 510, 255), (3, 4, 2, 508, 2), (9, 12, 4, 36, 18),
         (2, 2, 2, 64, 0), (130, 3, 1, 16, 8)]


@pytest.mark.parametrize("T,Q,K,d,r", HEADS)
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("weights,interleaved", [(True, False), (True, True), (False, False), (False, True)])
def test_head_norm_rotate(T, Q, K, d, r, ty, weights, interleaved):
    say(f"heads {T}x{Q}+{K}x{d} r={r} {ty} weights={weights} interleaved={interleaved}")
    q, k, pos, freq, qw, kw = head_inputs(T + d, T, Q, K, d, r, ty, weights)
    args = (pos, freq, qw, kw, 1e-5, interleaved)
    out = plain.head_norm_rotate(q, k, *args)
    dq, dk = (None if v is None else (rnd(i, *v.shape)).to(v.dtype).cuda() for i, v in ((21, q), (22, k)))
    g = plain.head_norm_rotate_grad(q, k, dq, dk, *args)
    e = float(np.float32(1e-5))
    for x, w, y, dy, dx, dw in ((q, qw, out[0], dq, g.dq, g.q_weight), (k, kw, out[1], dk, g.dk, g.k_weight)):
        if x is None:
            assert y is None and dx is None and dw is None
            continue
        assert y.dtype == dx.dtype == x.dtype and y.shape == dx.shape == x.shape
        want, size = ref.heads(f64(x), f64(w), host(pos), host(freq), e, interleaved)
        near(y, want, 32 * EPS * size, "forward")
        a, asize, b, bsize = ref.heads_grad(f64(x), f64(dy), f64(w), host(pos), host(freq), e, interleaved)
        near(dx, a, 96 * EPS * asize, "gradient")
        if w is None:
            assert dw is None
        else:
            near(dw, b, (32 + T * x.shape[1]) * EPS * bsize, "weight")


@pytest.mark.parametrize("T", [1, 33, 2500])
def test_heads_of_many_tokens(T):
    """More tokens than workgroups of the gradient."""
    q, k, pos, freq, qw, kw = head_inputs(31, T, 6, 2, 64, 32, "bf16")
    dq, dk = rnd(32, *q.shape).to(q.dtype).cuda(), rnd(33, *k.shape).to(k.dtype).cuda()
    got = plain.head_norm_rotate(q, k, pos, freq, qw, kw)
    g = plain.head_norm_rotate_grad(q, k, dq, dk, pos, freq, qw, kw)
    e = float(np.float32(1e-6))
    for x, w, y, dy, dx, dw in ((q, qw, got[0], dq, g.dq, g.q_weight), (k, kw, got[1], dk, g.dk, g.k_weight)):
        want, size = ref.heads(f64(x), f64(w), host(pos), host(freq), e, False)
        near(y, want, 32 * EPS * size, "forward")
        a, asize, b, bsize = ref.heads_grad(f64(x), f64(dy), f64(w), host(pos), host(freq), e, False)
        near(dx, a, 96 * EPS * asize, "gradient")
        near(dw, b, (32 + T * x.shape[1]) * EPS * bsize, "weight")
    again = plain.head_norm_rotate_grad(q, k, dq, dk, pos, freq, qw, kw)
    assert all(torch.equal(a, b) for a, b in zip(g, again))


def test_heads_at_far_positions():
    """An angle of 8 million turns and its neighbour differ by what the definition says."""
    T = 64
    q, _, _, freq, qw, _ = head_inputs(41, T, 2, 0, 128, 64, "f32")
    pos = on_gpu(8388607 - np.arange(T), torch.int64)
    got, _ = plain.head_norm_rotate(q, None, pos, freq, qw)
    want, size = ref.heads(f64(q), f64(qw), host(pos), host(freq), float(np.float32(1e-6)), False)
    near(got, want, 32 * EPS * size, "far")


def test_heads_of_other_strides():
    """Heads outside tokens, a gap between heads, one head out of many, and outputs with gaps through the C call."""
    x = (rnd(51, 6, 9, 70)).to(torch.bfloat16).cuda()
    pos, freq = torch.arange(9, device="cuda"), torch.tensor([1.0, 0.3, 0.01], device="cuda")
    for q in (x.transpose(0, 1)[:, :, :64], x[:, ::2, 6:], x[:, 3:4, :64], x[2:3, :, 1:65]):
        p = pos[:q.shape[0]].clone()
        want, _ = plain.head_norm_rotate(q.contiguous(), None, p, freq)
        got, _ = plain.head_norm_rotate(q, None, p, freq)
        assert torch.equal(got, want)
        dq = plain.head_norm_rotate_grad(q, None, q, None, p, freq).dq
        assert torch.equal(dq, plain.head_norm_rotate_grad(q.contiguous(), None, q.contiguous(), None, p, freq).dq)
    q = x[:, :, :64]
    at = pos[:6].clone()  # alive as long as its address is used
    want, _ = plain.head_norm_rotate(q, None, at, freq)
    p = plain._head_args(q, None, at, freq, None, None, 1e-6, False)
    out = torch.full((9, 6, 66), 7.0, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    assert nat.lib().ckks_plain_head_norm_rotate(C.byref(p), out.data_ptr(), 66, 6 * 66, None, 0, 0, stream) == 0
    assert torch.equal(out.transpose(0, 1)[:, :, :64], want) and out[..., 64:].eq(7).all()
    keep = x.clone()
    assert nat.lib().ckks_plain_head_norm_rotate(C.byref(p), q.data_ptr(), 9 * 70, 70, None, 0, 0, stream) == 0  # in place
    assert torch.equal(q, want) and torch.equal(x[..., 64:], keep[..., 64:])


def test_heads_in_place_in_joint_rows():
    """Queries and keys of a joint projection over themselves: values between them stay."""
    T, Q, K, d = 9, 4, 2, 64
    joint = rnd(53, T, (Q + 2 * K) * d).to(torch.bfloat16).cuda()
    q, k, v = (joint[:, a * d:b * d].view(T, b - a, d) for a, b in ((0, Q), (Q, Q + K), (Q + K, Q + 2 * K)))
    pos, freq = torch.arange(T, device="cuda") * 5, torch.tensor([1.0, 0.3], device="cuda")
    w = (1 + 0.1 * rnd(54, d)).to(torch.bfloat16).cuda()
    want, old = plain.head_norm_rotate(q, k, pos, freq, w, w), v.clone()
    p = plain._head_args(q, k, pos, freq, w, w, 1e-6, False)
    s = joint.stride(0)
    assert nat.lib().ckks_plain_head_norm_rotate(C.byref(p), q.data_ptr(), s, d, k.data_ptr(), s, d,
                                                 torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, old)


def test_heads_that_are_zero_or_not_finite():
    q, k, pos, freq, qw, kw = head_inputs(61, 4, 3, 1, 64, 32, "f32")
    q, k = q.clone(), k.clone()
    clean = plain.head_norm_rotate(q, k, pos, freq, qw, kw)
    q[1, 2], q[2, 0, 5], k[3, 0, 63] = 0.0, float("inf"), float("nan")
    out = plain.head_norm_rotate(q, k, pos, freq, qw, kw)
    assert not out[0][1, 2].any() and torch.isnan(out[0][2, 0]).any() and torch.isnan(out[1][3]).any()
    ok = torch.ones(4, 3, dtype=torch.bool)
    ok[1, 2] = ok[2, 0] = False
    assert torch.equal(out[0][ok], clean[0][ok]) and torch.equal(out[1][:3], clean[1][:3])
    z = torch.zeros(2, 1, 64, device="cuda")
    assert torch.isfinite(plain.head_norm_rotate_grad(z, None, z + 1, None, pos[:2].clone(), freq, qw).dq).all()


def test_heads_without_tokens():
    q, k, pos, freq, qw, kw = head_inputs(62, 4, 3, 1, 64, 32, "bf16")
    q, k, pos = q[:0], k[:0], pos[:0]
    out = plain.head_norm_rotate(q, k, pos, freq, qw, kw)
    assert out[0].shape == (0, 3, 64) and out[1].shape == (0, 1, 64)
    g = plain.head_norm_rotate_grad(q, k, q, k, pos, freq, qw, kw)
    assert not g.q_weight.any() and not g.k_weight.any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_heads_gradient_against_differences(interleaved):
    """Central differences of the 64-bit definition at the kernel's inputs, along random directions."""
    q, _, pos, freq, qw, _ = head_inputs(63, 5, 3, 0, 48, 20, "f32")
    dq = rnd(64, *q.shape).float().cuda()
    g = plain.head_norm_rotate_grad(q, None, dq, None, pos, freq, qw, None, 1e-6, interleaved)
    x, w, up = f64(q), f64(qw), f64(dq)
    f = lambda x, w: (ref.heads(x, w, host(pos), host(freq), 1e-6, interleaved)[0] * up).sum()  # noqa: E731
    h = 1e-6
    for seed in range(4):
        vx, vw = f64(rnd(70 + seed, *x.shape)), f64(rnd(80 + seed, *w.shape))
        slope = (f(x + h * vx, w + h * vw) - f(x - h * vx, w - h * vw)) / (2 * h)
        got = (f64(g.dq) * vx).sum() + (f64(g.q_weight) * vw).sum()
        # the differences: h^2 / 6 of third derivatives of order 1 and 2^-53 |f| / h; the kernel: 96 eps of its terms
        size = (np.abs(f64(g.dq) * vx)).sum() + (np.abs(f64(g.q_weight) * vw)).sum()
        assert abs(got - slope) < 256 * EPS * size + 1e-7 * size


def test_heads_autograd():
    q, k, pos, freq, qw, kw = head_inputs(65, 6, 4, 2, 64, 32, "bf16")
    leaves = [v.clone().requires_grad_() for v in (q, k, qw, kw)]
    out = plain.head_norm_rotate(leaves[0], leaves[1], pos, freq, leaves[2], leaves[3])
    a, b = rnd(66, *q.shape).to(q.dtype).cuda(), rnd(67, *k.shape).to(k.dtype).cuda()
    torch.autograd.backward(out, (a, b))
    g = plain.head_norm_rotate_grad(q, k, a, b, pos, freq, qw, kw)
    assert torch.equal(leaves[0].grad, g.dq) and torch.equal(leaves[1].grad, g.dk)
    assert torch.equal(leaves[2].grad, g.q_weight.to(qw.dtype)) and torch.equal(leaves[3].grad, g.k_weight.to(kw.dtype))
    # queries alone, an expanded gradient, one shared by all heads
    x = leaves[0]
    x.grad = None
    plain.head_norm_rotate(x, None, pos, freq, qw)[0].sum().backward()
    assert torch.equal(x.grad, plain.head_norm_rotate_grad(q, None, torch.ones_like(q), None, pos, freq, qw).dq)
    one, = torch.autograd.grad(plain.head_norm_rotate(x, leaves[1], pos, freq)[1].float().sum(), leaves[1])
    assert torch.equal(one, plain.head_norm_rotate_grad(q, k, torch.zeros_like(q), torch.ones_like(k), pos, freq).dk)
    g2, = torch.autograd.grad(plain.head_norm_rotate(x, None, pos, freq, qw)[0].square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="head_norm_rotate_grad has no gradient"):
        g2.sum().backward()
    with pytest.raises(RuntimeError, match="no gradient of inv_freq"):
        plain.head_norm_rotate(q, k, pos, freq.clone().requires_grad_())[0].sum().backward()


# ------------------------------------------------------------------ log probabilities

def check_score(z, tokens, top=0, temperature=None, allowed=None, grad=True, seed=5):
    B, V = z.shape
    tg = on_gpu(tokens, torch.int64)
    r = plain.token_logprobs(z, tg, top, temperature, allowed)
    want = ref.score(f64(z), tokens, top, None if temperature is None else temperature.cpu().numpy(), host(allowed))
    lm = np.where(np.isfinite(want["log_mass"]), want["log_mass"], 0)
    base = (V / 256 + 64 + 4 * want["far"] + 4 * lm) * EPS
    x_of = lambda lp, k: np.abs(np.where(np.isfinite(lp), lp, 0)) + k  # noqa: E731
    assert np.array_equal(f64(r.largest), want["largest"])
    near(r.log_mass, want["log_mass"], base, "log_mass")
    near(r.logprob, want["logprob"], base + 4 * EPS * x_of(want["logprob"], lm), "logprob")
    near(r.entropy, want["entropy"], (V / 256 + 64) * EPS * (1 + 2 * want["far"] + lm) + 8 * EPS * want["far"], "entropy")
    assert r.top_token.shape == r.top_logprob.shape == (B, top)
    assert np.array_equal(r.top_token.cpu().numpy(), want["top_token"])
    near(r.top_logprob, want["top_logprob"], base[:, None] + 4 * EPS * x_of(want["top_logprob"], lm[:, None]), "top")
    if grad:
        dl, dh = rnd(seed, B).float().cuda(), rnd(seed + 1, B).float().cuda()
        for a, b in ((dl, dh), (dl, None), (None, dh)):
            d = plain.token_logprobs_grad(z, tg, r, a, b, temperature, allowed)
            assert d.dtype == z.dtype and d.shape == z.shape
            g, size = ref.score_grad(want, tokens, f64(a), f64(b))
            lp = np.where(want["lp"] > -200, np.abs(want["lp"]), 0)
            h_off = (V / 256 + 64) * EPS * (1 + 2 * want["far"] + lm) + 8 * EPS * want["far"]
            off = base[:, None] + (8 + 8 * lp + 8 * lm[:, None]) * EPS
            p = np.exp(want["lp"])
            tol = off * size + p * (0 if b is None else np.abs(f64(b)) * (h_off + off.max(1)))[..., None] * want["inv_t"][:, None] \
                if b is not None else off * size
            weight = sum(0 if v is None else np.abs(f64(v))[:, None] * k for v, k in (
                (a, 1), (b, np.where(np.isfinite(want["lp"]), np.abs(want["lp"]), 0) + want["entropy"][:, None])))
            tol = tol + TINY * weight * want["inv_t"][:, None]
            near(d, g, np.where(want["possible"], tol, 0), "dlogits")
    return r


@pytest.mark.parametrize("B,V", [(1, 1), (3, 7), (2, 1000), (5, 2048), (3, 8200), (2, 50021), (300, 513)])
@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("top", [0, 1, 5, 64])
def test_token_logprobs(B, V, ty, top):
    say(f"token_logprobs {B}x{V} {ty} top {top}")
    z = wide(rnd(B + V, B, V) * 2.5, TYPE[ty], 5, 3)
    check_score(z, ints(1, B, -1, V + 1), top)
    check_score(z.contiguous(), ints(2, B, 0, V), top)


@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
def test_token_logprobs_masks_and_temperatures(ty):
    B, V = 12, 3001
    z = wide(rnd(3, B, V) * 3, TYPE[ty], 7, 4)
    buf = torch.from_numpy(np.random.default_rng(4).random((B, V + 3)) < 0.3).cuda()
    allowed = buf[:, 2:V + 2]
    allowed[2] = False                     # nothing
    allowed[3] = False
    allowed[3, 2999] = True                # one token
    allowed[5] = True
    z[5, :2990] = float("-inf")            # masked by the logits
    z[6, ::2] = float("nan")
    z[7, 100:] = torch.finfo(TYPE[ty]).min  # masks of the type's lowest value, which is a number
    z[8] = torch.finfo(TYPE[ty]).min
    t = torch.tensor([0.7, 1.3, 1, 0.5, 0, -1, 2, 1, 1, 1e-3, float("nan"), 0.9], device="cuda")
    tokens = ints(6, B, 0, V)
    tokens[3] = 2999
    tokens[7] = 50
    for top in (0, 7, 64):
        check_score(z, tokens, top, t, allowed)
        check_score(z, tokens, top, None, allowed)
        check_score(z, tokens, top, t)
    r = check_score(z, np.full(B, -1), 3, t, allowed)
    assert not r.logprob.any() and r.top_token[2].eq(-1).all() and r.entropy[2] == 0


@pytest.mark.parametrize("V", [1, 64, 5000, 70001])
@pytest.mark.parametrize("ty", ["bf16", "f32"])
def test_token_logprobs_of_equal_logits(V, ty):
    """Whole rows of equals, few values, and alternatives at the end of the row: the lowest indexes come first."""
    z = torch.zeros(6, V, dtype=TYPE[ty], device="cuda")
    z[1] = -0.0
    z[2] = -5.0
    z[2, V // 2:] = 3.0
    z[3] = on_gpu(ints(8, V, 0, 3), TYPE[ty])
    z[4] = torch.arange(V, device="cuda").to(TYPE[ty])
    z[5] = -torch.arange(V, device="cuda").to(TYPE[ty])
    check_score(z, ints(9, 6, 0, V), 64)
    check_score(z, ints(9, 6, 0, V), 1)


@pytest.mark.parametrize("period", [8, 512, 4096, 8192])
def test_token_logprobs_of_periodic_rows(period):
    """The largest logits all in one place of every period, in falling and in rising order."""
    V = 60000
    z = (rnd(14, 4, V) * 0.1).float()
    at = torch.arange(0, V, period)
    for row, slope in ((0, -1e-3), (1, 1e-3), (2, 0.0)):
        z[row, at] = 5 + slope * torch.arange(len(at))
    z[3, at] = float("-inf")
    check_score(z.cuda(), ints(10, 4, 0, V), 64)


@pytest.mark.parametrize("n", [1, 3])
def test_token_logprobs_of_infinite_logits(n):
    z = rnd(15, 3, 900).float().cuda()
    at = torch.tensor([5, 700, 899], device="cuda")[:n]
    z[:, at] = float("inf")
    z[1, 7] = float("nan")
    r = check_score(z, np.array([5, 6, 899]), 5, grad=False)
    d = plain.token_logprobs_grad(z, on_gpu([5, 6, 899], torch.int64), r, torch.ones(3, device="cuda"))
    assert torch.isfinite(d).all() and abs(float(d[0, 5]) - (1 - 1 / n)) < 1e-6 and d[0, 6] == 0
    if n == 3:
        assert abs(float(r.logprob[0]) + np.log(3)) < 1e-6 and abs(float(r.entropy[1]) - np.log(3)) < 1e-6


def test_token_logprobs_extreme_temperatures_and_sizes():
    V = 700
    t = torch.tensor([1e-45, 1e-38, 1e-30, 1e30, 3e38, float("inf"), 1, 1], device="cuda")
    z = (rnd(16, 8, V) * 3).float().cuda()
    z[6] *= 1e37
    z[7] *= 1e-38
    check_score(z, ints(11, 8, 0, V), 4, t, grad=False)
    r = plain.token_logprobs(z, torch.zeros(8, dtype=torch.int64, device="cuda"), 4, t)
    d = plain.token_logprobs_grad(z, torch.zeros(8, dtype=torch.int64, device="cuda"), r, None,
                                  torch.ones(8, device="cuda"), t)
    assert not torch.isnan(d).any()


def test_token_logprobs_offsets_past_32_bits():
    buf = torch.zeros(3 * (1 << 30) + 4096, dtype=torch.bfloat16, device="cuda")
    z = torch.as_strided(buf, (4, 1000), (1 << 30, 1))
    z.copy_((rnd(5, 4, 1000) * 2).to(torch.bfloat16))
    check_score(z, ints(12, 4, 0, 1000), 9)


def test_token_logprobs_of_the_largest_vocabulary():
    V = 1 << 24
    z = torch.zeros(1, V, dtype=torch.bfloat16, device="cuda")
    z[0, V - 1], z[0, 1 << 20] = 3.0, 2.0
    r = plain.token_logprobs(z, torch.tensor([V - 1], device="cuda"), 4)
    assert r.top_token.tolist() == [[V - 1, 1 << 20, 0, 1]]
    mass = 1 + np.exp(-1.0) + (V - 2) * np.exp(-3.0)
    near(r.log_mass, [np.log(mass)], (V / 256 + 64) * EPS, "log_mass")


def test_token_logprobs_grad_into_rows_of_a_wider_buffer():
    z = wide(rnd(17, 5, 3000) * 2, torch.bfloat16, 11, 5)
    tok = on_gpu(ints(13, 5, 0, 3000), torch.int64)
    r = plain.token_logprobs(z, tok)
    dl = torch.ones(5, device="cuda")
    want = plain.token_logprobs_grad(z, tok, r, dl)
    buf = torch.full((5, 3021), 9.0, dtype=torch.bfloat16, device="cuda")
    call = lambda out, stride: nat.lib().ckks_plain_token_logprobs_grad(  # noqa: E731
        0, z.data_ptr(), z.stride(0), tok.data_ptr(), None, None, 0, 5, 3000, r.entropy.data_ptr(),
        r.largest.data_ptr(), r.log_mass.data_ptr(), dl.data_ptr(), None, out, stride,
        torch.cuda.current_stream().cuda_stream)
    assert call(buf[:, 3:].data_ptr(), 3021) == 0
    torch.cuda.synchronize()
    assert torch.equal(buf[:, 3:3003], want) and buf[:, :3].eq(9).all() and buf[:, 3003:].eq(9).all()
    assert call(z.data_ptr(), z.stride(0)) == nat.EINVAL  # the logits are read while gradients are written


@pytest.mark.parametrize("B,V", [(1, 262144), (3, 70001), (5, 1 << 20), (100, 65536)])
@pytest.mark.parametrize("top", [0, 5, 64])
def test_token_logprobs_of_few_long_rows(B, V, top):
    """Rows in slices: equal logits across them, slices without a possible token, infinities in two of them."""
    z = (rnd(27, B, V) * 2).to(torch.bfloat16).cuda()
    z[0, V // 3:] = float("-inf")
    allowed = None
    if B > 1:
        z[1] = torch.arange(V, device="cuda").remainder(7).to(torch.bfloat16)
        z[2, :100] = -3.0
        z[2, 100:] = float("nan")
        allowed = torch.ones(B, V, dtype=torch.bool, device="cuda")
        allowed[0] = False
    check_score(z, ints(28, B, 0, V), top, None, allowed, grad=B < 100)
    z[0, 5] = z[0, V - 1] = float("inf")
    check_score(z, ints(28, B, 0, V), top, grad=False)


def test_token_logprobs_past_the_caches():
    """More than 128 MiB of logits."""
    check_score((rnd(29, 264, 131072) * 2).float().cuda(), ints(29, 264, 0, 131072), 3)


def test_token_logprobs_agree_with_sample():
    """The drawn tokens' log probabilities are those that sample reports, for every temperature and mask."""
    B, V = 40, 5000
    z = (rnd(18, B, V) * 2).to(torch.bfloat16).cuda()
    allowed = torch.from_numpy(np.random.default_rng(19).random((B, V)) < 0.5).cuda()
    allowed[11] = False
    g = on_gpu(-np.log(-np.log(np.random.default_rng(20).uniform(1e-9, 1 - 1e-9, (B, V)))), torch.float32)
    t = torch.linspace(-0.2, 2, B, device="cuda")
    token, logprob = plain.sample(z, g, t, allowed=allowed)
    r = plain.token_logprobs(z, token, 1, t, allowed)
    assert token[11] == -1 and r.logprob[11] == 0
    ok = token >= 0
    # each within V / 256 + 64 + 8 (10 + 10) of eps of the exact one
    assert (r.logprob[ok] - logprob[ok]).abs().max() < 2 * (V / 256 + 224) * EPS
    greedy = ~(t > 0) & ok
    assert greedy.any() and torch.equal(r.top_token[greedy, 0], token[greedy])


def test_the_examples_scores():
    """examples/next_token.py: the draws' log probabilities from both operators, and the likeliest in front."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import next_token
    r = next_token.main()
    s = r["scores"]
    assert (s.logprob - r["logprob"]).abs().max() < 2 * (next_token.VOCAB / 256 + 224) * EPS  # as above
    assert torch.equal(s.top_token[:, 0], r["logits"].argmax(1)) and (s.top_logprob.diff(dim=1) <= 0).all()
    assert (s.entropy > 0).all() and (s.logprob <= s.top_logprob[:, 0]).all()


def test_token_logprobs_grad_against_differences():
    B, V = 3, 60
    z, tokens = rnd(21, B, V).float().cuda(), ints(22, B, 0, V)
    t = torch.tensor([0.8, 1.0, 1.7], device="cuda")
    dl, dh = rnd(23, B).float().cuda(), rnd(24, B).float().cuda()
    tg = on_gpu(tokens, torch.int64)
    d = f64(plain.token_logprobs_grad(z, tg, plain.token_logprobs(z, tg, 0, t), dl, dh, t))
    def f(v):
        r = ref.score(v, tokens, 0, t.cpu().numpy())
        return (r["logprob"] * f64(dl) + r["entropy"] * f64(dh)).sum()
    h = 1e-6
    for i in range(20):
        v = f64(rnd(30 + i, B, V))
        slope = (f(f64(z) + h * v) - f(f64(z) - h * v)) / (2 * h)
        assert abs((d * v).sum() - slope) < (256 * EPS + 1e-7) * np.abs(d * v).sum() + 1e-8


def test_token_logprobs_autograd():
    z = (rnd(25, 6, 800) * 2).to(torch.bfloat16).cuda().requires_grad_()
    tok = on_gpu(ints(26, 6, -1, 800), torch.int64)
    r = plain.token_logprobs(z, tok, 3)
    (r.logprob.sum() * -1 + r.entropy.sum() * 0.5).backward()
    direct = plain.token_logprobs(z.detach(), tok, 3)
    assert all(torch.equal(a.detach(), b) for a, b in zip(r, direct))
    one = torch.ones(6, device="cuda")
    assert torch.equal(z.grad, plain.token_logprobs_grad(z.detach(), tok, direct, -one, 0.5 * one))
    g, = torch.autograd.grad(plain.token_logprobs(z, tok).logprob.sum(), z)
    assert torch.equal(g, plain.token_logprobs_grad(z.detach(), tok, direct, one))
    for name in ("top_logprob", "largest", "log_mass"):
        with pytest.raises(RuntimeError, match="logprob and entropy alone"):
            getattr(plain.token_logprobs(z, tok, 3), name).sum().backward()
    with pytest.raises(RuntimeError, match="temperature"):
        plain.token_logprobs(z, tok, 0, torch.ones(6, device="cuda", requires_grad=True)).logprob.sum().backward()
    g, = torch.autograd.grad(plain.token_logprobs(z, tok).logprob.sum(), z, create_graph=True)
    with pytest.raises(RuntimeError, match="token_logprobs_grad has no gradient"):
        g.sum().backward()


# ------------------------------------------------------------------ use

class Decoder:
    """One narrow layer around the operators: embedding, norm, queries and keys with their norm and rotation, a mix of
    them in torch, the tied vocabulary and the loss."""
    T, V, D, H, d = 48, 300, 64, 4, 16

    def __init__(self, dt, device):
        to = lambda v: v.to(dt).to(device)  # noqa: E731
        self.table, self.norm = to(rnd(1, self.V, self.D)), to(1 + 0.1 * rnd(2, self.D))
        self.proj = to(rnd(3, self.D, 2 * self.H * self.d) * 0.2)
        self.qw, self.kw = to(1 + 0.1 * rnd(4, self.d)), to(1 + 0.1 * rnd(5, self.d))
        self.tokens = torch.from_numpy(tokens_of("text", self.T, self.V)).to(device)
        self.tokens[-3:] = -1
        self.positions = torch.arange(self.T, device=device)
        self.freq = (100.0 ** (-torch.arange(8, dtype=torch.float64) / 8)).float().to(device)
        self.leaves = [self.table, self.norm, self.proj, self.qw, self.kw]

    def loss(self, embed, residual_norm, head_norm_rotate, token_logprobs):
        x = embed(self.tokens, self.table)
        h, u = residual_norm(x, torch.zeros_like(x), self.norm)
        joint = u @ self.proj
        n = self.H * self.d
        q, k = head_norm_rotate(joint[:, :n].view(-1, self.H, self.d), joint[:, n:].view(-1, self.H, self.d),
                                self.positions, self.freq, self.qw, self.kw)
        y = torch.tanh(q * k.flip(0)).reshape(-1, n)
        logits = (h + y) @ self.table.t()
        logprob, entropy = token_logprobs(logits, torch.roll(self.tokens, -1))[:2]
        return (entropy * 0.01 - logprob).sum() / self.T


def clear_decoder():
    """The loss and gradients in 64 bits on the CPU, by torch's own derivatives."""
    m = Decoder(torch.float64, "cpu")
    for v in m.leaves:
        v.requires_grad_()

    def embed(t, table):
        return torch.where((t >= 0)[:, None], table[t.clamp(min=0)], torch.zeros((), dtype=table.dtype))

    def norm(v, w):
        return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6) * w

    def heads(q, k, pos, freq, qw, kw):
        f = pos.double()[:, None, None] * freq.double()
        def turned(v):
            a, b = v.chunk(2, -1)
            return torch.cat([a * f.cos() - b * f.sin(), b * f.cos() + a * f.sin()], -1)
        return turned(norm(q, qw)), turned(norm(k, kw))

    def logprobs(z, t):
        lp = torch.log_softmax(z, -1)
        got = lp.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return torch.where(t >= 0, got, torch.zeros_like(got)), -(lp.exp() * lp).sum(-1)

    loss = m.loss(embed, lambda x, y, w: (x + y, norm(x + y, w)), heads, logprobs)
    loss.backward()
    return loss, [v.grad for v in m.leaves]


def test_a_decoders_loss_and_gradients():
    want, grads = clear_decoder()
    m = Decoder(torch.float32, "cuda")
    for v in m.leaves:
        v.requires_grad_()
    loss = m.loss(plain.embed, plain.residual_norm, plain.head_norm_rotate, plain.token_logprobs)
    loss.backward()
    # four products of at most 300 terms, two norms and a softmax in 32 bits between leaf and gradient, each with at
    # most 300 roundings of terms that cancel by less than 30: 6 * 300 * 30 eps of a gradient's size
    assert abs(float(loss.detach()) - float(want.detach())) < 6 * 300 * EPS * abs(float(want.detach()))
    for got, g in zip((v.grad for v in m.leaves), grads):
        off = (got.double().cpu() - g).norm() / g.norm()
        assert off < 6 * 300 * 30 * EPS, float(off)


def pass_through(state):
    """All operators once, forward and back, as tensors."""
    table, t, w, pos, freq, hw, into = state
    x = plain.embed(t, table, scale=1.5)
    h, u = plain.residual_norm(x, x, w)
    q, k = plain.head_norm_rotate(u[:, :96].view(-1, 3, 32), u[:, 96:].view(-1, 1, 32), pos, freq, hw, hw)
    logits = torch.cat([q.flatten(1), k.flatten(1), h], 1)
    r = plain.token_logprobs(logits, t, 6)
    dz = plain.token_logprobs_grad(logits, t, r, r.entropy, r.logprob)
    g = plain.head_norm_rotate_grad(q, k, q, k, pos, freq, hw, hw)
    return [x, q, k, *r, dz, *g, plain.embed_grad(dz[:, :128].contiguous(), t, table.shape[0]),
            plain.embed_grad(dz[:, 128:], t, table.shape[0], into=into.clone())]


def some_state(T=300, V=90):
    t = on_gpu(tokens_of("text", T, V), torch.int64)
    freq = (100.0 ** (-torch.arange(16, dtype=torch.float64) / 16)).float().cuda()
    return [(rnd(1, V, 128)).to(torch.bfloat16).cuda(), t, (1 + 0.1 * rnd(2, 128)).to(torch.bfloat16).cuda(),
            torch.arange(T, device="cuda") * 37, freq, (1 + 0.1 * rnd(3, 32)).to(torch.bfloat16).cuda(),
            rnd(4, V, 128).float().cuda()]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_tokens_on_another_stream_and_in_a_graph():
    state = some_state()
    want = [v.clone() for v in pass_through(state)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = pass_through(state)
    s.synchronize()
    assert same(want, got)
    graphs = []
    for _ in range(2):  # two graphs of the same operators, replayed in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = pass_through(state)
        graphs.append((graph, out))
    for n in range(4):
        state[0].mul_(1.25)
        state[1].copy_(torch.roll(state[1], 7))
        want = [v.clone() for v in pass_through(state)]
        torch.cuda.synchronize()
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(same(want, out) for _, out in graphs), n


def test_token_operators_refuse_forward_mode():
    from torch.autograd import forward_ad
    state = some_state(40, 20)
    table, t, w, pos, freq, hw, into = state
    z = rnd(6, 40, 20).float().cuda()
    heads = rnd(7, 40, 2, 32).float().cuda()
    r = plain.token_logprobs(z, t)
    calls = [(z, lambda v: plain.embed(t, v).sum()), (z, lambda v: plain.embed_grad(v, t, 9)),
             (heads, lambda v: plain.head_norm_rotate(v, None, pos, freq)[0]),
             (heads, lambda v: plain.head_norm_rotate_grad(heads, None, v, None, pos, freq).dq),
             (z, lambda v: plain.token_logprobs(v, t).logprob), (z, lambda v: plain.token_logprobs_grad(v, t, r, r.entropy))]
    for x, f in calls:
        with forward_ad.dual_level():
            with pytest.raises((RuntimeError, NotImplementedError), match="forward"):
                f(forward_ad.make_dual(x, torch.ones_like(x)))


def test_token_binding_refusals():
    x, t = torch.zeros(4, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    h, f, w = torch.zeros(4, 2, 64, device="cuda"), torch.ones(8, device="cuda"), torch.ones(64, device="cuda")
    r = plain.token_logprobs(x, t)
    bad = [(lambda: plain.embed(t.int(), x), "tokens"), (lambda: plain.embed(t[None], x), "tokens"),
           (lambda: plain.embed(t.cpu(), x), "tokens"), (lambda: plain.embed(t, x.double()), "table"),
           (lambda: plain.embed(t, x.t()), "table"), (lambda: plain.embed(t, x, dtype=torch.int8), "dtype"),
           (lambda: plain.embed(None, x), "tokens"), (lambda: plain.embed(t, None), "table"),
           (lambda: plain.embed_grad(x, t[:3], 9), "tokens"), (lambda: plain.embed_grad(x, t, 9, dtype=torch.int64), "dtype"),
           (lambda: plain.embed_grad(x, t, 9, into=x), "into"), (lambda: plain.embed_grad(x[0], t, 9), "drows"),
           (lambda: plain.head_norm_rotate(x, None, t, f), "q"), (lambda: plain.head_norm_rotate(h, h.half(), t, f), "k"),
           (lambda: plain.head_norm_rotate(h, h[:2], t, f), "k"), (lambda: plain.head_norm_rotate(h, h[..., :32], t, f), "k"),
           (lambda: plain.head_norm_rotate(h, None, t, f, None, w), "k_weight"),
           (lambda: plain.head_norm_rotate(h, h[:, :0], t, f), "k"), (lambda: plain.head_norm_rotate(h, None, t, None), "both"),
           (lambda: plain.head_norm_rotate(h, None, t[:3], f), "positions"),
           (lambda: plain.head_norm_rotate(h, None, t, f.double()), "inv_freq"),
           (lambda: plain.head_norm_rotate(h, None, t, f, w[:32]), "q_weight"),
           (lambda: plain.head_norm_rotate(h[..., ::2], None, t, f), "unit stride"),
           (lambda: plain.head_norm_rotate(h.double(), None, t, f), "q"),
           (lambda: plain.head_norm_rotate_grad(h, None, None, None, t, f), "dq"),
           (lambda: plain.head_norm_rotate_grad(h, None, h, h, t, f), "dk"),
           (lambda: plain.head_norm_rotate_grad(h, None, h[:, :1], None, t, f), "dq"),
           (lambda: plain.token_logprobs(x, t[:3]), "tokens"), (lambda: plain.token_logprobs(x, None), "tokens"),
           (lambda: plain.token_logprobs(x, t, 65), "top"), (lambda: plain.token_logprobs(x, t, -1), "top"),
           (lambda: plain.token_logprobs(x, t, 0, w), "temperature"), (lambda: plain.token_logprobs(x, t, 0, None, x), "allowed"),
           (lambda: plain.token_logprobs(h, t), "logits"), (lambda: plain.token_logprobs_grad(x, t, None), "scores"),
           (lambda: plain.token_logprobs_grad(x, t, r, w), "dlogprob"),
           (lambda: plain.token_logprobs_grad(x, t, r, None, r.entropy.double()), "dentropy"),
           (lambda: plain.token_logprobs_grad(x, t, plain.TokenLogprobs(*(v[:2] for v in r))), "scores")]
    for call, what in bad:
        with pytest.raises(ValueError, match=what):
            call()
    for call in (lambda: plain.head_norm_rotate(h[..., :63], None, t, f), lambda: plain.head_norm_rotate(h, None, t, w[:33]),
                 lambda: plain.head_norm_rotate(h[:, :1].expand(4, 3, 64), None, t, f),
                 lambda: plain.embed_grad(x, t, 9, into=x[:1].expand(9, 64)), lambda: plain.embed_grad(x, t, 4, into=x)):
        with pytest.raises(nat.CkksError):
            call()
