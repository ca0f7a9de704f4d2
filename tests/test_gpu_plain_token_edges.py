"""Embedding, heads and log probabilities (include/ckks_plain.h) where numbers,
layouts and uses are at the edge of what the calls take, against their
definitions in 64 bits (plain_token_ref).  Bounds as in test_gpu_plain_tokens."""
import numpy as np
import pytest

import plain_token_ref as ref
from gpu_util import require_gpu, say, torch
from rns_ckks_polynomial_amd import plain
from test_gpu_plain import EPS, TYPE, f64, rnd
from test_gpu_plain_tokens import check_embed_grad, check_score, head_inputs, host, ints, near, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()


# ------------------------------------------------------------------ log probabilities

@pytest.mark.parametrize("ty", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("temperature", [1e-45, 1e-38, 1e-37, 1e-36])
def test_gradient_at_tiny_temperatures(ty, temperature):
    """Rows whose largest logit is far above the others: p is 0 and 1, and the gradient 0, whatever 1 / temperature
    times its terms would be; and rows whose others are near it."""
    V = 5003
    z = -(1 + torch.rand(4, V, generator=torch.Generator().manual_seed(3)))
    at = torch.tensor([0, 17, V - 1, 2500])
    z[torch.arange(4), at] = torch.tensor([0.0, 0.0, 3.0, -0.5])
    z, tok = z.to(TYPE[ty]).cuda(), torch.where(torch.arange(4) == 2, 5, at).cuda()
    t = torch.full((4,), temperature, device="cuda")
    r = plain.token_logprobs(z, tok, 0, t)
    for dl in (None, 4.0, 50.0):
        for dh in (None, 1.0, -30.0):
            say(f"tiny {ty} {temperature} {dl} {dh}")
            each = lambda v: None if v is None else torch.full((4,), v, device="cuda")  # noqa: E731
            d = plain.token_logprobs_grad(z, tok, r, each(dl), each(dh), t)
            want = torch.zeros(4, V, dtype=torch.float64)
            if dl is not None:  # the third row's given token has p = 0, its largest p = 1
                want[2, 5], want[2, V - 1] = dl / max(temperature, 2.0 ** -127), -dl / max(temperature, 2.0 ** -127)
            # 1 / temperature and the product are rounded once each, then to the type; +-: infinite where it has no room
            low, high = ((want * (1 + s * 2.0 ** -22)).float().to(TYPE[ty]) for s in (-1, 1))
            d = d.cpu()
            assert ((d >= torch.minimum(low, high)) & (d <= torch.maximum(low, high))).all()
    near_ones = (rnd(5, 4, 300) * 2 * temperature).float().cuda()
    check_score(near_ones, ints(6, 4, 0, 300), 3, t)


@pytest.mark.parametrize("B,V", [(5, 300), (5, 70001)])
def test_distances_past_32_bits_and_infinite_temperatures(B, V):
    """Logits over the whole range at temperatures of its size, beside a NaN, and infinite ones at an infinite
    temperature; in slices too."""
    z = ((rnd(31, B, V).clamp(-3, 3)) * 1.1e38).float()
    z[1, V // 2] = float("nan")
    z[2, :V // 2], z[2, V // 2:] = 3e38, -3e38
    z[3, 7] = float("inf")
    z[4, 7] = z[4, V - 1] = float("inf")
    for t in (1e38, 3.4e38, float("inf")):
        say(f"distances {B}x{V} at {t}")
        r = plain.token_logprobs(z.cuda(), torch.tensor([0, 1, V - 1, 8, 7], device="cuda"), 4,
                                 torch.full((B,), t, device="cuda"))
        x = (z.double() - z.double().nan_to_num(-np.inf, np.inf).amax(1, keepdim=True)) / t
        x[3:] = -np.inf  # an infinite logit outweighs the finite ones
        x[3, 7] = x[4, 7] = x[4, V - 1] = 0
        x[x.isnan()] = -np.inf
        lp = torch.log_softmax(x, 1)
        bound = (V / 256 + 64 + 4 * 6 + 4 * np.log(V) + 4 * 24) * EPS  # |x| <= 6 / 1.1, and of log probabilities 24
        given = lp[torch.arange(B), torch.tensor([0, 1, V - 1, 8, 7])]
        for got, want in ((r.logprob, given), (r.log_mass, -lp.amax(1)), (r.top_logprob, lp.topk(4).values)):
            got = got.cpu().double()
            assert torch.equal(got == -np.inf, want == -np.inf)
            assert ((got - want).abs()[want > -np.inf] <= bound).all()
        entropy = -(lp.exp() * lp).nan_to_num(0).sum(1)
        assert ((r.entropy.cpu().double() - entropy).abs() <= bound * (1 + 2 * 6 + np.log(V))).all()


# ------------------------------------------------------------------ results and what autograd keeps of them

def some_scores(requires_grad=False):
    z = (rnd(41, 6, 700) * 2).float().cuda().requires_grad_(requires_grad)
    return z, on_gpu(ints(42, 6, -1, 700), torch.int64)


def test_results_are_tensors_of_their_own():
    """Writing to one result leaves what autograd holds of the others, and may be followed by it."""
    z, tok = some_scores()
    r = plain.token_logprobs(z, tok, 3)
    assert len({v.untyped_storage().data_ptr() for v in r}) == len(r) and not any(v._is_view() for v in r)
    w = torch.full((6,), 0.5, device="cuda", requires_grad=True)
    loss = (w * r.logprob).sum()
    kept = [v.clone() for v in r]
    r.entropy.add_(1)
    r.log_mass.zero_()
    loss.backward()
    assert torch.equal(w.grad, kept[0])
    w.grad = None
    r.largest.mul_(w)
    r.largest.sum().backward()
    assert torch.equal(w.grad, kept[4]) and torch.equal(r.logprob, kept[0])


def test_results_that_the_gradient_does_not_need_may_be_written():
    z, tok = some_scores(True)
    want, = torch.autograd.grad(plain.token_logprobs(z, tok, 3).logprob.neg().sum(), z)
    r = plain.token_logprobs(z, tok, 3)
    loss = r.logprob.neg_().sum()
    r.top_token.clamp_(min=0)
    with torch.no_grad():
        r.top_logprob.clamp_(min=-100)
    loss.backward()
    assert torch.equal(z.grad, want)


def test_heads_take_a_gradient_of_any_strides():
    """Rows of a gradient that share memory, as a window over a sequence gives them."""
    q, k = (rnd(43 + i, 7, 3, 64).to(torch.bfloat16).cuda().requires_grad_() for i in range(2))
    pos, freq = torch.arange(7, device="cuda"), torch.tensor([1.0, 0.3, 0.01], device="cuda")
    flat = rnd(45, 8192).to(torch.bfloat16).cuda()
    for strides in ((8, 64, 1), (192, 16, 1), (0, 64, 1), (1, 64, 64), (7, 5, 3)):
        say(f"gradient of strides {strides}")
        g = torch.as_strided(flat, (7, 3, 64), strides)
        want = plain.head_norm_rotate_grad(q.detach(), k.detach(), g.contiguous(), g.contiguous(), pos, freq)
        got = torch.autograd.grad(plain.head_norm_rotate(q, k, pos, freq), (q, k), (g, g))
        assert torch.equal(got[0], want.dq) and torch.equal(got[1], want.dk)


def test_heads_gradient_of_what_is_asked_for(monkeypatch):
    """Backward works on the queries or the keys alone where the other side is frozen, with the same results."""
    q, k, pos, freq, qw, kw = head_inputs(46, 40, 6, 2, 64, 32, "bf16")
    dq, dk = rnd(47, *q.shape).to(q.dtype).cuda(), rnd(48, *k.shape).to(k.dtype).cuda()
    whole = plain.head_norm_rotate_grad(q, k, dq, dk, pos, freq, qw, kw)
    heads, call = [], plain._call

    def record(name, device, p, *args):
        if name == "ckks_plain_head_norm_rotate_grad":
            heads.append((p._obj.q_heads, p._obj.k_heads))
        return call(name, device, p, *args)

    monkeypatch.setattr(plain, "_call", record)
    for frozen, worked in (((), (6, 2)), ((1, 3), (6, 0)), ((0, 2), (2, 0)), ((1,), (6, 2)), ((1, 2, 3), (6, 0)), ((0, 1, 2), (2, 0))):
        leaves = [v.detach().clone().requires_grad_(i not in frozen) for i, v in enumerate((q, k, qw, kw))]
        heads.clear()
        torch.autograd.backward(plain.head_norm_rotate(leaves[0], leaves[1], pos, freq, leaves[2], leaves[3]), (dq, dk))
        assert heads == [worked], frozen
        for i, (v, want) in enumerate(zip(leaves, whole)):
            if i in frozen:
                assert v.grad is None
            elif i < 2:
                assert torch.equal(v.grad, want)
            else:  # the terms may be added in another order: the bound of several steps, below
                x, dy = ((q, dq), (k, dk))[i - 2]
                _, _, b, bsize = ref.heads_grad(f64(x), f64(dy), f64((qw, kw)[i - 2]), host(pos), host(freq), 1e-6, False)
                near(v.grad, b, 256 * EPS * bsize, "weight")


# ------------------------------------------------------------------ sizes that take another form of a kernel

@pytest.mark.parametrize("T,Q,K,d,r,ty,interleaved,norm", [
    (4101, 32, 8, 128, 64, "bf16", False, True),   # 12 tokens a workgroup, four at a time; the last has 9
    (4101, 17, 2, 128, 48, "f32", True, True),     # 8, four at a time; the last has 5
    (5500, 6, 2, 64, 32, "f16", False, True),      # 20, ten at a time; the last has 20
    (5503, 6, 2, 64, 20, "bf16", True, True),      # the same; the last has 3
    (4101, 9, 40, 128, 64, "bf16", False, False),  # more heads of keys than of queries, no norm
])
def test_heads_gradient_of_workgroups_with_several_steps(T, Q, K, d, r, ty, interleaved, norm):
    """A workgroup's angles replaced between its steps, the next step's head fetched before, and the weights' sums
    carried over them.  A weight's sum adds up in a thread at most 60 terms (tokens times heads over groups of
    threads), 6 between lanes and 4 between waves, and of at most 1024 workgroups' 64 and 16: under 160 roundings, and
    each term is off by 96 eps as the gradient's are."""
    say(f"gradient of {T} x {Q} + {K} heads of {d} {ty}")
    q, k, pos, freq, qw, kw = head_inputs(71, T, Q, K, d, r, ty, norm)
    dq, dk = rnd(72, *q.shape).to(q.dtype).cuda(), rnd(73, *k.shape).to(k.dtype).cuda()
    got = plain.head_norm_rotate(q, k, pos, freq, qw, kw, 1e-6, interleaved)
    g = plain.head_norm_rotate_grad(q, k, dq, dk, pos, freq, qw, kw, 1e-6, interleaved)
    e = float(np.float32(1e-6))
    for x, w, y, dy, dx, dw in ((q, qw, got[0], dq, g.dq, g.q_weight), (k, kw, got[1], dk, g.dk, g.k_weight)):
        want, size = ref.heads(f64(x), f64(w), host(pos), host(freq), e, interleaved)
        near(y, want, 32 * EPS * size, "forward")
        a, asize, b, bsize = ref.heads_grad(f64(x), f64(dy), f64(w), host(pos), host(freq), e, interleaved)
        near(dx, a, 96 * EPS * asize, "gradient")
        if norm:
            near(dw, b, 256 * EPS * bsize, "weight")
    again = plain.head_norm_rotate_grad(q, k, dq, dk, pos, freq, qw, kw, 1e-6, interleaved)
    assert all(a is b or torch.equal(a, b) for a, b in zip(g, again))


@pytest.mark.parametrize("D", [1, 3, 7, 9, 2051, 2500, 3333, 4099, 9001])
@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("kind", ["text", "two", "one"])
def test_new_tables_gradient(D, out, kind):
    """Rows narrower than a vector and wider than 2048 columns in every type of the table, an odd number of rows of it
    (the last without a neighbour), tokens that do not occur, and runs of more rows than a chunk."""
    say(f"new table {D} {out} {kind}")
    check_embed_grad(151, 51, D, "bf16", out, kind, pad=3)
    check_embed_grad(67, 33, D, "f32", out, kind)
