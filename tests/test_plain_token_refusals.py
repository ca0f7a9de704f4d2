"""The C entry points of embedding, heads and log probabilities refuse what they
do not take, with the documented code and before any launch (so this runs
without a GPU: the addresses below are never followed)."""
import ctypes as C

import pytest

from rns_ckks_polynomial_amd import _native as nat

INV, ALIGN, UNSUP, WS = nat.EINVAL, nat.EALIGN, nat.EUNSUPPORTED, nat.EWORKSPACE
X, Y, H, U, W, G, Q, S, WSP = (0x10000000 * (i + 1) for i in range(9))
T, V, D = 8, 100, 64

EMB = dict(type=0, table=X, table_stride=D, vocab=V, cols=D, tokens=Y, rows=T, scale=1.0, out_type=0, out=H, out_stride=D)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INV), (dict(type=-1), INV), (dict(out_type=3), INV), (dict(table=None), INV), (dict(tokens=None), INV),
    (dict(out=None), INV), (dict(table_stride=D - 1), INV), (dict(out_stride=D - 1), INV), (dict(vocab=0), INV),
    (dict(cols=0), INV), (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(vocab=(1 << 24) + 1), UNSUP),
    (dict(cols=1 << 31, table_stride=1 << 31, out_stride=1 << 31), UNSUP), (dict(table=X + 1), ALIGN),
    (dict(tokens=Y + 4), ALIGN), (dict(out=H + 1), ALIGN), (dict(out=X), INV), (dict(out=X + 2 * D * (V - 1)), INV),
    (dict(out=Y + 8), INV),
])
def test_embed_arguments(kw, code):
    assert nat.lib().ckks_plain_embed(*{**EMB, **kw}.values(), None) == code


EMB8 = dict(q=X, q_stride=128, q_scale=W, vocab=V, cols=D, tokens=Y, rows=T, scale=1.0, out_type=0, out=H, out_stride=D)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(q_scale=None), INV), (dict(q_stride=64), INV), (dict(q_stride=192), INV),
    (dict(cols=129), INV), (dict(q=X + 8), ALIGN), (dict(q_scale=W + 2), ALIGN), (dict(out=W), INV), (dict(out=X + 128), INV),
    (dict(out_type=7), INV), (dict(tokens=None), INV),
])
def test_embed_i8_arguments(kw, code):
    assert nat.lib().ckks_plain_embed_i8(*{**EMB8, **kw}.values(), None) == code


EG = dict(type=0, drows=X, drows_stride=D, tokens=Y, rows=T, vocab=V, cols=D, scale=1.0, out_type=2, out=H, out_stride=D,
          add=0, ws=WSP, ws_bytes=1 << 24)


@pytest.mark.parametrize("add", [0, 1])
@pytest.mark.parametrize("kw,code", [
    (dict(type=3), INV), (dict(out_type=-1), INV), (dict(drows=None), INV), (dict(tokens=None), INV), (dict(out=None), INV),
    (dict(drows_stride=D - 1), INV), (dict(out_stride=D - 1), INV), (dict(vocab=0), INV), (dict(cols=0), INV),
    (dict(rows=-1), INV), (dict(vocab=(1 << 24) + 1), UNSUP), (dict(drows=X + 1), ALIGN), (dict(tokens=Y + 4), ALIGN),
    (dict(out=H + 2), ALIGN), (dict(out=X), INV), (dict(out=Y), INV), (dict(ws=X), INV), (dict(ws=Y), INV), (dict(ws=H), INV),
    (dict(ws=None), WS), (dict(ws_bytes=16), WS), (dict(ws=WSP + 8), ALIGN),
])
def test_embed_grad_arguments(kw, code, add):
    assert nat.lib().ckks_plain_embed_grad(*{**EG, "add": add, **kw}.values(), None) == code


def test_embed_grad_workspace():
    lib, n = nat.lib(), C.c_size_t()
    for rows in (T, 1000, 100000):
        assert lib.ckks_plain_embed_grad_workspace_size(rows, V, D, C.byref(n)) == 0 and n.value >= 4 * rows + 4 * V
        far = {"out": 1 << 50, "ws": 1 << 55}
        assert lib.ckks_plain_embed_grad(*{**EG, **far, "rows": rows, "ws_bytes": n.value - 1}.values(), None) == WS
    assert lib.ckks_plain_embed_grad_workspace_size(T, V, D, None) == INV
    assert lib.ckks_plain_embed_grad_workspace_size(T, 0, D, C.byref(n)) == INV


def at(what, token, head):
    return {f"{what}_token_stride": token, f"{what}_head_stride": head}


def heads(**kw):
    f = dict(type=0, interleaved=0, tokens=T, q_heads=4, k_heads=2, head_dim=D, rotary=D, q=X, k=Y,
             **at("q", 6 * D, D), **at("k", 6 * D, D), q_weight=W, k_weight=W + 4096, positions=G,
             inv_freq=S, eps=1e-6)
    f.update(kw)
    return nat.PlainHeads(**f)


BAD_HEADS = [
    (dict(type=3), INV), (dict(interleaved=2), INV), (dict(tokens=-1), INV), (dict(tokens=1 << 31), INV),
    (dict(q_heads=0), INV), (dict(k_heads=-1), INV), (dict(k_heads=0), INV), (dict(head_dim=0), INV),
    (dict(head_dim=63, rotary=62), UNSUP), (dict(rotary=63), UNSUP), (dict(rotary=66), INV), (dict(rotary=-2), INV),
    (dict(head_dim=514, **at("q", 1 << 15, 514), **at("k", 1 << 15, 514)), UNSUP),
    (dict(q_heads=65536), UNSUP), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(q=None), INV),
    (dict(k=None), INV), (dict(positions=None), INV), (dict(inv_freq=None), INV), (at("q", D - 1, D), INV),
    (at("k", 6 * D, D - 1), INV), (dict(q=X + 1), ALIGN), (dict(k=Y + 1), ALIGN),
    (dict(q_weight=W + 1), ALIGN), (dict(positions=G + 4), ALIGN), (dict(inv_freq=S + 2), ALIGN),
]
OUT = (H, 4 * D, D, U, 2 * D, D)


@pytest.mark.parametrize("kw,code", BAD_HEADS)
def test_heads_arguments(kw, code):
    lib, p = nat.lib(), heads(**kw)
    assert lib.ckks_plain_head_norm_rotate(C.byref(p), *OUT, None) == code
    g = nat.PlainHeadGrads(X + (1 << 27), Y + (1 << 27), 6 * 512, 512, 6 * 512, 512, H, U, 4 * 512, 512, 2 * 512, 512, Q,
                           Q + 4096)
    assert lib.ckks_plain_head_norm_rotate_grad(C.byref(p), C.byref(g), WSP, 1 << 20, None) == code


@pytest.mark.parametrize("out,code", [
    ((None, *OUT[1:]), INV), ((H, D, D, *OUT[3:]), INV), ((H, 4 * D, D - 1, *OUT[3:]), INV),
    ((H, 4 * D - 1, D, *OUT[3:]), INV), ((H + 1, *OUT[1:]), ALIGN), ((X, *OUT[1:]), INV), ((Y, *OUT[1:]), INV),
    ((*OUT[:3], H, *OUT[4:]), INV), ((W, *OUT[1:]), INV), ((G, *OUT[1:]), INV), ((S, *OUT[1:]), INV),
    ((*OUT[:3], None, *OUT[4:]), INV), ((*OUT[:3], Y, *OUT[4:]), INV), ((*OUT[:3], U + 1, *OUT[4:]), ALIGN),
])
def test_heads_outputs(out, code):
    p = heads()
    assert nat.lib().ckks_plain_head_norm_rotate(C.byref(p), *out, None) == code


def test_heads_beside_each_other_in_rows():
    """Parts of joint rows are apart where no element is shared, and not where one is (no tokens: nothing is launched;
    the pairs of ranges are looked at for two tokens and more, so by way of an error behind them: a workspace)."""
    lib = nat.lib()
    row = 8 * D * 2  # bytes of a token of 4 + 2 + 2 heads
    joint = dict(q=X, k=X + 4 * D * 2, **at("q", 8 * D, D), **at("k", 8 * D, D))
    p = heads(**joint)
    def grad(dq_in, dk_in, token=8 * D, **kw):
        g = nat.PlainHeadGrads(**{**HG, "dq_in": dq_in, "dk_in": dk_in, **at("dq_in", token, D), **at("dk_in", token, D), **kw})
        return lib.ckks_plain_head_norm_rotate_grad(C.byref(p), C.byref(g), None, 0, None)
    assert grad(H, H + 4 * D * 2) == WS                      # apart
    assert grad(H + 4 * D * 2, H) == WS                      # the other way round
    assert grad(H + 5 * D * 2, H) == INV                     # the queries' heads reach into the next token's keys
    assert grad(H, H + 3 * D * 2) == INV                     # the last query head is the first key
    assert grad(H, H + 7 * D * 2) == INV                     # the second key is the next token's first query
    assert grad(H, H + 4 * D * 2 + 5 * row) == WS            # rows further on
    assert grad(H + 5 * row, H + 4 * D * 2) == WS
    assert grad(X + 6 * D * 2, U) == INV                     # over the next token's queries
    # forward, into the values' place and over the other tensor
    call = lambda q, k: lib.ckks_plain_head_norm_rotate(C.byref(p), q, 8 * D, D, k, 8 * D, D, None)  # noqa: E731
    assert call(X, X) == INV and call(X + 4 * D * 2, U) == INV and call(H, X) == INV and call(X, X + 2 * D * 2) == INV


HG = dict(dq=X + (1 << 27), dk=Y + (1 << 27), **at("dq", 4 * D, D), **at("dk", 2 * D, D), dq_in=H, dk_in=U,
          **at("dq_in", 4 * D, D), **at("dk_in", 2 * D, D), q_weight=Q, k_weight=Q + 4096)


@pytest.mark.parametrize("kw,ws,code", [
    (dict(dq=None), WSP, INV), (dict(dk=None), WSP, INV), (dict(dq_in=None), WSP, INV), (dict(q_weight=None), WSP, INV),
    (dict(k_weight=None), WSP, INV), (at("dq", 1, D), WSP, INV), (dict(dq_in=X), WSP, INV),
    (dict(dq_in=X + (1 << 27)), WSP, INV), (dict(dk_in=H), WSP, INV), (dict(q_weight=H + 4), WSP, INV),
    (dict(k_weight=Q + 8), WSP, INV), (dict(q_weight=Q + 2), WSP, ALIGN), (at("dq_in", D, D), WSP, INV),
    ({}, None, WS), ({}, WSP + 4, ALIGN), ({}, H, INV), ({}, X, INV), ({}, Q, INV),
])
def test_heads_grad_arguments(kw, ws, code):
    p, g = heads(), nat.PlainHeadGrads(**{**HG, **kw})
    assert nat.lib().ckks_plain_head_norm_rotate_grad(C.byref(p), C.byref(g), ws, 1 << 20, None) == code


def test_heads_grad_workspace():
    lib, n, p = nat.lib(), C.c_size_t(), heads()
    assert lib.ckks_plain_head_grad_workspace_size(C.byref(p), C.byref(n)) == 0 and n.value > 0
    g = nat.PlainHeadGrads(**HG)
    assert lib.ckks_plain_head_norm_rotate_grad(C.byref(p), C.byref(g), WSP, n.value - 1, None) == WS
    assert lib.ckks_plain_head_norm_rotate_grad(C.byref(p), None, WSP, n.value, None) == INV
    assert lib.ckks_plain_head_grad_workspace_size(C.byref(p), None) == INV
    assert lib.ckks_plain_head_grad_workspace_size(None, C.byref(n)) == INV
    assert lib.ckks_plain_head_grad_workspace_size(C.byref(heads(q_weight=None, k_weight=None)), C.byref(n)) == 0
    assert n.value == 0


SC = dict(type=0, logits=X, logits_stride=V, tokens=Y, temperature=None, allowed=None, allowed_stride=0, rows=T, vocab=V,
          top=0, logprob=H, entropy=H + 4096, largest=H + 8192, log_mass=H + 12288, top_token=None, top_logprob=None, ws=WSP,
          ws_bytes=1 << 30)


@pytest.mark.parametrize("kw,code", [
    (dict(type=5), INV), (dict(logits=None), INV), (dict(tokens=None), INV), (dict(logits_stride=V - 1), INV),
    (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(vocab=0), INV), (dict(vocab=(1 << 24) + 1), UNSUP),
    (dict(top=-1), INV), (dict(top=65), UNSUP), (dict(top=3), INV), (dict(top_token=U), INV), (dict(top_logprob=U), INV),
    (dict(top=3, top_token=U), INV), (dict(logprob=None), INV), (dict(entropy=None), INV), (dict(largest=None), INV),
    (dict(log_mass=None), INV), (dict(allowed=G), INV), (dict(allowed=G, allowed_stride=V - 1), INV),
    (dict(logits=X + 1), ALIGN), (dict(tokens=Y + 4), ALIGN), (dict(temperature=W + 2), ALIGN), (dict(logprob=H + 2), ALIGN),
    (dict(top=1, top_token=U + 4, top_logprob=S), ALIGN), (dict(top=1, top_token=U, top_logprob=S + 2), ALIGN),
    (dict(logprob=X), INV), (dict(entropy=H), INV), (dict(largest=Y), INV), (dict(temperature=W, log_mass=W + 4), INV),
    (dict(allowed=G, allowed_stride=V, logprob=G), INV), (dict(top=2, top_token=U, top_logprob=U + 8), INV),
])
def test_score_arguments(kw, code):
    assert nat.lib().ckks_plain_token_logprobs(*{**SC, **kw}.values(), None) == code


def test_score_workspace():
    lib, n = nat.lib(), C.c_size_t()
    assert lib.ckks_plain_token_logprobs_workspace_size(T, V, 0, None) == INV
    assert lib.ckks_plain_token_logprobs_workspace_size(T, V, 65, C.byref(n)) == UNSUP
    assert lib.ckks_plain_token_logprobs_workspace_size(T, V, -1, C.byref(n)) == INV
    far = {"logits": 1 << 50, "ws": 1 << 55}
    for rows, vocab in ((1, V), (4, 131072), (1, 1 << 24), (5000, 1000)):
        assert lib.ckks_plain_token_logprobs_workspace_size(rows, vocab, 64, C.byref(n)) == 0
        if n.value:
            kw = {**SC, **far, "rows": rows, "vocab": vocab, "logits_stride": vocab, "ws_bytes": n.value - 1, "top": 64,
                  "top_token": U, "top_logprob": S}
            assert lib.ckks_plain_token_logprobs(*kw.values(), None) == WS
            assert lib.ckks_plain_token_logprobs(*{**kw, "ws": (1 << 55) + 8, "ws_bytes": n.value}.values(), None) == ALIGN
            assert lib.ckks_plain_token_logprobs(*{**kw, "ws": H}.values(), None) == INV


SG = dict(type=0, logits=X, logits_stride=V, tokens=Y, temperature=None, allowed=None, allowed_stride=0, rows=T, vocab=V,
          entropy=H, largest=H + 4096, log_mass=H + 8192, dlogprob=G, dentropy=G + 4096, dlogits=U, dlogits_stride=V)


@pytest.mark.parametrize("kw,code", [
    (dict(type=-1), INV), (dict(logits=None), INV), (dict(tokens=None), INV), (dict(entropy=None), INV),
    (dict(largest=None), INV), (dict(log_mass=None), INV), (dict(dlogits=None), INV), (dict(dlogits_stride=V - 1), INV),
    (dict(vocab=0), INV), (dict(vocab=(1 << 24) + 1), UNSUP), (dict(rows=-1), INV), (dict(dlogits=U + 1), ALIGN),
    (dict(entropy=H + 2), ALIGN), (dict(dlogprob=G + 1), ALIGN), (dict(dentropy=G + 2), ALIGN), (dict(dlogits=Y), INV),
    (dict(dlogits=X + 2), INV), (dict(dlogits=X), INV), (dict(dlogits=X, dlogits_stride=V + 1), INV), (dict(dlogits=H), INV), (dict(dlogits=G), INV),
    (dict(allowed=Q, allowed_stride=V, dlogits=Q), INV), (dict(allowed=Q), INV), (dict(temperature=S, dlogits=S), INV),
])
def test_score_grad_arguments(kw, code):
    assert nat.lib().ckks_plain_token_logprobs_grad(*{**SG, **kw}.values(), None) == code


def test_no_rows_is_valid():
    lib = nat.lib()
    assert lib.ckks_plain_embed(*{**EMB, "rows": 0, "table": None, "tokens": None, "out": None}.values(), None) == 0
    assert lib.ckks_plain_embed_grad(*{**EG, "rows": 0, "add": 1}.values(), None) == 0
    p = heads(tokens=0, q=None, k=None, positions=None)
    assert lib.ckks_plain_head_norm_rotate(C.byref(p), None, 0, 0, None, 0, 0, None) == 0
    assert lib.ckks_plain_token_logprobs(*{**SC, "rows": 0}.values(), None) == 0
    assert lib.ckks_plain_token_logprobs_grad(*{**SG, "rows": 0}.values(), None) == 0


def test_binding_wants_device_tensors():
    torch = pytest.importorskip("torch")
    from rns_ckks_polynomial_amd import plain
    x, t = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    for call in (lambda: plain.embed(t, x), lambda: plain.embed_grad(x, t, 4),
                 lambda: plain.head_norm_rotate(x[:, None], None, None, None), lambda: plain.token_logprobs(x, t),
                 lambda: plain.token_logprobs_grad(x, t, None)):
        with pytest.raises(ValueError, match="device tensor"):
            call()
