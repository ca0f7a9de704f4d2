"""Cases of further plaintext-side operators: a token's way in and out of an
encrypted decoder, and the heads between its projections and its attention.

- embed: rows of a table by token, scaled (the key holder's embedding before
         encryption); the table's gradient, summed by sorted tokens
- heads: norms of queries and keys for each head, and the rotation by position
         in the same pass; forward and gradient
- score: log probabilities of given tokens, entropy, the largest alternatives;
         forward, and forward with the logits' gradient

Where `own` is false `run` computes them from elementary torch operations in
32 bits (angles in 64); where it is true it calls the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4, "i8": 1}
EPS = 1e-6
ROW = 128            # rows of an 8-bit table start at multiples of this many bytes, zeros behind the last column
BASE = 1e6           # rotation frequencies BASE^(-2 i / rotary)


def listed():
    emb = dict(op="embed", backward=False, scale=1.0, padding=0.0)
    heads = dict(op="heads", backward=False, interleaved=False, q_norm=True, k_norm=True, far=0)
    score = dict(op="score", backward=False, top=0, masked=False, tempered=False, pad=0)
    return [
        # the tokens of one hop, before their encryption: latency alone
        dict(emb, name="embed 4 tokens", rows=4, vocab=32768, cols=2048, type="bf16", out="bf16"),
        # a long prompt over a large vocabulary, rows scaled by the root of their width
        dict(emb, name="embed prompt", rows=16384, vocab=131072, cols=4096, type="bf16", out="bf16", scale=64.0),
        # the vocabulary's 8-bit weights as the table (tied weights), nothing a multiple of anything, padded rows
        dict(emb, name="embed ragged 8-bit", rows=4099, vocab=50021, cols=5003, type="i8", out="f32", padding=0.1),
        # training step: the table's gradient of 8 sequences of 2048 tokens
        dict(emb, name="embed gradient", rows=16384, vocab=32768, cols=2048, type="bf16", out="f32", backward=True),
        # the same with odd sizes, scaled, a batch with padding, in 16 bits
        dict(emb, name="embed gradient ragged", rows=8191, vocab=20011, cols=2051, type="f16", out="f16", backward=True,
             scale=0.5, padding=0.2),
        # one hop's queries and keys (a 2048-wide hidden state in heads of 128): latency alone
        dict(heads, name="heads 4 tokens", tokens=4, q_heads=16, k_heads=8, dim=128, rotary=128, type="bf16"),
        # a long prompt's, out of the joint projection's rows, far into a sequence
        dict(heads, name="heads prompt", tokens=8192, q_heads=32, k_heads=8, dim=128, rotary=128, type="bf16",
             far=1000000),
        # training step of the same heads
        dict(heads, name="heads gradient", tokens=8192, q_heads=32, k_heads=8, dim=128, rotary=128, type="bf16",
             backward=True),
        # what was said by the tokens drawn, with the usual few alternatives, for one hop: latency alone
        dict(score, name="score 4 tokens", rows=4, vocab=32768, type="f32", top=5),
        # a prompt's tokens under a large vocabulary
        dict(score, name="score prompt", rows=2048, vocab=131072, type="bf16", top=20),
        # training step: log probabilities of the next tokens with an entropy bonus, and the logits' gradient
        dict(score, name="score gradient", rows=4096, vocab=32768, type="bf16", backward=True),
        # constrained decoding with temperatures and its gradient; odd sizes, rows of a wider buffer, rows without a
        # possible token
        dict(score, name="score masked gradient", rows=333, vocab=50021, type="f16", top=20, masked=True, tempered=True,
             pad=27, backward=True),
    ]


def _size(rng, low, high):
    """A size in [low, high], spread over its logarithm: a power of two, or an odd number."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    if rng.random() < 0.4:
        return min(high, max(low, 1 << round(math.log2(v))))
    return min(high, max(low, int(v) | 1))


def draw(rng):
    pick = rng.choice
    op = pick(["embed", "embed", "heads", "heads", "score", "score"])
    backward = rng.random() < 0.5
    if op == "embed":
        cols = _size(rng, 64, 8192)
        vocab = _size(rng, 1000, min(131072, (1 << (26 if backward else 28)) // cols))
        rows = _size(rng, 1, min(32768, (1 << 25) // cols))
        kind = pick(["bf16", "f16", "f32"] if backward else ["bf16", "f16", "f32", "i8"])
        return dict(op=op, backward=backward, rows=rows, vocab=vocab, cols=cols, type=kind,
                    out=pick(["bf16", "f16", "f32"]), scale=pick([1.0, 0.5, math.sqrt(cols)]), padding=pick([0.0, 0.2]))
    if op == "heads":
        dim = pick([32, 64, 64, 72, 80, 96, 128, 128, 128, 192, 256])
        k_heads = pick([0, 1, 2, 4, 8, 8, 16])
        q_heads = pick([1, 2, 3, 4, 7, 8]) * max(1, k_heads)
        while q_heads > 64:
            q_heads //= 2
        tokens = _size(rng, 1, min(16384, (1 << 25) // ((q_heads + k_heads) * dim)))
        return dict(op=op, backward=backward, tokens=tokens, q_heads=q_heads, k_heads=k_heads, dim=dim,
                    rotary=pick([dim, dim, dim // 2]), type=pick(["bf16", "bf16", "f16", "f32"]),
                    interleaved=rng.random() < 0.3, q_norm=rng.random() < 0.8, k_norm=rng.random() < 0.8,
                    far=pick([0, 100000, 4000000]))
    vocab = _size(rng, 1000, 262144)
    rows = _size(rng, 1, min(4096, (1 << (26 if backward else 27)) // vocab))
    return dict(op=op, backward=backward, rows=rows, vocab=vocab, type=pick(["bf16", "bf16", "f16", "f32"]),
                top=pick([0, 1, 5, 20, 64]), masked=rng.random() < 0.3, tempered=rng.random() < 0.4,
                pad=pick([0, 0, 27]))


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(v, dtype, pad):
    """v as rows of a buffer that is `pad` columns wider."""
    if not pad:
        return v.to(dtype)
    buf = torch.zeros(v.shape[0], v.shape[1] + pad, device="cuda", dtype=dtype)
    buf[:, :v.shape[1]] = v
    return buf[:, :v.shape[1]]


def _tokens(g, rows, vocab, padding):
    """Tokens of text: the r-th most frequent about as likely as 1 / r, spread over the vocabulary; -1 where a batch
    is padded."""
    rank = torch.exp(_rand(g, rows).double() * math.log(vocab)).long().clamp_(1, vocab) - 1
    t = (rank * 7919 + 13) % vocab
    if padding:
        t[_rand(g, rows) < padding] = -1
    return t


def _prepare_embed(g, c):
    T, V, D = c["rows"], c["vocab"], c["cols"]
    s = {"tokens": _tokens(g, T, V, c["padding"])}
    if c["backward"]:
        s["drows"] = (_randn(g, T, D) * 1e-2).to(TYPES[c["type"]])
    elif c["type"] == "i8":
        s["table"] = torch.zeros(V, -(-D // ROW) * ROW, device="cuda", dtype=torch.int8)
        s["table"][:, :D] = (_randn(g, V, D) * 32).round_().clamp_(-127, 127).to(torch.int8)
        s["table_scale"] = (0.5 + _rand(g, V)) / (32 * math.sqrt(D))
    else:
        s["table"] = (_randn(g, V, D) * 0.02).to(TYPES[c["type"]])
    return s


def _prepare_heads(g, c):
    T, Q, K, d, dt = c["tokens"], c["q_heads"], c["k_heads"], c["dim"], TYPES[c["type"]]
    # a joint projection's rows: queries, keys, values
    joint = _randn(g, T, (Q + 2 * K) * d) * 2 + 0.3 * _randn(g, 1, (Q + 2 * K) * d)
    joint = joint.to(dt)
    s = {"q": joint[:, :Q * d].view(T, Q, d), "k": joint[:, Q * d:(Q + K) * d].view(T, K, d) if K else None}
    s["q_weight"] = (1 + 0.1 * _randn(g, d)).to(dt) if c["q_norm"] else None
    s["k_weight"] = (1 + 0.1 * _randn(g, d)).to(dt) if K and c["k_norm"] else None
    # sequences packed one behind the other, each from a position of its own on
    length = max(1, T // 3)
    start = (_rand(g, 4).double() * (c["far"] + 1)).long()
    at = torch.arange(T, device="cuda")
    s["positions"] = start[at // length] + at % length
    r = c["rotary"] // 2
    s["inv_freq"] = (BASE ** (-torch.arange(r, device="cuda", dtype=torch.float64) / r)).float()
    if c["backward"]:
        s["dq"] = (_randn(g, T, Q, d) * 1e-2).to(dt)
        s["dk"] = (_randn(g, T, K, d) * 1e-2).to(dt) if K else None
    return s


def _prepare_score(g, c):
    B, V = c["rows"], c["vocab"]
    s = {"logits": _rows(_randn(g, B, V).mul_(2.5), TYPES[c["type"]], c["pad"])}
    s["tokens"] = (_rand(g, B).double() * V).long().clamp_(max=V - 1)
    if B >= 8:
        s["tokens"][B // 8::8] = -1          # rows behind a sequence's end
    s["allowed"], s["temperature"] = None, None
    if c["masked"]:
        s["allowed"] = _rand(g, B, V) < 0.3
        s["allowed"][torch.arange(B, device="cuda"), s["tokens"].clamp(min=0)] = True
        s["allowed"][B // 2::5] = _rand(g, len(range(B // 2, B, 5)), V) < 0.3  # what was said need not be allowed
        s["allowed"][B // 3::7] = False      # requests that may say nothing
    if c["tempered"]:
        s["temperature"] = 0.6 + 0.8 * _rand(g, B)
        s["temperature"][B // 5::9] = 0.0    # greedy requests: scored at temperature 1
    if c["backward"]:
        s["dlogprob"] = -_rand(g, B)
        s["dentropy"] = -0.01 * _rand(g, B)
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    make = {"embed": _prepare_embed, "heads": _prepare_heads, "score": _prepare_score}[case["op"]]
    return dict(make(g, case), case=dict(case))


# ------------------------------------------------------------------ plain forms, 32 bits

def _plain_embed(s):
    c, t = s["case"], s["tokens"]
    some = (t >= 0) & (t < c["vocab"])
    at = torch.where(some, t, torch.zeros_like(t))
    if c["backward"]:
        rows = torch.where(some[:, None], s["drows"].float() * c["scale"], torch.zeros((), device=t.device))
        grad = torch.zeros(c["vocab"], c["cols"], device=t.device, dtype=torch.float32)
        return {"table": grad.index_add_(0, at, rows).to(TYPES[c["out"]])}
    rows = s["table"][at][:, :c["cols"]].float()
    rows = rows * (c["scale"] * s["table_scale"][at][:, None]) if c["type"] == "i8" else rows * c["scale"]
    return {"rows": torch.where(some[:, None], rows, torch.zeros_like(rows)).to(TYPES[c["out"]])}


def _turned(x, cos, sin, interleaved):
    """x [T, H, d] with its first 2 r dimensions turned in r planes; cos, sin: [T, 1, r]"""
    r = cos.shape[-1]
    head, rest = x[..., :2 * r], x[..., 2 * r:]
    a, b = (head[..., 0::2], head[..., 1::2]) if interleaved else (head[..., :r], head[..., r:])
    a, b = a * cos - b * sin, b * cos + a * sin
    head = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([head, rest], -1)


def _plain_heads(s):
    c = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        x, w = s[name].float(), s[name + "_weight"]
        dt = s[name].dtype
        hat = x
        if w is not None:
            r = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
            hat = x * r
        if not c["backward"]:
            y = hat if w is None else hat * w.float()
            out[name] = _turned(y, cos, sin, c["interleaved"]).to(dt)
            continue
        dy = _turned(s["d" + name].float(), cos, -sin, c["interleaved"])
        if w is not None:
            out[name + "_weight"] = (dy * hat).sum((0, 1))
            a = dy * w.float()
            dy = r * (a - hat * (a * hat).mean(-1, keepdim=True))
        out["d" + name] = dy.to(dt)
    return out


def _plain_score(s):
    c = s["case"]
    z = s["logits"].float()
    B, V = z.shape
    valid = z > -math.inf
    if s["allowed"] is not None:
        valid = valid & s["allowed"]
    z = torch.where(valid, z, torch.full_like(z, -math.inf))
    t = torch.ones(B, 1, device=z.device) if s["temperature"] is None else s["temperature"][:, None]
    t = torch.where(t > 0, t, torch.ones_like(t))
    top = z.amax(1, keepdim=True)
    some = top > -math.inf
    d = torch.where(valid & some, (z - top) / t, torch.zeros_like(z))
    e = torch.where(valid, torch.exp(d), torch.zeros_like(z))
    mass = e.sum(1, keepdim=True)
    log_mass = torch.log(mass)
    p = torch.where(some, e / mass, torch.zeros_like(e))
    logp = torch.where(valid, d - log_mass, torch.zeros_like(d))
    entropy = -(p * logp).sum(1, keepdim=True)
    token = s["tokens"][:, None]
    given = (token >= 0) & (token < V)
    at = torch.where(given, token, torch.zeros_like(token))
    possible = given & valid.gather(1, at)
    logprob = torch.where(possible, logp.gather(1, at), torch.full_like(top, -math.inf))
    logprob = torch.where(given, logprob, torch.zeros_like(logprob))
    out = {"logprob": logprob[:, 0], "entropy": entropy[:, 0], "largest": top[:, 0], "log_mass": log_mass[:, 0]}
    if c["top"]:
        best, index = torch.sort(z, dim=1, descending=True, stable=True)
        best, index = best[:, :c["top"]], index[:, :c["top"]]
        there = best > -math.inf
        out["top_token"] = torch.where(there, index, torch.full_like(index, -1))
        out["top_logprob"] = torch.where(there, (best - top) / t - log_mass, torch.full_like(best, -math.inf))
    if c["backward"]:
        dl = torch.where(possible, s["dlogprob"][:, None], torch.zeros_like(top))
        g = -p * (dl + s["dentropy"][:, None] * (logp + entropy))
        g = g.scatter_add_(1, at, dl)
        out["dlogits"] = torch.where(valid, g / t, torch.zeros_like(g)).to(s["logits"].dtype)
    return out


def _own_score(s):
    from rns_ckks_polynomial_amd import plain
    c = s["case"]
    how = dict(temperature=s["temperature"], allowed=s["allowed"])
    r = plain.token_logprobs(s["logits"], s["tokens"], top=c["top"], **how)
    out = {"logprob": r.logprob, "entropy": r.entropy, "largest": r.largest, "log_mass": r.log_mass}
    if c["top"]:
        out["top_token"], out["top_logprob"] = r.top_token, r.top_logprob
    if c["backward"]:
        out["dlogits"] = plain.token_logprobs_grad(s["logits"], s["tokens"], r, s["dlogprob"], s["dentropy"], **how)
    return out


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"embed": _plain_embed, "heads": _plain_heads, "score": _plain_score}[c["op"]](s)
    from rns_ckks_polynomial_amd import plain
    if c["op"] == "embed":
        dt = TYPES[c["out"]]
        if c["backward"]:
            return {"table": plain.embed_grad(s["drows"], s["tokens"], c["vocab"], scale=c["scale"], dtype=dt)}
        table = plain.Int8Rows(s["table"], s["table_scale"], c["cols"]) if c["type"] == "i8" else s["table"]
        return {"rows": plain.embed(s["tokens"], table, scale=c["scale"], dtype=dt)}
    if c["op"] == "heads":
        how = dict(q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, interleaved=c["interleaved"])
        if c["backward"]:
            r = plain.head_norm_rotate_grad(s["q"], s["k"], s["dq"], s["dk"], s["positions"], s["inv_freq"], **how)
            return {k: v for k, v in r._asdict().items() if v is not None}
        q, k = plain.head_norm_rotate(s["q"], s["k"], s["positions"], s["inv_freq"], **how)
        return {"q": q} if k is None else {"q": q, "k": k}
    return _own_score(s)


# ------------------------------------------------------------------ bytes and operations

def work(case):
    c = case
    if c["op"] == "embed":
        T, V, D = c["rows"], c["vocab"], c["cols"]
        if c["backward"]:  # every row of the table's gradient is written, those of other tokens as zeros
            return {"bytes": T * (D * SIZE[c["type"]] + 8) + V * D * SIZE[c["out"]], "flops": 2 * T * D}
        return {"bytes": T * (D * (SIZE[c["type"]] + SIZE[c["out"]]) + 8 + (4 if c["type"] == "i8" else 0)),
                "flops": T * D}
    if c["op"] == "heads":
        n, b = c["tokens"] * (c["q_heads"] + c["k_heads"]) * c["dim"], SIZE[c["type"]]
        weights = c["dim"] * (c["q_norm"] + (c["k_norm"] if c["k_heads"] else 0))
        moved = (3 if c["backward"] else 2) * n * b + weights * (b + (4 if c["backward"] else 0))
        return {"bytes": moved + 8 * c["tokens"] + 2 * c["rotary"], "flops": (14 if c["backward"] else 7) * n}
    n, b = c["rows"] * c["vocab"], SIZE[c["type"]]
    moved = n * (b * (2 if c["backward"] else 1) + (1 if c["masked"] else 0))
    return {"bytes": moved + c["rows"] * (24 + 12 * c["top"] + (8 if c["backward"] else 0) + (4 if c["tempered"] else 0)),
            "flops": (14 if c["backward"] else 6) * n}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_embed(s):
    """Token by token: sorted tokens and differences of running sums would lose digits, so each distinct token's rows
    are added by one matrix of zeros and ones a block of tokens."""
    c = s["case"]
    T, V, D = c["rows"], c["vocab"], c["cols"]
    t = s["tokens"]
    if not c["backward"]:
        out = torch.zeros(T, D, device=t.device, dtype=torch.float64)
        have = torch.nonzero((t >= 0) & (t < V))[:, 0]
        factor = torch.full((have.numel(), 1), float(c["scale"]), device=t.device, dtype=torch.float64)
        if c["type"] == "i8":
            factor = factor * s["table_scale"].to(torch.float64)[t[have], None]
        out[have] = s["table"][t[have], :D].to(torch.float64) * factor
        return {"rows": out}
    out = torch.zeros(V, D, device=t.device, dtype=torch.float64)
    drows = s["drows"].to(torch.float64)
    kinds, kind_of = torch.unique(t, return_inverse=True)
    for first in range(0, kinds.numel(), 2048):
        last = min(first + 2048, kinds.numel())
        rows = torch.nonzero((kind_of >= first) & (kind_of < last))[:, 0]
        here = torch.zeros(last - first, rows.numel(), device=t.device, dtype=torch.float64)
        here[kind_of[rows] - first, torch.arange(rows.numel(), device=t.device)] = c["scale"]
        sums, ids = torch.mm(here, drows[rows]), kinds[first:last]
        good = (ids >= 0) & (ids < V)
        out[ids[good]] = sums[good]
    return {"table": out}


def _exact_heads(s):
    """Each pair of dimensions as one complex number: the rotation is a product with exp(i angle)."""
    c = s["case"]
    r = c["rotary"] // 2
    phase = s["positions"].to(torch.float64).outer(s["inv_freq"].to(torch.float64))
    unit = torch.polar(torch.ones_like(phase), phase)[:, None, :]
    dev = unit.device
    first = torch.arange(r, device=dev) * 2 if c["interleaved"] else torch.arange(r, device=dev)
    second = first + 1 if c["interleaved"] else first + r
    out = {}
    for name in ("q", "k"):
        if s[name] is None:
            continue
        x = s[name].to(torch.float64)
        w = s[name + "_weight"]
        d = x.shape[-1]
        size = torch.ones_like(x[..., :1])
        if w is not None:
            size = torch.sqrt(torch.linalg.vecdot(x, x)[..., None] / d + EPS)

        def turn(v, by):
            pair = torch.complex(v[..., first], v[..., second]) * by
            v = v.clone()
            v[..., first], v[..., second] = pair.real, pair.imag
            return v

        if not c["backward"]:
            out[name] = turn(x / size * (1.0 if w is None else w.to(torch.float64)), unit)
            continue
        dy = turn(s["d" + name].to(torch.float64), unit.conj())
        if w is not None:
            out[name + "_weight"] = torch.mm((x / size * dy).reshape(-1, d).t(),
                                             torch.ones(dy.shape[0] * dy.shape[1], 1, device=dev,
                                                        dtype=torch.float64))[:, 0]
            up = dy * w.to(torch.float64)
            dy = up / size - x * (torch.linalg.vecdot(up, x)[..., None] / (d * size ** 3))
        out["d" + name] = dy
    return out


def _exact_score(s):
    c = s["case"]
    B, V = c["rows"], c["vocab"]
    dev = s["logits"].device
    whole = lambda *n: torch.empty(*n, device=dev, dtype=torch.float64)  # noqa: E731
    out = {"logprob": whole(B), "entropy": whole(B), "largest": whole(B), "log_mass": whole(B)}
    if c["top"]:
        out["top_token"] = torch.full((B, c["top"]), -1, device=dev, dtype=torch.int64)
        out["top_logprob"] = torch.full((B, c["top"]), -math.inf, device=dev, dtype=torch.float64)
    if c["backward"]:
        out["dlogits"] = whole(B, V)
    step = max(1, (1 << 25) // V)
    for b in range(0, B, step):
        z = s["logits"][b:b + step].to(torch.float64)
        n = z.shape[0]
        no = torch.isnan(z) | (z == -math.inf)
        if s["allowed"] is not None:
            no |= ~s["allowed"][b:b + step]
        t = torch.ones(n, device=dev, dtype=torch.float64)
        if s["temperature"] is not None:
            t = s["temperature"][b:b + step].to(torch.float64)
            t = torch.where(t > 0, t, 1.0)
        z = z.masked_fill(no, -math.inf)
        top = z.max(1).values
        silent = top == -math.inf
        u = ((z - torch.where(silent, 0.0, top)[:, None]) / t[:, None])
        log_mass = torch.logsumexp(u, 1)
        lp = u - torch.where(silent, 0.0, log_mass)[:, None]
        p = torch.exp(lp)
        plogp = (p * lp).masked_fill(no, 0.0)
        out["entropy"][b:b + n] = -plogp.sum(1)
        out["largest"][b:b + n], out["log_mass"][b:b + n] = top, log_mass
        token = s["tokens"][b:b + step]
        inside = (token >= 0) & (token < V)
        row = torch.arange(n, device=dev)
        at = token.clamp(0, V - 1)
        out["logprob"][b:b + n] = torch.where(inside, lp[row, at], 0.0)
        if c["top"]:
            order = torch.argsort(z, dim=1, descending=True, stable=True)[:, :c["top"]]
            value = lp.gather(1, order)
            out["top_token"][b:b + n, :order.shape[1]] = torch.where(value == -math.inf, -1, order)
            out["top_logprob"][b:b + n, :order.shape[1]] = value
        if c["backward"]:
            dl = torch.where(inside & ~no[row, at], s["dlogprob"][b:b + step].to(torch.float64), 0.0)
            dh = s["dentropy"][b:b + step].to(torch.float64)
            # d logprob / d z = (one at the token - p) / t, d entropy / d z = -(p log p - p sum p log p) / t
            g = -dl[:, None] * p - dh[:, None] * (plogp - p * plogp.sum(1, keepdim=True))
            g[row, at] += dl
            out["dlogits"][b:b + n] = (g / t[:, None]).masked_fill(no, 0.0)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "heads": _exact_heads, "score": _exact_score}[case["op"]](s)
