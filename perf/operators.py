"""Cases of the plaintext-side operators: what the key holder of an encrypted
decoder computes in clear around it.

- norm:    residual stream + gated, optionally normalised block output, and the
           next block's norm; forward and gradient
- product: rows quantised to 8 bits times 8-bit weights with a scale for each channel
- project: norm with an 8-bit output feeding such a product (the decrypted
           hidden state on its way to the vocabulary)
- sample:  a token from logits by temperature, top-k, top-p and min-p

Where `own` is false `run` computes them from elementary torch operations in
32 bits; where it is true it calls the package.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
SCALE = 0.5          # residual scale of the norm cases
ROW = 128            # rows of 8-bit weights start at multiples of this many bytes, zeros behind the last column


def listed():
    norm = dict(op="norm", backward=False, bias=False, block=False, groups=0, pad=0)
    prod = dict(op="product", bias=False)
    samp = dict(op="sample", top_k=0, top_p=1.0, min_p=0.0, masked=False, pad=0)
    return [
        # one decrypted hop: 4 tokens of 2 x 1024 slots; latency alone
        dict(norm, name="norm 4 tokens", rows=4, cols=2048, type="bf16", kind="rms"),
        # a long prompt's residual stream, norm before and after the block and a gate for each channel
        dict(norm, name="norm prompt", rows=8192, cols=4096, type="bf16", kind="rms", block=True, groups=1),
        # ragged rows and columns, layer norm with biases, rows of a wider buffer
        dict(norm, name="norm ragged", rows=1021, cols=5003, type="f32", kind="layer", bias=True, block=True, pad=13),
        # training step of the same stream: 8 sequences, each with its own gate
        dict(norm, name="norm gradient", rows=16384, cols=2048, type="bf16", kind="rms", backward=True, block=True,
             groups=8),
        # the hop's hidden state through the final norm to the vocabulary
        dict(op="project", name="project 4 tokens", rows=4, cols=2048, channels=32768, type="bf16"),
        # one token to the vocabulary: reading the weights is all there is
        dict(prod, name="product token", rows=1, channels=32768, cols=2048, type="bf16", out="f32"),
        # a batch of decoding sequences through a wide projection
        dict(prod, name="product batch", rows=64, channels=8192, cols=8192, type="bf16", out="bf16"),
        # a prompt through the same projection: matrix cores alone
        dict(prod, name="product prompt", rows=8192, channels=8192, cols=8192, type="bf16", out="bf16"),
        # no size a multiple of anything
        dict(prod, name="product ragged", rows=777, channels=5003, cols=2051, type="f16", out="f16", bias=True),
        # one sequence's next token, the usual filters
        dict(samp, name="sample one", rows=1, vocab=32768, type="f32", top_k=50, top_p=0.95),
        # a batch over a large vocabulary, nucleus only
        dict(samp, name="sample batch", rows=256, vocab=131072, type="bf16", top_p=0.95),
        # constrained decoding: a mask of allowed tokens (some rows have none), min-p, logits in padded rows
        dict(samp, name="sample allowed", rows=33, vocab=50021, type="f16", min_p=0.05, top_k=1000, masked=True, pad=27),
    ]


def _size(rng, low, high):
    """A size in [low, high], spread over its logarithm: a power of two, or an odd number."""
    v = math.exp(rng.uniform(math.log(low), math.log(high)))
    if rng.random() < 0.4:
        return min(high, max(low, 1 << round(math.log2(v))))
    return min(high, max(low, int(v) | 1))


def draw(rng):
    op = rng.choice(["norm", "norm", "project", "product", "product", "sample", "sample"])
    pick = rng.choice
    if op == "norm":
        cols = _size(rng, 64, 8192)
        rows = _size(rng, 1, min(16384, (1 << 25) // cols))
        groups = pick([0, 1, 1, 2, 4])
        if groups:
            rows = max(groups, rows // groups * groups)
        kind = pick(["rms", "layer"])
        return dict(op=op, rows=rows, cols=cols, type=pick(["bf16", "bf16", "f16", "f32"]), kind=kind,
                    bias=kind == "layer" and rng.random() < 0.7, block=rng.random() < 0.6, groups=groups,
                    backward=rng.random() < 0.5, pad=pick([0, 0, 8, 13]))
    if op == "project":
        return dict(op=op, rows=_size(rng, 1, 64), cols=_size(rng, 512, 8192), channels=_size(rng, 512, 32768),
                    type=pick(["bf16", "f16"]))
    if op == "product":
        cols = _size(rng, 256, 8192)
        channels = _size(rng, 256, 32768)
        rows = _size(rng, 1, min(8192, (1 << 38) // (cols * channels)))
        return dict(op=op, rows=rows, channels=channels, cols=cols, type=pick(["bf16", "f16", "f32"]),
                    out=pick(["bf16", "f16", "f32"]), bias=rng.random() < 0.5)
    vocab = _size(rng, 1000, 262144)
    rows = _size(rng, 1, min(256, (1 << 25) // vocab))
    return dict(op=op, rows=rows, vocab=vocab, type=pick(["bf16", "f16", "f32"]), top_k=pick([0, 0, 1, 20, 50, 1000]),
                top_p=pick([1.0, 0.5, 0.9, 0.95]), min_p=pick([0.0, 0.0, 0.02, 0.1]), masked=rng.random() < 0.3,
                pad=pick([0, 0, 27]))


# ------------------------------------------------------------------ inputs

def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _rows(v, dtype, pad):
    """v as rows of a buffer that is `pad` columns wider."""
    if not pad:
        return v.to(dtype)
    buf = torch.zeros(v.shape[0], v.shape[1] + pad, device="cuda", dtype=dtype)
    buf[:, :v.shape[1]] = v
    return buf[:, :v.shape[1]]


def _norm_inputs(g, c):
    T, D, dt = c["rows"], c["cols"], TYPES[c["type"]]
    s = {"x": _rows(_randn(g, T, D) * 2 + _randn(g, 1, D), dt, c.get("pad", 0)),
         "y": _rows(_randn(g, T, D) + 0.1 * _randn(g, T, 1), dt, c.get("pad", 0))}
    p = {"next_weight": (1 + 0.1 * _randn(g, D)).to(dt)}
    if c.get("block"):
        p["block_weight"] = (0.5 + 0.1 * _randn(g, D)).to(dt)
    if c.get("bias"):
        p["next_bias"] = (0.1 * _randn(g, D)).to(dt)
        if c.get("block"):
            p["block_bias"] = (0.1 * _randn(g, D)).to(dt)
    if c.get("groups"):
        p["gate"] = torch.tanh(_randn(g, c["groups"], D)).to(dt)
    if c.get("backward"):
        s["dh"] = _rows(_randn(g, T, D) * 1e-2, dt, c.get("pad", 0))
        s["du"] = _rows(_randn(g, T, D) * 1e-2, dt, c.get("pad", 0))
    s["p"] = p
    return s


def _weight(g, channels, cols):
    """8-bit weights in rows of whole 128-byte pieces, and their scales."""
    q = torch.zeros(channels, -(-cols // ROW) * ROW, device="cuda", dtype=torch.int8)
    q[:, :cols] = (_randn(g, channels, cols) * 32).round_().clamp_(-127, 127).to(torch.int8)
    scale = (0.5 + torch.rand(channels, generator=g, device="cuda")) / (32 * math.sqrt(cols))
    return q, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c, op = case, case["op"]
    s = {"case": dict(c)}
    if op in ("norm", "project"):
        s.update(_norm_inputs(g, c if op == "norm" else dict(c, kind="rms")))
    if op == "project":
        s["w"], s["w_scale"] = _weight(g, c["channels"], c["cols"])
    if op == "product":
        s["x"] = _randn(g, c["rows"], c["cols"]).to(TYPES[c["type"]])
        s["w"], s["w_scale"] = _weight(g, c["channels"], c["cols"])
        s["bias"] = _randn(g, c["channels"]) if c["bias"] else None
    if op == "sample":
        B, V = c["rows"], c["vocab"]
        s["logits"] = _rows(_randn(g, B, V) * 2.5, TYPES[c["type"]], c["pad"])
        noise = torch.empty(B, V, device="cuda", dtype=torch.float32)
        s["gumbel"] = -noise.exponential_(generator=g).clamp_(min=1e-30).log_()
        t = 0.6 + 0.8 * torch.rand(B, generator=g, device="cuda")
        if B >= 8:
            t[B // 8::8] = 0.0          # greedy requests among the others
        s["temperature"] = t
        s["top_k"] = torch.full((B,), c["top_k"], device="cuda", dtype=torch.int32)
        s["top_p"] = torch.full((B,), c["top_p"], device="cuda", dtype=torch.float32)
        s["min_p"] = torch.full((B,), c["min_p"], device="cuda", dtype=torch.float32)
        s["allowed"] = None
        if c["masked"]:
            s["allowed"] = torch.rand(B, V, generator=g, device="cuda") < 0.3
            s["allowed"][B // 3::7] = False   # requests that may say nothing
    return s


# ------------------------------------------------------------------ plain forms, 32 bits

def _normed(v, kind):
    """(normalised rows, 1 / their deviation)"""
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    r = 1.0 / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
    return v * r, r


def _normed_grad(a, vhat, r, kind):
    d = a - vhat * (a * vhat).mean(1, keepdim=True)
    if kind == "layer":
        d = d - a.mean(1, keepdim=True)
    return d * r


def _gate(p, T):
    g = p.get("gate")
    return None if g is None else g.repeat_interleave(T // g.shape[0], dim=0)


def _norm_forward(x, y, p, kind):
    """h, u and what the gradient needs, from 32-bit inputs"""
    n, yhat, ry = y, None, None
    if "block_weight" in p:
        yhat, ry = _normed(y, kind)
        n = yhat * p["block_weight"]
        if "block_bias" in p:
            n = n + p["block_bias"]
    gate = _gate(p, x.shape[0])
    h = x + SCALE * (n if gate is None else gate * n)
    hhat, rh = _normed(h, kind)
    u = hhat * p["next_weight"]
    if "next_bias" in p:
        u = u + p["next_bias"]
    return h, u, n, yhat, ry, gate, hhat, rh


def _plain_norm(s):
    c, kind = s["case"], s["case"]["kind"]
    dt = TYPES[c["type"]]
    x, y, p = s["x"].float(), s["y"].float(), {k: v.float() for k, v in s["p"].items()}
    h, u, n, yhat, ry, gate, hhat, rh = _norm_forward(x, y, p, kind)
    if not c["backward"]:
        return {"h": h.to(dt), "u": u.to(dt)}
    dh, du = s["dh"].float(), s["du"].float()
    e = dh + _normed_grad(du * p["next_weight"], hhat, rh, kind)
    out = {"dx": e.to(dt), "next_weight": (du * hhat).sum(0)}
    dn = SCALE * e if gate is None else SCALE * gate * e
    dy = dn
    if "next_bias" in p:
        out["next_bias"] = du.sum(0)
    if gate is not None:
        G = p["gate"].shape[0]
        out["gate"] = (SCALE * e * n).view(G, -1, e.shape[1]).sum(1)
    if yhat is not None:
        out["block_weight"] = (dn * yhat).sum(0)
        if "block_bias" in p:
            out["block_bias"] = dn.sum(0)
        dy = _normed_grad(dn * p["block_weight"], yhat, ry, kind)
    out["dy"] = dy.to(dt)
    return out


def _quantised(x):
    scale = x.abs().amax(1, keepdim=True) / 127
    q = torch.where(scale == 0, torch.zeros_like(x), (x / scale).round().clamp(-127, 127))
    return q, scale


def _plain_product(x, s, cols):
    q, scale = _quantised(x)
    out = (q @ s["w"][:, :cols].float().t()) * scale * s["w_scale"]
    return out if s.get("bias") is None else out + s["bias"]


def _plain_sample(s):
    z = s["logits"].float()
    B, V = z.shape
    valid = z > -math.inf
    if s["allowed"] is not None:
        valid = valid & s["allowed"]
    z = torch.where(valid, z, torch.full_like(z, -math.inf))
    z, index = torch.sort(z, dim=1, descending=True, stable=True)
    valid, top = z > -math.inf, z[:, :1]
    greedy = ~(s["temperature"] > 0)[:, None]
    t = torch.where(greedy, torch.ones_like(top), s["temperature"][:, None])
    d = torch.where(z == top, torch.zeros_like(z), (z - top) / t)
    e = torch.where(valid, torch.exp(d), torch.zeros_like(z))
    rank = torch.arange(V, device=z.device)[None]
    k, p, m = s["top_k"][:, None], s["top_p"][:, None], s["min_p"][:, None]
    keep = valid & ((k <= 0) | (rank < k))
    mass = torch.where(keep, e, torch.zeros_like(e))
    before = torch.cumsum(mass, 1).roll(1, 1)
    keep = keep & ((p >= 1) | (before < p * mass.sum(1, keepdim=True)) | (rank == 0)) & ((e >= m) | (rank == 0))
    score = torch.where(keep, d + s["gumbel"].gather(1, index), torch.full_like(z, -math.inf))
    best = score.amax(1, keepdim=True)
    token = torch.where(keep & (score == best), index, torch.full_like(index, V)).amin(1, keepdim=True)
    token = torch.where(greedy, index[:, :1], token)
    at = (index == token).int().argmax(1, keepdim=True)
    logprob = torch.log(e.gather(1, at) / e.sum(1, keepdim=True))
    some = valid[:, :1]
    return {"token": torch.where(some, token, torch.full_like(token, -1))[:, 0],
            "logprob": torch.where(some, logprob, torch.full_like(logprob, -math.inf))[:, 0]}


def run(state):
    c, op = state["case"], state["case"]["op"]
    if own:
        from rns_ckks_polynomial_amd import plain
        if op == "norm":
            args = dict(state["p"], scale=SCALE, eps=EPS, kind=c["kind"])
            if not c["backward"]:
                h, u = plain.residual_norm(state["x"], state["y"], **args)
                return {"h": h, "u": u}
            grads = plain.residual_norm_grad(state["x"], state["y"], state["dh"], state["du"], **args)
            return {k: v for k, v in grads._asdict().items() if v is not None}
        if op == "sample":
            token, logprob = plain.sample(state["logits"], state["gumbel"], state["temperature"], top_k=state["top_k"],
                                          top_p=state["top_p"], min_p=state["min_p"], allowed=state["allowed"])
            return {"token": token, "logprob": logprob}
        w = plain.Int8Rows(state["w"], state["w_scale"], c["cols"])
        if op == "product":
            return {"out": plain.linear_i8(state["x"], w, bias=state["bias"], dtype=TYPES[c["out"]])}
        h, rows = plain.residual_norm_i8(state["x"], state["y"], scale=SCALE, eps=EPS, kind="rms", **state["p"])
        return {"h": h, "out": plain.matmul_i8(rows, w, dtype=TYPES[c["type"]])}
    if op == "norm":
        return _plain_norm(state)
    if op == "product":
        return {"out": _plain_product(state["x"].float(), state, c["cols"]).to(TYPES[c["out"]])}
    if op == "project":
        dt = TYPES[c["type"]]
        p = {k: v.float() for k, v in state["p"].items()}
        h, u = _norm_forward(state["x"].float(), state["y"].float(), p, "rms")[:2]
        return {"h": h.to(dt), "out": _plain_product(u, state, c["cols"]).to(dt)}
    return _plain_sample(state)


# ------------------------------------------------------------------ bytes and operations

def work(case):
    c, op = case, case["op"]
    if op == "norm":
        n, b = c["rows"] * c["cols"], SIZE[c["type"]]
        weights = 1 + c["groups"] + (1 if c["block"] else 0) + (1 + c["block"] if c["bias"] else 0)
        if c["backward"]:
            return {"bytes": 6 * n * b + c["cols"] * weights * (b + 4), "flops": 30 * n}
        return {"bytes": 4 * n * b + c["cols"] * weights * b, "flops": 12 * n}
    if op == "sample":
        # the noise is needed only where a token is kept: top_k of it; all of it without filters; with top_p or min_p
        # alone that depends on the values, and none is counted
        n = c["rows"] * c["vocab"]
        noise = min(c["top_k"], c["vocab"]) if c["top_k"] else 0 if c["top_p"] < 1 or c["min_p"] > 0 else c["vocab"]
        return {"bytes": n * (SIZE[c["type"]] + (1 if c["masked"] else 0)) + c["rows"] * (4 * noise + 28),
                "flops": 6 * n}
    M, N, K = c["rows"], c["channels"], c["cols"]
    flops = 2 * M * N * K
    if op == "project":
        b = SIZE[c["type"]]
        return {"bytes": 3 * M * K * b + K * b + N * K + 4 * N + M * N * b, "flops": flops + 12 * M * K}
    return {"bytes": M * K * SIZE[c["type"]] + N * K + 4 * N * (2 if c["bias"] else 1) + M * N * SIZE[c["out"]],
            "flops": flops + 4 * M * K}


# ------------------------------------------------------------------ the definitions in 64 bits

def _exact_norm(s, kind, scale, eps):
    """The definition row by row over (rows, cols) in 64 bits; the gradient by the chain rule through each mean."""
    d = lambda v: v.to(torch.float64)  # noqa: E731
    p = {k: d(v) for k, v in s["p"].items()}
    x, y = d(s["x"]), d(s["y"])
    T, D = x.shape

    def stats(v):
        mu = v.sum(1) / D if kind == "layer" else torch.zeros(T, device=v.device, dtype=torch.float64)
        return mu, ((v - mu[:, None]) ** 2).sum(1) / D + eps

    gate = torch.ones(1, D, device=x.device, dtype=torch.float64) if "gate" not in p else p["gate"]
    owner = torch.arange(T, device=x.device) * gate.shape[0] // T
    n = y
    if "block_weight" in p:
        mu_y, var_y = stats(y)
        n = (y - mu_y[:, None]) / var_y.sqrt()[:, None] * p["block_weight"] + p.get("block_bias", 0.0)
    h = x + scale * gate[owner] * n
    mu_h, var_h = stats(h)
    u = (h - mu_h[:, None]) / var_h.sqrt()[:, None] * p["next_weight"] + p.get("next_bias", 0.0)
    if "dh" not in s:
        return {"h": h, "u": u}
    dh, du = d(s["dh"]), d(s["du"])

    def through(up, v, mu, var, weight):
        """(gradient of the rows, of the weight, of the bias) of (v - mu) / sqrt(var) * weight + bias"""
        c = v - mu[:, None]
        dc = up * weight / var.sqrt()[:, None]
        dvar = -0.5 * (up * weight * c).sum(1) * var ** -1.5
        dc = dc + dvar[:, None] * 2 * c / D
        if kind == "layer":
            dc = dc - (dc.sum(1) / D)[:, None]
        return dc, (up * c / var.sqrt()[:, None]).sum(0), up.sum(0)

    back, dw, db = through(du, h, mu_h, var_h, p["next_weight"])
    total = dh + back
    out = {"dx": total, "next_weight": dw}
    if "next_bias" in p:
        out["next_bias"] = db
    if "gate" in p:
        out["gate"] = torch.zeros_like(gate).index_add_(0, owner, scale * total * n)
    dn = scale * gate[owner] * total
    out["dy"] = dn
    if "block_weight" in p:
        out["dy"], out["block_weight"], db = through(dn, y, mu_y, var_y, p["block_weight"])
        if "block_bias" in p:
            out["block_bias"] = db
    return out


def _exact_product(x, s, cols):
    """x: 64 bits.  A row's scale is held in 32 bits, and a quotient is rounded to 32 bits before it is rounded to a
    whole number: that is part of the definition (a tie is a tie of the 32-bit quotient)."""
    scale = (x.abs().max(1).values / 127).to(torch.float32).to(torch.float64)
    q = torch.zeros_like(x)
    some = scale > 0
    q[some] = torch.clamp(torch.round((x[some] / scale[some, None]).to(torch.float32)), -127, 127).to(torch.float64)
    sums = torch.mm(q, s["w"][:, :cols].to(torch.float64).t().contiguous())
    out = sums * (scale[:, None] * s["w_scale"].to(torch.float64)[None, :])
    return out if s.get("bias") is None else out + s["bias"].to(torch.float64)


def _exact_sample(s):
    z = s["logits"].to(torch.float64)
    B, V = z.shape
    tokens, logprobs = [], []
    for b in range(B):
        ok = ~torch.isnan(z[b]) & (z[b] != -math.inf)
        if s["allowed"] is not None:
            ok &= s["allowed"][b]
        ids = torch.nonzero(ok)[:, 0]
        if ids.numel() == 0:
            tokens.append(-1)
            logprobs.append(-math.inf)
            continue
        v = z[b][ids]
        t = float(s["temperature"][b])
        order = torch.argsort(v, descending=True, stable=True)
        ids, v = ids[order], v[order]
        weight = torch.exp((v - v[0]) / (t if t > 0 else 1.0))
        if t > 0:
            k, p, m = int(s["top_k"][b]), float(s["top_p"][b]), float(s["min_p"][b])
            last = min(k, ids.numel()) if k > 0 else ids.numel()
            kept = weight[:last]
            if p < 1:
                upto = torch.cumsum(kept, 0)
                last = 1 + int((upto[:-1] < p * upto[-1]).sum())
            last = max(1, min(last, int((weight >= m).sum())))
            score = (v[:last] - v[0]) / t + s["gumbel"][b][ids[:last]].to(torch.float64)
            at = int(ids[:last][score == score.max()].min())
            pos = int(torch.nonzero(ids == at)[0, 0])
        else:
            at, pos = int(ids[0]), 0
        tokens.append(at)
        logprobs.append(float(torch.log(weight[pos] / weight.sum())))
    return {"token": torch.tensor(tokens), "logprob": torch.tensor(logprobs, dtype=torch.float64)}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "norm":
        return _exact_norm(s, case["kind"], SCALE, EPS)
    if op == "product":
        return {"out": _exact_product(s["x"].to(torch.float64), s, case["cols"])}
    if op == "project":
        r = _exact_norm(s, "rms", SCALE, EPS)
        return {"h": r["h"], "out": _exact_product(r["u"], s, case["cols"])}
    return _exact_sample(s)
