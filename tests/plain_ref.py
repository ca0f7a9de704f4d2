"""The plaintext-side operators from their definitions in 64 bits (numpy on the
CPU), for the tests of the HIP kernels.  Shares no code with the package."""
import numpy as np

F64 = np.float64


def stats(v, kind, eps):
    mu = v.mean(1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    return mu, 1.0 / np.sqrt(((v - mu) ** 2).mean(1, keepdims=True) + eps)


def norm_forward(x, y, nw, nb=None, bw=None, bb=None, gate=None, scale=1.0, eps=1e-6, kind="rms"):
    """dict of h, u and the values on the way (all [T, D] in 64 bits)."""
    n, yhat, ry = y, None, None
    if bw is not None:
        mu, ry = stats(y, kind, eps)
        yhat = (y - mu) * ry
        n = yhat * bw + (0 if bb is None else bb)
    g = np.ones((1, x.shape[1])) if gate is None else gate.reshape(-1, x.shape[1])
    g = np.repeat(g, x.shape[0] // g.shape[0], axis=0) if x.shape[0] else g[:0]
    h = x + scale * g * n
    mu, rh = stats(h, kind, eps)
    hhat = (h - mu) * rh
    return dict(h=h, u=hhat * nw + (0 if nb is None else nb), n=n, yhat=yhat, ry=ry, g=g, hhat=hhat, rh=rh)


def norm_grad(x, y, dh, du, nw, nb=None, bw=None, bb=None, gate=None, scale=1.0, eps=1e-6, kind="rms"):
    """Gradients as a dict, and for each the sum or size of the absolute terms it is made of (for error bounds)."""
    f = norm_forward(x, y, nw, nb, bw, bb, gate, scale, eps, kind)

    def back(a, hat, r):
        d = a - hat * (a * hat).mean(1, keepdims=True)
        if kind == "layer":
            d = d - a.mean(1, keepdims=True)
        return r * d

    a = du * nw
    e = dh + back(a, f["hhat"], f["rh"])
    dn = scale * f["g"] * e
    out = {"dx": e, "dy": dn, "next_weight": (du * f["hhat"]).sum(0)}
    top = lambda v: np.abs(v).max(1, keepdims=True) if v.size else np.zeros((v.shape[0], 1))  # noqa: E731
    # largest absolute term on the way to a row's values
    size_e = top(dh) + f["rh"] * top(a) * (2 + top(f["hhat"]) ** 2)
    size = {"dx": size_e, "dy": np.abs(scale) * top(f["g"]) * size_e,
            "next_weight": (np.abs(du) * (np.abs(f["hhat"]) + top(f["hhat"]))).sum(0)}
    if nb is not None:
        out["next_bias"], size["next_bias"] = du.sum(0), np.abs(du).sum(0)
    if gate is not None:
        G, D = gate.reshape(-1, x.shape[1]).shape
        per = lambda v: v.reshape(G, -1, D).sum(1).reshape(gate.shape)  # noqa: E731
        out["gate"] = per(scale * e * f["n"])
        size["gate"] = per(np.abs(scale) * size_e * (np.abs(f["n"]) + top(f["n"])))
    if bw is not None:
        out["block_weight"] = (dn * f["yhat"]).sum(0)
        size["block_weight"] = (size["dy"] * (np.abs(f["yhat"]) + top(f["yhat"]))).sum(0)
        if bb is not None:
            out["block_bias"], size["block_bias"] = dn.sum(0), np.broadcast_to(size["dy"], dn.shape).sum(0)
        b = dn * bw
        out["dy"] = back(b, f["yhat"], f["ry"])
        size["dy"] = f["ry"] * size["dy"] * np.abs(bw).max() * (2 + top(f["yhat"]) ** 2)
    return out, size


def quantise(x32):
    """(q, scale) of float32 rows by the definition: 1/127, its product and the quotient in 32 bits, ties to even."""
    x32 = x32.astype(np.float32)
    top = np.abs(x32).max(1).astype(np.float32)
    with np.errstate(all="ignore"):
        s = (top * (np.float32(1) / np.float32(127))).astype(np.float32)
        s[~np.isfinite(top)] = np.nan
        v = np.rint((x32 / s[:, None]).astype(np.float32))
    q = np.where((s > 0)[:, None], np.clip(v, -127, 127), 0)
    return q.astype(np.int8), s


def sample(z, gumbel, temperature, top_k=None, top_p=None, min_p=None, allowed=None):
    """(token, logprob): a row at a time, one token at a time in falling order."""
    B, V = z.shape
    tokens, logprobs = np.empty(B, np.int64), np.empty(B, F64)
    for r in range(B):
        row = z[r].astype(np.float32)
        ok = ~np.isnan(row) & (row != -np.inf) & (True if allowed is None else allowed[r])
        ids = np.nonzero(ok)[0]
        if not len(ids):
            tokens[r], logprobs[r] = -1, -np.inf
            continue
        ids = ids[np.argsort(-row[ids], kind="stable")]
        top, t = row[ids[0]], np.float32(temperature[r])
        greedy = not t > 0
        t = np.float32(1) if greedy else t
        with np.errstate(all="ignore"):  # float32 steps, as defined
            d32 = np.where(row[ids] == top, np.float32(0), (row[ids] - top).astype(np.float32) / t).astype(np.float32)
            d64 = np.where(row[ids] == top, 0.0, (row[ids].astype(F64) - F64(top)) / F64(t))
        e = np.exp(d64)
        keep = ids[:1]
        if not greedy:
            last = len(ids)
            if top_k is not None and top_k[r] > 0:
                last = min(last, int(top_k[r]))
            if top_p is not None and top_p[r] < 1:
                total, mass, n = e[:last].sum(), 0.0, 0
                while n < last and (n == 0 or mass < F64(top_p[r]) * total):
                    mass += e[n]
                    n += 1
                last = n
            keep = [i for i in range(last) if i == 0 or not (min_p is not None and min_p[r] > 0)
                    or e[i] >= F64(min_p[r])]
            score = (d32[keep] + gumbel[r, ids[keep]].astype(np.float32)).astype(np.float32)
            best = score.max()
            keep = [min(ids[k] for k, s in zip(keep, score) if s == best)]
        tokens[r] = keep[0]
        at = int(np.nonzero(ids == keep[0])[0][0])
        logprobs[r] = d64[at] - np.log(e.sum())
    return tokens, logprobs
