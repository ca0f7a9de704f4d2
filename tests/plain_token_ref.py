"""Embedding, norm and rotation of heads, and token log probabilities from their
definitions in 64 bits (numpy on the CPU), for the tests of the HIP kernels.
Shares no code with the package."""
import numpy as np

F64 = np.float64


def embed_grad(drows, tokens, vocab, scale):
    """(gradient, sum of the absolute terms, how many terms) of each row of the table"""
    out, size = np.zeros((vocab, drows.shape[1])), np.zeros((vocab, drows.shape[1]))
    n = np.zeros((vocab, 1))
    for t, v in enumerate(tokens):
        if 0 <= v < vocab:
            out[v] += scale * drows[t]
            size[v] += np.abs(scale * drows[t])
            n[v] += 1
    return out, size, n


def pairs(r, interleaved):
    i = np.arange(r)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + r)


def turn(x, positions, inv_freq, interleaved, back=False):
    """x [T, H, d] turned; and the sizes |x_a| + |x_b| of what each element is made of"""
    y, size = x.copy(), np.abs(x)
    if inv_freq is None:
        return y, size
    f = positions.astype(F64)[:, None] * inv_freq.astype(F64)[None]
    c, s = np.cos(f)[:, None], np.sin(f)[:, None] * (-1 if back else 1)
    a, b = pairs(len(inv_freq), interleaved)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    both = size[..., a] + size[..., b]
    size[..., a], size[..., b] = both, both
    return y, size


def heads(x, w, positions, inv_freq, eps, interleaved):
    n = x if w is None else x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w
    return turn(n, positions, inv_freq, interleaved)


def heads_grad(x, dy, w, positions, inv_freq, eps, interleaved):
    """(dx, its size, dw, its size)"""
    dn, size = turn(dy, positions, inv_freq, interleaved, back=True)
    if w is None:
        return dn, size, None, None
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    hat = x * r
    a = dn * w
    dx = r * (a - hat * (a * hat).mean(-1, keepdims=True))
    abs_a = size * np.abs(w)
    dx_size = r * (abs_a + np.abs(hat) * (abs_a * np.abs(hat)).mean(-1, keepdims=True))
    return dx, dx_size, (dn * hat).sum((0, 1)), (size * np.abs(hat)).sum((0, 1))


def score(z, tokens, top=0, temperature=None, allowed=None):
    """dict of the results, of x - log mass (`lp`) and of what the error bounds go by"""
    B, V = z.shape
    r = dict(logprob=np.zeros(B), entropy=np.zeros(B), largest=np.full(B, -np.inf), log_mass=np.full(B, -np.inf),
             top_token=np.full((B, top), -1, np.int64), top_logprob=np.full((B, top), -np.inf),
             lp=np.full((B, V), -np.inf), far=np.zeros(B), inv_t=np.ones(B), possible=np.zeros((B, V), bool))
    for b in range(B):
        ok = ~np.isnan(z[b]) & (z[b] != -np.inf) & (True if allowed is None else allowed[b])
        ids = np.nonzero(ok)[0]
        t = F64(1) if temperature is None or not temperature[b] > 0 else max(F64(temperature[b]), 2.0 ** -127)
        inside = 0 <= tokens[b] < V
        r["inv_t"][b], r["possible"][b] = 1 / t, ok
        if not len(ids):
            r["logprob"][b] = -np.inf if inside else 0
            continue
        v = z[b][ids]
        m = v.max()
        with np.errstate(invalid="ignore"):
            x = np.where(v == m, 0.0, (v - m) / t)
        e = np.exp(x)
        lm = np.log(e.sum())
        lp = x - lm
        r["lp"][b, ids] = lp
        if inside:
            r["logprob"][b] = r["lp"][b, tokens[b]]
        p = np.exp(lp)
        r["entropy"][b] = -(p[p > 0] * lp[p > 0]).sum()
        r["far"][b] = -(p[p > 0] * x[p > 0]).sum()  # mean distance to the largest
        r["largest"][b], r["log_mass"][b] = m, lm
        order = np.argsort(-v, kind="stable")[:top]
        r["top_token"][b, :len(order)], r["top_logprob"][b, :len(order)] = ids[order], lp[order]
    return r


def score_grad(r, tokens, dl, dh):
    """(gradient, size of its terms) from score's results"""
    B, V = r["lp"].shape
    p = np.exp(r["lp"])
    lp = np.where(p > 0, r["lp"], 0)
    dl, dh = (np.zeros(B) if v is None else v for v in (dl, dh))
    inside = (tokens >= 0) & (tokens < V)
    at = np.where(inside, tokens, 0)
    inside &= r["possible"][np.arange(B), at]
    dl = np.where(inside, dl, 0)
    h = r["entropy"]
    with np.errstate(invalid="ignore"):
        g = -p * (dl[:, None] + dh[:, None] * (lp + h[:, None]))
    size = p * (np.abs(dl)[:, None] + np.abs(dh)[:, None] * (np.abs(lp) + h[:, None]))
    g[np.arange(B), at] += dl
    size[np.arange(B), at] += np.abs(dl)
    mask = r["possible"]
    return np.where(mask, g * r["inv_t"][:, None], 0), np.where(mask, size * r["inv_t"][:, None], 0)
