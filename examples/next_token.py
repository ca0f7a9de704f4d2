"""The next token of four sequences whose last layer ran on ciphertexts.

A hop is 4 tokens of a 2048-wide hidden state, 2 ciphertexts of 1024 slots
each.  The server multiplies them by a plaintext diagonal (the smallest layer
there is) and rescales, on the GPU; the key holder decrypts (with the CPU
oracle: decryption is host-side here) and, on the GPU again, in clear,

  residual stream + block output, final norm, 8-bit rows  (residual_norm_i8)
  product with the 8-bit vocabulary weights               (matmul_i8)
  temperature, top-k, top-p and a draw                    (sample)

Run from the repository's root: python examples/next_token.py
"""
from __future__ import annotations

import os
import sys

import numpy as np

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import oracle  # noqa: E402
from rns_ckks_polynomial_amd import synth  # noqa: E402

N, LEVEL, SLOTS, TOKENS, HALVES = 2048, 3, 1024, 4, 2
HIDDEN, VOCAB, SEED = SLOTS * HALVES, 8000, 0x7EC5
DELTA = 2.0 ** 59  # near the chain primes, so a rescale brings a product back to it


class KeyHolder:
    """Secret, encryption and decryption, on the host."""

    def __init__(self):
        oracle.build()
        self.ctx = oracle.Ctx(N, LEVEL, K=1, dnum=LEVEL)
        secret = synth.ternary(SEED, synth.TAG_SECRET, 0, N)
        self.secret = self.ctx.coeffs_to_ntt(secret, np.arange(LEVEL))

    def encrypt(self, values, j):
        m = self.ctx.encode(values.astype(np.complex128), DELTA, LEVEL)
        a = synth.uniform_mod(SEED, synth.TAG_ENC_A, np.arange(LEVEL) + 4096 * j, self.ctx.primes[:LEVEL], N)
        return self.ctx.encrypt(m, self.secret, a, synth.gaussian_ints(SEED, synth.TAG_ERROR, j, N), LEVEL)

    def decrypt(self, ct, scale, level):
        m = self.ctx.decrypt(ct, self.secret[:level], level)
        return self.ctx.decode(m, scale, level).real


def server(cts, diagonal_ntt):
    """Every ciphertext times the plaintext of its half, rescaled: device arrays in, device array out."""
    import torch

    from rns_ckks_polynomial_amd.api import Context
    g = Context(N, LEVEL, 1, LEVEL)
    ct = torch.from_numpy(cts).cuda()                                  # [tokens * halves][2][level][n]
    pt = torch.from_numpy(diagonal_ntt).cuda()                         # [halves][level][n]
    pt = pt[None, :, None].expand(TOKENS, HALVES, 2, LEVEL, N).contiguous().view(-1, LEVEL, N)
    out = g.rescale(g.pointwise_mul(ct.view(-1, LEVEL, N), pt).view(-1, 2, LEVEL, N))
    torch.cuda.synchronize()
    host = out.cpu().numpy()
    g.close()
    return host


def main():
    import torch

    from rns_ckks_polynomial_amd import plain
    rng = np.random.default_rng(SEED)
    x = rng.standard_normal((TOKENS, HIDDEN))                          # the hop's hidden state
    diagonal = rng.uniform(-0.5, 0.5, HIDDEN)

    holder = KeyHolder()
    cts = np.stack([holder.encrypt(half, 2 * t + h) for t in range(TOKENS)
                    for h, half in enumerate(x[t].reshape(HALVES, SLOTS))])
    pts = np.stack([holder.ctx.encode(d.astype(np.complex128), DELTA, LEVEL) for d in diagonal.reshape(HALVES, SLOTS)])
    back = server(cts, pts)
    scale = DELTA * DELTA / holder.ctx.q(LEVEL - 1)
    y = np.stack([holder.decrypt(ct, scale, LEVEL - 1) for ct in back]).reshape(TOKENS, HIDDEN)

    dev = lambda v, dt: torch.from_numpy(np.ascontiguousarray(v)).to(dt).cuda()  # noqa: E731
    norm = dev(1 + 0.1 * rng.standard_normal(HIDDEN), torch.float32)
    weights = plain.quantize_rows(dev(rng.standard_normal((VOCAB, HIDDEN)) * 0.1, torch.float32))  # laid out once
    gumbel = dev(-np.log(-np.log(rng.uniform(1e-9, 1 - 1e-9, (TOKENS, VOCAB)))), torch.float32)
    each = lambda v, dt=torch.float32: torch.full((TOKENS,), v, dtype=dt, device="cuda")  # noqa: E731

    h, rows = plain.residual_norm_i8(dev(x, torch.float32), dev(y, torch.float32), norm)
    logits = plain.matmul_i8(rows, weights, dtype=torch.float32)
    token, logprob = plain.sample(logits, gumbel, each(0.8), top_k=each(40, torch.int32), top_p=each(0.95))
    return {"y_error": float(np.abs(y - x * diagonal).max()), "logits": logits, "token": token, "logprob": logprob,
            "clear_logits": _clear_logits(x, x * diagonal, norm, weights)}


def _clear_logits(x, y, norm, weights):
    """The same logits without encryption or 8-bit activations, in 64 bits on the host."""
    h = x + y
    u = h / np.sqrt((h * h).mean(1, keepdims=True) + 1e-6) * norm.double().cpu().numpy()
    return u @ weights.dequantize().double().cpu().numpy().T


if __name__ == "__main__":
    r = main()
    off = np.abs(r["logits"].double().cpu().numpy() - r["clear_logits"])
    print(f"decrypted block output within {r['y_error']:.1e} of the clear one")
    print(f"logits within {off.max():.3f} of the clear ones (their deviation is {r['clear_logits'].std():.2f})")
    for t in range(TOKENS):
        print(f"sequence {t}: token {int(r['token'][t])}, log probability {float(r['logprob'][t]):.3f}")
