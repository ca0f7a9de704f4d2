"""MI355X-native RNS-CKKS arithmetic core (HIP kernels behind a C ABI).

`Context` (in .api) binds the C library; `plain` binds its plaintext-side
operators (embedding, norms, heads, 8-bit products, sampling, log probabilities); `synth` generates seeded inputs.
The bindings are imported lazily so CPU-only tools can use `synth` without
torch or the HIP library.
"""
__all__ = ["Context", "galois_rot", "galois_conj", "plain", "synth"]


def __getattr__(name):
    if name in ("Context", "galois_rot", "galois_conj"):
        from . import api
        return getattr(api, name)
    if name == "plain":
        from importlib import import_module
        return import_module(".plain", __name__)
    raise AttributeError(name)
