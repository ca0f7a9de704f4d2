"""The example from ciphertexts to tokens (examples/next_token.py): the
decrypted block output against the clear one, the logits against 64 bits, the
tokens against the definition on those logits."""
import os
import sys

import numpy as np
import pytest

from gpu_util import require_gpu, torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_next_token():
    require_gpu()
    import next_token
    r = next_token.main()
    # one product and a rescale at scale 2^59 with sigma = 3.2 errors: within 2^-20, as the other functional checks
    assert r["y_error"] < 2.0 ** -20
    # rounding to 8 bits moves a normalised value by half a step, about 4.5 / 127 / 2 uniformly, so a sum of 2048 of them
    # against weights of deviation 0.1 by a deviation of 4.5 / 254 / sqrt(3) * 0.1 * sqrt(2048) = 0.046: 6 of those
    off = np.abs(r["logits"].double().cpu().numpy() - r["clear_logits"])
    assert off.max() < 6 * 0.046
    token = r["token"].cpu().numpy()
    assert token.shape == (4,) and ((0 <= token) & (token < next_token.VOCAB)).all()
    # a token of the top 40, with its probability at temperature 0.8
    z = r["logits"].double().cpu().numpy() / np.float32(0.8)
    for t in range(4):
        assert (z[t] > z[t][token[t]]).sum() < 40
        want = z[t][token[t]] - z[t].max() - np.log(np.exp(z[t] - z[t].max()).sum())
        assert abs(float(r["logprob"][t]) - want) < 1e-5
    assert torch.isfinite(r["logprob"]).all()
