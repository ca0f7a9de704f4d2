"""Device code of the log probabilities and their gradient as host code (no GPU),
where numbers leave the range of 32 bits on the way to a result that is in it."""
from test_plain_tokens_on_host import _run


def test_gradient_at_tiny_temperatures(tmp_path):
    assert "gradient: ok" in _run(tmp_path, "logprob.hip", "score_grad_check.cpp")


def test_distances_past_32_bits_and_infinite_temperatures(tmp_path):
    assert "distances: ok" in _run(tmp_path, "logprob.hip", "score_distance_check.cpp")
