"""Device code of the heads as host code (no GPU): workgroups with several steps
of tokens."""
from test_plain_tokens_on_host import _run

SHARED = ("extern __shared__ float2 angles[];", "static float2 angles[1024];")


def test_workgroups_with_several_steps(tmp_path):
    assert "heads: ok" in _run(tmp_path, "heads.hip", "heads_check.cpp", [SHARED])
