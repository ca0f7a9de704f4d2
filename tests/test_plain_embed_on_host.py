"""Device code of the table's gradient as host code (no GPU)."""
from test_plain_tokens_on_host import _run

SHARED = ("extern __shared__ uint32_t places[];", "static uint32_t places[ORDER_WAVES << 9];")


def test_workgroups_of_columns_that_are_not_there(tmp_path):
    assert "sums: ok" in _run(tmp_path, "embed.hip", "embed_sum_check.cpp", [SHARED])
