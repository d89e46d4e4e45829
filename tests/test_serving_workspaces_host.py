"""Workspace sizes of the serving-step calls (no GPU needed)."""
import pytest

import bit_kv_cache_26_b200 as kvq
from test_serving_host import cache


@pytest.mark.parametrize("B,H,Gq", [(1, 8, 4), (1, 1, 1), (4, 4, 7), (3, 2, 16), (16, 8, 5), (256, 8, 4)])
def test_the_workspace_of_a_budget_serves_smaller_ones(B, H, Gq):
    c = cache(num_seqs=B, num_kv_heads=H, num_patterns=64, max_pages_per_seq=8192, num_pages=8192 * B, bits=4)
    sizes = [kvq.kvq_decode_pages_workspace_bytes(c, H * Gq, n) for n in range(1, 1200)]
    assert sizes == sorted(sizes)
    far = [kvq.kvq_decode_pages_workspace_bytes(c, H * Gq, n) for n in (1199, 4000, 8192, 1 << 20, (1 << 31) - 1)]
    assert far == sorted(far) and far[-1] <= 256 + B * H * Gq * 64 * 130 * 4
