"""kvq_norm_rope into outputs of unusual strides: heads before tokens, and rows of both dimensions interleaved."""
import pytest
import torch

from test_serving_gpu import D, gen, randn, rope_reference, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens,heads,T,H", [(37, 3, 128, 37 * 128), (2, 2, 384, 256), (3, 2, 256, 128 * 5 + 768), (2, 5, 640, 128), (4, 3, 136, 4 * 136), (4, 2, 256, 384), (3, 5, 384, 640)])
def test_outputs_of_unusual_strides(tokens, heads, T, H):
    import bit_kv_cache_26_b200 as kvq
    g = gen(T + H)
    x = randn(g, tokens, heads, D).to(torch.bfloat16)
    w = (1 + 0.3 * randn(g, D)).to(torch.bfloat16)
    pos = torch.arange(tokens, device="cuda", dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float32) / 64)
    flat = torch.full(((tokens - 1) * T + (heads - 1) * H + D,), 7.0, device="cuda", dtype=torch.bfloat16)
    out = torch.as_strided(flat, (tokens, heads, D), (T, H, 1))
    kvq.kvq_norm_rope(x, None, None, pos, inv, out, None, None, q_weight=w, eps=1e-6)
    within(out, *rope_reference(x, w, pos, inv, 128, False, 1e-6))
    rows = torch.zeros_like(flat, dtype=torch.bool)
    torch.as_strided(rows, (tokens, heads, D), (T, H, 1)).fill_(True)
    assert (flat[~rows] == 7.0).all()                                # what lies between them stays
