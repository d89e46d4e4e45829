"""kvq_norm_rope refuses output rows that overlap, whatever the order of its strides (answered on the host)."""
import itertools

import pytest

from test_serving_host import INVALID, rope, rows


def overlap(tokens, heads, T, H):
    at = sorted(t * T + h * H for t, h in itertools.product(range(tokens), range(heads)))
    return any(b - a < 128 for a, b in zip(at, at[1:]))


@pytest.mark.parametrize("tokens,heads,T,H", [(4, 2, 128, 128), (4, 3, 256, 128), (4, 2, 256, 376), (3, 5, 384, 648), (5, 5, 640, 136), (2, 2, 136, 200),
                                              (4, 3, 1024, 1032), (9, 4, 128, 1024)])
def test_overlapping_output_rows_are_refused(tokens, heads, T, H):
    assert overlap(tokens, heads, T, H)
    assert rope(q=rows(heads, out_tok_stride=T, out_head_stride=H), tokens=tokens) == INVALID
