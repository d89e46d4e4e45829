"""Page plans that stop, and plans over bad page ids (kvq_plan_pages), in both forms of the call: one launch, and two past
2048 sequences."""
import numpy as np
import pytest
import torch

from test_serving_gpu import check_plan, make_plan, plan_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import bit_kv_cache_26_b200 as m
    return m


@pytest.mark.parametrize("idle", [0, 300, 2100])                      # sequences without new tokens before the others
def test_the_status_names_the_limit_that_stopped_the_plan(kvq, idle):
    OVER, NONE = kvq.KVQ_DEV_OVERFLOW, kvq.KVQ_DEV_NO_PAGES
    go = lambda n, **kw: check_plan(kvq, [0] * (idle + len(n)), [0] * idle + n, 3, **kw)   # noqa: E731
    go([10, 20, 64, 64], most=25, free_n=3, want_bits=OVER)          # later requests' pages would pass the stack
    go([40, 40, 40, 40], most=100, free_n=3, want_bits=NONE)         # later requests' tokens would pass the slot map
    go([40, 40], most=60, free_n=3, want_bits=NONE)                  # one request passes both
    go([40, 0, 0], most=40, free_n=2, want_bits=0)                   # both to the brim
    go([40, 0, 0, 1], most=40, free_n=3, want_bits=OVER)
    go([40, 0, 0, 1], most=41, free_n=2, want_bits=NONE)
