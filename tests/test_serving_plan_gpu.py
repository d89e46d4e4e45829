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


@pytest.mark.parametrize("B", [3, 2100])
def test_tokens_of_invalid_pages_have_no_slot(kvq, B):
    # a hole in the held part of a table, and bad ids on the stack: in a chunk inside one long prompt, and in short requests
    L, n, maxp = [5, 40, 64] + [1] * (B - 3), [20, 2600, 33] + [0] * (B - 3), 90
    cache, t, table, free, free_n, most = make_plan(kvq, L, n, maxp)
    table[0, 0], table[1, 1] = -1, cache.num_pages
    free[free_n - 3], free[free_n - 40], free[free_n - 83] = -7, 2 ** 31 - 1, cache.num_pages
    cache.page_table.copy_(torch.from_numpy(table))
    t["free"].copy_(torch.from_numpy(free))
    cache.plan(t["new"], t["free"], t["count"], t["cu"], t["slots"][:most], t["pos"][:most], t["ids"][:most], cache.plan_workspace())
    wt, wcu, slots, pos, ids, left, _ = plan_reference(L, n, table, free, free_n, most)
    slots = np.array([s if 0 <= s < cache.num_pages * 32 else -1 for s in slots])
    assert (slots == -1).sum() > 20 + 24 + 3 * 30 - 32
    assert np.array_equal(t["slots"][:most].cpu().numpy(), slots)
    assert t["pos"][:most].tolist() == pos and t["ids"][:most].tolist() == ids and np.array_equal(t["cu"].cpu().numpy(), wcu)
    assert np.array_equal(cache.page_table.cpu().numpy(), wt) and int(t["count"]) == left
    assert cache.read_status() == kvq.KVQ_DEV_BAD_PAGE
