"""One workspace, zeroed once, under calls of different shapes and kinds in turn."""
import pytest
import torch

from test_serving_gpu import (D, G, attend, attend_reference, check_select, filled, gen, key_cache, make_plan,
                              plan_reference, random_lists, randn, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import bit_kv_cache_26_b200 as m
    return m


def test_select_of_batches_that_change_size(kvq):
    # 64, 128, 64, 300 and 600 groups, the first four with several CTAs each
    cases = []
    for B in (8, 16, 8, 75, 150, 16):
        H, pages = (8, 200) if B <= 16 else (4, 100)
        cache = key_cache(kvq, B, H, pages, torch.bfloat16, [pages * G - 3 - b for b in range(B)])
        g = gen(B)
        q = randn(g, B, 4 * H, D).to(torch.bfloat16)
        bounds = randn(g, cache.num_pages, H, 2, D).sort(2).values.to(torch.bfloat16)
        cases.append((cache, q, bounds))
    ws = torch.zeros(max(kvq.kvq_select_workspace_bytes(c.c) for c, _, _ in cases), dtype=torch.uint8, device="cuda")
    for cache, q, bounds in cases * 2:
        check_select(kvq, cache, q, bounds, 30, 1, 2, ws)


def test_attention_of_batches_that_change_size(kvq):
    # a long list's capacity (many splits) with few entries used, then other batches, heads and budgets
    cases = []
    for B, H, Gq, budget in ((8, 8, 4, 2100), (16, 8, 4, 2100), (8, 8, 4, 2100), (1, 2, 16, 64), (1, 8, 4, 72), (2, 8, 4, 72), (70, 4, 1, 5000),
                             (1, 1, 1, 280), (16, 8, 4, 2100)):
        cache = filled(kvq, B, H, 0, 4, 16, torch.bfloat16, lengths=[330 - b for b in range(B)])
        q = randn(gen(B), B, H * Gq, D).to(torch.bfloat16)
        lists, n = random_lists(cache, budget, B)
        cases.append((cache, q, lists, n))
    ws = torch.zeros(max(kvq.kvq_decode_pages_workspace_bytes(c.c, q.shape[1], lists.shape[-1]) for c, q, lists, _ in cases),
                     dtype=torch.uint8, device="cuda")
    for cache, q, lists, n in cases + cases[::-1]:
        within(attend(cache, q, lists, n, ws=ws), *attend_reference(kvq, cache, q, lists, n, D ** -0.5))


def test_one_workspace_for_plans_selections_and_attention(kvq):
    cache = filled(kvq, 1, 2, 0, 4, 16, torch.bfloat16, lengths=[140 * G - 9])
    q = randn(gen(2), 1, 8, D).to(torch.bfloat16)
    bounds = randn(gen(3), cache.num_pages, 2, 2, D).sort(2).values.to(torch.bfloat16)
    lists, n = random_lists(cache, 70, 1)
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    for B in (2100, 3, 4097):                                        # the plan's forms of two launches and of one
        L, new = [31 + b % 3 for b in range(B)], [b % 4 for b in range(B)]
        c, t, table, free, free_n, most = make_plan(kvq, L, new, 3)
        c.plan(t["new"], t["free"], t["count"], t["cu"], t["slots"][:most], t["pos"][:most], t["ids"][:most], ws)
        check_select(kvq, cache, q, bounds, 20, 1, 2, ws)
        within(attend(cache, q, lists, n, ws=ws), *attend_reference(kvq, cache, q, lists, n, D ** -0.5))
        wt, wcu, slots, pos, ids, left, bits = plan_reference(L, new, table, free, free_n, most)
        assert t["slots"][:most].tolist() == slots and t["pos"][:most].tolist() == pos and t["ids"][:most].tolist() == ids
        assert t["cu"].tolist() == wcu.tolist() and int(t["count"]) == left and c.read_status() == bits == 0


def test_the_workspace_of_a_budget_serves_smaller_ones(kvq):
    cache = filled(kvq, 1, 8, 0, 4, 64, torch.bfloat16, lengths=[130 * G - 7])
    q = randn(gen(2), 1, 32, D).to(torch.bfloat16)
    ws = torch.zeros(kvq.kvq_decode_pages_workspace_bytes(cache.c, 32, 128), dtype=torch.uint8, device="cuda")
    for budget in (128, 72, 73, 96, 5, 1, 110, 16):
        lists, n = random_lists(cache, budget, budget)
        within(attend(cache, q, lists, n, ws=ws), *attend_reference(kvq, cache, q, lists, n, D ** -0.5))
