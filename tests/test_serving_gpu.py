"""The serving-step entry points on a GPU against plain implementations in 64 bits: kvq_norm_rope, kvq_plan_pages,
kvq_page_bounds, kvq_select_pages, kvq_decode_attention_pages, and a run of them together.

Whole numbers and chosen values are compared exactly.  A 16-bit result is allowed half a step of its type,
finfo.eps / 2 of the value, plus the fp32 error of the arithmetic before it, bounded beside each comparison."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

D, G = 128, 32
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module")
def kvq():
    import bit_kv_cache_26_b200 as m
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def within(got, want, extra):
    """|got - want| <= half a step of got's type at want + extra (a bound or a tensor of bounds)."""
    step = torch.finfo(got.dtype).eps / 2
    tiny = torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps / 2   # half a subnormal step
    off = (got.double() - want).abs() - (want.abs() * step + (1 + step) * extra + tiny)
    assert not torch.isnan(got).any()
    assert float(off.max()) <= 0, f"beyond the bound by {float(off.max()):.3e}"


# ---- norms and rotation --------------------------------------------------------------------------

def rope_reference(x, w, pos, inv, rot, inter, eps):
    """(result, bound of the fp32 error): float64 by the formula.  Each product of the rotation carries a handful of
    fp32 roundings (norm, weight, cosine, the two products and their sum) and the angle's fp32 remainder 2 pi 2^-25:
    below 2^-20 of |u| + |v|."""
    y = x.double()
    if w is not None:
        y = y / ((y * y).mean(-1, keepdim=True) + eps).sqrt() * w.double()
    mag = y.abs()
    out, err = y.clone(), mag * 2.0 ** -20
    i = torch.arange(rot // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    if rot:
        ang = pos.double()[:, None, None] * inv.double()
        c, s = ang.cos(), ang.sin()
        out[..., a], out[..., b] = y[..., a] * c - y[..., b] * s, y[..., b] * c + y[..., a] * s
        err[..., a] = err[..., b] = (mag[..., a] + mag[..., b]) * 2.0 ** -20
    return out, err


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("tokens,hq,hk,rot,inter,norm", [
    (1, 1, 1, 128, False, True), (1, 32, 8, 128, True, False), (33, 28, 4, 64, False, True), (33, 28, 4, 96, True, True),
    (7, 5, 5, 16, False, True), (7, 5, 5, 0, False, True), (4737, 3, 1, 32, False, False), (5003, 2, 1, 112, True, True),
])
def test_norm_rope(kvq, dtype, tokens, hq, hk, rot, inter, norm):
    dt, g = DT[dtype], gen(tokens * 31 + rot)
    # a slice of a wider packed projection, so rows have free strides
    wide = randn(g, tokens, hq + 2 * hk + 1, D).to(dt)
    q, k, v = wide[:, :hq], wide[:, hq:hq + hk], wide[:, hq + hk:hq + 2 * hk]
    q[0, 0] = 0                                                     # a row without length
    qw, kw = ((1 + 0.3 * randn(g, D)).to(dt) for _ in range(2))
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    inv = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float32) / max(1, rot // 2))
    qo = torch.full((tokens, hq + 1, D), 7.0, dtype=dt, device="cuda")
    ko, vo = (torch.full((tokens, hk, D), 7.0, dtype=dt, device="cuda") for _ in range(2))
    kvq.kvq_norm_rope(q, k, v, pos, inv, qo[:, :hq], ko, vo, qw if norm else None, kw if norm else None, 1e-6, inter)
    within(qo[:, :hq], *rope_reference(q, qw if norm else None, pos, inv, rot, inter, 1e-6))
    within(ko, *rope_reference(k, kw if norm else None, pos, inv, rot, inter, 1e-6))
    assert torch.equal(vo.view(torch.int16), v.contiguous().view(torch.int16))
    assert (qo[:, hq] == 7.0).all()                                 # rows beside the output stay


@pytest.mark.parametrize("tokens,heads,weights,rot,inter", [
    (37, (8, 1, 1), "qk", 128, False), (37, (3, 1, 2), "k", 96, True), (1, (1, 1, 1), "q", 64, False), (20011, (1, 1, 1), "qk", 32, True),
    (37, (2, 3, 6), "", 128, False), (9001, (0, 2, 1), "k", 128, True), (513, (6, 0, 1), "q", 112, False),
])
def test_norm_rope_of_few_heads(kvq, tokens, heads, weights, rot, inter):
    dt, g = torch.bfloat16, gen(sum(heads) + rot)
    rows = [randn(g, tokens, n, D).to(dt) if n else None for n in heads]
    rows[2][0, 0, :4] = torch.tensor([float("nan"), float("inf"), -0.0, 0.0], device="cuda", dtype=dt)   # values pass as they are
    w = [(1 + 0.3 * randn(g, D)).to(dt) if n in weights else None for n in "qk"]
    pos = torch.randint(0, 1 << 20, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(rot // 2, device="cuda", dtype=torch.float32) / (rot // 2))
    out = [None if x is None else torch.full_like(x, 7.0) for x in rows]
    kvq.kvq_norm_rope(*rows, pos, inv, *out, *w, 1e-6, inter)
    for x, y, z in zip(rows[:2], out[:2], w):
        if x is not None:
            within(y, *rope_reference(x, z, pos, inv, rot, inter, 1e-6))
    assert torch.equal(out[2].view(torch.int16), rows[2].view(torch.int16))


def test_norm_rope_in_place_and_single_tensors(kvq):
    g = gen(3)
    x = randn(g, 45, 6, D).to(torch.bfloat16)
    w = (1 + 0.3 * randn(g, D)).to(torch.bfloat16)
    pos = torch.arange(45, device="cuda", dtype=torch.int32) * 1000 - 5000    # positions before zero turn back
    inv = 500000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float32) / 64)
    want, err = rope_reference(x, w, pos, inv, 128, False, 1e-5)
    out = torch.empty_like(x)
    kvq.kvq_norm_rope(None, x, None, pos, inv, None, out, None, k_weight=w, eps=1e-5)
    within(out, want, err)
    y = x.clone()
    kvq.kvq_norm_rope(y, None, None, pos, inv, y, None, None, q_weight=w, eps=1e-5)
    assert torch.equal(y, out)
    kvq.kvq_norm_rope(None, None, x, None, None, None, None, y)
    assert torch.equal(y, x)


def test_norm_rope_in_place_on_slices_and_without_tokens(kvq):
    g = gen(4)
    wide = randn(g, 77, 9, D).to(torch.float16)
    keep = wide.clone()
    w = (1 + 0.3 * randn(g, D)).to(torch.float16)
    pos = torch.arange(77, device="cuda", dtype=torch.int32)
    inv = 10000.0 ** (-torch.arange(48, device="cuda", dtype=torch.float32) / 48)
    q, k, v = wide[:, 1:6], wide[:, 6:8], wide[:, 8:]
    kvq.kvq_norm_rope(q, k, v, pos, inv, q, k, v, w, None, 1e-6)
    within(q, *rope_reference(keep[:, 1:6], w, pos, inv, 96, False, 1e-6))
    within(k, *rope_reference(keep[:, 6:8], None, pos, inv, 96, False, 1e-6))
    assert torch.equal(v, keep[:, 8:]) and torch.equal(wide[:, :1], keep[:, :1])
    none = wide[:0]
    kvq.kvq_norm_rope(none, None, none, pos[:0], inv, none, None, none)
    one = wide[5:6].clone()                                          # one token: a stride nobody reads
    out = torch.empty_like(one)
    kvq.kvq_norm_rope(one.as_strided((1, 9, D), (1, D, 1)), None, None, pos[5:6], inv, out, None, None, w)
    within(out, *rope_reference(one, w, pos[5:6], inv, 96, False, 1e-6))


# ---- page plans ----------------------------------------------------------------------------------

def plan_reference(L, n, table, free, count, most):
    """The plan one request after the other, in whole numbers."""
    table, (B, maxp) = table.copy(), table.shape
    cu, slots, pos, ids, left, bits, stop = [0], [], [], [], count, 0, False
    for b in range(B):
        ok = L[b] >= 0 and n[b] >= 0 and L[b] + n[b] <= maxp * G
        if not ok:
            bits |= 0x2
        held = -(-L[b] // G)
        need = -(-(L[b] + n[b]) // G) - held
        if ok and n[b] and not stop and (len(slots) + n[b] > most or need > left):
            stop = True
            bits |= 0x20 if need > left else 0x2
        elif ok and n[b] and stop:
            bits |= 0x20 | 0x2      # one of the two, by which sum passed its limit: not told apart here
        if ok and n[b] and not stop:
            for j in range(need):
                table[b, held + j] = free[left - 1 - j]
            left -= need
            for i in range(n[b]):
                p = L[b] + i
                slots.append(int(table[b, p // G]) * G + p % G)
                pos.append(p)
                ids.append(b)
        cu.append(len(slots))
    return table, np.array(cu), slots, pos, ids, left, bits


def make_plan(kvq, L, n, maxp, free_n=None, most=None, seed=0):
    B = len(L)
    rng = np.random.default_rng(seed)
    pages = rng.permutation(B * maxp).astype(np.int32).reshape(B, maxp)
    held = [max(0, min(maxp, -(-x // G))) for x in L]
    table = np.full((B, maxp), -1, np.int32)
    for b in range(B):
        table[b, :held[b]] = pages[b, :held[b]]
    free = np.concatenate([pages[b, held[b]:] for b in range(B)]) if B else np.zeros(0, np.int32)
    free_n = len(free) if free_n is None else free_n
    most = max(0, int(sum(max(0, x) for x in n))) if most is None else most
    cache = kvq.PagedKVCache(B, 1, maxp * G, 2, 1, page_order=torch.from_numpy(table))
    cache.seq_len.copy_(torch.tensor(L, dtype=torch.int32))
    t = dict(new=torch.tensor(n, dtype=torch.int32, device="cuda"), free=torch.from_numpy(free).cuda(),
             count=torch.tensor([free_n], dtype=torch.int32, device="cuda"),
             cu=torch.full((B + 1,), -7, dtype=torch.int32, device="cuda"),
             slots=torch.full((most + 3,), -7, dtype=torch.int64, device="cuda"),
             pos=torch.full((most + 3,), -7, dtype=torch.int32, device="cuda"),
             ids=torch.full((most + 3,), -7, dtype=torch.int32, device="cuda"))
    return cache, t, table, free, free_n, most


def check_plan(kvq, L, n, maxp, free_n=None, most=None, seed=0, want_bits=None):
    cache, t, table, free, free_n, most = make_plan(kvq, L, n, maxp, free_n, most, seed)
    ws = cache.plan_workspace()
    cache.plan(t["new"], t["free"], t["count"], t["cu"], t["slots"][:most], t["pos"][:most], t["ids"][:most], ws)
    wt, wcu, ws_, wp, wi, left, bits = plan_reference(L, n, table, free, free_n, most)
    tot = len(ws_)
    assert np.array_equal(t["cu"].cpu().numpy(), wcu)
    assert np.array_equal(cache.page_table.cpu().numpy(), wt)
    for key, want in (("slots", ws_), ("pos", wp), ("ids", wi)):
        got = t[key].cpu().numpy()
        assert np.array_equal(got[:tot], want), key
        assert (got[tot:] == -7).all(), key                          # past the plan: as it was
    assert int(t["count"]) == left
    got = cache.read_status()
    assert got == (bits if want_bits is None else want_bits)


@pytest.mark.parametrize("L,n,maxp", [
    ([0], [1], 1), ([31], [1], 1), ([32], [1], 2), ([5, 0, 64, 31], [0, 0, 0, 0], 3), ([5, 0, 64, 31, 32], [1, 1, 1, 1, 1], 3),
    ([0, 100, 0, 7], [65, 0, 31, 33], 4), ([17] * 300, [1] * 300, 2), ([0] * 3, [5000, 0, 4001], 160), ([40, 3], [4096, 8191], 400),
    ([100, 0], [530000, 7], 16600),
])
def test_plan(kvq, L, n, maxp):
    check_plan(kvq, L, n, maxp)


def test_plan_of_many_ragged_requests(kvq):
    rng = np.random.default_rng(1)
    for B, hi in ((1023, 3), (1025, 60), (2600, 40)):
        L = rng.integers(0, 100, B).tolist()
        n = (rng.integers(0, hi, B) * (rng.random(B) < 0.7)).tolist()
        check_plan(kvq, L, n, 6, seed=B)


def test_plan_drops_bad_requests_and_stops_when_something_runs_out(kvq):
    OVER, NONE = kvq.KVQ_DEV_OVERFLOW, kvq.KVQ_DEV_NO_PAGES
    check_plan(kvq, [0, 96, 5, -3, 0], [10, 33, -1, 4, 40], 4, want_bits=OVER)           # each alone gets nothing
    check_plan(kvq, [0, 0, 0, 10], [64, 32, 33, 1], 3, free_n=4, want_bits=NONE)          # the third finds one page of two
    check_plan(kvq, [0, 0, 0], [10, 10, 10], 3, most=20, want_bits=OVER)
    check_plan(kvq, [0, 0], [10, 10], 3, free_n=0, want_bits=NONE)
    check_plan(kvq, [10, 10], [10, 10], 3, free_n=0)                                       # no new page needed
    check_plan(kvq, [0] * 2000, [3] * 2000, 1, free_n=1500, want_bits=NONE)
    check_plan(kvq, [0] * 2000, [3] * 2000, 1, most=4200, want_bits=OVER)


# ---- page bounds ---------------------------------------------------------------------------------

def key_cache(kvq, B, H, maxp, dt, lengths, seed=0, **kw):
    order = torch.randperm(B * maxp, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
    c = kvq.PagedKVCache(B, H, maxp * G, kw.pop("bits", 2), kw.pop("P", 1), dtype=kvq.KVQ_BF16 if dt == torch.bfloat16 else kvq.KVQ_F16,
                         page_order=order, **kw)
    c.seq_len.copy_(torch.tensor(lengths, dtype=torch.int32))
    return c


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,L,n", [(1, [0], 1), (2, [31, 32, 0], 1), (3, [5, 64, 31, 0], 2), (8, [0, 1, 33], 31), (2, [7, 32], 33),
                                   (1, [0, 63], 257), (5, [9, 40, 0, 31], 100)])
def test_page_bounds(kvq, dtype, H, L, n):
    dt, g, B = DT[dtype], gen(n), len(L)
    maxp = -(-(max(L) + n) // G)
    cache = key_cache(kvq, B, H, maxp, dt, L)
    bounds = randn(g, cache.num_pages, H, 2, D).to(dt)
    want = bounds.float().cpu().numpy()
    k = randn(g, B, n, H, D).to(dt)
    kf, table = k.float().cpu().numpy(), cache.page_table.cpu().numpy()
    for b in range(B):
        for i in range(n):
            p, at = table[b, (L[b] + i) // G], (L[b] + i) % G
            want[p, :, 0] = kf[b, i] if at == 0 else np.minimum(want[p, :, 0], kf[b, i])
            want[p, :, 1] = kf[b, i] if at == 0 else np.maximum(want[p, :, 1], kf[b, i])
    cache.update_bounds(k, bounds)
    assert np.array_equal(bounds.float().cpu().numpy(), want)
    assert cache.read_status() == 0 and cache.seq_len.tolist() == L


def test_page_bounds_with_special_values_full_tables_and_bad_pages(kvq):
    dt = torch.bfloat16
    cache = key_cache(kvq, 3, 1, 2, dt, [0, 60, 0])
    k = torch.zeros(3, 5, 1, D, dtype=dt, device="cuda")
    k[0, 1, 0, 0], k[0, 2, 0, 1], k[0, 3, 0, 2] = float("nan"), float("inf"), float("-inf")
    bounds = torch.full((6, 1, 2, D), 9.0, dtype=dt, device="cuda")
    cache.page_table[2, 0] = 6                                       # no such page
    cache.update_bounds(k, bounds)
    at = int(cache.page_table[0, 0])
    assert torch.isnan(bounds[at, 0, :, 0]).all()
    assert bounds[at, 0, :, 1].tolist() == [0.0, math.inf] and bounds[at, 0, :, 2].tolist() == [-math.inf, 0.0]
    others = [p for p in range(6) if p != at]
    assert (bounds[others] == 9.0).all()                             # the full sequence and the bad page: as they were
    assert cache.read_status(clear=True) == kvq.KVQ_DEV_OVERFLOW | kvq.KVQ_DEV_BAD_PAGE


# ---- selection -----------------------------------------------------------------------------------

def halved(x):
    while x.shape[-1] > 1:
        n = x.shape[-1] // 2
        x = (x[..., :n] + x[..., n:]).astype(np.float32)
    return x[..., 0]


def select_reference(q, bounds, table, L, H, budget, sink, recent):
    """fp32 in the documented order (numpy), the choice by a stable sort."""
    B, Gq = q.shape[0], q.shape[1] // H
    lists = np.full((B, H, budget), -1, np.int32)
    count = np.zeros((B, H), np.int32)
    for b in range(B):
        n = -(-int(L[b]) // G)
        for h in range(H):
            if n <= budget:
                lists[b, h, :n], count[b, h] = np.arange(n), n
                continue
            slot = np.zeros((16, D), np.float32)
            slot[:Gq] = q[b, h * Gq:(h + 1) * Gq]
            up, dn = halved(np.maximum(slot, 0).T), halved(np.minimum(slot, 0).T)
            mid = np.arange(sink, n - recent)
            bd = bounds[table[b, mid], h]
            with np.errstate(invalid="ignore", over="ignore"):
                t = (up * bd[:, 1]).astype(np.float32) + (dn * bd[:, 0]).astype(np.float32)
                s = halved(halved(t.reshape(-1, 16, 8)))
            rank = sorted(range(len(mid)), key=lambda i: (0 if np.isnan(s[i]) else 1, -float(s[i]) if not np.isnan(s[i]) else 0.0, i))
            best = sorted(mid[rank[:budget - sink - recent]])
            lists[b, h], count[b, h] = [*range(sink), *best, *range(n - recent, n)], budget
    return lists, count


def check_select(kvq, cache, q, bounds, budget, sink, recent, ws=None):
    B, H = cache.B, cache.H
    lists = torch.full((B, H, budget), -5, dtype=torch.int32, device="cuda")
    count = torch.full((B, H), -5, dtype=torch.int32, device="cuda")
    ws = cache.select_workspace() if ws is None else ws
    cache.select(q, bounds, lists, count, ws, sink, recent)
    want, n = select_reference(q.float().cpu().numpy(), bounds.float().cpu().numpy(), cache.page_table.cpu().numpy(),
                               cache.seq_len.cpu().numpy(), H, budget, sink, recent)
    assert np.array_equal(count.cpu().numpy(), n)
    assert np.array_equal(lists.cpu().numpy(), want)
    return ws


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("H,Gq,L,budget,sink,recent", [
    (1, 1, [1], 1, 0, 1), (1, 4, [33, 0, 32], 1, 0, 1), (2, 7, [1000, 0, 31, 96], 3, 1, 2), (2, 16, [2048, 2047], 8, 1, 1),
    (3, 5, [4099, 17, 640], 20, 0, 1), (1, 3, [70000 * 32 - 5], 33, 2, 3), (1, 8, [20000], 64, 3, 5), (4, 4, [9000] * 3, 63, 1, 2), (1, 2, [300000], 200, 1, 4),
])
def test_select_pages(kvq, dtype, H, Gq, L, budget, sink, recent):
    dt, g, B = DT[dtype], gen(budget), len(L)
    maxp = max(1, -(-max(L) // G))
    cache = key_cache(kvq, B, H, maxp, dt, L)
    q = randn(g, B, H * Gq, D).to(dt)
    mid, half = randn(g, cache.num_pages, H, 1, D), randn(g, cache.num_pages, H, 1, D).abs()
    bounds = torch.cat([mid - half, mid + half], 2).to(dt)
    ws = check_select(kvq, cache, q, bounds, budget, sink, recent)
    # ties everywhere: every page of a head has one of three bounds, so the lower pages win
    bounds[:] = bounds[torch.randint(0, 3, (cache.num_pages,), generator=g, device="cuda")]
    check_select(kvq, cache, q, bounds, budget, sink, recent, ws)
    bounds[:] = 0
    check_select(kvq, cache, q, bounds, budget, sink, recent, ws)
    assert cache.read_status() == 0


def near_ties(Gq, pages, dt):
    """Queries and page bounds whose scores lie within a few units of the last place of each other: one channel, with a hi that
    varies and the lo that brings u hi + n lo back to the same value as nearly as the type can."""
    g = torch.Generator().manual_seed(Gq + pages)
    q = torch.zeros(1, Gq, D)
    q[0, :, 77] = torch.randn(Gq, generator=g) * 0.3 ** torch.arange(Gq)   # W+ and W- of many bits
    q = q.to(dt)
    u, n = q[0, :, 77].double().clamp(min=0).sum(), q[0, :, 77].double().clamp(max=0).sum()
    hi = (1 + torch.rand(pages, generator=g)).to(dt)
    lo = ((u * 1.5 - u * hi.double()) / n).to(dt)
    bounds = torch.zeros(pages, 1, 2, D, dtype=dt)
    bounds[:, 0, 0, 77], bounds[:, 0, 1, 77] = lo, hi
    return q, bounds


@pytest.mark.parametrize("Gq,pages,budget", [(5, 1200, 376), (16, 264, 117), (10, 4000, 840)])
def test_select_rounds_every_product_on_its_own(kvq, Gq, pages, budget):
    """(With one rounding of u hi + fl(n lo) each of these would choose other pages.)"""
    dt = torch.float16
    cache = key_cache(kvq, 1, 1, pages, dt, [pages * G])
    q, bounds = near_ties(Gq, pages, dt)
    placed = torch.empty_like(bounds)
    placed[cache.page_table[0].long().cpu()] = bounds
    check_select(kvq, cache, q.cuda(), placed.cuda(), budget, 0, 1)


def test_select_with_infinities_and_nan(kvq):
    dt, g = torch.float16, gen(9)
    cache = key_cache(kvq, 1, 1, 40, dt, [40 * G])
    q = randn(g, 1, 2, D).to(dt)
    bounds = randn(g, 40, 1, 2, D).sort(2).values.to(dt)
    table = cache.page_table[0].tolist()
    bounds[table[7], 0, 1, 3] = float("nan")
    bounds[table[20], 0, 1] = float("inf")
    bounds[table[30], 0, 0] = float("-inf")
    bounds[table[9], 0, :, :] = float("-inf")
    check_select(kvq, cache, q, bounds, 8, 1, 1)
    q[0, 0, 5] = float("nan")                                       # every score NaN: the lower pages
    check_select(kvq, cache, q, bounds, 8, 1, 1)


def test_select_ranks_invalid_pages_last(kvq):
    g = gen(2)
    cache = key_cache(kvq, 1, 1, 20, torch.bfloat16, [20 * G])
    bounds = randn(g, 20, 1, 2, D).sort(2).values.to(torch.bfloat16)
    cache.page_table[0, 4:12] = 99
    lists = torch.zeros(1, 1, 12, dtype=torch.int32, device="cuda")
    n = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    cache.select(randn(g, 1, 4, D).to(torch.bfloat16), bounds, lists, n, cache.select_workspace(), 0, 1)
    assert lists[0, 0].tolist() == [*range(0, 4), *range(12, 20)]
    assert cache.read_status() == kvq.KVQ_DEV_BAD_PAGE


# ---- attention over chosen pages -----------------------------------------------------------------

def filled(kvq, B, H, N, bits, P, dt, tx=0, seed=0, lengths=None, sets=1, v_rho=0.3, in_use=None, outlier=15.0):
    """A cache of N appended tokens (patterns: rows of the data), then cut to `lengths`' full pages is not possible, so
    each sequence is appended alone through a cache view of its own length."""
    g = gen(seed)
    lengths = [N] * B if lengths is None else lengths
    cache = key_cache(kvq, B, H, max(1, -(-max(lengths) // G)), dt, [0] * B, seed, bits=bits, P=P, transform=tx, num_sets=sets, v_rho=v_rho,
                      seq_to_set=torch.arange(B, dtype=torch.int32) % sets if sets > 1 else None,
                      patterns_in_use=in_use)
    k, v = randn(g, B, max(max(lengths), P), H, D), randn(g, B, max(max(lengths), P), H, D)
    k[..., 5:120:16] *= outlier
    if tx:
        cache.k_colscale.copy_(3 + 9 * torch.rand(sets, H, D, generator=g, device="cuda"))
        cache.v_colscale.copy_(3 + 9 * torch.rand(sets, H, D, generator=g, device="cuda"))
        cache.k_patterns.normal_(generator=g)
        cache.v_patterns.normal_(generator=g)
    else:
        cache.k_patterns.copy_(k[0, :P].transpose(0, 1))
        cache.v_patterns.copy_(v[0, :P].transpose(0, 1))
    if in_use:
        cache.k_patterns[:, :, in_use:] = float("nan")               # capacity that nothing may look at
        cache.v_patterns[:, :, in_use:] = float("nan")
    k, v = k.to(dt), v.to(dt)
    ws = cache.append_workspace()
    import ctypes
    for b, n in enumerate(lengths):
        if n == 0:
            continue
        one = kvq.kvq_cache()
        ctypes.memmove(ctypes.byref(one), ctypes.byref(cache.c), ctypes.sizeof(one))
        one.num_seqs = 1
        one.page_table += 4 * b * cache.maxp
        one.seq_len += 4 * b
        one.k_tail += 2 * b * H * G * D
        if one.seq_to_set:
            one.seq_to_set += 4 * b
        kvq.kvq_quantize_append(one, k[b:b + 1, :n].contiguous(), v[b:b + 1, :n].contiguous(), n, ws)
    assert cache.read_status() == 0 and cache.seq_len.tolist() == lengths
    return cache


def rebuilt(kvq, cache, b):
    n = int(cache.seq_len[b])
    k = torch.empty(n, cache.H, D, device="cuda")
    v = torch.empty_like(k)
    kvq.kvq_dequantize(cache.c, b, n, 0, n, k, v)
    return k.double(), v.double()


def attend_reference(kvq, cache, q, lists, counts, scale):
    """float64 softmax over the listed pages' tokens of the reconstructed cache, and a bound of the kernel's error.

    A logit is a sum of q_d s_d code, q_d z_d and q_d M_d, each below |q_d| 4 R_d (R the largest |k_d|), carried with 21 or
    more bits: off by at most delta = 2^-20 12 scale sum_d |q_d| R_d.  A softmax weight is then off by 2 delta of itself,
    which moves the output by 2 delta S, S = sum_t p_t max |v_t|; p s code, p z and W M, carried alike, by 2^-20 12 S; and
    each of the n tokens' weights in W is rounded to 2^-20 of the largest, 4 max_t p_t max |v_t| 2^-20 in the output."""
    B, H = cache.B, cache.H
    Gq = q.shape[1] // H
    out = torch.zeros(B, H * Gq, D, dtype=torch.float64, device="cuda")
    err = torch.zeros(B, H * Gq, 1, dtype=torch.float64, device="cuda")
    for b in range(B):
        if int(cache.seq_len[b]) == 0:
            continue
        k, v = rebuilt(kvq, cache, b)
        for h in range(H):
            pages = lists[b, h, :int(counts[b, h])].long()
            t = (pages[:, None] * G + torch.arange(G, device="cuda")).flatten()
            t = t[t < k.shape[0]]
            if len(t) == 0:
                continue
            qs = q[b, h * Gq:(h + 1) * Gq].double()
            p = torch.softmax(qs @ k[t, h].T * scale, -1)
            out[b, h * Gq:(h + 1) * Gq] = p @ v[t, h]
            delta = 2.0 ** -20 * 12 * scale * (qs.abs() @ k[:, h].abs().amax(0))
            each = p * v[t, h].abs().amax(-1)
            err[b, h * Gq:(h + 1) * Gq, 0] = (2 * delta + 2.0 ** -20 * 12) * each.sum(-1) + len(t) * 2.0 ** -20 * 4 * each.amax(-1)
    return out, err


def random_lists(cache, budget, seed, newest=True):
    B, H = cache.B, cache.H
    rng = np.random.default_rng(seed)
    lists, n = np.full((B, H, budget), -1, np.int32), np.zeros((B, H), np.int32)
    for b in range(B):
        pages = -(-int(cache.seq_len[b]) // G)
        for h in range(H):
            take = min(budget, pages) if rng.random() < 0.8 else int(rng.integers(0, min(budget, pages) + 1))
            pick = rng.permutation(pages)[:take]
            if newest and take and pages - 1 not in pick:
                pick[0] = pages - 1
            lists[b, h, :take], n[b, h] = pick, take
    return torch.from_numpy(lists).cuda(), torch.from_numpy(n).cuda()


def attend(cache, q, lists, n, scale=None, ws=None, **kw):
    out = torch.full((cache.B, q.shape[1], D), float("nan"), dtype=q.dtype, device="cuda")
    ws = cache.decode_pages_workspace(q.shape[1], lists.shape[-1]) if ws is None else ws
    cache.decode_pages(q, lists, n, out, ws, scale, **kw)
    return out


@pytest.mark.parametrize("dtype,bits,tx,H,Gq,P,lengths,budget", [
    ("bf16", 2, 0, 1, 1, 1, [1], 1), ("bf16", 4, 0, 2, 4, 16, [700, 0, 32, 31], 9), ("fp16", 2, 0, 2, 4, 64, [700, 5, 33, 96], 40),
    ("bf16", 4, 1, 2, 7, 8, [321, 64, 1], 6), ("fp16", 2, 1, 1, 7, 30, [1000, 999], 32), ("fp16", 4, 0, 1, 16, 255, [513, 512], 17),
    ("bf16", 2, 0, 3, 12, 100, [250, 640, 31], 8), ("bf16", 4, 0, 8, 4, 64, [5000], 64), ("fp16", 2, 0, 4, 2, 17, [2100] * 5, 33),
    ("bf16", 2, 0, 2, 5, 33, [4000] * 2, 126), ("fp16", 4, 1, 1, 9, 64, [3000, 40], 50),
    ("bf16", 4, 0, 1, 4, 64, [40007], 1251), ("fp16", 2, 0, 1, 8, 16, [9000, 8000], 6000), ("bf16", 2, 1, 1, 16, 255, [4001], 126),
])
def test_attention_over_pages(kvq, dtype, bits, tx, H, Gq, P, lengths, budget):
    dt = DT[dtype]
    cache = filled(kvq, len(lengths), H, 0, bits, P, dt, tx, seed=P, lengths=lengths)
    q = randn(gen(1), len(lengths), H * Gq, D).to(dt)
    for seed, newest, scale in ((0, True, D ** -0.5), (1, False, 0.3 * D ** -0.5)):
        lists, n = random_lists(cache, budget, seed, newest)
        out = attend(cache, q, lists, n, scale)
        within(out, *attend_reference(kvq, cache, q, lists, n, scale))
    assert cache.read_status() == 0


def test_attention_with_an_odd_number_of_partial_rows(kvq):
    # one query head of one sequence, a list long enough for splits through the workspace, of which there is an odd number
    cache = filled(kvq, 1, 1, 0, 4, 16, torch.bfloat16, lengths=[9000])
    q = randn(gen(2), 1, 1, D).to(torch.bfloat16)
    splits = lambda n: (kvq.kvq_decode_pages_workspace_bytes(cache.c, 1, n) - 256) // (130 * 4)   # noqa: E731
    odd = [n for n in range(17, 282) if splits(n) > 16 and splits(n) % 2]
    assert odd
    for budget in (odd[0], odd[len(odd) // 2], odd[-1]):
        lists, n = random_lists(cache, budget, 1)
        within(attend(cache, q, lists, n), *attend_reference(kvq, cache, q, lists, n, D ** -0.5))


def test_attention_over_every_page_is_decode_attention(kvq):
    cache = filled(kvq, 3, 2, 0, 4, 16, torch.bfloat16, lengths=[900, 31, 256])
    q = randn(gen(5), 3, 8, D).to(torch.bfloat16)
    lists = torch.arange(29, dtype=torch.int32, device="cuda").expand(3, 2, 29).contiguous()
    n = torch.tensor([[29, 29], [1, 1], [8, 8]], dtype=torch.int32, device="cuda")
    full = torch.empty(3, 8, D, device="cuda")
    cache.decode(q, full, cache.decode_workspace(8))
    out = attend(cache, q, lists, n)
    # the two kernels' errors: the tested 2e-3 of the largest value of decode attention, and half a step
    within(out, full.double(), 2e-3 * full.abs().amax(-1, keepdim=True).double())


def test_attention_sets_patterns_in_use_and_raw_values(kvq):
    # sequences with pattern sets of their own, half of each set's rows in use, and most values stored raw
    cache = filled(kvq, 3, 2, 0, 2, 16, torch.float16, lengths=[300, 40, 97], sets=3, v_rho=0.05, in_use=7)
    for s in range(1, 3):
        assert not torch.equal(cache.k_patterns[s, :, :7], torch.zeros_like(cache.k_patterns[s, :, :7]))
    q = randn(gen(6), 3, 8, D).to(torch.float16)
    lists, n = random_lists(cache, 10, 3)
    within(attend(cache, q, lists, n), *attend_reference(kvq, cache, q, lists, n, D ** -0.5))


def test_attention_list_order_duplicates_and_reuse(kvq):
    cache = filled(kvq, 2, 2, 0, 4, 8, torch.bfloat16, lengths=[640, 333])
    q = randn(gen(7), 2, 8, D).to(torch.bfloat16)
    ws = cache.decode_pages_workspace(8, 64)
    lists, n = random_lists(cache, 10, 4)
    first = attend(cache, q, lists, n, ws=ws)
    assert torch.equal(first, attend(cache, q, lists, n, ws=ws))      # same bits again, on the same workspace
    # a page listed twice counts twice
    twice = torch.cat([lists, lists[..., :1]], -1).contiguous()
    for b in range(2):
        for h in range(2):
            twice[b, h, int(n[b, h])] = lists[b, h, 0]
    within(attend(cache, q, twice, n + 1, ws=ws), *attend_reference(kvq, cache, q, twice, n + 1, D ** -0.5))
    within(attend(cache, q, lists, n, ws=ws), *attend_reference(kvq, cache, q, lists, n, D ** -0.5))


def test_attention_without_entries_is_zero_and_bad_entries_are_passed_over(kvq):
    cache = filled(kvq, 2, 1, 0, 2, 4, torch.bfloat16, lengths=[200, 70])
    q = randn(gen(8), 2, 3, D).to(torch.bfloat16)
    lists = torch.full((2, 1, 12), -1, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    assert (attend(cache, q, lists, n) == 0).all() and cache.read_status() == 0
    good = torch.tensor([[[6, 2]], [[0, 1]]], dtype=torch.int32, device="cuda")
    want = attend_reference(kvq, cache, q, good, torch.full_like(n, 2), D ** -0.5)
    lists[:, :, 4:6] = good                                          # entries that name no page of their sequence around them
    lists[0, 0, 0], lists[1, 0, 0], lists[1, 0, 1] = 7, 3, 2 ** 31 - 1
    n[:] = 12
    within(attend(cache, q, lists, n), *want)
    assert cache.read_status(clear=True) == kvq.KVQ_DEV_BAD_PAGE
    n[0], n[1] = 13, -1
    assert (attend(cache, q, lists, n) == 0).all()
    assert cache.read_status(clear=True) == kvq.KVQ_DEV_OVERFLOW
    was = int(cache.page_table[0, 2])
    cache.page_table[0, 2] = -4                                      # a listed page with an invalid id
    out = attend(cache, q, good, torch.full_like(n, 2))
    cache.page_table[0, 2] = was
    only = torch.tensor([[[6, -1]], [[0, 1]]], dtype=torch.int32, device="cuda")
    assert cache.read_status(clear=True) == kvq.KVQ_DEV_BAD_PAGE
    within(out, *attend_reference(kvq, cache, q, only, torch.tensor([[1], [2]], device="cuda"), D ** -0.5))


@pytest.mark.parametrize("B,H,Gq,budget,tx", [(40, 8, 4, 3, 0), (1, 1, 4, 8, 0), (1, 2, 5, 60, 1), (1, 1, 16, 60, 0), (3, 1, 8, 61, 1)])
def test_a_nan_in_a_query_shows_in_its_head_only(kvq, B, H, Gq, budget, tx):
    """(One group and 60 pages: splits that meet in the workspace; 8: in a cluster; 320 groups: none.)"""
    dt = torch.bfloat16
    cache = filled(kvq, B, H, 61 * G if B < 40 else 3 * G + 5, 4, 8, dt, tx=tx)
    q = randn(gen(5), B, H * Gq, D).to(dt)
    lists, n = random_lists(cache, budget, 6)
    assert n[0, 0] > 0
    want = attend(cache, q, lists, n)
    q[0, Gq // 2, 17] = float("nan")
    got = attend(cache, q, lists, n)
    assert torch.isnan(got[0, Gq // 2]).all()
    got[0, Gq // 2] = want[0, Gq // 2]
    # the others: the same sums up to an fp32 rounding of a rescaled weight (2^-24), so at most the neighbouring number
    assert torch.allclose(got.float(), want.float(), rtol=torch.finfo(dt).eps, atol=1e-6)


def test_attention_of_extreme_rows(kvq):
    # a zero query (every token weighs the same), one query head far above the others, and tiny values
    cache = filled(kvq, 1, 1, 0, 4, 4, torch.float16, lengths=[160])
    q = randn(gen(9), 1, 4, D).to(torch.float16)
    q[0, 0], q[0, 1], q[0, 2] = 0, q[0, 1] * 50, q[0, 2] * 2.0 ** -12
    lists, n = random_lists(cache, 5, 0)
    within(attend(cache, q, lists, n), *attend_reference(kvq, cache, q, lists, n, D ** -0.5))


def test_attention_when_the_largest_row_factors_do_not_count(kvq):
    # under the pre-transform, a page whose values are 2^14 times the others' but whose keys score far below
    cache = filled(kvq, 1, 1, 0, 4, 8, torch.float16, tx=1, lengths=[320])
    cb = 32 * D * 4 // 8
    for page, factor in ((3, 2.0 ** 14), (7, 2.0 ** -6)):
        f = cache.subblock(0, page, 0).view(torch.float32)
        f[(2 * cb + 2112) // 4:(2 * cb + 2240) // 4] = 0.0           # its keys are zero vectors
        f[(2 * cb + 2240) // 4:] *= factor
    q = (6 * randn(gen(3), 1, 4, D)).to(torch.float16)
    for order in ([3, 0, 1, 2, 4, 5, 6, 7, 8, 9], [9, 8, 7, 3, 2, 1, 0]):
        lists = torch.tensor(order, dtype=torch.int32, device="cuda").view(1, 1, -1).contiguous()
        n = torch.full((1, 1), len(order), dtype=torch.int32, device="cuda")
        want, err = attend_reference(kvq, cache, q, lists, n, D ** -0.5)
        assert float(want.abs().max()) < 100                         # page 3 has no weight
        within(attend(cache, q, lists, n), want, err)


# ---- streams, graphs, devices --------------------------------------------------------------------

def test_a_captured_step_replays_on_new_inputs(kvq):
    """rows -> bounds -> append + decode of one step -> selection -> attention, captured once and replayed."""
    B, H, Gq, steps, budget = 3, 2, 4, 40, 4
    caches = [filled(kvq, B, H, 0, 4, 8, torch.bfloat16, lengths=[150, 3, 64], seed=11) for _ in range(2)]
    # room for the steps: tables with more columns than the prefill needs
    for i, c in enumerate(caches):
        big = kvq.PagedKVCache(B, H, 320, 4, 8, v_rho=0.3)
        for b, n in enumerate((150, 3, 64)):
            for p in range(-(-n // G)):
                at, to = int(c.page_table[b, p]) * c.page_bytes, int(big.page_table[b, p]) * big.page_bytes
                big.pool[to:to + c.page_bytes] = c.pool[at:at + c.page_bytes]
        for name in ("seq_len", "k_tail", "k_patterns", "v_patterns"):
            getattr(big, name).copy_(getattr(c, name))
        caches[i] = big
    g = gen(12)
    w = (1 + 0.2 * randn(g, D)).to(torch.bfloat16)
    inv = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float32) / 64)
    qkv = [randn(g, B, (H * Gq + 2 * H), D).to(torch.bfloat16) for _ in range(steps)]

    class Step:
        def __init__(self, cache):
            self.c, z = cache, lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")   # noqa: E731
            self.x, self.q, self.k, self.v, self.out = z(B, H * Gq + 2 * H, D), z(B, H * Gq, D), z(B, H, D), z(B, H, D), z(B, H * Gq, D)
            self.full = torch.zeros(B, H * Gq, D, device="cuda")
            self.bounds = cache.bounds()
            self.lists = torch.zeros(B, H, budget, dtype=torch.int32, device="cuda")
            self.n = torch.zeros(B, H, dtype=torch.int32, device="cuda")
            self.ws = cache.step_workspace(H * Gq), cache.select_workspace(), cache.decode_pages_workspace(H * Gq, budget)

        def run(self):
            hq = H * Gq
            kvq.kvq_norm_rope(self.x[:, :hq], self.x[:, hq:hq + H], self.x[:, hq + H:], self.c.seq_len, inv, self.q, self.k, self.v, w, w)
            self.c.update_bounds(self.k.view(B, 1, H, D), self.bounds)
            self.c.step(self.k, self.v, self.q, self.full, self.ws[0])
            self.c.select(self.q, self.bounds, self.lists, self.n, self.ws[1])
            self.c.decode_pages(self.q, self.lists, self.n, self.out, self.ws[2])

    eager, replay = Step(caches[0]), Step(caches[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    saved = {n: getattr(replay.c, n).clone() for n in ("seq_len", "k_tail", "pool")}
    with torch.cuda.stream(s):
        replay.run()                                                 # warm-up, then its state put back
        for n, t in saved.items():
            getattr(replay.c, n).copy_(t)
        replay.bounds.zero_()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            replay.run()
    torch.cuda.current_stream().wait_stream(s)
    for t in range(steps):
        for x in (eager, replay):
            x.x.copy_(qkv[t])
        eager.run()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.n, replay.n) and torch.equal(eager.lists, replay.lists)
        assert torch.equal(eager.out, replay.out) and torch.equal(eager.k, replay.k)
        if t in (0, 1, 28, 29, steps - 1):
            within(eager.out, *attend_reference(kvq, eager.c, eager.q, eager.lists, eager.n, D ** -0.5))
    assert torch.equal(eager.bounds, replay.bounds)
    assert eager.c.read_status() == 0 and replay.c.read_status() == 0


def test_a_serving_run_from_an_empty_table(kvq):
    """Prompts, then steps of one token: plan -> rows -> bounds -> append -> selection -> attention, pages off one stack."""
    B, H, Gq, prompt, steps, budget, maxp = 3, 2, 4, 70, 45, 3, 6
    cache = kvq.PagedKVCache(B, H, maxp * G, 4, 8, page_order=torch.full((B * maxp,), -1, dtype=torch.int32), v_rho=0.3)
    g = gen(21)
    cache.k_patterns.normal_(generator=g)
    cache.v_patterns.normal_(generator=g)
    free = torch.randperm(cache.num_pages, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor([cache.num_pages], dtype=torch.int32, device="cuda")
    bounds, plan_ws, sel_ws = cache.bounds(), cache.plan_workspace(), cache.select_workspace()
    att_ws = cache.decode_pages_workspace(H * Gq, budget)
    lists, n = torch.zeros(B, H, budget, dtype=torch.int32, device="cuda"), torch.zeros(B, H, dtype=torch.int32, device="cuda")
    inv = 10000.0 ** (-torch.arange(64, device="cuda", dtype=torch.float32) / 64)
    w = (1 + 0.2 * randn(g, D)).to(torch.bfloat16)
    out = torch.zeros(B, H * Gq, D, dtype=torch.bfloat16, device="cuda")
    keys, length = [], 0
    for new in [prompt] + [1] * steps:
        T = B * new
        i32 = lambda *s: torch.full(s, -1, dtype=torch.int32, device="cuda")   # noqa: E731
        cu, pos, ids, slots = i32(B + 1), i32(T), i32(T), torch.full((T,), -1, dtype=torch.int64, device="cuda")
        cache.plan(torch.full((B,), new, dtype=torch.int32, device="cuda"), free, count, cu, slots, pos, ids, plan_ws)
        x = randn(g, T, H * Gq + 2 * H, D).to(torch.bfloat16)
        z = lambda h: torch.empty(T, h, D, dtype=torch.bfloat16, device="cuda")   # noqa: E731
        q, k, v = z(H * Gq), z(H), z(H)
        kvq.kvq_norm_rope(x[:, :H * Gq], x[:, H * Gq:H * Gq + H], x[:, H * Gq + H:], pos, inv, q, k, v, w, w)
        kb, vb = k.view(B, new, H, D), v.view(B, new, H, D)
        cache.update_bounds(kb, bounds)
        cache.append(kb, vb)
        keys.append(kb)
        length += new
        at = torch.arange(T, device="cuda")
        assert torch.equal(pos.long(), length - new + at % new) and torch.equal(ids.long(), at // new)
        assert torch.equal(slots, cache.page_table[ids.long(), pos.long() // G].long() * G + pos.long() % G)
        last = q.view(B, new, H * Gq, D)[:, -1].contiguous()
        cache.select(last, bounds, lists, n, sel_ws, sink=1, recent=1)
        cache.decode_pages(last, lists, n, out, att_ws)
        if length in (70, 71, 96, 97, 115):
            within(out, *attend_reference(kvq, cache, last, lists, n, D ** -0.5))
            want, wn = select_reference(last.float().cpu().numpy(), bounds.float().cpu().numpy(), cache.page_table.cpu().numpy(),
                                        cache.seq_len.cpu().numpy(), H, budget, 1, 1)
            assert np.array_equal(lists.cpu().numpy(), want) and np.array_equal(n.cpu().numpy(), wn)
    allk = torch.cat(keys, 1).float()
    for b in range(B):
        for p in range(-(-length // G)):
            rows = allk[b, p * G:(p + 1) * G]
            page = bounds[int(cache.page_table[b, p])].float()
            assert torch.equal(page[:, 0], rows.amin(0)) and torch.equal(page[:, 1], rows.amax(0))
    used = cache.page_table[cache.page_table >= 0]
    assert used.unique().numel() == used.numel() == B * 4 and int(count) == cache.num_pages - used.numel()
    assert cache.read_status() == 0 and cache.seq_len.tolist() == [length] * B


def test_two_calls_at_once_on_two_streams(kvq):
    cache = filled(kvq, 2, 2, 0, 4, 8, torch.bfloat16, lengths=[3000, 2000])
    qs = [randn(gen(s), 2, 8, D).to(torch.bfloat16) for s in range(2)]
    bounds = randn(gen(8), cache.num_pages, 2, 2, D).sort(2).values.to(torch.bfloat16)
    work = [dict(lists=torch.zeros(2, 2, 40, dtype=torch.int32, device="cuda"), n=torch.zeros(2, 2, dtype=torch.int32, device="cuda"),
                 out=torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda"), sel=cache.select_workspace(),
                 att=cache.decode_pages_workspace(8, 40), stream=torch.cuda.Stream()) for _ in range(2)]

    def go(w, q, stream):
        cache.select(q, bounds, w["lists"], w["n"], w["sel"], stream=stream)
        cache.decode_pages(q, w["lists"], w["n"], w["out"], w["att"], stream=stream)

    want = []
    for w, q in zip(work, qs):
        go(w, q, None)
        want.append((w["lists"].clone(), w["out"].clone()))
    for _ in range(20):
        for w in work:
            w["lists"].zero_()
            w["out"].zero_()
        torch.cuda.synchronize()
        for w, q in zip(work, qs):
            go(w, q, w["stream"])
        torch.cuda.synchronize()
        for w, (lists, out) in zip(work, want):
            assert torch.equal(w["lists"], lists) and torch.equal(w["out"], out)


@pytest.mark.parametrize("B", [3, 2100])
def test_a_captured_plan_pops_the_stack_on_every_replay(kvq, B):
    # both forms of the call (one launch, two): three steps of a token each, by replays of one graph
    L, n, maxp = [31] * B, [1] * B, 3
    cache, t, table, free, free_n, most = make_plan(kvq, L, n, maxp)
    ws = cache.plan_workspace()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        cache.plan(t["new"], t["free"], t["count"], t["cu"], t["slots"][:most], t["pos"][:most], t["ids"][:most], ws)
        cache.seq_len.add_(1)
    torch.cuda.current_stream().wait_stream(s)
    left = free_n
    for step in range(35):
        graph.replay()
        table, cu, slots, pos, ids, left, bits = plan_reference([31 + step] * B, n, table, free, left, most)
        if step in (0, 1, 33, 34):
            assert np.array_equal(cache.page_table.cpu().numpy(), table) and int(t["count"]) == left
            assert t["slots"][:most].tolist() == slots and t["pos"][:most].tolist() == pos and t["ids"][:most].tolist() == ids
    assert cache.read_status() == 0


FAILURE = """
    import sys
    sys.path.insert(0, {root!r})
    sys.path.insert(0, {tests!r})
    import torch
    import bit_kv_cache_26_b200 as kvq
    from test_serving_gpu import attend, filled, gen, random_lists, randn
    cache = filled(kvq, 2, 2, 0, 4, 8, torch.bfloat16, lengths=[300, 40])
    lists, n = random_lists(cache, 10, 0)
    attend(cache, randn(gen(0), 2, 8, 128).to(torch.bfloat16), lists, n)
    bits = cache.read_status(clear=True)
    assert bits & kvq.KVQ_DEV_TIMEOUT, hex(bits)
    assert torch.arange(1 << 20, device="cuda").sum().item() == (1 << 19) * ((1 << 20) - 1)
    print("timeout flagged")
"""


def test_expired_page_waits_are_flagged():
    # every page wait gives up at once: the status says so, the copies in flight are waited for, the context stays usable
    import os
    import subprocess
    import sys
    import textwrap

    from conftest import ROOT
    code = textwrap.dedent(FAILURE).format(root=ROOT, tests=os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], env=dict(os.environ, KVQ_TEST_WAIT_LIMIT="0"), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "timeout flagged" in r.stdout, r.stdout + r.stderr


def test_calls_on_a_stream_of_their_own(kvq):
    cache = filled(kvq, 2, 2, 0, 4, 8, torch.bfloat16, lengths=[640, 333])
    q = randn(gen(7), 2, 8, D).to(torch.bfloat16)
    bounds = randn(gen(8), cache.num_pages, 2, 2, D).sort(2).values.to(torch.bfloat16)
    lists = torch.zeros(2, 2, 8, dtype=torch.int32, device="cuda")
    n = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    ws = cache.select_workspace()
    cache.select(q, bounds, lists, n, ws)
    want = attend(cache, q, lists, n)
    torch.cuda.synchronize()
    lists.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    cache.select(q, bounds, lists, n, ws, stream=s)
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    cache.decode_pages(q, lists, n, out, cache.decode_pages_workspace(8, 8), stream=s)
    s.synchronize()
    assert torch.equal(out, want)


def test_the_binding_refuses_wrong_tensors(kvq):
    cache = filled(kvq, 2, 2, 0, 4, 8, torch.bfloat16, lengths=[64, 64])
    q = torch.zeros(2, 8, D, dtype=torch.bfloat16, device="cuda")
    lists, n = torch.zeros(2, 2, 4, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    ws = cache.decode_pages_workspace(8, 4)
    for args in ((q.half(), lists, n), (q, lists.long(), n), (q, lists, n[:1]), (q[:, :, ::2], lists, n), (q.cpu(), lists, n),
                 (q, lists.transpose(0, 1), n)):
        with pytest.raises(kvq.KvqError):
            cache.decode_pages(*args, torch.empty_like(q), ws)
    with pytest.raises(kvq.KvqError):
        cache.decode_pages(q, lists, n, torch.empty(2, 8, D, device="cuda"), ws)
    with pytest.raises(kvq.KvqError):
        cache.decode_pages(q, lists, n, torch.empty_like(q), ws[:64])
    with pytest.raises(kvq.KvqError):
        cache.update_bounds(torch.zeros(2, 1, 2, D, device="cuda"), cache.bounds())
    x = torch.zeros(4, 2, D, dtype=torch.bfloat16, device="cuda")
    for bad in (x[:, :1], x.half(), x[..., :64], x[:3]):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_norm_rope(x, None, None, None, None, bad, None, None)
    with pytest.raises(kvq.KvqError):                                # a rotation without positions
        kvq.kvq_norm_rope(x, None, None, None, torch.ones(64, device="cuda"), x, None, None)
