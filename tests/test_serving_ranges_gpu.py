"""Attention over chosen pages where weights and values span many powers of two, against float64.

A dominant token of small value (an attention sink) leaves the output to the small weights of the others, so the bound of
the error follows sum_t p_t |v_t| and not the largest weight: each logit is off by at most
delta = 2^-20 12 scale sum_d |q_d| R_d (R the largest |k_d|), which moves the output by 2 delta S, S = sum_t p_t max |v_t|, and
p s code, p z and W M (each below 4 |v|) are carried to 2^-20 of themselves: 2^-20 12 S."""
import pytest
import torch

from test_serving_gpu import D, DT, G, attend, gen, key_cache, randn, rebuilt, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    import bit_kv_cache_26_b200 as m
    return m


def sink_cache(kvq, dt, bits, Gq, pages, at, nats, values, tx=0, sink_value=0.0):
    """One sequence and KV head whose token `at` scores `nats` above the rest and has the value `sink_value`; the other
    values are near one of 16 patterns, of size `values`."""
    g, P, n = gen(pages + bits), 16, pages * G - 5
    cache = key_cache(kvq, 1, 1, pages, dt, [0], 1, bits=bits, P=P, transform=tx, v_rho=0.3)
    k, v = 0.05 * randn(g, n, D), torch.empty(n, D, device="cuda")
    sign = torch.where(randn(g, D) > 0, 1.0, -1.0)
    k[at] = sign * (nats / D ** 0.5)
    cache.k_patterns.copy_(k[1:P + 1])
    if tx:
        cache.k_colscale.fill_(1.0)
        cache.v_colscale.fill_(1.0)
        cache.k_patterns.normal_(generator=g)
        cache.v_patterns.normal_(generator=g)
        v = values * randn(g, n, D)
    else:
        cache.v_patterns.copy_(values * randn(g, P, D))
        pick = torch.randint(0, P, (n,), generator=g, device="cuda")
        v = cache.v_patterns[0, 0, pick] + 0.05 * values * randn(g, n, D)
    v[at] = sink_value
    cache.append(k.view(1, n, 1, D).to(dt), v.view(1, n, 1, D).to(dt))
    q = (sign + 0.02 * randn(g, 1, Gq, D)).to(dt)
    assert cache.read_status() == 0
    return cache, q


def check(kvq, cache, q, order):
    lists = torch.tensor(order, dtype=torch.int32, device="cuda").view(1, 1, -1)
    n = torch.full((1, 1), len(order), dtype=torch.int32, device="cuda")
    k, v = rebuilt(kvq, cache, 0)
    assert torch.isfinite(k).all() and torch.isfinite(v).all()
    t = (lists[0, 0].long()[:, None] * G + torch.arange(G, device="cuda")).flatten()
    t = t[t < k.shape[0]]
    k, v, qs, scale = k[t, 0], v[t, 0], q[0].double(), D ** -0.5
    p = torch.softmax(qs @ k.T * scale, -1)
    S = (p * v.abs().amax(-1)).sum(-1, keepdim=True)
    delta = 2.0 ** -20 * 12 * scale * (qs.abs() @ k.abs().amax(0))[:, None]
    out = attend(cache, q, lists, n)
    assert cache.read_status(clear=True) == 0
    within(out, (p @ v)[None], ((2 * delta + 2.0 ** -20 * 12) * S)[None])
    return p, S


@pytest.mark.parametrize("dtype,bits,Gq,pages,tx", [("bf16", 4, 4, 40, 0), ("fp16", 2, 3, 40, 0), ("bf16", 2, 7, 12, 0), ("fp16", 4, 16, 5, 0),
                                                    ("bf16", 4, 1, 1, 0), ("bf16", 4, 2, 9, 1)])
@pytest.mark.parametrize("nats", [10, 13, 16])
@pytest.mark.parametrize("last", [False, True])
def test_a_dominant_token_of_no_value_leaves_the_others(kvq, dtype, bits, Gq, pages, tx, nats, last):
    at = (pages - 1) * G + 9 if last else 0
    cache, q = sink_cache(kvq, DT[dtype], bits, Gq, pages, at, nats, 1.0, tx)
    for order in (list(range(pages)), list(range(pages))[::-1]):
        p, _ = check(kvq, cache, q, order)
        assert float(p.max(-1).values.min()) > 0.9 or nats < 13      # the sink has most of the weight


@pytest.mark.parametrize("dtype,bits,Gq,pages,tx", [("bf16", 4, 4, 40, 0), ("bf16", 2, 7, 12, 0), ("fp16", 2, 4, 40, 0), ("bf16", 2, 12, 5, 0),
                                                    ("bf16", 4, 2, 9, 1)])
@pytest.mark.parametrize("values,nats", [(1e-5, 0), (1e-6, 12), (1e-3, 14), (1e-3, 20), (3e-5, 16), (6e4, 0), (3e4, 12)])
def test_small_and_large_values_keep_their_bits(kvq, dtype, bits, Gq, pages, tx, values, nats):
    if dtype == "fp16":
        values = min(max(values, 1e-3), 1e3)                         # what the type holds, and what the reconstruction must stay below
    cache, q = sink_cache(kvq, DT[dtype], bits, Gq, pages, 0, nats, values, tx)
    for order in (list(range(pages)), list(range(pages))[::-1]):
        check(kvq, cache, q, order)
    if bits == 2 and values == 6e4 and tx == 0:                      # scales that no fp16 holds
        at = 2 * (G * D * bits // 8) + 1024
        assert float(cache.subblock(0, 1, 0)[at:at + 512].view(torch.float32).max()) > 2000


def test_pages_of_very_different_values(kvq):
    # pages whose values are 2^-20 .. 2^20 times the others', in both orders and alone
    cache, q = sink_cache(kvq, torch.bfloat16, 4, 5, 6, 0, 0, 1.0)
    at = 2 * (G * D * 4 // 8) + 1024
    for page, f in ((1, 2.0 ** -20), (3, 2.0 ** 20), (4, 2.0 ** -60)):
        sub = cache.subblock(0, page, 0)
        sub[at:at + 1024].view(torch.float32).mul_(f)                # scales and zeros
        sub[at + 1056:at + 1088] = 255                               # without patterns
    for order in ([0, 1, 2, 3, 4, 5], [3, 1, 0], [1, 4], [4], [1, 0], [5, 4, 3, 2, 1, 0]):
        check(kvq, cache, q, order)


@pytest.mark.parametrize("tx", [0, 1])
@pytest.mark.parametrize("pages", [1, 8, 64])                        # one CTA, a cluster, splits that meet in the workspace
def test_outputs_past_the_type_are_flagged(kvq, pages, tx):
    cache, q = sink_cache(kvq, torch.float16, 4, 4, pages, 0, 0, 1.0, tx)
    order = list(range(pages))
    at = 2 * (G * D * 4 // 8) + 1024
    for b in range(pages):                                           # values of 1 where they were, without patterns and transform
        sub = cache.subblock(0, b, 0)
        f = sub[at:at + 1024].view(torch.float32)
        f[:128], f[128:] = 0.0, 1.0
        sub[at + 1056:at + 1088] = 255
        if tx:
            sub[at + 1088 + 128:at + 1088 + 256].view(torch.float32).fill_(1.0)
    lists = torch.tensor(order, dtype=torch.int32, device="cuda").view(1, 1, -1)
    n = torch.full((1, 1), pages, dtype=torch.int32, device="cuda")
    base = attend(cache, q, lists, n).float().abs().max()            # (under the transform, one channel of its own size)
    assert cache.read_status() == 0
    for want, flagged in ((65500.0, False), (65600.0, True), (1e6, True)):
        for b in range(pages):
            cache.subblock(0, b, 0)[at + 512:at + 1024].view(torch.float32).fill_(want / float(base))
        out = attend(cache, q, lists, n)
        assert bool(torch.isinf(out).any()) == flagged
        assert cache.read_status(clear=True) == (kvq.KVQ_DEV_RANGE if flagged else 0)
