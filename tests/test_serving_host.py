"""Refusals of the serving-step entry points (kvq_norm_rope, kvq_plan_pages, kvq_page_bounds, kvq_select_pages,
kvq_decode_attention_pages): every bad argument is answered on the host, before anything is enqueued (no GPU needed)."""
import ctypes

import pytest
import torch

import bit_kv_cache_26_b200 as kvq

L = kvq._lib
INVALID, UNSUPPORTED, CAPACITY, WORKSPACE = (kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_CAPACITY,
                                             kvq.KVQ_ERR_WORKSPACE)
V = ctypes.c_void_p
BIG = 1 << 30


def cache(**kw):
    c = kvq.kvq_cache()
    c.num_seqs, c.num_kv_heads, c.head_dim, c.group, c.bits, c.num_patterns = 2, 2, 128, 32, 2, 16
    c.num_sets, c.max_pages_per_seq, c.num_pages, c.dtype = 1, 4, 8, 1
    c.page_pool = 256
    for f in ("page_table", "seq_len", "k_tail", "k_patterns", "v_patterns", "status"):
        setattr(c, f, 256)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def rows(heads=2, **kw):
    r = kvq.kvq_rows()
    r.in_, r.out, r.heads = 256, 256, heads
    r.in_tok_stride, r.in_head_stride, r.out_tok_stride, r.out_head_stride = 256, 128, 256, 128
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def rope(q=None, k=None, v=None, dtype=1, tokens=4, pos=256, inv=256, rot=128, eps=1e-6):
    ref = lambda r: ctypes.byref(r) if r is not None else None   # noqa: E731
    return L.kvq_norm_rope(ref(q), ref(k), ref(v), dtype, tokens, V(pos), V(inv), rot, 0, eps, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(rot=8), UNSUPPORTED), (dict(rot=144), UNSUPPORTED), (dict(rot=-16), UNSUPPORTED),
    (dict(tokens=-1), INVALID), (dict(tokens=1 << 31), CAPACITY), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(pos=None), INVALID), (dict(inv=None), INVALID),
    (dict(q=rows(in_=None)), INVALID), (dict(q=rows(out=None)), INVALID), (dict(q=rows(in_=8)), INVALID),
    (dict(q=rows(out=260)), INVALID), (dict(q=rows(weight=8)), INVALID), (dict(q=rows(heads=-1)), INVALID),
    (dict(q=rows(in_tok_stride=132)), INVALID), (dict(q=rows(out_head_stride=4)), INVALID),
    (dict(q=rows(in_head_stride=-128)), INVALID), (dict(q=rows(reserved=1)), INVALID), (dict(q=rows(heads=65536)), CAPACITY),
    (dict(v=rows(weight=256)), INVALID), (dict(q=rows(out_head_stride=0)), INVALID), (dict(q=rows(out_tok_stride=64)), INVALID),
])
def test_norm_rope_refuses(kw, status):
    assert rope(**{"q": rows(), **kw}) == status
    assert kvq.kvq_last_error()


def test_norm_rope_with_nothing_to_do():
    assert rope() == 0 and rope(q=rows(heads=0)) == 0 and rope(q=rows(in_=None), tokens=0) == 0


def plan(c=None, new_len=256, free=256, cap=8, count=256, left=256, cu=256, slots=256, pos=256, ids=256, most=64, ws=256, n=BIG):
    return L.kvq_plan_pages(ctypes.byref(c or cache()), V(new_len), V(free), cap, V(count), V(left), V(cu), V(slots), V(pos), V(ids),
                            most, V(ws), n, None)


@pytest.mark.parametrize("kw,status", [
    (dict(new_len=None), INVALID), (dict(free=None), INVALID), (dict(count=None), INVALID), (dict(left=None), INVALID),
    (dict(cu=None), INVALID), (dict(slots=None), INVALID), (dict(pos=None), INVALID), (dict(ids=None), INVALID),
    (dict(slots=264), INVALID), (dict(pos=260), INVALID), (dict(ids=260), INVALID), (dict(cap=-1), INVALID), (dict(most=-1), INVALID),
    (dict(most=(1 << 31) - 1), CAPACITY), (dict(ws=None), WORKSPACE), (dict(n=16), WORKSPACE), (dict(ws=258), INVALID),
    (dict(c=cache(page_table=None)), INVALID), (dict(c=cache(num_seqs=65536)), CAPACITY),
])
def test_plan_refuses(kw, status):
    assert plan(**kw) == status


def bounds(c=None, k=256, n=4, out=256):
    return L.kvq_page_bounds(ctypes.byref(c or cache()), V(k), n, V(out), None)


@pytest.mark.parametrize("kw,status", [
    (dict(k=None), INVALID), (dict(out=None), INVALID), (dict(k=264), INVALID), (dict(out=264), INVALID), (dict(n=-1), INVALID),
    (dict(n=129), CAPACITY), (dict(c=cache(dtype=3)), UNSUPPORTED),
])
def test_bounds_refuses(kw, status):
    assert bounds(**kw) == status


def select(c=None, q=256, hq=4, bnd=256, budget=8, sink=1, recent=2, lst=256, n=256, ws=256, wsn=BIG):
    return L.kvq_select_pages(ctypes.byref(c or cache()), V(q), hq, V(bnd), budget, sink, recent, V(lst), V(n), V(ws), wsn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(bnd=None), INVALID), (dict(lst=None), INVALID), (dict(n=None), INVALID), (dict(q=264), INVALID),
    (dict(bnd=264), INVALID), (dict(hq=3), UNSUPPORTED), (dict(hq=0), UNSUPPORTED), (dict(hq=34), UNSUPPORTED),
    (dict(budget=0), INVALID), (dict(budget=2), INVALID), (dict(sink=-1), INVALID), (dict(recent=0), INVALID),
    (dict(budget=2**31 - 1, sink=2**31 - 1, recent=2**31 - 1), INVALID), (dict(ws=None), WORKSPACE), (dict(wsn=8), WORKSPACE),
    (dict(ws=128), INVALID),
])
def test_select_refuses(kw, status):
    assert select(**kw) == status


def attend(c=None, q=256, hq=4, scale=0.1, lst=256, n=256, budget=8, out=256, ws=256, wsn=BIG):
    return L.kvq_decode_attention_pages(ctypes.byref(c or cache()), V(q), hq, scale, V(lst), V(n), budget, V(out), V(ws), wsn, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(lst=None), INVALID), (dict(n=None), INVALID), (dict(q=264), INVALID),
    (dict(out=264), INVALID), (dict(hq=3), UNSUPPORTED), (dict(hq=34), UNSUPPORTED), (dict(budget=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wsn=8), WORKSPACE), (dict(ws=128), INVALID), (dict(c=cache(bits=3)), UNSUPPORTED),
])
def test_attend_refuses(kw, status):
    assert attend(**kw) == status


def test_a_cache_without_sequences_is_no_work():
    c = cache(num_seqs=0)
    assert plan(c) == 0 and bounds(c) == 0 and select(c) == 0 and attend(c) == 0 and bounds(n=0) == 0


def test_workspace_sizes():
    c = cache()
    assert kvq.kvq_plan_workspace_bytes(c) == (2 + 4) * 4
    assert kvq.kvq_select_workspace_bytes(c) == 256 + 2 * 2 * 4 * 4
    small, large = (kvq.kvq_decode_pages_workspace_bytes(c, 4, n) for n in (1, 1024))
    assert 256 < small <= large
    assert kvq.kvq_decode_pages_workspace_bytes(c, 4, 0) == 0 and kvq.kvq_decode_pages_workspace_bytes(c, 0, 4) == 0


def test_the_binding_refuses_tensors_it_cannot_pass_on():
    # tensors in host memory, of another type or shape: refused before the library is called
    q = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    for bad in (q, q.float()):
        with pytest.raises(kvq.KvqError):
            kvq.kvq_norm_rope(bad, None, None, None, None, bad, None, None)
    with pytest.raises(kvq.KvqError):
        kvq.kvq_page_bounds(cache(), torch.zeros(2, 4, 2, 128), 4, torch.zeros(8, 2, 2, 128))
    kvq.kvq_norm_rope(None, None, None, None, None, None, None, None)   # nothing given, nothing done
