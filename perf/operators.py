"""The serving-step operators around the quantized paged cache, as measured calls.

Five operators of one decode / prefill step at long context, in the order a step runs them:

  rope      kvq_norm_rope               per-head RMS norm of queries and keys + position rotation, V split off
  plan      kvq_plan_pages              page tables, slot map and positions from request lengths
  bounds    kvq_page_bounds             per-page, per-channel minimum / maximum of the keys
  select    kvq_select_pages            the pages each (sequence, KV head) attends to, by an upper bound of its scores
  attend    kvq_decode_attention_pages  decode attention over the selected pages of the 2/4-bit cache

`own` False computes the plain form with elementary torch operations (fp32, angles in float64);
`own` True calls the library.  Shapes are those of this repository's workloads (8 KV / 32 query
heads at 8K-32K tokens, 4 KV / 28 query heads at 128K, 256 samples x 16K) and generic ones.
"""
import math

import torch

own = False

D, G = 128, 32                      # head_dim, tokens per page
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one decode step of 32 sequences at ~8K tokens: latency
        dict(name="rope_step_32", op="rope", tokens=32, hq=32, hk=8, rot=128, inter=False, norm=True, dtype="bf16", far=8704),
        # an odd chunk of a prompt, rotation of half the channels in adjacent pairs
        dict(name="rope_chunk_8191", op="rope", tokens=8191, hq=28, hk=4, rot=64, inter=True, norm=True, dtype="fp16", far=131072),
        # the whole prefill of 8 x 32768 tokens
        dict(name="rope_prefill_8x32k", op="rope", tokens=262144, hq=32, hk=8, rot=128, inter=False, norm=True, dtype="bf16", far=32768),
        # one token for each of 256 samples: latency
        dict(name="plan_step_256", op="plan", seqs=256, ctx=16000, new=1),
        # prompts of up to 16384 tokens for 256 samples
        dict(name="plan_prompts_256x16k", op="plan", seqs=256, ctx=0, new=16384),
        # one decode step of 32 sequences
        dict(name="bounds_step_32", op="bounds", seqs=32, hk=8, ctx=8600, new=1, dtype="bf16"),
        # the whole prefill of 8 x 32768 tokens
        dict(name="bounds_prefill_8x32k", op="bounds", seqs=8, hk=8, ctx=0, new=32768, dtype="bf16"),
        # one sequence at 32K, 64 of its 1024 pages: latency
        dict(name="select_1x32k", op="select", seqs=1, hk=8, gq=4, ctx=32768, budget=64, sink=1, recent=4, dtype="bf16"),
        # 256 samples at 16K, 128 of 512 pages
        dict(name="select_256x16k", op="select", seqs=256, hk=8, gq=4, ctx=16384, budget=128, sink=1, recent=4, dtype="bf16"),
        # one sequence at 32K in 4 bits, 64 pages: latency
        dict(name="attend_1x32k_4bit", op="attend", seqs=1, hk=8, gq=4, ctx=32768, budget=64, bits=4, tx=0, patterns=64, dtype="bf16"),
        # four sequences at 128K in 2 bits under the pre-transform, seven query heads a KV head
        dict(name="attend_4x128k_2bit_tx", op="attend", seqs=4, hk=4, gq=7, ctx=131072, budget=256, bits=2, tx=1, patterns=64, dtype="fp16"),
        # 256 samples at 16K in 4 bits, a quarter of the pages
        dict(name="attend_256x16k_4bit", op="attend", seqs=256, hk=8, gq=4, ctx=16384, budget=128, bits=4, tx=0, patterns=64, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "plan", "bounds", "select", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        hk = rng.choice([1, 2, 4, 8])
        hq = hk * rng.choice([1, 3, 4, 7, 8])
        tokens = _log(rng, 1, max(1, 262144 * 48 // (hq + 2 * hk) // 2))
        return dict(op=op, tokens=tokens, hq=hq, hk=hk, rot=rng.choice([32, 64, 96, 128]), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.8, dtype=dtype, far=_log(rng, 64, 1 << 20))
    if op == "plan":
        seqs = _log(rng, 1, 4096)
        return dict(op=op, seqs=seqs, ctx=_log(rng, 64, 32768), new=_log(rng, 1, min(131072, (1 << 22) // seqs)))
    if op == "bounds":
        seqs, hk = _log(rng, 1, 256), rng.choice([1, 2, 4, 8])
        return dict(op=op, seqs=seqs, hk=hk, ctx=_log(rng, 1, 16384) - 1, new=_log(rng, 1, min(32768, (1 << 21) // (seqs * hk))),
                    dtype=dtype)
    hk, gq = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 5, 7, 8, 16])
    if op == "select":
        seqs = _log(rng, 1, 256)
        pages = _log(rng, 64, min(8192, (1 << 20) // (seqs * hk)))
        ctx, budget = pages * G - rng.randint(0, G - 1), _log(rng, 8, min(512, pages // 2))
        sink, recent = rng.randint(0, 1), rng.randint(1, 3)
        return dict(op=op, seqs=seqs, hk=hk, gq=gq, ctx=ctx, budget=budget, sink=sink, recent=recent, dtype=dtype)
    seqs = _log(rng, 1, 128)
    ctx = _log(rng, 1, min(131072, (1 << 23) // (seqs * hk)))
    budget = _log(rng, 1, min(512, max(1, (1 << 17) // (seqs * hk))))
    return dict(op=op, seqs=seqs, hk=hk, gq=gq, ctx=ctx, budget=budget, bits=rng.choice([2, 4, 4]), tx=int(rng.random() < 0.3),
                patterns=_log(rng, 1, 128), dtype=dtype)


def _pages(tokens):
    return (tokens + G - 1) // G


def _sub_bytes(bits, tx):
    return 2 * (G * D * bits // 8) + 2112 + (256 if tx else 0)


def work(case):
    op = case["op"]
    if op == "rope":
        elems = case["tokens"] * (case["hq"] + 2 * case["hk"]) * D
        return {"bytes": 4 * elems + 4 * case["tokens"], "flops": 8 * case["tokens"] * (case["hq"] + case["hk"]) * D}
    if op == "plan":
        tokens = case["seqs"] * (case["new"] if case["new"] == 1 else 0.75 * case["new"])
        return {"bytes": 16 * tokens + 8 * tokens / G + 12 * case["seqs"], "flops": 0}
    if op == "bounds":
        rows = case["seqs"] * case["new"] * case["hk"]
        pages = case["seqs"] * _pages(case["new"]) * case["hk"]
        return {"bytes": rows * 2 * D + pages * 4 * D, "flops": 2 * rows * D}
    groups = case["seqs"] * case["hk"]
    heads = groups * case["gq"]
    if op == "select":
        pages = groups * _pages(case["ctx"])
        return {"bytes": pages * 4 * D + 2 * heads * D + 4 * groups * case["budget"], "flops": 4 * pages * D}
    pages = groups * min(case["budget"], _pages(case["ctx"]))
    return {"bytes": pages * _sub_bytes(case["bits"], case["tx"]) + 4 * heads * D + 2 * case["hk"] * case["patterns"] * 4 * D,
            "flops": 4 * pages * G * case["gq"] * D}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _randint(g, lo, hi, shape, dtype=torch.int32):
    return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)


def _lengths(g, seqs, ctx):
    """Ragged lengths up to ctx; in a batch one sequence still short of a page and one empty."""
    n = ctx - _randint(g, 0, max(1, ctx // 8), (seqs,))
    if seqs >= 4:
        n[1] = min(ctx, 17)
        n[2] = 0
    return n.to(torch.int32)


def _table(g, seqs, maxp):
    return torch.randperm(seqs * maxp, generator=g, device="cuda").to(torch.int32).reshape(seqs, maxp)


def _outliers(g, x):
    """Eight channels fifteen times as large as the rest, as keys have them."""
    x[..., torch.randperm(D, generator=g, device="cuda")[:8]] *= 15.0
    return x


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "rope":
        dt, t, hq, hk = DT[case["dtype"]], case["tokens"], case["hq"], case["hk"]
        s["qkv"] = torch.empty(t, (hq + 2 * hk) * D, dtype=dt, device="cuda")   # the packed projection's output
        s["qkv"].normal_(generator=g)
        s["qw"], s["kw"] = ((1.0 + 0.2 * _randn(g, D)).to(dt) for _ in range(2))
        s["pos"] = _randint(g, 0, case["far"], (t,))
        s["inv"] = 10000.0 ** (-torch.arange(case["rot"] // 2, device="cuda", dtype=torch.float32) / (case["rot"] // 2))
        s["q"] = torch.empty(t, hq, D, dtype=dt, device="cuda")
        s["k"], s["v"] = (torch.empty(t, hk, D, dtype=dt, device="cuda") for _ in range(2))
        if own:
            import bit_kv_cache_26_b200 as kvq

            s["kvq"] = kvq
        return s
    if op == "plan":
        b, ctx, new = case["seqs"], case["ctx"], case["new"]
        s["len"] = ctx - _randint(g, 0, max(1, ctx // 4), (b,)) if ctx else torch.zeros(b, dtype=torch.int32, device="cuda")
        s["new"] = (new - _randint(g, 0, max(1, new // 2), (b,))).to(torch.int32)
        s["maxp"] = _pages(ctx + new)
        pages = torch.randperm(b * s["maxp"], generator=g, device="cuda").to(torch.int32)
        held = (s["len"] + G - 1) // G
        s["table"] = torch.where(torch.arange(s["maxp"], device="cuda") < held[:, None], pages.reshape(b, -1), -1).to(torch.int32)
        s["free"] = pages.reshape(b, -1)[torch.arange(s["maxp"], device="cuda") >= held[:, None]].contiguous()
        s["count"] = torch.tensor([s["free"].numel()], dtype=torch.int32, device="cuda")
        s["left"] = torch.zeros_like(s["count"])
        s["cu"] = torch.zeros(b + 1, dtype=torch.int32, device="cuda")
        s["slots"] = torch.full((b * new,), -1, dtype=torch.int64, device="cuda")
        s["pos"], s["ids"] = (torch.full((b * new,), -1, dtype=torch.int32, device="cuda") for _ in range(2))
        if own:
            s |= _handle(b, 1, s["maxp"], 2, 1, torch.bfloat16, 0, s["table"], s["len"])
            s["ws"] = _workspace(s["kvq"].kvq_plan_workspace_bytes(s["cache"]))
        return s
    dt, b, hk = DT[case["dtype"]], case["seqs"], case["hk"]
    if op == "bounds":
        s["len"] = (case["ctx"] - _randint(g, 0, max(1, case["ctx"] // 8), (b,))).to(torch.int32)
        maxp = _pages(case["ctx"] + case["new"])
        s["table"] = _table(g, b, maxp)
        s["k_new"] = _outliers(g, _randn(g, b, case["new"], hk, D)).to(dt)
        s["bounds"] = _randn(g, b * maxp, hk, 2, D).sort(2).values.to(dt)
        if own:
            s |= _handle(b, hk, maxp, 2, 1, dt, 0, s["table"], s["len"])
        return s
    maxp = _pages(case["ctx"])
    s["len"], s["table"] = _lengths(g, b, case["ctx"]), _table(g, b, maxp)
    s["q"] = _randn(g, b, hk * case["gq"], D).to(dt)
    s["list"] = torch.full((b, hk, case["budget"]), -1, dtype=torch.int32, device="cuda")
    s["n"] = torch.zeros(b, hk, dtype=torch.int32, device="cuda")
    if op == "select":
        mid = _outliers(g, _randn(g, b * maxp, hk, 1, D))
        half = _outliers(g, 0.5 + _rand(g, b * maxp, hk, 1, D))
        s["bounds"] = torch.cat([mid - half, mid + half], 2).to(dt)
        del mid, half
        if own:
            s |= _handle(b, hk, maxp, 2, 1, dt, 0, s["table"], s["len"])
            s["ws"] = _workspace(s["kvq"].kvq_select_workspace_bytes(s["cache"]))
        return s
    # attend: pages of random codes with the scales, zeros and indices of real ones, and the selected pages
    bits, tx, P = case["bits"], case["tx"], case["patterns"]
    sb, cb, levels = _sub_bytes(bits, tx), G * D * bits // 8, (1 << bits) - 1
    pool = _randint(g, 0, 256, (b * maxp, hk, sb), torch.uint8)
    f = pool.view(torch.float32)
    scale = _outliers(g, 0.3 + 0.7 * _rand(g, 1, hk, D)) * 2.0 / levels           # per channel, K
    f[:, :, cb // 4:cb // 4 + D] = (0.5 + _rand(g, b * maxp, hk, D)) * scale
    f[:, :, cb // 4 + D:cb // 4 + 2 * D] = -f[:, :, cb // 4:cb // 4 + D] * (0.5 * levels)
    o = (2 * cb + 1024) // 4
    f[:, :, o:o + D] = (0.3 + 0.7 * _rand(g, b * maxp, hk, D)) * 2.0 / levels      # per token and 32 channels, V
    f[:, :, o + D:o + 2 * D] = -f[:, :, o:o + D].abs().mean() * (0.5 * levels)
    pool[:, :, 2 * cb + 2048:2 * cb + 2080] = _randint(g, 0, P, (b * maxp, hk, 32), torch.uint8)
    vidx = _randint(g, 0, P, (b * maxp, hk, 32), torch.uint8)
    pool[:, :, 2 * cb + 2080:2 * cb + 2112] = torch.where(_rand(g, b * maxp, hk, 32) < 0.05, 255, vidx).to(torch.uint8)
    if tx:
        f[:, :, (2 * cb + 2112) // 4:] = 0.5 + _rand(g, b * maxp, hk, 64)
    s["pool"] = pool
    s["kp"], s["vp"] = _outliers(g, _randn(g, 1, hk, P, D)), _randn(g, 1, hk, P, D)
    s["tail"] = _outliers(g, _randn(g, b, hk, G, D)).to(dt)
    s["kc"], s["vc"] = ((5.0 + 10.0 * _rand(g, 1, hk, D)) if tx else None for _ in range(2))
    s["out"] = torch.empty(b, hk * case["gq"], D, dtype=dt, device="cuda")
    # the newest page and a random choice of the others, in ascending order
    n = ((s["len"] + G - 1) // G).reshape(b, 1, 1)
    rank = _rand(g, b, hk, maxp)
    at = torch.arange(maxp, device="cuda")
    rank = torch.where(at == n - 1, 2.0, torch.where(at < n, rank, -1.0))
    take = min(case["budget"], maxp)
    best, idx = rank.topk(take, -1)
    idx = torch.where(best >= 0, idx, maxp).sort(-1).values
    s["list"][:, :, :take] = torch.where(idx < maxp, idx, -1).to(torch.int32)
    s["n"][:] = n[:, :, 0].clamp(max=case["budget"])
    # where each element's code sits in a page's words
    s["kat"], s["vat"] = _places(bits, G, D), _places(bits, D, G)
    s["chan"], s["vs_at"], s["vz_at"], s["tok"] = _orders()
    if own:
        s |= _handle(b, hk, maxp, bits, P, dt, tx, s["table"], s["len"], s)
        s["ws"] = _workspace(s["kvq"].kvq_decode_pages_workspace_bytes(s["cache"], hk * case["gq"], case["budget"]))
    return s


def _handle(b, hk, maxp, bits, P, dt, tx, table, length, s=None):
    """The cache struct over the state's own tensors (a user's program keeps it beside them)."""
    import bit_kv_cache_26_b200 as kvq

    c = kvq.kvq_cache()
    c.num_seqs, c.num_kv_heads, c.head_dim, c.group, c.bits = b, hk, D, G, bits
    c.num_patterns, c.num_sets, c.max_pages_per_seq, c.num_pages = P, 1, maxp, b * maxp
    c.dtype, c.transform = kvq.KVQ_BF16 if dt == torch.bfloat16 else kvq.KVQ_F16, tx
    # operators that only look at lengths and tables are given a cache whose other buffers stay untouched
    s = s or {k: torch.empty(256, dtype=torch.float32, device="cuda") for k in ("pool", "tail", "kp", "vp")}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.page_pool, c.page_table, c.seq_len = s["pool"].data_ptr(), table.data_ptr(), length.data_ptr()
    c.k_tail, c.k_patterns, c.v_patterns, c.status = s["tail"].data_ptr(), s["kp"].data_ptr(), s["vp"].data_ptr(), status.data_ptr()
    c.k_colscale = s["kc"].data_ptr() if tx else None
    c.v_colscale = s["vc"].data_ptr() if tx else None
    return dict(kvq=kvq, cache=c, keep=(None if "case" in s else s, status))


def _workspace(nbytes):
    return torch.zeros(max(256, nbytes), dtype=torch.uint8, device="cuda")


def _places(bits, rows, cols):
    """(word, bit) of element (row, col) of a code block, in the fragment order of the page layout."""
    r, c = torch.arange(rows, device="cuda")[:, None], torch.arange(cols, device="cuda")[None]
    lane = (r % 8) * 4 + (c % 8) // 2
    reg = ((r // 16) * (cols // 16) + c // 16) * 4 + (r % 16) // 8 + 2 * ((c % 16) // 8)
    per = 16 // bits
    w, bit = reg // per, bits * (reg % per) + 16 * (c % 2)
    return (w // 4) * 128 + lane * 4 + w % 4, bit.to(torch.int32)


def _orders():
    """Positions of a channel (K scales), of (token, channel) for V scales and zeros, and of a token."""
    c, t = torch.arange(D, device="cuda"), torch.arange(G, device="cuda")
    e = lambda x: x % 2 + 2 * ((x % 16) // 8)   # noqa: E731
    chan = (c // 16) * 16 + ((c % 8) // 2) * 4 + e(c)
    grp = (c // 32)[None]
    vs = (((t // 16) * 4 + e(t)) * 4 + (t % 8) // 2)[:, None] * 4 + grp
    return chan, vs, t[:, None] * 4 + grp, (t % 8) * 4 + t // 8


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    return {"rope": _rope, "plan": _plan, "bounds": _bounds, "select": _select, "attend": _attend}[s["case"]["op"]](s)


def _split(s):
    c = s["case"]
    t = s["qkv"].view(c["tokens"], c["hq"] + 2 * c["hk"], D)
    return t[:, :c["hq"]], t[:, c["hq"]:c["hq"] + c["hk"]], t[:, c["hq"] + c["hk"]:]


def _rope(s):
    c = s["case"]
    q, k, v = _split(s)
    qw, kw = (s["qw"], s["kw"]) if c["norm"] else (None, None)
    if own:
        s["kvq"].kvq_norm_rope(q, k, v, s["pos"], s["inv"], s["q"], s["k"], s["v"], q_weight=qw, k_weight=kw, eps=1e-6,
                               interleaved=c["inter"])
        return s["q"], s["k"], s["v"]
    angle = s["pos"].double()[:, None] * s["inv"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return _turn(q, qw, cos, sin, c), _turn(k, kw, cos, sin, c), v.contiguous()


def _turn(x, w, cos, sin, c):
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    rot = c["rot"]
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if c["inter"] else (y[..., :rot // 2], y[..., rot // 2:rot])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([u, v], -1).flatten(-2) if c["inter"] else torch.cat([u, v], -1)
    return torch.cat([turned, y[..., rot:]], -1).to(x.dtype)


def _plan(s):
    outs = dict(table=s["table"], cu=s["cu"], slots=s["slots"], pos=s["pos"], ids=s["ids"], left=s["left"])
    if own:
        s["kvq"].kvq_plan_pages(s["cache"], s["new"], s["free"], s["count"], s["left"], s["cu"], s["slots"], s["pos"], s["ids"],
                                s["ws"])
        return outs
    b, maxp, most = s["len"].numel(), s["maxp"], s["slots"].numel()
    have, new = s["len"].long(), s["new"].long()
    new = torch.where((new >= 0) & (have >= 0) & (have + new <= maxp * G), new, 0)
    held = (have + G - 1) // G
    need = (have + new + G - 1) // G - held
    upto, taken = new.cumsum(0), need.cumsum(0)
    served = (upto <= most) & (taken <= s["count"])
    total = torch.where(served, upto, 0).max()
    cu = torch.cat([total.new_zeros(1), torch.where(served, upto, total)])
    at = torch.arange(most, device="cuda")
    real = at < total
    ids = torch.searchsorted(cu[1:], at, right=True).clamp(max=b - 1)
    pos = have[ids] + at - cu[ids]
    page = torch.where(real, pos // G, 0)
    fresh = page - held[ids]
    top = (s["count"] - 1 - (taken - need)[ids] - fresh).clamp(0, s["free"].numel() - 1)
    phys = torch.where(fresh >= 0, s["free"][top], s["table"][ids, page]).long()
    to = torch.where(real & (pos % G == 0), ids * maxp + page, b * maxp)
    table = torch.cat([s["table"].flatten(), s["table"].new_zeros(1)])
    table[to] = phys.to(torch.int32)
    return dict(table=table[:-1].view(b, maxp), cu=cu.to(torch.int32), slots=torch.where(real, phys * G + pos % G, s["slots"]),
                pos=torch.where(real, pos.to(torch.int32), s["pos"]), ids=torch.where(real, ids.to(torch.int32), s["ids"]),
                left=(s["count"] - torch.where(served, taken, 0).max()).to(torch.int32))


def _bounds(s):
    c = s["case"]
    if own:
        s["kvq"].kvq_page_bounds(s["cache"], s["k_new"], c["new"], s["bounds"])
        return s["bounds"]
    b, maxp = s["table"].shape
    # the new tokens laid out from their page's first slot on; the places of others hold neutral values
    first = (s["len"] % G).long()
    room = _pages(c["new"] + G - 1)
    t = torch.arange(room * G, device="cuda") - first[:, None]
    real = (t >= 0) & (t < c["new"])
    rows = s["k_new"].float()[torch.arange(b, device="cuda")[:, None], t.clamp(0, c["new"] - 1)]
    rows = rows.view(b, room, G, c["hk"], D)
    real = real.view(b, room, G, 1, 1)
    lo = torch.where(real, rows, math.inf).amin(2)
    hi = torch.where(real, rows, -math.inf).amax(2)
    page = (s["len"] // G).long()[:, None] + torch.arange(room, device="cuda")
    touched = real.any(2)[..., 0, 0]
    phys = s["table"][torch.arange(b, device="cuda")[:, None], page.clamp(max=maxp - 1)].long()
    old = s["bounds"][phys].float()
    goes_on = ((page == (s["len"] // G)[:, None]) & (first > 0)[:, None])[..., None, None]
    lo = torch.where(goes_on, torch.minimum(lo, old[..., 0, :]), lo)
    hi = torch.where(goes_on, torch.maximum(hi, old[..., 1, :]), hi)
    s["bounds"][phys[touched]] = torch.stack([lo, hi], 3)[touched].to(s["bounds"].dtype)
    return s["bounds"]


def _fold(x):
    """fp32 sum over the last axis (a power of two) by halving: the upper half onto the lower, until one is left."""
    n = x.shape[-1] // 2
    return x[..., 0] if n == 0 else _fold(x[..., :n] + x[..., n:])


def _select(s):
    c = s["case"]
    if own:
        s["kvq"].kvq_select_pages(s["cache"], s["q"], c["hk"] * c["gq"], s["bounds"], c["budget"], c["sink"], c["recent"], s["list"],
                                  s["n"], s["ws"])
        return s["list"], s["n"]
    b, maxp = s["table"].shape
    q = torch.nn.functional.pad(s["q"].float().view(b, c["hk"], c["gq"], D), (0, 0, 0, 16 - c["gq"])).transpose(2, 3)
    up, down = _fold(q.clamp(min=0)), _fold(q.clamp(max=0))                       # [b, hk, D]
    lo_hi = s["bounds"][s["table"].long()].permute(0, 2, 1, 3, 4).float()          # [b, hk, pages, 2, D]
    terms = up[:, :, None] * lo_hi[..., 1, :] + down[:, :, None] * lo_hi[..., 0, :]
    score = _fold(_fold(terms.unflatten(-1, (16, 8))))                             # 8 neighbours first, then the 16 sums
    at = torch.arange(maxp, device="cuda")
    n = ((s["len"] + G - 1) // G).view(b, 1, 1)
    first = torch.where((at < c["sink"]) | (at >= n - c["recent"]), 0, 1) + 2 * (at >= n)   # forced, scored, absent
    order = score.sort(dim=-1, descending=True, stable=True).indices
    order = order.gather(-1, first.expand_as(order).gather(-1, order).sort(dim=-1, stable=True).indices)
    take = n.clamp(max=c["budget"])
    most = min(c["budget"], maxp)
    idx = torch.where(torch.arange(most, device="cuda") < take, order[..., :most], maxp).sort(-1).values
    picked = torch.where(idx < maxp, idx, -1).to(torch.int32)
    picked = torch.nn.functional.pad(picked, (0, c["budget"] - most), value=-1)
    return picked, take[:, :, 0].expand(b, c["hk"]).to(torch.int32).contiguous()


def _hadamard(dtype):
    i = torch.arange(D, device="cuda")
    bits = (i[:, None] & i[None])[..., None] >> torch.arange(7, device="cuda") & 1
    return (1 - 2 * (bits.sum(-1) % 2)).to(dtype)


def _attend(s):
    c = s["case"]
    scale = D ** -0.5
    if own:
        s["kvq"].kvq_decode_attention_pages(s["cache"], s["q"], c["hk"] * c["gq"], scale, s["list"], s["n"], s["out"], s["ws"])
        return s["out"]
    b, hk, gq, cb, k_n = c["seqs"], c["hk"], c["gq"], G * D * c["bits"] // 8, c["budget"]
    page = s["list"].long().clamp(min=0)
    at_b, at_h = torch.arange(b, device="cuda").view(b, 1, 1), torch.arange(hk, device="cuda").view(1, hk, 1)
    sub = s["pool"][s["table"][at_b, page].long(), at_h]                           # [b, hk, pages, bytes]
    f, words = sub.view(torch.float32), sub.view(torch.int32)
    mask = (1 << c["bits"]) - 1
    k = ((words[..., s["kat"][0]] >> s["kat"][1]) & mask).float()
    k = k * f[..., cb // 4 + s["chan"]][..., None, :] + f[..., cb // 4 + D + s["chan"]][..., None, :]
    kidx = sub[..., 2 * cb + 2048 + s["tok"]].long()
    k = k + s["kp"][0][at_h[..., None], kidx]
    v = ((words[..., cb // 4 + 256 + s["vat"][0]] >> s["vat"][1]) & mask).float().transpose(-1, -2)
    o = (2 * cb + 1024) // 4
    v = v * f[..., o + s["vs_at"]] + f[..., o + D + s["vz_at"]]
    vidx = sub[..., 2 * cb + 2080 + s["tok"]].long()
    v = v + torch.where((vidx < 255)[..., None], s["vp"][0][at_h[..., None], vidx.clamp(max=c["patterns"] - 1)], 0.0)
    if c["tx"]:
        H = _hadamard(torch.float32)
        o = (2 * cb + 2112) // 4
        k = f[..., o + s["tok"]][..., None] * ((k * s["kc"][0][:, None, None]) @ H) / D
        v = f[..., o + 32 + s["tok"]][..., None] * ((v * s["vc"][0][:, None, None]) @ H) / D
    length = s["len"].view(b, 1, 1).long()
    newest = (page == length // G)[..., None, None]
    k = torch.where(newest, s["tail"].float()[:, :, None], k).view(b, hk, k_n * G, D)
    v = v.reshape(b, hk, k_n * G, D)
    listed_ = torch.arange(k_n, device="cuda") < s["n"][..., None]
    real = (listed_[..., None] & (page[..., None] * G + torch.arange(G, device="cuda") < length[..., None])).view(b, hk, 1, k_n * G)
    score = (s["q"].float().view(b, hk, gq, D) @ k.transpose(-1, -2)) * scale
    score = torch.where(real, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.where(real, torch.exp(score - torch.where(top > -math.inf, top, 0.0)), 0.0)
    total = p.sum(-1, keepdim=True)
    out = (p @ torch.where(real.transpose(-1, -2), v, 0.0)) / torch.where(total > 0, total, 1.0)
    return out.view(b, hk * gq, D).to(s["q"].dtype)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op in ("plan", "select"):
        return None          # whole numbers only
    s = prepare(case, seed)
    if op == "rope":
        q, k, v = _split(s)
        weights = (s["qw"], s["kw"]) if case["norm"] else (None, None)
        return (*(_exact_turn(x, w, s, case) for x, w in zip((q, k), weights)), v.double())
    if op == "bounds":
        got = s["bounds"].double()
        b, n = case["seqs"], case["new"]
        pos = s["len"].long()[:, None] + torch.arange(n, device="cuda")
        page = s["table"].long().gather(1, pos // G)
        opened = page[pos % G == 0]
        got[opened, :, 0], got[opened, :, 1] = math.inf, -math.inf
        for h in range(case["hk"]):
            rows = s["k_new"][:, :, h].double().reshape(b * n, D)
            at = page.reshape(-1, 1).expand(-1, D)
            got[:, h, 0] = got[:, h, 0].scatter_reduce(0, at, rows, "amin")
            got[:, h, 1] = got[:, h, 1].scatter_reduce(0, at, rows, "amax")
        return got
    return _exact_attend(s, case)


def _exact_turn(x, w, s, case):
    rot = case["rot"]
    i = torch.arange(rot // 2, device="cuda")
    left, right = (2 * i, 2 * i + 1) if case["inter"] else (i, i + rot // 2)
    out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
    for t in range(0, x.shape[0], 16384):
        y = x[t:t + 16384].double()
        if w is not None:
            y = y / ((y * y).sum(-1, keepdim=True) / D + 1e-6).sqrt() * w.double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["pos"][t:t + 16384, None, None].double() * s["inv"].double())
        z = torch.complex(y[..., left], y[..., right]) * turn
        y[..., left], y[..., right] = z.real, z.imag
        out[t:t + 16384] = y
    return out


def _exact_attend(s, case):
    b, hk, gq, bits, P = case["seqs"], case["hk"], case["gq"], case["bits"], case["patterns"]
    cb, per = G * D * bits // 8, 16 // bits
    # the elements of a block in the order of its words, slots and halves: (row, col) by the layout read backwards
    def block(words, rows, cols):
        w = torch.arange(cb // 4, device="cuda")[:, None, None]
        slot, odd = torch.arange(per, device="cuda")[None, :, None], torch.arange(2, device="cuda")[None, None]
        lane, reg = (w % 128) // 4, ((w // 128) * 4 + w % 4) * per + slot
        ks, r = cols // 16, reg % 4
        row = 16 * (reg // 4 // ks) + 8 * (r % 2) + lane // 4
        col = 16 * (reg // 4 % ks) + 8 * (r // 2) + 2 * (lane % 4) + odd
        code = (words[:, :, None, None].long() >> (bits * slot + 16 * odd)) & ((1 << bits) - 1)
        out = torch.empty(words.shape[0], rows * cols, dtype=torch.float64, device="cuda")
        out[:, (row * cols + col).flatten()] = code.flatten(1).double()
        return out.view(-1, rows, cols)

    def unorder(x, order):            # x[:, i] belongs to element order[i]
        out = torch.empty_like(x)
        out[:, order] = x
        return out

    i = torch.arange(D, device="cuda")
    inner = lambda j: 2 * (j // 4 % 4) + j % 2 + 8 * (j // 2 % 2)   # noqa: E731
    ksc = 16 * (i // 16) + inner(i)
    vsc_tok = 16 * (i // 64) + 2 * (i // 4 % 4) + (i // 16) % 2 + 8 * (i // 32 % 2)
    tok = torch.arange(G, device="cuda")
    tok = tok // 4 + 8 * (tok % 4)
    H = _hadamard(torch.float64)
    out = torch.zeros(b, hk * gq, D, dtype=torch.float64, device="cuda")
    lengths, counts = s["len"].tolist(), s["n"].tolist()
    for x in range(b):
        for h in range(hk):
            n, L = counts[x][h], lengths[x]
            if n == 0 or L == 0:
                continue
            pages = s["list"][x, h, :n].long()
            sub = s["pool"][s["table"][x][pages].long(), h]
            f, words = sub.view(torch.float32).double(), sub.view(torch.int32)
            k = block(words[:, :cb // 4], G, D) * unorder(f[:, cb // 4:cb // 4 + D], ksc)[:, None]
            k = k + unorder(f[:, cb // 4 + D:cb // 4 + 2 * D], ksc)[:, None]
            k = k + s["kp"][0, h].double()[unorder(sub[:, 2 * cb + 2048:2 * cb + 2080], tok).long()]
            v = block(words[:, cb // 4 + 256:cb // 2 + 256], D, G).transpose(1, 2)
            o = (2 * cb + 1024) // 4
            vs = unorder(f[:, o:o + D], vsc_tok * 4 + i % 4).view(-1, G, 4)
            vz = f[:, o + D:o + 2 * D].view(-1, G, 4)
            v = v * vs.repeat_interleave(32, 2) + vz.repeat_interleave(32, 2)
            vidx = unorder(sub[:, 2 * cb + 2080:2 * cb + 2112], tok).long()
            v[vidx < 255] += s["vp"][0, h].double()[vidx[vidx < 255]]
            if case["tx"]:
                o = (2 * cb + 2112) // 4
                k = unorder(f[:, o:o + 32], tok)[..., None] * ((k * s["kc"][0, h].double()) @ H) / D
                v = unorder(f[:, o + 32:o + 64], tok)[..., None] * ((v * s["vc"][0, h].double()) @ H) / D
            if L % G:
                k[pages == L // G] = s["tail"][x, h].double()
            real = (pages[:, None] * G + torch.arange(G, device="cuda") < L).flatten()
            k, v = k.view(-1, D)[real], v.reshape(-1, D)[real]
            q = s["q"][x, h * gq:(h + 1) * gq].double()
            out[x, h * gq:(h + 1) * gq] = torch.softmax(q @ k.T * D ** -0.5, -1) @ v
    return out
