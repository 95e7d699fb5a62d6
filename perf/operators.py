"""The paged-cache operators, measured: planning a step on the GPU, appending
its keys and values, and the attention of its new tokens over the pages.

Shapes are the gpt-oss attention shapes of this repository (64 query heads, 8
key/value heads, head dim 64) and the smaller head counts of its tests.  A
case fixes every length, so that its work can be counted; the seed draws the
values and which page of the pool holds what.
"""
import math

import torch

own = False

D = 64
E4M3 = torch.float8_e4m3fn


def listed():
    return [
        # One token for each of 256 requests: the planning call before every decode step.
        dict(name="plan_decode_256", op="plan", batch=256, new_hi=1, chunked=0, finished=0, kv_lo=100, kv_hi=8192,
             page=64, window=0, spare=64),
        # A step that mixes prompt chunks, single tokens, idle and finished requests, for a
        # sliding-window layer group whose old pages go back to the pool.
        dict(name="plan_mixed_window", op="plan", batch=61, new_hi=2048, chunked=3, finished=9, kv_lo=0, kv_hi=6000,
             page=16, window=128, spare=16500),
        # One decode step's keys and values, cut out of a fused projection.
        dict(name="append_decode_64", op="append", tokens=64, pad=0, hq=64, hkv=8, page=64, e4m3=False),
        # A prompt of 16384 tokens, as in the 4 x 4096 prefill workload.
        dict(name="append_prefill_16k", op="append", tokens=16384, pad=0, hq=64, hkv=8, page=64, e4m3=False),
        # The same for an e4m3 cache: odd count, padding rows behind the last token.
        dict(name="append_e4m3_8191", op="append", tokens=8191, pad=65, hq=64, hkv=8, page=16, e4m3=True),
        # The smallest step: one request, one token.
        dict(name="attn_one_request", op="attn", batch=1, new_hi=1, chunked=0, kv_lo=4033, kv_hi=4033, hq=64, hkv=8,
             page=64, window=0, e4m3=False),
        # The decode step of the benchmark's decode key, at ragged lengths.
        dict(name="attn_decode_64x8k", op="attn", batch=64, new_hi=1, chunked=0, kv_lo=6000, kv_hi=8192, hq=64, hkv=8,
             page=64, window=0, e4m3=False),
        # The same over an e4m3 cache with short pages.
        dict(name="attn_decode_64x8k_e4m3", op="attn", batch=64, new_hi=1, chunked=0, kv_lo=6000, kv_hi=8192, hq=64,
             hkv=8, page=16, window=0, e4m3=True),
        # A decode step of a sliding-window layer: short key ranges, many requests.
        dict(name="attn_decode_w128", op="attn", batch=128, new_hi=1, chunked=0, kv_lo=50, kv_hi=8192, hq=64, hkv=8,
             page=16, window=128, e4m3=False),
        # A chunk of a long prompt: 2048 new tokens over 30720 cached ones, full causal.
        dict(name="attn_chunk_2k_of_32k", op="attn", batch=1, new_hi=2048, chunked=1, kv_lo=32768, kv_hi=32768, hq=64,
             hkv=8, page=64, window=0, e4m3=False),
        # Four chunks on a sliding-window layer.
        dict(name="attn_chunk_w128", op="attn", batch=4, new_hi=2048, chunked=1, kv_lo=3500, kv_hi=8000, hq=64, hkv=8,
             page=32, window=128, e4m3=False),
        # Chunks and single tokens together over an e4m3 cache, five query heads a group.
        dict(name="attn_mixed_e4m3", op="attn", batch=33, new_hi=700, chunked=8, kv_lo=700, kv_hi=4096, hq=40, hkv=8,
             page=16, window=0, e4m3=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attn", "attn"])
    page = rng.choice([16, 32, 64, 128])
    if op == "plan":
        window = rng.choice([0, 0, 100, 128, 1000])
        chunked = rng.choice([0, 1, 3, 8])
        batch = _log(rng, 1, 300)
        return dict(op="plan", batch=batch, new_hi=_log(rng, 2, 1500) if chunked else 1, chunked=chunked,
                    finished=rng.choice([0, 5, 11]), kv_lo=rng.randint(0, 60), kv_hi=_log(rng, 64, 8000), page=page,
                    window=window, spare=rng.choice([3, 40, 20000]))
    hq, hkv = rng.choice([(64, 8), (64, 8), (16, 2), (8, 8), (4, 1), (40, 8), (24, 8), (32, 2)])
    if op == "append":
        return dict(op="append", tokens=_log(rng, 1, 16000), pad=rng.choice([0, 0, 7, 300]), hq=hq, hkv=hkv, page=page,
                    e4m3=rng.random() < 0.5)
    window = rng.choice([0, 0, 0, 100, 128, 1000])
    chunked = rng.choice([0, 0, 1, 5])
    # Larger batches go with shorter lengths, so that no drawn case costs more than the largest listed one.
    batch = _log(rng, 1, 160)
    kv_hi = _log(rng, 64, max(128, min(24000, 400000 // batch)))
    if chunked == 1:
        batch, kv_hi = min(batch, 6), min(kv_hi, 14000)
    new_hi = min(_log(rng, 2, 1500), kv_hi) if chunked else rng.choice([1, 1, 1, 2, 4])
    return dict(op="attn", batch=batch, new_hi=new_hi, chunked=chunked, kv_lo=min(kv_hi, max(new_hi, kv_hi // 3)),
                kv_hi=kv_hi, hq=hq, hkv=hkv, page=page, window=window, e4m3=rng.random() < 0.4)


def _spread(lo, hi, b, salt):
    """The b-th of a set of lengths spread over [lo, hi]."""
    return lo + int((hi - lo + 1) * ((b * 0.6180339887 + salt) % 1.0)) if hi > lo else lo


def _lens(case):
    """(tokens in the cache after the step, new tokens) of every request of an attention case."""
    kv = [_spread(case["kv_lo"], case["kv_hi"], b, 0.37) for b in range(case["batch"])]
    every = case["chunked"]
    if every == 0:  # decode: the same few tokens for every request
        new = [min(case["new_hi"], k) for k in kv]
    elif every == 1:  # chunks only; the first one has the full length
        new = [min(k, case["new_hi"] if b == 0 else _spread(max(1, case["new_hi"] // 2), case["new_hi"], b, 0.11))
               for b, k in enumerate(kv)]
    else:  # a chunk every so many requests, single tokens between them
        new = [min(k, _spread(max(1, case["new_hi"] // 4), case["new_hi"], b, 0.2) if b % every == 0 else 1)
               for b, k in enumerate(kv)]
    return kv, new


def _plan_lens(case):
    """(cached tokens, new tokens or -1 for a finished request) of every request of a planning case."""
    cached = [_spread(case["kv_lo"], case["kv_hi"], b, 0.37) for b in range(case["batch"])]
    new = []
    for b in range(case["batch"]):
        if case["finished"] and b % case["finished"] == case["finished"] - 1:
            new.append(-1)
        elif case["chunked"] and b % case["chunked"] == 0:
            new.append(_spread(0, case["new_hi"], b, 0.2))
        else:
            new.append(1)
    return cached, new


def _max_pages(case):
    return -(-(case["kv_hi"] + case["new_hi"]) // case["page"]) + 1


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = dict(device="cuda")
    page = case["page"]
    if case["op"] == "plan":
        cached, new = _plan_lens(case)
        first = [max(0, c - 40 - case["window"]) // page if case["window"] else 0 for c in cached]
        held = [(b, j) for b, c in enumerate(cached) for j in range(first[b], -(-c // page))]
        pages = len(held) + case["spare"]
        ids = torch.randperm(pages, generator=gen, **dev).int()
        table = torch.full((case["batch"], _max_pages(case)), -1, dtype=torch.int32, **dev)
        if held:
            at = torch.tensor(held, **dev)
            table[at[:, 0], at[:, 1]] = ids[: len(held)]
        head = int(torch.randint(0, pages, (1,), generator=gen, **dev))
        ring = torch.full((pages,), -1, dtype=torch.int32, **dev)
        ring[(head + torch.arange(case["spare"], **dev)) % pages] = ids[len(held):]
        as_int = lambda v: torch.tensor(v, dtype=torch.int32, **dev)  # noqa: E731
        return dict(case=case, cached=as_int(cached), new=as_int(new), table=table, ring=ring,
                    pool=as_int([head, case["spare"]]), first=as_int(first), tokens=sum(max(0, n) for n in new) + 5)
    hq, hkv = case["hq"], case["hkv"]
    kind = E4M3 if case["e4m3"] else torch.bfloat16
    scales = (torch.rand((2, hkv), generator=gen, **dev) * 0.004 + 0.008) if case["e4m3"] else None

    def values(*shape):
        return torch.randn(shape, generator=gen, dtype=torch.bfloat16, **dev)

    def cache(pages):
        c = torch.empty((2, pages, page, hkv, D), dtype=kind, **dev)
        for i in range(2):  # stale tokens of earlier requests lie where no request owns a slot
            x = values(pages, page, hkv, D)
            c[i] = (x.float() / scales[i][:, None]).clamp(-448, 448).to(kind) if case["e4m3"] else x
        return c

    if case["op"] == "append":
        tokens, pad = case["tokens"], case["pad"]
        pages = -(-tokens // page) + 3
        order = torch.randperm(pages, generator=gen, **dev)
        at = torch.arange(tokens, **dev)
        slots = torch.full((tokens + pad,), -1, dtype=torch.int32, **dev)
        slots[:tokens] = (order[at // page] * page + at % page).int()
        qkv = values(tokens + pad, hq + 2 * hkv, D)
        return dict(case=case, k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], slots=slots, cache=cache(pages), scales=scales)
    kv, new = _lens(case)
    held = [-(-k // page) for k in kv]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=gen, **dev).int()
    table = torch.full((case["batch"], max(held) + 1), -1, dtype=torch.int32, **dev)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = order[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    qkv = values(cu[-1], hq + 2 * hkv, D)
    return dict(case=case, kv=kv, new=new, cu=cu, q=qkv[:, :hq], cache=cache(pages), table=table, scales=scales,
                cu_seqlens=torch.tensor(cu, dtype=torch.int32, **dev),
                kv_lens=torch.tensor(kv, dtype=torch.int32, **dev),
                sinks=torch.randn((hq,), generator=gen, **dev))


def run(state):
    op = state["case"]["op"]
    if own:
        from sink_sliding_window_b200 import ops
        case = state["case"]
        if op == "plan":
            cu, kv, slots, pool, first = ops.paged_plan(
                state["cached"], state["new"], state["table"], state["ring"], state["pool"], case["page"],
                state["tokens"], case["window"], state["first"])
            return cu, kv, slots, state["table"], state["ring"], pool, first
        k_scale, v_scale = (None, None) if state["scales"] is None else (state["scales"][0], state["scales"][1])
        if op == "append":
            return ops.paged_append(state["k"], state["v"], state["slots"], state["cache"][0], state["cache"][1],
                                    k_scale, v_scale)
        return ops.paged_attn(state["q"], state["cache"][0], state["cache"][1], state["table"], state["cu_seqlens"],
                              state["kv_lens"], state["sinks"], case["window"], max_new=max(state["new"]),
                              k_scale=k_scale, v_scale=v_scale)
    if op == "plan":
        return _plain_plan(state)
    if op == "append":
        return _plain_append(state)
    return _plain_attn(state)


def _plain_plan(s):
    page, window = s["case"]["page"], s["case"]["window"]
    table, ring = s["table"], s["ring"]
    wide, size = table.shape[1], ring.shape[0]
    c, n, first = s["cached"].long(), s["new"].long(), s["first"].long()
    head, count = s["pool"].long()[0], s["pool"].long()[1]
    gone, plus = n < 0, n.clamp(min=0)
    cu = torch.cat([plus.new_zeros(1), plus.cumsum(0)])
    held = (c + page - 1) // page
    need = torch.where(gone | (c + plus > wide * page), 0, (c + plus + page - 1) // page - held)
    upto = need.cumsum(0)
    fits = ~gone & (c + plus <= wide * page) & ((need == 0) | (upto <= count))
    popped = torch.where(fits & (need > 0), upto, 0).max()
    kv = torch.where(fits, c + plus, torch.where(gone, 0, c))
    drop = torch.maximum(first, (c - window + 1).clamp(min=0) // page) if window > 0 else first
    # The slot of every new token, and the table entries of the new pages.
    t = torch.arange(s["tokens"], device=c.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=c.shape[0] - 1)
    at = c[b] + t - cu[b]
    j = (at // page).clamp(max=wide - 1)
    fresh = j >= held[b]
    taken = ring[(head + upto[b] - need[b] + j - held[b]) % size]
    where = torch.where(fresh, taken, table[b, j])
    live = (t < cu[-1]) & fits[b]
    slots = torch.where(live, where * page + at % page, -1)
    # What goes back to the pool: before the table changes.
    col = torch.arange(wide, device=c.device)
    back = table[(col >= first[:, None]) & (col < torch.where(gone, held, drop)[:, None])]
    opens = live & fresh & (at % page == 0)
    table[b[opens], j[opens]] = where[opens]
    ring[(head + count + torch.arange(back.shape[0], device=c.device)) % size] = back
    pool = torch.stack([(head + popped) % size, count - popped + back.shape[0]])
    return tuple(x.int() for x in (cu, kv, slots)) + (table, ring, pool.int(), torch.where(gone, 0, drop).int())


def _plain_append(s):
    k_cache, v_cache = s["cache"][0], s["cache"][1]
    live = s["slots"] >= 0
    to = s["slots"][live].long()
    for i, (x, c) in enumerate(((s["k"], k_cache), (s["v"], v_cache))):
        rows = x[live]
        if s["scales"] is not None:
            rows = (rows.float() * (1.0 / s["scales"][i])[:, None]).clamp(-448, 448).to(E4M3)
            c.view(torch.uint8).view(-1, *c.shape[2:])[to] = rows.view(torch.uint8)
        else:
            c.view(-1, *c.shape[2:])[to] = rows
    return k_cache, v_cache


def _gathered(s, rows, first, pages, i):
    """Keys (i = 0) or values (i = 1) on `pages` pages of the requests `rows`, [rows, slots, hkv, D] in 32 bits."""
    col = (first[:, None] + torch.arange(pages, device="cuda")).clamp(max=s["table"].shape[1] - 1)
    x = s["cache"][i][s["table"][rows].gather(1, col).clamp(min=0).long()].flatten(1, 2).float()
    return x if s["scales"] is None else x * s["scales"][i][:, None]


def _plain_rows(s, rows, new, length):
    """The attention of the requests `rows`, all with `new` new tokens and at most `length` keys."""
    hq, hkv, window, page = (s["case"][key] for key in ("hq", "hkv", "window", "page"))
    take = s["cu_seqlens"][rows].long()[:, None] + torch.arange(new, device="cuda")
    q = s["q"][take].float().view(len(rows), new, hkv, hq // hkv, D)
    # From the page of the first key that a window leaves in sight.
    first = (s["kv_lens"][rows].long() - new - window + 1).clamp(min=0) // page * (window > 0)
    pages = -(-length // page)
    if window > 0:
        pages = min(pages, -(-(window + new - 1) // page) + 1)
    k, v = _gathered(s, rows, first, pages, 0), _gathered(s, rows, first, pages, 1)
    x = torch.matmul(q.permute(0, 2, 1, 3, 4).flatten(2, 3), k.permute(0, 2, 3, 1)) * D ** -0.5
    x = x.view(len(rows), hkv, new, hq // hkv, pages * page)
    i = (s["kv_lens"][rows, None] - new + torch.arange(new, device="cuda"))[:, :, None]
    j = (first[:, None] * page + torch.arange(pages * page, device="cuda"))[:, None]
    seen = (j <= i) & ((i - j < window) if window > 0 else True)
    x = torch.where(seen[:, None, :, None], x, -math.inf)
    sink = s["sinks"].view(hkv, 1, hq // hkv)
    top = torch.maximum(x.amax(-1), sink)
    p = (x - top[..., None]).exp()
    total = p.sum(-1) + (sink - top).exp()
    y = torch.matmul(p.flatten(2, 3), v.transpose(1, 2)).view(*total.shape, D) / total[..., None]
    return take, y.permute(0, 2, 1, 3, 4).flatten(2, 3), (top + total.log()).permute(1, 3, 0, 2).flatten(0, 1)


def _plain_attn(s):
    out = torch.empty((s["cu"][-1], s["case"]["hq"], D), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((s["case"]["hq"], s["cu"][-1]), device="cuda")
    # Requests with the same few new tokens go together, a longer chunk by itself.
    few = sorted({n for n in s["new"] if n <= 4})
    groups = [[b for b, n in enumerate(s["new"]) if n == m] for m in few] + [[b] for b, n in enumerate(s["new"]) if n > 4]
    for rows in groups:
        take, y, l = _plain_rows(s, torch.tensor(rows, device="cuda"), s["new"][rows[0]], max(s["kv"][b] for b in rows))
        out[take] = y.to(torch.bfloat16)
        lse[:, take] = l
    return out, lse


def work(case):
    if case["op"] == "plan":
        cached, new = _plan_lens(case)
        tokens = sum(max(0, n) for n in new) + 5
        fresh = sum(-(-(c + n) // case["page"]) - -(-c // case["page"]) for c, n in zip(cached, new) if n > 0)
        return dict(bytes=4 * (6 * case["batch"] + tokens + 2 * fresh), flops=0)
    size = 1 if case["e4m3"] else 2
    if case["op"] == "append":
        return dict(bytes=case["tokens"] * (2 * case["hkv"] * D * (2 + size) + 4), flops=0)
    keys = pairs = tokens = 0
    for k, n in zip(*_lens(case)):
        w = case["window"] if case["window"] > 0 else k
        keys += min(k, n - 1 + w)
        pairs += sum(min(w, k - n + t + 1) for t in range(n))
        tokens += n
    return dict(bytes=keys * 2 * case["hkv"] * D * size + tokens * case["hq"] * (2 * D * 2 + 4),
                flops=4 * D * pairs * case["hq"])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return _exact_plan(s)
    if case["op"] == "append":
        return _exact_append(s)
    hq, hkv, page, window = case["hq"], case["hkv"], case["page"], case["window"]
    out = torch.empty((s["cu"][-1], hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((hq, s["cu"][-1]), dtype=torch.float64, device="cuda")
    for b, (length, new) in enumerate(zip(s["kv"], s["new"])):
        slots = [int(p) for p in s["table"][b, : -(-length // page)].tolist()]
        rows = slice(s["cu"][b], s["cu"][b + 1])
        place = torch.arange(length - new, length, device="cuda")[:, None] - torch.arange(length, device="cuda")[None, :]
        masked = (place < 0) | (place >= (window if window > 0 else length + 1))
        for g in range(hkv):
            k, v = (torch.cat([s["cache"][i, p, :, g].double() for p in slots])[:length] if length <= 512 else
                    s["cache"][i, slots, :, g].double().reshape(-1, D)[:length] for i in range(2))
            if s["scales"] is not None:
                k, v = k * s["scales"][0, g].double(), v * s["scales"][1, g].double()
            for h in range(g * (hq // hkv), (g + 1) * (hq // hkv)):
                logits = (s["q"][rows, h].double() @ k.T / math.sqrt(D)).masked_fill_(masked, -math.inf)
                logits = torch.cat([logits, s["sinks"][h].double().expand(new, 1)], 1)
                lse[h, rows] = torch.logsumexp(logits, 1)
                out[rows, h] = torch.softmax(logits, 1)[:, :-1] @ v
    return out, lse


def _exact_append(s):
    page, got = s["case"]["page"], []
    for i, x in enumerate((s["k"], s["v"])):
        x, c = x.double(), s["cache"][i].double()
        if s["scales"] is not None:
            x = (x / s["scales"][i].double()[:, None]).clamp(-448.0, 448.0)
            step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
            x = torch.round(x / step) * step  # to the nearest of a binade's eight values, ties to the even one
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        to = s["slots"][keep].long()
        c[to // page, to % page] = x[keep]
        got.append(c)
    return got


def _exact_plan(s):
    """The step request by request, as one would plan it by hand."""
    page, window = s["case"]["page"], s["case"]["window"]
    table, ring = s["table"].tolist(), s["ring"].tolist()
    size, (head, count) = len(ring), s["pool"].tolist()
    old = [list(row) for row in table]
    free = [ring[(head + i) % size] for i in range(count)]
    cu, kv, slots, first, back, used, asked = [0], [], [], [], [], 0, 0
    for b, (c, n, low) in enumerate(zip(s["cached"].tolist(), s["new"].tolist(), s["first"].tolist())):
        held = -(-c // page)
        if n < 0:
            back += old[b][low:held]
            cu.append(cu[-1])
            kv.append(0)
            first.append(0)
            continue
        drop = max(low, max(0, c - window + 1) // page) if window > 0 else low
        back += old[b][low:drop]
        first.append(drop)
        cu.append(cu[-1] + n)
        need = -(-(c + n) // page) - held
        if c + n > len(table[b]) * page:
            need, ok = 0, False
        else:
            asked += need
            ok = need == 0 or asked <= count
        if ok:
            for j in range(held, held + need):
                table[b][j] = free[used]
                used += 1
        kv.append(c + n if ok else c)
        slots += [table[b][p // page] * page + p % page if ok else -1 for p in range(c, c + n)]
    slots += [-1] * (s["tokens"] - len(slots))
    for i, p in enumerate(back):
        ring[(head + count + i) % size] = p
    as_int = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return tuple(as_int(v) for v in (cu, kv, slots, table, ring, [(head + used) % size, count - used + len(back)], first))
