"""sink_attn_paged_plan: the planned step against the one planned by hand, on
the lengths, pools and windows where it can go wrong; its refusals (CPU)."""
import ctypes
import random

import pytest
import torch

from sink_sliding_window_b200 import build, ops
from tests.paged_util import plan


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.load()


def _state(rng, cached, new, page, window, spare, max_pages, with_first):
    """A pool and a table that own what the lengths say."""
    first = [rng.randint(0, max(0, c - window) // page) if window and c > window else 0 for c in cached]
    if not with_first:
        first = [0] * len(cached)
    held = [-(-c // page) for c in cached]
    n = sum(h - f for h, f in zip(held, first)) + spare
    n = max(n, 1)
    ids = list(range(n))
    rng.shuffle(ids)
    table = [[-1] * max_pages for _ in cached]
    for b in range(len(cached)):
        for j in range(first[b], held[b]):
            table[b][j] = ids.pop()
    head = rng.randrange(n)
    ring = [-1] * n
    count = len(ids)
    for i, p in enumerate(ids):
        ring[(head + i) % n] = p
    return table, ring, [head, count], first


def _run(cached, new, table, ring, pool, page, max_tokens, window, first, **kw):
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    tb, rg = t(table), t(ring)
    got = ops.paged_plan(t(cached), t(new), tb, rg, t(pool), page, max_tokens, window,
                         None if first is None else t(first), **kw)
    torch.cuda.synchronize()
    cu, kv, slots, pool_out, first_out = got
    return [cu.tolist(), kv.tolist(), slots.tolist(), tb.tolist(), rg.tolist(), pool_out.tolist(),
            None if first_out is None else first_out.tolist()]


def _compare(got, want):
    for name, g, w in zip(("cu_seqlens", "kv_lens", "slot_map", "block_table", "free_pages", "pool", "first_page"),
                          got, want):
        if g is not None:
            assert g == list(w), name


CASES = [  # batch, longest, most new, page, window, spare
    (1, 0, 1, 16, 0, 1), (1, 40, 1, 16, 0, 4), (3, 100, 40, 32, 0, 40), (33, 300, 1, 64, 0, 40),
    (65, 500, 300, 16, 0, 3000), (40, 900, 60, 16, 100, 300), (257, 200, 3, 128, 16, 300), (31, 64, 5000, 1024, 0, 300),
    (1025, 90, 4, 16, 20, 1025), (4096, 20, 2, 16, 1, 4096),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "b%d-l%d-n%d-p%d-w%d" % c[:5])
def test_plan_matches_by_hand(case):
    batch, longest, most, page, window, spare = case
    rng = random.Random(batch * 7 + page)
    cached = [rng.choice([0, rng.randint(0, longest)]) for _ in range(batch)]
    new = [rng.choice([-1, 0, 1, rng.randint(0, most)]) for _ in range(batch)]
    max_pages = -(-(longest + most) // page) + 1
    table, ring, pool, first = _state(rng, cached, new, page, window, spare, max_pages, True)
    tokens = sum(max(0, n) for n in new)
    for max_tokens in {tokens, tokens + 37}:
        got = _run(cached, new, table, ring, pool, page, max_tokens, window, first)
        assert ops.device_error() == 0
        _compare(got, plan(cached, new, table, ring, pool, page, max_tokens, window, first))


@pytest.mark.gpu
def test_plan_without_first_page_and_all_ended():
    cached, new, page = [33, 0, 64, 17], [-1, -5, -1, -1], 16
    table, ring, pool, _ = _state(random.Random(1), cached, new, page, 0, 3, 6, False)
    got = _run(cached, new, table, ring, pool, page, 5, 0, None)
    _compare(got, plan(cached, new, table, ring, pool, page, 5))
    assert got[5][1] == 3 + 3 + 4 + 2


@pytest.mark.gpu
@pytest.mark.parametrize("spare", [0, 1, 3, 5])
def test_plan_pool_runs_dry(spare):
    """Requests are served in order while pages last; one that needs none is
    served anyway, and the others keep their lengths."""
    cached, new, page = [16, 15, 30, 32, 16, 1], [17, 1, 3, 16, 1, 2], 16
    table, ring, pool, _ = _state(random.Random(2), cached, new, page, 0, spare, 5, False)
    want = plan(cached, new, table, ring, pool, page, sum(new))
    _compare(_run(cached, new, table, ring, pool, page, sum(new), 0, None), want)
    assert ops.device_error() == (0x202 if spare < 5 else 0)
    assert want[1][1] == 16 and want[1][5] == 3


@pytest.mark.gpu
def test_plan_records_lengths_that_do_not_fit():
    """A request longer than its table row gets nothing; a step with more
    tokens than the slot map keeps every write inside it."""
    cached, new, page = [30, 5], [4, 3], 16
    table, ring, pool, _ = _state(random.Random(3), cached, new, page, 0, 4, 2, False)
    got = _run(cached, new, table, ring, pool, page, 7, 0, None)
    assert ops.device_error() == 0x204
    _compare(got, plan(cached, new, table, ring, pool, page, 7))
    assert got[1] == [30, 8] and got[2][:4] == [-1] * 4
    guard = torch.full((16,), 77, dtype=torch.int32, device="cuda")
    got = _run([0, 5], [4, 3], table, ring, pool, page, 5, 0, None, slot_map=guard[:5])
    assert ops.device_error() == 0x204
    assert guard[5:].tolist() == [77] * 11 and len(got[2]) == 5
    assert _run([-3], [1], [[-1, -1]], ring, pool, page, 1, 0, None)[2] == [-1]
    assert ops.device_error() == 0x204
    # A table entry outside the pool gives no slot.
    assert _run([5], [1], [[99, -1]], ring, pool, page, 1, 0, None)[2] == [-1]
    assert ops.device_error() == 0x203


@pytest.mark.gpu
def test_plan_in_place_over_many_steps():
    """The lengths, the pool and the given-back pages updated in place, step
    after step, with requests that end and start again: every page is always
    owned once, by a request or by the pool."""
    rng = random.Random(5)
    B, page, window, max_pages, N = 9, 16, 40, 12, 70
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    cached, first, pool = t([0] * B), t([0] * B), t([0, N])
    table, ring = t([[-1] * max_pages] * B), t(list(range(N)))
    h = dict(cached=[0] * B, first=[0] * B, pool=[0, N], table=[[-1] * max_pages] * B, ring=list(range(N)))
    for _ in range(60):
        new = [rng.choice([-1, 0, 1, 1, 1, rng.randint(0, 30)]) for _ in range(B)]
        new = [n if c + max(n, 0) <= max_pages * page else -1 for c, n in zip(h["cached"], new)]
        tokens = sum(max(0, n) for n in new)
        cu, kv, slots, _, _ = ops.paged_plan(cached, t(new), table, ring, pool, page, tokens + 3, window, first,
                                             kv_lens=cached, pool_out=pool, first_page_out=first)
        want = plan(h["cached"], new, h["table"], h["ring"], h["pool"], page, tokens + 3, window, h["first"])
        _compare([cu.tolist(), cached.tolist(), slots.tolist(), table.tolist(), ring.tolist(), pool.tolist(),
                  first.tolist()], want)
        h.update(cached=want[1], table=want[3], ring=want[4], pool=want[5], first=want[6])
        owned = [h["table"][b][j] for b in range(B) for j in range(h["first"][b], -(-h["cached"][b] // page))]
        owned += [h["ring"][(h["pool"][0] + i) % N] for i in range(h["pool"][1])]
        assert sorted(owned) == list(range(N))
    ops.device_error()


@pytest.mark.gpu
def test_plan_captured_and_replayed_with_new_lengths():
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    page, N, B = 16, 64, 3
    rng = random.Random(9)
    cached, new = t([0] * B), t([1] * B)
    table, ring, pool = t([[-1] * 8] * B), t(list(range(N))), t([5, N])
    outs = dict(cu_seqlens=t([0] * (B + 1)), kv_lens=t([0] * B), slot_map=t([0] * 64), pool_out=t([0, 0]))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    saved = table.clone()
    with torch.cuda.stream(stream):
        ops.paged_plan(cached, new, table, ring, pool, page, 64, **outs)
        table.copy_(saved)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ops.paged_plan(cached, new, table, ring, pool, page, 64, **outs)
    torch.cuda.current_stream().wait_stream(stream)
    for _ in range(4):
        n = [rng.randint(0, 20) for _ in range(B)]
        new.copy_(t(n))
        table.copy_(saved)
        graph.replay()
        torch.cuda.synchronize()
        want = plan([0] * B, n, saved.tolist(), list(range(N)), [5, N], page, 64)
        _compare([outs["cu_seqlens"].tolist(), outs["kv_lens"].tolist(), outs["slot_map"].tolist(), table.tolist(),
                  ring.tolist(), outs["pool_out"].tolist(), None], want)


def _args(d, ptr=4096, **kw):
    a = dict(cached=ptr, new=ptr, table=ptr, ring=ptr, pool=ptr, first=None, window=0, cu=ptr, kv=ptr, slots=ptr,
             pool_out=ptr, first_out=None)
    a.update(kw)
    P = ctypes.c_void_p
    return (ctypes.byref(d) if d is not None else None, P(a["cached"]), P(a["new"]), P(a["table"]), P(a["ring"]),
            P(a["pool"]), P(a["first"]), a["window"], P(a["cu"]), P(a["kv"]), P(a["slots"]), P(a["pool_out"]),
            P(a["first_out"]), None)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), 2), (dict(max_tokens=-1), 2), (dict(max_pages=0), 2), (dict(page_size=0), 2),
    (dict(num_pages=0), 2), (dict(page_size=48), 4), (dict(page_size=8), 4), (dict(page_size=2048), 4),
    (dict(batch=4097), 4), (dict(num_pages=1 << 28), 4), (dict(max_pages=1 << 26), 4), (dict(max_tokens=(1 << 30) + 1), 4),
])
def test_plan_rejects_bad_sizes(L, bad, code):
    s = dict(batch=2, max_tokens=8, max_pages=4, page_size=16, num_pages=8)
    s.update(bad)
    assert L.sink_attn_paged_plan(*_args(ops.PlanDims(**s))) == code


def test_plan_rejects_bad_pointers(L):
    d = ops.PlanDims(2, 8, 4, 16, 8)
    assert L.sink_attn_paged_plan(*_args(None)) == 1
    for name in ("cached", "new", "table", "ring", "pool", "cu", "kv", "slots", "pool_out"):
        assert L.sink_attn_paged_plan(*_args(d, **{name: None})) == 1, name
        assert L.sink_attn_paged_plan(*_args(d, **{name: 4098})) == 3, name
    assert L.sink_attn_paged_plan(*_args(d, window=5)) == 1
    assert L.sink_attn_paged_plan(*_args(d, first=4096)) == 1
    assert L.sink_attn_paged_plan(*_args(d, first=4096, first_out=4097)) == 3
    d.batch = 0
    assert L.sink_attn_paged_plan(*_args(d)) == 0


def test_plan_binding_refuses_host_tensors(L):
    z = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.paged_plan(z, z, z.view(2, 1), z, z, 16, 4)
