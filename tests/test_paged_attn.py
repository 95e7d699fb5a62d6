"""sink_attn_paged_append and sink_attn_paged_attn (CUDA, through the C ABI)
against the definition in 64 bits: lengths around tile and page ends, head
layouts, windows, sinks, layouts of the cache, stale slots that hold NaN, and
the three paged calls together as a serving loop uses them.  Refusals: CPU."""
import ctypes

import numpy as np
import pytest
import torch

from sink_sliding_window_b200 import build, ops
from tests.paged_util import NAN_CODE, Paged, quantise


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.load()


KINDS = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])


# ------------------------------------------------------------------ append
@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("layout", ["token", "head", "fused"])
@pytest.mark.parametrize("tokens,hkv,page", [(1, 8, 64), (33, 1, 16), (300, 3, 128), (1000, 8, 16)])
def test_append(e4m3, layout, tokens, hkv, page):
    """Every new row is in its slot, bit for bit; skipped rows and all other
    slots are as they were."""
    p = Paged([5], [1], hkv, hkv, page, e4m3=e4m3, layout=layout, extra_pages=-(-tokens // page) + 2)
    gen = torch.Generator().manual_seed(tokens)
    qkv = torch.randn((tokens, 4 + 2 * hkv, 64), generator=gen).to(torch.bfloat16)
    qkv[0, 4:, 0] = 1e5  # saturates in e4m3
    k, v = qkv[:, 4:4 + hkv], qkv[:, 4 + hkv:]
    slots = torch.randperm(p.pages * page, generator=gen)[:tokens].int()
    slots[tokens // 2::3] = -1
    dev = qkv.cuda()
    store = p.store.cuda()
    kc, vc = p.views(store)
    scales = (p.k_scale.cuda(), p.v_scale.cuda()) if e4m3 else (None, None)
    got = ops.paged_append(dev[:, 4:4 + hkv], dev[:, 4 + hkv:], slots.cuda(), kc, vc, *scales)
    torch.cuda.synchronize()
    assert got[0] is kc and got[1] is vc and ops.device_error() == 0
    want = p.store.clone()
    for x, c, s in zip((k, v), p.views(want), (p.k_scale, p.v_scale)):
        codes = quantise(x, s)[0] if e4m3 else x
        for t, z in enumerate(slots.tolist()):
            if z >= 0:
                c[z // page, z % page] = codes[t]
    bits = torch.uint8 if e4m3 else torch.int16
    assert torch.equal(store.cpu().view(bits), want.view(bits))


@pytest.mark.gpu
def test_append_records_a_slot_outside_the_pool():
    p = Paged([5], [1], 1, 1, 16)
    kc, vc = p.views(p.store.cuda())
    before = kc.clone()
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    ops.paged_append(x, x, torch.tensor([p.pages * 16, -7], dtype=torch.int32, device="cuda"), kc, vc)
    assert ops.device_error() == 0x203
    assert torch.equal(kc.view(torch.int16), before.view(torch.int16))


@pytest.mark.gpu
def test_append_past_32_bit_offsets():
    """Slots whose element offset does not fit 32 bits."""
    pages, page, hkv = (1 << 32) // (64 * 64 * 8) + 3, 64, 8
    if torch.cuda.mem_get_info()[0] < 20 << 30:
        pytest.skip("needs 20 GB")
    kc = torch.zeros((pages, page, hkv, 64), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((2, hkv, 64), device="cuda").to(torch.bfloat16)
    slots = torch.tensor([pages * page - 1, 3], dtype=torch.int32, device="cuda")
    ops.paged_append(x, x, slots, kc, kc.clone())
    assert ops.device_error() == 0
    assert torch.equal(kc[-1, -1], x[0]) and torch.equal(kc[0, 3], x[1]) and not kc[1:-1].any()
    # ... and attention over the last pages of such a pool.
    p = Paged([200], [3], 16, 8, page)
    for j in range(4):
        part = p.k[0][j * page:(j + 1) * page].cuda()
        kc[pages - 4 + j, :part.shape[0]] = part
    p.vd = p.kd  # the values are the keys here
    table = torch.arange(pages - 4, pages, dtype=torch.int32, device="cuda").view(1, 4)
    a = p.device()
    out, lse = ops.paged_attn(a["q"], kc, kc, table, a["cu_seqlens"], a["kv_lens"], a["sinks"])
    p.check(out, lse)


# --------------------------------------------------------------- attention
EDGES = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300, 1000]


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("window", [0, 1, 100, 128])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_one_token(e4m3, window, page):
    p = Paged(EDGES, [1] * len(EDGES), 16, 2, page, window, e4m3, seed=window + page)
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("layout", ["token", "head", "fused"])
def test_cache_layouts(e4m3, layout):
    p = Paged([300, 77, 1], [70, 1, 1], 8, 2, 32, 0, e4m3, seed=3, layout=layout)
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (3, 1), (10, 2), (7, 1), (24, 2), (16, 1), (32, 1), (33, 1), (64, 1), (128, 1), (100, 1)])
def test_head_groups(e4m3, hq, hkv):
    """Any number of query heads per key/value head, one and several tokens."""
    for new in ([1, 1, 1, 1], [2, 0, 5, 3], [40, 1, 17, 130]):
        p = Paged([129, 64, 200, 300], new, hq, hkv, 16, 0, e4m3, seed=hq)
        p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("window", [0, 5, 100, 128, 1000])
def test_chunks(e4m3, window):
    """Chunks of every length over cached tokens, whole prompts among them."""
    kv = [1, 40, 128, 129, 300, 513, 777, 1024]
    new = [1, 40, 127, 2, 200, 513, 64, 333]
    p = Paged(kv, new, 8, 2, 16, window, e4m3, seed=window)
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("window", [0, 128])
def test_mixed_batch(e4m3, window):
    """Chunks, single tokens and idle requests in one call."""
    kv = [900, 33, 0, 257, 64, 1200, 5, 17, 128, 600, 0, 1]
    new = [300, 1, 0, 1, 0, 1, 5, 1, 1, 2, 0, 1]
    p = Paged(kv, new, 16, 2, 64, window, e4m3, seed=window)
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_many_idle_requests(e4m3):
    """A batch far larger than the step: most requests are idle."""
    kv, new = [0] * 700, [0] * 700
    for b, (k, n) in zip((0, 3, 31, 32, 350, 698, 699), ((9, 9), (70, 1), (400, 1), (400, 33), (128, 1), (1, 1), (65, 2))):
        kv[b], new[b] = k, n
    p = Paged(kv, new, 8, 1, 16, 0, e4m3, seed=1)
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_long_context_splits(e4m3):
    """Few rows over many keys: the key range is split and joined."""
    for kv, new in (([20000], [1]), ([9000, 20001], [4, 1]), ([16000], [40])):
        p = Paged(kv, new, 8, 1, 64, 0, e4m3, seed=4)
        p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_sinks(e4m3):
    """Sinks off, far below, far above the logits."""
    sinks = [-np.inf, -1e4, 0.0, 1e4, 0.5, -30.0, 30.0, -np.inf]
    for kv, new in (([300, 1, 65, 0], [1, 1, 2, 0]), ([300, 64], [100, 64])):
        p = Paged(kv, new, 8, 1, 16, 0, e4m3, seed=6, sinks=sinks)
        p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_wide_logits(e4m3):
    """Large logits: the running maximum is raised again and again."""
    for kv, new in (([1500, 700], [1, 1]), ([900], [200])):
        p = Paged(kv, new, 8, 1, 32, 0, e4m3, seed=7, std=2.5)
        p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_one_key_far_above_the_others(e4m3):
    """A key e^12 above thousands of others that together weigh a few percent
    of it: the small weights may not be lost."""
    p = Paged([6000], [1], 8, 1, 64, 0, e4m3, seed=8)
    k = torch.zeros_like(p.k[0])
    k[100] = 1.0
    p.q[:] = 12.0 / 8.0
    p.k[0] = k
    codes = quantise(k, p.k_scale)[0] if e4m3 else k
    p.kd[0] = quantise(k, p.k_scale)[1] if e4m3 else k.double()
    kc = p.views(p.store)[0]
    for j, page in enumerate(p.table[0, :94].tolist()):
        part = codes[j * 64:(j + 1) * 64]
        kc[page, :part.shape[0]] = part
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_rows_that_see_nothing(e4m3):
    """A request whose kv_lens says less than its new tokens (one the plan
    had no room for): rows before position 0 see no key, out = 0, lse = sink."""
    p = Paged([3, 50], [1, 1], 8, 1, 16, 0, e4m3, seed=9)
    a = p.device()
    for n in (6, 80):
        q = torch.randn((n + 1, 8, 64), device="cuda").to(torch.bfloat16)
        cu = torch.tensor([0, n, n + 1], dtype=torch.int32, device="cuda")
        out, lse = ops.paged_attn(q, a["k_cache"], a["v_cache"], a["block_table"], cu, a["kv_lens"], a["sinks"],
                                  k_scale=a["k_scale"], v_scale=a["v_scale"])
        assert ops.device_error() == 0
        assert not out[:n - 3].any() and torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
        assert torch.equal(lse[:, :n - 3], a["sinks"][:, None].expand(8, n - 3).contiguous()) or \
            torch.allclose(lse[:, :n - 3], a["sinks"][:, None], rtol=2e-7, atol=2e-7)


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("new", [[1, 1], [50, 3]])
def test_rows_behind_the_last_request_are_left(e4m3, new):
    p = Paged([90, 60], new, 8, 2, 16, 0, e4m3, seed=10, pad_rows=9)
    out = torch.full((p.rows, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((8, p.rows), 7.0, device="cuda")
    p.check(*p.run(ops, out=out, lse=lse))
    assert (out[p.T:] == 7).all() and (lse[:, p.T:] == 7).all()


@pytest.mark.gpu
@KINDS
def test_strided_queries_and_scale(e4m3):
    p = Paged([90, 300], [1, 33], 8, 2, 16, 0, e4m3, seed=11)
    a = p.device()
    qkv = torch.full((p.T, 12, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    qkv[:, :8] = a.pop("q")
    a.pop("max_new")
    out, lse = ops.paged_attn(qkv[:, :8], a["k_cache"], a["v_cache"], a["block_table"], a["cu_seqlens"],
                              a["kv_lens"], a["sinks"], scale=0.3, k_scale=a["k_scale"], v_scale=a["v_scale"])
    torch.cuda.synchronize()
    p.check(out, lse, scale=0.3)


@pytest.mark.gpu
@KINDS
def test_a_needed_page_outside_the_pool_is_recorded(e4m3):
    """The other request's rows are right, nothing is read out of range."""
    for new in ([1, 1], [40, 40]):
        p = Paged([300, 200], new, 8, 1, 16, 0, e4m3, seed=12)
        a = p.device()
        for bad in (-1, p.pages, 1 << 30):
            a["block_table"][0, 7] = bad
            out, lse = ops.paged_attn(a["q"], a["k_cache"], a["v_cache"], a["block_table"], a["cu_seqlens"],
                                      a["kv_lens"], a["sinks"], max_new=a["max_new"], k_scale=a["k_scale"],
                                      v_scale=a["v_scale"])
            assert ops.device_error() == 0x203
            good = p.reference()
            r = slice(new[0], p.T)
            assert ((out[r].double().cpu() - good[0][r]).abs() <= good[2][r]).all()


@pytest.mark.gpu
def test_lengths_that_do_not_fit_are_recorded():
    """More rows than total_tokens, or than max_new: device error 0x205, and
    every access stays inside the tensors."""
    p = Paged([300, 200], [40, 2], 8, 1, 16, 0, seed=13)
    a = p.device()
    args = (a["q"], a["k_cache"], a["v_cache"], a["block_table"])
    guard = torch.full((p.T + 8, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 40, p.T + 500], dtype=torch.int32, device="cuda")
    ops.paged_attn(*args, cu, a["kv_lens"], a["sinks"], out=guard[:p.T])
    assert ops.device_error() == 0x205 and (guard[p.T:] == 7).all()
    ops.paged_attn(*args, a["cu_seqlens"], a["kv_lens"], a["sinks"], max_new=2)
    assert ops.device_error() == 0x205
    out, lse = ops.paged_attn(*args, a["cu_seqlens"], a["kv_lens"], a["sinks"], max_new=40)
    assert ops.device_error() == 0
    p.check(out, lse)


@pytest.mark.gpu
@KINDS
def test_same_answer_twice_and_two_streams_at_once(e4m3):
    """Two calls that overlap on two streams, each with its own workspace,
    give what they give alone, bit for bit."""
    ps = [Paged([3000, 900], [1, 1], 16, 2, 16, 0, e4m3, seed=14), Paged([1500, 900], [600, 1], 16, 2, 16, 0, e4m3, seed=15)]
    alone = [p.run(ops) for p in ps]
    args = [p.device() for p in ps]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ps]
    got = []
    for _ in range(3):
        for a, s in zip(args, streams):
            b = dict(a)
            got.append(ops.paged_attn(b.pop("q"), b.pop("k_cache"), b.pop("v_cache"), b.pop("block_table"),
                                      b.pop("cu_seqlens"), b.pop("kv_lens"), b.pop("sinks"), **b, stream=s))
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, alone[i % 2][0]) and torch.equal(l, alone[i % 2][1])


@pytest.mark.gpu
@KINDS
def test_serving_loop(e4m3):
    """Plan, append and attention together: prompts in chunks, then single
    tokens, on a full-causal and on a window-64 layer with a pool of their
    own each; the second pool is too small for the whole context and lives on
    the pages its window gives back.  A captured decode step is replayed at
    the end.  Every row equals the definition over the whole history."""
    B, hq, hkv, page, W = 4, 8, 2, 16, 64
    gen = torch.Generator(device="cuda").manual_seed(1)
    total = [150, 37, 260, 5]
    hist = [torch.randn((n, hq + 2 * hkv, 64), generator=gen, device="cuda").to(torch.bfloat16) for n in total]
    sinks = torch.randn((hq,), generator=gen, device="cuda")
    scales = [torch.full((hkv,), 0.01, device="cuda") for _ in range(2)] if e4m3 else [None, None]
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    layers = []
    for window, pages in ((0, 40), (W, 32)):
        kind = torch.uint8 if e4m3 else torch.bfloat16
        cache = torch.full((2, pages, page, hkv, 64), NAN_CODE if e4m3 else float("nan"), dtype=kind, device="cuda")
        layers.append(dict(window=window, cache=cache, table=t([[-1] * 17] * B), ring=t(list(range(pages))),
                           pool=t([0, pages]), lens=t([0] * B), first=t([0] * B), out=[[] for _ in range(B)],
                           lse=[[] for _ in range(B)]))
    done = [0] * B
    step = 0
    while any(d < n for d, n in zip(done, total)):
        chunk = 60 if step < 3 else 1 if step % 7 else 9
        new = [min(chunk, n - d) for d, n in zip(done, total)]
        x = torch.cat([h[d:d + m] for h, d, m in zip(hist, done, new)])
        pad = torch.cat([x, torch.zeros_like(x[:3])])
        for y in layers:
            cu, _, slots, _, _ = ops.paged_plan(y["lens"], t(new), y["table"], y["ring"], y["pool"], page, pad.shape[0],
                                                y["window"], y["first"], kv_lens=y["lens"], pool_out=y["pool"],
                                                first_page_out=y["first"])
            ops.paged_append(pad[:, hq:hq + hkv], pad[:, hq + hkv:], slots, y["cache"][0], y["cache"][1], *scales)
            out, lse = ops.paged_attn(pad[:, :hq], y["cache"][0], y["cache"][1], y["table"], cu, y["lens"], sinks,
                                      y["window"], max_new=max(new), k_scale=scales[0], v_scale=scales[1])
            assert ops.device_error() == 0
            at = 0
            for b, m in enumerate(new):
                y["out"][b].append(out[at:at + m].cpu())
                y["lse"][b].append(lse[:, at:at + m].cpu())
                at += m
        done = [d + m for d, m in zip(done, new)]
        step += 1
    for y in layers:
        assert y["lens"].tolist() == total
        p = Paged([1], [1], hq, hkv, page, y["window"], e4m3)
        p.kv, p.new, p.T = total, total, sum(total)
        p.cu = np.concatenate([[0], np.cumsum(total)])
        p.q, p.sinks = torch.cat([h[:, :hq] for h in hist]).cpu(), sinks.cpu()
        parts = [[h[:, a:a + hkv].cpu() for h in hist] for a in (hq, hq + hkv)]
        p.kd, p.vd = ([quantise(x, s.cpu())[1] if e4m3 else x.double() for x in part] for part, s in zip(parts, scales))
        p.check(torch.cat([torch.cat(o) for o in y["out"]]), torch.cat([torch.cat(o, 1) for o in y["lse"]], 1))


@pytest.mark.gpu
@KINDS
def test_captured_step_replayed_with_new_lengths(e4m3):
    """A step captured once serves other lengths, cached and new, as long as
    they stay within max_new and the padded rows."""
    ps = [Paged([40, 900, 300], n, 8, 2, 16, 0, e4m3, seed=s, pad_rows=48 - sum(n)) for s, n in
          enumerate(([1, 1, 1], [40, 0, 3], [0, 30, 1]))]
    a = ps[0].device()
    wide = max(p.pages for p in ps)
    assert wide == ps[0].pages
    out = torch.zeros((48, 8, 64), dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros((8, 48), device="cuda")
    a.pop("max_new")
    args = [a.pop(k) for k in ("q", "k_cache", "v_cache", "block_table", "cu_seqlens", "kv_lens", "sinks")]
    kw = dict(a, out=out, lse=lse, max_new=40)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ops.paged_attn(*args, **kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            ops.paged_attn(*args, **kw)
    torch.cuda.synchronize()
    for p in ps:
        b = p.device()
        for x, name in zip(args, ("q", "k_cache", "v_cache", "block_table", "cu_seqlens", "kv_lens", "sinks")):
            x.copy_(b[name])
        for name in ("k_scale", "v_scale"):
            if e4m3:
                kw[name].copy_(b[name])
        graph.replay()
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        p.check(out, lse)


# ---------------------------------------------------------- refusals (CPU)
def _dims(**kw):
    d = dict(batch=2, total_tokens=4, max_new=2, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=9,
             max_pages=4, page_stride=2048, token_stride=128, head_stride=64, q_stride=512)
    d.update(kw)
    return ops.PagedDims(**d)


def _call(L, d, e4m3=False, window=0, scale=0.125, ws=1 << 40, **kw):
    P = ctypes.c_void_p
    names = ["q", "k", "v", "table", "cu", "kv"] + (["ks", "vs"] if e4m3 else []) + ["sinks"]
    a = {n: 4096 for n in names + ["out", "lse", "workspace"]}
    a.update(kw)
    f = L.sink_attn_paged_attn_e4m3 if e4m3 else L.sink_attn_paged_attn
    return f(None if d is None else ctypes.byref(d), *[P(a[n]) for n in names], window, scale, P(a["out"]), P(a["lse"]),
             P(a["workspace"]), ws, None)


@pytest.mark.parametrize("bad,code", [
    (dict(batch=-1), 2), (dict(total_tokens=-1), 2), (dict(max_new=0), 2), (dict(num_kv_heads=0), 2),
    (dict(num_q_heads=0), 2), (dict(num_q_heads=7), 2), (dict(head_dim=128), 4), (dict(page_size=0), 2),
    (dict(page_size=8), 4), (dict(page_size=24), 4), (dict(page_size=2048), 4), (dict(num_pages=0), 2),
    (dict(num_pages=1 << 27), 4), (dict(max_pages=0), 2), (dict(max_pages=1 << 27), 4), (dict(num_q_heads=258), 4),
    (dict(page_stride=2044), 3), (dict(token_stride=-128), 2), (dict(q_stride=513), 3), (dict(head_stride=68), 3),
])
def test_attn_rejects_bad_sizes(L, bad, code):
    assert _call(L, _dims(**bad)) == code
    if "max_new" not in bad and "num_q_heads" not in bad and "max_pages" not in bad and "batch" not in bad and "q_stride" not in bad:
        P = ctypes.c_void_p
        assert L.sink_attn_paged_append(ctypes.byref(_dims(**bad)), P(4096), P(4096), 512, 512, P(4096), P(4096),
                                        P(4096), None) == code


def test_attn_rejects_bad_pointers_scale_and_workspace(L):
    d = _dims()
    assert _call(L, None) == 1
    for e4m3 in (False, True):
        names = ["q", "k", "v", "table", "cu", "kv", "sinks", "out", "lse"] + (["ks", "vs"] if e4m3 else [])
        for n in names:
            assert _call(L, d, e4m3, **{n: None}) == 1, n
            assert _call(L, d, e4m3, **{n: 4098}) == 3, n
        assert _call(L, d, e4m3, workspace=None) == 7
        assert _call(L, d, e4m3, workspace=4096 + 128) == 7
        assert _call(L, d, e4m3, ws=0) == 7
        for s in (0.0, -1.0, float("nan"), float("inf")):
            assert _call(L, d, e4m3, scale=s) == 4
    # A byte cache needs rows that are multiples of 16 elements apart.
    assert _call(L, _dims(head_stride=72), True) == 3
    assert L.sink_attn_paged_workspace_size(ctypes.byref(_dims(head_dim=32))) == 0
    assert L.sink_attn_paged_workspace_size(ctypes.byref(d)) > 0
    assert _call(L, _dims(total_tokens=0), q=None) == 0 and _call(L, _dims(batch=0), q=None) == 0


def test_append_rejects_bad_pointers(L):
    P = ctypes.c_void_p
    good = [4096, 4096, 512, 512, 4096, 4096, 4096]
    def call(d, args):
        return L.sink_attn_paged_append(None if d is None else ctypes.byref(d), P(args[0]), P(args[1]), args[2],
                                        args[3], P(args[4]), P(args[5]), P(args[6]), None)
    assert call(None, good) == 1
    for i in (0, 1, 4, 5, 6):
        assert call(_dims(), good[:i] + [None] + good[i + 1:]) == 1
        assert call(_dims(), good[:i] + [4098] + good[i + 1:]) == 3
    assert call(_dims(), good[:2] + [-8] + good[3:]) == 2 and call(_dims(), good[:2] + [12] + good[3:]) == 3
    assert call(_dims(total_tokens=0), [None] * 2 + [512, 512] + [None] * 3) == 0
    assert L.sink_attn_paged_append_e4m3(ctypes.byref(_dims()), P(4096), P(4096), 512, 512, P(4096), P(4096), P(4096),
                                         None, P(4096), None) == 1


def test_binding_refuses_host_tensors_and_wrong_types(L):
    kc = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        ops.paged_attn(q, kc, kc, i.view(1, 2), i, i[:1], torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA"):
        ops.paged_append(q[:, :2], q[:, :2], i, kc, kc)
    with pytest.raises(ValueError, match="bfloat16"):
        ops.paged_append(q[:, :2], q[:, :2], i, kc.float(), kc)
