"""sink_attn_paged_attn over sizes, strides and schedules: drawn batches of
every kind, units that are cut (with parts that hold no key), CTAs that take
several turns, a workspace of any content, defaults and refusals."""
import ctypes
import random

import pytest
import torch

from sink_sliding_window_b200 import build, ops
from tests.paged_util import Paged


@pytest.fixture(scope="module")
def L():
    build.build()
    return ops.load()


KINDS = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])


@pytest.mark.gpu
@pytest.mark.parametrize("seed", range(24))
def test_drawn_batches(seed):
    rng = random.Random(seed)
    hq, hkv = rng.choice([(64, 8), (16, 2), (8, 8), (4, 1), (40, 8), (24, 8), (32, 2), (12, 3), (10, 5), (20, 10), (72, 12)])
    batch = rng.choice([1, 2, 3, 7, 20])
    kind = rng.choice(["one", "few", "chunk", "mixed"])
    kv, new = [], []
    for _ in range(batch):
        n = rng.choice([1, rng.randint(1, 40), rng.randint(1, 300), rng.randint(1, 700)])
        m = {"one": 1, "few": rng.randint(1, 5), "chunk": rng.randint(1, 200),
             "mixed": rng.choice([0, 1, 1, 2, rng.randint(1, 90)])}[kind]
        kv.append(n)
        new.append(min(m, n))
    if not any(new):
        new[0] = 1
    p = Paged(kv, new, hq, hkv, rng.choice([16, 32, 64, 128, 1024]), rng.choice([0, 0, 1, 17, 100, 128, 500]),
              rng.random() < 0.5, seed=seed, layout=rng.choice(["token", "head", "fused"]), pad_rows=rng.choice([0, 3]))
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("window", [0, 100])
def test_more_units_than_ctas(e4m3, window):
    """A unit of 2 (e4m3: 4) tokens and far more of them than CTAs run at
    once: CTAs take up to four turns."""
    p = Paged([700, 100, 350, 611], [700, 100, 300, 33], 256, 2, 32, window, e4m3, seed=1)
    p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_parts_without_keys(e4m3):
    """Few units over a long context are cut into more parts than the short
    requests beside them have key tiles."""
    for kv, new in (([9000, 70, 300], [40, 40, 33]), ([5000, 65], [70, 65]), ([12000], [9])):
        p = Paged(kv, new, 8, 1, 64, 0, e4m3, seed=2)
        p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("heads", [(64, 2), (64, 1), (48, 1), (96, 2), (24, 3), (128, 2)])
def test_several_warps_a_head(e4m3, heads):
    """17 to 64 query rows a head, whole and cut, over a window too."""
    for kv, new, window in (([70, 3000, 33], [1, 1, 1], 0), ([500, 90], [1, 1], 64)):
        p = Paged(kv, new, *heads, 16, window, e4m3, seed=sum(heads))
        p.check(*p.run(ops))


@pytest.mark.gpu
@KINDS
def test_workspace_of_any_content(e4m3):
    """Nothing is expected of the workspace, and one call's content is no
    matter to the next."""
    calls = [Paged([5000, 300], [1, 1], 8, 1, 16, 0, e4m3, seed=3), Paged([4000, 64, 900], [60, 1, 1], 8, 1, 16, 0, e4m3, seed=4)]
    ws = torch.full((200 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
    for p in calls + calls[::-1]:
        p.check(*p.run(ops, workspace=ws))


@pytest.mark.gpu
@KINDS
def test_default_max_new_and_padding(e4m3):
    """max_new left out: a decode step with padded rows goes through both kernels."""
    p = Paged([900, 20, 333], [1, 1, 1], 16, 2, 16, 0, e4m3, seed=5, pad_rows=40)
    a = p.device()
    out, lse = ops.paged_attn(a["q"], a["k_cache"], a["v_cache"], a["block_table"], a["cu_seqlens"], a["kv_lens"],
                              a["sinks"], k_scale=a["k_scale"], v_scale=a["v_scale"])
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    p.check(out, lse)


@pytest.mark.gpu
@KINDS
def test_strides_of_single_elements(e4m3):
    """One token, one key/value head, one page: their strides mean nothing."""
    p = Paged([40], [1], 4, 1, 64, 0, e4m3, seed=6, extra_pages=0)
    a = p.device()
    odd = lambda t: t.as_strided(t.shape, (3,) + t.stride()[1:2] + (5, 1))  # noqa: E731
    q = a["q"].as_strided(a["q"].shape, (7, 64, 1))
    out, lse = ops.paged_attn(q, odd(a["k_cache"]), a["v_cache"], a["block_table"], a["cu_seqlens"], a["kv_lens"],
                              a["sinks"], k_scale=a["k_scale"], v_scale=a["v_scale"])
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    p.check(out, lse)


@pytest.mark.gpu
@KINDS
@pytest.mark.parametrize("new", [[1, 1], [50, 3]])
def test_windows_beyond_all_positions(e4m3, new):
    p = Paged([300, 200], new, 8, 2, 16, 0, e4m3, seed=7)
    a = p.device()
    for window in (300, (1 << 31) - 1, -5):
        out, lse = ops.paged_attn(a["q"], a["k_cache"], a["v_cache"], a["block_table"], a["cu_seqlens"], a["kv_lens"],
                                  a["sinks"], window, k_scale=a["k_scale"], v_scale=a["v_scale"])
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        p.check(out, lse)


@pytest.mark.gpu
def test_two_graphs_with_a_workspace_each():
    """Captured calls replayed on two streams at once."""
    ps = [Paged([3000, 900], [1, 1], 16, 2, 16, 0, seed=8), Paged([1500, 900], [200, 1], 16, 2, 16, 0, seed=9)]
    graphs = []
    for p in ps:
        a = p.device()
        args = [a.pop(k) for k in ("q", "k_cache", "v_cache", "block_table", "cu_seqlens", "kv_lens", "sinks")]
        a.update(out=torch.zeros((p.T, 16, 64), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros((16, p.T), device="cuda"),
                 workspace=torch.empty(200 << 20, dtype=torch.uint8, device="cuda"))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            ops.paged_attn(*args, **a)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                ops.paged_attn(*args, **a)
        graphs.append((graph, stream, a, args))
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, _, _ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    for p, (_, _, a, _) in zip(ps, graphs):
        p.check(a["out"], a["lse"])


@pytest.mark.gpu
@KINDS
def test_rows_counted_twice_stay_inside(e4m3):
    """cu_seqlens that go back and forth make far more units than T rows can:
    recorded, and nothing outside of the call's tensors is written."""
    p = Paged([4000] * 8, [8] * 8, 8, 1, 64, 0, e4m3, seed=11, pad_rows=5)
    a = p.device()
    n = 64
    cu = torch.tensor([0, p.T] * (n // 2) + [0], dtype=torch.int32, device="cuda")
    lens = torch.full((n,), 4000, dtype=torch.int32, device="cuda")
    table = a["block_table"].repeat(n // 8, 1).contiguous()
    d = ops.PagedDims(n, p.rows, p.rows, 8, 1, 64, 64, p.pages, p.max_pages, a["k_cache"].stride(0), a["k_cache"].stride(1),
                      64, a["q"].stride(0))
    need = ops.load().sink_attn_paged_workspace_size(ctypes.byref(d))
    ws = torch.full((need + (8 << 20),), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((p.rows + 64, 8, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    for order in (cu, cu.flip(0).contiguous()):
        ops.paged_attn(a["q"], a["k_cache"], a["v_cache"], table, order, lens, a["sinks"], out=out[:p.rows],
                       k_scale=a["k_scale"], v_scale=a["v_scale"], workspace=ws[:need])
        torch.cuda.synchronize()
        assert ops.device_error() == 0x205
        assert (ws[need:] == 0x5A).all() and (out[p.rows:] == 7).all()


@pytest.mark.gpu
def test_empty_step_and_empty_batch():
    p = Paged([40, 3], [1, 1], 4, 1, 16, 0, seed=10)
    a = p.device()
    out, lse = ops.paged_attn(a["q"][:0], a["k_cache"], a["v_cache"], a["block_table"], a["cu_seqlens"] * 0, a["kv_lens"],
                              a["sinks"])
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    out, lse = ops.paged_attn(a["q"], a["k_cache"], a["v_cache"], a["block_table"][:0], a["cu_seqlens"][:1],
                              a["kv_lens"][:0], a["sinks"])
    assert out.shape == (2, 4, 64) and ops.device_error() == 0


# ---------------------------------------------------------- refusals (CPU)
@pytest.mark.parametrize("bad,code", [
    (dict(page_stride=0), 2), (dict(token_stride=56), 2), (dict(head_stride=0), 2), (dict(page_stride=1 << 38), 4),
    (dict(q_stride=0), 2), (dict(q_stride=504), 2), (dict(q_stride=1 << 38), 4), (dict(batch=4097), 4),
    (dict(batch=4096, max_pages=1 << 20), 4), (dict(total_tokens=1 << 29, max_new=1 << 29), 4),
])
def test_attn_rejects_strides_and_batches(L, bad, code):
    d = dict(batch=2, total_tokens=4, max_new=2, num_q_heads=8, num_kv_heads=2, head_dim=64, page_size=16, num_pages=9,
             max_pages=4, page_stride=2048, token_stride=128, head_stride=64, q_stride=512)
    d.update(bad)
    P = ctypes.c_void_p
    a = [P(4096)] * 6
    assert L.sink_attn_paged_attn(ctypes.byref(ops.PagedDims(**d)), *a, P(4096), 0, 0.125, P(4096), P(4096), P(4096),
                                  1 << 40, None) == code


def test_workspace_size_covers_every_split(L):
    """It grows with nothing but the kind of work, and is never 0 for valid sizes."""
    d = dict(batch=3, total_tokens=4, max_new=1, num_q_heads=8, num_kv_heads=1, head_dim=64, page_size=16, num_pages=9,
             max_pages=4, page_stride=1024, token_stride=64, head_stride=64, q_stride=512)
    size = lambda **kw: L.sink_attn_paged_workspace_size(ctypes.byref(ops.PagedDims(**{**d, **kw})))  # noqa: E731
    assert 0 < size() <= size(max_new=4) <= size(max_new=4, total_tokens=4000, max_pages=4096)
    assert size(total_tokens=1 << 20, max_new=1 << 20, max_pages=1 << 16, batch=64) < 400 << 20
