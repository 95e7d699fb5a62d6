"""Paged attention at the largest batch, over pages that several requests
share, and called from several threads at once."""
import random
import threading

import pytest
import torch

from sink_sliding_window_b200 import build, ops
from tests.paged_util import Paged

pytestmark = pytest.mark.gpu
KINDS = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


@KINDS
@pytest.mark.parametrize("chunks", [False, True])
def test_4096_requests(e4m3, chunks):
    rng = random.Random(chunks)
    kv = [rng.choice([0, 1, 16, 17, rng.randint(1, 40)]) for _ in range(4096)]
    new = [min(n, rng.choice([0, 1, 1])) for n in kv]
    if chunks:
        for b in (0, 77, 2000, 4095):
            kv[b], new[b] = 300 + b % 7, 100 + b % 11
    p = Paged(kv, new, 2, 1, 16, 0, e4m3, seed=21)
    p.check(*p.run(ops))


def test_one_more_is_refused():
    p = Paged([1] * 4097, [1] * 4097, 1, 1, 16)
    a = p.device()
    with pytest.raises(ops.SinkAttnError, match="UNSUPPORTED"):
        ops.paged_attn(a["q"], a["k_cache"], a["v_cache"], a["block_table"], a["cu_seqlens"], a["kv_lens"], a["sinks"])


@KINDS
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 1, 3], [70, 90, 50]])
def test_requests_that_share_pages(e4m3, new):
    """A common prefix of 64 tokens in the same four pages of every request."""
    kv = [64 + n + 7 * i for i, n in enumerate(new)]
    p = Paged(kv, new, 8, 2, 16, 0, e4m3, seed=22)
    for b in (1, 2):
        p.table[b, :4] = p.table[0, :4]
        for x in (p.kd, p.vd):
            x[b][:64] = x[0][:64]
    p.check(*p.run(ops))


@KINDS
def test_two_threads_at_once(e4m3):
    """Each on a stream of its own; the interpreter is free during the calls."""
    ps = [Paged([900, 300], [1, 1], 16, 2, 16, 0, e4m3, seed=23), Paged([700, 300], [150, 1], 16, 2, 16, 0, e4m3, seed=24)]
    alone = [p.run(ops) for p in ps]
    args = [p.device() for p in ps]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        stream = torch.cuda.Stream()
        for _ in range(50):
            got[i].append(ops.paged_attn(**args[i], stream=stream))
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    for i in (0, 1):
        assert len(got[i]) == 50
        for o, l in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(l, alone[i][1])
