"""The few-rows kernel beside the chunk kernel starts without waiting for the
kernels before the call: it reads the call's inputs through L2 only (a test of
the source, CPU), and sees what those kernels wrote just before (GPU)."""
import os
import re

import pytest
import torch

from sink_sliding_window_b200 import build, ops
from tests.paged_util import Paged

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sink_sliding_window_b200", "csrc")
INPUTS = ("q", "k_scale", "v_scale", "table", "cu", "kv_lens", "sinks")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name,load", [("paged_attn.cuh", "paged_load<kL2>("), ("paged_rows.cuh", "paged_load<kBeside>(")])
def test_inputs_are_read_through_l2(name, load):
    code = _code(name)
    for field in INPUTS:
        for m in re.finditer(rf"\bp\.{field}\b(?!\s*=[^=])", code):
            before = code[:m.start()]
            line = before[before.rfind(";") + 1:] + code[m.start():code.index(";", m.start())]
            # Either loaded by paged_load or made into an address that is (q's rows).
            assert load in before[before.rfind(";") + 1:] or "src =" in line, line.strip()
            assert f"p.{field}[" not in line and not re.search(rf"(?<![\w)])\*\s*\(?p\.{field}\b", line), line.strip()
    for m in re.finditer(r"\bsrc \+ 16", code):  # and nothing but paged_load follows such an address
        assert load in code[code[:m.start()].rfind("=") + 1:m.start()]


def test_the_kernel_asks_for_it_everywhere():
    code = _code("paged_rows.cuh")
    calls = re.findall(r"\b(paged_(?:request|check|entry|load))(<\w+>)?\(", code)
    assert len(calls) >= 12 and all(t == "<kBeside>" for _, t in calls), calls
    body = _code("paged_attn.cuh")
    body = body[body.index("paged_load("):]
    assert "kL2 ? __ldcg(at)" in body[:body.index("}")]
    launch = _code("sink_attn.cu")
    assert "beside ? launch_rows<kF8, kR, true>" in launch


KINDS = pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])


@pytest.mark.gpu
@KINDS
def test_inputs_written_just_before_the_call(e4m3):
    """Steps of chunks and single tokens over the same buffers, which copies
    on the same stream fill again before every call: each gives, bit for bit,
    what it gives when nothing else is under way."""
    build.build()
    names = ("q", "k_cache", "v_cache", "block_table", "cu_seqlens", "kv_lens", "sinks", "k_scale", "v_scale")
    kv = [[900, 700, 40, 333, 1200, 64], [64, 1200, 700, 900, 333, 40], [333, 40, 900, 64, 700, 1200]]
    new = [[150, 1, 1, 2, 1, 1], [1, 1, 150, 1, 2, 1], [2, 1, 1, 1, 150, 1]]
    ps = [Paged(k, n, 16, 2, 16, 0, e4m3, seed=40 + i) for i, (k, n) in enumerate(zip(kv, new))]
    args = [p.device() for p in ps]
    want = []
    for p, a in zip(ps, args):
        out, lse = p.run(ops)
        p.check(out, lse)
        want.append((out, lse))
    buf = {n: None if args[0][n] is None else args[0][n].clone() for n in names}
    got = []
    for i in range(60):
        a = args[i % 3]
        for n in names:
            if buf[n] is not None:
                buf[n].copy_(a[n])
        got.append(ops.paged_attn(*(buf[n] for n in names[:7]), max_new=150, k_scale=buf["k_scale"], v_scale=buf["v_scale"]))
    torch.cuda.synchronize()
    assert ops.device_error() == 0
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 3][0]) and torch.equal(l, want[i % 3][1]), i
