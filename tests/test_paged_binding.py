"""The native binding of the paged calls: numbers that do not fit, and tensors
that have a device but no memory, are refused with a Python exception before
the library is called.  CPU: tensors of a fake mode stand for CUDA ones."""
import subprocess
import sys

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from sink_sliding_window_b200 import build, ops


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def _fake():
    """The arguments of the three calls, on a device, without memory."""
    with FakeTensorMode():
        i = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
        h = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        plan = dict(cached_lens=i(2), new_lens=i(2), block_table=i(2, 4), free_pages=i(8), pool=i(2), page_size=16,
                    max_tokens=4, first_page=i(2))
        append = dict(k_new=h(4, 2, 64), v_new=h(4, 2, 64), slot_map=i(4), k_cache=h(8, 16, 2, 64), v_cache=h(8, 16, 2, 64))
        attn = dict(q=h(4, 8, 64), k_cache=h(8, 16, 2, 64), v_cache=h(8, 16, 2, 64), block_table=i(2, 4), cu_seqlens=i(3),
                    kv_lens=i(2), sinks=torch.empty(8, device="cuda"))
    return dict(paged_plan=plan, paged_append=append, paged_attn=attn)


BIG = [1 << 31, -(1 << 31) - 1, sys.maxsize, 1 << 80]


@pytest.mark.parametrize("value", BIG)
@pytest.mark.parametrize("call,name", [("paged_plan", "window"), ("paged_plan", "max_tokens"), ("paged_plan", "page_size"),
                                       ("paged_attn", "window"), ("paged_attn", "max_new")])
def test_numbers_beyond_32_bits_are_refused(call, name, value):
    with pytest.raises(ValueError, match="32 bits|whole number|negative"):
        getattr(ops, call)(**{**_fake()[call], name: value})


@pytest.mark.parametrize("call", ["paged_plan", "paged_append", "paged_attn"])
def test_tensors_without_memory_are_refused(call):
    with pytest.raises((RuntimeError, ValueError), match="data|storage|pointer"):
        getattr(ops, call)(**_fake()[call])


@pytest.mark.gpu
@pytest.mark.parametrize("value", BIG)
def test_a_planned_window_beyond_32_bits_raises(value):
    """In a process of its own: a call that ends the process fails the test, not the run."""
    code = f"""
import torch
from sink_sliding_window_b200 import ops
t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
args = (t([3, 4]), t([1, 1]), t([[0, -1], [1, -1]]), t([2, 3, -1, -1]), t([0, 2]), 16, 2)
try:
    ops.paged_plan(*args, window={value}, first_page=t([0, 0]))
except ValueError as e:
    print("refused:", e)
cu = ops.paged_plan(*args, window=(1 << 31) - 1, first_page=t([0, 0]))[0]
print("then:", cu.tolist(), ops.device_error())
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "refused:" in r.stdout and "then: [0, 1, 2] 0" in r.stdout


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch):
    """Neither found up to date nor loaded: the file names what it is for."""
    here = build.binding_path()
    assert torch.__version__ in here and sys.implementation.cache_tag in here
    assert ops._paged_calls().__file__ == here
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    monkeypatch.setattr(ops, "_paged", None)
    assert build.binding_path() != here
    with pytest.raises(RuntimeError, match="torch-0.0.1"):
        ops._paged_calls()


def test_the_library_is_built_without_torch():
    """As before there was a binding: torch is not needed for libsinkattn.so."""
    code = ("import sys; sys.modules['torch'] = None\n"
            "from sink_sliding_window_b200 import build\n"
            "build._newer = lambda target, sources: target == build.LIB\n"  # no binding is up to date
            "import os; print(os.path.exists(build.build()))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "True", r.stderr[-2000:]
