"""A wait that ran out and what a call reports about its inputs are recorded
apart: neither hides the other, whichever came first."""
import pytest
import torch

from sink_sliding_window_b200 import build, ops

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    ops.device_error(), ops.device_error()


def _dry():
    """A planned step whose pool is empty (0x202)."""
    t = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ops.paged_plan(t([16]), t([1]), t([[0, -1]]), t([-1, -1]), t([0, 0]), 16, 1)


def _small_ring():
    """A decode ring smaller than its window (0x201)."""
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    ops.decode(h(1, 2, 8, 64), h(1, 2, 2, 64), h(1, 2, 2, 64), h(1, 64, 2, 64), h(1, 64, 2, 64),
               torch.tensor([200], dtype=torch.int32, device="cuda"), torch.zeros(8, device="cuda"), 64, max_seqlen=202)


@pytest.mark.parametrize("report,code", [(_dry, 0x202), (_small_ring, 0x201)])
def test_an_input_does_not_hide_a_wait(report, code):
    report()
    assert ops.selftest_wait(2_000_000)[1] == 0x107
    assert ops.device_error() == code
    assert ops.device_error() == 0


def test_a_wait_does_not_hide_an_input():
    out = torch.full((4,), -1, dtype=torch.int32, device="cuda")
    import ctypes
    assert ops.load().sink_attn_selftest_wait(2_000_000, ctypes.c_void_p(out.data_ptr()),
                                              ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    _dry()
    assert [ops.device_error() for _ in range(3)] == [0x107, 0x202, 0]


def test_the_first_of_each_kind_stays():
    _small_ring()
    _dry()
    assert [ops.device_error() for _ in range(2)] == [0x201, 0]
