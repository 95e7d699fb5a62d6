"""Planning steps in which a request is refused: the requests behind it get
the rows, slots and pages that they would have had, whatever it asked for."""
import pytest
import torch

from sink_sliding_window_b200 import build, ops
from tests.paged_util import plan

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def _t(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(cached, new, table, ring, pool, page, max_tokens, window=0, first=None):
    tb, rg = _t(table), _t(ring)
    cu, kv, slots, pool_out, first_out = ops.paged_plan(_t(cached), _t(new), tb, rg, _t(pool), page, max_tokens, window,
                                                        None if first is None else _t(first))
    return dict(cu=cu.tolist(), kv=kv.tolist(), slots=slots.tolist(), table=tb.tolist(), ring=rg.tolist(),
                pool=pool_out.tolist(), first=None if first is None else first_out.tolist(), error=ops.device_error())


def _expect(got, want):
    for name, w in zip(("cu", "kv", "slots", "table", "ring", "pool"), want):
        assert got[name] == list(w), name


@pytest.mark.parametrize("behind", [1, 40, 1100])
@pytest.mark.parametrize("asked", [27, 28, 32, 33, 40, 3000])
def test_more_tokens_than_a_table_row_holds(asked, behind):
    """One request of 5 tokens in a row of 32 asks for too many, and others
    of 5 tokens stand in front of it and behind it."""
    page, B = 16, behind + 2
    cached = [5] * B
    new = [3, asked] + [3 + b % 9 for b in range(behind)]
    table = [[b, -1] for b in range(B)]
    ring = list(range(B, 2 * B)) + [-1] * B
    tokens = sum(new)
    got = _run(cached, new, table, ring, [0, B], page, tokens)
    _expect(got, plan(cached, new, table, ring, [0, B], page, tokens))
    assert got["cu"][1:3] == [3, 3 + asked] and got["error"] == (0x204 if asked > 27 else 0)
    assert (got["slots"][3:3 + asked] == [-1] * asked) == (asked > 27)
    assert min(got["slots"][3 + asked:]) >= 0


def test_rows_behind_an_overlong_request_reach_their_own_pages():
    """Planned, appended and attended to: the healthy request's keys are its
    own rows, and its output is what it is alone."""
    page, hq, hkv = 16, 8, 2
    gen = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, sinks = rnd(43, hq + 2 * hkv, 64), torch.zeros(hq, device="cuda")
    cache = [rnd(6, page, hkv, 64) for _ in range(2)]
    table, ring = _t([[-1, -1], [4, -1]]), _t([0, 1, 2, 3, 5, -1])
    before = [c.clone() for c in cache]
    cu, kv, slots, _, _ = ops.paged_plan(_t([0, 5]), _t([40, 3]), table, ring, _t([0, 5]), page, 43)
    ops.paged_append(x[:, hq:hq + hkv], x[:, hq + hkv:], slots, *cache)
    out, _ = ops.paged_attn(x[:, :hq], *cache, table, cu, kv, sinks, max_new=40)
    assert ops.device_error() == 0x204
    assert kv.tolist() == [0, 8]
    for c, b, at in zip(cache, before, (hq, hq + hkv)):
        b[4, 5:8] = x[40:, at:at + hkv]
        assert torch.equal(c, b)
    alone, _ = ops.paged_attn(x[40:, :hq], *cache, table[1:], _t([0, 3]), kv[1:], sinks, max_new=40)
    assert ops.device_error() == 0 and torch.equal(out[40:], alone)


MOST = (1 << 31) - 1


@pytest.mark.parametrize("huge", [1 << 20, 1 << 30, MOST])
def test_sums_of_tokens_end_at_31_bits(huge):
    """Requests that ask for as many tokens as the type holds, at several
    places: nobody's rows wrap around to the front."""
    page, B = 16, 2500
    cached, new = [5] * B, [2] * B
    for b in (700, 701, 1800, 2499):
        new[b] = huge
    table = [[b] for b in range(B)]
    got = _run(cached, new, table, [-1] * B, [0, 0], page, 4000)
    cu = [0]
    for n in new:
        cu.append(min(cu[-1] + n, MOST))
    assert got["cu"] == cu and got["error"] == 0x204
    assert got["kv"] == [5 if n == huge else 7 for n in new]
    assert got["slots"] == [b * page + 5 + i for b in range(700) for i in range(2)] + [-1] * 2600
    assert got["table"] == table and got["pool"] == [0, 0]


@pytest.mark.parametrize("max_tokens", [0, 1, 30, 100, 2000])
def test_pages_of_tokens_behind_the_slot_map(max_tokens):
    """A step with more tokens than the slot map: the lengths count them, so
    the table holds their pages."""
    page, B = 16, 60
    cached, new = [(7 * b) % 33 for b in range(B)], [(11 * b) % 70 for b in range(B)]
    held = [-(-c // page) for c in cached]
    ids = list(range(sum(held)))
    table = [[ids.pop() for _ in range(h)] + [-1] * (7 - h) for h in held]
    N = sum(held) + 300
    ring = list(range(sum(held), N)) + [-1] * sum(held)
    got = _run(cached, new, table, ring, [0, 300], page, max_tokens)
    _expect(got, plan(cached, new, table, ring, [0, 300], page, max_tokens))
    assert got["error"] == (0x204 if sum(new) > max_tokens else 0)


@pytest.mark.parametrize("window,gone", [(1, 4), (16, 3), (17, 3), (18, 2), (40, 1), (48, 1), (49, 1), (50, 0), (200, 0)])
@pytest.mark.parametrize("first", [0, 2])
def test_a_full_row_gives_back_what_its_window_leaves(window, gone, first):
    """A request whose row of 64 tokens is full and that asks for one more is
    refused, and gives back the pages wholly before its window all the same
    (position 64 - window + 1 is the first that anyone sees)."""
    page = 16
    table = [[0, 1, 2, 3], [4, 5, -1, -1]]
    for b in range(first):
        table[0][b] = -1
    back = list(range(first, max(first, gone)))
    other = 1 if window == 1 else 0  # the other request's first page, which it gave back before
    got = _run([64, 17], [1, 20], table, [6, 7] + [-1] * 6, [0, 2], page, 21, window, [first, other])
    assert got["error"] == 0x204 and got["kv"] == [64, 37] and got["cu"] == [0, 1, 21]
    assert got["slots"][:2] == [-1, 5 * page + 1]
    assert got["first"] == [max(first, gone), other]
    assert got["table"] == [table[0], [4, 5, 6, -1]]
    assert got["ring"] == [6, 7] + back + [-1] * (6 - len(back))
    assert got["pool"] == [1, 1 + len(back)]
