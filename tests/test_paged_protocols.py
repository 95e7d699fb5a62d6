"""Models of the mbarrier protocols of the paged attention kernels (few rows;
chunks over bf16 and e4m3 pages), run under random interleavings (CPU only).

The same model of barriers, tensor-core queue and TMA completions as the other
kernels' (test_barrier_protocols.py).  Besides phases and deadlocks it checks
that no copy or widening writes a buffer that is still read, and that no MMA is
in flight when a chunk CTA goes on to its next round.  The models
follow the kernels' barrier use and are kept in step with them by hand."""
import random

import pytest

from tests.test_barrier_protocols import Bar, _run, _wait


class Buffer:
    """A stage: written by copies, read by threads or MMAs."""

    def __init__(self, name):
        self.name, self.readers, self.holds = name, 0, None

    def write(self, what):
        assert self.readers == 0, f"{self.name}: written while {self.holds} is read"
        self.holds = what

    def begin(self, what):
        assert self.holds == what, f"{self.name}: holds {self.holds}, {what} wanted"
        self.readers += 1

    def end(self):
        self.readers -= 1


def _steps(n, rng):
    for _ in range(rng.randrange(n + 1)):
        yield "step"


# --------------------------------------------------------------- few rows
def rows_model(counts, warps, stages, boxes, rng):
    """One CTA of the few-rows kernel: counts[g] blocks of worker g, `warps`
    warps a worker, copies of `boxes` boxes for K and as many for V."""
    groups = len(counts)
    full = [[Bar(("full", g, s), 1) for s in range(stages)] for g in range(groups)]
    empty = [[Bar(("empty", g, s), warps) for s in range(stages)] for g in range(groups)]
    buf = [[Buffer((g, s)) for s in range(stages)] for g in range(groups)]
    tma, done = [], []

    def copies():
        for i in range(max(counts)):
            s, turn = i % stages, i // stages
            for g in range(groups):
                if i >= counts[g]:
                    continue
                if turn > 0:
                    yield from _wait(empty[g][s], turn - 1)
                full[g][s].arrive(expect_tx=2 * boxes)
                buf[g][s].write(i)
                tma.extend([lambda g=g, s=s: full[g][s].complete_tx(1)] * (2 * boxes))
                yield "step"

    def attend(g, w):
        for i in range(counts[g]):
            s, turn = i % stages, i // stages
            yield from _wait(full[g][s], turn)
            buf[g][s].begin(i)
            yield from _steps(3, rng)
            buf[g][s].end()
            empty[g][s].arrive()
            yield "step"
        done.append((g, w))

    _run([copies()] + [attend(g, w) for g in range(groups) for w in range(warps)], [], tma, rng)
    assert len(done) == groups * warps


@pytest.mark.parametrize("counts", [[1], [2], [7], [3, 9], [0, 5, 4], [8, 8, 8, 8], [0, 0, 1]])
@pytest.mark.parametrize("stages", [3, 6])
def test_rows_protocol(counts, stages):
    for seed in range(15):
        rng = random.Random(seed)
        rows_model(counts, rng.choice([1, 2, 3, 8]), stages, rng.choice([1, 2, 4]), rng)


# ----------------------------------------------------------------- chunks
def chunk_model(codes, tiles, rounds, rng):
    """A chunk CTA over several rounds (n_half 64-key steps, `live` of its `tiles`
    query tiles hold tokens); codes: e4m3, with a copying and two widening
    warps.  The barriers' phases run on from round to round."""
    bars = {}
    state = dict(bars=bars, ring=0, q=0, s=[0] * tiles, copied=0)
    for i, (n_half, live) in enumerate(rounds):
        following = (rounds[i + 1][0] + 1) // 2 if i + 1 < len(rounds) else 0
        _chunk_round(codes, tiles, live, n_half, rng, state, following)


def _chunk_round(codes, tiles, live, n_half, rng, state, following):
    n_tiles = (n_half + 1) // 2
    # The copying warp is ahead: it ends the round with the next one's first tiles.
    copy_to = state["ring"] + n_tiles + min(following, 1 if codes else 2)
    bars, ring, q0, s0 = state["bars"], state["ring"], state["q"], list(state["s"])
    # What the copying warp works out for the round: the ring's place and parities.
    state["ring"] += n_tiles
    state["q"] += n_half > 0
    for w in range(live):
        state["s"][w] += n_half

    def bar(name, count=1):
        return bars.setdefault(name, Bar(name, count))

    bar("q_full"), bar("q_conv", tiles), bar("o_full")
    for s in range(2):
        bar(("k_full", s), 2 if codes else 1), bar(("v_full", s), 2 if codes else 1), bar(("kv_empty", s))
    for s in range(4):
        bar(("codes_full", s)), bar(("codes_empty", s))
    for w in range(tiles):
        bar(("s_full", w)), bar(("p_full", w))
    if "buffers" not in state:
        state["buffers"] = [[Buffer((n, s)) for s in range(k)] for n, k in (("K", 2), ("V", 2), ("codes", 4), ("S", tiles))]
    k_buf, v_buf, c_buf, s_tmem = state["buffers"]
    tc, tma, ended = [], [], []

    def mma():
        if n_half == 0:
            ended.append("mma")
            return
        bar("q_full").arrive(expect_tx=tiles)
        tma.extend([lambda: bar("q_full").complete_tx(1)] * tiles)
        yield from _wait(bar("q_conv") if codes else bar("q_full"), q0)
        yield from _wait(bar(("k_full", ring % 2)), ring // 2)

        def qk(w, h):
            j = ring + h // 2
            k_buf[j % 2].begin(j)

            def run():
                k_buf[j % 2].end()
                s_tmem[w].write(("S", h))
            tc.append(run)
            tc.append(lambda: bar(("s_full", w)).arrive())

        for w in range(live):
            qk(w, 0)
        yield "step"
        for h in range(n_half):
            j, hn = ring + h // 2, h + 1
            jn = ring + hn // 2
            yield from _wait(bar(("v_full", j % 2)), j // 2)
            if hn < n_half:
                yield from _wait(bar(("k_full", jn % 2)), jn // 2)
            for w in range(live):
                yield from _wait(bar(("p_full", w)), s0[w] + h)
                v_buf[j % 2].begin(j)
                s_tmem[w].begin(("P", h))

                def pv(w=w, j=j):
                    v_buf[j % 2].end()
                    s_tmem[w].end()
                tc.append(pv)
                if hn < n_half:
                    qk(w, hn)
                yield "step"
            if h % 2 == 1 or h == n_half - 1:
                tc.append(lambda j=j: bar(("kv_empty", j % 2)).arrive())
        tc.append(lambda: bar("o_full").arrive())
        ended.append("mma")

    def copy_tiles():
        for j in range(state["copied"], copy_to):
            s = j % 2
            if j >= 2:
                yield from _wait(bar(("kv_empty", s)), j // 2 - 1)
            for buf, name in ((k_buf, "k_full"), (v_buf, "v_full")):
                bar((name, s)).arrive(expect_tx=2)
                buf[s].write(j)
                tma.extend([lambda name=name, s=s: bar((name, s)).complete_tx(1)] * 2)
                yield "step"
        ended.append("copy")

    def copy_codes():
        for q in range(4 * state["copied"], 4 * copy_to):
            s = q % 4
            if q >= 4:
                yield from _wait(bar(("codes_empty", s)), q // 4 - 1)
            bar(("codes_full", s)).arrive(expect_tx=1)
            c_buf[s].write(q)
            tma.append(lambda s=s: bar(("codes_full", s)).complete_tx(1))
            yield "step"
        ended.append("copy")

    def widen(which):
        for q in range(4 * ring + which, 4 * (ring + n_tiles), 2):
            j, e = q // 4, q % 4
            s = j % 2
            if e < 2 and j >= 2:
                yield from _wait(bar(("kv_empty", s)), j // 2 - 1)
            yield from _wait(bar(("codes_full", q % 4)), q // 4)
            c_buf[q % 4].begin(q)
            yield from _steps(2, rng)
            (k_buf if e < 2 else v_buf)[s].write(j)
            c_buf[q % 4].end()
            bar(("codes_empty", q % 4)).arrive()
            bar(("k_full" if e < 2 else "v_full", s)).arrive()
            yield "step"
        ended.append("widen")

    def softmax(w):
        if n_half == 0 or w >= live:
            if codes and n_half:
                bar("q_conv").arrive()
            ended.append("softmax")
            return
        if codes:
            yield from _wait(bar("q_full"), q0)
            bar("q_conv").arrive()
        for h in range(n_half):
            yield from _wait(bar(("s_full", w)), s0[w] + h)
            s_tmem[w].begin(("S", h))
            yield from _steps(3, rng)
            s_tmem[w].end()
            s_tmem[w].write(("P", h))
            if rng.random() < 0.2:  # a step with keys that nobody sees: rows of V are zeroed
                j = ring + h // 2
                yield from _wait(bar(("v_full", j % 2)), j // 2)
                assert v_buf[j % 2].holds == j
            bar(("p_full", w)).arrive()
            yield "step"
        yield from _wait(bar("o_full"), q0)
        ended.append("softmax")

    agents = [mma()] + [softmax(w) for w in range(tiles)]
    agents += [copy_codes(), widen(0), widen(1)] if codes else [copy_tiles()]

    def sync():  # the CTA's barrier at the end of a round: Q and TMEM change hands
        while len(ended) < len(agents) - 1:
            yield "blocked"
        assert not tc, "in flight at the end of a round"

    agents.append(sync())
    _run(agents, tc, tma, rng)
    state["copied"] = copy_to


@pytest.mark.parametrize("codes,tiles", [(False, 2), (True, 4)], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("n_half", [0, 1, 2, 3, 4, 5, 9, 12])
def test_chunk_protocol(codes, tiles, n_half):
    for seed in range(12):
        rng = random.Random(seed)
        chunk_model(codes, tiles, [(n_half, rng.randint(1, tiles))], rng)


@pytest.mark.parametrize("codes,tiles", [(False, 2), (True, 4)], ids=["bf16", "e4m3"])
def test_chunk_protocol_over_rounds(codes, tiles):
    for seed in range(30):
        rng = random.Random(seed)
        chunk_model(codes, tiles, [(rng.choice([0, 1, 2, 3, 3, 4, 5]), rng.randint(1, tiles)) for _ in range(7)], rng)


def test_model_sees_a_stage_freed_too_early():
    """A worker whose stages are freed by fewer warps than read them."""
    def broken(seed):
        rng = random.Random(seed)
        full, empty, buf = [Bar("f", 1) for _ in range(2)], [Bar("e", 1) for _ in range(2)], [Buffer(s) for s in range(2)]
        tma = []

        def copies():
            for i in range(12):
                if i >= 2:
                    yield from _wait(empty[i % 2], i // 2 - 1)
                full[i % 2].arrive(expect_tx=1)
                buf[i % 2].write(i)
                tma.append(lambda i=i: full[i % 2].complete_tx(1))
                yield "step"

        def attend(frees):
            for i in range(12):
                yield from _wait(full[i % 2], i // 2)
                buf[i % 2].begin(i)
                yield from _steps(3, rng)
                buf[i % 2].end()
                if frees:
                    empty[i % 2].arrive()
                yield "step"

        _run([copies(), attend(True), attend(False)], [], tma, rng)

    caught = 0
    for seed in range(20):
        try:
            broken(seed)
        except AssertionError:
            caught += 1
    assert caught > 0
