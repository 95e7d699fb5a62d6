"""Paged attention over e4m3 codes, held to the rounding that its kernels have:
softmax weights of 11 bits (fp16).  The bound tells them from weights of 8 bits
(bf16), which a plain form on the CPU shows.

With x the logits, M the largest visible one, pi_j the weights in 64 bits and
`out` their sum over the values, the kernels compute
  out' = bf16((sum_j w_j v_j) / l),  w_j = fp16(2^(x_j - m)),  l = sum_j 2^(x_j - m) + 2^(s - m)
with m a reference that is never above M (it is a maximum of keys met before,
and never the sink).  So, with fp32 sums and K = 2^-18 (1 + max_j sum_d |q_d k_jd| scale)
the error of a logit and of its exponential (64 products of 11- and 4-bit
numbers summed in fp32, the maximum's rounding, ex2's 2^-22):
  each weight: half a step of fp16, 2^-11 of it, or below 2^-14 half the
    smallest step, 2^-25 of 2^m and so of the largest weight;
  logits: K in the sum and K in l;
  sums over n keys, 16 a step, one rounding or truncation (2^-23) each, the
    same in l, and 32 more for rescaling, joining and the scales: (n / 8 + 32) 2^-23;
  the result's half step, 2^-8 of it.
    e = (2^-11 + 2 K + (n / 8 + 32) 2^-23) sum_j pi_j |v_j| + 2^-25 max_j pi_j sum_j |v_j|
    |out' - out| <= e + 2^-8 (|out| + e)."""
import math

import pytest
import torch

from sink_sliding_window_b200 import build, ops
from tests.paged_util import Paged


def reference(p, scale=0.125):
    """(out, bound) [T, Hq, 64] in 64 bits."""
    rows, bounds = [], []
    for b, (n, m) in enumerate(zip(p.kv, p.new)):
        q = p.q[int(p.cu[b]):int(p.cu[b + 1])].double()
        G = p.hq // p.hkv
        k, v = (x[b].repeat_interleave(G, 1) for x in (p.kd, p.vd))
        d = torch.arange(n - m, n)[:, None] - torch.arange(n)[None, :]
        seen = (d >= 0) & ((d < p.window) if p.window > 0 else True)
        x = torch.einsum("thd,jhd->htj", q, k) * scale
        x = torch.where(seen, x, -math.inf)
        s = p.sinks.double()[:, None, None].expand(-1, m, 1)
        pi = torch.softmax(torch.cat([x, s], 2), 2)[..., :-1]
        out = torch.einsum("htj,jhd->thd", pi, v)
        a = torch.einsum("htj,jhd->thd", pi, v.abs())
        every = torch.einsum("tj,jhd->thd", seen.double(), v.abs())
        big = torch.where(seen, torch.einsum("thd,jhd->htj", q.abs(), k.abs()) * scale, 0.0).amax(2)
        K = 2.0 ** -18 * (1 + big.T[..., None])
        e = (2.0 ** -11 + 2 * K + (n / 8 + 32) * 2.0 ** -23) * a + 2.0 ** -25 * pi.amax(2).T[..., None] * every
        rows.append(out)
        bounds.append(e + 2.0 ** -8 * (out.abs() + e))
    return torch.cat(rows), torch.cat(bounds)


def plain(p, kind, scale=0.125):
    """The same with weights rounded to `kind` (64-bit otherwise), and the result to bf16."""
    rows = []
    for b, (n, m) in enumerate(zip(p.kv, p.new)):
        q = p.q[int(p.cu[b]):int(p.cu[b + 1])].double()
        k, v = (x[b].repeat_interleave(p.hq // p.hkv, 1) for x in (p.kd, p.vd))
        d = torch.arange(n - m, n)[:, None] - torch.arange(n)[None, :]
        x = torch.einsum("thd,jhd->htj", q, k) * scale
        x = torch.where((d >= 0) & ((d < p.window) if p.window > 0 else True), x, -math.inf)
        top = x.amax(2, keepdim=True)
        w = torch.exp(x - top)
        total = w.sum(2, keepdim=True) + torch.exp(p.sinks.double()[:, None, None] - top)
        rows.append(torch.einsum("htj,jhd->thd", w.to(kind).double() / total, v).to(torch.bfloat16).double())
    return torch.cat(rows)


CASES = [  # kv, new, query heads, key/value heads, page, window, std
    ([1, 2, 3, 15, 17, 64, 65, 129, 300, 1000], [1] * 10, 16, 2, 16, 0, 1.0),
    ([5, 40, 129, 700], [1] * 4, 16, 2, 64, 100, 1.0),
    ([70, 3000, 33], [1, 1, 1], 64, 2, 16, 0, 1.0),
    ([129, 64, 200, 300], [2, 4, 5, 3], 8, 2, 16, 0, 1.0),
    ([1, 40, 128, 300, 513], [1, 40, 127, 200, 64], 8, 2, 16, 0, 1.0),
    ([1, 40, 128, 300, 513], [1, 40, 127, 200, 64], 8, 2, 16, 128, 1.0),
    ([900, 33, 257, 1200], [150, 1, 1, 2], 16, 2, 64, 0, 1.0),
    ([2500], [40], 8, 1, 64, 0, 1.0),
    ([1500, 700], [1, 1], 8, 1, 32, 0, 2.5),
    ([900], [100], 8, 1, 32, 0, 2.5),
]


def _id(c):
    return f"kv{max(c[0])}-n{max(c[1])}-g{c[2] // c[3]}-w{c[5]}-s{c[6]}"


def _paged(i):
    kv, new, hq, hkv, page, window, std = CASES[i]
    return Paged(kv, new, hq, hkv, page, window, True, seed=100 + i, std=std)


@pytest.mark.gpu
@pytest.mark.parametrize("i", range(len(CASES)), ids=lambda i: _id(CASES[i]))
def test_weights_of_eleven_bits(i):
    build.build()
    p = _paged(i)
    got, _ = p.run(ops)
    out, bound = reference(p)
    ratio = ((got[:p.T].double().cpu() - out).abs() / bound.clamp(min=1e-30)).max().item()
    print(f"{_id(CASES[i])}: {ratio:.3f} of the bound")
    assert ratio <= 1, f"{ratio:.2f} of the bound"


@pytest.mark.parametrize("i", [0, 3, 4, 8], ids=lambda i: _id(CASES[i]))
def test_the_bound_tells_eleven_bits_from_eight(i):
    p = _paged(i)
    out, bound = reference(p)
    assert ((plain(p, torch.float16) - out).abs() <= bound).all()
    assert ((plain(p, torch.bfloat16) - out).abs() > bound).any()
