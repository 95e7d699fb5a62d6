"""Plain forms and fixtures of the paged-cache tests: a step planned request
by request, a pool with pages in random order whose unowned slots hold NaN,
and the attention definition in 64 bits."""
import math

import numpy as np
import torch

NAN_CODE = 0x7F  # e4m3 NaN


def plan(cached, new, table, ring, pool, page, max_tokens, window=0, first=None):
    """The planning step by hand, on Python lists.  Returns the same seven
    results the call gives: cu, kv, slots, table, ring, pool, first."""
    table, ring = [list(r) for r in table], list(ring)
    size, (head, count) = len(ring), pool
    old = [list(r) for r in table]
    free = [ring[(head + i) % size] for i in range(count)]
    cu, kv, slots, first_out, back = [0], [], [], [], []
    used = asked = 0
    for b, (c, n) in enumerate(zip(cached, new)):
        held = -(-c // page)
        low = min(first[b], held) if first is not None else 0
        if n < 0:
            back += old[b][low:held]
            cu.append(cu[-1]), kv.append(0), first_out.append(0)
            continue
        fine = c + n <= len(table[b]) * page
        drop = max(low, max(0, c - window + 1) // page) if window > 0 and fine else low
        back += old[b][low:drop]
        first_out.append(drop)
        cu.append(cu[-1] + n)
        need = -(-(c + n) // page) - held if fine else 0
        asked += need
        ok = fine and (need == 0 or asked <= count)
        if ok:
            for j in range(held, held + need):
                table[b][j] = free[used]
                used += 1
        kv.append(c + n if ok else c)
        slots += [table[b][p // page] * page + p % page if ok else -1 for p in range(c, c + n)]
    slots = (slots + [-1] * max_tokens)[:max_tokens]
    for i, p in enumerate(back):
        ring[(head + count + i) % size] = p
    return cu, kv, slots, table, ring, [(head + used) % size, count - used + len(back)], first_out


def quantise(x, scale):
    """bf16 [..., H, 64] -> (e4m3 codes as uint8, the fp64 values they stand for)."""
    y = (x.float() * (1.0 / scale)[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return y.view(torch.uint8), y.double() * scale.double()[:, None]


class Paged:
    """Requests with kv[b] tokens of which the last new[b] are new, laid out
    on pages.  CPU tensors; device() gives the call's arguments.

    layout: "token" ([page][token][head]), "head" ([page][head][token]) or
    "fused" (keys and values of a page beside one another)."""

    def __init__(self, kv, new, hq, hkv, page, window=0, e4m3=False, seed=0, layout="token", stale=float("nan"),
                 std=1.0, sinks=None, drop=True, pad_rows=0, extra_pages=2):
        gen = torch.Generator().manual_seed(seed)
        self.kv, self.new, self.hq, self.hkv, self.page, self.window = list(kv), list(new), hq, hkv, page, window
        self.e4m3, self.layout = e4m3, layout
        B, T = len(kv), sum(new)
        self.T, self.rows = T, T + pad_rows
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        rnd = lambda *s: (torch.randn(s, generator=gen) * std).to(torch.bfloat16)  # noqa: E731
        self.q = rnd(self.rows, hq, 64)
        self.k = [rnd(n, hkv, 64) for n in kv]
        self.v = [rnd(n, hkv, 64) for n in kv]
        self.sinks = torch.randn((hq,), generator=gen) if sinks is None else torch.as_tensor(sinks, dtype=torch.float32)
        self.k_scale = torch.rand((hkv,), generator=gen) * 0.004 + 0.008 if e4m3 else None
        self.v_scale = torch.rand((hkv,), generator=gen) * 0.004 + 0.008 if e4m3 else None
        held = [-(-n // page) for n in kv]
        self.pages = sum(held) + extra_pages
        order = torch.randperm(self.pages, generator=gen).tolist()
        self.max_pages = max(held + [1]) + 1
        table = np.full((B, self.max_pages), -1, np.int32)
        kind = torch.uint8 if e4m3 else torch.bfloat16
        shape = {"token": (2, self.pages, page, hkv, 64), "head": (2, self.pages, hkv, page, 64),
                 "fused": (self.pages, 2, page, hkv, 64)}[layout]
        self.store = torch.full(shape, NAN_CODE if e4m3 else stale, dtype=kind)
        kc, vc = self.views(self.store)
        self.kd, self.vd = [], []
        at = 0
        for b, n in enumerate(kv):
            ids = order[at:at + held[b]]
            at += held[b]
            # With a window, pages that no new query can see may be gone.
            gone = max(0, n - new[b] - window + 1) // page if window > 0 and drop else 0
            table[b, :held[b]] = ids
            table[b, :gone] = -1
            for x, c, s, keep in ((self.k[b], kc, self.k_scale, self.kd), (self.v[b], vc, self.v_scale, self.vd)):
                codes, exact = quantise(x, s) if e4m3 else (x, x.double())
                keep.append(exact)
                for j in range(gone, held[b]):
                    part = codes[j * page:(j + 1) * page]
                    c[ids[j], :part.shape[0]] = part
        self.table = torch.from_numpy(table)

    def views(self, store):
        if self.layout == "fused":
            return store[:, 0], store[:, 1]
        if self.layout == "head":
            return store[0].transpose(1, 2), store[1].transpose(1, 2)
        return store[0], store[1]

    def device(self):
        kc, vc = self.views(self.store.cuda())
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        return dict(q=c(self.q), k_cache=kc, v_cache=vc, block_table=c(self.table),
                    cu_seqlens=torch.from_numpy(self.cu).cuda(),
                    kv_lens=torch.tensor(self.kv, dtype=torch.int32, device="cuda"), sinks=c(self.sinks),
                    window=self.window, max_new=max(self.new + [1]), k_scale=c(self.k_scale), v_scale=c(self.v_scale))

    def run(self, ops, **kw):
        a = self.device()
        out, lse = ops.paged_attn(a.pop("q"), a.pop("k_cache"), a.pop("v_cache"), a.pop("block_table"),
                                  a.pop("cu_seqlens"), a.pop("kv_lens"), a.pop("sinks"), **a, **kw)
        torch.cuda.synchronize()
        assert ops.device_error() == 0
        return out, lse

    def reference(self, scale=0.125):
        """out [T, Hq, 64], lse [Hq, T] in 64 bits, and for each the bound on
        the kernel's error.

        out: the weights p_j are rounded to 16 bits (half a step, 2^-8 of
        each) before they multiply the values, the result once more; the
        fp32 logits, exponentials and sums add less than 1/16 of that:
          2^-8 (|out| + sum_j pi_j |v_j|) * 17/16.
        Over e4m3 codes the weights are fp16, half a step of which is 2^-11 of
        each, or 2^-25 of the largest for those below fp16's range.  This
        bound allows them what bf16 weights have, and
          + 2^-21 max_j pi_j sum_j |v_j|;
        test_paged_rounding.py holds them to their own.
        lse: fp32 logits x (64 products of 16-bit numbers, |error| at most
        2^-18 of sum |q_d k_d| scale, the running maximum's rounding and
        ex2's 2^-22 with them): 2^-18 (1 + max_j sum_d |q_d k_d| scale)."""
        g_ = self.hq // self.hkv
        out, bo = torch.zeros((self.T, self.hq, 64), dtype=torch.float64), torch.zeros((self.T, self.hq, 64), dtype=torch.float64)
        lse, bl = torch.zeros((self.hq, self.T), dtype=torch.float64), torch.zeros((self.hq, self.T), dtype=torch.float64)
        for b, (n, m) in enumerate(zip(self.kv, self.new)):
            r = slice(int(self.cu[b]), int(self.cu[b + 1]))
            if m == 0:
                continue
            d = torch.arange(n - m, n)[:, None] - torch.arange(n)[None, :]
            seen = (d >= 0) & ((d < self.window) if self.window > 0 else True)
            for h in range(self.hq):
                k, v = self.kd[b][:, h // g_], self.vd[b][:, h // g_]
                q = self.q[r, h].double()
                x = torch.where(seen, q @ k.T * scale, -math.inf)
                s = self.sinks[h].double().expand(m, 1)
                full = torch.cat([x, s], 1)
                lse[h, r] = torch.logsumexp(full, 1)
                pi = torch.nan_to_num(torch.exp(full - lse[h, r][:, None]), nan=0.0)[:, :-1]
                out[r, h] = pi @ v
                a = pi @ v.abs()
                bo[r, h] = 2.0 ** -8 * 17 / 16 * (out[r, h].abs() + a)
                if self.e4m3 and n:
                    bo[r, h] += 2.0 ** -21 * pi.amax(1)[:, None] * (seen.double() @ v.abs())
                if n:
                    big = torch.where(seen, q.abs() @ k.abs().T * scale, 0.0).amax(1)
                    bl[h, r] = 2.0 ** -18 * (1 + big + s[:, 0].abs().nan_to_num(posinf=0.0))
                else:
                    bl[h, r] = 2.0 ** -18 * (1 + s[:, 0].abs().nan_to_num(posinf=0.0))
        return out, lse, bo, bl

    def check(self, out, lse, scale=0.125):
        ro, rl, bo, bl = self.reference(scale)
        o, l = out[:self.T].double().cpu(), lse[:, :self.T].double().cpu()
        assert torch.isfinite(o).all()
        assert torch.equal(torch.isfinite(l), torch.isfinite(rl))
        worst = ((o - ro).abs() / bo.clamp(min=1e-30)).max().item() if o.numel() else 0.0
        assert ((o - ro).abs() <= bo + 1e-30).all(), f"out: {worst:.2f} of the bound"
        fin = torch.isfinite(rl)
        e = torch.where(fin, (l - rl).abs(), 0.0)
        assert (e <= bl).all(), f"lse: error {e.max().item():.3e}, {(e / bl).max().item():.2f} of the bound"
        return worst
