"""A ragged batch over a paged cache, and its attention and append from their
definitions in 64 bits."""
from __future__ import annotations

import math
import random

import torch

from megatron_tensor_transformer_plan_b200 import tpl

D = 128
BASE = 500000.0


def plan_of(nq, nkv, t=1, rope=True, f32=False, layers=1, H=None, F=None):
    flags = tpl.TPL_NORM | tpl.TPL_RESIDUAL | (tpl.TPL_ROPE if rope else 0) | (tpl.TPL_FP32_WEIGHTS if f32 else 0)
    return tpl.Plan(tpl.make_dims(H or nq * D, nq, nkv, D, F or 2 * nq * D, layers, 1e-5, flags, BASE if rope else 0.0), t)


class Case:
    """kv_len: keys per sequence (this call's tokens included); news: tokens
    per sequence (None: one token each); shared: keys in common pages."""

    def __init__(self, dev, nq, nkv, t, page, kv_len, news=None, shared=0, dtype=torch.float32, seed=0, rows_before=0,
                 rows_behind=0, spare_entries=2, fill=None, q_scale=2.0):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rnd = random.Random(seed)
        self.nq, self.nkv, self.t, self.page, self.kv_len, self.shared, self.dev = nq, nkv, t, page, kv_len, shared, dev
        n = len(kv_len)
        entries = max(1, (max(kv_len) + page - 1) // page, shared // page) + spare_entries
        need = [(x + page - 1) // page for x in kv_len]
        pages = list(range(shared // page + sum(need) + 3))
        rnd.shuffle(pages)
        self.n_pages = len(pages)
        common = [pages.pop() for _ in range(shared // page)]
        # entries that hold no key name no page at all
        self.pages = [[common[e] if e < len(common) else pages.pop() if e < need[b] else 0x7ffffff0 for e in range(entries)]
                      for b in range(n)]
        wide = torch.full((n, entries + 3), -5, dtype=torch.int32)
        wide[:, :entries] = torch.tensor(self.pages, dtype=torch.int32)
        self.table = wide.to(dev)[:, :entries]
        self.lens = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        if news is None:
            self.news, self.start, self.q_start = [1] * n, list(range(n)), None
            self.tokens = n
        else:
            self.news, self.start, at = news, [], rows_before
            for x in news:
                self.start.append(at)
                at += x
            self.q_start = torch.tensor(self.start + [at], dtype=torch.int32, device=dev)
            self.tokens = at + rows_behind
        shape = (t, self.n_pages, nkv // t, page, D)

        def normal(s, dt, scale=1.0):
            return torch.empty(s, dtype=dt, device=dev).normal_(0.0, scale, generator=g)

        self.k, self.v = normal(shape, torch.bfloat16), normal(shape, torch.bfloat16)
        if fill is not None:  # everything that is no key of any sequence
            hole = torch.ones((self.n_pages, page), dtype=torch.bool, device=dev)
            for b, x in enumerate(kv_len):
                at = torch.arange(x, device=dev)
                hole[torch.tensor(self.pages[b], device=dev)[at // page], at % page] = False
            if shared:
                hole[torch.tensor(common, device=dev)] = False
            for pool in (self.k, self.v):
                pool.permute(1, 3, 0, 2, 4)[hole] = fill
        self.q = normal((self.tokens, nq, D), dtype, q_scale)

    def kv(self, plan):
        return plan.paged_kv(self.k, self.v)

    def batch(self, plan):
        return plan.paged_batch(self.table, self.lens, self.q_start, self.tokens)

    def rows(self):
        """(sequence, row of q, position) of every token."""
        for b, (x, new) in enumerate(zip(self.kv_len, self.news)):
            for i in range(new):
                yield b, self.start[b] + i, x - new + i

    def keys(self, b, pool):
        """The keys of sequence b: fp64 [kv_len][n_kv][128]."""
        at = torch.arange(self.kv_len[b], device=self.dev)
        x = pool[:, torch.tensor(self.pages[b], device=self.dev)[at // self.page], :, at % self.page]  # [len][t][nkv/t][d]
        return x.double().flatten(1, 2)

    def expected(self, window=0, sinks=0, q_bits=24, p_bits=24):
        """(o, lse, bound on o, bound on lse), from the definition in fp64.

        The bounds count the kernels' roundings.  With q kept to q_bits, a
        logit is off by E = sum|q k| / sqrt(d) * (2^-q_bits + 128 * 2^-24) (the
        second term: 128 fp32 additions).  A probability is then off by E and
        by its own rounding 2^-p_bits, and sums over n keys in fp32 by n *
        2^-24; o adds half a step of bf16, 2^-8 of its value."""
        o = torch.zeros((self.tokens, self.nq, D), dtype=torch.float64, device=self.dev)
        lse = torch.full((self.tokens, self.nq), -math.inf, dtype=torch.float64, device=self.dev)
        tol, ltol = torch.zeros_like(o), torch.zeros_like(lse)
        g = self.nq // self.nkv
        for b, new in enumerate(self.news):
            n = self.kv_len[b]
            if n == 0 or new == 0:
                continue
            K, V = self.keys(b, self.k), self.keys(b, self.v)
            rows = slice(self.start[b], self.start[b] + new)
            pos = torch.arange(n - new, n, device=self.dev)[:, None]
            key = torch.arange(n, device=self.dev)[None]
            seen = key <= pos
            if window:
                seen &= (key > pos - window) | (key < sinks)
            q = self.q[rows].double().unflatten(1, (self.nkv, g)).permute(1, 2, 0, 3)  # [nkv][g][new][d]
            Kt = K.permute(1, 2, 0)[:, None]
            hide = ~seen
            s = (q @ Kt / math.sqrt(D)).masked_fill(hide, -math.inf)
            top = s.amax(-1, keepdim=True)
            top = torch.where(top == -math.inf, torch.zeros_like(top), top)
            p = torch.exp(s - top)
            den = p.sum(-1, keepdim=True)
            some = den > 0
            p = torch.where(some, p / den.clamp_min(1e-300), torch.zeros_like(p))
            Vt = V.permute(1, 0, 2)[:, None]
            # hidden values may be anything: they have no part in the sums
            used = seen.any(0)
            Vt = torch.where(used[None, None, :, None], Vt, torch.zeros_like(Vt))
            Ka = torch.where(used[None, None, None], Kt, torch.zeros_like(Kt)).abs()
            E = (q.abs() @ Ka).masked_fill(hide, 0).amax(-1, keepdim=True) / math.sqrt(D)
            E = E * (2.0 ** -q_bits + 128 * 2.0 ** -24)
            out, mag = p @ Vt, p @ Vt.abs()
            rel = 2 * E + 2.0 ** -p_bits + (n + 64) * 2.0 ** -24 + 2.0 ** -20
            o[rows] = out.permute(2, 0, 1, 3).flatten(1, 2)
            tol[rows] = (2 * rel * mag + 2.0 ** -8 * out.abs() + 1e-30).permute(2, 0, 1, 3).flatten(1, 2)
            z = torch.where(some, top + den.clamp_min(1e-300).log(), torch.full_like(den, -math.inf))
            lse[rows] = z.squeeze(-1).permute(2, 0, 1).flatten(1, 2)
            lt = E + (n + 64) * 2.0 ** -24 + 2.0 ** -20 * (1 + torch.where(some, z, torch.zeros_like(z)).abs())
            ltol[rows] = lt.squeeze(-1).permute(2, 0, 1).flatten(1, 2)
        return o, lse, tol, ltol


def outputs(case, dtype=torch.bfloat16):
    o = torch.full((case.tokens, case.nq * D), float("nan"), dtype=dtype, device=case.dev)
    return o, torch.full((case.tokens, case.nq), float("nan"), dtype=torch.float32, device=case.dev)


def check(case, o, lse, window=0, sinks=0, q_bits=24, p_bits=24):
    """Every row of a sequence within its bound; the others as they were (NaN)."""
    ref, ref_lse, tol, ltol = case.expected(window, sinks, q_bits, p_bits)
    mine = torch.zeros(case.tokens, dtype=torch.bool, device=case.dev)
    for b, new in enumerate(case.news):
        mine[case.start[b]:case.start[b] + new] = True
    o = o.view(case.tokens, case.nq, D).double()
    assert torch.isnan(o[~mine]).all() and torch.isnan(lse[~mine]).all(), "a row of no sequence was written"
    bad = ~((o[mine] - ref[mine]).abs() <= tol[mine])
    assert not bad.any(), (f"{int(bad.sum())} of {bad.numel()} outputs off, first at {bad.nonzero()[0].tolist()}, worst "
                           f"{float(((o[mine] - ref[mine]).abs() / tol[mine]).nan_to_num(1e9).max()):.3g} bounds")
    want, got = ref_lse[mine], lse[mine].double()
    empty = want == -math.inf
    assert (got[empty] == -math.inf).all(), "an empty row's lse"
    assert ((got - want).abs()[~empty] <= ltol[mine][~empty]).all(), "lse"


def turned(x, pos, base=BASE):
    """RoFormer's rotation of x [..., 128] (fp64) by position, half-split pairs."""
    e = torch.arange(D // 2, dtype=torch.float64, device=x.device)
    ang = pos.double()[:, None, None] * base ** (-2.0 * e / D)
    a, b = x[..., :64], x[..., 64:]
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], dim=-1)
