"""What the paged-cache calls do at the edges of what a batch may hold."""
import math
import os
import subprocess
import sys

import pytest
import torch

from megatron_tensor_transformer_plan_b200 import tpl
from tests.paged_util import D, Case, check, outputs, plan_of
from tests.test_gpu_paged import PROMPT_P, TOKEN_Q, q_bits, run_attn, workspace

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def run_shared(plan, c, shared, ws=None):
    o, lse = outputs(c)
    plan.paged_attn_shared(c.kv(plan), c.batch(plan), shared, c.q, o, workspace(plan, c) if ws is None else ws, lse=lse)
    torch.cuda.synchronize()
    assert plan.last_device_error() == tpl.TPL_OK
    return o, lse


# ---- a prefix that no sequence fills ------------------------------------------

INSIDE = [
    # nq, nkv, t, page, shared, kv_len
    (8, 8, 1, 16, 48, [33]),
    (64, 8, 8, 64, 1024, [700, 650, 0, 3]),
    (40, 8, 2, 32, 992, [961] * 40),
    (32, 32, 2, 128, 1536, [1, 0, 2]),
    (16, 1, 1, 256, 512, [0, 0]),
    (4, 4, 1, 16, 4096, [130, 129]),       # whole tiles that nobody sees
    (24, 8, 1, 64, 1536, [1500] * 50),
    (16, 8, 2, 32, 1024, [10] * 33 + [801] + [5] * 3),
    (16, 8, 2, 32, 1024, [100] * 35 + [1030, 3]),   # (filled by one, the 36th)
]


@pytest.mark.parametrize("p", INSIDE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("stale", [NAN, INF])
def test_a_prefix_that_no_sequence_fills(gpu, p, dtype, stale):
    """Slots of the prefix behind the longest sequence hold anything, and the
    table names no page where nothing is seen."""
    nq, nkv, t, page, shared, kv_len = p
    plan = plan_of(nq, nkv, t)
    c = Case(gpu, nq, nkv, t, page, kv_len, shared=shared, dtype=dtype, seed=page)
    top = max(kv_len)
    for key in range(min(top, shared), shared):
        for pool in (c.k, c.v):
            pool[:, c.pages[0][key // page], :, key % page] = stale
    c.table[:, (top + page - 1) // page:] = -3
    o, lse = run_shared(plan, c, shared)
    check(c, o, lse, 0, 0, q_bits(c, False), PROMPT_P)


# ---- starts that are out of range ------------------------------------------------

STARTS = [
    # q_start with n_tokens = 60, the rows that some sequence validly has
    ([0, 50, 20, 60], [(0, 0, 20), (2, 20, 60)]),       # (rows 20 .. 49 lie in two sequences: either may lack them)
    ([70, 75], []),
    ([-5, -2], []),
    ([0, 10, 61, 62, 70], [(0, 0, 10)]),
    ([60, 65], []),
    ([-1, 10, 30], [(1, 10, 30)]),
    ([0, 10, 10, 5], [(0, 0, 10)]),
]


@pytest.mark.parametrize("p", STARTS)
def test_append_reports_starts_out_of_range(gpu, p):
    starts, valid = p
    plan = plan_of(16, 8, 2, rope=False)
    n, tokens, page = len(starts) - 1, 60, 16
    c = Case(gpu, 16, 8, 2, page, [100] * n, [0] * n, seed=2)
    q_start = torch.tensor(starts, dtype=torch.int32, device=gpu)
    batch = plan.paged_batch(c.table, c.lens, q_start, tokens)
    k, v = (torch.randn((tokens, 8, D), device=gpu) for _ in "kv")
    want = c.k.clone(), c.v.clone()
    loose = torch.zeros((c.n_pages, page), dtype=torch.bool, device=gpu)  # slots that may or may not be written
    for b, first, end in valid:
        for r in range(first, end):
            pos = 100 - starts[b + 1] + r
            for pool, x in zip(want, (k, v)):
                pool[:, c.pages[b][pos // page], :, pos % page] = x[r].to(torch.bfloat16).unflatten(0, (2, 4))
    for b in range(n):
        if 0 <= starts[b] <= starts[b + 1] <= tokens:
            for r in range(starts[b], starts[b + 1]):
                if sum(starts[x] <= r < starts[x + 1] <= tokens and starts[x] >= 0 for x in range(n)) > 1:
                    pos = 100 - starts[b + 1] + r
                    loose[c.pages[b][pos // page], pos % page] = True
    plan.paged_append(c.kv(plan), batch, k, v)
    assert plan.last_device_error() == tpl.TPL_EDEVICE
    for pool, w in zip((c.k, c.v), want):
        same = (pool == w).permute(1, 3, 0, 2, 4).flatten(2).all(-1)
        assert (same | loose).all()
    assert plan.last_device_error() == tpl.TPL_OK


# ---- logits beyond fp32 -----------------------------------------------------------

def overflowing(gpu, nq, nkv, kv_len, low, dtype, news=None, shared=0):
    """Every q is 2^66; the first `low` keys are -2^66 (their logits fall below
    fp32's range, a weight of 0), the others give logits of deviation 1."""
    c = Case(gpu, nq, nkv, 1, 64, kv_len, news, shared=shared, dtype=dtype, seed=3)
    c.q.fill_(2.0 ** 66)
    c.k.mul_(2.0 ** -66)
    for b, n in enumerate(kv_len):
        for key in range(min(low, n)):
            c.k[:, c.pages[b][key // 64], :, key % 64] = -2.0 ** 66
    return c


@pytest.mark.parametrize("kind", ["tokens", "prompts", "shared"])
@pytest.mark.parametrize("heads", [(16, 8), (32, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("low", [20, 64, 200])
def test_logits_below_the_range(gpu, kind, heads, dtype, low):
    """A key whose logit overflows to -inf has no weight; a token that sees
    only such keys gets what one that sees no key gets."""
    nq, nkv = heads
    kv_len = [300, 1300, 40, 150]
    news = [7, 30, 40, 1] if kind == "prompts" else None
    shared = 128 if kind == "shared" else 0
    if shared:
        kv_len = [300, 1300, 140, 129]
    plan = plan_of(nq, nkv, 1)
    c = overflowing(gpu, nq, nkv, kv_len, low, dtype, news, shared)
    o, lse = run_shared(plan, c, shared) if shared else run_attn(plan, c)
    o = o.view(-1, nq, D).double()
    g = nq // nkv
    for b, row, pos in c.rows():
        if pos < low:
            assert (o[row] == 0).all() and (lse[row] == -INF).all(), (b, pos)
            continue
        K, V = c.keys(b, c.k)[low:pos + 1], c.keys(b, c.v)[low:pos + 1]
        q = c.q[row].double().unflatten(0, (nkv, g))
        s = torch.einsum("jgd,kjd->jgk", q, K) / math.sqrt(D)
        p = torch.softmax(s, -1)
        ref, mag = torch.einsum("jgk,kjd->jgd", p, V).flatten(0, 1), torch.einsum("jgk,kjd->jgd", p, V.abs()).flatten(0, 1)
        # q is exact; a logit adds 128 products in fp32, a weight rounds to p_bits, the sums add in fp32
        E = torch.einsum("jgd,kjd->jgk", q.abs(), K.abs()).amax(-1).flatten()[:, None] / math.sqrt(D) * 128 * 2.0 ** -24
        n = pos + 1 - low
        p_bits = TOKEN_Q if kind == "tokens" else PROMPT_P
        rel = 2 * E + 2.0 ** -p_bits + (n + 64) * 2.0 ** -24 + 2.0 ** -20
        assert ((o[row] - ref).abs() <= 2 * rel * mag + 2.0 ** -8 * ref.abs()).all(), (b, pos)
        z = torch.logsumexp(s, -1).flatten()
        lt = E[:, 0] + (n + 64) * 2.0 ** -24 + 2.0 ** -20 * (1 + z.abs())
        assert ((lse[row].double() - z).abs() <= lt).all(), (b, pos)


# ---- keys that are no numbers -------------------------------------------------------

@pytest.mark.parametrize("kind", ["tokens", "prompts", "shared own", "shared prefix"])
def test_a_seen_key_that_is_no_number_is_seen(gpu, kind):
    """NaN among the keys that a token sees gives it NaN, also where all keys
    of one part of the work are NaN; other sequences do not notice."""
    news = [3, 2, 5] if kind == "prompts" else None
    shared = 1024 if kind.startswith("shared") else 0
    plan = plan_of(16, 8, 1)
    c = Case(gpu, 16, 8, 1, 64, [1025, 1100, 1025 + 64], news, shared=shared, seed=4)
    for key in range(1024, 1025) if kind == "shared own" else range(256, 512):
        c.k[:, c.pages[0][key // 64], :, key % 64] = NAN
    o, lse = run_shared(plan, c, shared) if shared else run_attn(plan, c)
    o = o.view(-1, 16, D)
    for b, row, _ in c.rows():
        hit = b == 0 or kind == "shared prefix"
        assert torch.isnan(o[row]).all() == hit and torch.isnan(lse[row]).all() == hit
        assert hit or (torch.isfinite(o[row]).all() and torch.isfinite(lse[row]).all())


# ---- calls that follow each other ---------------------------------------------------

def test_own_keys_appended_by_the_call_before(gpu):
    """Behind a shared prefix the kernel of the sequences' own keys starts under
    the prefix's; it has to see what an append just before wrote.  Step after step
    with other keys and queries, against the same steps one kernel at a time."""
    plan = plan_of(32, 8, 2)
    shared, own, steps = 256, 700, 40
    c = Case(gpu, 32, 8, 2, 64, [shared + own] * 4, shared=shared, seed=6)
    kv, batch, ws = c.kv(plan), c.batch(plan), workspace(plan, c)
    start = torch.arange(5, dtype=torch.int32, device=gpu) * own
    prompts = plan.paged_batch(c.table, c.lens, start, 4 * own)
    g = torch.Generator(device=gpu)
    g.manual_seed(1)
    k, v = (torch.randn((4, 4 * own, 8, D), generator=g, device=gpu) for _ in "kv")
    q = torch.randn((4, 4, 32, D), generator=g, device=gpu)

    def step(s, wait):
        o, lse = outputs(c)
        plan.paged_append(kv, prompts, k[s % 4], v[(s + s // 4) % 4])
        if wait:
            torch.cuda.synchronize()
        plan.paged_attn_shared(kv, batch, shared, q[(s + s // 7) % 4], o, ws, lse=lse)
        if wait:
            torch.cuda.synchronize()
        return o, lse

    got = [step(s, False) for s in range(steps)]
    for s in range(steps):
        o, lse = step(s, True)
        assert torch.equal(o, got[s][0]) and torch.equal(lse, got[s][1]), s
    assert plan.last_device_error() == tpl.TPL_OK


def test_first_calls_of_a_process_are_captured(gpu):
    """Append, tokens, prompts and a shared prefix, captured in a process that has
    launched none of them before."""
    code = """
import torch
from megatron_tensor_transformer_plan_b200 import tpl
from tests.paged_util import D, Case, check, outputs, plan_of
gpu = torch.device("cuda:0")
plan = plan_of(20, 4, 4, rope=False)
runs = []
for kind in ("tokens", "prompts", "shared"):
    c = Case(gpu, 20, 4, 4, 64, [700, 165, 130], [40, 3, 9] if kind == "prompts" else None,
             shared=128 if kind == "shared" else 0, seed=9)
    k, v = (torch.randn((c.tokens, 4, D), device=gpu) for _ in "kv")
    runs.append((kind, c, k, v, outputs(c), c.kv(plan), c.batch(plan), plan.paged_workspace(3, c.tokens)))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    for kind, c, k, v, (o, lse), kv, batch, ws in runs:
        plan.paged_append(kv, batch, k, v)
        if kind == "shared":
            plan.paged_attn_shared(kv, batch, 128, c.q, o, ws, lse=lse)
        else:
            plan.paged_attn(kv, batch, c.q, o, ws, lse=lse)
for _ in range(3):
    for r in runs:
        r[4][0].fill_(float("nan")), r[4][1].fill_(float("nan"))
    graph.replay()
    torch.cuda.synchronize()
    assert plan.last_device_error() == tpl.TPL_OK
    for kind, c, k, v, (o, lse), *_ in runs:
        check(c, o, lse, 0, 0, 16, 16 if kind == "tokens" else 8)
print("captured first: ok")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first: ok" in r.stdout, r.stdout + r.stderr


# ---- plans with fp32 outputs ----------------------------------------------------------

def test_fp32_outputs_are_closer_than_bf16(gpu):
    """Few keys and small queries, so that the bound is far below a bf16 step."""
    plan = plan_of(24, 8, 2, f32=True)
    c = Case(gpu, 24, 8, 2, 32, [7, 1, 3, 30, 0], seed=5, q_scale=0.1)
    o, lse = run_attn(plan, c, dtype=torch.float32)
    ref, ref_lse, tol, ltol = c.expected(0, 0, TOKEN_Q, TOKEN_Q)
    tol = tol - 2.0 ** -8 * ref.abs() + 2.0 ** -24 * ref.abs()  # fp32 in place of bf16 outputs
    live = slice(0, 4)
    o = o.view(5, 24, D).double()
    assert ((o - ref).abs() <= tol).all()
    assert ((lse.double() - ref_lse).abs()[live] <= ltol[live]).all() and (lse[4] == -INF).all()
    rounded = ref.to(torch.bfloat16).double()
    assert ((rounded - ref).abs() > tol)[live].double().mean() > 0.5  # (bf16 outputs would not pass)


# ---- numbers outside their range: the others' results -----------------------------------

@pytest.mark.parametrize("kind, bad", [(kind, bad) for kind in ("tokens", "prompts", "shared")
                                       for bad in ("page", "page below", "length", "length below")] + [("prompts", "start")])
def test_the_other_sequences_of_a_bad_one(gpu, kind, bad):
    """Every other sequence is right, and an append writes its slots and no others."""
    news = [5, 6, 7] if kind == "prompts" else None
    shared = 64 if kind == "shared" else 0
    plan = plan_of(32, 8, 2, rope=False)
    c = Case(gpu, 32, 8, 2, 64, [300, 400, 500], news, shared=shared, seed=1)
    wrong = 1
    if bad.startswith("page"):
        c.table[1, 6] = -1 if bad == "page below" else c.n_pages
    elif bad.startswith("length"):
        c.lens[1] = -9 if bad == "length below" else c.table.shape[1] * 64 + 1
    else:
        c.q_start[3], wrong = c.tokens + 1, 2
    o, lse = outputs(c)
    kv, batch, ws = c.kv(plan), c.batch(plan), workspace(plan, c)
    if kind == "shared":
        plan.paged_attn_shared(kv, batch, shared, c.q, o, ws, lse=lse)
    else:
        plan.paged_attn(kv, batch, c.q, o, ws, lse=lse)
    assert plan.last_device_error() == tpl.TPL_EDEVICE
    ref, ref_lse, tol, ltol = c.expected(0, 0, TOKEN_Q, TOKEN_Q if kind == "tokens" else PROMPT_P)
    rows = [r for b, r, _ in c.rows() if b != wrong]
    assert ((o.view(-1, 32, D).double() - ref).abs() <= tol)[rows].all()
    assert ((lse.double() - ref_lse).abs() <= ltol)[rows].all()
    k, v = (torch.randn((c.tokens, 8, D), device=gpu) for _ in "kv")
    want = c.k.clone(), c.v.clone()
    for b, r, pos in c.rows():
        if b != wrong:
            for pool, x in zip(want, (k, v)):
                pool[:, c.pages[b][pos // 64], :, pos % 64] = x[r].to(torch.bfloat16).unflatten(0, (2, 4))
    plan.paged_append(kv, batch, k, v)
    assert plan.last_device_error() == tpl.TPL_EDEVICE
    assert torch.equal(c.k, want[0]) and torch.equal(c.v, want[1])
    assert plan.last_device_error() == tpl.TPL_OK


# ---- padding and full tables --------------------------------------------------------------

@pytest.mark.parametrize("kind", ["tokens", "prompts", "shared"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_padded_rows_hold_anything(gpu, kind, dtype):
    """Queries of inactive tokens and of rows that no sequence has may be NaN; the
    longest sequence fills its row of the table to the last slot."""
    news = [200, 5, 3, 4] if kind == "prompts" else None
    shared = 128 if kind == "shared" else 0
    plan = plan_of(16, 8, 2)
    c = Case(gpu, 16, 8, 2, 32, [150, 0, 512, 3], news, shared=shared, dtype=dtype, seed=8, spare_entries=0,
             rows_before=2 if news else 0, rows_behind=70 if news else 0, fill=NAN)
    assert c.table.shape[1] * 32 == 512
    idle = torch.ones(c.tokens, dtype=torch.bool, device=gpu)
    idle[[r for _, r, pos in c.rows() if pos >= 0]] = False
    q = c.q.clone()
    c.q[idle] = NAN
    o, lse = run_shared(plan, c, shared) if shared else run_attn(plan, c)
    c.q = q
    check(c, o, lse, 0, 0, q_bits(c, kind == "tokens"), TOKEN_Q if kind == "tokens" else PROMPT_P)
