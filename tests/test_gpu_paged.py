"""The paged-cache calls against their definitions in 64 bits: appending with
the rotation, attention of single tokens and of prompts (window, sinks), and
attention behind a shared prefix."""
import random

import pytest
import torch

from megatron_tensor_transformer_plan_b200 import tpl
from tests.paged_util import D, Case, check, outputs, plan_of, turned

pytestmark = pytest.mark.gpu

TOKEN_Q = 16   # single tokens: q (fp32) and P as bf16 hi + lo, 2^-9 * 2^-9 and the sign of lo
PROMPT_P = 8   # prompts and prefixes: P as one bf16, half a step


def q_bits(case, single):
    return 24 if case.q.dtype == torch.bfloat16 else TOKEN_Q


def workspace(plan, case):
    return plan.paged_workspace(len(case.kv_len), case.tokens)


def run_attn(plan, case, window=0, sinks=0, ws=None, dtype=torch.bfloat16):
    o, lse = outputs(case, dtype)
    plan.paged_attn(case.kv(plan), case.batch(plan), case.q, o, workspace(plan, case) if ws is None else ws,
                    window=window, sinks=sinks, lse=lse)
    torch.cuda.synchronize()
    assert plan.last_device_error() == tpl.TPL_OK
    return o, lse


# ---- append -------------------------------------------------------------------

APPEND = [
    # nq, nkv, t, page, kv_len, news, dtype, rope
    (8, 8, 1, 16, [1], None, torch.float32, True),
    (32, 8, 4, 64, [1, 0, 77, 4096, 65, 64], None, torch.bfloat16, True),
    (40, 8, 2, 32, [131072, 5, 33], None, torch.float32, True),
    (16, 2, 2, 256, [300, 2, 257, 9], [300, 2, 1, 0], torch.bfloat16, True),
    (24, 8, 8, 128, [500, 17, 1, 130], [123, 20, 1, 2], torch.float32, True),
    (48, 4, 1, 16, [900, 31], [513, 31], torch.bfloat16, False),
    (64, 8, 8, 64, [65, 129, 700] * 20, None, torch.float32, False),
    (8, 1, 1, 32, [800, 3, 1400, 0], [700, 5, 1301, 2], torch.float32, True),
    (1, 1, 1, 16, [40] * 700, None, torch.bfloat16, True),
]


@pytest.mark.parametrize("p", APPEND)
@pytest.mark.parametrize("place", ["apart", "slices", "in place", "no q"])
def test_append(gpu, p, place):
    nq, nkv, t, page, kv_len, news, dtype, rope = p
    plan = plan_of(nq, nkv, t, rope)
    c = Case(gpu, nq, nkv, t, page, kv_len, news, dtype=dtype, seed=3, rows_before=2 if news else 0,
             rows_behind=3 if news else 0)
    g = torch.Generator(device=gpu)
    g.manual_seed(8)
    fused = torch.empty((c.tokens, nq + 2 * nkv, D), dtype=dtype, device=gpu).normal_(generator=g)
    q, k, v = fused[:, :nq], fused[:, nq:nq + nkv], fused[:, nq + nkv:]
    if place == "apart":
        q, k, v = q.contiguous(), k.transpose(0, 1).contiguous().transpose(0, 1), v.flatten(1)
    q0, k0, v0 = q.clone().double(), k.clone().double(), v.clone().unflatten(1, (nkv, D)) if v.dim() == 2 else v.clone()
    k_pool, v_pool = c.k.clone(), c.v.clone()
    q_out = q if place == "in place" else torch.full((c.tokens, nq, D), 7.0, dtype=dtype, device=gpu)
    before = q_out.clone()
    if place == "no q":
        plan.paged_append(c.kv(plan), c.batch(plan), k, v)
    else:
        plan.paged_append(c.kv(plan), c.batch(plan), k, v, q, q_out)
    torch.cuda.synchronize()
    assert plan.last_device_error() == tpl.TPL_OK

    live = [(b, r, pos) for b, r, pos in c.rows() if pos >= 0]
    b, r, pos = (torch.tensor(x, device=gpu) for x in zip(*live))
    pages = torch.tensor(c.pages, device=gpu)[b, pos // page]
    # fp32: the angle's rounding, sine, cosine and two products, 2^-20 of |a| + |b| in all
    half = 2.0 ** -8
    slack = 2.0 ** -20 if rope else 0.0

    def off(x):
        return slack * (x[..., :64].abs() + x[..., 64:].abs()).repeat(1, 1, 2)

    want = turned(k0[r], pos) if rope else k0[r]
    got = c.k.permute(1, 3, 0, 2, 4)[pages, pos % page].flatten(1, 2).double()
    assert ((got - want).abs() <= half * want.abs() + off(k0[r])).all()
    got_v = c.v.permute(1, 3, 0, 2, 4)[pages, pos % page].flatten(1, 2)
    assert torch.equal(got_v, v0[r].to(torch.bfloat16))
    for pool, old in ((c.k, k_pool), (c.v, v_pool)):  # no other slot changes
        a, o = pool.permute(1, 3, 0, 2, 4).clone(), old.permute(1, 3, 0, 2, 4).clone()
        a[pages, pos % page], o[pages, pos % page] = 0, 0
        assert torch.equal(a, o)
    if place != "no q":
        want = turned(q0[r], pos) if rope else q0[r]
        q_half = half if dtype == torch.bfloat16 else 2.0 ** -24
        assert ((q_out[r].double() - want).abs() <= q_half * want.abs() + off(q0[r])).all()
        rest = torch.ones(c.tokens, dtype=torch.bool, device=gpu)
        rest[r] = False
        assert torch.equal(q_out[rest], before[rest])


# ---- single tokens ------------------------------------------------------------

DECODE = [
    # nq, nkv, t, page, kv_len, window, sinks
    (1, 1, 1, 16, [1], 0, 0),
    (32, 32, 2, 16, [518], 0, 0),
    (64, 8, 4, 64, [8193, 1, 0, 63, 64, 65, 3000], 0, 0),
    (40, 8, 8, 32, [0, 0, 129], 0, 0),
    (48, 4, 1, 256, [255, 256, 257, 5000], 0, 0),
    (32, 2, 2, 128, [4097, 130, 2], 0, 0),
    (16, 1, 1, 64, [20011], 0, 0),
    (8, 1, 1, 16, [1000, 17, 4096], 1, 0),
    (64, 8, 8, 16, [9000, 4100, 4096, 3, 0, 4101], 4096, 4),
    (24, 8, 4, 64, [700, 333, 90, 128], 64, 33),
    (20, 4, 2, 32, [700, 333, 90, 128, 129], 37, 128),
    (24, 2, 1, 256, [5000, 1500, 257], 1000, 1),
    (8, 8, 1, 16, [1, 2, 3] * 300, 2, 1),
    (16, 8, 2, 64, [100, 2000], 2 ** 31 - 1, 2 ** 31 - 1),
    (16, 8, 2, 64, [100, 2000], 5, 2 ** 31 - 1),
]


@pytest.mark.parametrize("p", DECODE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_tokens(gpu, p, dtype):
    nq, nkv, t, page, kv_len, window, sinks = p
    plan = plan_of(nq, nkv, t)
    c = Case(gpu, nq, nkv, t, page, kv_len, dtype=dtype, seed=len(kv_len), fill=float("nan"))
    o, lse = run_attn(plan, c, window, sinks)
    check(c, o, lse, window, sinks, q_bits(c, True), TOKEN_Q)
    o2, lse2 = run_attn(plan, c, window, sinks)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_tokens_fp32_plan_and_strided_queries(gpu):
    plan = plan_of(24, 8, 2, f32=True)
    c = Case(gpu, 24, 8, 2, 32, [300, 1, 77], seed=5)
    wide = torch.randn((3, 48, D + 4), device=gpu) * 2
    c.q = wide[:, ::2, :D]
    assert c.q.stride(1) == 2 * (D + 4)
    o, lse = run_attn(plan, c, dtype=torch.float32)
    ref, ref_lse, tol, _ = c.expected(0, 0, TOKEN_Q, TOKEN_Q)
    assert ((o.view(3, 24, D).double() - ref).abs() <= tol).all()  # (the bound allows for bf16 outputs)
    assert float((o.view(3, 24, D).double() - ref).abs().max()) < 2.0 ** -8  # fp32 outputs: far closer


def test_tokens_skipped_pages_are_not_read(gpu):
    """Behind a window the table may name no page, and the pages may hold anything."""
    plan = plan_of(16, 8, 1)
    c = Case(gpu, 16, 8, 1, 32, [3000, 999], seed=6)
    ref = run_attn(plan, c, 100, 40)
    for b, n in enumerate(c.kv_len):
        for e in range(2, (n - 100) // 32):  # keys 64 .. lie behind the sinks and before the window
            c.k[:, c.pages[b][e]] = float("inf")
            c.v[:, c.pages[b][e]] = float("nan")
            c.table[b, e] = -7
    got = run_attn(plan, c, 100, 40)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))


# ---- prompts ------------------------------------------------------------------

PROMPT = [
    # nq, nkv, t, page, kv_len, news, window, sinks
    (4, 4, 1, 16, [1], [1], 0, 0),
    (64, 8, 8, 64, [130, 129, 40], [130, 1, 7], 0, 0),
    (40, 8, 2, 32, [937, 300, 64], [37, 300, 20], 0, 0),
    (32, 32, 2, 128, [700, 256], [257, 256], 0, 0),
    (48, 4, 4, 256, [1000, 0, 513, 20], [400, 0, 1, 0], 0, 0),
    (16, 1, 1, 16, [2100, 33], [90, 33], 0, 0),
    (24, 8, 8, 64, [5, 200, 300], [9, 150, 1], 0, 0),          # tokens before the first position
    (64, 8, 8, 128, [3000, 100, 1500], [800, 100, 257], 300, 16),
    (20, 4, 2, 16, [1500, 90], [333, 90], 1, 0),
    (16, 8, 2, 32, [1500, 700], [1100, 700], 129, 133),
    (8, 8, 1, 64, [6000], [40], 1000, 200),
    (32, 8, 1, 256, [2000, 3], [700, 3], 64, 2 ** 31 - 1),
    (32, 8, 1, 256, [20, 600], [40, 300], 2 ** 31 - 1, 0),
    (8, 4, 1, 64, [3, 1, 2] * 150, [3, 1, 1] * 150, 2, 1),
    (16, 16, 8, 64, [9000], [1], 0, 0),
]


@pytest.mark.parametrize("p", PROMPT)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompts(gpu, p, dtype):
    nq, nkv, t, page, kv_len, news, window, sinks = p
    plan = plan_of(nq, nkv, t)
    c = Case(gpu, nq, nkv, t, page, kv_len, news, dtype=dtype, seed=len(kv_len) + page, rows_before=1, rows_behind=5,
             fill=float("nan"))
    o, lse = run_attn(plan, c, window, sinks)
    check(c, o, lse, window, sinks, q_bits(c, False), PROMPT_P)
    o2, lse2 = run_attn(plan, c, window, sinks)
    same = ~torch.isnan(lse)
    assert torch.equal(o.view(c.tokens, nq, D)[same], o2.view(c.tokens, nq, D)[same]) and torch.equal(lse[same], lse2[same])


def test_prompt_rows_that_see_large_and_small_logits(gpu):
    """Logits that rise along the keys by far more than an exponent's range."""
    plan = plan_of(8, 2, 1)
    c = Case(gpu, 8, 2, 1, 64, [900, 700], [500, 700], dtype=torch.bfloat16, seed=2)
    c.q.fill_(8.0)
    for b in range(2):
        at = torch.arange(c.kv_len[b], device=gpu)
        ramp = ((at.float() / 50 - 5).to(torch.bfloat16))[:, None, None].expand(-1, 1, 2)
        rows = c.k.permute(1, 3, 0, 2, 4)
        rows[torch.tensor(c.pages[b], device=gpu)[at // 64], at % 64] = ramp[..., None].expand(-1, 1, 2, D)
    o, lse = run_attn(plan, c)
    check(c, o, lse, 0, 0, 24, PROMPT_P)


# ---- a shared prefix ----------------------------------------------------------

SHARED = [
    # nq, nkv, t, page, shared, kv_len
    (4, 4, 1, 16, 16, [17]),
    (64, 8, 4, 64, 1024, [1025, 1500, 1030, 2000, 1100]),
    (40, 8, 2, 32, 992, [1200] * 30 + [993]),
    (32, 32, 2, 16, 1536, [1700, 1537, 1600]),
    (48, 4, 4, 256, 512, [600, 700] * 20),
    (16, 1, 1, 128, 2048, [2049 + 7 * i for i in range(40)]),
    (64, 8, 8, 64, 4096, [0, 1, 100, 4095, 4096, 4097, 5000, 0]),   # sequences that end inside the prefix
    (24, 8, 8, 64, 640, [300, 64, 640]),                             # none has keys of its own
    (8, 1, 1, 64, 192, [200 + i for i in range(150)]),
]


@pytest.mark.parametrize("p", SHARED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared(gpu, p, dtype):
    nq, nkv, t, page, shared, kv_len = p
    plan = plan_of(nq, nkv, t)
    c = Case(gpu, nq, nkv, t, page, kv_len, shared=shared, dtype=dtype, seed=page, fill=float("nan"))
    ws = workspace(plan, c)
    for _ in range(2):
        o, lse = outputs(c)
        plan.paged_attn_shared(c.kv(plan), c.batch(plan), shared, c.q, o, ws, lse=lse)
        torch.cuda.synchronize()
        assert plan.last_device_error() == tpl.TPL_OK
        check(c, o, lse, 0, 0, q_bits(c, False), PROMPT_P)
    # the prefix is read through row 0 of the table only
    c.table[1:, :shared // page] = -3
    o2, lse2 = outputs(c)
    plan.paged_attn_shared(c.kv(plan), c.batch(plan), shared, c.q, o2, ws, lse=lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert plan.last_device_error() == tpl.TPL_OK


def test_shared_of_nothing_is_attention(gpu):
    plan = plan_of(16, 8, 1)
    c = Case(gpu, 16, 8, 1, 32, [300, 1, 64], seed=1)
    o, lse = outputs(c)
    plan.paged_attn_shared(c.kv(plan), c.batch(plan), 0, c.q, o, workspace(plan, c), lse=lse)
    o2, lse2 = run_attn(plan, c)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# ---- streams, graphs, batches in use -------------------------------------------

def test_lse_may_be_left_out_and_an_empty_batch_is_nothing(gpu):
    plan = plan_of(16, 8, 1)
    c = Case(gpu, 16, 8, 1, 32, [300, 1, 64], seed=1)
    o, _ = outputs(c)
    plan.paged_attn(c.kv(plan), c.batch(plan), c.q, o, workspace(plan, c))
    assert torch.equal(o, run_attn(plan, c)[0])
    ws = workspace(plan, c)
    empty = plan.paged_batch(c.table[:0], c.lens[:0])
    plan.paged_attn(c.kv(plan), empty, c.q[:0], o[:0], ws)
    plan.paged_attn_shared(c.kv(plan), empty, 0, c.q[:0], o[:0], ws)
    plan.paged_append(c.kv(plan), empty, c.q[:0, :8], c.q[:0, :8])
    none = plan.paged_batch(c.table, c.lens, torch.zeros(4, dtype=torch.int32, device=gpu), 0)
    plan.paged_attn(c.kv(plan), none, c.q[:0], o[:0], ws)
    # rows that belong to no sequence
    idle = plan.paged_batch(c.table, c.lens, torch.zeros(4, dtype=torch.int32, device=gpu), 3)
    o.fill_(5.0)
    plan.paged_attn(c.kv(plan), idle, c.q, o, ws)
    assert (o == 5.0).all() and plan.last_device_error() == tpl.TPL_OK


def test_one_workspace_serves_smaller_batches(gpu):
    plan = plan_of(64, 8, 1)
    big = Case(gpu, 64, 8, 1, 64, [500] * 40, shared=256, seed=4)
    ws = workspace(plan, big)
    for c in (Case(gpu, 64, 8, 1, 64, [3000, 70], seed=5), Case(gpu, 64, 8, 1, 64, [3000, 70], [30, 3], seed=5)):
        o, lse = run_attn(plan, c, ws=ws)
        ref = run_attn(plan, c)
        assert torch.equal(o, ref[0]) and torch.equal(lse, ref[1])


@pytest.mark.parametrize("kind", ["tokens", "prompts", "shared"])
def test_graph_follows_the_arrays(gpu, kind):
    """A captured step (append, then attention) replayed while the batch grows."""
    plan = plan_of(32, 8, 2)
    news = [3, 1, 7] if kind == "prompts" else None
    last = [700, 129, 400]
    c = Case(gpu, 32, 8, 2, 64, last, news, shared=64 if kind == "shared" else 0, seed=7)
    steps = 3
    step_new = c.news
    q, k, v = (torch.randn((steps, c.tokens, h, D), device=gpu) for h in (32, 8, 8))
    q_in, k_in, v_in, q_out = q[0].clone(), k[0].clone(), v[0].clone(), torch.empty_like(q[0])
    o, lse = outputs(c)
    kv, batch, ws = c.kv(plan), c.batch(plan), workspace(plan, c)

    def step():
        plan.paged_append(kv, batch, k_in, v_in, q_in, q_out)
        if kind == "shared":
            plan.paged_attn_shared(kv, batch, 64, q_out, o, ws, lse=lse)
        else:
            plan.paged_attn(kv, batch, q_out, o, ws, window=200, sinks=3, lse=lse)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k0, v0 = c.k.clone(), c.v.clone()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.k.copy_(k0)
    c.v.copy_(v0)
    lens = [x - s * (steps - 1) for x, s in zip(last, step_new)]
    results = []
    for s in range(steps):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q_in.copy_(q[s]), k_in.copy_(k[s]), v_in.copy_(v[s])
        graph.replay()
        results.append((o.clone(), lse.clone()))
        lens = [x + n for x, n in zip(lens, step_new)]
    torch.cuda.synchronize()
    c.k.copy_(k0)
    c.v.copy_(v0)
    lens = [x - s * (steps - 1) for x, s in zip(last, step_new)]
    for s in range(steps):
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        q_in.copy_(q[s]), k_in.copy_(k[s]), v_in.copy_(v[s])
        step()
        assert torch.equal(o, results[s][0]) and torch.equal(lse, results[s][1])
        lens = [x + n for x, n in zip(lens, step_new)]
    c.q = q_out
    check(c, o, lse, 0 if kind == "shared" else 200, 0 if kind == "shared" else 3, TOKEN_Q, PROMPT_P)
    assert plan.last_device_error() == tpl.TPL_OK


def test_two_streams_with_a_workspace_each(gpu):
    plan = plan_of(64, 8, 1)
    cs = [Case(gpu, 64, 8, 1, 64, [2000, 300, 5], seed=1), Case(gpu, 64, 8, 1, 64, [1500, 3], [200, 3], seed=2)]
    want = [run_attn(plan, c) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs, wss = [outputs(c) for c in cs], [workspace(plan, c) for c in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, (o, lse), ws in zip(cs, streams, outs, wss):
            with torch.cuda.stream(s):
                plan.paged_attn(c.kv(plan), c.batch(plan), c.q, o, ws, lse=lse)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_numbers_outside_their_range_are_reported(gpu):
    """Page ids, lengths and starts that the kernels' own checks catch: the
    call returns, the error word is set, the other sequences are right, and
    nothing outside the sequence's own slots is written."""
    plan = plan_of(32, 8, 2)
    for bad in ("page", "page below", "length", "length below", "start"):
        for kind in ("tokens", "prompts", "shared"):
            if bad == "start" and kind != "prompts":
                continue
            news = [5, 6, 7] if kind == "prompts" else None
            c = Case(gpu, 32, 8, 2, 64, [300, 400, 500], news, shared=64 if kind == "shared" else 0, seed=1)
            ws = workspace(plan, c)
            if bad.startswith("page"):
                c.table[1, 6] = -1 if bad == "page below" else c.n_pages
            elif bad.startswith("length"):
                c.lens[1] = -9 if bad == "length below" else c.table.shape[1] * 64 + 1
            else:
                c.q_start[3] = c.tokens + 1
            o, lse = outputs(c)
            kv, batch = c.kv(plan), c.batch(plan)
            if kind == "shared":
                plan.paged_attn_shared(kv, batch, 64, c.q, o, ws, lse=lse)
            else:
                plan.paged_attn(kv, batch, c.q, o, ws, lse=lse)
            assert plan.last_device_error() == tpl.TPL_EDEVICE, (bad, kind)
            ref, _, tol, _ = c.expected(0, 0, TOKEN_Q, PROMPT_P)
            rows = slice(c.start[0], c.start[0] + c.news[0])
            assert ((o.view(-1, 32, D).double() - ref).abs() <= tol)[rows].all()
            old = c.k.clone()
            plan.paged_append(kv, batch, torch.ones((c.tokens, 8, D), device=gpu), torch.ones((c.tokens, 8, D), device=gpu))
            assert plan.last_device_error() == tpl.TPL_EDEVICE, (bad, kind)
            changed = (c.k != old).permute(1, 3, 0, 2, 4).flatten(2).any(-1).sum()
            assert int(changed) <= sum(c.news)
            assert plan.last_device_error() == tpl.TPL_OK


# ---- the ends of the ranges -------------------------------------------------------

def moved_to_the_end(c, n_pages):
    """The same batch in a pool of n_pages pages, its pages the last ones."""
    shift = n_pages - c.n_pages
    for name in ("k", "v"):
        small = getattr(c, name)
        big = torch.empty((small.shape[0], n_pages, *small.shape[2:]), dtype=small.dtype, device=small.device)
        big[:, shift:] = small
        setattr(c, name, big)
    c.pages = [[p + shift if p < c.n_pages else p for p in row] for row in c.pages]
    c.table += torch.where(c.table < c.n_pages, shift, 0).to(torch.int32) * (c.table >= 0)
    c.n_pages = n_pages
    return c


@pytest.mark.parametrize("kind", ["tokens", "prompts", "shared"])
def test_offsets_beyond_32_bits(gpu, kind):
    """20.5 million rows of the pool: 2.6e9 values, 5.2 GB each for k and v."""
    plan = plan_of(16, 2, 2)
    news = [40, 3] if kind == "prompts" else None
    c = moved_to_the_end(Case(gpu, 16, 2, 2, 256, [1000, 513], news, shared=256 if kind == "shared" else 0, seed=3), 40000)
    k = torch.randn((c.tokens, 2, D), device=gpu)
    v = torch.randn((c.tokens, 2, D), device=gpu)
    plan.paged_append(c.kv(plan), c.batch(plan), k, v)
    for b, r, pos in c.rows():
        want = v[r].to(torch.bfloat16)
        assert torch.equal(c.v[:, c.pages[b][pos // 256], :, pos % 256].flatten(0, 1), want)
    if kind == "shared":
        o, lse = outputs(c)
        plan.paged_attn_shared(c.kv(plan), c.batch(plan), 256, c.q, o, workspace(plan, c), lse=lse)
        assert plan.last_device_error() == tpl.TPL_OK
    else:
        o, lse = run_attn(plan, c)
    check(c, o, lse, 0, 0, TOKEN_Q, TOKEN_Q if kind == "tokens" else PROMPT_P)


@pytest.mark.parametrize("kind", ["tokens", "prompts", "shared"])
def test_a_batch_that_sees_nothing(gpu, kind):
    plan = plan_of(16, 8, 1)
    n = 1024
    c = Case(gpu, 16, 8, 1, 16, [0] * n, [1] * n if kind == "prompts" else None, shared=32 if kind == "shared" else 0, seed=3,
             fill=float("nan"))
    o, lse = outputs(c)
    if kind == "shared":
        plan.paged_attn_shared(c.kv(plan), c.batch(plan), 32, c.q, o, workspace(plan, c), lse=lse)
    else:
        plan.paged_attn(c.kv(plan), c.batch(plan), c.q, o, workspace(plan, c), lse=lse)
    assert (o == 0).all() and (lse == -float("inf")).all() and plan.last_device_error() == tpl.TPL_OK


@pytest.mark.parametrize("seed", range(12))
def test_many_sequences_of_any_length(gpu, seed):
    rnd = random.Random(seed)
    nkv = rnd.choice([1, 2, 4, 8])
    nq = nkv * rnd.choice([1, 2, 3, 5, 7, 8, 9, 11, 16])
    t = rnd.choice([x for x in (1, 2, 4) if nkv % x == 0])
    page = rnd.choice([16, 32, 64, 128, 256])
    n = rnd.choice([1, 2, 33, 147, 1024]) if seed else 1024
    top = max(3, 40000 // n)
    kv_len = [rnd.choice([0, 1, rnd.randrange(top), rnd.randrange(top)]) for _ in range(n)]
    kind = seed % 3
    news = [rnd.randrange(0, 1 + min(x, 2 + 600 // n)) if rnd.random() < 0.9 else 0 for x in kv_len] if kind == 1 else None
    window, sinks = (rnd.choice([0, 1, 63, 64, 65, 300]), rnd.choice([0, 1, 64, 200])) if kind < 2 else (0, 0)
    shared = page * rnd.randrange(1, 9) if kind == 2 else 0
    plan = plan_of(nq, nkv, t)
    dtype = rnd.choice([torch.float32, torch.bfloat16])
    c = Case(gpu, nq, nkv, t, page, kv_len, news, shared=shared, dtype=dtype, seed=seed, rows_behind=1 if news else 0,
             fill=float("nan"))
    if kind == 2:
        o, lse = outputs(c)
        plan.paged_attn_shared(c.kv(plan), c.batch(plan), shared, c.q, o, workspace(plan, c), lse=lse)
        assert plan.last_device_error() == tpl.TPL_OK
    else:
        o, lse = run_attn(plan, c, window, sinks)
    check(c, o, lse, window, sinks, q_bits(c, kind == 0), TOKEN_Q if kind == 0 else PROMPT_P)


def test_captured_before_any_eager_call(gpu):
    """A graph whose first launches are the captured ones (its own process state aside)."""
    plan = plan_of(20, 4, 4)
    c = Case(gpu, 20, 4, 4, 64, [700, 65, 3], seed=9)
    o, lse = outputs(c)
    kv, batch, ws = c.kv(plan), c.batch(plan), workspace(plan, c)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.paged_attn(kv, batch, c.q, o, ws, lse=lse)
    for _ in range(3):
        o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(c, o, lse, 0, 0, TOKEN_Q, TOKEN_Q)
    assert plan.last_device_error() == tpl.TPL_OK
